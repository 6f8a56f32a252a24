"""Gradients of the sequence operators under what training programs do around autograd:
activation checkpointing, saved-tensor hooks, frozen inputs, captured backward passes."""
import pytest
import torch
import torch.utils.checkpoint

import embedding_columns_amd as E
import test_gpu_attention as attention
import test_gpu_recurrence as recurrence

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def attend(d, dout, q_like=lambda t: t):
    names = [n for n in ("q", "k", "v", "bias") if d.get(n) is not None]
    leaves = {n: d[n].detach().clone().requires_grad_() for n in names}
    out = E.cross_attention(**{**d, **{n: q_like(t) for n, t in leaves.items()}})
    return out, [leaves[n] for n in names], [dout]


def scan(d, dy, dlast, q_like=lambda t: t):
    names = [n for n in ("x", "gate", "state") if d.get(n) is not None]
    leaves = {n: d[n].detach().clone().requires_grad_() for n in names}
    outs = E.gated_recurrence(**{**d, **{n: q_like(t) for n, t in leaves.items()}})
    return list(outs), [leaves[n] for n in names], [dy, dlast]


class Overwritten:
    """Saved-tensor hooks that keep a copy and spoil what was saved, as freed and reused
    memory would; only what the operators made or were given as temporaries is spoiled."""

    def __enter__(self):
        self.spoil = []

        def pack(t):
            kept = t.detach().clone()
            if t.is_floating_point() and not t.is_leaf:
                self.spoil.append(t.detach())
            return kept
        self.hooks = torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.clone())
        self.hooks.__enter__()
        return self

    def __exit__(self, *args):
        self.hooks.__exit__(*args)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_under_hooks(dtype):
    d, dout = attention.make(dtype, [3, 140], [90, 2100], 4, 2, 64, buckets=9, masked=0.2, seed=31)
    out, leaves, given = attend(d, dout)
    want = torch.autograd.grad(out, leaves, given)
    with Overwritten() as hooks:
        out, leaves, given = attend(d, dout, lambda t: t * 1)
    for t in hooks.spoil:
        t.fill_(float("nan"))
    got = torch.autograd.grad(out, leaves, given)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[70, 3], [5000]])
def test_recurrence_under_hooks(dtype, lengths):
    d, dy, dlast = recurrence.make(dtype, lengths, 66, masked=0.2, seed=32)
    outs, leaves, given = scan(d, dy, dlast)
    want = torch.autograd.grad(outs, leaves, given)
    with Overwritten() as hooks:
        outs, leaves, given = scan(d, dy, dlast, lambda t: t * 1)
    for t in hooks.spoil:
        t.fill_(float("nan"))
    got = torch.autograd.grad(outs, leaves, given)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_checkpointing_and_offloading(dtype):
    """A block of both operators: its inputs and intermediates are dropped, or moved to the host,
    between the passes, and their memory is used again."""
    d, dout = attention.make(dtype, [3, 140], [90, 700], 4, 4, 64, buckets=9, masked=0.2, seed=33)
    x, gate = d["k"].flatten(1), d["v"].flatten(1)

    def block(q, x, gate, bias):
        y, _ = E.gated_recurrence(x * 2, gate * 2, d["k_offsets"] + 0, mask=d["mask"] + 0)
        rows = y.view(d["k"].shape)
        return E.cross_attention(q * 2, rows * 2, rows, d["q_offsets"] + 0, d["k_offsets"] + 0,
                                 mask=d["mask"] + 0, bias=bias * 2, boundaries=d["boundaries"] + 0,
                                 q_pos=d["q_pos"] + 0, k_pos=d["k_pos"] + 0)

    def gradients(call):
        leaves = [t.detach().clone().requires_grad_() for t in (d["q"], x, gate, d["bias"])]
        out = call(*leaves)
        reused = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in (1 << 10, 1 << 16, 1 << 18)
                  for _ in range(20)]
        out.backward(dout)
        del reused
        return [out] + [t.grad for t in leaves]

    def offloaded(*leaves):
        with torch.autograd.graph.save_on_cpu():
            return block(*leaves)

    want = gradients(block)
    for call in (lambda *t: torch.utils.checkpoint.checkpoint(block, *t, use_reentrant=False),
                 lambda *t: torch.utils.checkpoint.checkpoint(block, *t, use_reentrant=True), offloaded):
        assert all(torch.equal(a, b) for a, b in zip(gradients(call), want))
