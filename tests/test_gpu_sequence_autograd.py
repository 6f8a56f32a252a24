"""Gradients of the sequence operators under what training programs do around autograd:
activation checkpointing, saved-tensor hooks, frozen inputs, broadcast gradients, captured
backward passes."""
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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [([3, 140], [90, 700]), ([1, 2], [9000, 5003])])
def test_each_gradient_alone(dtype, shape):
    """Frozen inputs change no bit of the others' gradients: the bias's without the keys' among them."""
    d, dout = attention.make(dtype, *shape, 4, 2, 64, buckets=9, masked=0.2, seed=34)
    out, leaves, given = attend(d, dout)
    want = dict(zip(("q", "k", "v", "bias"), torch.autograd.grad(out, leaves, given)))
    for name in want:
        leaf = d[name].detach().clone().requires_grad_()
        got = torch.autograd.grad(E.cross_attention(**{**d, name: leaf}), leaf, dout)[0]
        assert torch.equal(got, want[name]), name
    r, dy, dlast = recurrence.make(dtype, shape[1], 66, masked=0.2, seed=35)
    outs, leaves, given = scan(r, dy, dlast)
    want = dict(zip(("x", "gate", "state"), torch.autograd.grad(outs, leaves, given)))
    for name in want:
        leaf = r[name].detach().clone().requires_grad_()
        got = torch.autograd.grad(list(E.gated_recurrence(**{**r, name: leaf})), leaf, [dy, dlast])[0]
        assert torch.equal(got, want[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_that_are_broadcast(dtype):
    """A sum's gradient is one number seen from everywhere (strides of zero)."""
    d, dout = attention.make(dtype, [3, 140], [90, 700], 4, 2, 64, buckets=9, masked=0.2, seed=36)
    r, dy, dlast = recurrence.make(dtype, [90, 700], 66, masked=0.2, seed=37)
    for make, one in ((lambda: attend(d, torch.ones_like(dout)), lambda t: t.sum()),
                      (lambda: attend(d, torch.ones_like(dout)), lambda t: t.sum(2).sum()),
                      (lambda: scan(r, torch.ones_like(dy), None), lambda t: t.sum()),
                      (lambda: scan(r, torch.ones_like(dy), None), lambda t: t.sum(0).sum())):
        outs, leaves, given = make()
        out = outs[0] if isinstance(outs, list) else outs
        want = torch.autograd.grad(out, leaves, given[:1])
        outs, leaves, _ = make()
        got = torch.autograd.grad(one(outs[0] if isinstance(outs, list) else outs), leaves)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_captured_training_step(dtype):
    """Forward and backward in one graph, replayed on new values between eager work."""
    d, dout = attention.make(dtype, [1, 150], [2000, 300], 4, 4, 64, buckets=9, masked=0.2, seed=38)
    leaves = [d[n].clone().requires_grad_() for n in ("q", "k", "v", "bias")]

    def step():
        q, k, v, bias = leaves
        y, last = E.gated_recurrence(k.flatten(1), v.flatten(1), d["k_offsets"], mask=d["mask"])
        out = E.cross_attention(**{**d, "q": q, "k": y.view(k.shape), "v": v, "bias": bias})
        return [out, last] + list(torch.autograd.grad([out, last], leaves, [dout, torch.ones_like(last)]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        with torch.no_grad():
            for t in leaves:
                t.mul_(-1.25)
        eager = step()
        for t in captured:
            t.detach().zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
