"""The encoder operators' 64-bit forms against torch's own differentiation and against
differences, on the CPU."""
import pytest
import torch

import encoder_reference as R


def _delta_inputs(seed, lens, kh, h, dk, dv, masked):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen, dtype=torch.float64)
    n = sum(lens)
    k = randn(n, kh, dk)
    t = dict(q=randn(n, kh, dk), k=k / k.norm(dim=-1, keepdim=True), v=randn(n, h, dv),
             gate=randn(n, h) + 1, beta=randn(n, h), state=randn(len(lens), h, dk, dv))
    off = torch.tensor([0] + list(lens)).cumsum(0).int()
    mask = (torch.rand(n, generator=gen) > 0.3).to(torch.uint8) if masked else None
    return t, off, mask, randn(n, h, dv), randn(len(lens), h, dk, dv)


def _plain(t, off, mask):
    """o and last by differentiable torch operations, step by step."""
    g = t["v"].shape[1] // t["q"].shape[1]
    outs, lasts = [], []
    for s in range(len(off) - 1):
        S = t["state"][s]
        for i in range(int(off[s]), int(off[s + 1])):
            if mask is not None and not mask[i]:
                outs.append(torch.zeros_like(t["v"][i]))
                continue
            q, k = t["q"][i].repeat_interleave(g, 0), t["k"][i].repeat_interleave(g, 0)
            S = torch.sigmoid(t["gate"][i])[:, None, None] * S
            u = torch.sigmoid(t["beta"][i])[:, None] * (t["v"][i] - (S * k[:, :, None]).sum(1))
            S = S + k[:, :, None] * u[:, None, :]
            outs.append((S * q[:, :, None]).sum(1) * q.shape[1] ** -0.5)
        lasts.append(S)
    return torch.stack(outs), torch.stack(lasts)


@pytest.mark.parametrize("masked", [False, True])
def test_delta_is_torchs(masked):
    t, off, mask, do, dlast = _delta_inputs(1, [7, 0, 1, 40], 2, 4, 5, 3, masked)
    ref = R.delta(offsets=off, mask=mask, do=do, dlast=dlast, **t)
    leaves = {n: x.requires_grad_() for n, x in t.items()}
    o, last = _plain(leaves, off, mask)
    grads = torch.autograd.grad([o, last], list(leaves.values()), [do, dlast])
    got = dict(zip(("d" + n for n in leaves), grads), o=o.detach(), last=last.detach())
    for name, (val, _) in ref.items():
        assert torch.allclose(val, got[name], rtol=1e-10, atol=1e-12), name


def test_delta_by_differences():
    t, off, mask, do, dlast = _delta_inputs(2, [9, 3], 1, 2, 4, 3, True)
    ref = R.delta(offsets=off, mask=mask, do=do, dlast=dlast, **t)

    def loss():
        out = R.delta(offsets=off, mask=mask, **t)
        return (out["o"][0] * do).sum() + (out["last"][0] * dlast).sum()
    gen = torch.Generator().manual_seed(3)
    for name in t:
        d = torch.randn(t[name].shape, generator=gen, dtype=torch.float64)
        keep, step = t[name], 1e-5
        t[name] = keep + step * d
        up = loss()
        t[name] = keep - step * d
        down = loss()
        t[name] = keep
        want = (ref["d" + name][0] * d).sum()
        # a central difference is off by step^2 / 6 of the third derivative, order one here,
        # and by the sums' own rounding over the step
        assert abs((up - down) / (2 * step) - want) < 1e-7 * (1 + abs(want)), name


def test_layer_norm_is_torchs():
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(3, 5, 7, generator=gen, dtype=torch.float64).requires_grad_()
    w, b = (torch.randn(7, generator=gen, dtype=torch.float64).requires_grad_() for _ in range(2))
    dy = torch.randn(3, 5, 7, generator=gen, dtype=torch.float64)
    ref = R.layer_norm(x, w, b, dy=dy)
    y = torch.nn.functional.layer_norm(x, (7,), w, b)
    got = dict(zip(("dx", "dweight", "dbias"), torch.autograd.grad(y, (x, w, b), dy)), y=y)
    for name, (val, _) in ref.items():
        assert torch.allclose(val, got[name], rtol=1e-10, atol=1e-12), name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_is_its_own_transpose(layout):
    gen = torch.Generator().manual_seed(5)
    x, y = (torch.randn(6, 2, 10, generator=gen, dtype=torch.float64) for _ in range(2))
    pos = torch.tensor([0, 1, -3, 1 << 30, 77, 2], dtype=torch.int32)
    f = torch.rand(4, generator=gen, dtype=torch.float64)
    a, _ = R.rotary(x, pos, f, layout, 1.25)
    b, _ = R.rotary(y, pos, f, layout, 1.25, back=True)
    assert torch.allclose((a * y)[..., :8].sum(), (x * b)[..., :8].sum(), rtol=1e-10)
    assert torch.equal(a[..., 8:], x[..., 8:])
    # turning by the sum of two positions is turning twice
    twice, _ = R.rotary(R.rotary(x, pos // 2, f, layout)[0], pos - pos // 2, f, layout)
    assert torch.allclose(twice, R.rotary(x, pos, f, layout)[0], atol=1e-6)
