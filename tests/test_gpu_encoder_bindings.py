"""The encoder operators by the bindings of their C entry points, with buffers of the caller's own:
the same bits as by gated_delta, gated_delta_step, layer_norm and rotary."""
import pytest
import torch

import embedding_columns_amd as E
from test_gpu_delta import BF16, F32, call, make

pytestmark = pytest.mark.gpu


def _u8(n):
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


def _delta_desc(t, dtype):
    n, kh, dk = t["q"].shape
    h, dv = t["v"].shape[1:]
    return E.DeltaDesc(dtype=dtype, samples=t["offsets"].numel() - 1, key_heads=kh, heads=h, dk=dk, dv=dv, scale=dk ** -0.5,
                       n=n, q=t["q"].data_ptr(), k=t["k"].data_ptr(), v=t["v"].data_ptr(), gate=t["gate"].data_ptr(),
                       beta=t["beta"].data_ptr(), q_stride=kh * dk, q_head_stride=dk, k_stride=kh * dk, k_head_stride=dk,
                       v_stride=h * dv, v_head_stride=dv, gate_stride=h, beta_stride=h, offsets=t["offsets"].data_ptr(),
                       mask=t["mask"].data_ptr(), state=t["state"].data_ptr())


@pytest.mark.parametrize("dtype,code", [(F32, E.F32), (BF16, E.BF16)])
@pytest.mark.parametrize("dk,dv", [(64, 32), (40, 24)])
def test_delta(dk, dv, dtype, code):
    t = make([70, 0, 45], 2, 4, dk, dv, dtype, masked=0.1, seed=71)
    want = call(t)
    desc = _delta_desc(t, code)
    kept, forward, backward = E.emb_delta_query(desc)
    got = {"o": torch.empty_like(t["v"]), "last": torch.empty_like(t["state"])}
    saved = _u8(kept)
    E.emb_delta_forward(desc, got["o"], got["last"], saved, _u8(forward))
    for x in ("q", "k", "v", "gate", "beta", "state"):
        got["d" + x] = torch.empty_like(t[x])
    E.emb_delta_backward(desc, saved, t["do"], t["dlast"], got["dq"], got["dk"], got["dv"], got["dgate"], got["dbeta"],
                         got["dstate"], _u8(backward))
    for x in want:
        assert torch.equal(got[x], want[x]), x
    none, forward, zero = E.emb_delta_query(desc, training=False)
    assert none == zero == 0
    o, last = torch.empty_like(t["v"]), torch.empty_like(t["state"])
    E.emb_delta_forward(desc, o, last, None, _u8(forward))
    assert torch.equal(o, want["o"]) and torch.equal(last, want["last"])


@pytest.mark.parametrize("dtype,code", [(F32, E.F32), (BF16, E.BF16)])
def test_delta_step(dtype, code):
    t = make([1] * 5, 2, 4, 64, 32, dtype, masked=0.5, seed=72)
    state, other = t["state"].clone(), t["state"].clone()
    want = E.gated_delta_step(*(t[x] for x in ("q", "k", "v", "gate", "beta")), state)
    o = torch.empty_like(want)
    E.emb_delta_step(_delta_desc(t, code), other, o)
    assert torch.equal(o, want) and torch.equal(other, state)


@pytest.mark.parametrize("dtype,code", [(F32, E.F32), (BF16, E.BF16)])
def test_norm(dtype, code):
    gen = torch.Generator().manual_seed(73)
    x, dy = (torch.randn(60, 3, 40, generator=gen).to(dtype).cuda() for _ in range(2))
    w, b = (torch.randn(40, generator=gen).cuda() for _ in range(2))
    wide = torch.zeros(60, 5, 40, dtype=dtype, device="cuda")
    wide[:, 1:4] = dy
    leaves = [v.clone().requires_grad_() for v in (x, w, b)]
    y = E.layer_norm(*leaves)
    grads = torch.autograd.grad(y, leaves, dy)
    desc = E.NormDesc(dtype=code, channels=40, inner=3, eps=1e-5, rows=180, x=x.data_ptr(), x_stride=120, x_inner_stride=40,
                      weight=w.data_ptr(), bias=b.data_ptr())
    out, stats = torch.empty_like(x), torch.empty(180, 2, device="cuda")
    E.emb_norm_forward(desc, out, stats)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    E.emb_norm_backward(desc, stats, wide[:, 1:4], dx, dw, db, _u8(E.emb_norm_query(desc)))
    for a, b in zip((out, dx, dw, db), (y,) + grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("back", [False, True])
def test_rotary(back):
    gen = torch.Generator().manual_seed(74)
    q, k = torch.randn(30, 4, 32, generator=gen).cuda(), torch.randn(50, 2, 32, generator=gen).cuda()
    qp, kp = (torch.randint(0, 1 << 30, (n,), generator=gen).int().cuda() for n in (30, 50))
    f = E.rotary_frequencies(24)
    want = E.rotary(q, k, qp, kp, -f if back else f, scale=1.25)
    out = torch.empty_like(q), torch.empty_like(k)
    sides = [E.RotaryRows(x=x.data_ptr(), y=y.data_ptr(), pos=p.data_ptr(), n=x.shape[0], stride=x.stride(0),
                          head_stride=x.stride(1), heads=x.shape[1]) for x, y, p in zip((q, k), out, (qp, kp))]
    desc = E.RotaryDesc(dtype=E.F32, layout=0, dim=32, pairs=12, scale=1.25, frequencies=f.data_ptr(), q=sides[0], k=sides[1])
    E.emb_rotary_turn(desc, back=back)
    for a, b in zip(out, want):
        assert torch.equal(a, b)
