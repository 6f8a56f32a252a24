"""Rotary positions' kernel against the 64-bit form, with the bounds of encoder_reference.py."""
import pytest
import torch

import embedding_columns_amd as E
import encoder_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def rows(n, heads, dim, dtype, seed, longest=1 << 31):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, dim, generator=gen).to(dtype).cuda()
    pos = torch.randint(-longest, longest, (n,), generator=gen).clamp(-2 ** 31, 2 ** 31 - 1).int()
    ends = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    pos[:min(n, 5)] = ends[:n]
    return x, pos.cuda()


def check(got, x, pos, f, layout, scale, back=False):
    val, bound = R.rotary(x, pos, f, layout, scale, back)
    off = (got.cpu().double() - val).abs()
    assert got.shape == val.shape and (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,part", [(2, 2), (16, 16), (64, 64), (128, 128), (128, 64), (40, 24), (40, 30), (7, 6), (33, 0),
                                      (96, 32), (256, 256), (1024, 1024)])
def test_sizes(dim, part, layout, dtype):
    q, qp = rows(37, 4, dim, dtype, 1)
    k, kp = rows(70, 2, dim, dtype, 2)
    f = E.rotary_frequencies(part)
    q.requires_grad_()
    k.requires_grad_()
    a, b = E.rotary(q, k, qp, kp, f, layout, 1.5)
    check(a.detach(), q, qp, f, layout, 1.5)
    check(b.detach(), k, kp, f, layout, 1.5)
    da, db = torch.randn_like(a), torch.randn_like(b)
    dq, dk = torch.autograd.grad([a, b], [q, k], [da, db])
    check(dq, da, qp, f, layout, 1.5, back=True)
    check(dk, db, kp, f, layout, 1.5, back=True)
    with torch.no_grad():
        assert torch.equal(E.rotary(q, None, qp, None, f, layout, 1.5)[0], a)


@pytest.mark.parametrize("n_q,n_k", [(1, 1), (1, 0), (0, 3), (0, 0), (2000, 1), (5, 30001)])
def test_counts(n_q, n_k):
    f = E.rotary_frequencies(32)
    q, qp = rows(n_q, 3, 32, BF16, 3)
    k, kp = rows(n_k, 1, 32, BF16, 4)
    a, b = E.rotary(q, k, qp, kp, f)
    check(a, q, qp, f, "half", 1.0)
    check(b, k, kp, f, "half", 1.0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(layout, dtype):
    q, qp = rows(50, 4, 64, dtype, 5)
    k, kp = rows(50, 2, 64, dtype, 6)
    f = E.rotary_frequencies(48)
    want = E.rotary(q, k, qp, kp, f, layout)
    wide = torch.full((50, 7, 71), float("nan"), dtype=dtype, device="cuda")
    wide[:, 1:5, 3:67] = q
    turned = k.transpose(0, 1).contiguous().transpose(0, 1)
    got = E.rotary(wide[:, 1:5, 3:67], turned, qp, kp, f, layout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    both = torch.cat([q, k], 1)                          # as one projection's rows hold them
    got = E.rotary(both[:, :4], both[:, 4:], qp, kp, f, layout)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = q[:1, :1].expand(50, 4, 64)
    check(E.rotary(one, None, qp, None, f, layout)[0], one, qp, f, layout, 1.0)
    leaf = q.detach().requires_grad_()
    out = E.rotary(leaf, None, qp, None, f, layout)[0]
    ones = torch.ones(1, 1, 1, dtype=dtype, device="cuda").expand(out.shape)
    check(torch.autograd.grad(out, leaf, ones)[0], ones, qp, f, layout, 1.0, back=True)


def test_one_side_wanted():
    f = E.rotary_frequencies(16)
    q, qp = rows(9, 2, 16, F32, 7)
    k, kp = rows(11, 2, 16, F32, 8)
    k.requires_grad_()
    a, b = E.rotary(q, k, qp, kp, f)
    db = torch.randn_like(b)
    check(torch.autograd.grad(b, k, db)[0], db, kp, f, "half", 1.0, back=True)
    q2, k2 = q.clone().requires_grad_(), k.detach().clone().requires_grad_()
    a, b = E.rotary(q2, k2, qp, kp, f)
    grads = torch.autograd.grad(a.sum(), [q2, k2], allow_unused=True)
    assert grads[1] is None or not grads[1].any()


def test_frequencies():
    f = E.rotary_frequencies(64, base=500.0)
    j = torch.arange(32, dtype=torch.float64)
    assert torch.allclose(f.cpu(), 500.0 ** (-j / 32), rtol=1e-14)
    assert torch.allclose(E.rotary_frequencies(64, factor=4.0).cpu() * 4, E.rotary_frequencies(64).cpu(), rtol=1e-14)
    slow = E.rotary_frequencies(64, factor=8.0, trained=2048).cpu()
    plain = E.rotary_frequencies(64).cpu()
    turns = 2048 * plain / (2 * torch.pi)
    assert torch.equal(slow[turns >= 32], plain[turns >= 32])
    assert torch.allclose(slow[turns <= 1] * 8, plain[turns <= 1], rtol=1e-14)
    assert (slow[1:] < slow[:-1]).all()
    # unusual ones: zero, negative, large, beyond the range
    odd = torch.tensor([0.0, -0.7, 1e6, 2e9, float("nan"), 6.283185307179586], dtype=torch.float64, device="cuda")
    q, qp = rows(20, 1, 12, F32, 9, longest=1000)
    qp[:5] = torch.tensor([0, 1, -1, 900, -900])
    got = E.rotary(q, None, qp, None, odd, "interleaved")[0]
    assert got[..., 6:10].isnan().all()
    fine = odd.clone()
    fine[3:5] = 0
    val, bound = R.rotary(q, qp, fine, "interleaved")
    for at in (slice(0, 6), slice(10, 12)):
        assert ((got.cpu().double() - val).abs() <= bound)[..., at].all()


def test_captured():
    f = E.rotary_frequencies(64)
    q, qp = rows(100, 4, 64, BF16, 10)
    k, kp = rows(300, 2, 64, BF16, 11)
    E.rotary(q, k, qp, kp, f)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = E.rotary(q, k, qp, kp, f)
    for i in range(3):
        q.copy_(rows(100, 4, 64, BF16, 12 + i)[0])
        kp.copy_(rows(300, 2, 64, BF16, 22 + i)[1])
        graph.replay()
        want = E.rotary(q, k, qp, kp, f)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_refusals_on_the_gpu():
    f = E.rotary_frequencies(16)
    q, qp = rows(4, 2, 16, F32, 13)
    with pytest.raises(ValueError, match="layout"):
        E.rotary(q, None, qp, None, f, layout="quarter")
    with pytest.raises(ValueError, match="positions"):
        E.rotary(q, None, qp.long(), None, f)
    with pytest.raises(ValueError, match="frequencies"):
        E.rotary(q, None, qp, None, f.float())
    with pytest.raises(E.EmbError, match="pairs"):
        E.rotary(q, None, qp, None, E.rotary_frequencies(18))
    with pytest.raises(ValueError, match="no gradient of the frequencies"):
        E.rotary(q, None, qp, None, f.clone().requires_grad_())
    with pytest.raises(E.EmbError, match="scale"):
        E.rotary(q, None, qp, None, f, scale=float("inf"))
    with pytest.raises(ValueError, match="one head size"):
        E.rotary(q, q[..., :8], qp, qp, f)
    with pytest.raises(ValueError, match="even"):
        E.rotary_frequencies(7)
