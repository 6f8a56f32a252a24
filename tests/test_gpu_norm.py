"""Layer norm's kernels against the 64-bit form, with the bounds of encoder_reference.py."""
import pytest
import torch

import embedding_columns_amd as E
import encoder_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(shape, dtype, affine=(True, True), seed=0, mean=0.5):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(shape, generator=gen) * 2 + mean).to(dtype).cuda()
    w = torch.randn(shape[-1], generator=gen).cuda() if affine[0] else None
    b = torch.randn(shape[-1], generator=gen).cuda() if affine[1] else None
    return x, w, b, torch.randn(shape, generator=gen).to(dtype).cuda()


def call(x, w, b, dy, eps=1e-5):
    leaves = [t.detach().requires_grad_() for t in (x, w, b) if t is not None]
    it = iter(leaves)
    y = E.layer_norm(next(it), None if w is None else next(it), None if b is None else next(it), eps)
    names = ["dx"] + ["dweight"] * (w is not None) + ["dbias"] * (b is not None)
    return {"y": y.detach(), **dict(zip(names, torch.autograd.grad(y, leaves, dy)))}


def check(x, w, b, dy, got, eps=1e-5):
    ref = R.layer_norm(x, w, b, eps, dy)
    for name, t in got.items():
        val, bound = ref[name]
        off = (t.cpu().double() - val).abs()
        assert t.shape == val.shape and (off <= bound).all(), (name, float((off / bound).max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,c", [(1, 1), (3, 2), (1000, 7), (5, 8), (70, 64), (33, 100), (257, 256), (9, 511), (65, 512),
                                    (300, 513), (20, 1000), (7, 1025), (40, 2048), (6, 2049), (5, 4097), (3, 8191), (2, 8200),
                                    (2, 16384)])
def test_sizes(rows, c, dtype):
    t = make((rows, c), dtype)
    check(*t, call(*t))
    y = E.layer_norm(*t[:3])
    assert torch.equal(y, call(*t)["y"])


@pytest.mark.parametrize("affine", [(False, False), (True, False), (False, True)])
def test_without_parameters(affine):
    t = make((77, 96), BF16, affine, seed=1)
    check(*t, call(*t))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    x, w, b, dy = make((50, 6, 40), dtype, seed=2)
    want = call(x, w, b, dy)
    check(x, w, b, dy, want)
    wide = torch.full((50, 8, 45), float("nan"), dtype=dtype, device="cuda")
    wide[:, 1:7, 3:43] = x
    gy = torch.full((50, 6, 43), float("nan"), dtype=dtype, device="cuda")
    gy[..., 1:41] = dy
    got = call(wide[:, 1:7, 3:43], w, b, gy[..., 1:41])
    turned = call(x.transpose(0, 1).contiguous().transpose(0, 1), w, b, dy.transpose(1, 2).contiguous().transpose(1, 2))
    columns = call(x[:, 2], w, b, dy[:, 2])
    for name in want:
        assert torch.equal(got[name], want[name]) and torch.equal(turned[name], want[name]), name
    check(x[:, 2], w, b, dy[:, 2], columns)
    check(x, w, b, dy[:1, :1].expand(x.shape), call(x, w, b, dy[:1, :1].expand(x.shape)))
    same = x[:1].expand(x.shape)
    check(same, w, b, dy, call(same, w, b, dy))


def test_other_shapes():
    x, w, b, dy = make((2, 3, 4, 16), F32, seed=3)
    check(x, w, b, dy, call(x, w, b, dy))
    check(x[0, 0, 0], w, b, dy[0, 0, 0], call(x[0, 0, 0], w, b, dy[0, 0, 0]))
    for shape in ((0, 8), (3, 0, 8)):
        t = make(shape, F32)
        got = call(*t)
        assert got["y"].shape == shape and not got["dweight"].any() and not got["dbias"].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_values(dtype):
    """Rows far from zero, rows of one value, large and small rows; a row of NaN keeps to itself."""
    x, w, b, dy = make((12, 200), dtype, seed=4)
    x[0] = 7.0
    x[1] = 0.0
    x[2] *= 1e15
    x[3] *= 1e-12
    x[4] += 100.0
    got = call(x, w, b, dy)
    check(x, w, b, dy, got)
    assert torch.equal(got["y"][1].float(), b.to(dtype).float())
    y = E.layer_norm(x, w, b)
    x[5, 3] = float("nan")
    x[6, 0] = float("inf")
    bad = E.layer_norm(x, w, b)
    assert bad[5:7].isnan().all() and torch.equal(torch.cat([bad[:5], bad[7:]]), torch.cat([y[:5], y[7:]]))


def test_the_same_bits_and_many_rows():
    t = make((30011, 128), BF16, seed=5)
    first = call(*t)
    check(*t, first)
    for _ in range(2):
        again = call(*t)
        for name in first:
            assert torch.equal(first[name], again[name]), name


def test_frozen_parts():
    x, w, b, dy = make((30, 64), F32, seed=6)
    want = call(x, w, b, dy)
    for which, name in enumerate(("dx", "dweight", "dbias")):
        ins = [t.detach().requires_grad_(i == which) for i, t in enumerate((x, w, b))]
        got, = torch.autograd.grad(E.layer_norm(*ins), [ins[which]], dy)
        assert torch.equal(got, want[name])


def test_captured():
    x, w, b, dy = make((500, 256), BF16, seed=7)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(x, w, b, dy)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(x, w, b, dy)
    for i in range(3):
        x.copy_(make((500, 256), BF16, seed=8 + i)[0])
        graph.replay()
        eager = call(x, w, b, dy)
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(got[name], eager[name]), name


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 16, device="cuda")
    with pytest.raises(ValueError, match="weight"):
        E.layer_norm(x, torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError, match="weight"):
        E.layer_norm(x.bfloat16(), torch.zeros(16, device="cuda", dtype=BF16))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        E.layer_norm(x.half())
    with pytest.raises(ValueError, match="last dimension"):
        E.layer_norm(x.t())
    with pytest.raises(E.EmbError, match="eps"):
        E.layer_norm(x, eps=-1.0)
    with pytest.raises(E.EmbError, match="16384"):
        E.layer_norm(torch.zeros(1, 16385, device="cuda"))
