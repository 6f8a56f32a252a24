"""Cross attention with a bucket bias against its definition in 64 bits (sequence_reference
derives the bounds), at the sizes, masks, strides and values where it can go wrong."""
import math

import pytest
import torch

import embedding_columns_amd as E
import sequence_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def offsets(lengths, first=0):
    t = [first]
    for n in lengths:
        t.append(t[-1] + n)
    return torch.tensor(t, dtype=torch.int32, device="cuda")


def make(dtype, q_len, k_len, heads, kv_heads, dim, buckets=0, masked=0.0, seed=0, spread=1000):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    nq, nk = sum(q_len), sum(k_len)

    def normal(*shape, dtype=dtype):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    d = dict(q=normal(nq, heads, dim), k=normal(nk, kv_heads, dim), v=normal(nk, kv_heads, dim),
             q_offsets=offsets(q_len), k_offsets=offsets(k_len))
    if masked:
        d["mask"] = (torch.rand(nk, generator=gen, device="cuda") >= masked).to(torch.uint8)
    if buckets:
        d["bias"] = normal(buckets, heads, dtype=F32)
        edges = torch.randint(-spread, spread, (buckets - 1,), generator=gen, device="cuda")
        d["boundaries"] = edges.sort().values.to(torch.int32)
        d["q_pos"] = torch.randint(-spread, spread, (nq,), generator=gen, device="cuda").int()
        d["k_pos"] = torch.randint(-spread, spread, (nk,), generator=gen, device="cuda").int()
    return d, normal(nq, heads, dim)


def run(d, dout=None, **more):
    if dout is None:
        return {"out": E.cross_attention(**d, **more)}
    names = [n for n in ("q", "k", "v", "bias") if d.get(n) is not None]
    leaves = {n: d[n].detach().requires_grad_() for n in names}
    out = E.cross_attention(**{**d, **leaves}, **more)
    grads = torch.autograd.grad(out, [leaves[n] for n in names], dout)
    return {"out": out, **{"d" + n: g for n, g in zip(names, grads)}}


def check(d, dout, **more):
    got = run(d, dout, **more)
    want = ref.attention(**d, dout=dout, **more)
    for name in got:
        ref.check(got[name], want[name], name)
    alone = run(d, **more)["out"]
    assert torch.equal(alone, got["out"])
    return got


RAGGED = [([1], [1]), ([0, 3, 0, 1], [5, 0, 0, 31]), ([31, 1, 33], [33, 32, 31]),
          ([2, 130, 7], [129, 64, 300]), ([300, 1], [127, 255]), ([5] * 40, [17] * 40)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q_len,k_len", RAGGED)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 32), (4, 2, 64), (6, 2, 40), (2, 2, 128)])
def test_lengths(dtype, q_len, k_len, heads, kv_heads, dim):
    check(*make(dtype, q_len, k_len, heads, kv_heads, dim, buckets=9, masked=0.2, seed=1))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [1, 5, 8, 12, 33, 72, 127])
def test_odd_head_sizes(dtype, dim):
    check(*make(dtype, [3, 70], [40, 9], 3, 1, dim, buckets=4, seed=2))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("buckets", [0, 1, 2, 64, 65, 256])
def test_bucket_counts(dtype, buckets):
    check(*make(dtype, [33, 5], [100, 70], 2, 1, 32, buckets=buckets, masked=0.1, seed=3))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_keys_split_over_workgroups(dtype):
    check(*make(dtype, [1, 2], [9000, 5003], 4, 2, 64, buckets=16, masked=0.3, seed=4, spread=5))
    check(*make(dtype, [1], [4097], 1, 1, 128, seed=5))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_few_keys(dtype):
    check(*make(dtype, [700, 900], [3, 130], 2, 1, 64, buckets=7, seed=6))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,kv_heads,dim", [(16, 16, 32), (16, 16, 64), (32, 16, 40), (16, 16, 128),
                                                (16, 16, 33)])
def test_large_batches_share_key_tiles(dtype, heads, kv_heads, dim):
    """Enough rows for workgroups of 128 of them, whose wavefronts share their tiles of keys."""
    d, dout = make(dtype, [1500, 37, 1000, 0, 2048], [70, 300, 129, 50, 0], heads, kv_heads, dim,
                   buckets=9, masked=0.2, seed=22)
    check(d, dout)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_batches_with_sorted_positions(dtype):
    d, dout = make(dtype, [1500, 700, 1100], [200, 333, 65], 16, 16, 64, buckets=33, seed=23)
    d["k_pos"] = torch.cat([torch.arange(n) for n in (200, 333, 65)]).int().cuda() * 40
    d["q_pos"] = torch.cat([torch.arange(n) * 7 for n in (1500, 700, 1100)]).int().cuda()
    edges = [-3000, -200, -7, -1] + [int(1.4 ** j) + j for j in range(28)]
    d["boundaries"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
    check(d, dout)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_samples(dtype):
    gen = torch.Generator().manual_seed(24)
    q_len = torch.randint(0, 3, (4500,), generator=gen).tolist()
    k_len = torch.randint(0, 6, (4500,), generator=gen).tolist()
    check(*make(dtype, q_len, k_len, 1, 1, 16, buckets=3, masked=0.2, seed=25))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [32, 128])
def test_the_largest_table(dtype, dim):
    """256 buckets of 16 heads on one key head: the most that LDS holds beside the tiles."""
    check(*make(dtype, [3, 9], [150, 40], 16, 1, dim, buckets=256, seed=26))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sorted_positions(dtype):
    d, dout = make(dtype, [40, 200], [500, 700], 4, 4, 64, buckets=12, masked=0.1, seed=7)
    d["k_pos"] = torch.arange(1200, dtype=torch.int32, device="cuda")
    d["q_pos"] = torch.arange(240, dtype=torch.int32, device="cuda") * 5
    check(d, dout)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nothing_left_for_a_row(dtype):
    d, dout = make(dtype, [4, 40, 3], [20, 200, 33], 2, 1, 32, buckets=5, masked=0.1, seed=8)
    d["mask"][20:220] = 0
    got = check(d, dout)
    assert not got["out"][4:44].any() and not got["dq"][4:44].any()
    assert not got["dk"][20:220].any() and not got["dv"][20:220].any()
    d["mask"][:] = 0
    got = check(d, dout)
    assert all(not g.any() for g in got.values())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf, torch.finfo(BF16).min])
def test_masked_places_are_never_read_into_results(dtype, junk):
    d, dout = make(dtype, [4, 140], [90, 200], 2, 1, 64, buckets=5, masked=0.4, seed=9)
    clean = run(d, dout)
    for name in ("k", "v"):
        d[name][d["mask"] == 0] = junk
    got = run(d, dout)
    for name in got:
        assert torch.equal(got[name], clean[name]), name
    # a sample that is masked whole gives zero even to rows that are not finite
    d["mask"][:90] = 0
    d["q"][0] = math.nan
    assert not run(d)["out"][:4].any()


@pytest.mark.parametrize("low", [-math.inf, torch.finfo(F32).min, -1e30])
def test_a_bias_that_shuts_buckets(low):
    d, dout = make(F32, [3, 50], [60, 80], 2, 2, 32, buckets=4, seed=10)
    d["bias"][1] = low
    d["bias"][3, 1] = low
    if low == -math.inf:
        d["q_pos"][0] = 10 ** 6              # all its keys in the last bucket, shut for head 1
        got = check(d, dout)
        assert not got["out"][0, 1].any()
    else:
        got, want = run(d, dout), ref.attention(**d, dout=dout)
        for name in ("out", "dq", "dk", "dv"):
            assert torch.isfinite(got[name]).all()
            assert torch.allclose(got[name].cpu().double(), want[name][0], rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_positions_at_the_ends_of_int32(dtype):
    d, dout = make(dtype, [5, 40], [40, 50], 1, 1, 32, buckets=6, seed=11)
    lo, hi = -2 ** 31, 2 ** 31 - 1
    d["q_pos"][:] = torch.tensor([lo, hi, 0, -1, 1] * 9, dtype=torch.int32)
    d["k_pos"][:] = torch.tensor([hi, lo, lo + 1, 0, hi - 1] * 18, dtype=torch.int32)
    d["boundaries"][:] = torch.tensor([lo + 1, -1, 0, 0, hi], dtype=torch.int32)
    check(d, dout)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift", [0, 1])
def test_strided_and_shifted_views(dtype, shift):
    """Heads and rows out of a fused projection, and rows that start off 16-byte alignment."""
    d, dout = make(dtype, [3, 140], [50, 200], 4, 4, 64, buckets=5, seed=12)
    want = run(d, dout)
    fused = torch.zeros(250, 3, 4, 64 + 8 + shift, dtype=dtype, device="cuda")
    fused[:, 1, :, shift:64 + shift] = d["k"]
    fused[:, 2, :, shift:64 + shift] = d["v"]
    by_head = torch.zeros(4, 143, 64 + shift, dtype=dtype, device="cuda")
    by_head[:, :, shift:] = d["q"].transpose(0, 1)
    v = dict(d, k=fused[:, 1, :, shift:64 + shift], v=fused[:, 2, :, shift:64 + shift],
             q=by_head[:, :, shift:].transpose(0, 1))
    wide = torch.zeros(143, 4, 128, dtype=dtype, device="cuda")
    wide[:, :, :64] = dout
    got = run(v, wide[:, :, :64])
    for name in want:
        assert torch.equal(got[name], want[name]), name


def test_broadcast_keys_get_the_sum_of_their_gradients():
    d, dout = make(F32, [9, 30], [40, 70], 4, 4, 32, seed=13)
    one = d["k"][:, :1].contiguous().requires_grad_()
    out = E.cross_attention(**{**d, "k": one.expand(-1, 4, -1)})
    got = torch.autograd.grad(out, one, dout)[0]
    full = run({**d, "k": one.detach().expand(-1, 4, -1).contiguous()}, dout)
    assert torch.allclose(got, full["dk"].sum(1, keepdim=True), rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_no_sample_give_zero(dtype):
    d, dout = make(dtype, [2, 9, 45, 4], [60, 33, 80, 7], 2, 1, 32, buckets=5, masked=0.1, seed=14)
    d["q_offsets"], d["k_offsets"] = offsets([9, 45], first=2), offsets([33, 80], first=60)
    got = check(d, dout)
    assert not got["out"][:2].any() and not got["out"][56:].any()
    assert not got["dk"][:60].any() and not got["dv"][173:].any()


@pytest.mark.parametrize("nq,nk,samples", [(0, 0, 0), (0, 5, 1), (5, 0, 1), (0, 0, 3), (4, 4, 0)])
def test_empty_batches(nq, nk, samples):
    d, dout = make(F32, [nq], [nk], 2, 1, 32, buckets=3, seed=15)
    z = torch.zeros(samples + 1, dtype=torch.int32, device="cuda")
    d["q_offsets"], d["k_offsets"] = z.clone(), z.clone()
    if samples:
        d["q_offsets"][1:], d["k_offsets"][1:] = nq, nk
    got = run(d, dout)
    assert all(not g.any() for g in got.values())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_every_time(dtype):
    d, dout = make(dtype, [60, 200], [3000, 700], 4, 2, 64, buckets=9, masked=0.1, seed=16, spread=50)
    first = run(d, dout)
    for _ in range(3):
        again = run(d, dout)
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_scale_and_large_scores():
    d, dout = make(F32, [20], [300], 2, 2, 64, seed=17)
    d["q"] *= 30
    check(d, dout, scale=0.5)
    check(d, dout, scale=1e-6)


def test_against_differences():
    """<gradient, direction> against central differences of the operator itself.

    With h = 2^-6 and inputs and directions of unit size, a sum of 2 x 23 x 16 outputs has a
    third derivative of at most a few hundred along the direction (each factor of the
    softmax's third derivative is a centred score, |dim^-1/2 (q.dk + dq.k)| ~ 1.5), so the
    truncation h^2 / 6 f''' stays under 0.02 on values of order 10; the outputs' rounding
    gives 1e-7 x 700 / 2h < 0.005."""
    d, dout = make(F32, [3, 20], [40, 50], 2, 1, 16, buckets=5, masked=0.1, seed=18)
    grads = run(d, dout)
    gen = torch.Generator(device="cuda").manual_seed(19)
    h = 2.0 ** -6
    for name in ("q", "k", "v", "bias"):
        way = torch.randn(d[name].shape, generator=gen, device="cuda")
        way /= way.double().norm().item() ** 0.5      # a direction that moves few scores far

        def value(sign):
            return (run({**d, name: d[name] + sign * h * way})["out"].double() * dout.double()).sum()
        slope = float(value(1) - value(-1)) / (2 * h)
        want = float((grads["d" + name].double() * way.double()).sum())
        assert abs(slope - want) < 0.03, (name, slope, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_another_stream_and_a_graph(dtype):
    d, dout = make(dtype, [1, 150], [2000, 300], 4, 2, 64, buckets=9, seed=20)
    want = run(d, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(d, dout)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = E.cross_attention(**d)
    for _ in range(3):
        d["q"].mul_(-1)
        eager = E.cross_attention(**d)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_offsets_past_32_bits():
    """Rows of a cache whose element offsets pass 2^32."""
    stride = 1 << 16
    n = 70_000                                     # 70,000 rows of 65,536 elements: 9.2 GB
    cache = torch.empty(n * stride, dtype=BF16, device="cuda").view(n, stride)
    d, dout = make(BF16, [0, 3], [0, 100], 2, 1, 64, seed=21)
    cache[n - 100:, :64], cache[n - 100:, 64:128] = d["k"][:, 0], d["v"][:, 0]
    want = run(d)["out"]
    far = dict(d, k=cache[:, :64].view(n, 1, 64), v=cache[:, 64:128].view(n, 1, 64),
               k_offsets=torch.tensor([0, n - 100, n], dtype=torch.int32, device="cuda"))
    assert torch.equal(run(far)["out"], want)


def test_refusals():
    d, _ = make(F32, [3], [9], 2, 1, 32, buckets=4)
    bad = [({"q": d["q"].to(BF16)}, ValueError), ({"q": d["q"].double()}, ValueError),
           ({"q": d["q"].cpu()}, ValueError), ({"q": d["q"][0]}, ValueError),
           ({"q": d["q"].transpose(1, 2)}, ValueError), ({"k": d["k"][:, :, :16]}, ValueError),
           ({"v": d["v"][:5]}, ValueError), ({"q_offsets": d["q_offsets"].long()}, ValueError),
           ({"k_offsets": offsets([4, 5])}, ValueError), ({"bias": d["bias"].to(BF16)}, ValueError),
           ({"bias": d["bias"][:, :1]}, ValueError), ({"q_pos": None}, ValueError),
           ({"k_pos": d["k_pos"].long()}, ValueError), ({"boundaries": d["boundaries"][:2]}, ValueError),
           ({"mask": torch.ones(8, dtype=torch.uint8, device="cuda")}, ValueError),
           ({"scale": 0.0}, E.EmbError), ({"scale": -1.0}, E.EmbError), ({"scale": math.nan}, E.EmbError),
           ({"k": d["k"].expand(-1, 1, -1).repeat(1, 3, 1), "v": d["v"].repeat(1, 3, 1)}, E.EmbError)]
    for change, kind in bad:
        with pytest.raises(kind):
            E.cross_attention(**{**d, **change})
    big, _ = make(F32, [3], [9], 1, 1, 129)
    with pytest.raises(E.EmbError, match="dim"):
        E.cross_attention(**big)
    with pytest.raises(E.EmbError, match="256"):
        E.cross_attention(**make(F32, [3], [9], 1, 1, 32, buckets=257)[0])
    assert E.cross_attention(**d).shape == (3, 2, 32)
