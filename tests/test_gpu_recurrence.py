"""The gated recurrence against its definition in 64 bits (sequence_reference derives the
bounds), at the lengths, masks, strides and values where it can go wrong."""
import math

import pytest
import torch

import embedding_columns_amd as E
import sequence_reference as ref
from test_gpu_attention import offsets

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(dtype, lengths, channels, state=True, masked=0.0, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(lengths)

    def normal(*shape, dtype=dtype, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).to(dtype)

    d = dict(x=normal(n, channels), gate=normal(n, channels, mean=2.0, std=2.0),
             offsets=offsets(lengths))
    if state:
        d["state"] = normal(len(lengths), channels, dtype=F32)
    if masked:
        d["mask"] = (torch.rand(n, generator=gen, device="cuda") >= masked).to(torch.uint8)
    return d, normal(n, channels), normal(len(lengths), channels, dtype=F32)


def run(d, dy=None, dlast=None):
    if dy is None:
        y, last = E.gated_recurrence(**d)
        return {"y": y, "last": last}
    names = [n for n in ("x", "gate", "state") if d.get(n) is not None]
    leaves = {n: d[n].detach().requires_grad_() for n in names}
    y, last = E.gated_recurrence(**{**d, **leaves})
    outs, given = ([y, last], [dy, dlast]) if dlast is not None else ([y], [dy])
    grads = torch.autograd.grad(outs, [leaves[n] for n in names], given)
    return {"y": y, "last": last, **{"d" + n: g for n, g in zip(names, grads)}}


def check(d, dy, dlast):
    got, want = run(d, dy, dlast), ref.recurrence(**d, dy=dy, dlast=dlast)
    for name in got:
        ref.check(got[name], want[name], name)
    alone = run(d)
    assert torch.equal(alone["y"], got["y"]) and torch.equal(alone["last"], got["last"])
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[1], [0, 1, 0, 17], [15, 16, 17], [127, 128, 129], [300, 2, 700],
                                     [5] * 60, [1] * 130])
@pytest.mark.parametrize("channels", [1, 3, 64, 130])
def test_lengths(dtype, lengths, channels):
    check(*make(dtype, lengths, channels, masked=0.2, seed=1))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", [[1500], [1024, 3000], [2048, 0, 1025, 5000]])
def test_long_sequences_are_split(dtype, lengths):
    check(*make(dtype, lengths, 70, masked=0.1, seed=2))
    check(*make(dtype, lengths, 20, state=False, seed=3))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_samples_of_very_different_lengths(dtype):
    """Many samples, long, short and empty ones beside one another, none of them cut."""
    gen = torch.Generator().manual_seed(16)
    lengths = torch.randint(0, 700, (130,), generator=gen).tolist()
    lengths[3], lengths[50], lengths[129] = 0, 1, 0
    check(*make(dtype, lengths, 130, masked=0.1, seed=17))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("channels", [33, 96])
def test_short_samples_with_a_long_one(dtype, channels):
    """A mean between 33 and 128 rows: four wavefronts, and one sample of many of their blocks."""
    gen = torch.Generator().manual_seed(20)
    lengths = torch.randint(0, 100, (40,), generator=gen).tolist()
    lengths[7], lengths[8], lengths[39] = 1300, 0, 64
    assert 32 < sum(lengths) // 40 <= 128
    check(*make(dtype, lengths, channels, masked=0.1, seed=21))


def test_many_samples():
    gen = torch.Generator().manual_seed(18)
    lengths = torch.randint(0, 4, (5000,), generator=gen).tolist()
    check(*make(F32, lengths, 3, masked=0.1, seed=19))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_state_or_mask_or_last_gradient(dtype):
    d, dy, _ = make(dtype, [40, 200], 34, state=False, seed=4)
    check(d, dy, None)


def test_only_the_last_state_has_a_gradient():
    d, _, dlast = make(F32, [40, 2000], 34, seed=5)
    leaves = {n: d[n].clone().requires_grad_() for n in ("x", "gate", "state")}
    _, last = E.gated_recurrence(**{**d, **leaves})
    got = torch.autograd.grad(last, list(leaves.values()), dlast)
    want = ref.recurrence(**d, dy=torch.zeros_like(d["x"]), dlast=dlast)
    for name, g in zip(("dx", "dgate", "dstate"), got):
        ref.check(g, want[name], name)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_masked_rows_are_never_read_into_results(dtype, junk):
    for lengths in ([30, 5], [1400, 200]):
        d, dy, dlast = make(dtype, lengths, 66, masked=0.4, seed=6)
        d["mask"][-5:] = 0
        clean = run(d, dy, dlast)
        out = d["mask"] == 0
        d["x"][out], d["gate"][out] = junk, junk
        got = run(d, dy, dlast)
        for name in got:
            assert torch.equal(got[name], clean[name]), name
        assert not got["dx"][out].any() and not got["dgate"][out].any()


def test_gates_at_their_ends():
    """Gates that let all through or nothing, infinities among them, keep or take exactly."""
    d, dy, dlast = make(F32, [6, 40], 8, seed=7)
    d["gate"][:, 0], d["gate"][:, 1] = math.inf, -math.inf
    d["gate"][:, 2], d["gate"][:, 3] = 200.0, -200.0
    got = run(d, dy, dlast)
    first = torch.cat([d["state"][0:1].expand(6, -1), d["state"][1:2].expand(40, -1)])
    for c in (0, 2):
        assert torch.equal(got["y"][:, c], first[:, c])
    for c in (1, 3):
        assert torch.equal(got["y"][:, c], d["x"][:, c])
        assert torch.equal(got["dx"][:6, c][:-1], dy[:5, c])
    assert all(torch.isfinite(t).all() for t in got.values())
    assert not got["dgate"][:, :4].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_rows(dtype):
    d, dy, dlast = make(dtype, [90, 1, 300], 64, masked=0.1, seed=8)
    want = run(d, dy, dlast)
    for shift in (0, 1):
        fused = torch.zeros(391, 2 * 64 + 1 + shift, dtype=dtype, device="cuda")
        fused[:, shift:64 + shift], fused[:, 64 + shift:128 + shift] = d["x"], d["gate"]
        v = dict(d, x=fused[:, shift:64 + shift], gate=fused[:, 64 + shift:128 + shift])
        got = run(v, dy, dlast)
        for name in want:
            assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_of_no_sample_give_zero(dtype):
    d, dy, dlast = make(dtype, [7, 60, 1500, 9], 10, seed=9)
    d["offsets"] = offsets([60, 1500], first=7)
    d["state"], dlast = d["state"][:2], dlast[:2]
    got = check(d, dy, dlast)
    for name in ("y", "dx", "dgate"):
        assert not got[name][:7].any() and not got[name][-9:].any()


@pytest.mark.parametrize("n,samples", [(0, 0), (0, 3), (4, 0)])
def test_empty_batches(n, samples):
    d, dy, dlast = make(F32, [n], 6, seed=10)
    d["offsets"] = torch.zeros(samples + 1, dtype=torch.int32, device="cuda")
    d["state"] = torch.randn(samples, 6, device="cuda")
    got = run(d, dy, torch.ones(samples, 6, device="cuda"))
    assert torch.equal(got["last"], d["state"]) and not got["y"].any() and not got["dx"].any()
    assert torch.equal(got["dstate"], torch.ones(samples, 6, device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,channels", [(0, 5), (1, 1), (3, 7), (65, 256)])
def test_step_equals_a_scan_of_one_row(dtype, rows, channels):
    d, _, _ = make(dtype, [1] * rows, channels, seed=11)
    want = ref.recurrence(**d)
    state = d["state"].clone()
    y = E.gated_recurrence_step(d["x"], d["gate"], state)
    ref.check(y, want["y"], "y")
    ref.check(state, want["last"], "last")
    wide = torch.zeros(rows, channels + 3, dtype=dtype, device="cuda")
    wide[:, 1:channels + 1] = d["x"]
    again, out = d["state"].clone(), torch.empty_like(y)
    assert E.gated_recurrence_step(wide[:, 1:channels + 1], d["gate"], again, out=out) is out
    assert torch.equal(out, y) and torch.equal(again, state)


def test_steps_follow_the_scan():
    d, _, _ = make(F32, [50], 64, seed=12)
    y, last = E.gated_recurrence(**d)
    state = d["state"].clone()
    for t in range(50):
        got = E.gated_recurrence_step(d["x"][t:t + 1], d["gate"][t:t + 1], state)
        assert torch.allclose(got[0], y[t], rtol=1e-5, atol=1e-6)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-6)


def test_against_differences():
    """<gradient, direction> against central differences of the operator itself: h = 2^-6,
    outputs of order one, directions of unit norm scaled to 3; truncation h^2 / 6 f''' is
    under 4e-5 x 27 x 5 and rounding under 1e-7 x 1000 / 2h."""
    d, dy, dlast = make(F32, [5, 60], 8, masked=0.1, seed=13)
    grads = run(d, dy, dlast)
    gen = torch.Generator(device="cuda").manual_seed(14)
    h = 2.0 ** -6
    for name in ("x", "gate", "state"):
        way = torch.randn(d[name].shape, generator=gen, device="cuda")
        way *= 3 / float(way.norm())

        def value(sign):
            r = run({**d, name: d[name] + sign * h * way})
            return (r["y"].double() * dy.double()).sum() + (r["last"].double() * dlast.double()).sum()
        slope = float(value(1) - value(-1)) / (2 * h)
        want = float((grads["d" + name].double() * way.double()).sum())
        assert abs(slope - want) < 0.01, (name, slope, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_same_bits_other_stream_and_graph(dtype):
    d, dy, dlast = make(dtype, [300, 4000], 64, masked=0.1, seed=15)
    want = run(d, dy, dlast)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(d, dy, dlast)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, last = E.gated_recurrence(**d)
    for _ in range(3):
        d["x"].mul_(-1)
        eager = run(d)
        y.zero_(), last.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager["y"]) and torch.equal(last, eager["last"])


def test_refusals():
    d, _, _ = make(F32, [3, 4], 6)
    bad = [{"x": d["x"].to(BF16)}, {"x": d["x"].double(), "gate": d["gate"].double()},
           {"x": d["x"].cpu()}, {"gate": d["gate"][:, :4]}, {"x": d["x"].t()},
           {"offsets": d["offsets"].long()}, {"state": d["state"][:1]},
           {"state": d["state"].to(BF16)}, {"mask": torch.ones(6, dtype=torch.uint8, device="cuda")}]
    for change in bad:
        with pytest.raises(ValueError):
            E.gated_recurrence(**{**d, **change})
    with pytest.raises(E.EmbError, match="channels"):
        E.gated_recurrence(d["x"][:, :0], d["gate"][:, :0], d["offsets"])
    with pytest.raises(ValueError):
        E.gated_recurrence_step(d["x"], d["gate"], d["state"])
    with pytest.raises(ValueError):
        E.gated_recurrence_step(d["x"][:2].requires_grad_(), d["gate"][:2], d["state"])
