"""The gated delta rule's kernels against the 64-bit form, with bounds derived in
encoder_reference.py, at the sizes, masks, strides and values where they can go wrong."""
import pytest
import torch

import embedding_columns_amd as E
import encoder_reference as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(lens, kh=1, h=1, dk=32, dv=32, dtype=F32, state=True, masked=0.0, seed=0, before=0, behind=0):
    """Inputs on the GPU; `before` and `behind` rows belong to no sample."""
    gen = torch.Generator().manual_seed(seed)
    n = before + sum(lens) + behind

    def randn(*s):
        return torch.randn(*s, generator=gen)
    k = randn(n, kh, dk) + 0.3
    t = dict(q=randn(n, kh, dk), k=k / k.norm(dim=-1, keepdim=True).clamp(min=1e-3) * 0.99, v=randn(n, h, dv),
             gate=randn(n, h) * 2 + 2, beta=randn(n, h) * 1.5)
    t = {name: x.to(dtype).cuda() for name, x in t.items()}
    t["state"] = randn(len(lens), h, dk, dv).cuda() if state else None
    t["offsets"] = torch.tensor([before] + list(lens)).cumsum(0).int().cuda()
    t["mask"] = (torch.rand(n, generator=gen) >= masked).to(torch.uint8).cuda() if masked else None
    t["do"] = randn(n, h, dv).to(dtype).cuda()
    t["dlast"] = randn(len(lens), h, dk, dv).cuda()
    return t


NAMES = ("q", "k", "v", "gate", "beta", "state")


def call(t, train=True, scale=None):
    ins = {x: t[x] for x in NAMES}
    if not train:
        o, last = E.gated_delta(**ins, offsets=t["offsets"], mask=t["mask"], scale=scale)
        return {"o": o, "last": last}
    leaves = {x: v.detach().requires_grad_() for x, v in ins.items() if v is not None}
    o, last = E.gated_delta(**{**ins, **leaves}, offsets=t["offsets"], mask=t["mask"], scale=scale)
    grads = torch.autograd.grad([o, last], list(leaves.values()), [t["do"], t["dlast"]])
    return dict(zip(("d" + x for x in leaves), grads), o=o.detach(), last=last.detach())


def check(t, got, scale=None):
    train = "dq" in got
    ref = R.delta(*(t[x] for x in NAMES[:5]), t["offsets"], t["state"], t["mask"], scale,
                  t["do"] if train else None, t["dlast"])
    assert set(ref) == set(got)
    for name, (val, bound) in ref.items():
        x = got[name].cpu().double()
        assert x.shape == val.shape, name
        off = (x - val).abs()
        assert torch.isfinite(x).all(), name
        assert (off <= bound).all(), (name, float(off.max()), float((off / bound).max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lens", [[1], [31], [32], [33], [64, 0, 5, 1], [0, 0, 3], [100, 65, 2, 0]])
def test_lengths(lens, dtype):
    t = make(lens, 2, 2, 32, 32, dtype)
    check(t, call(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (16, 24), (33, 31), (40, 72), (64, 64), (72, 8), (96, 100), (128, 128),
                                   (127, 96), (8, 128), (128, 4)])
def test_head_sizes(dk, dv, dtype):
    t = make([37, 70], 1, 2, dk, dv, dtype, seed=1)
    check(t, call(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kh,h", [(1, 1), (1, 3), (2, 6), (3, 3), (1, 8)])
def test_shared_heads(kh, h, dtype):
    t = make([45, 20], kh, h, 24, 40, dtype, masked=0.2, seed=2)
    check(t, call(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state", [True, False])
def test_forward_alone(state, dtype):
    t = make([90, 3, 0, 33], 2, 4, 64, 32, dtype, state=state, masked=0.1, seed=3)
    check(t, call(t, train=False))
    check(t, call(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_rows_hold_anything(dtype):
    """Masked rows of infinities and NaN, a sample without a kept row, rows of no sample."""
    t = make([40, 33, 70], 2, 2, 32, 64, dtype, masked=0.4, seed=4, before=5, behind=40)
    off = t["offsets"].tolist()
    t["mask"][off[1]:off[2]] = 0
    out = (t["mask"] == 0).nonzero()[:, 0]
    nobody = torch.cat([torch.arange(off[0]), torch.arange(off[3], t["q"].shape[0])]).cuda()
    want = call(t)
    for name in ("q", "k", "v", "gate", "beta", "do"):
        for i, rows in enumerate((out, nobody)):
            t[name][rows[0::2]] = float("nan")
            t[name][rows[1::2]] = float("inf")
    got = call(t)
    for name in got:
        assert torch.equal(got[name], want[name]), name
    for name in ("o", "dq", "dk", "dv", "dgate", "dbeta"):
        assert not got[name][out].any() and not got[name][nobody].any(), name
    assert torch.equal(got["last"][1], t["state"][1])
    assert torch.equal(got["dstate"][1], t["dlast"][1])
    for name in ("q", "k", "v", "gate", "beta", "do"):
        t[name][out] = 0
        t[name][nobody] = 0
    check(t, got)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gates_at_their_ends(dtype):
    """Gates that forget all or nothing, in one chunk, and writes that are all or nothing."""
    t = make([70, 40], 1, 2, 32, 32, dtype, seed=5)
    inf = float("inf")
    for name in ("gate", "beta"):
        t[name][3] = inf
        t[name][10] = -inf
        t[name][20] = -500.0
        t[name][21] = 500.0
        t[name][40] = -inf
        t[name][80:90] = -30.0
    got = call(t)
    check(t, got)
    assert not got["dgate"][3].any() and not got["dgate"][10].any() and not got["dbeta"][40].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_same_key_again(dtype):
    """Every row writes at one key: the system of a chunk is as far from the identity as it gets."""
    t = make([96], 1, 1, 32, 32, dtype, seed=6)
    t["k"][:] = t["k"][:1]
    t["gate"][:] = 8.0
    t["beta"][:] = 6.0
    check(t, call(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides(dtype):
    t = make([50, 14], 2, 4, 32, 32, dtype, seed=7)
    want = call(t)
    big = {}
    for name in ("q", "k", "v", "gate", "beta", "do"):
        x = t[name]
        wide = torch.zeros(x.shape[0], *(s + 3 for s in x.shape[1:]), dtype=dtype, device="cuda") + float("nan")
        part = wide[(slice(None),) + tuple(slice(1, 1 + s) for s in x.shape[1:])]
        part.copy_(x)
        big[name] = part
    got = call({**t, **big})
    for name in want:
        assert torch.equal(got[name], want[name]), name
    # heads before rows
    turned = {x: t[x].transpose(0, 1).contiguous().transpose(0, 1) for x in ("q", "k", "v", "do")}
    got = call({**t, **turned})
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_broadcast_inputs(dtype):
    """One row and one head for all: their gradients are summed by autograd."""
    t = make([40], 2, 2, 32, 32, dtype, state=False, seed=8)
    one = {x: t[x][:1, :1].detach().clone().requires_grad_() for x in ("q", "k", "v")}
    full = {x: one[x].expand(t[x].shape) for x in one}
    o, _ = E.gated_delta(**full, gate=t["gate"], beta=t["beta"], offsets=t["offsets"])
    ones = torch.ones(1, 1, 1, dtype=dtype, device="cuda").expand(o.shape)
    got = torch.autograd.grad(o, list(one.values()), ones)
    t.update({x: full[x].detach().contiguous() for x in full}, do=ones.contiguous(), dlast=torch.zeros_like(t["dlast"]))
    each = call(t)
    check(t, each)
    for name, g in zip(one, got):
        want = each["d" + name].sum((0, 1), keepdim=True)
        size = each["d" + name].double().abs().sum((0, 1), keepdim=True)
        u = R.unit(dtype)
        assert ((g.double() - want.double()).abs() <= 2 * u * size).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_same_bits(dtype):
    t = make([300, 77, 200], 2, 4, 64, 64, dtype, masked=0.1, seed=9)
    first = call(t)
    for _ in range(3):
        again = call(t)
        for name in first:
            assert torch.equal(first[name], again[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cut_anywhere(dtype):
    """A sequence in two calls, the state handed over, is the sequence in one: what differs is
    where the chunks begin."""
    t = make([150], 1, 2, 32, 48, dtype, seed=10)
    whole = call(t, train=False)
    for cut in (1, 32, 77):
        state, outs = t["state"], []
        for rows in (slice(0, cut), slice(cut, 150)):
            part = {x: t[x][rows] for x in ("q", "k", "v", "gate", "beta")}
            off = torch.tensor([0, rows.stop - rows.start], dtype=torch.int32, device="cuda")
            o, state = E.gated_delta(**part, offsets=off, state=state)
            outs.append(o)
        check({**t}, {"o": torch.cat(outs), "last": state})
    assert whole["o"].shape == (150, 2, 48)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 32), (128, 128), (40, 72), (127, 127), (1, 1), (5, 128), (128, 3), (64, 20)])
def test_step(dk, dv, dtype):
    t = make([1] * 9, 2, 4, dk, dv, dtype, seed=11)
    check(t, call(t, train=False))
    state = t["state"].clone()
    version = state._version
    o = E.gated_delta_step(t["q"], t["k"], t["v"], t["gate"], t["beta"], state)
    check(t, {"o": o, "last": state})
    assert state._version > version
    out = torch.empty_like(o)
    state = t["state"].clone()
    assert E.gated_delta_step(t["q"], t["k"], t["v"], t["gate"], t["beta"], state, out=out) is out
    assert torch.equal(out, o)


def test_step_by_step_is_the_scan():
    t = make([60, 60], 1, 2, 64, 64, F32, seed=12)
    want = call(t, train=False)
    state = t["state"].clone()
    rows = torch.arange(2, device="cuda") * 60
    outs = []
    for i in range(60):
        outs.append(E.gated_delta_step(*(t[x][rows + i] for x in NAMES[:5]), state))
    o = torch.stack(outs, 1).reshape(120, 2, 64)
    check(t, {"o": o, "last": state})
    assert want["last"].shape == state.shape


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nothing_to_do(dtype):
    t = make([0, 0], 1, 2, 16, 16, dtype)
    got = call(t)
    assert torch.equal(got["last"], t["state"]) and torch.equal(got["dstate"], t["dlast"])
    assert got["o"].shape == (0, 2, 16) and got["dq"].shape == (0, 1, 16)
    t = make([], 1, 2, 16, 16, dtype, behind=3, state=False)
    got = call(t)
    assert not got["o"].any() and not got["dk"].any() and got["last"].shape == (0, 2, 16, 16)
    z = torch.empty(0, 1, 16, dtype=dtype, device="cuda")
    s = torch.empty(0, 1, 16, 16, device="cuda")
    assert E.gated_delta_step(z, z, z, z[..., 0], z[..., 0], s).shape == (0, 1, 16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scale_and_other_stream(dtype):
    t = make([80], 1, 1, 32, 32, dtype, seed=13)
    want = call(t, scale=-2.5)
    check(t, want, scale=-2.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(t, scale=-2.5)
    side.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long(dtype):
    """Many chunks of one sequence beside short ones."""
    t = make([700, 3, 90], 1, 2, 64, 64, dtype, masked=0.05, seed=14)
    check(t, call(t))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 32), (40, 72), (128, 96)])
def test_few_long_samples(dk, dv, dtype):
    """A few samples long enough to be walked in segments, which are joined afterwards."""
    t = make([4300, 0, 3000, 1300], 1, 2, dk, dv, dtype, masked=0.05, seed=17, before=3, behind=2)
    got = call(t)
    check(t, got)
    alone = call(t, train=False)
    # the same samples among so many that none is cut: both sides' states are off by what a
    # chunk's sums lose and a memory of some 50 rows passes on
    many = 64
    n = t["q"].shape[0]
    cat = {x: torch.cat([t[x]] * many) for x in ("q", "k", "v", "gate", "beta", "do", "mask", "state", "dlast")}
    off = torch.cat([t["offsets"].long()[:-1] + i * n for i in range(many)] + [t["offsets"].long()[-1:] + (many - 1) * n])
    # each copy's last sample ends where the next one's first begins: the rows between are masked
    nobody = torch.ones(n, dtype=torch.bool, device="cuda")
    nobody[3:-2] = False
    cat["mask"][nobody.repeat(many)] = 0
    whole = call({**cat, "offsets": off.int()})
    for name, a in {**got, **{x: alone[x] for x in alone}}.items():
        b = whole[name][:a.shape[0]].double()
        u = 2 * R.unit(dtype) if a.dtype is BF16 else (2 * (dk + dv) + 400) * R.E32
        assert ((a.double() - b).norm() <= u * b.norm()).item(), (name, ((a.double() - b).norm() / b.norm()).item())


def test_a_captured_step_of_training():
    t = make([100, 40], 2, 2, 64, 64, BF16, seed=15)
    want = call(t)
    ins = {x: t[x].clone() for x in NAMES}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call({**t, **ins})
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call({**t, **ins})
    for i in range(3):
        other = make([100, 40], 2, 2, 64, 64, BF16, seed=16 + i)
        for x in NAMES:
            ins[x].copy_(other[x])
        graph.replay()
        eager = call({**other, "do": t["do"], "dlast": t["dlast"], "offsets": t["offsets"]})
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(got[name], eager[name]), name
    assert set(want) == set(got)


def test_refusals_on_the_gpu():
    t = make([10], 1, 2, 16, 16)
    args = {x: t[x] for x in NAMES[:5]}
    off = t["offsets"]
    with pytest.raises(ValueError, match="do not fit"):
        E.gated_delta(**{**args, "k": t["k"][:, :, :8]}, offsets=off)
    with pytest.raises(ValueError, match="do not fit"):
        E.gated_delta(**{**args, "gate": t["gate"][:5]}, offsets=off)
    with pytest.raises(ValueError, match="share their type"):
        E.gated_delta(**{**args, "beta": t["beta"].bfloat16()}, offsets=off)
    with pytest.raises(ValueError, match="state"):
        E.gated_delta(**args, offsets=off, state=t["state"][:, :1])
    with pytest.raises(ValueError, match="offsets"):
        E.gated_delta(**args, offsets=off.long())
    with pytest.raises(ValueError, match="last dimension"):
        E.gated_delta(**{**args, "q": t["q"].repeat_interleave(2, 2)[..., ::2]}, offsets=off)
    with pytest.raises(E.EmbError, match="128"):
        big = torch.zeros(4, 1, 129, device="cuda")
        E.gated_delta(big, big, big, big[..., 0], big[..., 0], torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="no gradient"):
        E.gated_delta_step(t["q"][:1].requires_grad_(), *(t[x][:1] for x in NAMES[1:5]), t["state"])
    v = t["v"].clone().requires_grad_()
    o, _ = E.gated_delta(**{**args, "v": v}, offsets=off)
    with pytest.raises(RuntimeError, match="first derivatives"):
        torch.autograd.grad(o.sum(), v, create_graph=True)
