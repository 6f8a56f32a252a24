"""The gated delta rule where rows hold NaN or infinities and are not masked: what the definition
makes of them, and nothing else, is not finite."""
import pytest
import torch

import embedding_columns_amd as E
import encoder_reference as R
from test_gpu_delta import BF16, F32, NAMES, call, make

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
ROWS = ("q", "k", "v", "gate", "beta", "do")


def reference(t):
    return R.delta(*(t[x] for x in NAMES[:5]), t["offsets"], t["state"], t["mask"], None, t["do"], t["dlast"])


def check(clean, bad, got, forward=False):
    """What is finite in the 64-bit form of the bad inputs depends on no bad value, so that the
    form of the clean ones has the same values there, and its bounds hold."""
    ref, want = reference(clean), reference(bad)
    for name, x in got.items():
        x = x.cpu().double()
        finite = torch.isfinite(want[name][0])
        assert torch.equal(torch.isfinite(x), finite), (name, (torch.isfinite(x) != finite).nonzero()[:8].tolist())
        val, bound = ref[name]
        assert ((x - val).abs() <= bound)[finite].all(), name


def both(t, name, at, value):
    bad = {**t, name: t[name].clone()}
    bad[name][at] = value
    return bad


def run(t, name, at, value):
    bad = both(t, name, at, value)
    check(t, bad, call(bad))
    check(t, bad, call(bad, train=False))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("row", [0, 5, 15, 16, 20, 31, 37, 89])
@pytest.mark.parametrize("name", ROWS)
def test_a_row_of_nan(name, row, dtype):
    """Rows at the ends and inside of chunks of 32 rows and of their halves."""
    t = make([90, 40], 1, 2, 40, 24, dtype, masked=0.1, seed=31)
    t["mask"][row] = 1
    run(t, name, row, NAN)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_one_infinite_element(name, value, dtype):
    t = make([30, 70], 2, 4, 64, 64, dtype, seed=32)
    run(t, name, (55, 1, 33), value)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (32, 16), (100, 72), (128, 128)])
def test_head_sizes(dk, dv, dtype):
    t = make([45, 50], 1, 2, dk, dv, dtype, seed=33)
    for name in ("q", "k", "v", "gate", "do"):
        run(t, name, (20, 0, dk // 2 if name in "qk" else dv // 2)[:t[name].dim()], NAN)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [NAN, INF])
@pytest.mark.parametrize("name", ["state", "dlast"])
def test_a_state(name, value, dtype):
    """One element of the first state, or of what comes for the last: its column alone."""
    t = make([40, 33, 5], 2, 2, 32, 48, dtype, masked=0.2, seed=34)
    run(t, name, (1, 0, 7, 30), value)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_rows_under_a_state_that_is_not_finite(dtype):
    """They give zero and keep the state as it is, the finite numbers beside the infinity too."""
    t = make([70, 20], 1, 2, 32, 16, dtype, seed=35)
    t["mask"] = torch.ones(90, dtype=torch.uint8, device="cuda")
    t["mask"][40:70] = 0
    t["mask"][70:] = 0
    t["state"][1, 0, 5, 2] = INF
    t["v"][10] = NAN
    o, last = E.gated_delta(*(t[x] for x in NAMES[:5]), offsets=t["offsets"], state=t["state"], mask=t["mask"])
    assert o[10:40].isnan().all() and not o[40:].any() and torch.isfinite(o[:10]).all()
    assert torch.equal(last[1], t["state"][1])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_samples_keep_to_themselves(dtype):
    """A sample of nothing but NaN among others, which have the same bits as without it."""
    t = make([50, 33, 64, 7], 2, 4, 64, 32, dtype, seed=36)
    want = call(t)
    off = t["offsets"].tolist()
    bad = {**t, **{x: t[x].clone() for x in ROWS}}
    for x in ROWS:
        bad[x][off[1]:off[2]] = NAN
    got = call(bad)
    rows = torch.ones(off[-1], dtype=torch.bool, device="cuda")
    rows[off[1]:off[2]] = False
    for name in want:
        keep = torch.tensor([True, False, True, True], device="cuda") if name in ("last", "dstate") else rows
        assert torch.equal(got[name][keep], want[name][keep]), name
        assert not torch.isfinite(got[name][~keep]).any(), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_cut_samples(name, dtype):
    """A sample that is walked in segments, bad in its second of three."""
    t = make([2500], 1, 1, 16, 16, dtype, seed=37)
    run(t, name, 1500, NAN)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_largest_keys(dtype):
    """Keys whose products pass fp32 make what the definition makes of them in fp32: not the rows
    before them."""
    t = make([64], 1, 1, 32, 32, dtype, seed=38)
    t["k"][40] = 1e30
    t["k"][41] = 1e30
    o, last = E.gated_delta(*(t[x] for x in NAMES[:5]), offsets=t["offsets"], state=t["state"])
    assert torch.isfinite(o[:40]).all() and not torch.isfinite(last).all()
