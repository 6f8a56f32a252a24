"""The gated delta rule over samples long enough to be cut into segments of 1024 rows, whose states
are chained afterwards: against the same samples walked whole, with a memory that reaches over
several segments, so that every link of the chain shows."""
import math

import pytest
import torch

import encoder_reference as R
from test_gpu_delta import BF16, F32, call, make

pytestmark = pytest.mark.gpu

ROWS = ("q", "k", "v", "gate", "beta", "do")


def long_memory(lens, dk, dv, dtype, seed):
    t = make(lens, 1, 1, dk, dv, dtype, masked=0.05, seed=seed)
    t["gate"] = (t["gate"] * 0.5 + 8.0).to(dtype)        # a segment forgets a tenth to a third by this,
    t["beta"] = (t["beta"] * 0.5 - 5.5).to(dtype)        # and as much by its writes
    return t


def whole(t, samples):
    """The same call with so many more samples, of a row each, that none is cut."""
    more = 64
    extra = make([1] * more, 1, 1, t["q"].shape[2], t["v"].shape[2], t["q"].dtype, seed=99)
    both = {x: torch.cat([t[x], extra[x]]) for x in ROWS + ("state", "dlast")}
    both["mask"] = torch.cat([t["mask"], torch.ones(more, dtype=torch.uint8, device="cuda")])
    both["offsets"] = torch.cat([t["offsets"], t["offsets"][-1] + torch.arange(1, more + 1, device="cuda").int()])
    n = t["q"].shape[0]
    return {x: y[:samples] if x in ("last", "dstate") else y[:n] for x, y in call(both).items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 24), (64, 128), (96, 40), (128, 128), (8, 16)])
@pytest.mark.parametrize("lens", [[2048], [2049], [3072], [4000], [5100], [6144], [8200], [9216], [12300], [20000],
                                  [10241, 0, 1024, 5000], [1, 4097, 6000]])
def test_segments(lens, dk, dv, dtype):
    """A chunk's errors are 4 x 2^-24 of the state (eight stages' roundings), those of up to 640
    chunks are carried on and add up as independent ones, on either side."""
    t = long_memory(lens, dk, dv, dtype, seed=sum(lens) + dk)
    got, want = call(t), whole(t, len(lens))
    chunks = sum(lens) / 32
    far = 8 * math.sqrt(chunks) * 2.0 ** -24
    for name in want:
        a, b = got[name].double(), want[name].double()
        # each side of a rounded output is off by at most u of itself besides (a few large elements
        # of dgate can all be a step apart, so that no fewer can be asked for)
        tol = far if got[name].dtype == F32 else 2 * R.unit(dtype) + far
        assert ((a - b).norm() <= tol * b.norm()).item(), (name, ((a - b).norm() / b.norm()).item(), tol)


def test_the_memory_reaches():
    """What the test above is for: without the state at one end the other end's is another.  Five segments
    keep about a quarter of it; the gradient at the first row is that of 32 x 64 numbers of order one (a
    length of 45) beside some 3500 rows' q dO / 8 (5.6 each, 330 together): 45 / 4 / 330 is 0.03."""
    t = long_memory([5100], 64, 32, F32, seed=1)
    got, without = call(t), call({**t, "state": torch.zeros_like(t["state"]), "dlast": torch.zeros_like(t["dlast"])})
    for name in ("last", "dstate"):
        assert (got[name] - without[name]).norm() > 0.01 * got[name].norm(), name
