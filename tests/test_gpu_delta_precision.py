"""The gated delta rule's arithmetic: bf16 calls compute what fp32 calls do from the same numbers,
to the bit, and round it once; fp32 results are within a few roundings of the 64-bit form's over
a whole tensor; a sample's results do not depend on what else is in the call."""
import pytest
import torch

import encoder_reference as R
from test_gpu_delta import BF16, F32, NAMES, call, make

pytestmark = pytest.mark.gpu

ROWS = ("q", "k", "v", "gate", "beta", "do")


def alone(t, s):
    """Sample s by itself."""
    off = t["offsets"][s:s + 2]
    rows = slice(int(off[0]), int(off[1]))
    one = {x: t[x][rows] for x in ROWS}
    one.update(state=None if t["state"] is None else t["state"][s:s + 1], dlast=t["dlast"][s:s + 1],
               mask=None if t["mask"] is None else t["mask"][rows], offsets=off - off[0])
    return one, rows


def as_f32(t):
    return {**t, **{x: t[x].float() for x in ROWS}}


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_sample_in_a_large_batch(dtype):
    """The same bits alone and among so many that what is kept for the gradients passes 32 MB."""
    lens = [((53 * i) % 211) + 60 for i in range(48)]
    t = make(lens, 4, 4, 128, 128, dtype, masked=0.1, seed=21)
    got = call(t)
    for s in (0, 7, 31, 47):
        one, rows = alone(t, s)
        for name, x in call(one).items():
            where = slice(s, s + 1) if name in ("last", "dstate") else rows
            assert torch.equal(x, got[name][where]), (s, name)


CASES = [([100, 65, 2, 0], 2, 2, 32, 32), ([37, 70], 1, 2, 40, 72), ([300, 77], 1, 2, 16, 128), ([90] * 20, 4, 4, 128, 128),
         ([200, 333], 2, 4, 64, 64), ([150], 1, 1, 96, 24), ([4300, 3000], 1, 1, 64, 32)]


def both(case, seed, strong=False):
    lens, kh, h, dk, dv = case
    t = make(lens, kh, h, dk, dv, BF16, masked=0.05, seed=seed)
    if strong:                                           # states that the rows' own writes are small beside
        t["state"] *= 8.0
        t["dlast"] *= 8.0
    return call(t), call(as_f32(t))


@pytest.mark.parametrize("case", CASES)
def test_bf16_states_are_fp32s(case):
    got, want = both(case, 22)
    for name in ("last", "dstate"):
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("strong", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_bf16_is_fp32_rounded_once(case, strong):
    got, want = both(case, 23, strong)
    for name in want:
        x = want[name] if name in ("last", "dstate") else want[name].to(BF16)
        assert torch.equal(got[name], x), (name, ((got[name] != x).double().mean()).item())


@pytest.mark.parametrize("strong", [False, True])
@pytest.mark.parametrize("case", CASES[:6])
def test_fp32_over_whole_tensors(case, strong):
    """A chunk's rows pass some eight stages whose roundings are 2^-24 of their terms each (in rows,
    in the state and in what meets them), and a state that remembers some 50 rows passes two
    chunks: as independent errors sqrt(16) 2^-24 of the terms' length.  Four times as much is let
    through, for terms that are longer than their sum."""
    lens, kh, h, dk, dv = case
    t = make(lens, kh, h, dk, dv, F32, masked=0.05, seed=24)
    if strong:
        t["state"] *= 8.0
        t["dlast"] *= 8.0
    got = call(t)
    ref = R.delta(*(t[x] for x in NAMES[:5]), t["offsets"], t["state"], t["mask"], None, t["do"], t["dlast"])
    for name, (val, _) in ref.items():
        off = (got[name].cpu().double() - val).norm() / val.norm().clamp(min=1e-30)
        assert off <= 16 * 2.0 ** -24, (name, off.item())
