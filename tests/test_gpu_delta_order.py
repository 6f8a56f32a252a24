"""The gated delta rule over more samples than walks run at once: they begin from the longest on, and
which one begins when changes nothing."""
import pytest
import torch

from test_gpu_delta import BF16, F32, call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("samples", [129, 200])
def test_many_samples(samples, dtype):
    gen = torch.Generator().manual_seed(samples)
    lens = torch.randint(0, 200, (samples,), generator=gen)
    lens[::7] = 133                                      # the same length often, and none
    lens[5::11] = 0
    t = make(lens.tolist(), 1, 3, 32, 32, dtype, masked=0.1, seed=samples, before=2, behind=1)
    got = call(t)
    check(t, got)
    alone = call(t, train=False)
    assert torch.equal(alone["o"], got["o"]) and torch.equal(alone["last"], got["last"])


def part(t, first, last):
    """Samples first .. last - 1 by themselves."""
    off = t["offsets"][first:last + 1]
    rows = slice(int(off[0]), int(off[-1]))
    some = {x: t[x][rows] for x in ("q", "k", "v", "gate", "beta", "do")}
    some.update(state=t["state"][first:last], dlast=t["dlast"][first:last], mask=None, offsets=off - off[0])
    return some, rows


@pytest.mark.parametrize("samples", [1023, 1024, 1025])
def test_as_many_as_are_ordered(samples):
    """The same bits as in parts that have too few walks to be ordered."""
    gen = torch.Generator().manual_seed(samples)
    t = make(torch.randint(30, 150, (samples,), generator=gen).tolist(), 1, 1, 8, 16, F32, seed=samples)
    got = call(t)
    for first in range(0, samples, 205):
        some, rows = part(t, first, min(first + 205, samples))
        for name, x in call(some).items():
            where = slice(first, first + 205) if name in ("last", "dstate") else rows
            assert torch.equal(x, got[name][where]), (first, name)


def test_a_sample_is_what_it_is_alone():
    """Every sample's rows and state to the bit, wherever its walk stands in the order."""
    lens = [((37 * i) % 171) for i in range(150)]
    t = make(lens, 2, 2, 64, 64, BF16, seed=1)
    got = call(t)
    for s in (0, 1, 37, 71, 149):
        one, rows = part(t, s, s + 1)
        for name, x in call(one).items():
            where = slice(s, s + 1) if name in ("last", "dstate") else rows
            assert torch.equal(x, got[name][where]), (s, name)


@pytest.mark.parametrize("samples", [8, 40])
def test_states_kept_either_way(samples):
    """bf16 gradients with the states before the chunks kept in fp32 (few of them) and in bf16."""
    gen = torch.Generator().manual_seed(samples)
    t = make(torch.randint(20, 200, (samples,), generator=gen).tolist(), 1, 4, 128, 128, BF16, masked=0.1, seed=samples)
    check(t, call(t))
