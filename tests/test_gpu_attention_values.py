"""Cross attention where values are not finite or lie far apart: each stays where the
definition has it."""
import math

import pytest
import torch

import sequence_reference as ref
from test_gpu_attention import BF16, F32, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("entry", [math.inf, math.nan, 3e38])
@pytest.mark.parametrize("heads,kv_heads,q_len", [(2, 1, [4, 40]), (16, 16, [1500, 2048])])
def test_a_masked_key_brings_no_bias(dtype, entry, heads, kv_heads, q_len):
    """A table's entry whose bucket holds masked keys alone takes no part, whatever it is:
    masked keys beside others in a block of keys, and whole blocks of them."""
    d, dout = make(dtype, q_len, [300, 200], heads, kv_heads, 32, buckets=5, seed=27)
    d["mask"] = torch.ones(500, dtype=torch.uint8, device="cuda")
    d["mask"][[3, 40, 41, 99, 310]] = 0
    d["mask"][128:160] = 0                            # half a tile of 64, one of 32
    d["mask"][192:256] = 0
    d["boundaries"] = torch.tensor([-50, 0, 50, 1000], dtype=torch.int32, device="cuda")
    d["q_pos"] = d["q_pos"] % 30
    d["k_pos"] = torch.where(d["mask"] == 0, -5000, d["k_pos"] % 100).int()     # masked: last bucket
    d["bias"][4] = 0
    want = run(d, dout)
    ref.check(want["out"], ref.attention(**d)["out"], "out")
    d["bias"][4] = entry
    got = run(d, dout)
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("junk", [math.nan, math.inf])
@pytest.mark.parametrize("heads,kv_heads,q_len", [(2, 1, [4, 40, 5]), (16, 16, [1500, 300, 1700])])
def test_rows_without_keys_have_no_gradient(dtype, junk, heads, kv_heads, q_len):
    """Whatever arrives as the gradient of an output that no key made."""
    d, dout = make(dtype, q_len, [20, 200, 70], heads, kv_heads, 32, buckets=5, masked=0.1, seed=28)
    rows = slice(q_len[0], q_len[0] + q_len[1])
    d["mask"][20:220] = 0                             # the second sample's
    d["bias"][4, 1] = -math.inf
    d["boundaries"][3], d["q_pos"][1] = 5000, 10 ** 6      # the second row, of head 1 alone
    want = run(d, dout)
    assert not want["out"][rows].any() and not want["out"][1, 1].any()
    dout[rows], dout[1, 1] = junk, junk
    d["q"][rows] = junk
    got = run(d, dout)
    assert not got["dq"][rows].any() and not got["dk"][20:220].any() and not got["dv"][20:220].any()
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_masked_keys_have_no_gradient(dtype):
    """Not even from a row whose own gradient is not finite."""
    d, dout = make(dtype, [4, 40], [90, 200], 2, 1, 32, buckets=5, masked=0.4, seed=29)
    dout[2], dout[30, 1] = math.nan, math.inf
    got = run(d, dout)
    out = d["mask"] == 0
    assert not got["dk"][out].any() and not got["dv"][out].any()


def neighbours(dtype, keys):
    """32 rows that share a block with buckets of their own: row i's keys in bucket i // 4."""
    d, dout = make(dtype, [32], [keys], 1, 1, 32, buckets=8, seed=30)
    d["k_pos"][:] = 0
    d["q_pos"][:] = torch.arange(32, dtype=torch.int32) // 4
    d["boundaries"] = torch.arange(1, 8, dtype=torch.int32, device="cuda")
    return d, dout


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("junk", [math.nan, math.inf])
@pytest.mark.parametrize("row", [0, 13, 31])
def test_a_bucket_gets_its_own_gradients_alone(dtype, junk, row):
    d, dout = neighbours(dtype, 32)
    want = run(d, dout)["dbias"]
    dout[row] = junk
    got = run(d, dout)["dbias"]
    others = torch.arange(8, device="cuda") != row // 4
    assert torch.equal(got[others], want[others]) and not torch.isfinite(got[row // 4]).any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("large", [0, 3, 7])
def test_a_small_bucket_beside_a_large_one(dtype, large):
    """Each bucket's sum within the bound of its own terms."""
    d, dout = neighbours(dtype, 150)
    dout[4 * large:4 * large + 4] *= 2.0 ** 24
    ref.check(run(d, dout)["dbias"], ref.attention(**d, dout=dout)["dbias"], "dbias")
