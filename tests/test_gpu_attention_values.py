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
