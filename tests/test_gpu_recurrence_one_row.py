"""Batches of a single row, whose stride no other row depends on, through the recurrence."""
import pytest
import torch

import embedding_columns_amd as E
import sequence_reference as ref
from test_gpu_recurrence import BF16, F32, check, make, run

pytestmark = pytest.mark.gpu


def one_row(values, stride, at_front=0):
    """`values` [1, C] as a view whose single row has another stride than C."""
    c = values.shape[1]
    big = torch.full((at_front + max(stride, c) * 2,), 9, dtype=values.dtype, device=values.device)
    view = big.as_strided((1, c), (stride, 1), at_front)
    view.copy_(values)
    return view


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("channels", [1, 64, 77, 130])
@pytest.mark.parametrize("stride", [0, 1, 5, 1 << 21])
def test_one_row_of_any_stride(dtype, channels, stride):
    """The stride of a single row says nothing: a transposed column's is 1, a broadcast row's 0."""
    d, dy, dlast = make(dtype, [1], channels, seed=22)
    want = check(d, dy, dlast)
    v = dict(d, x=one_row(d["x"], stride), gate=one_row(d["gate"], stride, at_front=1))
    assert v["x"].stride() == (stride, 1) and v["x"].is_contiguous()
    got = run(v, one_row(dy, stride), dlast)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    state = d["state"].clone()
    y = E.gated_recurrence_step(v["x"], v["gate"], state)
    ref.check(y, ref.recurrence(**d)["y"], "y")
    ref.check(state, ref.recurrence(**d)["last"], "last")
