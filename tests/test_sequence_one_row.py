"""The recurrence's descriptor of a single row, on the host."""
import ctypes as C

import pytest

import embedding_columns_amd as E
from test_abi import L  # noqa: F401  (the fixture that builds the library where there is none)
from test_sequence_abi import recurrence


@pytest.mark.parametrize("stride", [-1 << 40, -1, 0, 1, 63, 1 << 21, 1 << 62])
def test_one_row_has_no_stride(L, stride):  # noqa: F811
    """Of a batch of one row (or none) no stride is read, and none is refused."""
    rows, need = C.c_int64(), C.c_size_t()
    for n in (0, 1):
        d = recurrence(n=n, x_stride=stride, gate_stride=stride)
        assert E.lib().emb_recurrence_query(C.byref(d), C.byref(rows), C.byref(need)) == 0
    two = recurrence(n=2, x_stride=stride, gate_stride=stride)
    assert E.lib().emb_recurrence_query(C.byref(two), C.byref(rows), C.byref(need)) == (2 if stride > 63 else 1)
