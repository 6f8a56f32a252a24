"""The gated delta rule's limits on rows, samples and heads: the query refuses what the calls refuse,
and takes what a launch can hold."""
import ctypes as C

import pytest

import embedding_columns_amd as E
from test_abi import L  # noqa: F401
from test_encoder_abi import delta

BIG = 1 << 62


def statuses(desc, training):
    a = C.c_size_t()
    query = E.lib().emb_delta_query(C.byref(desc), training, C.byref(a), C.byref(a), C.byref(a))
    # a workspace of no size where keys have to be packed: what the sizes allow ends at that, before any launch
    saved = 4096 if training else None
    forward = E.lib().emb_delta_forward(C.byref(desc), 4096, 4096, saved, 4096, BIG, None) if query else \
        E.lib().emb_delta_forward(C.byref(desc), 4096, 4096, saved, None, 0, None)
    return query, forward


@pytest.mark.parametrize("training", [0, 1])
@pytest.mark.parametrize("kw", [dict(n=9_000_000), dict(n=1 << 28), dict(n=(1 << 31) - 65536, dk=32), dict(n=1 << 28, dk=60, dv=20),
                                dict(samples=1 << 20, heads=4), dict(samples=1 << 16, heads=64, dv=16)])
def test_what_a_launch_holds(L, kw, training):  # noqa: F811
    assert statuses(delta(k=4100, **kw), training) == (0, 3)


@pytest.mark.parametrize("kw,training", [
    (dict(n=(1 << 31) - 65536), 1),                      # gradients of keys of 64: two wavefronts every 32 rows
    (dict(n=(1 << 31) - 65536, samples=1 << 20, dk=32), 0),
    (dict(samples=1 << 24, heads=4), 0), (dict(samples=1 << 20, heads=64, dv=128), 1),
])
def test_what_it_does_not(L, kw, training):  # noqa: F811
    assert statuses(delta(**kw), training) == (2, 2)
    assert "too many" in E.emb_last_error()


def test_workspaces_go_by_what_is_packed(L):  # noqa: F811
    """Keys and queries that are read in place take no room in the backward's workspace."""
    n, rows = 1000, 1000 * 2 * 64 * 2
    ready = E.emb_delta_query(delta(n=n))
    one, two = E.emb_delta_query(delta(n=n, k=4100)), E.emb_delta_query(delta(n=n, k=4100, q=4100))
    assert ready[0] == one[0] == two[0]
    for i in (1, 2):
        assert rows <= one[i] - ready[i] < rows + 256 and two[i] - one[i] == one[i] - ready[i]
