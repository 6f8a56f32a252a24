"""The sequence operators' host side: descriptors match the header, sizes are told without
a GPU, and bad arguments come back as a status before any launch."""
import ctypes as C
import os
import re

import pytest

import embedding_columns_amd as E
from test_abi import L  # noqa: F401  (the fixture that builds the library where there is none)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "emb.h")
SIZES = {"int32_t": 4, "float": 4, "int64_t": 8}


def attention(**kw):
    d = dict(dtype=E.BF16, heads=4, kv_heads=2, dim=64, samples=8, buckets=0, scale=0.125, n_q=100,
             n_k=5000, q=4096, k=4096, v=4096, q_stride=256, q_head_stride=64, k_stride=128,
             k_head_stride=64, v_stride=128, v_head_stride=64, q_offsets=4096, k_offsets=4096)
    d.update(kw)
    return E.AttentionDesc(**d)


def recurrence(**kw):
    d = dict(dtype=E.BF16, samples=8, channels=64, n=1000, x=4096, gate=4096, x_stride=64,
             gate_stride=64, offsets=4096)
    d.update(kw)
    return E.RecurrenceDesc(**d)


@pytest.mark.parametrize("name,desc", [("emb_attention", E.AttentionDesc), ("emb_recurrence", E.RecurrenceDesc)])
def test_descriptors_match_the_header(name, desc):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), src, flags=re.S).group(1)
    fields = []
    for decl in body.split(";"):
        decl = " ".join(decl.split())
        if not decl:
            continue
        kind, names = re.match(r"(?:const )?(\w+) (.*)", decl).groups()
        for n in names.split(","):
            fields.append((n.strip(" *"), 8 if "*" in n else SIZES[kind]))
    ours = [(n, getattr(desc, n).size) for n, _ in desc._fields_]
    assert fields == ours


def test_sizes_without_a_gpu(L):  # noqa: F811
    one, two, rows = C.c_size_t(), C.c_size_t(), C.c_int64()
    few = E.emb_attention_query(attention(n_k=100))
    assert few[0] == 0 and few[1] >= 100 * 4 * 4
    # one query row over a long cache: its keys are split and the parts need room
    split = E.emb_attention_query(attention(samples=1, n_q=1, n_k=100_000))
    assert split[0] >= 2 * 4 * 64 * 4
    biased = E.emb_attention_query(attention(buckets=32))
    assert biased[1] > E.emb_attention_query(attention())[1]
    assert E.emb_recurrence_query(recurrence()) == (1000 // 8 + 10, 0)
    assert E.emb_recurrence_query(recurrence(samples=1, n=100_000))[1] > 0
    assert E.lib().emb_attention_query(None, C.byref(one), C.byref(two)) == 1
    assert E.lib().emb_attention_query(C.byref(attention()), None, C.byref(two)) == 1
    assert E.lib().emb_recurrence_query(None, C.byref(rows), C.byref(one)) == 1


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dtype=2), 1, "dtype"), (dict(heads=3), 1, "kv_heads"), (dict(heads=0), 1, "heads"),
    (dict(kv_heads=0), 1, "kv_heads"), (dict(dim=0), 1, "dim"), (dict(dim=129), 2, "128"),
    (dict(samples=-1), 1, "samples"), (dict(n_q=-1), 1, "n_q"), (dict(n_q=1 << 31), 2, "2^31"),
    (dict(n_k=(1 << 31) - 1), 2, "2^31"), (dict(n_q=1 << 30), 2, "2^31"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"), (dict(buckets=-1), 1, "buckets"),
    (dict(buckets=257), 2, "256"), (dict(heads=64, kv_heads=1, buckets=65), 2, "4096"),
    (dict(q_stride=-1), 1, "strides"), (dict(heads=1 << 17, kv_heads=1 << 17), 2, "65535"),
])
def test_attention_refuses(L, kw, status, msg):  # noqa: F811
    one, two = C.c_size_t(), C.c_size_t()
    assert E.lib().emb_attention_query(C.byref(attention(**kw)), C.byref(one), C.byref(two)) == status
    assert msg in E.emb_last_error()


def test_attention_calls_refuse_buffers(L):  # noqa: F811
    fwd, bwd = E.lib().emb_attention_forward, E.lib().emb_attention_backward
    ok = dict(q_offsets=4096, k_offsets=4096)
    for kw, msg in [(dict(q_offsets=None), "offsets"), (dict(q=None), "q, k and v"),
                    (dict(v=None), "q, k and v"), (dict(k=4097), "aligned"),
                    (dict(buckets=4), "bias"), (dict(buckets=4, bias=4096, q_pos=4096, k_pos=4096), "bias"),
                    (dict(buckets=4, bias=4098, q_pos=4096, k_pos=4096, boundaries=4096), "4-byte")]:
        d = attention(**{**ok, **kw})
        assert fwd(C.byref(d), 4096, None, None, None, 0, None) == 1 and msg in E.emb_last_error()
        assert bwd(C.byref(d), 4096, 4096, 4096, 4096, 256, 64, 4096, None, None, None, None, 0, None) == 1
        assert msg in E.emb_last_error()
    d = attention()
    assert fwd(C.byref(d), None, None, None, None, 0, None) == 1
    assert fwd(C.byref(d), 4098, None, None, None, 0, None) == 1
    assert fwd(None, 4096, None, None, None, 0, None) == 1
    split = attention(samples=1, n_q=1, n_k=100_000)
    assert fwd(C.byref(split), 4096, None, None, None, 0, None) == 3
    assert fwd(C.byref(split), 4096, None, None, 4096, 256, None) == 3
    assert fwd(C.byref(split), 4096, None, None, 4100, 1 << 30, None) == 3

    def back(d=d, out=4096, rest=4096, lse=4096, dout=4096, dq=4096, dk=None, dv=None, dbias=None, ws=None, n=0):
        return bwd(C.byref(d), out, rest, lse, dout, 256, 64, dq, dk, dv, dbias, ws, n, None)
    assert back(out=None) == back(rest=None) == back(lse=None) == back(dout=None) == back(dq=None) == 1
    assert back(dk=4096) == 1 and "together" in E.emb_last_error()
    assert back(dbias=4096) == 1 and "dbias" in E.emb_last_error()
    assert back(dq=4098) == 1
    assert back() == 3


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dtype=5), 1, "dtype"), (dict(samples=-1), 1, "samples"), (dict(channels=0), 1, "channels"),
    (dict(channels=(1 << 20) + 1, x_stride=1 << 21, gate_stride=1 << 21), 2, "2^20"),
    (dict(n=-1), 1, "n must"), (dict(n=1 << 31), 2, "2^31"), (dict(x_stride=63), 1, "strides"),
    (dict(gate_stride=1 << 21), 2, "2^21"),
])
def test_recurrence_refuses(L, kw, status, msg):  # noqa: F811
    rows, need = C.c_int64(), C.c_size_t()
    assert E.lib().emb_recurrence_query(C.byref(recurrence(**kw)), C.byref(rows), C.byref(need)) == status
    assert msg in E.emb_last_error()


def test_recurrence_calls_refuse_buffers(L):  # noqa: F811
    fwd, bwd, step = (E.lib().emb_recurrence_forward, E.lib().emb_recurrence_backward,
                      E.lib().emb_recurrence_step)
    d = recurrence()
    assert fwd(None, 4096, 4096, None, None, 0, None) == 1
    assert fwd(C.byref(d), None, 4096, None, None, 0, None) == 1
    assert fwd(C.byref(d), 4096, None, None, None, 0, None) == 1
    for kw in (dict(offsets=None), dict(x=None), dict(gate=4097), dict(state=4098)):
        assert fwd(C.byref(recurrence(**kw)), 4096, 4096, None, None, 0, None) == 1
    assert fwd(C.byref(recurrence(samples=1, n=100_000)), 4096, 4096, None, None, 0, None) == 3
    assert bwd(C.byref(d), None, 4096, None, 4096, 4096, None, None, 0, None) == 1
    assert bwd(C.byref(d), 4096, 4096, None, 4096, None, None, None, 0, None) == 1
    assert bwd(C.byref(d), 4096, 4097, None, 4096, 4096, None, None, 0, None) == 1
    assert step(E.F32, 0, 8, None, 8, None, 8, None, None, None) == 0
    assert step(E.F32, 4, 8, 4096, 8, 4096, 8, None, 4096, None) == 1
    assert step(E.F32, 4, 0, 4096, 8, 4096, 8, 4096, 4096, None) == 1
    assert step(9, 4, 8, 4096, 8, 4096, 8, 4096, 4096, None) == 1
