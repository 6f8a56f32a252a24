"""The encoder operators' host side: descriptors match the header, sizes are told without a
GPU, and bad arguments come back as a status before any launch."""
import ctypes as C
import os
import re

import pytest
import torch

import embedding_columns_amd as E
from test_abi import L  # noqa: F401  (the fixture that builds the library where there is none)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "emb.h")
SIZES = {"int32_t": 4, "float": 4, "int64_t": 8, "emb_rotary_rows": C.sizeof(E.RotaryRows)}


def delta(**kw):
    d = dict(dtype=E.BF16, samples=8, key_heads=2, heads=4, dk=64, dv=32, scale=0.125, n=1000, q=4096,
             k=4096, v=4096, gate=4096, beta=4096, q_stride=128, q_head_stride=64, k_stride=128,
             k_head_stride=64, v_stride=128, v_head_stride=32, gate_stride=4, beta_stride=4,
             offsets=4096)
    d.update(kw)
    return E.DeltaDesc(**d)


def norm(**kw):
    d = dict(dtype=E.BF16, channels=64, inner=1, eps=1e-5, rows=100, x=4096, x_stride=64)
    d.update(kw)
    return E.NormDesc(**d)


def rotary(q=None, k=None, **kw):
    side = dict(x=4096, y=4096, pos=4096, n=10, stride=128, head_stride=64, heads=2)
    d = dict(dtype=E.BF16, layout=0, dim=64, pairs=32, scale=1.0, frequencies=4096,
             q=E.RotaryRows(**{**side, **(q or {})}), k=E.RotaryRows(**{**side, **(k or {})}))
    d.update(kw)
    return E.RotaryDesc(**d)


@pytest.mark.parametrize("name,desc", [("emb_delta", E.DeltaDesc), ("emb_norm", E.NormDesc),
                                       ("emb_rotary_rows", E.RotaryRows), ("emb_rotary", E.RotaryDesc)])
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
    assert fields == [(n, getattr(desc, n).size) for n, _ in desc._fields_]


def test_sizes_without_a_gpu(L):  # noqa: F811
    a = C.c_size_t()
    saved, forward, backward = E.emb_delta_query(delta())
    # the states before every 32 rows and what was written at every row
    assert saved >= 1000 // 32 * 4 * 64 * 32 * 2 + 1000 * 4 * 32 * 2
    assert backward > 1000 // 32 * 4 * 64 * 32 * 2
    inference = E.emb_delta_query(delta(), training=False)
    assert inference[0] == inference[2] == 0 and 0 < inference[1] < saved
    # heads that are no multiple of 32, or lie unaligned, are packed first
    assert E.emb_delta_query(delta(dk=60), training=False)[1] > inference[1]
    assert E.emb_delta_query(delta(k=4100), training=False)[1] > inference[1]
    assert E.emb_norm_query(norm()) >= 2 * 64 * 4
    assert E.emb_norm_query(norm(rows=0)) == 0
    assert E.lib().emb_delta_query(None, 1, C.byref(a), C.byref(a), C.byref(a)) == 1
    assert E.lib().emb_delta_query(C.byref(delta()), 1, None, C.byref(a), C.byref(a)) == 1
    assert E.lib().emb_norm_query(None, C.byref(a)) == 1
    assert E.lib().emb_norm_query(C.byref(norm()), None) == 1


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dtype=2), 1, "dtype"), (dict(samples=-1), 1, "samples"), (dict(n=-1), 1, "n must"),
    (dict(heads=3), 1, "key_heads"), (dict(key_heads=0), 1, "key_heads"), (dict(heads=0), 1, "key_heads"),
    (dict(dk=0), 1, "dk"), (dict(dv=-1), 1, "dk"), (dict(dk=129), 2, "128"), (dict(dv=129), 2, "128"),
    (dict(heads=1 << 16, key_heads=1), 2, "65535"), (dict(scale=float("nan")), 1, "scale"),
    (dict(scale=float("inf")), 1, "scale"), (dict(n=1 << 31), 2, "2^31"), (dict(samples=1 << 25), 2, "2^24"),
    (dict(q_stride=-1), 1, "strides"), (dict(v_head_stride=-5), 1, "strides"),
    (dict(k_stride=(1 << 21) + 1), 2, "2^21"),
])
def test_delta_refuses(L, kw, status, msg):  # noqa: F811
    a = C.c_size_t()
    assert E.lib().emb_delta_query(C.byref(delta(**kw)), 1, C.byref(a), C.byref(a), C.byref(a)) == status
    assert msg in E.emb_last_error()


def test_delta_calls_refuse_buffers(L):  # noqa: F811
    fwd, bwd, step = E.lib().emb_delta_forward, E.lib().emb_delta_backward, E.lib().emb_delta_step
    big = 1 << 40
    for kw in (dict(offsets=None), dict(q=None), dict(gate=None), dict(v=4097), dict(beta=4097), dict(state=4098)):
        d = delta(**kw)
        assert fwd(C.byref(d), 4096, 4096, None, 4096, big, None) == 1
        assert bwd(C.byref(d), 4096, 4096, 128, 32, None, 4096, 4096, 4096, 4096, 4096, None, 4096, big, None) == 1
    d = delta()
    assert fwd(None, 4096, 4096, None, 4096, big, None) == 1
    assert fwd(C.byref(d), None, 4096, None, 4096, big, None) == 1
    assert fwd(C.byref(d), 4096, None, None, 4096, big, None) == 1
    assert fwd(C.byref(d), 4096, 4096, 4100, 4096, big, None) == 1
    assert fwd(C.byref(d), 4096, 4096, None, 4096, 16, None) == 3
    assert fwd(C.byref(d), 4096, 4096, None, None, big, None) == 3
    assert fwd(C.byref(d), 4096, 4096, None, 4100, big, None) == 3

    def back(saved=4096, dout=4096, s=128, hs=32, dlast=None, dq=4096, dk=4096, dv=4096, dg=4096, db=4096,
             dstate=None, ws=4096, n=big):
        return bwd(C.byref(d), saved, dout, s, hs, dlast, dq, dk, dv, dg, db, dstate, ws, n, None)
    assert back(saved=None) == back(saved=4100) == back(dout=None) == back(dq=None) == back(db=None) == 1
    assert back(dout=4097) == back(dg=4097) == back(dlast=4098) == back(dstate=4098) == back(s=-1) == 1
    assert back(s=1 << 22) == 2 and back(n=1024) == back(ws=None) == back(ws=4100) == 3
    assert bwd(None, 4096, 4096, 128, 32, None, 4096, 4096, 4096, 4096, 4096, None, 4096, big, None) == 1
    assert step(None, 4096, 4096, None) == 1
    assert step(C.byref(delta(n=0)), None, None, None) == 0
    assert step(C.byref(d), None, 4096, None) == step(C.byref(d), 4096, None, None) == 1
    assert step(C.byref(d), 4098, 4096, None) == step(C.byref(delta(q=4097)), 4096, 4096, None) == 1
    assert step(C.byref(delta(n=1 << 24)), 4096, 4096, None) == 2


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dtype=7), 1, "dtype"), (dict(channels=0), 1, "channels"), (dict(inner=0), 1, "inner"),
    (dict(channels=16385), 2, "16384"), (dict(rows=-1), 1, "rows"), (dict(rows=7, inner=2), 1, "rows"),
    (dict(x_stride=-1), 1, "strides"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(eps=float("inf")), 1, "eps"), (dict(rows=1 << 41), 2, "2^40"),
])
def test_norm_refuses(L, kw, status, msg):  # noqa: F811
    a = C.c_size_t()
    assert E.lib().emb_norm_query(C.byref(norm(**kw)), C.byref(a)) == status
    assert msg in E.emb_last_error()


def test_norm_calls_refuse_buffers(L):  # noqa: F811
    fwd, bwd = E.lib().emb_norm_forward, E.lib().emb_norm_backward
    d = norm()
    assert fwd(None, 4096, None, None) == fwd(C.byref(d), None, None, None) == fwd(C.byref(d), 4097, None, None) == 1
    assert fwd(C.byref(d), 4096, 4098, None) == fwd(C.byref(norm(x=None)), 4096, None, None) == 1
    assert fwd(C.byref(norm(weight=4098)), 4096, None, None) == 1
    assert fwd(C.byref(norm(rows=0, x=None)), None, None, None) == 0

    def back(stats=4096, dy=4096, s=64, dx=4096, dw=4096, db=None, ws=4096, n=1 << 30):
        return bwd(C.byref(d), stats, dy, s, 0, dx, dw, db, ws, n, None)
    assert back(stats=None) == back(dy=None) == back(dx=None) == back(dy=4097) == back(dw=4098) == back(s=-1) == 1
    assert back(ws=None) == back(n=16) == back(ws=4098) == back(dw=None, db=4096, n=0) == 3


@pytest.mark.parametrize("kw,status,msg", [
    (dict(dtype=7), 1, "dtype"), (dict(layout=2), 1, "layout"), (dict(dim=0), 1, "dim"), (dict(pairs=33), 1, "pairs"),
    (dict(pairs=-1), 1, "pairs"), (dict(dim=1025), 2, "1024"), (dict(scale=float("nan")), 1, "scale"),
    (dict(frequencies=None), 1, "frequencies"), (dict(frequencies=4100), 1, "frequencies"),
    (dict(q=dict(n=-1)), 1, "n must"), (dict(k=dict(heads=0)), 1, "heads"), (dict(q=dict(n=1 << 31)), 2, "2^31"),
    (dict(k=dict(heads=1024)), 2, "2^16"), (dict(q=dict(stride=-1)), 1, "strides"), (dict(q=dict(x=None)), 1, "given"),
    (dict(k=dict(pos=None)), 1, "given"), (dict(k=dict(y=4097)), 1, "aligned"), (dict(q=dict(pos=4098)), 1, "aligned"),
])
def test_rotary_refuses(L, kw, status, msg):  # noqa: F811
    assert E.lib().emb_rotary_turn(C.byref(rotary(**kw)), 0, None) == status
    assert msg in E.emb_last_error()
    assert E.lib().emb_rotary_turn(None, 0, None) == 1
    none = dict(n=0, x=None, y=None, pos=None, heads=0)
    assert E.lib().emb_rotary_turn(C.byref(rotary(q=none, k=none)), 0, None) == 0


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 1, 8)
    with pytest.raises(ValueError, match="GPU"):
        E.gated_delta(x, x, x, x[..., 0], x[..., 0], torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        E.gated_delta_step(x, x, x, x[..., 0], x[..., 0], torch.zeros(4, 1, 8, 8))
    with pytest.raises(ValueError, match="GPU"):
        E.layer_norm(x)
    with pytest.raises(ValueError, match="GPU"):
        E.rotary(x, None, torch.zeros(4, dtype=torch.int32), None, E.rotary_frequencies(8, device="cpu"))
    with torch.no_grad(), pytest.raises(TypeError):
        E.rotary([1.0], None, None, None, E.rotary_frequencies(8, device="cpu"))


def test_tangents_are_refused():
    import torch.autograd.forward_ad as fwAD
    x = torch.zeros(4, 1, 8)
    with fwAD.dual_level():
        dual = fwAD.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError, match="forward-mode"):
            E.layer_norm(dual)
        with pytest.raises(RuntimeError, match="forward-mode"):
            E.rotary(dual, None, torch.zeros(4, dtype=torch.int32), None, E.rotary_frequencies(8, device="cpu"))
        with pytest.raises(RuntimeError, match="forward-mode"):
            E.gated_delta(dual, x, x, x[..., 0], x[..., 0], torch.tensor([0, 4], dtype=torch.int32))


def test_frequencies_refuse():
    with pytest.raises(ValueError, match="even"):
        E.rotary_frequencies(5, device="cpu")
    with pytest.raises(ValueError, match="positive"):
        E.rotary_frequencies(8, base=0.0, device="cpu")
    with pytest.raises(ValueError, match="low"):
        E.rotary_frequencies(8, factor=2.0, trained=100, low=3.0, high=2.0, device="cpu")
