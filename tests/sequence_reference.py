"""Plain 64-bit forms of the sequence operators on the CPU, sample by sample, with a
bound on the error that the kernels' roundings can make of each value.

Attention.  With u the unit roundoff of the activations' type (2^-24 fp32, 2^-8 bf16: 8 significant bits)
and e = 2^-24 that of the accumulators:
 - a score is a product of dim terms in fp32, so it is off by at most
   e (dim + 4) scale sum|q||k|, plus 8 e of |score| + |lse| + |bias| in the scaling and the
   exponent; a probability then by at most d = 2 max(that) + 16 e of itself;
 - bf16 probabilities and score gradients are rounded once more (u each) where they
   enter a product; a sum of n terms adds (n + 8) e; the result is rounded (u).
Every bound below is u |value| + (u' + d + (n + 8) e) (sum of the terms' magnitudes),
u' being u for bf16 and 0 for fp32."""
import math

import torch

E32 = 2.0 ** -24


def unit(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else E32


def buckets_of(apart, boundaries):
    """#{m : boundaries[m] <= apart}, apart saturated to int32."""
    apart = apart.clamp(-2 ** 31, 2 ** 31 - 1)
    n = torch.zeros_like(apart)
    for b in boundaries.tolist():
        n += apart >= b
    return n


def attention(q, k, v, q_offsets, k_offsets, mask=None, bias=None, boundaries=None, q_pos=None,
              k_pos=None, scale=None, dout=None):
    """{name: (value, bound)} for out, lse and, with dout, dq, dk, dv, dbias."""
    dtype, u = q.dtype, unit(q.dtype)
    uw = u if dtype == torch.bfloat16 else 0.0
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    qo, ko = q_offsets.tolist(), k_offsets.tolist()
    mask = None if mask is None else mask.cpu()
    heads, kv_heads, dim = q.shape[1], k.shape[1], q.shape[2]
    group = heads // kv_heads
    scale = dim ** -0.5 if scale is None else scale
    z = torch.zeros_like
    val = {"out": z(q), "lse": torch.full(q.shape[:2], -math.inf, dtype=torch.float64)}
    mag = {"out": z(q)}
    err = {"out": z(q), "lse": z(val["lse"])}
    if dout is not None:
        dout = dout.detach().cpu().double()
        for name, t in (("dq", q), ("dk", k), ("dv", v)):
            val[name], err[name] = z(t), z(t)
        if bias is not None:
            val["dbias"] = torch.zeros(bias.shape, dtype=torch.float64)
            err["dbias"] = z(val["dbias"])
    if bias is not None:
        table = bias.detach().cpu().double()
        q_pos, k_pos, boundaries = q_pos.cpu().long(), k_pos.cpu().long(), boundaries.cpu().long()
    for b in range(len(qo) - 1):
        rows = torch.arange(qo[b], qo[b + 1])
        cols = torch.arange(ko[b], ko[b + 1])
        if mask is not None:
            cols = cols[mask[cols] != 0]
        if not rows.numel() or not cols.numel():
            continue
        n, nr = cols.numel(), rows.numel() * group
        if bias is not None:
            bucket = buckets_of(q_pos[rows][:, None] - k_pos[cols][None, :], boundaries)
        for h in range(heads):
            qh, kh, vh = q[rows, h], k[cols, h // group], v[cols, h // group]
            s = qh @ kh.t() * scale
            size = qh.abs() @ kh.abs().t() * scale
            if bias is not None:
                add = table[:, h][bucket]
                s = s + add
                fine = add[torch.isfinite(add)]
                top_bias = float(fine.abs().max()) if fine.numel() else 0.0
            else:
                top_bias = 0.0
            top = s.amax(1, keepdim=True)
            dead = torch.isinf(top) & (top < 0)
            p = torch.exp(s - torch.where(dead, torch.zeros_like(top), top))
            total = p.sum(1, keepdim=True)
            p = p / torch.where(dead, torch.ones_like(total), total)
            lse = (top + torch.log(total))[:, 0]
            ends = lse[torch.isfinite(lse)]
            reach = float(ends.abs().max()) if ends.numel() else 0.0
            d = 2 * E32 * ((dim + 4 + 8) * float(size.max()) + 8 * (reach + top_bias)) + 16 * E32
            val["lse"][rows, h] = lse
            err["lse"][rows, h] = d + (n + 8) * E32 + E32 * lse.abs()
            val["out"][rows, h] = p @ vh
            err["out"][rows, h] = u * (p @ vh).abs() + (uw + d + (n + 8) * E32) * (p @ vh.abs())
            if dout is None:
                continue
            do = dout[rows, h]
            dp = do @ vh.t()
            dpa = do.abs() @ vh.abs().t()
            delta = (p * dp).sum(1, keepdim=True)
            delta_a = (p * dpa).sum(1, keepdim=True)
            ds = p * (dp - delta)
            f = d + (n + nr + dim + 8) * E32
            # what fp32 leaves of a score gradient: its terms' magnitudes, and delta's
            dsa = 2 * f * p * (dpa + delta_a)
            ka, qa = kh.abs(), qh.abs()
            val["dq"][rows, h] = scale * (ds @ kh)
            err["dq"][rows, h] = scale * (uw * ((p * dp).abs() @ ka + delta.abs() * (p @ ka))
                                          + dsa @ ka + f * ((p * dpa) @ ka + delta_a * (p @ ka)))
            val["dk"][cols, h // group] += scale * (ds.t() @ qh)
            err["dk"][cols, h // group] += scale * ((uw + f) * (ds.abs().t() @ qa) + dsa.t() @ qa)
            val["dv"][cols, h // group] += p.t() @ do
            err["dv"][cols, h // group] += (uw + f) * (p.t() @ do.abs())
            if bias is not None:
                val["dbias"][:, h] += torch.bincount(bucket.flatten(), ds.flatten(), len(table))
                err["dbias"][:, h] += torch.bincount(
                    bucket.flatten(), (dsa + (nr + n) * E32 * ds.abs()).flatten(), len(table))
    for name in ("dq", "dk", "dv"):
        if name in val:
            err[name] += u * val[name].abs()
    if "dbias" in val:
        err["dbias"] += E32 * len(qo) * val["dbias"].abs()
    return {name: (val[name], err[name]) for name in val}


def recurrence(x, gate, offsets, state=None, mask=None, dy=None, dlast=None):
    """{name: (value, bound)} for y, last and, with dy, dx, dgate, dstate.

    sigmoid(gate) and its complement are off by 8 e of themselves (an exponential of an
    argument up to ~20 and a reciprocal); each step multiplies by a <= 1 and adds, so the
    state's error obeys the state's own recurrence on magnitudes, 16 e a step, which the
    loop below carries along.  The same holds backward.  Outputs are rounded once (u)."""
    dtype, u = x.dtype, unit(x.dtype)
    x, gate = x.detach().cpu().double(), gate.detach().cpu().double()
    off = offsets.tolist()
    n, c = x.shape
    a, na = 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(gate))
    if mask is not None:
        out = mask.cpu() == 0
        a[out], na[out] = 1.0, 0.0
        x = torch.where(out[:, None], torch.zeros_like(x), x)
    y, ye = torch.zeros(n, c, dtype=torch.float64), torch.zeros(n, c, dtype=torch.float64)
    before, be = torch.zeros_like(y), torch.zeros_like(y)
    last = torch.zeros(len(off) - 1, c, dtype=torch.float64)
    le = torch.zeros_like(last)
    for b in range(len(off) - 1):
        h = torch.zeros(c, dtype=torch.float64) if state is None else state[b].detach().cpu().double()
        e = torch.zeros(c, dtype=torch.float64)
        for t in range(off[b], off[b + 1]):
            before[t], be[t] = h, e
            e = a[t] * e + 16 * E32 * (a[t] * h.abs() + na[t] * x[t].abs())
            h = a[t] * h + na[t] * x[t]
            y[t], ye[t] = h, e
        last[b], le[b] = h, e
    res = {"y": (y, u * y.abs() + ye), "last": (last, le + E32 * last.abs())}
    if dy is None:
        return res
    dy = dy.detach().cpu().double()
    g, ge = torch.zeros_like(y), torch.zeros_like(y)
    dstate, dse = torch.zeros_like(last), torch.zeros_like(last)
    for b in range(len(off) - 1):
        h = torch.zeros(c, dtype=torch.float64) if dlast is None else dlast[b].detach().cpu().double()
        e = torch.zeros(c, dtype=torch.float64)
        for t in range(off[b + 1] - 1, off[b] - 1, -1):
            e = e + 16 * E32 * (h.abs() + dy[t].abs())
            h = h + dy[t]
            g[t], ge[t] = h, e
            e, h = a[t] * e + 16 * E32 * a[t] * h.abs(), a[t] * h
        dstate[b], dse[b] = h, e
    dx, diff = na * g, before - x
    res["dx"] = (dx, u * dx.abs() + na * ge + 32 * E32 * dx.abs())
    dg = a * na * diff * g
    res["dgate"] = (dg, u * dg.abs() + a * na * (diff.abs() * ge + g.abs() * (
        be + 4 * E32 * (before.abs() + x.abs()))) + 64 * E32 * dg.abs())
    res["dstate"] = (dstate, dse + E32 * dstate.abs())
    if mask is not None:
        for name in ("dx", "dgate"):
            res[name][0][out], res[name][1][out] = 0.0, 0.0
    return res


def check(got, expected, name):
    """Every element of `got` within its bound of the 64-bit value (and 1e-30, for exact zeros)."""
    value, bound = expected
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (name, got.shape, value.shape)
    if not got.numel():
        return
    same = got == value                     # infinities included
    off = (got - value).abs()
    bad = ~same & ~(off <= bound + 1e-30)
    assert not bad.any(), (name, int(bad.sum()), float((off / (bound + 1e-30))[bad].max()),
                           [int(i) for i in bad.nonzero()[0]])
