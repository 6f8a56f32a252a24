"""Plain 64-bit forms of the encoder's operators on the CPU (the gated delta rule, layer norm,
rotary positions), with a bound on the error that the kernels' roundings can make of each value.

With u the unit roundoff of the activations' type (2^-24 fp32, 2^-8 bf16) and e = 2^-24 that of
the accumulators, every result is rounded once (u |value|), and

Gated delta rule.  An error in the state is passed on by a (I - b k k^T), which for keys of at
most unit length never makes it longer, and local errors are at most a small multiple of e of
the terms that are summed: in 2-norm they add up to (n + sums' lengths) e of the terms'
magnitudes, which are taken here from true u, dr with their signs dropped.  For bf16 the
states, u and z that gradients read are rounded once more, two of them in one term at most, and
what outputs are made of carries 16 bits: 3 u and 2^-14 cover them.

Layer norm.  Means over c terms are off by at most (c / 64 + 10) e of the terms' mean magnitude
(64 lanes and a tree; 1024 of them for long rows), which enters xh once and once through r.

Rotary positions.  The angle is exact to 3e-9, sine and cosine to 1e-7, two products and a sum."""
import torch

E32 = 2.0 ** -24


def unit(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else E32


def _norm(t):
    return t.norm(dim=-1, keepdim=True)


def delta(q, k, v, gate, beta, offsets, state=None, mask=None, scale=None, do=None, dlast=None):
    """{name: (value, bound)} for o, last and, with do, the gradients."""
    dtype = v.dtype
    u, bf = unit(dtype), v.dtype == torch.bfloat16
    q, k, v, gate, beta = (t.detach().cpu().double() for t in (q, k, v, gate, beta))
    n, kh, dk = q.shape
    h, dv = v.shape[1:]
    g = h // kh
    scale = dk ** -0.5 if scale is None else scale
    off = offsets.tolist()
    samples = len(off) - 1
    keep = torch.ones(n, dtype=torch.bool) if mask is None else mask.cpu() != 0
    train = do is not None
    S0 = torch.zeros(samples, h, dk, dv, dtype=torch.float64) if state is None else state.detach().cpu().double()
    Q, K = q.repeat_interleave(g, 1), k.repeat_interleave(g, 1)
    a, b = torch.sigmoid(gate), torch.sigmoid(beta)
    z = torch.zeros_like
    val = {"o": z(v), "last": S0.clone()}
    bound = {"o": z(v), "last": 8 * E32 * S0.abs()}
    if train:
        do = do.detach().cpu().double()
        dlast = z(S0) if dlast is None else dlast.detach().cpu().double()
        for name, t in (("dq", Q), ("dk", K), ("dv", v), ("dgate", a), ("dbeta", b)):
            val[name], bound[name] = z(t), z(t)
        val["dstate"], bound["dstate"] = dlast.clone(), 8 * E32 * dlast.abs()
    ru = 3 * u if bf else 0.0
    out16 = 2.0 ** -14 if bf else 0.0
    for s in range(samples):
        rows = [t for t in range(off[s], off[s + 1]) if keep[t]]
        local = (4 * len(rows) + 2 * (dk + dv) + 200) * E32
        S, A = S0[s].clone(), S0[s].abs()
        before, us, abs_before = [], [], []
        for t in rows:
            before.append(S)
            abs_before.append(A)
            S = a[t][:, None, None] * S
            ut = b[t][:, None] * (v[t] - torch.einsum("hij,hi->hj", S, K[t]))
            S = S + K[t][:, :, None] * ut[:, None, :]
            A = a[t][:, None, None] * A + K[t].abs()[:, :, None] * ut.abs()[:, None, :]
            us.append(ut)
            val["o"][t] = scale * torch.einsum("hij,hi->hj", S, Q[t])
            mag = abs(scale) * torch.einsum("hij,hi->hj", A, Q[t].abs())
            bound["o"][t] = u * val["o"][t].abs() + (out16 + local) * (mag + _norm(mag))
        val["last"][s] = S
        bound["last"][s] = 8 * E32 * S.abs() + local * (A + A.flatten(1).norm(dim=1)[:, None, None])
        if not train:
            continue
        D, B = dlast[s].clone(), dlast[s].abs()
        most_dgate = torch.zeros(h, dtype=torch.float64)
        for t in reversed(rows):
            old, aold, ut = before.pop(), abs_before.pop(), us.pop()
            at, bt = a[t][:, None, None], b[t][:, None]
            new = at * old + K[t][:, :, None] * ut[:, None, :]
            anew = at * aold + K[t].abs()[:, :, None] * ut.abs()[:, None, :]
            val["dq"][t] = scale * torch.einsum("hij,hj->hi", new, do[t])
            mag = {"dq": abs(scale) * torch.einsum("hij,hj->hi", anew, do[t].abs())}
            D = D + scale * Q[t][:, :, None] * do[t][:, None, :]
            B = B + abs(scale) * Q[t].abs()[:, :, None] * do[t].abs()[:, None, :]
            du = torch.einsum("hij,hi->hj", D, K[t])
            dr = bt * du
            val["dv"][t] = dr
            mag_u = torch.einsum("hij,hi->hj", B, K[t].abs())
            mag["dv"] = bt * mag_u
            val["dk"][t] = torch.einsum("hij,hj->hi", D, ut) - torch.einsum("hij,hj->hi", at * old, dr)
            mag["dk"] = torch.einsum("hij,hj->hi", B, ut.abs()) + torch.einsum("hij,hj->hi", at * aold, mag["dv"])
            # d beta = du . (v - a S k) b (1 - b), and b (v - a S k) is u
            val["dbeta"][t] = (1 - b[t]) * (du * ut).sum(-1)
            mag["dbeta"] = (1 - b[t]) * (mag_u * ut.abs()).sum(-1)
            da = (D * old).sum((-1, -2)) - (dr * torch.einsum("hij,hi->hj", old, K[t])).sum(-1)
            val["dgate"][t] = a[t] * (1 - a[t]) * da
            mag["dgate"] = (1 - a[t]) * ((B * at * aold).sum((-1, -2)) +
                                         (mag["dv"] * torch.einsum("hij,hi->hj", at * aold, K[t].abs())).sum(-1))
            most_dgate = torch.maximum(most_dgate, mag["dgate"] / (1 - a[t]).clamp(min=1e-3))
            D = at * (D - K[t][:, :, None] * dr[:, None, :])
            B = at * (B + K[t].abs()[:, :, None] * dr.abs()[:, None, :])
            for name, m in mag.items():
                r = 0.0 if name == "dv" else ru
                spread = _norm(m) if m.dim() == 2 else m
                bound[name][t] = u * val[name][t].abs() + r * m + 2 * local * (m + spread)
        if rows:
            # Pairs of rows of a chunk enter the gradients of the gates between them, as the
            # difference of two sums over all of a chunk's pairs: at most 32 times the largest
            # gate's terms, in at most 40 additions.
            bound["dgate"][rows] += 32 * 40 * E32 * most_dgate
        val["dstate"][s] = D
        bound["dstate"][s] = 8 * E32 * D.abs() + 2 * local * (B + B.flatten(1).norm(dim=1)[:, None, None])
    if train:
        for name in ("dq", "dk"):                        # of shared heads: summed, rounded once
            whole = val[name].view(n, kh, g, dk).sum(2)
            part = bound[name] - u * val[name].abs()
            val[name], bound[name] = whole, u * whole.abs() + part.view(n, kh, g, dk).sum(2)
        if state is None:
            del val["dstate"], bound["dstate"]
    return {name: (val[name], bound[name] + 1e-30) for name in val}


def layer_norm(x, weight=None, bias=None, eps=1e-5, dy=None):
    u = unit(x.dtype)
    x = x.detach().cpu().double()
    c = x.shape[-1]
    w = torch.ones(c, dtype=torch.float64) if weight is None else weight.detach().cpu().double()
    b = torch.zeros(c, dtype=torch.float64) if bias is None else bias.detach().cpu().double()
    sums = (c / 64 + 10) * E32
    mean = x.mean(-1, keepdim=True)
    r = ((x - mean) ** 2).mean(-1, keepdim=True).add(eps).rsqrt()
    xh = (x - mean) * r
    off = r * (sums * x.abs().mean(-1, keepdim=True) + 2 * E32 * (x - mean).abs())   # of xh by the mean
    # the sum of squares is off by its own length and by twice the mean's error
    rel = 2 * sums + r * r * sums * x.abs().mean(-1, keepdim=True) * (x - mean).abs().mean(-1, keepdim=True) + 4 * E32
    dxh = off + xh.abs() * rel
    y = xh * w + b
    out = {"y": (y, u * y.abs() + dxh * w.abs() + 4 * E32 * ((xh * w).abs() + b.abs()) + 1e-30)}
    if dy is None:
        return out
    dy = dy.detach().cpu().double()
    gw = dy * w
    m1, m2 = gw.mean(-1, keepdim=True), (gw * xh).mean(-1, keepdim=True)
    dx = r * (gw - m1 - xh * m2)
    e1 = sums * gw.abs().mean(-1, keepdim=True)
    e2 = sums * (gw * xh).abs().mean(-1, keepdim=True) + (gw.abs() * dxh).mean(-1, keepdim=True)
    mag = gw.abs() + m1.abs() + (xh * m2).abs()
    out["dx"] = (dx, u * dx.abs() + r * (e1 + xh.abs() * e2 + dxh * m2.abs() + (8 * E32 + rel) * mag) + 1e-30)
    dy, xh, dxh = (t.reshape(-1, c) for t in (dy, xh, dxh))
    n = len(dy)
    add = (n + 40) * E32
    out["dweight"] = ((dy * xh).sum(0), (dy.abs() * dxh).sum(0) + add * (dy * xh).abs().sum(0) + 1e-30)
    out["dbias"] = (dy.sum(0), add * dy.abs().sum(0) + 1e-30)
    return out


def rotary(x, pos, frequencies, layout="half", scale=1.0, back=False):
    u = unit(x.dtype)
    x, f = x.detach().cpu().double(), frequencies.cpu()
    pairs = f.numel()
    t = torch.outer(pos.cpu().double(), f)[:, None] * (-1.0 if back else 1.0)
    i = torch.arange(pairs)
    at, bt = (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = x[..., at], x[..., bt]
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., at] = scale * (a * t.cos() - b * t.sin())
    y[..., bt] = scale * (b * t.cos() + a * t.sin())
    # the reference's own angle is off by 2^-53 of itself
    far = 2.0 ** -52 * t.abs() + 1e-7 + 4 * E32
    bound[..., at] = bound[..., bt] = abs(scale) * far * (a.abs() + b.abs())
    return y, bound + u * y.abs() * (bound > 0) + 1e-30
