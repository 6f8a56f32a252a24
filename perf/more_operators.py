"""The operators of a behaviour encoder's block at the sizes of real use: the gated delta
rule (a recurrence with a matrix state; scan, training step and single steps of serving),
layer norm and rotary positions, each with a plain form in elementary torch operations.

A case's `lengths` seeds its jagged lengths, so that a case's work is the same for
every seed of its values."""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64                   # rows that the plain delta rule takes together


def _delta(name, op, train, dtype, samples, n, key_heads, heads, dk, dv, state, masked, lengths):
    return {"name": name, "op": op, "train": train, "dtype": dtype, "samples": samples,
            "k_lo": n[0], "k_hi": n[1], "key_heads": key_heads, "heads": heads, "dk": dk, "dv": dv,
            "state": state, "masked": masked, "lengths": lengths}


def _norm(name, train, dtype, rows, channels, affine):
    return {"name": name, "op": "norm", "train": train, "dtype": dtype, "rows": rows,
            "channels": channels, "affine": affine}


def _rotary(name, train, dtype, n_q, n_k, heads, kv_heads, dim, part, layout, stretch, longest):
    return {"name": name, "op": "rotary", "train": train, "dtype": dtype, "n_q": n_q, "n_k": n_k,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "part": part, "layout": layout,
            "stretch": stretch, "longest": longest}


def listed():
    return [
        # one user's history of a request, encoded from nothing: latency alone counts
        _delta("delta_one_user", "delta", False, "bf16", 1, (50, 50), 4, 4, 32, 32, False, 0.0, 1),
        # states of a batch of histories of the long-sequence workload's lengths, some
        # positions masked, from stored states
        _delta("delta_histories", "delta", False, "bf16", 256, (200, 2000), 4, 4, 64, 64, True,
               0.1, 2),
        # lifelong histories of a few users: too few sequences to fill the chip by themselves
        _delta("delta_lifelong", "delta", False, "bf16", 2, (60000, 65537), 4, 4, 64, 128, True, 0.0,
               3),
        # a training step of the encoder on the workload's lengths
        _delta("train_delta", "delta", True, "bf16", 64, (200, 2000), 4, 4, 128, 128, False, 0.0, 4),
        # full precision, shared key heads, head sizes that are no powers of two, samples
        # without a history
        _delta("train_delta_odd_f32", "delta", True, "f32", 19, (0, 333), 2, 6, 40, 72, True, 0.2, 5),
        # one event for each of a batch of users: the state moves one step
        _delta("step_delta_users", "step", False, "bf16", 64, (1, 1), 4, 4, 64, 64, True, 0.0, 6),
        # the rows of one user's history before a layer: latency alone counts
        _norm("norm_one_user", False, "bf16", 50, 256, True),
        # a training step over all rows of a batch of histories
        _norm("train_norm", True, "bf16", 140771, 512, True),
        # full precision, wide rows of an odd count
        _norm("train_norm_wide_f32", True, "f32", 8191, 5000, True),
        # one candidate and one user's history
        _rotary("rotary_one_user", False, "bf16", 1, 50, 4, 4, 64, 64, "half", 1.0, 1 << 24),
        # a training step of attention between two long sequences: elapsed seconds as positions
        _rotary("train_rotary", True, "bf16", 14321, 14207, 8, 8, 128, 128, "half", 1.0, 1 << 24),
        # full precision, part of an odd head, neighbouring pairs, slowed for longer histories
        _rotary("train_rotary_part_f32", True, "f32", 301, 65537, 6, 3, 40, 24, "interleaved", 8.0,
                1 << 30),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    case = _draw(rng)
    return {key: value for key, value in case.items() if key != "name"}


def _draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["delta", "delta", "delta", "step", "norm", "norm", "rotary", "rotary"])
    train = op != "step" and rng.random() < 0.5
    wide = 1 if dtype == "bf16" else 2
    if op == "norm":
        channels = _log(rng, 8, 8192)
        if rng.random() < 0.5:
            channels = (channels + 7) // 8 * 8
        rows = _log(rng, 1, 2 ** 26 // (channels * wide))
        return _norm("", train, dtype, rows, channels, rng.random() < 0.8)
    if op == "rotary":
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        dim = rng.choice([16, 24, 32, 40, 64, 64, 96, 128])
        part = dim if rng.random() < 0.6 else 2 * rng.randint(1, dim // 2)
        most = 2 ** 24 // (dim * wide)
        return _rotary("", train, dtype, _log(rng, 1, most // heads), _log(rng, 1, most // kv), heads, kv, dim,
                       part, rng.choice(["half", "interleaved"]), rng.choice([1.0, 1.0, 4.0, 16.0]),
                       _log(rng, 64, 1 << 30))
    key_heads = rng.choice([1, 2, 3, 4])
    heads = key_heads * rng.choice([1, 1, 2, 4])
    dk, dv = (rng.choice([16, 24, 32, 40, 64, 64, 72, 96, 128]) for _ in range(2))
    lengths = rng.randrange(1, 1 << 20)
    if op == "step":
        return _delta("", op, False, dtype, _log(rng, 1, 2 ** 24 // (heads * dk * dv)), (1, 1), key_heads,
                      heads, dk, dv, True, 0.0, lengths)
    hi = _log(rng, 1, 8000 if train else 66000)
    most = 2 ** 25 // (wide * heads * max(dk, dv) * max(hi, 64))
    samples = max(1, min(1024, _log(rng, 1, max(1, most))))
    return _delta("", op, train, dtype, samples, (rng.randint(0 if samples > 8 else 1, hi), hi), key_heads, heads, dk, dv,
                  rng.random() < 0.5, rng.choice([0.0, 0.1, 0.3]), lengths)


# ------------------------------------------------------------------- inputs

def _lengths(case):
    rng = random.Random(case["lengths"])
    return [rng.randint(case["k_lo"], case["k_hi"]) for _ in range(case["samples"])]


def _frequencies(case):
    """Radians a step of each pair; a stretched table slows the pairs that turn less than
    32 times over 4096 steps, the slowest (less than once) by the whole factor."""
    pairs, stretch = case["part"] // 2, case["stretch"]
    freq = [10000.0 ** (-j / pairs) for j in range(pairs)]
    if stretch != 1.0:
        for j, f in enumerate(freq):
            turns = 4096 * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            freq[j] = f * (keep + (1.0 - keep) / stretch)
    return freq


def prepare(case, seed):
    device = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=device).manual_seed(seed)
    dtype, train = DTYPES[case["dtype"]], case["train"]

    def normal(*shape, mean=0.0, std=1.0, dtype=dtype):
        t = torch.randn(*shape, generator=gen, device=device)
        return t.mul_(std).add_(mean).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        n, c = case["rows"], case["channels"]
        # rows of a size of their own each, off zero, and a channel that stands out, as
        # sums of a few layers are
        size = torch.rand(n, 1, generator=gen, device=device).mul_(2).add_(0.2)
        x = torch.randn(n, c, generator=gen, device=device).mul_(size).add_(0.3)
        x[:, c // 3] += 6.0
        s["x"] = x.to(dtype).requires_grad_(train)
        s["weight"] = s["bias"] = None
        if case["affine"]:
            s["weight"] = normal(c, mean=1.0, std=0.2, dtype=torch.float32).requires_grad_(train)
            s["bias"] = normal(c, std=0.2, dtype=torch.float32).requires_grad_(train)
        if train:
            s["dy"] = normal(n, c)
        return s
    if case["op"] == "rotary":
        d = case["dim"]
        s["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=device)
        for x, n, heads in (("q", case["n_q"], case["heads"]), ("k", case["n_k"], case["kv_heads"])):
            s[x] = normal(n, heads, d).requires_grad_(train)
            s[x + "_pos"] = torch.randint(-case["longest"] // 8, case["longest"], (n,), generator=gen,
                                          device=device, dtype=torch.int32)
            if train:
                s["d" + x] = normal(n, heads, d)
        s["scale"] = 1.0 if case["stretch"] == 1.0 else 0.1 * math.log(case["stretch"]) + 1.0
        return s
    lens = _lengths(case)
    n = sum(lens) if case["op"] == "delta" else case["samples"]
    b, kh, h, dk, dv = (case[x] for x in ("samples", "key_heads", "heads", "dk", "dv"))
    # unit queries and keys; keys have a part in common, as those of related items do
    for x, mean in (("q", 0.0), ("k", 0.4)):
        t = torch.randn(n, kh, dk, generator=gen, device=device) + mean
        s[x] = (t / t.norm(dim=-1, keepdim=True)).to(dtype).requires_grad_(train)
    s["v"] = normal(n, h, dv).requires_grad_(train)
    s["gate"] = normal(n, h, mean=4.0, std=2.0).requires_grad_(train)     # mostly remembering
    s["beta"] = normal(n, h, std=1.5).requires_grad_(train)
    s["state"] = (normal(b, h, dk, dv, std=0.3, dtype=torch.float32).requires_grad_(train)
                  if case["state"] else None)
    if case["op"] == "step":
        return s
    total = [0]
    for m in lens:
        total.append(total[-1] + m)
    s["offsets"] = torch.tensor(total, dtype=torch.int32, device=device)
    s["longest"] = max(lens)
    s["mask"] = None
    if case["masked"]:
        s["mask"] = (torch.rand(n, generator=gen, device=device) >= case["masked"]).to(torch.uint8)
        if b > 1:
            s["mask"][total[1]:total[2]] = 0                              # a sample loses every row
    if train:
        s["do"] = normal(n, h, dv)
        s["dlast"] = normal(b, h, dk, dv, std=0.3, dtype=torch.float32)
    return s


# -------------------------------------------------------------- plain forms

def _plain_norm(s):
    case, dtype = s["case"], s["x"].dtype
    x = s["x"].detach().float()
    mean = x.mean(-1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)
    xh = x * rstd
    affine = s["weight"] is not None
    y = xh * s["weight"].detach() + s["bias"].detach() if affine else xh
    out = {"y": y.to(dtype)}
    if not case["train"]:
        return out
    dy = s["dy"].float()
    g = dy * s["weight"].detach() if affine else dy
    out["dx"] = (rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))).to(dtype)
    if affine:
        out["dweight"], out["dbias"] = (dy * xh).sum(0), dy.sum(0)
    return out


def _plain_turned(x, pos, s, back):
    """Pairs of x turned by their positions' angles (back: the other way)."""
    case, half = s["case"], s["case"]["part"] // 2
    angle = pos.double()[:, None] * s["freq"]
    cos = (angle.cos() * s["scale"]).float()[:, None]
    sin = (angle.sin() * (-s["scale"] if back else s["scale"])).float()[:, None]
    f = x.detach().float()
    out = f.clone()
    if case["layout"] == "half":
        a, b = slice(0, half), slice(half, 2 * half)
    else:
        a, b = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    out[..., a] = f[..., a] * cos - f[..., b] * sin
    out[..., b] = f[..., b] * cos + f[..., a] * sin
    return out.to(x.dtype)


def _plain_rotary(s):
    out = {"q": _plain_turned(s["q"], s["q_pos"], s, False),
           "k": _plain_turned(s["k"], s["k_pos"], s, False)}
    if s["case"]["train"]:
        out["dq"] = _plain_turned(s["dq"], s["q_pos"], s, True)
        out["dk"] = _plain_turned(s["dk"], s["k_pos"], s, True)
    return out


def _plain_step(s):
    g = s["case"]["heads"] // s["case"]["key_heads"]
    q, k = (s[x].float().repeat_interleave(g, 1) for x in ("q", "k"))
    a, b = torch.sigmoid(s["gate"].float())[..., None], torch.sigmoid(s["beta"].float())[..., None]
    old = s["state"] * a[..., None]
    u = b * (s["v"].float() - (old * k[..., None]).sum(-2))
    s["state"].copy_(old + k[..., None] * u[..., None, :])
    o = (s["state"] * q[..., None]).sum(-2) * s["case"]["dk"] ** -0.5
    return {"o": o.to(s["v"].dtype), "last": s["state"]}


def _plain_delta(s):
    """Chunks of rows: what each does to the state it is given as products of matrices, for
    all chunks side by side; the state goes through them one after another."""
    case = s["case"]
    b, kh, h, dk, dv = (case[x] for x in ("samples", "key_heads", "heads", "dk", "dv"))
    n, dtype, dev = s["v"].shape[0], s["v"].dtype, s["v"].device
    scale = dk ** -0.5
    chunks = max(1, -(-s["longest"] // CHUNK))
    off = s["offsets"].long()
    place = torch.arange(chunks * CHUNK, device=dev)
    there = place < (off[1:] - off[:-1])[:, None]
    index = (off[:-1, None] + place).clamp(max=max(n - 1, 0)) * there
    keep = there if s["mask"] is None or not n else there & (s["mask"][index] != 0)

    def leaf(x):
        return None if x is None else x.detach().float().requires_grad_(case["train"])

    q, k, v, gate, beta, state = (leaf(s[x]) for x in ("q", "k", "v", "gate", "beta", "state"))

    def cut(t, heads):               # [b, heads, chunks, CHUNK, ...], zero where no row is kept
        t = t[index] if n else t.new_zeros((b, chunks * CHUNK) + t.shape[1:])
        t = t * keep.view(keep.shape + (1,) * (t.dim() - 2))
        t = t.transpose(1, 2).reshape((b, heads, chunks, CHUNK) + t.shape[3:])
        return t.repeat_interleave(h // heads, 1)

    with torch.set_grad_enabled(case["train"]):
        rows = keep.view(b, 1, chunks, CHUNK)
        Q, K, V = cut(q, kh), cut(k, kh), cut(v, h)
        decay = torch.nn.functional.logsigmoid(cut(gate, h)).double() * rows
        B = (torch.sigmoid(cut(beta, h)) * rows)[..., None]
        total = decay.cumsum(-1)
        low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
        apart = (total[..., :, None] - total[..., None, :]).masked_fill(~low, 0.0)
        between = apart.exp().float() * low
        G = total.exp().float()[..., None]
        W = (total[..., -1:] - total).exp().float()[..., None]
        M = torch.matmul(K, K.transpose(-1, -2).contiguous()) * between * B
        M = M.tril(-1)
        # the inverse of I + M: blocks on the diagonal twice as large each time
        N = torch.eye(CHUNK, device=dev).expand_as(M)
        size = 1
        place = torch.arange(CHUNK, device=dev)
        while size < CHUNK:
            block = place // size
            lower = (block[:, None] % 2 == 1) & (block[None, :] == block[:, None] - 1)
            N = N - torch.matmul(torch.matmul(N, M * lower), N)
            size *= 2
        P = torch.matmul(Q, K.transpose(-1, -2).contiguous()) * between * scale
        Y, X = torch.matmul(N, B * V), torch.matmul(N, B * G * K)
        Q, K = Q * G * scale, (K * W).transpose(-1, -2).contiguous()
        S = state if state is not None else V.new_zeros(b, h, dk, dv)
        outs = []
        for c in range(chunks):
            U = Y[:, :, c] - torch.matmul(X[:, :, c], S)
            outs.append(torch.matmul(Q[:, :, c], S) + torch.matmul(P[:, :, c], U))
            S = S * G[:, :, c, -1:] + torch.matmul(K[:, :, c], U)
        o = torch.stack(outs, 2).reshape(b, h, chunks * CHUNK, dv).transpose(1, 2)
        o = o.new_zeros(n, h, dv).index_put((index[keep],), o[keep]) if n else 1.0 * v
    out = {"o": o.detach().to(dtype), "last": S.detach()}
    if not case["train"]:
        return out
    leaves = {"q": q, "k": k, "v": v, "gate": gate, "beta": beta}
    if state is not None:
        leaves["state"] = state
    grads = torch.autograd.grad([o, S], list(leaves.values()), [s["do"].float(), s["dlast"]],
                                allow_unused=True)
    for name, leaf, grad in zip(leaves, leaves.values(), grads):
        grad = torch.zeros_like(leaf) if grad is None else grad
        out["d" + name] = grad.to(torch.float32 if name == "state" else dtype)
    return out


# ------------------------------------------------------------------ one pass

PLAIN = {"norm": _plain_norm, "rotary": _plain_rotary, "delta": _plain_delta, "step": _plain_step}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    import embedding_columns_amd as E
    if op == "step":
        o = E.gated_delta_step(s["q"], s["k"], s["v"], s["gate"], s["beta"], s["state"])
        return {"o": o, "last": s["state"]}
    if op == "norm":
        y = E.layer_norm(s["x"], s["weight"], s["bias"])
        if not case["train"]:
            return {"y": y}
        wanted = [s["x"]] + ([s["weight"], s["bias"]] if s["weight"] is not None else [])
        return {"y": y, **dict(zip(("dx", "dweight", "dbias"), torch.autograd.grad(y, wanted, s["dy"])))}
    if op == "rotary":
        q, k = E.rotary(s["q"], s["k"], s["q_pos"], s["k_pos"], s["freq"], layout=case["layout"],
                        scale=s["scale"])
        if not case["train"]:
            return {"q": q, "k": k}
        dq, dk = torch.autograd.grad([q, k], [s["q"], s["k"]], [s["dq"], s["dk"]])
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    o, last = E.gated_delta(s["q"], s["k"], s["v"], s["gate"], s["beta"], s["offsets"],
                            state=s["state"], mask=s["mask"])
    if not case["train"]:
        return {"o": o, "last": last}
    names = ["q", "k", "v", "gate", "beta"] + (["state"] if s["state"] is not None else [])
    grads = torch.autograd.grad([o, last], [s[x] for x in names], [s["do"], s["dlast"]])
    return {"o": o, "last": last, **{"d" + x: g for x, g in zip(names, grads)}}


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        n, c = case["rows"], case["channels"]
        affine = 8 * c if case["affine"] else 0
        if case["train"]:
            return {"bytes": 4 * n * c * size + 2 * affine, "flops": 20 * n * c}
        return {"bytes": 2 * n * c * size + affine, "flops": 8 * n * c}
    if case["op"] == "rotary":
        elements = (case["n_q"] * case["heads"] + case["n_k"] * case["kv_heads"]) * case["dim"]
        passes = 2 if case["train"] else 1
        return {"bytes": passes * 2 * elements * size + 4 * (case["n_q"] + case["n_k"]),
                "flops": passes * 3 * elements}
    b, kh, h, dk, dv = (case[x] for x in ("samples", "key_heads", "heads", "dk", "dv"))
    n = sum(_lengths(case)) if case["op"] == "delta" else b
    rows = n * size * (2 * kh * dk + 2 * h * dv + 2 * h) + (n if case["masked"] else 0)
    states = 4 * b * h * dk * dv * (2 if case["state"] else 1)
    # products with the state: two reads and one update of it, and two more times that backwards
    if not case["train"]:
        return {"bytes": rows + states, "flops": 6 * n * h * dk * dv}
    return {"bytes": 2 * rows + 2 * states, "flops": 20 * n * h * dk * dv}


# ---------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if case["train"] and case.get("k_hi", 0) > 9000:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "delta": _exact_delta,
            "step": _exact_step}[case["op"]](s)


def _exact_norm(s):
    """Differentiated by way of the mean and the variance, as the chain rule has it."""
    x = s["x"].detach().double()
    c = x.shape[1]
    w = s["weight"].detach().double() if s["weight"] is not None else x.new_ones(c)
    mean, var = x.sum(1) / c, x.var(1, correction=0) + 1e-5
    apart = x - mean[:, None]
    out = {"y": apart / var.sqrt()[:, None] * w}
    if s["bias"] is not None:
        out["y"] += s["bias"].detach().double()
    if not s["case"]["train"]:
        return out
    dy = s["dy"].double()
    dxh = dy * w
    dvar = -0.5 * (dxh * apart).sum(1) * var ** -1.5
    dmean = -dxh.sum(1) / var.sqrt()
    out["dx"] = dxh / var.sqrt()[:, None] + (2 * dvar[:, None] * apart + dmean[:, None]) / c
    if s["weight"] is not None:
        out["dweight"] = (dy * apart / var.sqrt()[:, None]).sum(0)
        out["dbias"] = dy.sum(0)
    return out


def _exact_rotary(s):
    """Complex numbers multiplied by exp(i angle)."""
    part, layout = s["case"]["part"], s["case"]["layout"]

    def turned(x, pos, sign):
        x = x.detach().double()
        by = torch.polar(torch.full((1, 1), float(s["scale"]), dtype=torch.float64, device=x.device),
                         sign * torch.outer(pos.double(), s["freq"]))[:, None]
        head = x[..., :part]
        if layout == "half":
            z = torch.complex(*[t.contiguous() for t in head.chunk(2, -1)]) * by
            head = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.view_as_complex(head.reshape(head.shape[:-1] + (-1, 2)).contiguous()) * by
            head = torch.view_as_real(z).flatten(-2)
        return torch.cat([head, x[..., part:]], -1)

    out = {x: turned(s[x], s[x + "_pos"], 1.0) for x in ("q", "k")}
    if s["case"]["train"]:
        out.update({"d" + x: turned(s["d" + x], s[x + "_pos"], -1.0) for x in ("q", "k")})
    return out


def _moved(S, q, k, v, a, b):
    """One step of the definition: the new state, what was written and what is read."""
    S = a[..., None, None] * S
    u = b[..., None] * (v - torch.matmul(k[..., None, :], S)[..., 0, :])
    S = torch.addcmul(S, k[..., :, None], u[..., None, :])
    return S, u, torch.matmul(q[..., None, :], S)[..., 0, :]


def _in_64(s):
    case = s["case"]
    g = case["heads"] // case["key_heads"]
    q, k = (s[x].detach().double().repeat_interleave(g, 1) for x in ("q", "k"))
    gate, beta = s["gate"].detach().double(), s["beta"].detach().double()
    return q * case["dk"] ** -0.5, k, s["v"].detach().double(), torch.sigmoid(gate), torch.sigmoid(beta)


def _exact_step(s):
    q, k, v, a, b = _in_64(s)
    S, _, o = _moved(s["state"].double(), q, k, v, a, b)
    return {"o": o, "last": S}


def _exact_delta(s):
    """Step by step through time, all samples side by side, the longest first; backwards
    over stretches of steps whose states are made again."""
    case = s["case"]
    bs, kh, h, dk, dv = (case[x] for x in ("samples", "key_heads", "heads", "dk", "dv"))
    q, k, v, a, b = _in_64(s)
    if s["mask"] is not None:
        q[s["mask"] == 0] = 0
        a[s["mask"] == 0], b[s["mask"] == 0] = 1.0, 0.0
    off = s["offsets"].long()
    n = off[1:] - off[:-1]
    order = torch.argsort(n, descending=True, stable=True)
    sizes = n[order].tolist()
    alive, m = [], bs
    for t in range(s["longest"]):
        while m and sizes[m - 1] <= t:
            m -= 1
        alive.append(m)
    start = off[:-1][order]
    S = s["state"].detach().double()[order] if s["state"] is not None else v.new_zeros(bs, h, dk, dv)
    o = torch.zeros_like(v)
    stretch, kept = 40, []
    for t, m in enumerate(alive):
        if case["train"] and t % stretch == 0:
            kept.append(S.clone())
        at = start[:m] + t
        new, _, o[at] = _moved(S[:m], q[at], k[at], v[at], a[at], b[at])
        if m == bs:
            S = new
        else:
            S[:m] = new
    back = torch.argsort(order)
    out = {"o": o, "last": S[back]}
    if not case["train"]:
        return out
    do, E = s["do"].double(), s["dlast"].double()[order]
    dq, dk_, dv_, da, db = (torch.zeros_like(x) for x in (q, k, v, a, b))
    for c in reversed(range(len(kept))):
        steps = range(c * stretch, min(len(alive), (c + 1) * stretch))
        S, before = kept[c], []
        for t in steps:
            m = alive[t]
            at = start[:m] + t
            before.append(S[:m])
            S = _moved(S[:m], q[at], k[at], v[at], a[at], b[at])[0]
        for t in reversed(steps):
            m = alive[t]
            at = start[:m] + t
            old, qt, kt, at_, bt = before.pop(), q[at], k[at], a[at], b[at]
            new, u, _ = _moved(old, qt, kt, v[at], at_, bt)
            dot = do[at]
            dq[at] = torch.matmul(new, dot[..., None])[..., 0]
            D = torch.addcmul(E[:m], qt[..., :, None], dot[..., None, :])      # into the new state
            du = torch.matmul(kt[..., None, :], D)[..., 0, :]
            dr = bt[..., None] * du
            read = torch.matmul(kt[..., None, :], old)[..., 0, :]
            dv_[at] = dr
            db[at] = (du * (v[at] - at_[..., None] * read)).sum(-1)
            dk_[at] = (torch.matmul(D, u[..., None]) - at_[..., None, None]
                       * torch.matmul(old, dr[..., None]))[..., 0]
            da[at] = (D * old).sum((-1, -2)) - (dr * read).sum(-1)
            E[:m] = at_[..., None, None] * torch.addcmul(D, kt[..., :, None], dr[..., None, :], value=-1)
    rows = torch.zeros(len(v), dtype=torch.bool, device=v.device)
    if len(v):
        rows[:] = True if s["mask"] is None else s["mask"] != 0
    g = h // kh
    dq, dk_ = ((x * rows[:, None, None]).view(-1, kh, g, dk).sum(2) for x in (dq * dk ** -0.5, dk_))
    out.update(dq=dq, dk=dk_, dv=dv_, dgate=da * a * (1 - a) * rows[:, None],
               dbeta=db * b * (1 - b) * rows[:, None])
    if s["state"] is not None:
        out["dstate"] = E[back]
    return out
