"""Cases of the operators around a layer's aggregation: dropout from a
counter-based generator, the dense layer (product with bias, activation,
dropout and residual in its epilogue) with its gradients, and group norm with
an activation over the rows of each graph, with its gradients.

Formulas (T = round(65536 p), s = 65536 / (65536 - T), 0 for T = 65536):

  dropout   Out[r, j] = keep(r, j) ? s X[r, j] : 0  (+ addend[r, j]),
            keep(r, j) = u(r, j) >= T with u the 16-bit draw number j % 8 of
            the Philox4x32-10 block at counter (j / 8, node(r), call, 1), key
            (seed low, seed high): draw e is the low (e even) or high (e odd)
            half of word e / 2.
  dense     Z = X W + b;  Out = R + dropout(act(Z));  backward:
            dZ = act'(Z) dropout(G);  dX = dZ W^T;  dW = X^T dZ;  db = 1^T dZ.
  norm      per graph (rows seg[i] .. seg[i + 1] - 1) and group of adjacent
            columns: xhat = (x - mean) rstd, rstd = 1 / sqrt(var + eps);
            Out = act(xhat w + v);  backward with a = act'(xhat w + v) G:
            dw = sum a xhat, dv = sum a over all rows;  dX = rstd (h - mean(h)
            - xhat mean(h xhat)), h = a w, means over the group.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_ES = {"f32": 4, "bf16": 2}
_EPS = 1e-5
_SLOPE = 0.01


def listed():
    return [
        # the hidden rows of a small citation graph between two layers: launch latency
        {"name": "dropout_tiny_f32", "op": "dropout", "dtype": "f32", "n": 2708, "d": 16, "p": 0.5, "nodes": False, "addend": False},
        # a partition's halo rows, each under its global node id, odd width
        {"name": "dropout_halo_bf16", "op": "dropout", "dtype": "bf16", "n": 262144, "d": 602, "p": 0.1, "nodes": True, "addend": False},
        # a hidden layer of a 2.45M-node graph, added to the residual stream
        {"name": "dropout_large_bf16", "op": "dropout", "dtype": "bf16", "n": 2450000, "d": 256, "p": 0.5, "nodes": False, "addend": True},
        # first layer of a small citation graph: few rows, long odd sum, 16 columns
        {"name": "dense_fwd_tiny_f32", "op": "dense_fwd", "dtype": "f32", "m": 2708, "k": 1433, "n": 16, "act": "relu", "p": 0.5, "residual": False},
        # one query node's row through a wide layer
        {"name": "dense_fwd_row_bf16", "op": "dense_fwd", "dtype": "bf16", "m": 1, "k": 512, "n": 2048, "act": "silu", "p": 0.0, "residual": True},
        # hidden residual layer of a 2.45M-node graph in training
        {"name": "dense_fwd_large_bf16", "op": "dense_fwd", "dtype": "bf16", "m": 2450000, "k": 256, "n": 256, "act": "gelu", "p": 0.1, "residual": True},
        # the 233K-node graph's 602 features in fp32, backward
        {"name": "dense_bwd_odd_f32", "op": "dense_bwd", "dtype": "f32", "m": 232965, "k": 602, "n": 128, "act": "leaky_relu", "p": 0.5, "residual": False},
        # the same hidden residual layer, backward
        {"name": "dense_bwd_large_bf16", "op": "dense_bwd", "dtype": "bf16", "m": 2450000, "k": 256, "n": 256, "act": "gelu", "p": 0.1, "residual": True},
        # a batch of small graphs (about 25 nodes each), 8 groups
        {"name": "norm_fwd_batch_bf16", "op": "norm_fwd", "dtype": "bf16", "n": 102400, "c": 256, "groups": 8, "graphs": 4096, "act": "relu"},
        # one large graph, every channel on its own
        {"name": "norm_fwd_large_bf16", "op": "norm_fwd", "dtype": "bf16", "n": 2450000, "c": 256, "groups": 256, "graphs": 1, "act": "gelu"},
        # a batch of small graphs, backward, odd width, fp32
        {"name": "norm_bwd_batch_f32", "op": "norm_bwd", "dtype": "f32", "n": 30011, "c": 100, "groups": 10, "graphs": 1200, "act": "silu"},
        # one large graph as a whole, backward
        {"name": "norm_bwd_large_bf16", "op": "norm_bwd", "dtype": "bf16", "n": 2450000, "c": 256, "groups": 32, "graphs": 1, "act": "relu"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dropout", "dense_fwd", "dense_bwd", "norm_fwd", "norm_bwd"])
    dt = rng.choice(["f32", "bf16"])
    act = rng.choice(["none", "relu", "leaky_relu", "gelu", "silu"])
    p = rng.choice([0.0, 0.1, 0.3, 0.5, 0.6])
    most = 2450000 * 256 // (2 if dt == "f32" else 1)
    while True:
        rows = _log_int(rng, 1, 2450000)
        if op == "dropout":
            d = _log_int(rng, 1, 2048)
            if rows * d <= most:
                return {"op": op, "dtype": dt, "n": rows, "d": d, "p": p or 0.2, "nodes": rng.random() < 0.5, "addend": rng.random() < 0.5}
        elif op in ("dense_fwd", "dense_bwd"):
            k, n = _log_int(rng, 1, 2048), _log_int(rng, 1, 2048)
            if rows * max(k, n) <= most and rows * k * n <= most * (256 if dt == "bf16" else 128):
                return {"op": op, "dtype": dt, "m": rows, "k": k, "n": n, "act": act, "p": p, "residual": rng.random() < 0.5}
        else:
            c = _log_int(rng, 1, 1024 if dt == "f32" else 2048)
            groups = rng.choice([g for g in range(1, c + 1) if c % g == 0])
            graphs = rng.choice([1, _log_int(rng, 1, max(1, min(rows, 100000)))])
            # (statistics of eight values at least, on average)
            if rows * c <= most and rows * c >= 8 * groups * graphs:
                return {"op": op, "dtype": dt, "n": rows, "c": c, "groups": groups, "graphs": graphs, "act": act}


# ---- inputs ------------------------------------------------------------------------

def _pitched(rows, d, dtype):
    """[rows, d] view whose rows start on 16 bytes (128 where they are wider than 64)."""
    es = _ES[dtype]
    line = 128 if d * es > 64 else 16
    ld = (d * es + line - 1) // line * line // es
    return torch.zeros((rows, ld), dtype=_DT[dtype], device="cuda")[:, :d]


def _normal(rows, d, dtype, g, scale=1.0, shift=None):
    x = torch.randn((rows, d), generator=g, device="cuda")
    x *= scale
    if shift is not None:
        x += shift
    out = _pitched(rows, d, dtype)
    out.copy_(x)
    return out


def _drop_args(case, seed):
    return {"p": case["p"], "seed": 0x9E3779B97F4A7C15 ^ (seed * 0x100000001B3 % (1 << 63)), "call": seed % 1000}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op = case["dtype"], case["op"]
    s = {"case": dict(case)}
    if op == "dropout":
        n, d = case["n"], case["d"]
        s["x"] = _normal(n, d, dt, g)
        s["add"] = _normal(n, d, dt, g) if case["addend"] else None
        s["nodes"] = torch.randint(0, 1 << 31, (n,), generator=g, device="cuda", dtype=torch.int32) if case["nodes"] else None
        s["out"] = _pitched(n, d, dt)
        s["drop"] = _drop_args(case, seed)
    elif op in ("dense_fwd", "dense_bwd"):
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _normal(m, k, dt, g)
        s["w"] = (torch.randn((k, n), generator=g, device="cuda") * math.sqrt(2.0 / (k + n))).to(_DT[dt])
        s["b"] = torch.rand(n, generator=g, device="cuda") * 0.2 - 0.1
        s["drop"] = _drop_args(case, seed)
        if op == "dense_fwd":
            s["res"] = _normal(m, n, dt, g) if case["residual"] else None
            s["out"] = _pitched(m, n, dt)
            s["z_out"] = _pitched(m, n, dt) if case["act"] != "none" else None
        else:
            s["z"] = _normal(m, n, dt, g, 0.8) if case["act"] != "none" else None
            s["g"] = _normal(m, n, dt, g, 0.05)
            s["dx"] = _pitched(m, k, dt)
    else:
        n, c, graphs = case["n"], case["c"], case["graphs"]
        shift = torch.randn(c, generator=g, device="cuda") * 0.5 + 0.3
        s["x"] = _normal(n, c, dt, g, 1.3, shift)
        s["w"] = torch.rand(c, generator=g, device="cuda") + 0.5
        s["v"] = torch.randn(c, generator=g, device="cuda") * 0.2
        cuts = torch.randint(0, n + 1, (graphs - 1,), generator=g, device="cuda", dtype=torch.int64).sort().values
        s["seg"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts,
                              torch.full((1,), n, dtype=torch.int64, device="cuda")])
        s["out"] = _pitched(n, c, dt)
        if op == "norm_bwd":
            s["g"] = _normal(n, c, dt, g, 0.05)
            s["mean"], s["rstd"] = _norm_stats(s["x"], s["seg"], case["groups"])
    return s


# ---- plain forms --------------------------------------------------------------------

def _keep(rows, d, drop, nodes, device):
    """keep(r, j) as truth values and the scale s, by Philox4x32-10 in 64-bit whole numbers."""
    T = int(math.floor(drop["p"] * 65536 + 0.5))
    if T == 65536:
        return torch.zeros((rows, d), dtype=torch.bool, device=device), 0.0
    m32 = 0xFFFFFFFF
    nb = (d + 7) // 8
    ids = nodes.to(torch.int64) & m32 if nodes is not None else torch.arange(rows, device=device)
    c0 = torch.arange(nb, device=device)[None, :].expand(rows, nb)
    c1 = ids[:, None].expand(rows, nb)
    c2 = torch.full((1, 1), drop["call"], dtype=torch.int64, device=device).expand(rows, nb)
    c3 = torch.ones((1, 1), dtype=torch.int64, device=device).expand(rows, nb)
    k0, k1 = drop["seed"] & m32, drop["seed"] >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32, ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    u = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], -1)
    return (u >= T).reshape(rows, nb * 8)[:, :d], 65536.0 / (65536 - T)


def _drop(x, drop, nodes=None):
    if drop["p"] == 0.0:
        return x
    keep, s = _keep(x.shape[0], x.shape[1], drop, nodes, x.device)
    return torch.where(keep, x * s, torch.zeros((), dtype=x.dtype, device=x.device))


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "leaky_relu":
        return torch.where(z > 0, z, z * _SLOPE)
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "leaky_relu":
        return torch.where(z > 0, torch.ones_like(z), torch.full_like(z, _SLOPE))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "silu":
        e = 1.0 / (1.0 + torch.exp(-z))
        return e * (1.0 + z * (1.0 - e))
    return torch.ones_like(z)


def _seg_of_rows(seg, n):
    return torch.searchsorted(seg[1:].contiguous(), torch.arange(n, device=seg.device), right=True)


def _seg_sums(v, seg):
    """Sums of v's rows (float64) over each graph: differences of running sums."""
    run_ = torch.cumsum(v.t().contiguous(), 1)
    run_ = torch.cat([torch.zeros_like(run_[:, :1]), run_], 1)
    return (run_[:, seg[1:]] - run_[:, seg[:-1]]).t()


def _group_sums(v, groups):
    return v.reshape(v.shape[0], groups, -1).sum(-1, dtype=torch.float64)


def _norm_stats(x, seg, groups):
    n, c = x.shape
    cnt = ((seg[1:] - seg[:-1]) * (c // groups)).to(torch.float64).clamp(min=1)[:, None]
    xf = x.float()
    mean = _seg_sums(_group_sums(xf, groups), seg) / cnt
    of = _seg_of_rows(seg, n)
    cen = xf.reshape(n, groups, -1) - mean.float()[of][:, :, None]
    # (about the rounded mean; the rounding's own part of the spread taken back)
    var = _seg_sums((cen * cen).sum(-1, dtype=torch.float64), seg) / cnt - (mean - mean.float().double()) ** 2
    return mean.float(), (1.0 / torch.sqrt(var.clamp(min=0) + _EPS)).float()


def _like(x, buf):
    """x rounded once into rows of buf's pitch."""
    out = torch.empty_strided(buf.shape, buf.stride(), dtype=buf.dtype, device=buf.device)
    out.copy_(x)
    return out


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        y = _drop(s["x"].float(), s["drop"], s["nodes"])
        if s["add"] is not None:
            y = y + s["add"].float()
        return {"out": _like(y, s["out"])}
    if op == "dense_fwd":
        z = torch.matmul(s["x"].float(), s["w"].float()) + s["b"]
        y = _drop(_act(z, c["act"]), s["drop"])
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"out": _like(y, s["out"]), "z": _like(z, s["z_out"]) if s["z_out"] is not None else None}
    if op == "dense_bwd":
        dz = _drop(s["g"].float(), s["drop"])
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"].float(), c["act"])
        return {"dw": torch.matmul(s["x"].float().t(), dz), "db": dz.sum(0),
                "dx": _like(torch.matmul(dz, s["w"].float().t()), s["dx"])}
    n, ch, groups, seg = c["n"], c["c"], c["groups"], s["seg"]
    xf = s["x"].float()
    of = _seg_of_rows(seg, n)
    mean, rstd = _norm_stats(s["x"], seg, groups) if op == "norm_fwd" else (s["mean"], s["rstd"])
    xhat = ((xf.reshape(n, groups, -1) - mean[of][:, :, None]) * rstd[of][:, :, None]).reshape(n, ch)
    if op == "norm_fwd":
        return {"out": _like(_act(xhat * s["w"] + s["v"], c["act"]), s["out"]), "mean": mean, "rstd": rstd}
    # (the sign of z decides a step of the gradient: z in 64 bits for it)
    if c["act"] in ("relu", "leaky_relu"):
        z = ((xf.double().reshape(n, groups, -1) - mean[of][:, :, None]) * rstd[of][:, :, None]).reshape(n, ch) * s["w"] + s["v"]
    else:
        z = xhat * s["w"] + s["v"]
    a = _act_grad(z, c["act"]).float() * s["g"].float()
    ah = a * xhat
    h = a * s["w"]
    cnt = ((seg[1:] - seg[:-1]) * (ch // groups)).to(torch.float64).clamp(min=1)[:, None]
    m1 = (_seg_sums(_group_sums(h, groups), seg) / cnt).float()[of][:, :, None]
    m2 = (_seg_sums(_group_sums(h * xhat, groups), seg) / cnt).float()[of][:, :, None]
    h3, x3 = h.reshape(n, groups, -1), xhat.reshape(n, groups, -1)
    dx = ((h3 - m1 - x3 * m2) * rstd[of][:, :, None]).reshape(n, ch)
    return {"dw": ah.sum(0, dtype=torch.float64).float(), "dv": a.sum(0, dtype=torch.float64).float(), "dx": _like(dx, s["out"])}


# ---- the framework's calls ------------------------------------------------------------

def _own(s):
    import sparse_aggregation_gemm_amd as sag
    c = s["case"]
    op = c["op"]
    if op == "dropout":
        drop = sag.Drop(nodes=s["nodes"], **s["drop"])
        return {"out": sag.dropout(s["x"], drop, addend=s["add"], Out=s["out"])}
    if op == "dense_fwd":
        out, z, _ = sag.dense_layer_forward(s["x"], s["w"], s["b"], act=c["act"], slope=_SLOPE, drop=sag.Drop(**s["drop"]),
                                            residual=s["res"], want_z=s["z_out"] is not None, Out=s["out"], Z=s["z_out"])
        return {"out": out, "z": z}
    if op == "dense_bwd":
        ctx = sag.DenseCtx(s["x"], s["w"], c["act"], _SLOPE, sag.Drop(**s["drop"]))
        dw, db, dx = sag.dense_layer_backward(ctx, s["z"], s["g"], dX=s["dx"])
        return {"dw": dw, "db": db, "dx": dx}
    if op == "norm_fwd":
        out, ctx = sag.group_norm_forward(s["x"], c["groups"], s["w"], s["v"], seg=s["seg"], eps=_EPS, act=c["act"],
                                          slope=_SLOPE, Out=s["out"])
        return {"out": out, "mean": ctx.mean, "rstd": ctx.rstd}
    ctx = sag.GroupNormCtx(s["x"], c["groups"], s["w"], s["v"], s["seg"], s["mean"], s["rstd"], c["act"], _SLOPE)
    dw, dv, dx = sag.group_norm_backward(ctx, s["g"], dX=s["out"])
    return {"dw": dw, "dv": dv, "dx": dx}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def work(case):
    es, op = _ES[case["dtype"]], case["op"]
    if op == "dropout":
        e = case["n"] * case["d"]
        return {"bytes": es * e * (3 if case["addend"] else 2) + (4 * case["n"] if case["nodes"] else 0), "flops": e}
    if op in ("dense_fwd", "dense_bwd"):
        m, k, n = case["m"], case["k"], case["n"]
        z = 0 if case["act"] == "none" else 1
        if op == "dense_fwd":
            return {"bytes": es * (m * k + k * n + m * n * (1 + z + (1 if case["residual"] else 0))) + 4 * n, "flops": 2 * m * k * n}
        return {"bytes": es * (2 * m * k + k * n + m * n * (1 + z)) + 4 * (k * n + n), "flops": 4 * m * k * n}
    e, g = case["n"] * case["c"], case["graphs"]
    stats = 8 * g * case["groups"] + 8 * (g + 1)
    if op == "norm_fwd":
        return {"bytes": 2 * es * e + stats + 8 * case["c"], "flops": 10 * e}
    return {"bytes": 3 * es * e + stats + 16 * case["c"], "flops": 20 * e}


# ---- the definition in 64 bits ----------------------------------------------------------

def _mul_hi_lo(a, b):
    """High and low words of the 32 x 32-bit product, by 16-bit halves."""
    al, ah, bl, bh = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    low, mid1, mid2 = al * bl, ah * bl, al * bh
    mid = (low >> 16) + (mid1 & 0xFFFF) + (mid2 & 0xFFFF)
    return ah * bh + (mid1 >> 16) + (mid2 >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _exact_factor(rows, d, drop, nodes):
    """The factor (0 or s) of each element, in float64; one draw per element."""
    T = np.floor(np.float64(drop["p"]) * 65536.0 + 0.5)
    if T == 0:
        return 1.0
    j = torch.arange(d, device="cuda")
    r = torch.arange(rows, device="cuda") if nodes is None else nodes.long() % (1 << 32)
    block = j.div(8, rounding_mode="floor").unique()
    x = [block.repeat(rows, 1), r[:, None].repeat(1, block.numel()), torch.full((rows, block.numel()), drop["call"], device="cuda"),
         torch.full((rows, block.numel()), 1, device="cuda")]
    key = [drop["seed"] % (1 << 32), drop["seed"] // (1 << 32)]
    for i in range(10):
        hi0, lo0 = _mul_hi_lo(x[0], 0xD2511F53)
        hi1, lo1 = _mul_hi_lo(x[2], 0xCD9E8D57)
        x = [hi1 ^ x[1] ^ ((key[0] + i * 0x9E3779B9) % (1 << 32)), lo1, hi0 ^ x[3] ^ ((key[1] + i * 0xBB67AE85) % (1 << 32)), lo0]
    out = torch.zeros((rows, d), dtype=torch.float64, device="cuda")
    for e in range(min(8, d)):
        cols = j[e::8]
        u = (x[e // 2][:, :cols.numel()] >> (16 * (e % 2))) % 65536
        out[:, e::8] = (u.double() >= T).double() * (65536.0 / (65536.0 - T) if T < 65536 else 0.0)
    return out


def _exact_act(z, act):
    """(act(z), act'(z)) in float64."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "leaky_relu":
        f = 1.0 + (_SLOPE - 1.0) * (z <= 0).double()
        return z * f, f
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    return z, torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dropout":
        y = s["x"].double() * _exact_factor(case["n"], case["d"], s["drop"], s["nodes"])
        return {"out": y if s["add"] is None else y + s["add"].double()}
    if op in ("dense_fwd", "dense_bwd"):
        f = _exact_factor(case["m"], case["n"], s["drop"], None)
        x, w = s["x"].double(), s["w"].double()
        if op == "dense_fwd":
            z = torch.addmm(s["b"].double(), x, w)
            y = _exact_act(z, case["act"])[0] * f
            if s["res"] is not None:
                y += s["res"].double()
            return {"out": y, "z": z if s["z_out"] is not None else None}
        dz = s["g"].double() * f
        if s["z"] is not None:
            dz *= _exact_act(s["z"].double(), case["act"])[1]
        return {"dw": x.t() @ dz, "db": dz.sum(0), "dx": dz @ w.t()}
    n, c, q = case["n"], case["c"], case["groups"]
    d = c // q
    lens = s["seg"].diff()
    of = torch.arange(lens.numel(), device="cuda").repeat_interleave(lens)

    def per_graph(v):          # [n, c] -> means [graphs, q]
        if lens.numel() == 1:
            t = v.reshape(n, q, d).sum((0, 2))[None]
        else:
            t = torch.zeros((lens.numel(), q), dtype=torch.float64, device="cuda").index_add_(0, of, v.reshape(n, q, d).sum(2))
        return t / (lens * d).clamp(min=1)[:, None]

    def spread(t):             # [graphs, q] -> [n, c]
        return t[of].repeat_interleave(d, 1)

    x = s["x"].double()
    w, v = s["w"].double(), s["v"].double()
    if op == "norm_fwd":
        mean = per_graph(x)
        x -= spread(mean)
        rstd = (per_graph(x * x) + _EPS).rsqrt()
        return {"out": _exact_act(x * spread(rstd) * w + v, case["act"])[0], "mean": mean, "rstd": rstd}
    rstd = spread(s["rstd"].double())
    xhat = (x - spread(s["mean"].double())) * rstd
    a = _exact_act(xhat * w + v, case["act"])[1] * s["g"].double()
    h = a * w
    dx = rstd * (h - spread(per_graph(h)) - xhat * spread(per_graph(h * xhat)))
    return {"dw": (a * xhat).sum(0), "dv": a.sum(0), "dx": dx}
