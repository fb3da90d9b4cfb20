"""Dropout, the dense layer and group norm on the GPU against the float64
oracle on the same stored inputs.

Bounds.  u = 2^-24 (half a step of fp32) and ut = finfo(dtype).eps / 2 for the
one rounding of an output.  An activation or its derivative is taken to cost
16 u of its argument's size (and the GELU of a bf16 result what fit() says), a sum of n terms n u of the sum of their sizes (whatever
the order).  These are worst cases; the exact-integer tests below leave no room."""
import numpy as np
import pytest
import torch

import gen
from oracle import block as ob, layers as olay

pytestmark = pytest.mark.gpu

sag = pytest.importorskip("sparse_aggregation_gemm_amd")
from gpu_util import DEV, bits16, f64, say, to_dev, to_dev_dense  # noqa: E402

U = 2.0 ** -24
TD = {"f32": torch.float32, "bf16": torch.bfloat16}
UT = {k: torch.finfo(v).eps / 2 for k, v in TD.items()}
LIP = 1.13                       # largest slope of any of the activations


def fit(kind, dt, z):
    """What GELU's tail costs where the result is rounded to bf16: z Phi(z) is
    max(z, 0) - |z| (1 - Phi(|z|)), and the five-term fit of the second factor
    is off by 3.1e-5 of it at most (its polynomial against log_ndtr in 64 bits
    on [0, 14]: 3.110e-5); at most 5.3e-6, where half a step of bf16 at 1 is 3.9e-3."""
    return 3.2e-5 * np.abs(z) * torch.special.ndtr(torch.from_numpy(-np.abs(z))).numpy() if kind == "gelu" and dt == "bf16" else 0.0


def mat(g, rows, d, dt, integers=False, scale=1.0):
    x = g.integers(-4, 5, (rows, d)).astype(np.float32) if integers else (scale * g.standard_normal((rows, d))).astype(np.float32)
    return to_dev_dense(gen.f32_to_bf16_bits(x) if dt == "bf16" else x, dt)


def within(got, ref, tol):
    err = np.abs(f64(got) - ref) - tol
    assert np.all(np.isfinite(f64(got))), "not finite"
    assert err.size == 0 or err.max() <= 0, f"over the bound by {err.max():.3e} at {np.unravel_index(err.argmax(), err.shape)}"


def raw(t):
    """The bits of a result, to compare two runs."""
    return bits16(t) if t.dtype == torch.bfloat16 else t.detach().contiguous().cpu().view(torch.int32).numpy()


# ---- dropout ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", [(1, 1), (1, 8), (3, 7), (300, 16), (77, 100), (129, 602), (5, 4099), (2, 20000), (1025, 9)])
@pytest.mark.parametrize("p,nodes,add", [(0.5, False, False), (0.1, True, True), (0.9, False, True)])
def test_dropout(dt, n, d, p, nodes, add):
    say(f"dropout {dt} {n}x{d} p={p} nodes={nodes} add={add}")
    g = np.random.default_rng(n * 31 + d)
    X = mat(g, n, d, dt)
    A = mat(g, n, d, dt) if add else None
    ids = g.integers(-2 ** 31, 2 ** 31, n).astype(np.int32) if nodes else None
    seed, call = int(g.integers(0, 2 ** 63)), 5
    f = ob.drop_factor(n, d, p, seed, call, ids, 40)
    out = sag.dropout(X, sag.Drop(p, seed, call, to_dev(ids) if nodes else None, 40), addend=A)
    ref = ob.drop(f64(X), f)
    tol = U * np.abs(ref)
    if add:
        ref = ref + f64(A)
        tol = tol + U * np.abs(ref)
    within(out, ref, tol * 1.01 + UT[dt] * np.abs(ref))
    if not add:
        assert np.array_equal(f64(out) == 0, (f == 0) | (f64(X) == 0))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dropout_ends_of_p_and_special_values(dt):
    say(f"dropout ends {dt}")
    g = np.random.default_rng(2)
    X = mat(g, 50, 33, dt)
    X[3, 5], X[4, 6], X[5, 7] = float("nan"), float("inf"), -float("inf")
    assert np.array_equal(raw(sag.dropout(X, sag.Drop(0.0, 1))), raw(X))
    assert not raw(sag.dropout(X, sag.Drop(1.0, 1))).any()
    assert np.array_equal(raw(sag.dropout(X, sag.Drop(2.0 ** -18, 1))), raw(X))     # rounds to 0
    for seed in range(6):
        f = ob.drop_factor(50, 33, 0.5, seed)
        y = f64(sag.dropout(X, sag.Drop(0.5, seed)))
        assert np.isnan(y[3, 5]) == (f[3, 5] > 0) and np.isinf(y[4, 6]) == (f[4, 6] > 0)
        assert np.isinf(y[5, 7]) == (f[5, 7] > 0) and np.isfinite(y).sum() >= y.size - 3
    assert sag.dropout(X[:0], sag.Drop(0.5, 1)).shape == (0, 33)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dropout_in_place_strides_and_rows_outside(dt):
    """Out = X, Out = addend, an operand of another pitch, and rows around the
    view that stay as they were."""
    say(f"dropout in place {dt}")
    g = np.random.default_rng(3)
    drop = sag.Drop(0.4, 11, 2)
    big = mat(g, 60, 72, dt)
    X = big[10:40, :44]                      # a wider pitch, rows and columns outside
    ref = sag.dropout(mat_copy(X), drop)
    keep = raw(big).copy()
    sag.dropout(X, drop, Out=X)
    assert np.array_equal(raw(X), raw(ref))
    after = raw(big)
    after[10:40, :44] = keep[10:40, :44]
    assert np.array_equal(after, keep)
    A = mat(g, 30, 44, dt)
    ref = sag.dropout(X, drop, addend=A)
    sag.dropout(X, drop, addend=A, Out=A)
    assert np.array_equal(raw(A), raw(ref))


def mat_copy(t):
    out = sag.empty_dense(t.shape[0], t.shape[1], t.dtype, t.device)
    out.copy_(t)
    return out


def test_dropout_of_a_partition_is_the_whole_graphs():
    """With node ids for stream ids a partition's rows get the masks they have
    in the whole graph, in either type and at any pitch."""
    say("dropout partition")
    g = np.random.default_rng(4)
    X = mat(g, 200, 50, "f32")
    whole = f64(sag.dropout(X, sag.Drop(0.5, 77, 1)))
    ids = g.permutation(200)[:60].astype(np.int32)
    part = f64(sag.dropout(mat_copy(X[torch.from_numpy(ids).long().to(DEV)]), sag.Drop(0.5, 77, 1, nodes=to_dev(ids))))
    assert np.array_equal(part, whole[ids])
    assert np.array_equal(f64(sag.dropout(mat_copy(X[120:]), sag.Drop(0.5, 77, 1, row0=120))), whole[120:])
    ones = mat_copy(torch.ones_like(X[:, :50], dtype=torch.bfloat16))
    assert np.array_equal(f64(sag.dropout(ones, sag.Drop(0.5, 77, 1))) > 0, ob.drop_factor(200, 50, 0.5, 77, 1) > 0)


# ---- dense layer --------------------------------------------------------------------------

SIZES = [(1, 1, 1), (3, 7, 5), (129, 100, 47), (128, 64, 128), (257, 602, 130), (700, 256, 256), (33, 1433, 16),
         (2, 130, 300), (1, 512, 2048), (511, 65, 64), (64, 2100, 72), (300, 31, 1025)]


def dense_case(dt, M, K, N, kind, p, res, bias=True, seed=0):
    g = np.random.default_rng(M * 7 + K * 3 + N + seed)
    X = mat(g, M, K, dt)
    W = mat(g, K, N, dt, scale=float(np.sqrt(1.0 / K))).contiguous()
    b = to_dev(g.uniform(-0.5, 0.5, N).astype(np.float32)) if bias else None
    R = mat(g, M, N, dt) if res else None
    drop = sag.Drop(p, int(g.integers(0, 2 ** 63)), 9) if p is not None else None
    f = ob.drop_factor(M, N, p, drop.seed, 9) if drop else np.ones((M, N))
    return g, X, W, b, R, drop, f


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("kind,p,res", [("gelu", 0.1, True), ("relu", None, False), ("silu", 0.5, False), ("none", 0.3, True),
                                        ("leaky_relu", None, True)])
def test_dense_forward(dt, M, K, N, kind, p, res):
    say(f"dense forward {dt} M={M} K={K} N={N} {kind} p={p} res={res}")
    _, X, W, b, R, drop, f = dense_case(dt, M, K, N, kind, p, res)
    out, z, _ = sag.dense_layer_forward(X, W, b, act=kind, slope=0.1, drop=drop, residual=R, want_z=True)
    x, w, bb = f64(X), f64(W), f64(b)
    Z, Out = ob.dense_forward(x, w, bb, kind, 0.1, f, f64(R) if res else None)
    ez = (K + 1) * U * (np.abs(x) @ np.abs(w) + np.abs(bb))
    within(z, Z, ez + UT[dt] * np.abs(Z) + 1e-30)
    eo = f * (LIP * ez + 16 * U * np.abs(Z) + fit(kind, dt, Z)) + 3 * U * np.abs(f * Z) + U * np.abs(Out)
    within(out, Out, eo + UT[dt] * (np.abs(Out) + eo) + 1e-30)
    # the same call again, without Z: the same bits
    out2, z2, _ = sag.dense_layer_forward(X, W, b, act=kind, slope=0.1, drop=drop, residual=R, want_z=False)
    assert z2 is None and np.array_equal(raw(out2), raw(out))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", SIZES + [(2049, 64, 96)])
@pytest.mark.parametrize("kind,p", [("gelu", 0.1), ("relu", 0.5), ("silu", None), ("none", None), ("leaky_relu", 0.3)])
def test_dense_backward(dt, M, K, N, kind, p):
    say(f"dense backward {dt} M={M} K={K} N={N} {kind} p={p}")
    g, X, W, _, _, drop, f = dense_case(dt, M, K, N, kind, p, False, seed=1)
    Z = mat(g, M, N, dt)
    G = mat(g, M, N, dt)
    if M > 2:
        Z[1, 0] = 0.0                              # the step of ReLU
    dW, db, dX = sag.dense_layer_backward(sag.DenseCtx(X, W, kind, 0.1, drop), Z if kind != "none" else None, G)
    x, w, z, gg = f64(X), f64(W), f64(Z), f64(G)
    dZ, rW, rb, rX = ob.dense_backward(x, w, z, kind, 0.1, f, gg)
    ez = np.abs(gg) * f * (16 * U * (1 + np.abs(z)) if kind in ("gelu", "silu") else 0) + 3 * U * np.abs(dZ)
    # dZ in the weight gradient's products: three bf16 parts, (2^-8)^3, or two from 2^15 rows on; exact without rounding
    keep = 0.0 if dt == "f32" or kind in ("none", "relu") else (2.0 ** -24 if M < 2 ** 15 else 2.0 ** -16)
    within(dX, rX, ((ez + (UT[dt] if dt == "bf16" else 0) * np.abs(dZ)) @ np.abs(w).T + N * U * np.abs(dZ) @ np.abs(w).T) * 1.01
           + UT[dt] * np.abs(rX) * 1.01 + 1e-30)
    within(dW, rW, np.abs(x).T @ (ez + keep * np.abs(dZ)) + (M + 2) * U * np.abs(x).T @ np.abs(dZ) + 1e-30)
    within(db, rb, (ez + keep * np.abs(dZ)).sum(0) + (M + 2) * U * np.abs(dZ).sum(0) + 1e-30)
    again = sag.dense_layer_backward(sag.DenseCtx(X, W, kind, 0.1, drop), Z if kind != "none" else None, G, want_dX=False)
    assert again[2] is None and np.array_equal(raw(again[0]), raw(dW)) and np.array_equal(raw(again[1]), raw(db))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", [(1, 64, 128), (97, 130, 47), (600, 256, 256), (4100, 100, 72), (130, 700, 300)])
def test_dense_exact_integers(dt, M, K, N):
    """Small whole numbers, p = 0.5 (scale 2): every sum is exact in fp32, so
    each output is the exact value rounded once."""
    say(f"dense integers {dt} M={M} K={K} N={N}")
    g = np.random.default_rng(M + K + N)
    X, W, R, G = mat(g, M, K, dt, True), mat(g, K, N, dt, True).contiguous(), mat(g, M, N, dt, True), mat(g, M, N, dt, True)
    b = to_dev(g.integers(-3, 4, N).astype(np.float32))
    drop = sag.Drop(0.5, 21, 3)
    f = ob.drop_factor(M, N, 0.5, 21, 3)
    out, z, ctx = sag.dense_layer_forward(X, W, b, act="relu", drop=drop, residual=R)
    rnd = olay.round_bf16 if dt == "bf16" else (lambda v: v)
    Z, Out = ob.dense_forward(f64(X), f64(W), f64(b), "relu", 0.0, f, f64(R))
    assert np.array_equal(f64(z), rnd(Z)) and np.array_equal(f64(out), rnd(Out))
    dW, db, dX = sag.dense_layer_backward(ctx, z, G)
    _, rW, rb, rX = ob.dense_backward(f64(X), f64(W), f64(z), "relu", 0.0, f, f64(G))
    assert np.array_equal(f64(dW), rW) and np.array_equal(f64(db), rb) and np.array_equal(f64(dX), rnd(rX))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dense_pitches_in_place_and_garbage_padding(dt):
    """Operands of different pitches whose padding holds NaN, Out written over
    the residual, and rows outside a view left alone."""
    say(f"dense pitches {dt}")
    g = np.random.default_rng(6)
    M, K, N = 150, 45, 52
    nan = float("nan")

    def holed(rows, d, pitch):
        buf = torch.full((rows + 4, pitch), nan, dtype=TD[dt], device=DEV)
        buf[2:2 + rows, :d] = torch.from_numpy(g.standard_normal((rows, d)).astype(np.float32)).to(DEV).to(TD[dt])
        return buf, buf[2:2 + rows, :d]

    _, X = holed(M, K, 48)
    rb, R = holed(M, N, 88)
    zb, Z = holed(M, N, 56)
    W = mat(g, K, N, dt).contiguous()
    drop = sag.Drop(0.25, 5)
    ref, zr, ctx = sag.dense_layer_forward(mat_copy(X), W, None, act="gelu", drop=drop, residual=mat_copy(R))
    sag.dense_layer_forward(X, W, None, act="gelu", drop=drop, residual=R, Out=R, Z=Z)
    assert np.array_equal(raw(R), raw(ref)) and np.array_equal(raw(Z), raw(zr))
    for buf, d in ((rb, N), (zb, N)):
        assert torch.isnan(buf[:2]).all() and torch.isnan(buf[-2:]).all() and torch.isnan(buf[:, d:]).all()
    db_, D = holed(M, K, 56)
    _, Gv = holed(M, N, 64)
    want = sag.dense_layer_backward(ctx, zr, mat_copy(Gv))
    got = sag.dense_layer_backward(sag.DenseCtx(X, W, "gelu", 0.01, drop), Z, Gv, dX=D)
    for a, b in zip(got, want):
        assert np.array_equal(raw(a), raw(b))
    assert torch.isnan(db_[:2]).all() and torch.isnan(db_[-2:]).all() and torch.isnan(db_[:, K:]).all()


def test_dense_no_rows():
    say("dense no rows")
    X, W = sag.empty_dense(0, 40, torch.float32, DEV), torch.ones(40, 24, device=DEV)
    out, z, ctx = sag.dense_layer_forward(X, W, act="silu")
    assert out.shape == (0, 24) and z.shape == (0, 24)
    dW, db, dX = sag.dense_layer_backward(ctx, z, out)
    assert dX.shape == (0, 40) and not dW.any() and not db.any()


@pytest.mark.parametrize("kind", ["gelu", "silu", "leaky_relu"])
def test_dense_gradient_by_differences(kind):
    """The gradients against central differences of the forward pass in fp32:
    the loss sum(G Out) along one random direction of each operand.  Step
    h = 2^-7: the difference's own error is h^2 / 6 of the third derivative
    (below 1e-4 of the sums) and 2^-23 |loss| / h."""
    say(f"dense differences {kind}")
    g = np.random.default_rng(8)
    M, K, N = 40, 30, 20
    X, W, G = mat(g, M, K, "f32"), mat(g, K, N, "f32", scale=0.2).contiguous(), mat(g, M, N, "f32")
    b = to_dev(g.standard_normal(N).astype(np.float32))
    drop = sag.Drop(0.3, 4)

    def loss(x, w, bb):
        return float((f64(sag.dense_layer_forward(x, w, bb, act=kind, slope=0.2, drop=drop)[0]) * f64(G)).sum())

    _, z, ctx = sag.dense_layer_forward(X, W, b, act=kind, slope=0.2, drop=drop)
    dW, db, dX = sag.dense_layer_backward(ctx, z, G)
    h = 2.0 ** -7 if kind != "leaky_relu" else 2.0 ** -13
    size = float(np.abs(f64(dX)).sum())
    for i, grad in ((0, dX), (1, dW), (2, db)):
        args = [X, W, b]
        v = torch.from_numpy(g.choice([-1.0, 1.0], tuple(grad.shape)).astype(np.float32)).to(DEV) / grad.numel() ** 0.5
        def at(s):
            a = list(args)
            a[i] = mat_copy(a[i] + s * v) if i != 1 and a[i].dim() == 2 else (a[i] + s * v).contiguous()
            return loss(*a)
        num = (at(h) - at(-h)) / (2 * h)
        want = float((f64(grad) * f64(v)).sum())
        assert abs(num - want) < 2e-3 * size / 10


# ---- group norm ---------------------------------------------------------------------------

def norm_case(dt, n, d, groups, seg, seed=0, offset=2.0):
    g = np.random.default_rng(n * 13 + d * 5 + groups + seed)
    x = (g.standard_normal((n, d)) * g.uniform(0.5, 2.0, d) + offset * g.standard_normal(d)).astype(np.float32)
    X = to_dev_dense(gen.f32_to_bf16_bits(x) if dt == "bf16" else x, dt)
    w = g.uniform(0.5, 1.5, d).astype(np.float32)
    b = g.standard_normal(d).astype(np.float32)
    return g, X, to_dev(w), to_dev(b), None if seg is None else to_dev(np.asarray(seg, np.int64))


def cuts(n, graphs, seed):
    g = np.random.default_rng(seed)
    return [0] + sorted(g.integers(0, n + 1, graphs - 1).tolist()) + [n]


NORMS = [(1, 1, 1, None), (1, 8, 2, None), (7, 3, 3, None), (300, 256, 8, None), (1000, 100, 10, None), (5000, 64, 64, None),
         (40, 2048, 1, None), (333, 602, 7, cuts(333, 20, 1)), (2000, 128, 1, cuts(2000, 300, 2)), (64, 96, 96, [0, 0, 10, 10, 10, 64]),
         (500, 24, 4, [5, 6, 7, 200, 200, 470]), (12, 16, 2, [3, 3, 3]), (9000, 32, 32, cuts(9000, 7, 3)), (257, 1024, 16, cuts(257, 257, 4))]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,groups,seg", NORMS)
@pytest.mark.parametrize("kind", ["none", "relu", "gelu"])
def test_norm_forward(dt, n, d, groups, seg, kind):
    if dt == "f32" and d > 1024:                    # refused: fp32 rows end at 1024
        with pytest.raises(sag._lib.SagError, match="1024"):
            sag.group_norm_forward(mat(np.random.default_rng(0), n, d, dt), groups)
        return
    say(f"norm forward {dt} n={n} d={d} groups={groups} graphs={1 if seg is None else len(seg) - 1} {kind}")
    _, X, w, b, sd = norm_case(dt, n, d, groups, seg)
    seg_h = [0, n] if seg is None else seg
    base = sag.empty_dense(n, d, TD[dt], DEV, fill=7.0)
    out, ctx = sag.group_norm_forward(X, groups, w, b, seg=sd, eps=1e-3, act=kind, Out=base)
    x = f64(X)
    mean, rstd = ob.norm_stats(x, groups, seg_h, 1e-3)
    # statistics: pairwise sums of few terms each; 64 u of the values' size
    big = np.abs(x).max() if x.size else 1.0
    within(ctx.mean, mean, 64 * U * big)
    # var: relative 64 u, and the mean's own error squared is far below it
    within(ctx.rstd, rstd, 64 * U * rstd)
    m32, r32 = f64(ctx.mean), f64(ctx.rstd)
    ref = ob.norm_forward(x, groups, seg_h, f64(w), f64(b), kind, 0.01, m32, r32, np.full((n, d), 7.0))
    D = d // groups
    tol = np.zeros((n, d))
    for i in range(len(seg_h) - 1):
        r = slice(seg_h[i], seg_h[i + 1])
        xw = np.abs((x[r] - np.repeat(m32[i], D)) * np.repeat(r32[i], D) * f64(w))
        z = (x[r] - np.repeat(m32[i], D)) * np.repeat(r32[i], D) * f64(w) + f64(b)
        tol[r] = LIP * 5 * U * (xw + np.abs(f64(b))) + 16 * U * (xw + np.abs(f64(b))) + fit(kind, dt, z)
    within(out, ref, tol * 1.01 + UT[dt] * np.abs(ref))
    # rows of no graph were left as they were
    own = np.zeros(n, bool)
    for i in range(len(seg_h) - 1):
        own[seg_h[i]:seg_h[i + 1]] = True
    assert np.all(f64(out)[~own] == 7.0)
    # in place: the same bits
    Y = mat_copy(X)
    sag.group_norm_forward(Y, groups, w, b, seg=sd, eps=1e-3, act=kind, Out=Y)
    assert np.array_equal(raw(Y)[own], raw(out)[own]) and np.array_equal(raw(Y)[~own], raw(X)[~own])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,groups,seg", NORMS)
@pytest.mark.parametrize("kind", ["none", "relu", "silu", "leaky_relu"])
def test_norm_backward(dt, n, d, groups, seg, kind):
    if dt == "f32" and d > 1024:                    # refused: fp32 rows end at 1024
        with pytest.raises(sag._lib.SagError, match="1024"):
            sag.group_norm_forward(mat(np.random.default_rng(0), n, d, dt), groups)
        return
    say(f"norm backward {dt} n={n} d={d} groups={groups} graphs={1 if seg is None else len(seg) - 1} {kind}")
    g, X, w, b, sd = norm_case(dt, n, d, groups, seg, 1)
    seg_h = [0, n] if seg is None else seg
    G = mat(g, n, d, dt)
    _, ctx = sag.group_norm_forward(X, groups, w, b, seg=sd, eps=1e-3, act=kind, slope=0.2)
    base = sag.empty_dense(n, d, TD[dt], DEV, fill=7.0)
    dw, db, dX = sag.group_norm_backward(ctx, G, dX=base)
    x, gg, ww, bb, mean, rstd = f64(X), f64(G), f64(w), f64(b), f64(ctx.mean), f64(ctx.rstd)
    rw, rb, rX = ob.norm_backward(x, groups, seg_h, ww, bb, kind, 0.2, mean, rstd, gg, np.full((n, d), 7.0))
    D = d // groups
    tX, tw, tb = np.zeros((n, d)), np.zeros(d), np.zeros(d)
    own = np.zeros(n, bool)
    S = 512 * U                                     # terms a thread, the threads of a column and of a group
    for i in range(len(seg_h) - 1):
        r = slice(seg_h[i], seg_h[i + 1])
        if seg_h[i] >= seg_h[i + 1]:
            continue
        own[r] = True
        rs = np.repeat(rstd[i], D)
        xh = (x[r] - np.repeat(mean[i], D)) * rs
        z = xh * ww + bb
        a = ob.act_grad(z, kind, 0.2) * gg[r]
        ez = 5 * U * (np.abs(xh * ww) + np.abs(bb))
        # ReLU's side is decided exactly; silu'' is at most 1/2
        ea = np.abs(gg[r]) * ((ez + 16 * U * (1 + np.abs(z))) if kind == "silu" else 2 * U)
        h, eh = np.abs(a * ww), ea * np.abs(ww) + U * np.abs(a * ww)
        ex = 2 * U * np.abs(xh)
        tw += (ea * np.abs(xh) + np.abs(a) * ex).sum(0) + S * np.abs(a * xh).sum(0)
        tb += ea.sum(0) + S * np.abs(a).sum(0)

        def gm(v):
            return np.repeat(v.reshape(-1, groups, D).mean((0, 2)), D)

        m1, m2 = gm(h), gm(h * np.abs(xh))
        e1, e2 = gm(eh) + S * m1, gm(eh * np.abs(xh) + h * ex) + S * m2
        tX[r] = rs * (eh + e1 + np.abs(xh) * e2 + ex * m2 + 4 * U * (h + m1 + np.abs(xh) * m2))
    within(dw, rw, tw * 1.01 + 1e-30)
    within(db, rb, tb * 1.01 + 1e-30)
    within(dX, rX, tX * 1.01 + UT[dt] * (np.abs(rX) + tX))
    assert np.all(f64(dX)[~own] == 7.0)
    # without dX, and written over G: the same bits
    dw2, db2, none = sag.group_norm_backward(ctx, G, want_dX=False)
    assert none is None and np.array_equal(raw(dw2), raw(dw)) and np.array_equal(raw(db2), raw(db))
    G2 = mat_copy(G)
    sag.group_norm_backward(ctx, G2, dX=G2)
    assert np.array_equal(raw(G2)[own], raw(dX)[own]) and np.array_equal(raw(G2)[~own], raw(G)[~own])


@pytest.mark.parametrize("groups", [1, 32])
def test_norm_of_a_large_mean(groups):
    """Values of 1000 with a spread of 1: the variance survives (fp32 sums of
    squares would lose all of it)."""
    say(f"norm large mean groups={groups}")
    g = np.random.default_rng(9)
    x = (1000.0 + g.standard_normal((6000, 32))).astype(np.float32)
    x[0] = 5000.0                                   # and an outlier first
    X = to_dev_dense(x, "f32")
    _, ctx = sag.group_norm_forward(X, groups, eps=0.0)
    mean, rstd = ob.norm_stats(x.astype(np.float64), groups, [0, 6000], 0.0)
    within(ctx.mean, mean, 4 * U * 1000 * np.ones_like(mean))
    # each value's rounding about a thread's mean: u 5000 against a spread of 1
    within(ctx.rstd, rstd, 2.0 ** -10 * rstd)


def test_norm_step_of_relu_is_decided_exactly():
    """Channels whose affine puts z within rounding of 0 on both sides: the
    gradient's mask is the sign of the exact (x - mean) rstd w + b."""
    say("norm relu step")
    g = np.random.default_rng(10)
    n, d = 4000, 8
    X = to_dev_dense(g.standard_normal((n, d)).astype(np.float32), "f32")
    _, c0 = sag.group_norm_forward(X, d)
    x, m, r = f64(X), f64(c0.mean)[0], f64(c0.rstd)[0]
    w = np.ones(d, np.float32)
    b = (-(x[17] - m) * r).astype(np.float32)      # z of row 17 is within half a step of 0
    ctx = sag.GroupNormCtx(X, d, to_dev(w), to_dev(b), None, c0.mean, c0.rstd, "relu")
    G = to_dev_dense(np.repeat((np.arange(n)[:, None] == 17).astype(np.float32), d, 1), "f32")
    _, db, _ = sag.group_norm_backward(ctx, G)
    z = (x[17] - m) * r + b.astype(np.float64)
    assert np.array_equal(f64(db), (z > 0).astype(np.float64))


# ---- together -----------------------------------------------------------------------------

class Block:
    """h + dense(A dropout(act(norm(h)))) and its gradient, as a residual GCN
    block runs them, with the library's own aggregation between."""

    def __init__(self, dt, seed=3, counter=None):
        w = gen.make_config(2, 0.002)
        src, dst = w.edges
        self.n = w.n_global
        self.b = sag.csr_build_normalize(to_dev(src), to_dev(dst), self.n, 0, self.n, True, True, "gcn")
        sag.csr_schedule(self.b.A, 256)
        sag.csr_schedule(self.b.AT, 256)
        g = np.random.default_rng(seed)
        self.d, self.dt = 48, dt
        self.H = mat(g, self.n, self.d, dt)
        self.W = mat(g, self.d, self.d, dt, scale=0.2).contiguous()
        self.bias = to_dev(g.standard_normal(self.d).astype(np.float32))
        self.gw = to_dev(g.uniform(0.5, 1.5, self.d).astype(np.float32))
        self.gb = to_dev(g.standard_normal(self.d).astype(np.float32))
        self.G = mat(g, self.n, self.d, dt)
        self.seg = to_dev(np.array([0, self.n // 3, self.n // 2, self.n], np.int64))
        self.d1 = sag.Drop(0.5, 1, counter=counter)
        self.d2 = sag.Drop(0.2, 2, counter=counter)

    def run(self):
        N, nctx = sag.group_norm_forward(self.H, 4, self.gw, self.gb, seg=self.seg, act="silu")
        P = sag.dropout(N, self.d1)
        Q = sag.spmm_csr(self.b.A, P)
        out, z, dctx = sag.dense_layer_forward(Q, self.W, self.bias, act="gelu", drop=self.d2, residual=self.H)
        dW, db, dQ = sag.dense_layer_backward(dctx, z, self.G)
        dP = sag.spmm_csr_t(self.b.AT, dQ)
        dN = sag.dropout(dP, self.d1)
        dgw, dgb, dH = sag.group_norm_backward(nctx, dN)
        dH = sag.dropout(dH, sag.Drop(0.0, 0), addend=self.G)          # plus the residual's gradient
        return out, dW, db, dgw, dgb, dH


def test_residual_block_against_the_oracle():
    """The run of them in fp32 against the float64 oracle: each stage adds
    rounding of the order of its sums; 1e-4 of each output's largest value is
    some 100 times their worst (rows of up to ~1000 terms, u = 6e-8)."""
    say("residual block")
    from oracle import csr as ocsr
    B = Block("f32")
    out, dW, db, dgw, dgb, dH = [f64(t) for t in B.run()]
    w = gen.make_config(2, 0.002)
    src, dst = w.edges
    o = ocsr.build(src, dst, B.n, 0, B.n, True, True, "gcn")
    A = np.zeros((B.n, B.n))
    for r in range(B.n):
        s, e = o.A.indptr[r], o.A.indptr[r + 1]
        A[r, o.A.indices[s:e]] = o.A.values[s:e]
    H, W, G = f64(B.H), f64(B.W), f64(B.G)
    seg = B.seg.cpu().tolist()
    m, rs = ob.norm_stats(H, 4, seg, 1e-5)
    N = ob.norm_forward(H, 4, seg, f64(B.gw), f64(B.gb), "silu", 0, m, rs, np.zeros_like(H))
    f1, f2 = ob.drop_factor(B.n, B.d, 0.5, 1), ob.drop_factor(B.n, B.d, 0.2, 2)
    Q = A @ ob.drop(N, f1)
    Z, Out = ob.dense_forward(Q, W, f64(B.bias), "gelu", 0, f2, H)
    _, rW, rb, rQ = ob.dense_backward(Q, W, Z, "gelu", 0, f2, G)
    rgw, rgb, rH = ob.norm_backward(H, 4, seg, f64(B.gw), f64(B.gb), "silu", 0, m, rs, ob.drop(A.T @ rQ, f1), np.zeros_like(H))
    for name, got, ref in (("out", out, Out), ("dW", dW, rW), ("db", db, rb), ("dgw", dgw, rgw), ("dgb", dgb, rgb), ("dH", dH, rH + G)):
        assert np.abs(got - ref).max() <= 1e-4 * np.abs(ref).max(), name


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_block_in_a_graph(dt):
    """Captured and replayed several times with eager work between: equal to
    the eager run bit for bit, with a device word that advances the masks."""
    say(f"block graph {dt}")
    counter = torch.zeros(1, dtype=torch.int32, device=DEV)
    B = Block(dt, counter=counter)
    want = []
    for c in range(4):
        counter.fill_(c)
        want.append([raw(t).copy() for t in B.run()])
    assert not np.array_equal(want[0][0], want[1][0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = B.run()
    for c in (0, 2, 1, 3, 0):
        counter.fill_(c)
        torch.randn(1000, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want[c]):
            assert np.array_equal(raw(a), b)
        B.run()
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """The same calls on two streams at a time, each with workspaces of its
    own, give what they give alone."""
    say("block two streams")
    blocks = [Block("bf16", 3), Block("bf16", 4)]
    want = [[raw(t).copy() for t in b.run()] for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, b in enumerate(blocks):
            with torch.cuda.stream(streams[i]):
                got[i] = b.run()
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert np.array_equal(raw(a), b)
