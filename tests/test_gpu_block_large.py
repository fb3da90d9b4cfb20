"""The dense layer and group norm where outputs have many tiles and batches
many graphs: from 512 tiles of 32 x 32 (512 graphs) on other kernels run than
at the sizes of test_gpu_block, under the same bounds."""
import numpy as np
import pytest
import torch

import test_gpu_block as tb
from oracle import block as ob

pytestmark = pytest.mark.gpu

sag = pytest.importorskip("sparse_aggregation_gemm_amd")
from gpu_util import DEV, f64, say, to_dev  # noqa: E402

# Out of 64 columns or fewer, of more, of several tiles across; ragged in each size
FORWARD = [(9001, 33, 64), (8200, 1, 40), (2100, 70, 300), (1025, 130, 1000), (70, 65, 8200), (4200, 256, 128)]
# dX of up to 64, 128, 256 and more columns (bf16 beyond 256 stores dZ)
BACKWARD = [(9001, 40, 16), (17000, 7, 3), (5000, 100, 72), (3001, 200, 65), (2500, 256, 300), (1500, 400, 130), (515, 1030, 33),
            (33000, 40, 33), (33000, 300, 20)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", FORWARD)
@pytest.mark.parametrize("kind,p,res", [("gelu", 0.1, True), ("relu", None, False), ("silu", 0.5, False), ("none", None, True)])
def test_dense_forward_of_many_tiles(dt, M, K, N, kind, p, res):
    tb.test_dense_forward(dt, M, K, N, kind, p, res)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", BACKWARD)
@pytest.mark.parametrize("kind,p", [("gelu", 0.1), ("relu", 0.5), ("silu", None), ("none", 0.2), ("none", None), ("leaky_relu", None)])
def test_dense_backward_of_many_tiles(dt, M, K, N, kind, p):
    tb.test_dense_backward(dt, M, K, N, kind, p)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", [(9001, 40, 64), (5000, 100, 136), (3001, 200, 260), (1500, 400, 500)])
def test_dense_exact_integers_of_many_tiles(dt, M, K, N):
    tb.test_dense_exact_integers(dt, M, K, N)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", [(150, 45, 52), (9001, 45, 52), (3001, 199, 201), (1500, 401, 403)])
def test_dense_padding_of_nan_and_rows_outside(dt, M, K, N):
    """Padding that holds NaN reaches no result, Out is written over the
    residual and dX over X, and nothing is written outside the views."""
    say(f"dense NaN padding {dt} M={M} K={K} N={N}")
    g = np.random.default_rng(16)

    def holed(rows, d, extra):
        buf = torch.full((rows + 4, (d + 7) // 8 * 8 + extra), float("nan"), dtype=tb.TD[dt], device=DEV)
        buf[2:2 + rows, :d] = torch.from_numpy(g.standard_normal((rows, d)).astype(np.float32)).to(DEV).to(tb.TD[dt])
        return buf, buf[2:2 + rows, :d]

    xb, X = holed(M, K, 8)
    rb, R = holed(M, N, 32)
    zb, Z = holed(M, N, 0)
    W = tb.mat(g, K, N, dt).contiguous()
    b = to_dev(g.standard_normal(N).astype(np.float32))
    drop = sag.Drop(0.25, 5)
    ref, zr, _ = sag.dense_layer_forward(tb.mat_copy(X), W, b, act="gelu", drop=drop, residual=tb.mat_copy(R))
    sag.dense_layer_forward(X, W, b, act="gelu", drop=drop, residual=R, Out=R, Z=Z)
    assert np.array_equal(tb.raw(R), tb.raw(ref)) and np.array_equal(tb.raw(Z), tb.raw(zr))
    _, G = holed(M, N, 16)
    db_, D = holed(M, K, 16)
    want = sag.dense_layer_backward(sag.DenseCtx(tb.mat_copy(X), W, "gelu", 0.01, drop), zr, tb.mat_copy(G))
    got = sag.dense_layer_backward(sag.DenseCtx(X, W, "gelu", 0.01, drop), Z, G, dX=D)
    for a, c in zip(got, want):
        assert np.array_equal(tb.raw(a), tb.raw(c))
    for buf, d in ((rb, N), (zb, N), (db_, K), (xb, K)):
        assert torch.isnan(buf[:2]).all() and torch.isnan(buf[-2:]).all() and torch.isnan(buf[:, d:]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("M,K,N", [(60, 40, 50), (9001, 40, 50), (3001, 200, 260), (1500, 400, 300)])
def test_dense_dropped_values_are_zero_whatever_they_were(dt, M, K, N):
    """p = 1 leaves the residual and no gradient; where a value is dropped, NaN
    and infinity in Z or in the gradient leave nothing."""
    say(f"dense dropped values {dt} M={M} K={K} N={N}")
    g = np.random.default_rng(17)
    X, R, G = tb.mat(g, M, K, dt), tb.mat(g, M, N, dt), tb.mat(g, M, N, dt)
    W = tb.mat(g, K, N, dt, scale=0.1).contiguous()
    out, z, ctx = sag.dense_layer_forward(X, W, act="gelu", drop=sag.Drop(1.0, 3), residual=R)
    assert np.array_equal(tb.raw(out), tb.raw(R)) and f64(z).any()
    for t in sag.dense_layer_backward(ctx, z, G):
        assert not f64(t).any()
    drop = sag.Drop(0.5, 8, 1)
    f = ob.drop_factor(M, N, 0.5, 8, 1)
    bad = X.clone()
    Xn = tb.mat_copy(bad)
    Xn[5, 3], Xn[M - 1, 0] = float("nan"), float("inf")
    out, z, _ = sag.dense_layer_forward(Xn, W, act="relu", drop=drop, residual=R)
    o, r = f64(out), f64(R)
    assert np.array_equal(np.isnan(f64(z)).any(1), np.arange(M) == 5)
    assert np.array_equal(o[f == 0], r[f == 0]) and np.isfinite(np.delete(o, [5, M - 1], 0)).all()
    # gradients that are not finite, only where they are dropped
    hole = torch.from_numpy((f == 0) & (g.random((M, N)) < 0.1)).to(DEV)
    Z = tb.mat(g, M, N, dt)
    want = sag.dense_layer_backward(sag.DenseCtx(X, W, "gelu", 0.0, drop), Z, G)
    G[hole] = float("nan")
    Z[hole] = float("inf")
    got = sag.dense_layer_backward(sag.DenseCtx(X, W, "gelu", 0.0, drop), Z, G)
    for a, c in zip(got, want):
        assert np.array_equal(tb.raw(a), tb.raw(c))


NORMS = [(13000, 256, 8, tb.cuts(13000, 700, 1)), (9000, 100, 10, tb.cuts(9000, 600, 2)), (20000, 8, 2, tb.cuts(20000, 1500, 3)),
         (6000, 40, 40, tb.cuts(6000, 1300, 4)), (9000, 250, 1, tb.cuts(9000, 520, 5)), (3000, 128, 4, tb.cuts(3000, 9000, 6)),
         (5000, 602, 7, tb.cuts(5000, 800, 7)), (40000, 16, 1, tb.cuts(38000, 513, 8))]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,groups,seg", NORMS)
@pytest.mark.parametrize("kind", ["none", "relu", "gelu"])
def test_norm_forward_of_many_graphs(dt, n, d, groups, seg, kind):
    tb.test_norm_forward(dt, n, d, groups, seg, kind)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d,groups,seg", NORMS)
@pytest.mark.parametrize("kind", ["relu", "silu"])
def test_norm_backward_of_many_graphs(dt, n, d, groups, seg, kind):
    tb.test_norm_backward(dt, n, d, groups, seg, kind)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("graphs", [3, 600])
def test_norm_keeps_a_bad_value_in_its_graph_and_group(dt, graphs):
    """NaN and infinity spoil their own graph and group alone; padding columns
    that hold NaN spoil nothing."""
    say(f"norm bad values {dt} graphs={graphs}")
    g = np.random.default_rng(18)
    n, d, groups = graphs * 20, 60, 4
    buf = torch.full((n, 72), float("nan"), dtype=tb.TD[dt], device=DEV)
    X = buf[:, :d]
    X.copy_(torch.from_numpy(g.standard_normal((n, d)).astype(np.float32)))
    seg = to_dev(np.arange(graphs + 1, dtype=np.int64) * 20)
    want, _ = sag.group_norm_forward(tb.mat_copy(X), groups, seg=seg, act="relu")
    X[25, 17], X[59, 59] = float("nan"), float("inf")
    got, ctx = sag.group_norm_forward(X, groups, seg=seg, act="none")
    spoilt = np.zeros((n, d), bool)
    spoilt[20:40, 15:30] = spoilt[40:60, 45:60] = True
    assert np.array_equal(np.isnan(f64(got)), spoilt)
    assert np.array_equal(np.maximum(f64(got), 0)[~spoilt], f64(want)[~spoilt])
    G = tb.mat(g, n, d, dt)
    dX = f64(sag.group_norm_backward(ctx, G)[2])
    assert np.array_equal(np.isnan(dX), spoilt)


def test_norm_of_a_large_mean_by_wavefronts():
    """Short graphs of values about 1000 with a spread of 1."""
    say("norm large mean, short graphs")
    g = np.random.default_rng(19)
    x = (1000.0 + g.standard_normal((600 * 12, 32))).astype(np.float32)
    seg = np.arange(601, dtype=np.int64) * 12
    _, ctx = sag.group_norm_forward(tb.to_dev_dense(x, "f32"), 2, seg=to_dev(seg), eps=0.0)
    mean, rstd = ob.norm_stats(x.astype(np.float64), 2, seg.tolist(), 0.0)
    tb.within(ctx.mean, mean, 4 * tb.U * 1000 * np.ones_like(mean))
    # the squares' own rounding, and the mean's error squared: (4 u 1000)^2 against a variance above 1/2
    tb.within(ctx.rstd, rstd, 64 * tb.U * rstd)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [8, 20000])
def test_activations_of_infinity(dt, rows):
    """Plus infinity stays itself in every activation, NaN stays NaN, and
    ReLU and GELU of minus infinity are their limit 0."""
    say(f"activations of infinity {dt} rows={rows}")
    X = tb.mat_copy(torch.ones(rows, 1, dtype=tb.TD[dt], device=DEV))
    X[1], X[2], X[3] = float("inf"), -float("inf"), float("nan")
    W = torch.ones(1, 40, dtype=tb.TD[dt], device=DEV)
    for kind in ("none", "relu", "leaky_relu", "gelu", "silu"):
        y = f64(sag.dense_layer_forward(X, W, act=kind)[0])
        assert (y[1] == np.inf).all() and np.isnan(y[3]).all() and np.isfinite(np.delete(y, [1, 2, 3], 0)).all(), kind
        if kind in ("relu", "gelu"):
            assert (y[2] == 0).all(), kind


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("graphs", [0, 1, 600])
def test_norm_without_rows(dt, graphs):
    say(f"norm no rows {dt} graphs={graphs}")
    X = sag.empty_dense(0, 40, tb.TD[dt], DEV)
    seg = to_dev(np.zeros(graphs + 1, np.int64))
    w = torch.full((40,), 2.0, device=DEV)
    out, ctx = sag.group_norm_forward(X, 4, w, seg=seg, eps=0.25, act="gelu")
    assert out.shape == (0, 40) and ctx.mean.shape == (graphs, 4)
    assert not f64(ctx.mean).any() and np.all(f64(ctx.rstd) == 2.0)
    dw, db, dX = sag.group_norm_backward(ctx, X)
    assert dX.shape == (0, 40) and not f64(dw).any() and not f64(db).any()


def test_norm_of_rows_in_no_graph():
    """Rows before the first graph and behind the last of many, with NaN in
    them, stay as they were in Out and in dX and count nowhere."""
    say("norm rows in no graph")
    g = np.random.default_rng(20)
    n, d = 6000, 32
    X, G = tb.mat(g, n, d, "bf16"), tb.mat(g, n, d, "bf16")
    seg = np.sort(g.integers(50, n - 70, 601)).astype(np.int64)
    lo, hi = int(seg[0]), int(seg[-1])
    want, c0 = sag.group_norm_forward(X, 4, seg=to_dev(seg), act="silu")
    w0, b0, x0 = sag.group_norm_backward(c0, G)
    X[:lo], X[hi:], G[:lo], G[hi:] = (float("nan"),) * 4
    out, dX = (sag.empty_dense(n, d, torch.bfloat16, DEV, fill=3.0) for _ in range(2))
    _, ctx = sag.group_norm_forward(X, 4, seg=to_dev(seg), act="silu", Out=out)
    dw, db, _ = sag.group_norm_backward(ctx, G, dX=dX)
    for a, b in ((out, want), (dX, x0)):
        assert np.array_equal(tb.raw(a[lo:hi]), tb.raw(b[lo:hi])) and (f64(a[:lo]) == 3).all() and (f64(a[hi:]) == 3).all()
    assert np.array_equal(tb.raw(dw), tb.raw(w0)) and np.array_equal(tb.raw(db), tb.raw(b0))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_large_calls_in_a_graph_and_in_one_workspace(dt):
    """The tiled kernels and wavefronts' graphs captured, replayed with a mask
    that advances and eager work between, and two calls one after the other in
    one workspace: equal to eager calls with workspaces of their own."""
    say(f"large calls captured {dt}")
    g = np.random.default_rng(21)
    M, K, N = 5000, 100, 136
    X, R, G = tb.mat(g, M, K, dt), tb.mat(g, M, N, dt), tb.mat(g, M, N, dt)
    W = tb.mat(g, K, N, dt, scale=0.1).contiguous()
    seg = to_dev(np.asarray(tb.cuts(M, 700, 9), np.int64))
    counter = torch.zeros(1, dtype=torch.int32, device=DEV)
    drop = sag.Drop(0.3, 5, counter=counter)
    ws = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)

    def run(ws=None):
        out, z, ctx = sag.dense_layer_forward(X, W, act="gelu", drop=drop, residual=R, ws=ws)
        y, nctx = sag.group_norm_forward(out, 4, seg=seg, act="silu", ws=ws)
        dw, db, dy = sag.group_norm_backward(nctx, G, ws=ws)
        dW, dc, dX = sag.dense_layer_backward(ctx, z, dy, ws=ws)
        return y, dw, db, dW, dc, dX

    want = []
    for c in range(3):
        counter.fill_(c)
        want.append([tb.raw(t).copy() for t in run()])
        assert all(np.array_equal(a, tb.raw(b)) for a, b in zip(want[-1], run(ws)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(ws)
    for c in (0, 2, 1, 0, 2):
        counter.fill_(c)
        torch.randn(1000, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a, tb.raw(b)) for a, b in zip(want[c], outs)), c


def test_rows_past_32_bits():
    """4.6 G elements a matrix: the last rows come out as they do in a call of
    their own (small whole numbers, so that every sum is exact; group norm
    within a step of bf16, as its sums are cut elsewhere)."""
    say("rows past 32 bits")
    n, d, m = 2 ** 24 + 2 ** 20 + 5, 256, 3001
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free memory")

    def tail(seed):
        g = np.random.default_rng(seed)
        small = tb.mat(g, m, d, "bf16", True)
        big = torch.zeros(n, d, dtype=torch.bfloat16, device=DEV)
        big[n - m:] = small
        return big, small

    (X, x), (G, g) = tail(30), tail(31)
    W = tb.mat(np.random.default_rng(32), d, d, "bf16", True).contiguous()
    far, near = sag.Drop(0.5, 3, row0=5), sag.Drop(0.5, 3, row0=5 + n - m)
    assert np.array_equal(tb.raw(sag.dropout(X, far)[n - m:]), tb.raw(sag.dropout(x, near)))
    out, z, ctx = sag.dense_layer_forward(X, W, act="relu", drop=far, residual=G)
    o, y, c = sag.dense_layer_forward(x, W, act="relu", drop=near, residual=g)
    assert np.array_equal(tb.raw(out[n - m:]), tb.raw(o)) and np.array_equal(tb.raw(z[n - m:]), tb.raw(y))
    del out
    for a, b in zip(sag.dense_layer_backward(ctx, z, G), sag.dense_layer_backward(c, y, g)):
        assert np.array_equal(tb.raw(a[n - m:] if a.shape[0] == n else a), tb.raw(b))
    del z, ctx
    seg = np.array([0, 7, n - m, n - m + 20, n], np.int64)
    out, ctx = sag.group_norm_forward(X, 8, seg=to_dev(seg), act="none")
    o, c = sag.group_norm_forward(x, 8, seg=to_dev(np.array([0, 20, m], np.int64)), act="none")
    tb.within(out[n - m:], f64(o), 2.0 ** -7 * np.abs(f64(o)) + 1e-6)
    got, want = sag.group_norm_backward(ctx, G), sag.group_norm_backward(c, g)
    # (a step of bf16 of each value, and where terms cancel 2^-20 of their size)
    tb.within(got[2][n - m:], f64(want[2]), 2.0 ** -7 * np.abs(f64(want[2])) + 1e-4)
