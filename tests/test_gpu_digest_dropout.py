"""Dropout in DIGEST's exchange (sparse_aggregation_gemm_amd.digest) against
the oracle: each layer reads its local and halo rows dropped out by the masks
of their global ids, its input gradient passes the same masks before it goes
on and before its halo rows return, the stores keep undropped rows, and the
overlapped and one-stream runs give the same bits.

Bounds as in the exchange's test without dropout (relative to the
absolute-value bound, whose entries the mask scales as it does the gradient);
the dropped input is the layer's input times the factor, with one rounding of
the product to fp32 and one to the stored type."""
import numpy as np
import pytest
import torch

import gen
import test_gpu_digest as td
from oracle import block as obl, csr as ocsr, layers as olay, lowbit as olb

pytestmark = pytest.mark.gpu

sag = pytest.importorskip("sparse_aggregation_gemm_amd")
from sparse_aggregation_gemm_amd.digest import StaleExchange  # noqa: E402
from gpu_util import DEV, f64, say, to_dev, to_dev_dense, tol  # noqa: E402


class Share:
    def __init__(self, cfg, scale, model, dt, dims, relu, seed):
        w = gen.make_config(cfg, scale)
        src, dst = w.edges
        args = (w.n_global, w.lo, w.hi, w.symmetrize, w.self_loops, "gcn" if model == "gcn" else "mean")
        self.ob = ocsr.build(src, dst, *args)
        self.gb = sag.csr_build_normalize(to_dev(src), to_dev(dst), *args)
        sag.csr_schedule(self.gb.A, 256)
        sag.csr_schedule(self.gb.AT, 256)
        self.model, self.dt, self.dims, self.relu, L = model, dt, dims, relu, len(dims) - 1
        self.n_l, self.n_h, self.L = self.ob.n_local, self.ob.n_halo, L
        assert self.n_h > 0
        g = np.random.default_rng(seed)
        self.stores0 = [td._stored(g.standard_normal((w.n_global, d)), dt) for d in dims[:-1]]
        self.H0 = td._stored(g.standard_normal((self.n_l, dims[0])), dt)
        k = 2 if model == "sage" else 1
        self.Ws = [td._stored(g.uniform(-0.3, 0.3, (k * dims[l], dims[l + 1])), dt) for l in range(L)]
        self.bs = [g.uniform(-0.1, 0.1, dims[l + 1]).astype(np.float32) for l in range(L)]
        self.G = td._stored(g.standard_normal((self.n_l, dims[L])), dt)
        self.local = np.arange(w.lo, w.hi, dtype=np.int32)
        self.halo_rows = ocsr.halo_rows(self.ob, 0)
        self.ids = np.concatenate([self.local, self.gb.halo_gid.cpu().numpy()]).astype(np.int32)

    def exchange(self, **kw):
        dt = self.dt
        self.stores = [to_dev_dense(s, dt) for s in self.stores0]
        self.gstores = [sag.empty_dense(*s.shape, t.dtype, DEV, fill=0.0) for s, t in zip(self.stores0, self.stores)]
        return StaleExchange(self.gb, self.model, self.dims, self.relu, self.stores, self.gstores, to_dev(self.local), **kw)

    def step(self, ex, **kw):
        dt = self.dt
        res = ex.step(to_dev_dense(self.H0, dt), [to_dev_dense(x, dt).contiguous() for x in self.Ws],
                      [to_dev(x) for x in self.bs], to_dev_dense(self.G, dt), **kw)
        torch.cuda.synchronize()
        return res

    def bits(self, res):
        return [td._bits(x) for x in (res.out, *res.dW, *res.db, *self.stores, *self.gstores)]


@pytest.mark.parametrize("cfg,scale,model,dt,dims,relu", [
    (5, 0.002, "gcn", "f32", [48, 64, 24], [True, False]), (5, 0.002, "gcn", "bf16", [48, 64, 24], [True, True]),
    (3, 1 / 64, "sage", "f32", [30, 64, 16], [True, True]), (3, 1 / 64, "sage", "bf16", [32, 64, 16], [True, False])])
@pytest.mark.parametrize("p", [(0.5, 0.25), (0.0, 0.5)])
def test_exchange_with_dropout(cfg, scale, model, dt, dims, relu, p):
    say(f"digest dropout cfg={cfg} {model} {dt} dims={dims} p={p}")
    S = Share(cfg, scale, model, dt, dims, relu, 4)
    runs = {}
    for overlap in (True, False):
        ex = S.exchange(dropout=p, seed=99)
        runs[overlap] = []
        for call in (0, 1):
            before = [f64(s) for s in S.stores]
            gbefore = [f64(s) for s in S.gstores]
            res = S.step(ex, overlap=overlap, want_dH0=True, call=call)
            runs[overlap].append(S.bits(res))
            if not overlap:
                continue
            outs = [f64(ex.H[l + 1][:S.n_l]) for l in range(S.L - 1)] + [f64(res.out)]
            grads = olay.as_f64(S.G, dt)
            for l in reversed(range(S.L)):
                local = olay.as_f64(S.H0, dt) if l == 0 else outs[l - 1]
                H = np.concatenate([local, before[l][S.halo_rows]])
                f = obl.drop_factor(len(H), dims[l], p[l], 99, call * S.L + l, S.ids) if p[l] else np.ones_like(H)
                X = H
                if p[l]:
                    X = f64(ex.dropped[l])
                    half = torch.finfo(ex.dropped[l].dtype).eps / 2
                    assert np.all(np.abs(X - f * H) <= (2.0 ** -23 + half) * np.abs(f * H))
                Out, Yd, dW, db, dH, (dWd, dbd, dHd) = td._oracle_layer(
                    model, S.ob.A, S.ob.AT, X, S.n_l, olay.as_f64(S.Ws[l], dt), S.bs[l], relu[l], outs[l], grads, True)
                got = f64(res.dH[l])
                for name, a, r, den in (("out", outs[l], Out, Yd), ("dW", f64(res.dW[l]), dW, dWd),
                                        ("db", f64(res.db[l]), db, dbd), ("dH", got, f * dH, f * dHd)):
                    assert td._err(a, r, den) <= tol(dt), f"layer {l} {name}"
                exp = gbefore[l].astype(np.float32)
                exp[S.halo_rows] += got[S.n_l:].astype(np.float32)
                assert np.array_equal(td._bits(S.gstores[l]), td._store_bits(exp, dt)), f"grad store {l}"
                grads = got[:S.n_l]
            for l in range(S.L - 1):
                exp = olb.push(before[l + 1], outs[l], S.local, 0)
                assert np.array_equal(td._bits(S.stores[l + 1]), td._store_bits(exp, dt)), f"store {l + 1}"
    for a, b in zip(runs[True], runs[False]):
        for x, y in zip(a, b):
            assert np.array_equal(x, y), "overlapped and one-stream runs differ"
    assert not np.array_equal(runs[True][0][0], runs[True][1][0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_probability_zero_is_the_run_without(dt):
    say(f"digest dropout zero {dt}")
    S = Share(5, 0.002, "gcn", dt, [48, 64, 24], [True, False], 5)
    want = S.bits(S.step(S.exchange(), want_dH0=True))
    got = S.bits(S.step(S.exchange(dropout=[0.0, 0.0], seed=3), want_dH0=True, call=7))
    assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_refusals():
    say("digest dropout refusals")
    S = Share(5, 0.002, "gcn", "f32", [16, 16, 16], [True, False], 6)
    for bad in ([0.5], [0.5, 1.5], [-0.1, 0.0], [float("nan"), 0.0]):
        with pytest.raises(ValueError, match="one dropout probability"):
            S.exchange(dropout=bad)
