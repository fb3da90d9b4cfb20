"""Refusals of dropout, the dense layer and group norm: the binding's checks of
shapes, types and values, and the C ABI's before any launch (no GPU)."""
import ctypes
from dataclasses import replace

import pytest
import torch

sag = pytest.importorskip("sparse_aggregation_gemm_amd")
L = sag._lib


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


D = sag.Drop(0.5, 1)


def test_dropout_binding():
    with pytest.raises(ValueError, match="must be 2-D"):
        sag.dropout(z(4), D)
    with pytest.raises(TypeError, match="unsupported dtype"):
        sag.dropout(z(4, 8, dtype=torch.float16), D)
    with pytest.raises(ValueError, match="addend has shape"):
        sag.dropout(z(4, 8), D, addend=z(4, 7))
    with pytest.raises(TypeError, match="Out is torch.bfloat16"):
        sag.dropout(z(4, 8), D, Out=z(4, 8, dtype=torch.bfloat16))
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError, match="p must lie"):
            sag.dropout(z(4, 8), replace(D, p=p))
    with pytest.raises(ValueError, match="nodes has shape"):
        sag.dropout(z(4, 8), replace(D, nodes=torch.zeros(3, dtype=torch.int32)))
    with pytest.raises(TypeError, match="nodes is torch.int64"):
        sag.dropout(z(4, 8), replace(D, nodes=torch.zeros(4, dtype=torch.int64)))
    with pytest.raises(ValueError, match="contiguous"):
        sag.dropout(z(4, 8), replace(D, nodes=torch.zeros(8, dtype=torch.int32)[::2]))
    with pytest.raises(ValueError, match="counter"):
        sag.dropout(z(4, 8), replace(D, counter=torch.zeros(2, dtype=torch.int32)))
    with pytest.raises(ValueError, match="counter"):
        sag.dropout(z(4, 8), replace(D, counter=torch.zeros(1, dtype=torch.int64)))


def test_operands_must_be_on_the_gpu():
    with pytest.raises(ValueError, match="must be on the GPU"):
        sag.dropout(z(4, 8), D)
    with pytest.raises(ValueError, match="must be on the GPU"):
        sag.dense_layer_forward(z(6, 8), z(8, 5))
    with pytest.raises(ValueError, match="must be on the GPU"):
        sag.group_norm_forward(z(6, 8), 2)


def test_dense_binding():
    X, W = z(6, 8), z(8, 5)
    with pytest.raises(ValueError, match="W has shape"):
        sag.dense_layer_forward(X, z(7, 5))
    with pytest.raises(TypeError, match="W is torch.bfloat16"):
        sag.dense_layer_forward(X, z(8, 5, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="b has shape"):
        sag.dense_layer_forward(X, W, z(6))
    with pytest.raises(ValueError, match="residual has shape"):
        sag.dense_layer_forward(X, W, residual=z(5, 5))
    with pytest.raises(ValueError, match="Out has shape"):
        sag.dense_layer_forward(X, W, Out=z(6, 4))
    with pytest.raises(ValueError, match="Z has shape"):
        sag.dense_layer_forward(X, W, Z=z(7, 5))
    with pytest.raises(ValueError, match="unknown activation 'tanh'"):
        sag.dense_layer_forward(X, W, act="tanh")
    ctx = sag.DenseCtx(X, W, "relu")
    with pytest.raises(ValueError, match="needs Z"):
        sag.dense_layer_backward(ctx, None, z(6, 5))
    with pytest.raises(ValueError, match="G_out has shape"):
        sag.dense_layer_backward(ctx, z(6, 5), z(6, 4))
    with pytest.raises(ValueError, match="dX has shape"):
        sag.dense_layer_backward(ctx, z(6, 5), z(6, 5), dX=z(6, 5))


def test_norm_binding():
    X = z(6, 8)
    with pytest.raises(ValueError, match="groups must divide"):
        sag.group_norm_forward(X, 3)
    with pytest.raises(ValueError, match="groups must divide"):
        sag.group_norm_forward(X, 0)
    with pytest.raises(ValueError, match="weight has shape"):
        sag.group_norm_forward(X, 2, z(7))
    with pytest.raises(ValueError, match="seg must be 1-D"):
        sag.group_norm_forward(X, 2, seg=torch.zeros(0, dtype=torch.int64))
    with pytest.raises(TypeError, match="seg is torch.int32"):
        sag.group_norm_forward(X, 2, seg=torch.zeros(3, dtype=torch.int32))
    ctx = sag.GroupNormCtx(X, 2, None, None, None, z(1, 2), z(1, 2))
    with pytest.raises(ValueError, match="G_out has shape"):
        sag.group_norm_backward(ctx, z(5, 8))
    with pytest.raises(ValueError, match="mean has shape"):
        sag.group_norm_backward(replace(ctx, mean=z(2, 2)), z(6, 8))


fake = ctypes.c_void_p(1 << 20)
BIG = 1 << 40


def drop(**kw):
    d = L.SagDrop(p=0.5, seed=1)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def test_dropout_abi():
    lib = L.lib()

    def call(x=fake, ldx=8, n=4, d=8, dt=0, dr=None, add=None, out=fake, ldo=8):
        return lib.sag_dropout(x, ldx, n, d, dt, drop() if dr is None else dr, add, 8, out, ldo, None)
    assert call(dt=2) == L.SAG_E_INVALID
    assert call(x=None) == L.SAG_E_INVALID
    assert call(out=None) == L.SAG_E_INVALID
    assert call(n=-1) == L.SAG_E_INVALID
    assert call(ldo=4) == L.SAG_E_INVALID
    assert call(ldx=10) == L.SAG_E_ALIGN
    assert call(add=ctypes.c_void_p(8)) == L.SAG_E_ALIGN
    assert lib.sag_dropout(fake, 8, 4, 8, 0, None, None, 0, fake, 8, None) == L.SAG_E_INVALID
    for p in (-0.5, 1.01, float("nan"), float("inf")):
        assert call(dr=drop(p=p)) == L.SAG_E_INVALID
    assert call(dr=drop(row0=-1)) == L.SAG_E_INVALID
    assert call(dr=drop(row0=(1 << 32) - 3)) == L.SAG_E_INVALID
    assert b"32 bits" in lib.sag_last_error()
    assert call(n=0) == L.SAG_OK


def test_dense_abi():
    lib = L.lib()

    def fwd(M=4, x=fake, K=8, w=fake, N=8, act=1, slope=0.1, dr=None, r=None, dt=0, out=fake, ldo=8, ws=fake, nb=BIG):
        return lib.sag_dense_layer_forward(M, x, 8, K, w, None, N, act, slope, dr, r, 8, dt, None, 0, out, ldo, ws, nb, None)
    assert fwd(dt=7) == L.SAG_E_INVALID
    assert fwd(M=-1) == L.SAG_E_INVALID
    assert fwd(K=0) == L.SAG_E_INVALID and fwd(N=0) == L.SAG_E_INVALID
    assert fwd(K=(1 << 24) + 1) == L.SAG_E_UNSUPPORTED
    assert fwd(act=5) == L.SAG_E_INVALID and fwd(act=-1) == L.SAG_E_INVALID
    assert fwd(slope=float("nan")) == L.SAG_E_INVALID
    assert fwd(x=None) == L.SAG_E_INVALID and fwd(w=None) == L.SAG_E_INVALID and fwd(out=None) == L.SAG_E_INVALID
    assert fwd(ldo=6) == L.SAG_E_INVALID and fwd(N=5, ldo=6) == L.SAG_E_ALIGN
    assert fwd(r=ctypes.c_void_p(4)) == L.SAG_E_ALIGN
    assert fwd(dr=drop(p=2.0)) == L.SAG_E_INVALID
    big = 100_000                                  # rows of more tiles than need no workspace
    assert fwd(M=big, nb=16) == L.SAG_E_WORKSPACE and fwd(M=big, ws=None) == L.SAG_E_WORKSPACE
    assert fwd(M=big, ws=ctypes.c_void_p(8)) == L.SAG_E_WORKSPACE
    assert lib.sag_dense_forward_workspace_bytes(4, 8, 8, 0) == 0
    assert lib.sag_dense_forward_workspace_bytes(big, 8, 8, 0) > 0
    assert fwd(M=0) == L.SAG_OK

    def bwd(M=4, x=fake, K=8, w=fake, N=8, act=1, zz=fake, g=fake, dw=fake, db=fake, dx=fake, dt=0, nb=BIG):
        return lib.sag_dense_layer_backward(M, x, 8, K, w, N, act, 0.1, None, zz, 8, g, 8, dw, db, dx, 8, dt, fake, nb, None)
    assert bwd(dt=7) == L.SAG_E_INVALID
    assert bwd(zz=None) == L.SAG_E_INVALID
    assert bwd(g=None) == L.SAG_E_INVALID
    assert bwd(x=None) == L.SAG_E_INVALID
    assert bwd(w=None) == L.SAG_E_INVALID
    assert bwd(nb=64) == L.SAG_E_WORKSPACE
    assert lib.sag_dense_forward_workspace_bytes(4, 0, 8, 0) == 0
    assert lib.sag_dense_backward_workspace_bytes(-1, 8, 8, 0) == 0
    assert lib.sag_dense_backward_workspace_bytes(1000, 8, 8, 1) > 0


def test_norm_abi():
    lib = L.lib()

    def fwd(n=4, d=8, groups=2, seg=None, n_seg=1, eps=1e-5, act=0, dt=0, out=fake, mean=fake, nb=BIG, x=fake):
        return lib.sag_group_norm_forward(x, 4096, n, d, groups, seg, n_seg, None, None, eps, act, 0.1, dt, out, 4096, mean, fake,
                                          fake, nb, None)
    assert fwd(dt=3) == L.SAG_E_INVALID
    assert fwd(n=-1) == L.SAG_E_INVALID and fwd(d=0) == L.SAG_E_INVALID
    assert fwd(groups=3) == L.SAG_E_INVALID and fwd(groups=0) == L.SAG_E_INVALID
    assert fwd(n_seg=2) == L.SAG_E_INVALID and fwd(n_seg=-1) == L.SAG_E_INVALID
    assert fwd(seg=fake, n_seg=1 << 24) == L.SAG_E_UNSUPPORTED
    assert fwd(d=1032, groups=1) == L.SAG_E_UNSUPPORTED and fwd(d=2056, groups=1, dt=1) == L.SAG_E_UNSUPPORTED
    assert fwd(eps=-1.0) == L.SAG_E_INVALID and fwd(eps=float("nan")) == L.SAG_E_INVALID
    assert fwd(act=9) == L.SAG_E_INVALID
    assert fwd(x=None) == L.SAG_E_INVALID and fwd(out=None) == L.SAG_E_INVALID and fwd(mean=None) == L.SAG_E_INVALID
    assert fwd(nb=8) == L.SAG_E_WORKSPACE
    assert fwd(seg=fake, n_seg=0) == L.SAG_OK

    def bwd(g=fake, dx=fake, mean=fake, nb=BIG, n_seg=1, seg=None):
        return lib.sag_group_norm_backward(fake, 8, 4, 8, 2, seg, n_seg, None, None, 0, 0.1, mean, fake, g, 8, fake, fake, dx, 8,
                                           0, fake, nb, None)
    assert bwd(g=None) == L.SAG_E_INVALID
    assert bwd(mean=None) == L.SAG_E_INVALID
    assert bwd(dx=ctypes.c_void_p(8)) == L.SAG_E_ALIGN
    assert bwd(nb=8) == L.SAG_E_WORKSPACE
    assert lib.sag_group_norm_forward_workspace_bytes(100, 64, 4, 3, 1) > 0
    assert lib.sag_group_norm_forward_workspace_bytes(100, 4096, 4, 3, 1) == 0


def test_drop_struct_layout_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f[0] for f in L.SagDrop._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "sag.h"\nint main(void) {\n'
                   '    printf("%zu\\n", sizeof(sag_drop));\n' +
                   "".join(f'    printf("%zu\\n", offsetof(sag_drop, {n}));\n' for n in fields) + "    return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(L.SagDrop)] + [getattr(L.SagDrop, n).offset for n in fields]


@pytest.mark.parametrize("dt", [L.SAG_F32, L.SAG_BF16])
def test_a_workspace_for_many_rows_serves_fewer(dt):
    lib = L.lib()
    rows = sorted({1, 2, 63, 64, 65, 1000, 16383, 16384, 32767, 32768, 33000, 2 ** 20, 2 ** 24 + 1}
                  | {int(1.07 ** i) for i in range(1, 250)})

    def grows(f):
        sizes = [f(m) for m in rows]
        bad = [(a, x, b, y) for a, x, b, y in zip(rows, sizes, rows[1:], sizes[1:]) if y < x]
        assert not bad, bad[:3]

    for k, n in ((1, 1), (100, 47), (256, 256), (257, 300), (1500, 2000)):
        grows(lambda m: lib.sag_dense_forward_workspace_bytes(m, k, n, dt))
        if dt == L.SAG_BF16:       # (fp32 takes the plain product's workspace, for the size it is asked for)
            grows(lambda m: lib.sag_dense_backward_workspace_bytes(m, k, n, dt))
    for d, groups, graphs in ((1, 1, 1), (100, 10, 7), (256, 8, 600), (1000, 1, 5000), (64, 64, 1)):
        grows(lambda m: lib.sag_group_norm_forward_workspace_bytes(m, d, groups, graphs, dt))
        grows(lambda m: lib.sag_group_norm_backward_workspace_bytes(m, d, groups, graphs, dt))
