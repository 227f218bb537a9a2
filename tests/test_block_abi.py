"""C ABI of the block library on the host (no GPU): it loads next to the
attention library, exports every function include/sparse_block.h declares,
links the CUDA runtime statically, and sizes its workspace (0 for shapes it
refuses)."""

import ctypes
import os
import re
import subprocess

import pytest

from factorized_block_sparse_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def sb():
    build.build_block_lib()
    from factorized_block_sparse_b200 import sparse_block

    return sparse_block


def test_every_declared_block_function_is_exported(sb):
    text = open(os.path.join(ROOT, "include", "sparse_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(sparse_block_\w+)\s*\(", text))
    assert declared == set(sb.EXPORTS)
    raw = ctypes.CDLL(sb.LIB_PATH)
    for name in declared:
        assert hasattr(raw, name), name


def test_block_library_links(sb):
    out = subprocess.run(["ldd", sb.LIB_PATH], capture_output=True, text=True).stdout
    assert "libsparse_attn.so" in out and "libcublas" in out
    assert "libcudart.so" not in out and "libcuda.so" not in out


def test_block_workspace_size(sb):
    from factorized_block_sparse_b200 import sparse_attn as sa

    lay = sa.Layout("fixed", 1024, 128, 32, 64)
    ws = sb.lib.sparse_block_workspace_size
    n = ws(2, 1024, 4, 64, lay.handle)
    mc = 2 * 1024 * 4 * 64 * 2  # one [M, C] bf16 tensor
    # activations of the recomputed forward and their gradients (38 [M, C] tensors) + the attention's workspace
    assert n >= 38 * mc + sa.sparse_attn_bwd_workspace_size(2, 4, 1024, 64, lay)
    assert ws(2, 1024, 4, 48, lay.handle) == 0        # D outside {32, 64, 128}
    assert ws(1, 1024, 64, 128, lay.handle) == 0      # H * D above 6144
    assert ws(0, 1024, 4, 64, lay.handle) == 0
    assert ws(1, 1024, 4, 64, None) == 0


def test_gelu_argument_checks(sb):
    # refused before anything reaches the device (no GPU needed)
    from factorized_block_sparse_b200 import sparse_attn as sa

    f = sb.lib.sparse_block_gelu
    a, b, c = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
    assert f(None, b, None, 8, None) == sa.SA_ERR_INVALID_ARG           # u null
    assert f(a, None, None, 8, None) == sa.SA_ERR_INVALID_ARG           # g null
    assert f(a, b, None, 12, None) == sa.SA_ERR_INVALID_ARG             # n not a multiple of 8
    assert f(ctypes.c_void_p(0x10008), b, None, 8, None) == sa.SA_ERR_INVALID_ARG  # u not 16-byte aligned
    assert f(a, b, ctypes.c_void_p(0x30004), 8, None) == sa.SA_ERR_INVALID_ARG     # dgelu not aligned
    assert f(a, b, a, 8, None) == sa.SA_ERR_INVALID_ARG                 # dgelu is u
    assert f(a, b, b, 8, None) == sa.SA_ERR_INVALID_ARG                 # dgelu is g
    assert f(a, b, c, 0, None) == sa.SA_OK                              # nothing to do


def test_layer_norm_and_clip_argument_checks(sb):
    # refused before anything reaches the device (no GPU needed)
    from factorized_block_sparse_b200 import sparse_attn as sa

    INV, UNS, WS = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED, sa.SA_ERR_WORKSPACE
    A, Bp, Cp, Dp, Ep = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000

    def fwd(x=A, ldx=64, g=Bp, b=Cp, y=Dp, ldy=64, mean=Ep, rstd=0x60000, M=4, C=64, eps=1e-5, dt=0):
        return sb.lib.sparse_block_layer_norm_fwd(x, ldx, g, b, y, ldy, mean, rstd, M, C, eps, dt, None)

    for kw in (dict(x=None), dict(g=None), dict(y=None), dict(M=-1), dict(C=0), dict(ldx=63), dict(ldy=63), dict(dt=3),
               dict(dt=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=A + 1), dict(b=Cp + 2),
               dict(mean=Ep + 2), dict(y=A, ldx=64, ldy=72), dict(dt=2, x=A + 2)):
        assert fwd(**kw) == INV, kw
    assert fwd(C=16385, ldx=16385, ldy=16385) == UNS
    assert fwd(M=0) == sa.SA_OK
    size = sb.lib.sparse_block_layer_norm_bwd_workspace_size
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 16385) == 0 and size(0, 64) > 0

    def bwd(x=A, ldx=64, g=Bp, dy=Cp, lddy=64, mean=Dp, rstd=Ep, dx=0x60000, lddx=64, dg=0x70000, db=0x80000, M=4, C=64,
            dt=0, ws=0x90000, wb=1 << 30):
        return sb.lib.sparse_block_layer_norm_bwd(x, ldx, g, dy, lddy, mean, rstd, dx, lddx, dg, db, M, C, dt, ws, wb, None)

    for kw in (dict(x=None), dict(g=None), dict(dy=None), dict(mean=None), dict(rstd=None), dict(dx=None), dict(dg=None),
               dict(M=-1), dict(C=0), dict(ldx=63), dict(lddy=63), dict(lddx=63), dict(dt=5), dict(dx=A, lddx=72),
               dict(dx=Cp, lddx=72), dict(db=0x70000), dict(dy=Cp + 1), dict(dg=0x70002)):
        assert bwd(**kw) == INV, kw
    assert bwd(C=20000, ldx=20000, lddy=20000, lddx=20000) == UNS
    assert bwd(ws=None) == WS and bwd(ws=0x90010) == WS and bwd(wb=100) == WS

    VP, SZ, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int

    def clip(g=(A, Bp), o=(A, Bp), n=(16, 16), dt=(0, 2), mx=1.0, norm=Ep, ws=0x90000, wb=1 << 20, count=None):
        k = len(g)
        return sb.lib.sparse_block_clip_grads(k if count is None else count, (VP * k)(*g), (VP * k)(*o) if o else None,
                                              (SZ * k)(*n), (I * k)(*dt), mx, norm, ws, wb, None)

    for kw in (dict(count=-1), dict(norm=None), dict(norm=Ep + 2), dict(mx=-1.0), dict(mx=float("nan")), dict(dt=(0, 3)),
               dict(g=(0, Bp)), dict(g=(A + 1, Bp)), dict(g=(A, Bp + 2)), dict(o=(A, 0)), dict(o=(A, Bp + 2)),
               dict(n=(16, 1 << 41)),
               dict(g=(A, A), dt=(0, 0)),                       # one buffer twice
               dict(g=(A, Bp), o=(Bp, A)),                      # written over another gradient
               dict(o=(A + 16, Bp)), dict(o=(Cp, Cp)), dict(o=(Cp, Cp + 16), dt=(0, 0))):
        assert clip(**kw) == INV, kw
    assert clip(ws=None) == WS and clip(ws=0x90008) == WS and clip(wb=64) == WS
