"""Packed attention without a GPU: the library's exports and refusals, and
the float64 oracle against torch's own attention, autograd and differences."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from factorized_block_sparse_b200 import build
from oracle import packed

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pa():
    build.build_packed_lib()
    from factorized_block_sparse_b200 import packed_attn

    return packed_attn


def test_every_declared_function_is_exported(pa):
    text = open(os.path.join(ROOT, "include", "packed_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(packed_attn_\w+)\s*\(", text))
    assert declared == set(pa.EXPORTS)
    raw = ctypes.CDLL(pa.LIB_PATH)
    for name in declared:
        assert hasattr(raw, name), name
    out = subprocess.run(["ldd", pa.LIB_PATH], capture_output=True, text=True).stdout
    assert "libcuda.so" not in out and "libcudart.so" not in out


def test_layout(pa):
    from factorized_block_sparse_b200 import sparse_attn as sa

    assert pa.Layout([]).rows == 0
    assert pa.Layout([0, 0]).rows == 0
    assert pa.Layout([1, 0, 300]).rows == 301
    for bad in ([-1], [5, -3], [1 << 31]):
        with pytest.raises(ValueError):
            pa.Layout(bad)
    with pytest.raises(sa.SparseAttnError):
        pa.Layout([(1 << 31) - 1])  # past the row limit
    with pytest.raises(sa.SparseAttnError):
        pa.Layout([1 << 30, 1 << 30])
    f = pa.lib.packed_attn_layout
    h = ctypes.c_void_p()
    one = np.array([4], dtype=np.int32)
    assert f(None, 1, ctypes.byref(h)) == sa.SA_ERR_INVALID_ARG
    assert f(one.ctypes.data, -1, ctypes.byref(h)) == sa.SA_ERR_INVALID_ARG
    assert f(one.ctypes.data, 1, None) == sa.SA_ERR_INVALID_ARG
    pa.lib.packed_attn_layout_free(None)
    assert pa.lib.packed_attn_layout_rows(None) == -1
    lay = pa.Layout([3])
    lay.close()
    lay.close()
    with pytest.raises(ValueError):
        lay.handle


def test_workspace_size(pa):
    from factorized_block_sparse_b200 import sparse_attn as sa

    lay = pa.Layout([100, 300])
    ws = pa.lib.packed_attn_bwd_workspace_size
    assert ws(8, 2, 64, lay.handle) > 0
    assert ws(8, 3, 64, lay.handle) == 0  # not a multiple
    assert ws(8, 2, 48, lay.handle) == 0
    assert ws(0, 1, 64, lay.handle) == 0
    assert ws(8, 2, 64, None) == 0
    with pytest.raises(sa.SparseAttnError):
        pa.workspace(8, 3, 64, lay, "cpu")


class _View(ctypes.Structure):  # pa_tensor
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def _t(addr, rs=256, hs=64):
    return ctypes.byref(_View(addr, rs, hs))


def test_argument_checks(pa):
    # refused before anything reaches the device
    from factorized_block_sparse_b200 import sparse_attn as sa

    INV, UNS = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED
    lay = pa.Layout([100, 300])
    base = dict(q=_t(0x10000), k=_t(0x20000, 128), v=_t(0x30000, 128), o=_t(0x40000), lse=0x50000, ls=400, rows=400, hq=4,
                hkv=2, d=64, dt=0, scale=0.125, lay=lay.handle)

    def fwd(**kw):
        a = {**base, **kw}
        return pa.lib.packed_attn_fwd(a["q"], a["k"], a["v"], a["o"], a["lse"], a["ls"], a["rows"], a["hq"], a["hkv"],
                                      a["d"], a["dt"], a["scale"], a["lay"], None)

    def bwd(**kw):
        a = {**base, "dO": _t(0x60000), "dq": _t(0x70000), "dk": _t(0x80000, 128), "dv": _t(0x90000, 128),
             "ws": 0x100000, "wb": 1 << 40, **kw}
        return pa.lib.packed_attn_bwd(a["q"], a["k"], a["v"], a["o"], a["lse"], a["ls"], a["dO"], a["dq"], a["dk"],
                                      a["dv"], a["rows"], a["hq"], a["hkv"], a["d"], a["dt"], a["scale"], a["lay"],
                                      a["ws"], a["wb"], None)

    for f in (fwd, bwd):
        assert f(d=48) == UNS and f(d=256) == UNS
        for bad in (dict(hq=0), dict(hkv=0), dict(hq=3), dict(rows=399), dict(rows=1 << 31), dict(dt=2), dict(dt=-1),
                    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                    dict(lay=None), dict(lse=None), dict(ls=399), dict(hq=65536 * 2),
                    dict(q=None), dict(k=None), dict(v=None), dict(o=None),
                    dict(q=_t(0)), dict(q=_t(0x10008)), dict(q=_t(0x10000, 257)), dict(k=_t(0x20000, 0)),
                    dict(v=_t(0x30000, 128, 63)), dict(v=_t(0x30000, -128, 64))):
            assert f(**bad) == INV, bad
    for bad in (dict(o=_t(0x10000)), dict(o=_t(0x40000, 128, 64)), dict(o=_t(0x40000, 256, 32)),
                dict(o=_t(0x40000, 64, 64))):
        assert fwd(**bad) == INV, bad
    for bad in (dict(dO=None), dict(dq=None), dict(dk=_t(0x20000, 128)), dict(dk=_t(0x70000, 128)),
                dict(dv=_t(0x90000, 64, 64)), dict(dq=_t(0x60000))):
        assert bwd(**bad) == INV, bad
    for bad in (dict(ws=None), dict(ws=0x100010), dict(wb=64)):
        assert bwd(**bad) == sa.SA_ERR_WORKSPACE, bad
    # nothing to do: no device work either
    none = pa.Layout([0])
    assert fwd(lay=none.handle, rows=0) == sa.SA_OK and bwd(lay=none.handle, rows=0) == sa.SA_OK


def test_lengths_that_are_not_integers(pa):
    for bad in ([1.5, 2.0], [True, False], ["3"], np.array([4.0]), torch.tensor([2.5])):
        with pytest.raises(ValueError):
            pa.Layout(bad)
    for good in ([3, 0], (3,), np.array([3], dtype=np.uint8), torch.tensor([3]), np.array([3], dtype=np.int64), [], range(3)):
        assert pa.Layout(good).rows == 3 * (len(good) > 0)


def test_misaligned_lse(pa):
    from factorized_block_sparse_b200 import sparse_attn as sa

    lay = pa.Layout([100])
    q, k, v, o = _t(0x10000), _t(0x20000, 128), _t(0x30000, 128), _t(0x40000)
    for lse in (0x50001, 0x50002):
        assert pa.lib.packed_attn_fwd(q, k, v, o, lse, 100, 100, 4, 2, 64, 0, 0.125, lay.handle,
                                      None) == sa.SA_ERR_INVALID_ARG
        assert pa.lib.packed_attn_bwd(q, k, v, o, lse, 100, _t(0x60000), _t(0x70000), _t(0x80000, 128),
                                      _t(0x90000, 128), 100, 4, 2, 64, 0, 0.125, lay.handle, 0x100000, 1 << 40,
                                      None) == sa.SA_ERR_INVALID_ARG


def test_stream_of_another_device(pa):
    from types import SimpleNamespace

    s = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError):
        pa._on_stream(s, torch.device("cuda", 0))


def test_binding_refusals(pa):
    lay = pa.Layout([4])
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.forward(q, q, q, lay)  # not on a CUDA device
    with pytest.raises(ValueError):
        pa.forward(q[0], q, q, lay)
    with pytest.raises(ValueError):
        pa.forward(q, q[:3], q[:3], lay)
    with pytest.raises(ValueError):
        pa.forward(q, q, q[:, :1], lay)
    with pytest.raises(ValueError):
        pa.forward(q[:3], q[:3], q[:3], lay)


# ------------------------------------------------------------ the oracle itself
CASES = [([5], 1, 1, 8), ([1, 7, 0, 4], 2, 2, 4), ([6, 3], 4, 2, 4), ([9], 6, 1, 4)]


def _inputs(lengths, hq, hkv, d, tail=2, seed=0):
    rng = np.random.default_rng(seed)
    T = sum(lengths) + tail
    return [rng.standard_normal((T, h, d)) for h in (hq, hkv, hkv, hq)]


@pytest.mark.parametrize("lengths,hq,hkv,d", CASES)
@pytest.mark.parametrize("scale", [None, 0.7])
def test_oracle_equals_torch_attention_and_autograd(lengths, hq, hkv, d, scale):
    q, k, v, dO = _inputs(lengths, hq, hkv, d)
    o, lse, mag = packed.forward(q, k, v, lengths, scale)
    g = packed.backward(q, k, v, o, lse, dO, lengths, scale)
    c = packed.starts(lengths)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    loss = 0
    for a, b in zip(c[:-1], c[1:]):
        if a == b:
            continue
        rep = lambda t: t[a:b].repeat_interleave(hq // hkv, dim=1).transpose(0, 1)[None]  # noqa: E731
        ref = torch.nn.functional.scaled_dot_product_attention(tq[a:b].transpose(0, 1)[None], rep(tk), rep(tv),
                                                               is_causal=True, scale=scale)
        np.testing.assert_allclose(o[a:b], ref[0].transpose(0, 1).detach().numpy(), atol=1e-12)
        loss = loss + (ref[0].transpose(0, 1) * torch.tensor(dO[a:b])).sum()
    loss.backward()
    for got, t in zip(g[:3], (tq, tk, tv)):
        np.testing.assert_allclose(got, t.grad.numpy(), atol=1e-12)
    assert (mag + 1e-12 >= np.abs(o)).all()
    rows = c[-1]
    assert not o[rows:].any() and not g[0][rows:].any() and not g[1][rows:].any() and not g[2][rows:].any()


def test_oracle_gradients_equal_differences():
    lengths, hq, hkv, d = [4, 2], 2, 1, 3
    q, k, v, dO = _inputs(lengths, hq, hkv, d, tail=0, seed=3)
    o, lse, _ = packed.forward(q, k, v, lengths)
    grads = packed.backward(q, k, v, o, lse, dO, lengths)[:3]
    h = 1e-6
    for x, g in zip((q, k, v), grads):
        for idx in np.ndindex(x.shape):
            keep = x[idx]
            x[idx] = keep + h
            up = (packed.forward(q, k, v, lengths)[0] * dO).sum()
            x[idx] = keep - h
            dn = (packed.forward(q, k, v, lengths)[0] * dO).sum()
            x[idx] = keep
            assert abs((up - dn) / (2 * h) - g[idx]) <= 1e-6 * max(1.0, abs(g[idx]))
