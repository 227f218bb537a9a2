"""Thin Python binding of the C ABI in ``include/packed_attn.h``: causal
attention over packed sequences of different lengths, with grouped heads.

Argument marshalling only: the computation runs in the CUDA kernels of
``libpacked_attn.so``.  ``q`` is ``[T, Hq, D]``, ``k`` and ``v``
``[T, Hkv, D]`` (bf16 or fp16, the last dimension contiguous, rows and heads
at any stride that is a multiple of 8 elements, so slices of a fused
projection are taken as they are); the sequences of the layout lie one
behind another in the rows.  ``lse`` is float32 ``[Hq, T]``.  The stream is
torch's current stream of the tensors' device unless one is given.  On a
given stream the caller orders the work before and behind a call (the inputs
are to be ready there, and results belong to it); tensors may be dropped as soon
as the call has returned.  There is no CPU fallback: if the library is missing,
loading this module raises.

Use::

    lay = pa.Layout([4096, 17, 901])           # built once per batch
    o, lse = pa.forward(q, k, v, lay)
    dq, dk, dv = pa.backward(q, k, v, o, lse, dO, lay)
"""

import ctypes
import os
from array import array

import numpy as np
import torch

from . import sparse_attn as sa

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpacked_attn.so")

# Every entry point declared in include/packed_attn.h.
EXPORTS = ("packed_attn_layout", "packed_attn_layout_free", "packed_attn_layout_rows", "packed_attn_layout_upload",
           "packed_attn_fwd", "packed_attn_bwd_workspace_size", "packed_attn_bwd", "packed_attn_status")


def load_library(path=None):
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m factorized_block_sparse_b200.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    I, VP, SZ, L64, F = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
    T = VP  # pa_tensor, see _descs
    lib.packed_attn_layout.argtypes = [VP, I, ctypes.POINTER(VP)]
    lib.packed_attn_layout.restype = I
    lib.packed_attn_layout_free.argtypes = [VP]
    lib.packed_attn_layout_free.restype = None
    lib.packed_attn_layout_rows.argtypes = [VP]
    lib.packed_attn_layout_rows.restype = L64
    lib.packed_attn_layout_upload.argtypes = [VP, VP]
    lib.packed_attn_layout_upload.restype = I
    lib.packed_attn_fwd.argtypes = [T, T, T, T, VP, L64, L64, I, I, I, I, F, VP, VP]
    lib.packed_attn_fwd.restype = I
    lib.packed_attn_bwd_workspace_size.argtypes = [I, I, I, VP]
    lib.packed_attn_bwd_workspace_size.restype = SZ
    lib.packed_attn_bwd.argtypes = [T, T, T, T, VP, L64, T, T, T, T, L64, I, I, I, I, F, VP, VP, SZ, VP]
    lib.packed_attn_bwd.restype = I
    lib.packed_attn_status.argtypes = [VP]
    lib.packed_attn_status.restype = I
    return lib


lib = load_library()


class Layout:
    """Owns a ``pa_layout*`` of the given sequence lengths (host integers)."""

    def __init__(self, lengths):
        self._h = ctypes.c_void_p()
        wide = np.asarray(lengths).reshape(-1)
        if wide.size and wide.dtype.kind not in "iu":
            raise ValueError(f"sequence lengths must be integers, got {wide.dtype}")
        if wide.size and (wide.min() < 0 or wide.max() > np.iinfo(np.int32).max):
            raise ValueError("sequence lengths must be at least 0 and fit 32 bits")
        self.lengths = tuple(int(n) for n in wide)
        arr = np.ascontiguousarray(wide, dtype=np.int32)  # (after the range check)
        h = ctypes.c_void_p()
        sa._check(lib.packed_attn_layout(arr.ctypes.data, int(arr.size), ctypes.byref(h)), "packed_attn_layout")
        self._h = h
        self.rows = int(lib.packed_attn_layout_rows(h))

    @property
    def handle(self):
        if not self._h.value:
            raise ValueError("the layout is closed")
        return self._h

    def upload(self, device=None, stream=None):
        """Tables to ``device`` (default: the current one); needed before a call is captured into a graph."""
        with torch.cuda.device(device):
            sa._check(lib.packed_attn_layout_upload(self.handle, sa._stream_ptr(stream)), "packed_attn_layout_upload")

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            lib.packed_attn_layout_free(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _check_tensors(q, k, v, layout, more=()):
    """Shapes, types, strides and devices of a call; returns (T, Hq, Hkv, D, type code)."""
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("expected q [T, Hq, D] and k, v [T, Hkv, D]")
    T, Hq, D = qs
    Hkv = ks[1]
    if ks[0] != T or ks[2] != D or v.shape != ks:
        raise ValueError(f"k and v must be [{T}, Hkv, {D}], got {tuple(ks)} and {tuple(v.shape)}")
    if T < layout.rows:
        raise ValueError(f"the layout has {layout.rows} rows, the tensors {T}")
    dt, index = q.dtype, q.get_device() if q.is_cuda else None
    if dt is torch.bfloat16:
        code = 0
    elif dt is torch.float16:
        code = 1
    else:
        raise ValueError(f"expected bf16 or fp16 tensors, got {dt}")
    for name, t, shape in (("q", q, qs), ("k", k, ks), ("v", v, ks), *more):
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        if t.dtype is not dt or t.get_device() != index:
            raise ValueError(f"{name} must be a {dt} tensor on the CUDA device of q")
        if t.stride(2) != 1 and D > 1:
            raise ValueError(f"the last dimension of {name} must be contiguous")
    return T, Hq, Hkv, D, code


def _descs(*tensors):
    """The C views (``pa_tensor``: address, row and head stride) of ``[T, H, D]`` tensors: an array and their addresses
    in it.  The strides of extents of 1 carry no meaning and are not read."""
    flat = []
    for t in tensors:
        rows, heads, _ = t.stride()
        flat += t.data_ptr(), rows, heads
    a = array("q", flat)
    at = a.buffer_info()[0]
    return a, range(at, at + 24 * len(tensors), 24)


def _check_lse(lse, Hq, T, q):
    if tuple(lse.shape) != (Hq, T) or lse.dtype != torch.float32 or lse.device != q.device:
        raise ValueError(f"lse must be float32 [{Hq}, {T}] on the device of q")
    if T > 1 and lse.stride(1) != 1:
        raise ValueError("the rows of lse must be contiguous")
    return lse.stride(0) if Hq > 1 else T


# torch's current stream of a device as an integer, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, stream, what, fn, *args):
    """``fn(*args, stream)`` with ``device`` as the current one, on the given stream or torch's current one of it."""
    if stream is None:
        s = _raw_stream(device.index)
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if device.index == torch.cuda.current_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(device):
            st = fn(*args, s)
    if st:
        raise sa.SparseAttnError(st, what)


def _fwd(q, k, v, o, lse, ls, dims, layout, stream, scale):
    T, Hq, Hkv, D, code = dims
    views, at = _descs(q, k, v, o)  # (kept until the call has read them)
    _call(q.device, stream, "packed_attn_fwd", lib.packed_attn_fwd, *at, lse.data_ptr(), ls, T, Hq, Hkv, D, code,
          D ** -0.5 if scale is None else float(scale), layout.handle)


def _bwd(q, k, v, o, lse, ls, dO, dq, dk, dv, dims, layout, ws, stream, scale):
    T, Hq, Hkv, D, code = dims
    if ws.device != q.device or not ws.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the device of q")
    views, at = _descs(q, k, v, o, dO, dq, dk, dv)  # (kept until the call has read them)
    _call(q.device, stream, "packed_attn_bwd", lib.packed_attn_bwd, *at[:4], lse.data_ptr(), ls, *at[4:], T, Hq, Hkv,
          D, code, D ** -0.5 if scale is None else float(scale), layout.handle, ws.data_ptr(), ws.numel() * ws.element_size())


def packed_attn_fwd(q, k, v, o, lse, layout, stream=None, scale=None):
    """Writes ``o`` and ``lse`` in place (C ABI call); ``scale`` None is 1/sqrt(D)."""
    dims = _check_tensors(q, k, v, layout, (("o", o, q.shape),))
    _fwd(q, k, v, o, lse, _check_lse(lse, dims[1], dims[0], q), dims, layout, stream, scale)
    if stream is not None:
        sa._record(stream, q.device, q, k, v, o, lse)


def packed_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, layout, ws, stream=None, scale=None):
    """Writes ``dq``, ``dk``, ``dv`` in place (C ABI call); ``scale`` None is 1/sqrt(D)."""
    dims = _check_tensors(q, k, v, layout, (("o", o, q.shape), ("dO", dO, q.shape), ("dq", dq, q.shape),
                                            ("dk", dk, k.shape), ("dv", dv, k.shape)))
    _bwd(q, k, v, o, lse, _check_lse(lse, dims[1], dims[0], q), dO, dq, dk, dv, dims, layout, ws, stream, scale)
    if stream is not None:
        sa._record(stream, q.device, q, k, v, o, lse, dO, dq, dk, dv, ws)


def packed_attn_status(stream=None):
    return int(lib.packed_attn_status(sa._stream_ptr(stream)))


# ------------------------------------------------------------ conveniences
def _on_stream(stream, device):
    """A context of the stream that a call runs on, for its allocations and its launches."""
    return torch.cuda.stream(sa._torch_stream(stream, device))


def _new(like, rows):
    """A contiguous tensor of the shape, type and device of another, zero in the rows behind the last sequence."""
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    if rows < t.shape[0]:
        t[rows:].zero_()
    return t


def workspace(Hq, Hkv, D, layout, device):
    n = int(lib.packed_attn_bwd_workspace_size(Hq, Hkv, D, layout.handle))
    if n == 0:
        raise sa.SparseAttnError(sa.SA_ERR_INVALID_ARG, "packed_attn_bwd_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def forward(q, k, v, layout, stream=None, scale=None):
    """Allocates ``o`` and ``lse`` (zero in rows behind the last sequence) and runs the forward pass."""
    dims = _check_tensors(q, k, v, layout)
    if stream is not None:
        with _on_stream(stream, q.device):
            out = forward(q, k, v, layout, scale=scale)
        sa._record(stream, q.device, q, k, v)
        return out
    T, Hq, rows = dims[0], dims[1], layout.rows
    o = _new(q, rows)
    lse = torch.empty(Hq, T, dtype=torch.float32, device=q.device)
    if rows < T:
        lse[:, rows:].zero_()
    _fwd(q, k, v, o, lse, T, dims, layout, None, scale)
    return o, lse


def backward(q, k, v, o, lse, dO, layout, ws=None, stream=None, scale=None):
    """Allocates ``dq``, ``dk``, ``dv`` (zero in rows behind the last sequence), and a workspace if none is given."""
    dims = _check_tensors(q, k, v, layout, (("o", o, q.shape), ("dO", dO, q.shape)))
    T, Hq, Hkv, D, _ = dims
    ls = _check_lse(lse, Hq, T, q)
    if stream is not None:
        with _on_stream(stream, q.device):
            out = backward(q, k, v, o, lse, dO, layout, ws, scale=scale)
        sa._record(stream, q.device, q, k, v, o, lse, dO, ws)
        return out
    rows = layout.rows
    dq, dk, dv = _new(q, rows), _new(k, rows), _new(v, rows)
    if ws is None:
        ws = workspace(Hq, Hkv, D, layout, q.device)
    _bwd(q, k, v, o, lse, ls, dO, dq, dk, dv, dims, layout, ws, None, scale)
    return dq, dk, dv
