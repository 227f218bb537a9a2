"""Thin Python binding of the C ABI in ``include/sparse_block.h``: the Sparse
Transformer block around the attention op.

Argument marshalling only: the block runs in ``libsparse_block.so`` (CUDA
kernels for the layer norms, GELU and head layout, cuBLAS and cuBLASLt for
the projections, ``libsparse_attn.so`` for the attention).  Tensors are
``torch.Tensor`` objects on a CUDA device: activations bf16 ``[B, N, C]``
with ``C = H * D``, projection weights bf16 ``[in, out]``, layer-norm
parameters and parameter gradients float32.  With ``stream=`` the caller orders
the work before and behind a call; tensors may be dropped as soon as it has
returned.  There is no CPU fallback.
"""

import ctypes
import os
from array import array

import torch

from . import sparse_attn as sa

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparse_block.so")

PARAMS = ("ln1_g", "ln1_b", "w_qkv", "w_o", "ln2_g", "ln2_b", "w_1", "w_2")
EXPORTS = ("sparse_block_workspace_size", "sparse_block_fwd", "sparse_block_bwd", "sparse_block_gelu",
           "sparse_block_layer_norm_fwd", "sparse_block_layer_norm_bwd_workspace_size", "sparse_block_layer_norm_bwd",
           "sparse_block_clip_workspace_size", "sparse_block_clip_grads")


class _Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in PARAMS]


def load_library(path=None):
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m factorized_block_sparse_b200.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    I, VP, SZ = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER(_Params)
    lib.sparse_block_workspace_size.argtypes = [I, I, I, I, VP]
    lib.sparse_block_workspace_size.restype = SZ
    lib.sparse_block_fwd.argtypes = [VP, P, VP, I, I, I, I, VP, VP, SZ, VP]
    lib.sparse_block_fwd.restype = I
    lib.sparse_block_bwd.argtypes = [VP, VP, P, VP, P, I, I, I, I, VP, VP, SZ, VP]
    lib.sparse_block_bwd.restype = I
    lib.sparse_block_gelu.argtypes = [VP, VP, VP, SZ, VP]
    lib.sparse_block_gelu.restype = I
    L64, F = ctypes.c_int64, ctypes.c_float
    lib.sparse_block_layer_norm_fwd.argtypes = [VP, L64, VP, VP, VP, L64, VP, VP, L64, I, F, I, VP]
    lib.sparse_block_layer_norm_fwd.restype = I
    lib.sparse_block_layer_norm_bwd_workspace_size.argtypes = [L64, I]
    lib.sparse_block_layer_norm_bwd_workspace_size.restype = SZ
    lib.sparse_block_layer_norm_bwd.argtypes = [VP, L64, VP, VP, L64, VP, VP, VP, L64, VP, VP, L64, I, I, VP, SZ, VP]
    lib.sparse_block_layer_norm_bwd.restype = I
    lib.sparse_block_clip_workspace_size.argtypes = []
    lib.sparse_block_clip_workspace_size.restype = SZ
    lib.sparse_block_clip_grads.argtypes = [I, VP, VP, VP, VP, ctypes.c_double, VP, VP, SZ, VP]
    lib.sparse_block_clip_grads.restype = I
    return lib


lib = load_library()


def _struct(d):
    return _Params(*[ctypes.c_void_p(d[n].data_ptr()) for n in PARAMS])


def _dims(x, H):
    B, N, C = (int(s) for s in x.shape)
    if C % H:
        raise ValueError("C must be a multiple of H")
    return B, N, C // H


def workspace(B, N, H, D, layout, device):
    import torch

    n = int(lib.sparse_block_workspace_size(B, N, H, D, layout.handle))
    if n == 0:
        raise sa.SparseAttnError(sa.SA_ERR_INVALID_ARG, "sparse_block_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def sparse_block_fwd(x, params, y, H, layout, ws, stream=None):
    B, N, D = _dims(x, H)
    p = _struct(params)
    sa._check(lib.sparse_block_fwd(sa._ptr(x), ctypes.byref(p), sa._ptr(y), B, N, H, D, layout.handle, sa._ptr(ws),
                                   ws.numel(), sa._stream_ptr(stream)), "sparse_block_fwd")


def sparse_block_bwd(x, dy, params, dx, grads, H, layout, ws, stream=None):
    B, N, D = _dims(x, H)
    p, g = _struct(params), _struct(grads)
    sa._check(lib.sparse_block_bwd(sa._ptr(x), sa._ptr(dy), ctypes.byref(p), sa._ptr(dx), ctypes.byref(g), B, N, H,
                                   D, layout.handle, sa._ptr(ws), ws.numel(), sa._stream_ptr(stream)),
              "sparse_block_bwd")


def forward(x, params, H, layout, ws=None, stream=None):
    """Allocates ``y`` (and a workspace if none is given) and runs the block."""
    import torch

    B, N, D = _dims(x, H)
    ws = workspace(B, N, H, D, layout, x.device) if ws is None else ws
    y = torch.empty_like(x)
    sparse_block_fwd(x, params, y, H, layout, ws, stream)
    if stream is not None:
        sa._record(stream, x.device, x, *(params[n] for n in PARAMS), y, ws)
    return y


def backward(x, dy, params, H, layout, ws=None, stream=None, max_norm=None):
    """``(dx, grads)``: grads holds float32 tensors of the parameters' shapes.
    With ``max_norm`` the gradients are clipped by their global norm in place
    (``clip_grads``) and the result is ``(dx, grads, norm)``."""
    import torch

    B, N, D = _dims(x, H)
    ws = workspace(B, N, H, D, layout, x.device) if ws is None else ws
    dx = torch.empty_like(x)
    grads = {n: torch.empty(params[n].shape, dtype=torch.float32, device=x.device) for n in PARAMS}
    sparse_block_bwd(x, dy, params, dx, grads, H, layout, ws, stream)
    if stream is not None:
        sa._record(stream, x.device, x, dy, *(params[n] for n in PARAMS), dx, *grads.values(), ws)
    if max_norm is not None:
        return dx, grads, clip_grads(grads, max_norm, stream=stream)
    return dx, grads


def sparse_block_gelu(u, g, dgelu=None, stream=None):
    sa._check(lib.sparse_block_gelu(sa._ptr(u), sa._ptr(g), sa._ptr(dgelu) if dgelu is not None else None,
                                    u.numel(), sa._stream_ptr(stream)), "sparse_block_gelu")


def gelu(u, grad=False, stream=None):
    """``gelu(u)`` (and ``gelu'(u)`` when ``grad``) of a bf16 tensor with a multiple of 8 elements."""
    import torch

    g = torch.empty_like(u)
    d = torch.empty_like(u) if grad else None
    sparse_block_gelu(u, g, d, stream)
    return (g, d) if grad else g


# ------------------------------------------------------------ layer norm
def _dtype(t):
    dt = t.dtype
    if dt is torch.bfloat16:
        return 0
    if dt is torch.float16:
        return 1
    if dt is torch.float32:
        return 2
    raise ValueError(f"expected a bf16, fp16 or float32 tensor, got {dt}")


def _rows(name, t):
    """``(rows, C, row stride)`` of a tensor whose leading dimensions are one run of rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must have at least one channel")
    C = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // C, C, C
    if C > 1 and t.stride(-1) != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    rows, ld = 1, C
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if rows > 1 and st != rows * ld:
            raise ValueError(f"the leading dimensions of {name} must be rows at one stride")
        if rows == 1:
            ld = st
        rows *= n
    if rows > 1 and ld < C:
        raise ValueError(f"the rows of {name} overlap")
    return rows, C, (ld if rows > 1 else C)


def _vector(name, t, C, device):
    if t.dtype is not torch.float32 or t.device != device or t.shape != (C,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [{C}] tensor on {device}")
    return t.data_ptr()


def _on(device, stream):
    """A context of the device and the stream that a call runs on, for its allocations and its launch."""
    import contextlib

    if stream is not None:
        stream = sa._torch_stream(stream, device)
    cm = contextlib.ExitStack()
    if device.index != torch.cuda.current_device():
        cm.enter_context(torch.cuda.device(device))
    if stream is not None:
        cm.enter_context(torch.cuda.stream(stream))
    return cm


# torch's current stream of a device as an integer, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _here(device, stream):
    """Whether a call runs on the current device and its current stream, so that it needs no context."""
    return stream is None and device.index == torch.cuda.current_device()


def layer_norm(x, g, b=None, eps=1e-5, stream=None):
    """``(y, mean, rstd)`` of rows ``x [..., C]`` (bf16, fp16 or float32; rows at any one stride): y of x's type and
    shape, contiguous; mean and rstd float32 of the leading shape, for ``layer_norm_backward``.  ``g`` and ``b`` are
    float32 ``[C]``; without ``b`` there is no bias."""
    dev = x.device
    M, C, ld = _rows("x", x)
    dt = _dtype(x)
    gp = _vector("g", g, C, dev)
    bp = None if b is None else _vector("b", b, C, dev)
    if not _here(dev, stream):
        with _on(dev, stream):
            out = layer_norm(x, g, b, eps)
        if stream is not None:
            sa._record(stream, dev, x, g, b)
        return out
    y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if x.dim() == 2:
        mean = torch.empty(M, dtype=torch.float32, device=dev)
    else:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    if M:
        st = lib.sparse_block_layer_norm_fwd(x.data_ptr(), ld, gp, bp, y.data_ptr(), C, mean.data_ptr(), rstd.data_ptr(),
                                             M, C, eps, dt, _raw_stream(dev.index))
        if st:
            raise sa.SparseAttnError(st, "sparse_block_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_backward(x, g, dy, mean, rstd, bias=True, stream=None):
    """``(dx, dg, db)`` from ``layer_norm``'s input, gain and statistics and the upstream gradient ``dy``: dx of x's
    type and shape, contiguous; dg and db float32 ``[C]`` (db None without ``bias``)."""
    dev = x.device
    M, C, ld = _rows("x", x)
    dt = _dtype(x)
    if dy.shape != x.shape or dy.dtype is not x.dtype or dy.device != dev:
        raise ValueError(f"dy must be a {x.dtype} tensor of shape {tuple(x.shape)} on {dev}")
    ldd = _rows("dy", dy)[2]
    gp = _vector("g", g, C, dev)
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype is not torch.float32 or t.shape != x.shape[:-1] or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(x.shape[:-1])} on {dev}")
    if not _here(dev, stream):
        with _on(dev, stream):
            out = layer_norm_backward(x, g, dy, mean, rstd, bias)
        if stream is not None:
            sa._record(stream, dev, x, g, dy, mean, rstd)
        return out
    dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    if M == 0:
        return dx, torch.zeros_like(g), torch.zeros_like(g) if bias else None
    dg = torch.empty_like(g)
    db = torch.empty_like(g) if bias else None
    n = lib.sparse_block_layer_norm_bwd_workspace_size(M, C)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    st = lib.sparse_block_layer_norm_bwd(x.data_ptr(), ld, gp, dy.data_ptr(), ldd, mean.data_ptr(), rstd.data_ptr(),
                                         dx.data_ptr(), C, dg.data_ptr(), db.data_ptr() if bias else None, M, C, dt,
                                         ws.data_ptr(), n, _raw_stream(dev.index))
    if st:
        raise sa.SparseAttnError(st, "sparse_block_layer_norm_bwd")
    return dx, dg, db


# ------------------------------------------------- norm and clipping of gradients
_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _clip(grads, max_norm, out, stream):
    in_place = out is grads
    if isinstance(grads, dict):
        if isinstance(out, dict) and not in_place:  # by name: the two may be in different orders
            if out.keys() != grads.keys():
                raise ValueError("the outputs must have the gradients' names")
            out = [out[n] for n in grads]
        grads = list(grads.values())
    else:
        grads = list(grads)
    outs = grads if in_place else None if out is None else list(out.values()) if isinstance(out, dict) else list(out)
    if not grads:
        raise ValueError("expected at least one gradient")
    if outs is not None and len(outs) != len(grads):
        raise ValueError(f"{len(grads)} gradients, {len(outs)} outputs")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("gradients must be CUDA tensors")
    index = dev.index
    for t in grads:
        if t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"gradients must be contiguous tensors on {dev}")
    codes = [_CODES.get(t.dtype, -1) for t in grads]
    if -1 in codes:
        raise ValueError(f"expected bf16, fp16 or float32 gradients, got {grads[codes.index(-1)].dtype}")
    if outs is not None and not in_place:
        for t, o in zip(grads, outs):
            if o.shape != t.shape or o.dtype is not t.dtype or o.get_device() != index or not o.is_contiguous():
                raise ValueError("an output must be a contiguous tensor of its gradient's shape, type and device")
    if not _here(dev, stream):
        with _on(dev, stream):
            norm = _clip(grads, max_norm, grads if in_place else outs, None)
        if stream is not None:
            sa._record(stream, dev, *grads, *(() if in_place or outs is None else outs))
        return norm
    # host arrays of pointers, counts and types; the call has read them when it returns
    gp = array("Q", [t.data_ptr() for t in grads])
    op = None if outs is None else gp if in_place else array("Q", [t.data_ptr() for t in outs])
    counts, types = array("Q", [t.numel() for t in grads]), array("i", codes)
    buf = torch.empty(64 + CLIP_WORKSPACE // 4, dtype=torch.float32, device=dev)  # the norm, and 256 bytes behind it the workspace
    at = buf.data_ptr()
    st = lib.sparse_block_clip_grads(len(grads), gp.buffer_info()[0], None if op is None else op.buffer_info()[0],
                                     counts.buffer_info()[0], types.buffer_info()[0], float(max_norm), at, at + 256,
                                     CLIP_WORKSPACE, _raw_stream(index))
    if st:
        raise sa.SparseAttnError(st, "sparse_block_clip_grads")
    return buf[0]


CLIP_WORKSPACE = int(lib.sparse_block_clip_workspace_size())


def grad_norm(grads, stream=None):
    """The norm of all gradients (a list or dict of contiguous bf16, fp16 or float32 tensors) taken as one vector, as
    a float32 scalar tensor on their device."""
    return _clip(grads, 0.0, None, stream)


def clip_grads(grads, max_norm, out=None, stream=None):
    """Multiplies every gradient by ``min(1, max_norm / (norm + 1e-6))``, in place or into the tensors of ``out``, and
    returns ``norm``, the global norm before it (a float32 scalar tensor on the device; nothing waits for it)."""
    return _clip(grads, max_norm, grads if out is None else out, stream)
