"""The training operators together, as a step over packed documents uses them:
the attention half of a pre-activation block, h = x + attn(LN(x) Wqkv) Wo,
its backward pass by hand, and the clipping of all gradients; against the same
formulas in float64.

Tolerance.  On the way to h the activations a, q/k/v, o and h are rounded to
bf16, and so are the attention's weights; the gradients pass through do, dq,
dk, dv, da and dx as well: about ten roundings of at most 2^-8 of a value each,
whose errors are independent, so relative L2 at most sqrt(10) 2^-8 = 1.2e-2
(a rounding's own root mean square is 0.58 of its bound, which is the room).
"""

import numpy as np
import pytest
import torch

from factorized_block_sparse_b200 import synth
from oracle import packed

pytestmark = pytest.mark.gpu

REL = 1.2e-2


def f64(t):
    return t.detach().cpu().double().numpy()


def close(name, got, ref):
    got = f64(got)
    assert np.isfinite(got).all(), name
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= REL, f"{name}: relative L2 {rel:.2e}"


def step(pa, sb, x, dy, p, layout, hq, hkv, d, max_norm, ws=None):
    """One step: (h, gradients by name, norm before the clipping)."""
    T, C = x.shape
    a, mean, rstd = sb.layer_norm(x, p["g"], p["b"])
    qkv = (a @ p["w_qkv"]).view(T, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    o, lse = pa.forward(q, k, v, layout)
    h = torch.addmm(x, o.view(T, hq * d), p["w_o"])
    # backward
    do = (dy @ p["w_o"].t()).view(T, hq, d)
    dqkv = torch.empty_like(qkv)
    pa.packed_attn_bwd(q, k, v, o, lse, do, dqkv[:, :hq], dqkv[:, hq:hq + hkv], dqkv[:, hq + hkv:], layout,
                       pa.workspace(hq, hkv, d, layout, x.device) if ws is None else ws)
    dqkv = dqkv.view(T, -1)
    da = dqkv @ p["w_qkv"].t()
    dx, dg, db = sb.layer_norm_backward(x, p["g"], da, mean, rstd)
    grads = {"w_o": o.view(T, -1).t() @ dy, "w_qkv": a.t() @ dqkv, "g": dg, "b": db}
    norm = sb.clip_grads(grads, max_norm)
    return h, dx + dy, grads, norm


def reference(x, dy, p, lengths, hq, hkv, d):
    eps = 1e-5
    m = x.mean(-1, keepdims=True)
    r = 1 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    xh = (x - m) * r
    a = xh * p["g"] + p["b"]
    T = x.shape[0]
    qkv = (a @ p["w_qkv"]).reshape(T, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    o, lse, _ = packed.forward(q, k, v, lengths)
    h = x + o.reshape(T, -1) @ p["w_o"]
    do = (dy @ p["w_o"].T).reshape(T, hq, d)
    dq, dk, dv, _ = packed.backward(q, k, v, o, lse, do, lengths)
    dqkv = np.concatenate([dq, dk, dv], 1).reshape(T, -1)
    t = (dqkv @ p["w_qkv"].T)
    g = {"w_o": o.reshape(T, -1).T @ dy, "w_qkv": a.T @ dqkv, "g": (t * xh).sum(0), "b": t.sum(0)}
    t = t * p["g"]
    dx = r * (t - t.mean(-1, keepdims=True) - xh * (t * xh).mean(-1, keepdims=True)) + dy
    return h, dx, g


def make(lengths, hq, hkv, d, device):
    T, C, W = sum(lengths), hq * d, (hq + 2 * hkv) * d
    bf = torch.bfloat16
    n = lambda shape, s, f=1.0: torch.from_numpy(synth.normal_f32(shape, s) * np.float32(f))  # noqa: E731
    p = {"g": 1 + 0.1 * n((C,), 82), "b": 0.1 * n((C,), 83), "w_qkv": n((C, W), 84, C ** -0.5).to(bf),
         "w_o": n((C, C), 85, C ** -0.5).to(bf)}
    return n((T, C), 80).to(bf).to(device), n((T, C), 81).to(bf).to(device), {k: v.to(device) for k, v in p.items()}


@pytest.mark.parametrize("lengths,hq,hkv,d", [([300, 17, 1, 211], 4, 2, 64), ([129, 384], 4, 1, 128)])
def test_training_step_over_packed_documents(cuda_device, lengths, hq, hkv, d):
    from factorized_block_sparse_b200 import packed_attn as pa
    from factorized_block_sparse_b200 import sparse_block as sb

    x, dy, p = make(lengths, hq, hkv, d, cuda_device)
    layout = pa.Layout(lengths)
    ref_h, ref_dx, ref_g = reference(f64(x), f64(dy), {k: f64(v) for k, v in p.items()}, lengths, hq, hkv, d)
    ref_norm = np.sqrt(sum((v ** 2).sum() for v in ref_g.values()))
    h, dx, grads, norm = step(pa, sb, x, dy, p, layout, hq, hkv, d, 0.5 * ref_norm)
    assert pa.packed_attn_status() == 0
    close("h", h, ref_h)
    close("dx", dx, ref_dx)
    assert abs(float(norm) - ref_norm) <= REL * ref_norm
    scale = 0.5 * ref_norm / float(norm)
    for name in ref_g:
        close(name, grads[name], ref_g[name] * scale)
    # the clipped gradients have the norm asked for (bf16 weights' gradients round once more)
    assert abs(float(sb.grad_norm(grads)) - 0.5 * ref_norm) <= 2.0 ** -8 * ref_norm


def test_training_step_captured(cuda_device):
    """The whole step in one CUDA graph, replayed on other inputs, equals the eager step bit for bit."""
    from factorized_block_sparse_b200 import packed_attn as pa
    from factorized_block_sparse_b200 import sparse_block as sb

    lengths, hq, hkv, d = [300, 17, 1, 211], 4, 2, 64
    x, dy, p = make(lengths, hq, hkv, d, cuda_device)
    layout = pa.Layout(lengths)
    layout.upload(cuda_device)
    ws = pa.workspace(hq, hkv, d, layout, cuda_device)
    eager = step(pa, sb, x, dy, p, layout, hq, hkv, d, 1.0, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # the products' library sets itself up outside the capture
        step(pa, sb, x, dy, p, layout, hq, hkv, d, 1.0, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step(pa, sb, x, dy, p, layout, hq, hkv, d, 1.0, ws)
    x2, dy2 = x.flip(0).contiguous(), dy.flip(0).contiguous()
    want2 = step(pa, sb, x2, dy2, p, layout, hq, hkv, d, 1.0, ws)
    keep = x.clone(), dy.clone()
    for a, b, want in ((keep[0], keep[1], eager), (x2, dy2, want2)):
        x.copy_(a)
        dy.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and torch.equal(out[3], want[3])
        for name in want[2]:
            assert torch.equal(out[2][name], want[2][name]), name


def test_streams_given_as_handles(cuda_device):
    # 0 is the legacy default stream; another stream's handle stands for it
    from factorized_block_sparse_b200 import packed_attn as pa
    from factorized_block_sparse_b200 import sparse_block as sb

    lay = pa.Layout([200, 57])
    q, k, v, dO = (torch.from_numpy(synth.normal_f32((257, 2, 64), 90 + i)).to(torch.bfloat16).to(cuda_device)
                   for i in range(4))
    x = q.reshape(257, 128)
    g = torch.ones(128, device=cuda_device)

    def run(stream):
        o, lse = pa.forward(q, k, v, lay, stream=stream)
        d = pa.backward(q, k, v, o, lse, dO, lay, stream=stream)
        y, mean, rstd = sb.layer_norm(x, g, stream=stream)
        e = sb.layer_norm_backward(x, g, y, mean, rstd, stream=stream)
        out = [torch.empty_like(t) for t in d]
        norm = sb.clip_grads(d, 0.1, out=out, stream=stream)
        torch.cuda.synchronize()
        return [o, lse, *d, y, mean, rstd, *e, *out, norm]

    ref = run(None)
    side = torch.cuda.Stream(device=cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    for stream in (0, side.cuda_stream, side):
        before = torch.cuda.current_stream()
        for a, b in zip(ref, run(stream)):
            assert torch.equal(a, b)
        assert torch.cuda.current_stream() == before
