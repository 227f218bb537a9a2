"""Tensors that a caller drops behind a call on another stream than their own:
their memory is not handed out while that stream may still use it.  The side
stream is held up by a sleep kernel first, so that the call's work has not run
when the tensors go; nothing is written to the memory that comes back.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

M, C = 4096, 512  # tensors of 4 MB and more: blocks of their own in torch's allocator


@pytest.fixture(scope="module")
def calls():
    """{name: (make inputs, call of them on a stream, which of the inputs are dropped)}"""
    from factorized_block_sparse_b200 import packed_attn as pa
    from factorized_block_sparse_b200 import sparse_block as sb

    lay = pa.Layout([M - 96, 96])

    def qkv(dev):
        return [torch.randn(M, 8, 64, device=dev).to(torch.bfloat16) for _ in range(3)]

    def attn(dev):
        q, k, v = qkv(dev)
        o, lse = pa.forward(q, k, v, lay)
        return [q, k, v, o, lse.repeat(64, 1)[:8], torch.randn_like(q)]

    def rows(dev):
        return [torch.randn(M, C, device=dev), torch.ones(C, device=dev)]

    def norm(dev):
        x, g = rows(dev)
        _, mean, rstd = sb.layer_norm(x, g)
        return [x, g, torch.randn_like(x), mean, rstd]

    def low(i, s):
        o, lse = torch.empty_like(i[0]), torch.empty(8, M, device=i[0].device)
        pa.packed_attn_fwd(*i, o, lse, lay, stream=s)
        return o, lse

    def low_bwd(i, s):
        outs = [torch.empty_like(t) for t in i[:3]]
        pa.packed_attn_bwd(*i, *outs, lay, pa.workspace(8, 8, 64, lay, i[0].device), stream=s)
        return outs

    from factorized_block_sparse_b200 import sparse_attn as sa
    from factorized_block_sparse_b200 import synth

    strided = sa.Layout("strided", M, 64, 0, 64)

    def dense(dev):
        return [torch.randn(1, 8, M, 64, device=dev).to(torch.bfloat16) for _ in range(3)]

    def dense_bwd(dev):
        i = dense(dev)
        o, lse = sa.forward(*i, strided)
        return [*i, o, lse, torch.randn_like(o)]

    def block(dev):
        p = {n: t.to(dev) for n, t in synth.block_params(C).items()}
        return [torch.randn(1, M, C, device=dev).to(torch.bfloat16) for _ in range(2)] + [p]

    return {
        "sparse_attn.forward": (dense, lambda i, s: sa.forward(*i, strided, stream=s), (0, 1, 2)),
        "sparse_attn.backward": (dense_bwd, lambda i, s: sa.backward(*i, strided, stream=s), (0, 1, 2, 3, 5)),
        "block forward": (block, lambda i, s: sb.forward(i[0], i[2], 8, strided, stream=s), (0,)),
        "block backward": (block, lambda i, s: sb.backward(*i, 8, strided, stream=s, max_norm=0.5), (0, 1)),
        "forward": (qkv, lambda i, s: pa.forward(*i, lay, stream=s), (0, 1, 2)),
        "backward": (attn, lambda i, s: pa.backward(*i, lay, stream=s), (0, 1, 2, 3, 4, 5)),
        "packed_attn_fwd": (qkv, low, (0, 1, 2)),
        "packed_attn_bwd": (attn, low_bwd, (0, 1, 2, 3, 4, 5)),
        "layer_norm": (rows, lambda i, s: sb.layer_norm(*i, stream=s), (0,)),
        "layer_norm_backward": (norm, lambda i, s: sb.layer_norm_backward(*i, stream=s), (0, 2)),
        "grad_norm": (rows, lambda i, s: sb.grad_norm(i, stream=s), (0,)),
        "clip_grads": (rows, lambda i, s: sb.clip_grads(i, 0.5, stream=s), (0,)),
    }


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", ["forward", "backward", "packed_attn_fwd", "packed_attn_bwd", "layer_norm",
                                  "layer_norm_backward", "grad_norm", "clip_grads", "sparse_attn.forward",
                                  "sparse_attn.backward", "block forward", "block backward"])
def test_dropped_tensors_keep_their_memory(cuda_device, calls, name, as_handle):
    make, call, which = calls[name]
    side = torch.cuda.Stream(device=cuda_device)
    s = side.cuda_stream if as_handle else side
    with torch.cuda.stream(side):
        call(make(cuda_device), s)  # tables, modules and the stream's own blocks are there before the stream is held up
    torch.cuda.synchronize()
    inputs = make(cuda_device)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(300_000_000)
    out = call(inputs, s)
    gone = {inputs[i].untyped_storage().data_ptr(): inputs[i].untyped_storage().nbytes() for i in which}
    del inputs
    new = [torch.empty(n, dtype=torch.uint8, device=cuda_device) for n in gone.values() for _ in range(2)]
    held = not side.query()
    back = [t for t in new if t.data_ptr() in gone]
    torch.cuda.synchronize()
    assert held  # the call had not run yet
    assert not back
    del out


def test_a_stream_named_inside_its_capture(cuda_device):
    from factorized_block_sparse_b200 import packed_attn as pa
    from factorized_block_sparse_b200 import sparse_block as sb

    lay = pa.Layout([300, 41])
    lay.upload(cuda_device)
    q, k, v, dO = (torch.randn(341, 2, 64, device=cuda_device).to(torch.bfloat16) for _ in range(4))
    g = torch.ones(128, device=cuda_device)

    def run(stream):
        o, lse = pa.forward(q, k, v, lay, stream=stream)
        d = pa.backward(q, k, v, o, lse, dO, lay, stream=stream)
        y, mean, rstd = sb.layer_norm(q.view(341, 128), g, stream=stream)
        e = sb.layer_norm_backward(q.view(341, 128), g, y, mean, rstd, stream=stream)
        out = [torch.empty_like(t) for t in d]
        return [o, lse, *d, y, *e, *out, sb.clip_grads(d, 0.1, out=out, stream=stream)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = run(s)
    for _ in range(2):
        for t in (q, k, v, dO):
            t.copy_(torch.randn_like(t))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(run(None), got))


class _Handle:
    """A stream of another library: nothing but its handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("of", [lambda s: _Handle(s.cuda_stream), lambda s: 1, lambda s: 2, lambda s: 0])
def test_streams_that_are_not_torchs(cuda_device, of):
    # an object with a handle; the legacy default stream by its other name, and the calling thread's default stream
    from factorized_block_sparse_b200 import packed_attn as pa
    from factorized_block_sparse_b200 import sparse_attn as sa
    from factorized_block_sparse_b200 import sparse_block as sb

    side = torch.cuda.Stream(device=cuda_device)
    s = of(side)
    lay, strided = pa.Layout([200, 56]), sa.Layout("strided", 256, 16, 0, 16)
    q, k, v, dO = (torch.randn(256, 2, 64, device=cuda_device).to(torch.bfloat16) for _ in range(4))
    o, lse = pa.forward(q, k, v, lay)
    b = [t.transpose(0, 1).contiguous()[None] for t in (q, k, v, dO)]
    bo, bl = sa.forward(*b[:3], strided)
    want = sa.backward(*b[:3], bo, bl, b[3], strided)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    torch.cuda.synchronize()
    pa.packed_attn_fwd(q, k, v, o2, lse2, lay, stream=s)
    bo2, bl2 = sa.forward(*b[:3], strided, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(bo, bo2) and torch.equal(bl, bl2)
    got = sa.backward(*b[:3], bo, bl, b[3], strided, stream=s)
    torch.cuda.synchronize()
    grads = pa.backward(q, k, v, o, lse, dO, lay)
    x, g = q.reshape(256, 128), torch.ones(128, device=cuda_device)
    norm, total = sb.layer_norm(x, g), sb.grad_norm(grads)
    torch.cuda.synchronize()
    o3, lse3 = pa.forward(q, k, v, lay, stream=s)
    mine = [o3, lse3, *pa.backward(q, k, v, o, lse, dO, lay, stream=s), *sb.layer_norm(x, g, stream=s), sb.grad_norm(grads, stream=s)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((o, lse, *grads, *norm, total), mine))
    assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])  # (dq adds up in any order)
