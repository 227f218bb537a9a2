"""Layer norm and gradient clipping as calls of their own, on the GPU, against
plain float64 formulas.

Tolerances.  u is half a step of the output's type; every output is rounded
to it once.  e = 2^-24 is half a step of float32; a sum of C terms is taken by
threads of at most 32 terms each and a tree of ten levels, below 64 roundings,
so 64 e of the sum of magnitudes bounds it (the statistics' errors enter y, dx
through the same magnitudes).  dg and db add up rows: one rounding a row that
a thread visits (at most 64 in these cases) and 64 for the partial sums, 128 e
of the sum of magnitudes.  The norm is summed in float64 and rounded once to
float32; a clipped gradient takes two float32 roundings and its own.
"""

import numpy as np
import pytest
import torch

from factorized_block_sparse_b200 import synth

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E = 2.0 ** -24
EPS = 1e-5
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def sb():
    from factorized_block_sparse_b200 import sparse_block

    return sparse_block


def f64(t):
    return t.detach().cpu().double().numpy()


def within(name, got, ref, bound):
    got = f64(got)
    assert np.isfinite(got).all(), name
    over = np.abs(got - ref) - bound
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, f"{name}{at}: got {got[at]:.9g}, reference {ref[at]:.9g}, bound {bound[at]:.3g}"


def check_fwd(x, g, b, y, mean, rstd, eps=EPS):
    xd, gd = f64(x), f64(g)
    bd = f64(b) if b is not None else np.zeros_like(gd)
    m = xd.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((xd - m) ** 2).mean(-1, keepdims=True) + eps)
    ref = (xd - m) * r * gd + bd
    a = np.abs(xd).mean(-1, keepdims=True)
    within("mean", mean, m[..., 0], 64 * E * a[..., 0] + 1e-45)
    # the mean's error d enters the variance as d^2, next to 64 roundings of the sum
    d2 = (64 * E * a) ** 2 * r ** 2
    within("rstd", rstd, r[..., 0], ((64 * E + d2) * r)[..., 0])
    slop = 64 * E * ((np.abs(xd) + a) * r * np.abs(gd) + np.abs(bd)) + (64 * E + d2) * np.abs(ref - bd)
    u = U[y.dtype]
    within("y", y, ref, u * np.abs(ref) + (1 + u) * slop + TINY[y.dtype])


def check_bwd(x, g, dy, mean, rstd, dx, dg, db):
    xd, gd, dd = f64(x), f64(g), f64(dy)
    m, r = f64(mean)[..., None], f64(rstd)[..., None]
    xh, t = (xd - m) * r, dd * gd
    C = xd.shape[-1]
    ref = r * (t - t.sum(-1, keepdims=True) / C - xh * ((t * xh).sum(-1, keepdims=True) / C))
    mags = r * (np.abs(t) + np.abs(t).mean(-1, keepdims=True) + np.abs(xh) * np.abs(t * xh).mean(-1, keepdims=True))
    u = U[dx.dtype]
    within("dx", dx, ref, u * np.abs(ref) + (1 + u) * 80 * E * mags + TINY[dx.dtype])
    flat = lambda z: z.reshape(-1, C)  # noqa: E731
    within("dg", dg, flat(dd * xh).sum(0), 130 * E * flat(np.abs(dd * xh)).sum(0) + 1e-45)
    if db is not None:
        within("db", db, flat(dd).sum(0), 128 * E * flat(np.abs(dd)).sum(0) + 1e-45)


def draw(M, C, dtype, pad, device, seed=0):
    x = torch.from_numpy(synth.normal_f32((M, C + pad), 40 + seed) * 1.5 + 0.25).to(dtype).to(device)[:, :C]
    dy = torch.from_numpy(synth.normal_f32((M, C + pad), 41 + seed)).to(dtype).to(device)[:, :C]
    g = torch.from_numpy(1.0 + 0.1 * synth.normal_f32((C,), 42 + seed)).to(device)
    b = torch.from_numpy(0.1 * synth.normal_f32((C,), 43 + seed)).to(device)
    return x, dy, g, b


# every width path: a warp or a block a row, one to four words a thread, odd widths, widths read again per pass
SHAPES = [(1, 1, 0), (3, 2, 0), (5, 31, 0), (7, 33, 3), (1, 64, 0), (9, 100, 4), (130, 128, 0), (33, 136, 8), (64, 255, 0),
          (300, 256, 0), (17, 512, 0), (40, 520, 24), (3, 1001, 0), (50, 1024, 0), (21, 1032, 0), (11, 2048, 0),
          (6, 2047, 1), (9, 2049, 0), (5, 4096, 0), (4, 4104, 16), (3, 6143, 0), (7, 6144, 0), (2, 6145, 0), (5, 8192, 0),
          (3, 8200, 0), (2, 16384, 0), (2, 16383, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C,pad", SHAPES)
def test_layer_norm(cuda_device, sb, M, C, pad, dtype):
    x, dy, g, b = draw(M, C, dtype, pad, cuda_device)
    y, mean, rstd = sb.layer_norm(x, g, b)
    check_fwd(x, g, b, y, mean, rstd)
    dx, dg, db = sb.layer_norm_backward(x, g, dy, mean, rstd)
    check_bwd(x, g, dy, mean, rstd, dx, dg, db)
    # without a bias, and the same bits again
    y0, _, _ = sb.layer_norm(x, g)
    check_fwd(x, g, None, y0, mean, rstd)
    dx2, dg2, none = sb.layer_norm_backward(x, g, dy, mean, rstd, bias=False)
    assert none is None and torch.equal(dx, dx2) and torch.equal(dg, dg2)


@pytest.mark.parametrize("M,C,pad", [(4000, 768, 0), (4000, 765, 0), (3600, 1000, 1), (2500, 2968, 8), (2500, 2967, 2),
                                     (1200, 4095, 1), (1100, 6144, 0), (1100, 6143, 1), (700, 8192, 0), (500, 9000, 3)])
def test_many_wide_rows(cuda_device, sb, M, C, pad):
    # several rows a block, so that the rings go round; what lies between the rows is NaN.  A column's sum runs over at
    # most 27 rows of a block, then 37 blocks' sums of a group and the 32 groups: under check_bwd's 128 roundings.
    x, dy, g, b = draw(M, C, torch.bfloat16, pad, cuda_device)
    if pad:
        for t in (x, dy):
            t.as_strided((M, pad), (C + pad, 1), t.storage_offset() + C).fill_(float("nan"))
    y, mean, rstd = sb.layer_norm(x, g, b)
    check_fwd(x, g, b, y, mean, rstd)
    out = sb.layer_norm_backward(x, g, dy, mean, rstd)
    check_bwd(x, g, dy, mean, rstd, *out)


@pytest.mark.parametrize("M,C", [(20000, 64), (9001, 512), (5000, 1001), (3000, 2048)])
def test_many_rows(cuda_device, sb, M, C):
    x, dy, g, b = draw(M, C, torch.bfloat16, 0, cuda_device)
    y, mean, rstd = sb.layer_norm(x, g, b)
    check_fwd(x, g, b, y, mean, rstd)
    out = sb.layer_norm_backward(x, g, dy, mean, rstd)
    check_bwd(x, g, dy, mean, rstd, *out)
    again = sb.layer_norm_backward(x, g, dy, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(out, again))


def test_rows_far_from_zero_constant_rows_and_eps(cuda_device, sb):
    x, dy, g, b = draw(16, 384, torch.float32, 0, cuda_device)
    y, mean, rstd = sb.layer_norm(x + 1000.0, g, b)
    check_fwd(x + 1000.0, g, b, y, mean, rstd)
    c = torch.full((4, 384), 3.0, device=cuda_device)
    y, mean, rstd = sb.layer_norm(c, g, b, eps=1e-3)
    assert torch.equal(y, b.expand(4, 384)) and (mean == 3.0).all()
    within("rstd", rstd, np.full(4, 1e-3 ** -0.5), np.full(4, 1e-5))
    y, _, _ = sb.layer_norm(x, g, b, eps=0.0)
    assert torch.isfinite(y).all()


def test_a_row_that_is_not_finite_stays_alone(cuda_device, sb):
    for C in (96, 1001, 2048):
        x, dy, g, b = draw(9, C, torch.bfloat16, 0, cuda_device)
        y, _, _ = sb.layer_norm(x, g, b)
        x2 = x.clone()
        x2[4, 0] = float("inf")
        y2, _, _ = sb.layer_norm(x2, g, b)
        rest = [0, 1, 2, 3, 5, 6, 7, 8]
        assert torch.equal(y[rest], y2[rest]) and torch.isnan(y2[4]).any()


def test_shapes_strides_and_places(cuda_device, sb):
    x, dy, g, b = draw(24, 96, torch.bfloat16, 0, cuda_device)
    want = sb.layer_norm(x, g, b)
    got = sb.layer_norm(x.view(2, 3, 4, 96), g, b)
    assert got[0].shape == (2, 3, 4, 96) and got[1].shape == (2, 3, 4)
    assert torch.equal(got[0].view(24, 96), want[0]) and torch.equal(got[2].view(24), want[2])
    one = sb.layer_norm(x[0], g, b)  # a single row without leading dimensions
    assert one[1].shape == () and torch.equal(one[0], want[0][0])
    every = sb.layer_norm(x[::3], g, b)  # rows at a larger stride
    assert torch.equal(every[0], want[0][::3])
    # columns of a wider tensor whose rows start at odd elements
    wide = torch.zeros((24, 131), dtype=torch.bfloat16, device=cuda_device)
    wide[:, 33:129] = x
    got = sb.layer_norm(wide[:, 33:129], g, b)
    check_fwd(x, g, b, *got)
    back = sb.layer_norm_backward(wide[:, 33:129], g, dy, want[1], want[2])
    check_bwd(x, g, dy, want[1], want[2], *back)
    # no rows
    y, mean, _ = sb.layer_norm(x[:0], g, b)
    assert y.shape == (0, 96) and mean.shape == (0,)
    _, dg, db = sb.layer_norm_backward(x[:0], g, dy[:0], want[1][:0], want[2][:0])
    assert not dg.any() and not db.any()
    # a stream of its own
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sb.layer_norm(x, g, b, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0])


def test_layer_norm_in_place(cuda_device, sb):
    from factorized_block_sparse_b200 import sparse_attn as sa

    for C in (96, 1024, 1001, 8200):
        x, dy, g, b = draw(20, C, torch.float16, 0, cuda_device)
        x, dy = x.contiguous(), dy.contiguous()
        y, mean, rstd = sb.layer_norm(x, g, b)
        dx, dg, db = sb.layer_norm_backward(x, g, dy, mean, rstd)
        s = sa._stream_ptr(None)
        z = x.clone()
        assert sb.lib.sparse_block_layer_norm_fwd(sa._ptr(z), C, sa._ptr(g), sa._ptr(b), sa._ptr(z), C, None, None, 20, C,
                                                  EPS, 1, s) == 0
        assert torch.equal(z, y)
        ws = torch.empty(sb.lib.sparse_block_layer_norm_bwd_workspace_size(20, C), dtype=torch.uint8, device=cuda_device)
        for into in (0, 1):
            zx, zd = x.clone(), dy.clone()
            dst = (zx, zd)[into]
            assert sb.lib.sparse_block_layer_norm_bwd(sa._ptr(zx), C, sa._ptr(g), sa._ptr(zd), C, sa._ptr(mean),
                                                      sa._ptr(rstd), sa._ptr(dst), C, sa._ptr(dg), sa._ptr(db), 20, C, 1,
                                                      sa._ptr(ws), ws.numel(), s) == 0
            assert torch.equal(dst, dx)


def test_layer_norm_gradients_equal_differences(cuda_device, sb):
    x, dy, g, b = draw(2, 5, torch.float32, 0, cuda_device)
    x, dy = x.contiguous(), dy.contiguous()
    _, mean, rstd = sb.layer_norm(x, g, b)
    dx, dg, db = sb.layer_norm_backward(x, g, dy, mean, rstd)

    def loss(xd, gd, bd):
        m = xd.mean(-1, keepdims=True)
        r = 1.0 / np.sqrt(((xd - m) ** 2).mean(-1, keepdims=True) + EPS)
        return (((xd - m) * r * gd + bd) * f64(dy)).sum()

    args = [f64(x), f64(g), f64(b)]
    for a, grad in zip(args, (dx, dg, db)):
        for i in np.ndindex(a.shape):
            keep, h = a[i], 1e-5
            a[i] = keep + h
            up = loss(*args)
            a[i] = keep - h
            dn = loss(*args)
            a[i] = keep
            # differences in float64 are good to about 1e-9, the float32 gradients to about 1e-5
            assert abs((up - dn) / (2 * h) - float(f64(grad)[i])) <= 2e-5 * max(1.0, abs(float(f64(grad)[i])))


# ------------------------------------------------------------------ clipping
def grads_of(sizes, types, device, scale=1.0, seed=0):
    return [(torch.from_numpy(synth.normal_f32((n,), 60 + seed + i)) * (scale * 10.0 ** -(i % 4))).to(types[i % len(types)]).to(device)
            for i, n in enumerate(sizes)]


def check_clip(sb, grads, max_norm, norm_rtol=2.0 ** -23):
    ref = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    c = min(1.0, max_norm / (ref + 1e-6))
    n0 = sb.grad_norm(grads)
    assert n0.shape == () and abs(float(n0.double()) - ref) <= norm_rtol * ref
    outs = [torch.full_like(g, 9.0) for g in grads]
    keep = [g.clone() for g in grads]
    n1 = sb.clip_grads(grads, max_norm, out=outs)
    assert torch.equal(n0, n1)
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))  # gradients as they were
    for g, o in zip(grads, outs):
        if g.numel():
            r = f64(g) * c
            within("clipped", o, r, (U[g.dtype] + 2 ** -22) * np.abs(r) + TINY[g.dtype])
    n2 = sb.clip_grads(grads, max_norm)  # in place
    assert torch.equal(n0, n2)
    assert all(torch.equal(a, b) for a, b in zip(outs, grads))


@pytest.mark.parametrize("types", [[torch.float32], [torch.bfloat16], [torch.float16], TYPES])
@pytest.mark.parametrize("factor", [0.25, 4.0])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], [16384, 16385, 8, 100003], [7] * 130, [1 << 20, 3, 1 << 18],
                                   list(range(1, 260))])
def test_clip(cuda_device, sb, sizes, types, factor):
    grads = grads_of(sizes, types, cuda_device)
    ref = float(np.sqrt(sum((f64(g) ** 2).sum() for g in grads)))
    check_clip(sb, grads, ref * factor)


def test_clip_misaligned_and_shaped(cuda_device, sb):
    base = grads_of([4099], [torch.bfloat16], cuda_device)[0]
    grads = [base[1:2000].clone(), base[2001:4099]]
    grads[0] = base.clone()[1:2000]  # starts two bytes off a 16-byte boundary
    check_clip(sb, grads, 0.5)
    d = {"w": torch.ones((3, 4, 5), device=cuda_device), "b": torch.zeros((), device=cuda_device)}
    n = sb.clip_grads(d, 1.0)
    assert abs(float(n) - 60 ** 0.5) < 1e-5 and torch.allclose(d["w"], torch.full_like(d["w"], 60 ** -0.5))


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_clip_sums_do_not_overflow_or_vanish(cuda_device, sb, scale):
    grads = [t * scale for t in grads_of([1000, 4096, 50], [torch.float32, torch.bfloat16], cuda_device)]
    check_clip(sb, grads, scale)


def test_clip_outputs_by_name(cuda_device, sb):
    # dicts whose names come in different orders, of one shape
    a, b = grads_of([300, 300], [torch.float32], cuda_device)
    out = {"b": torch.empty_like(b), "a": torch.empty_like(a)}
    norm = sb.clip_grads({"a": a, "b": b}, 0.5, out=out)
    same = [torch.empty_like(a), torch.empty_like(b)]
    assert torch.equal(norm, sb.clip_grads([a, b], 0.5, out=same))
    assert torch.equal(out["a"], same[0]) and torch.equal(out["b"], same[1])
    with pytest.raises(ValueError):
        sb.clip_grads({"a": a, "b": b}, 0.5, out={"a": same[0], "c": same[1]})


def test_clip_values_that_are_not_finite(cuda_device, sb):
    g = [torch.ones(100, device=cuda_device), torch.ones(10, dtype=torch.bfloat16, device=cuda_device)]
    g[0][7] = float("inf")
    n = sb.clip_grads(g, 1.0)
    assert torch.isinf(n) and torch.isnan(g[0][7]) and (g[0][:7] == 0).all() and (g[1] == 0).all()
    g[1][3] = float("nan")
    n = sb.clip_grads(g, 1.0)
    assert torch.isnan(n) and torch.isnan(g[0]).all() and torch.isnan(g[1]).all()
    z = [torch.zeros(33, device=cuda_device)]
    assert float(sb.clip_grads(z, 1.0)) == 0.0 and not z[0].any()
    z[0] += 1.0
    sb.clip_grads(z, 0.0)
    assert not z[0].any()


def test_clip_captured_replayed_and_two_at_once(cuda_device, sb):
    g = grads_of([5000, 70001], [torch.float32], cuda_device)
    o = [torch.empty_like(t) for t in g]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        n = sb.clip_grads(g, 1.0, out=o)
        x = sb.layer_norm(g[0].view(50, 100), g[1][:100].contiguous())
    for k in (1.0, 3.0):
        for t, f in zip(g, grads_of([5000, 70001], [torch.float32], cuda_device, scale=k)):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        ref = np.sqrt(sum((f64(t) ** 2).sum() for t in g))
        assert abs(float(n.double()) - ref) <= 2 ** -23 * ref
        check_fwd(g[0].view(50, 100), g[1][:100], None, *x)
    a, b = grads_of([300000], [torch.float32], cuda_device), grads_of([400000], [torch.float32], cuda_device, seed=9)
    want = [sb.grad_norm(a), sb.grad_norm(b)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [sb.grad_norm(x, stream=q) for x, q in zip((a, b), ss)]
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_refusals(cuda_device, sb):
    from factorized_block_sparse_b200 import sparse_attn as sa

    x, dy, g, b = draw(4, 96, torch.bfloat16, 0, cuda_device)
    for call in (lambda: sb.layer_norm(x.double(), g), lambda: sb.layer_norm(x, g[:95]), lambda: sb.layer_norm(x, g.half()),
                 lambda: sb.layer_norm(x.cpu(), g), lambda: sb.layer_norm(x.t(), g), lambda: sb.layer_norm(x[:1].expand(4, 96), g),
                 lambda: sb.layer_norm_backward(x, g, dy.float(), x[:, 0].float(), x[:, 0].float()),
                 lambda: sb.layer_norm_backward(x, g, dy, x[:, 0], x[:, 0]),
                 lambda: sb.clip_grads([], 1.0), lambda: sb.clip_grads([x.t()], 1.0), lambda: sb.clip_grads([x.long()], 1.0),
                 lambda: sb.clip_grads([x], 1.0, out=[x.float()]), lambda: sb.clip_grads([x], 1.0, out=[])):
        with pytest.raises(ValueError):
            call()
    x = x.contiguous()
    for call in (lambda: sb.layer_norm(x, g, eps=-1.0), lambda: sb.layer_norm(x, g, eps=float("nan")),
                 lambda: sb.layer_norm(torch.zeros((2, 16385), device=cuda_device), torch.zeros(16385, device=cuda_device)),
                 lambda: sb.clip_grads([x], -1.0), lambda: sb.clip_grads([x], float("nan")),
                 lambda: sb.clip_grads([x, x], 1.0),                      # the same gradient twice, in place
                 lambda: sb.clip_grads([x[0], x[1]], 1.0, out=[x[1], x[0]]),
                 lambda: sb.clip_grads([x[:2], x[2:]], 1.0, out=[x[1:3], x[2:]])):
        with pytest.raises(sa.SparseAttnError):
            call()
    # the same gradient twice counts twice where nothing is written
    assert abs(float(sb.grad_norm([x, x])) ** 2 - 2 * float((x.float() ** 2).sum())) < 1e-2


def test_block_backward_with_clipping(cuda_device, sb):
    from factorized_block_sparse_b200 import sparse_attn as sa

    B, N, H, D = 1, 256, 2, 64
    xin, p = synth.block_inputs(B, N, H * D), synth.block_params(H * D)
    lay = sa.Layout("strided", N, 16, 0, 16)
    x, dy = xin["x"].to(cuda_device), xin["dy"].to(cuda_device)
    pd = {k: v.to(cuda_device) for k, v in p.items()}
    dx, g = sb.backward(x, dy, pd, H, lay)
    dx2, g2, norm = sb.backward(x, dy, pd, H, lay, max_norm=0.5)
    ref = np.sqrt(sum((f64(t) ** 2).sum() for t in g.values()))
    # the block's gradient sums may differ in their last bits from run to run
    assert abs(float(norm) - ref) <= 1e-3 * ref
    assert abs(np.sqrt(sum((f64(t) ** 2).sum() for t in g2.values())) - 0.5) <= 1e-3
