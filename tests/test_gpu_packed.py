"""Packed causal attention on the GPU against the float64 oracle
(oracle.packed), element by element.

Tolerances.  u is half a step of the tensors' type (2^-8 of a value in bf16,
2^-11 in fp16).  Forward: every P is rounded once before its product with v
and o once at the end, so |o - ref| <= u (sum_j P_ij |v_j| + |ref|), plus the
float32 arithmetic: scores, exponential and row sum are good to a few 1e-5 of
P at the score sizes drawn here, taken as 2e-4 sum P |v|.  lse: the float32
scores' error, 2^-24 D max|s| and the logarithm's, taken as 1e-4.  Backward
(from the same rounded o and float32 lse as the oracle gets): dv like o,
u (sum P |dO| + |ref|); dk and dq: dS is rounded once,
u (scale sum |dS| |q| + |ref|), and dP - delta cancels float32 values good to
a few 1e-6 of their terms (|dP|, |delta| <= about 50 here), taken as
5e-4 scale sum P |q|.  In fp16 a rounded P or dS below 2^-14 is off by up to
2^-25 whatever its size: 2^-25 sum |dO| (or scale sum |q|) on top.
"""

import numpy as np
import pytest
import torch

from factorized_block_sparse_b200 import synth
from oracle import packed

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SUB = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}

# lengths, Hq, Hkv, D, dtype
CASES = [
    ([1], 1, 1, 64, torch.bfloat16),
    ([2], 1, 1, 128, torch.float16),
    ([128], 2, 2, 64, torch.bfloat16),
    ([127, 129], 2, 1, 128, torch.bfloat16),
    ([1, 2, 3, 255, 256, 257], 4, 2, 64, torch.float16),
    ([300, 0, 5, 513], 6, 2, 128, torch.bfloat16),
    ([700], 8, 1, 64, torch.bfloat16),
    ([64, 64, 65, 191], 3, 3, 128, torch.float16),
    ([1000, 24], 2, 2, 64, torch.bfloat16),
    ([385, 129, 1], 5, 1, 128, torch.bfloat16),
    ([130, 40], 4, 4, 32, torch.bfloat16),
    ([257, 3, 128], 6, 3, 32, torch.float16),
    ([1] * 40 + [2] * 30, 4, 2, 64, torch.bfloat16),
    ([512, 640], 16, 2, 128, torch.bfloat16),
    # more tiles x heads than SMs: query heads or row tiles of an item in pairs
    ([130, 300, 77] * 6, 8, 4, 128, torch.bfloat16),
    ([130, 257, 300, 128, 1] * 3, 9, 3, 64, torch.float16),
    ([385, 100] * 5, 10, 10, 128, torch.float16),
    ([600, 1, 513], 24, 2, 64, torch.bfloat16),
    ([129, 384] * 6, 6, 6, 32, torch.bfloat16),
    ([700] * 3, 12, 6, 32, torch.float16),
    # few key tiles with many steps each: their steps in parts, some of them empty
    ([900, 300, 40], 6, 2, 128, torch.float16),
    ([1999], 2, 1, 64, torch.bfloat16),
    ([1500], 1, 1, 128, torch.bfloat16),
    ([1100, 3], 4, 1, 32, torch.float16),
]


@pytest.fixture(scope="module")
def pa():
    from factorized_block_sparse_b200 import packed_attn

    return packed_attn


def draw(T, hq, hkv, d, dtype, seed=0, q_scale=1.0):
    mk = lambda h, s, f=1.0: (torch.from_numpy(synth.normal_f32((T, h, d), s + seed)) * f).to(dtype)  # noqa: E731
    return mk(hq, 0, q_scale), mk(hkv, 1), mk(hkv, 2), mk(hq, 3)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(name, got, ref, bound):
    got = f64(got)
    assert np.isfinite(got).all(), name
    over = np.abs(got - ref) - bound
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 0, f"{name}{at}: got {got[at]:.6g}, reference {ref[at]:.6g}, bound {bound[at]:.3g}"


def check_forward(q, k, v, o, lse, lengths, scale=None, lse_tol=1e-4):
    u = U[q.dtype]
    ref, rl, mag = packed.forward(f64(q), f64(k), f64(v), lengths, scale)
    n = sum(lengths)
    check("o", o[:n], ref[:n], u * (mag[:n] + np.abs(ref[:n])) + 2e-4 * mag[:n] + SUB[q.dtype] * 4)
    check("lse", lse[:, :n], rl[:, :n], np.full_like(rl[:, :n], lse_tol))


def check_backward(q, k, v, o, lse, dO, grads, lengths, scale=None):
    u, s = U[q.dtype], SUB[q.dtype]
    dq, dk, dv, m = packed.backward(f64(q), f64(k), f64(v), f64(o), f64(lse), f64(dO), lengths, scale)
    n = sum(lengths)
    for name, got, ref, b in (
            ("dq", grads[0], dq, u * (m["dq_ds"] + np.abs(dq)) + 5e-4 * m["dq_p"] + s * m["dq_n"]),
            ("dk", grads[1], dk, u * (m["dk_ds"] + np.abs(dk)) + 5e-4 * m["dk_p"] + s * m["dk_n"]),
            ("dv", grads[2], dv, u * (m["dv_p"] + np.abs(dv)) + 2e-4 * m["dv_p"] + s * m["dv_n"])):
        # a float32 result rounds to the type's own subnormals near zero
        check(name, got[:n], ref[:n], b[:n] + s + 1e-30)


@pytest.mark.parametrize("lengths,hq,hkv,d,dtype", CASES)
def test_forward_and_backward(cuda_device, pa, lengths, hq, hkv, d, dtype):
    q, k, v, dO = (t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, dtype))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    assert pa.packed_attn_status() == 0
    check_forward(q, k, v, o, lse, lengths)
    grads = pa.backward(q, k, v, o, lse, dO, lay)
    assert pa.packed_attn_status() == 0
    check_backward(q, k, v, o, lse, dO, grads, lengths)
    # every sum has a fixed order: the same bits again
    o2, lse2 = pa.forward(q, k, v, lay)
    again = pa.backward(q, k, v, o, lse, dO, lay)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("scale", [0.02, 0.5])
def test_explicit_scale(cuda_device, pa, scale):
    lengths, hq, hkv, d = [200, 333], 4, 2, 64
    q, k, v, dO = (t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay, scale=scale)
    check_forward(q, k, v, o, lse, lengths, scale)
    check_backward(q, k, v, o, lse, dO, pa.backward(q, k, v, o, lse, dO, lay, scale=scale), lengths, scale)


def test_peaked_rows(cuda_device, pa):
    # scores up to about +-100: rows that one key owns, and a running maximum that moves by much
    lengths = [500]
    q, k, v, dO = (t.to(cuda_device) for t in draw(500, 2, 2, 64, torch.bfloat16, q_scale=16.0))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    # scores of size 100 carry 16 times the float32 error of the unit ones
    check_forward(q, k, v, o, lse, lengths, lse_tol=1e-3)


def _strided(t, how):
    T, h, d = t.shape
    if how == "fused":  # heads of several tensors side by side in a row
        buf = torch.full((T, h + 3, d), float("nan"), dtype=t.dtype, device=t.device)
        out = buf[:, 2:2 + h]
    elif how == "heads-first":
        out = torch.empty((h, T, d), dtype=t.dtype, device=t.device).transpose(0, 1)
    else:  # padded rows and heads
        buf = torch.full((T, h + 1, d + 8), float("nan"), dtype=t.dtype, device=t.device)
        out = buf[:, :h, :d]
    out.copy_(t)
    return out


@pytest.mark.parametrize("how", ["fused", "heads-first", "padded"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_strides(cuda_device, pa, how, d):
    lengths, hq, hkv = [150, 77, 260], 4, 2
    base = [t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16, seed=5)]
    q, k, v, dO = (_strided(t, how) for t in base)
    lay = pa.Layout(lengths)
    ws = pa.workspace(hq, hkv, d, lay, cuda_device)
    o, lse = _strided(torch.zeros_like(base[0]), how), torch.empty((hq, sum(lengths) + 5), device=cuda_device)[:, :-5]
    pa.packed_attn_fwd(q, k, v, o, lse, lay)
    check_forward(q, k, v, o, lse, lengths)
    outs = [_strided(torch.zeros_like(t), how) for t in base[:3]]
    pa.packed_attn_bwd(q, k, v, o, lse, dO, *outs, lay, ws)
    check_backward(q, k, v, o, lse, dO, outs, lengths)
    if how == "padded":  # the gaps between heads and rows were not written
        for t in (o, *outs):
            whole = t._base
            assert torch.isnan(whole[:, -1]).all() and torch.isnan(whole[:, :, d:]).all()


def test_rows_behind_the_last_sequence_stay(cuda_device, pa):
    lengths, T, hq, hkv, d = [130, 61], 230, 4, 2, 64
    q, k, v, dO = (t.to(cuda_device) for t in draw(T, hq, hkv, d, torch.bfloat16))
    n = sum(lengths)
    for t in (q, k, v, dO):
        t[n:] = float("nan")
    lay = pa.Layout(lengths)
    o, lse = torch.full_like(q, 7.0), torch.full((hq, T), 7.0, device=cuda_device)
    pa.packed_attn_fwd(q, k, v, o, lse, lay)
    check_forward(q[:n], k[:n], v[:n], o, lse, lengths)
    outs = [torch.full_like(t, 7.0) for t in (q, k, v)]
    pa.packed_attn_bwd(q, k, v, o, lse, dO, *outs, lay, pa.workspace(hq, hkv, d, lay, cuda_device))
    check_backward(q[:n], k[:n], v[:n], o[:n], lse[:, :n], dO[:n], outs, lengths)
    for t in (o, *outs):
        assert (t[n:] == 7.0).all()
    assert (lse[:, n:] == 7.0).all()
    # the allocating calls leave zeros there
    o2, lse2 = pa.forward(q, k, v, lay)
    assert not o2[n:].any() and not lse2[:, n:].any()
    assert not any(t[n:].any() for t in pa.backward(q, k, v, o, lse, dO, lay))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_sequences_do_not_touch_one_another(cuda_device, pa, d, value):
    # the middle sequence holds values that are not finite; the others come out as without it
    lengths, hq, hkv = [130, 70, 200], 4, 2
    x = [t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16)]
    lay = pa.Layout(lengths)
    o, lse = pa.forward(*x[:3], lay)
    ref = (o, *pa.backward(*x[:3], o, lse, x[3], lay))
    y = [t.clone() for t in x]
    for t in y:
        t[130:200] = value
    o2, lse2 = pa.forward(*y[:3], lay)
    got = (o2, *pa.backward(*y[:3], o2, lse2, y[3], lay))
    for name, a, b in zip(("o", "dq", "dk", "dv"), ref, got):
        for part in (slice(0, 130), slice(200, 400)):
            assert torch.equal(a[part], b[part]), name
    assert torch.equal(lse[:, :130], lse2[:, :130]) and torch.equal(lse[:, 200:], lse2[:, 200:])
    assert pa.packed_attn_status() == 0


def test_later_rows_do_not_reach_earlier_tiles(cuda_device, pa):
    # causality: changing the rows from 256 on changes nothing before them, in o and in no gradient of those rows' own terms
    q, k, v, dO = (t.to(cuda_device) for t in draw(400, 2, 2, 64, torch.bfloat16))
    lay = pa.Layout([400])
    o, lse = pa.forward(q, k, v, lay)
    k2, v2 = k.clone(), v.clone()
    k2[256:] = float("inf")
    v2[256:] = float("nan")
    o2, lse2 = pa.forward(q, k2, v2, lay)
    assert torch.equal(o[:256], o2[:256]) and torch.equal(lse[:, :256], lse2[:, :256])


def test_another_stream_and_two_calls_at_once(cuda_device, pa):
    lengths, hq, hkv, d = [900, 333, 12], 4, 2, 64
    lay = pa.Layout(lengths)
    sets = [[t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16, seed=10 * i)] for i in range(2)]
    want = []
    for x in sets:
        o, lse = pa.forward(*x[:3], lay)
        want.append((o, lse, *pa.backward(*x[:3], o, lse, x[3], lay)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for x, s in zip(sets, streams):
        o, lse = pa.forward(*x[:3], lay, stream=s)
        got.append((o, lse, *pa.backward(*x[:3], o, lse, x[3], lay, stream=s)))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_and_replayed(cuda_device, pa):
    lengths, hq, hkv, d = [300, 129], 4, 2, 128
    lay = pa.Layout(lengths)
    x = [t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16)]
    ws = pa.workspace(hq, hkv, d, lay, cuda_device)
    fresh = pa.Layout(lengths)  # not on the device: refused inside a capture
    lay.upload(cuda_device)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    refused = False
    with torch.cuda.graph(g, stream=s):
        o, lse = pa.forward(*x[:3], lay)
        grads = pa.backward(*x[:3], o, lse, x[3], lay, ws=ws)
        try:
            pa.forward(*x[:3], fresh)
        except Exception as e:  # SparseAttnError
            refused = "status 1" in str(e)
    assert refused
    for seed in (0, 20):
        for t, n in zip(x, draw(sum(lengths), hq, hkv, d, torch.bfloat16, seed=seed)):
            t.copy_(n)
        g.replay()
        torch.cuda.synchronize()
        check_forward(*x[:3], o, lse, lengths)
        check_backward(*x[:3], o, lse, x[3], grads, lengths)
    assert pa.packed_attn_status() == 0


def test_offsets_beyond_32_bits(cuda_device, pa):
    # q and o hold 2^31 elements and more; the last sequence equals the same rows on their own
    hq, hkv, d, T = 128, 1, 64, (1 << 18) + 200
    lengths = [200] * (T // 200)
    lengths.append(T - sum(lengths))
    lengths = [n for n in lengths if n]
    g = torch.Generator(device=cuda_device).manual_seed(1)
    q = torch.empty((T, hq, d), dtype=torch.bfloat16, device=cuda_device).normal_(generator=g)
    k, v = (torch.empty((T, hkv, d), dtype=torch.bfloat16, device=cuda_device).normal_(generator=g) for _ in range(2))
    assert q.numel() > 1 << 31
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    n = lengths[-1] + lengths[-2]
    small = pa.Layout(lengths[-2:])
    o2, lse2 = pa.forward(q[-n:], k[-n:], v[-n:], small)
    assert torch.equal(o[-n:], o2) and torch.equal(lse[:, -n:], lse2)
    dO = q.flip(0)
    dq, dk, dv = pa.backward(q, k, v, o, lse, dO, lay)
    r = pa.backward(q[-n:], k[-n:], v[-n:], o2, lse2, dO[-n:], small)
    assert torch.equal(dq[-n:], r[0])
    # dk and dv: the small call, with few key tiles, takes their sums in parts, so in another order; both against the oracle
    for dkv in ((dk[-n:], dv[-n:]), r[1:]):
        check_backward(q[-n:], k[-n:], v[-n:], o2, lse2, dO[-n:], (dq[-n:], *dkv), lengths[-2:])
    assert pa.packed_attn_status() == 0


def test_refusals_on_the_gpu(cuda_device, pa):
    from factorized_block_sparse_b200 import sparse_attn as sa

    lay = pa.Layout([10])
    q = torch.zeros((10, 2, 64), dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError):
        pa.forward(q.float(), q.float(), q.float(), lay)
    with pytest.raises(ValueError):
        pa.forward(q, q.half(), q.half(), lay)
    with pytest.raises(ValueError):
        pa.forward(q, q.transpose(1, 2).contiguous().transpose(1, 2), q, lay)
    with pytest.raises(sa.SparseAttnError):
        pa.forward(q, q[:, :1].expand(10, 2, 64), q, lay)  # heads that share their memory
    with pytest.raises(sa.SparseAttnError):
        pa.forward(torch.zeros((10, 2, 68), dtype=torch.bfloat16, device=cuda_device)[..., 4:], q, q, lay)
    o, lse = pa.forward(q, q, q, lay)
    with pytest.raises(sa.SparseAttnError):
        pa.packed_attn_fwd(q, q, q, q, lse, lay)
    with pytest.raises(ValueError):
        pa.packed_attn_fwd(q, q, q, o, lse.double(), lay)
    with pytest.raises(sa.SparseAttnError):
        pa.backward(q, q, q, o, lse, q, lay, ws=torch.empty(64, dtype=torch.uint8, device=cuda_device))


def test_a_layout_freed_during_a_capture(cuda_device, pa):
    # a garbage collector may drop another batch's layout at any time: the capture under way stays whole
    lengths, hq, hkv, d = [200, 90], 2, 1, 64
    x = [t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16)]
    lay, other = pa.Layout(lengths), pa.Layout([64, 64])
    lay.upload(cuda_device)
    other.upload(cuda_device)
    want = pa.forward(*x[:3], lay)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        o, lse = pa.forward(*x[:3], lay)
        other.close()
        o2, _ = pa.forward(*x[:3], lay)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(o2, want[0]) and torch.equal(lse, want[1])


def test_a_long_sequence_sampled(cuda_device, pa):
    # 40000 rows in one sequence behind a short one: rows and keys here and there against the oracle's formulas
    lengths, hq, hkv, d = [77, 40000], 2, 1, 64
    q, k, v, dO = (t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    dq, dk, dv = pa.backward(q, k, v, o, lse, dO, lay)
    assert pa.packed_attn_status() == 0
    u, c = U[torch.bfloat16], d ** -0.5
    kk, vv = (t[77:, 0].double() for t in (k, v))
    for h in range(hq):
        qq, gg, oo = (t[77:, h].double() for t in (q, dO, o))
        L = lse[h, 77:].double()
        delta = (gg * oo).sum(-1)
        for i in (0, 127, 128, 20001, 39999):  # a query row
            s = c * (kk[:i + 1] @ qq[i])
            p = torch.exp(s - torch.logsumexp(s, 0))
            ref, mag = p @ vv[:i + 1], p @ vv[:i + 1].abs()
            assert ((o[77 + i, h].double() - ref).abs() <= u * (mag + ref.abs()) + 2e-4 * mag).all()
            assert abs(float(lse[h, 77 + i]) - float(torch.logsumexp(s, 0))) <= 1e-4
            p = torch.exp(s - L[i])
            ds = p * (vv[:i + 1] @ gg[i] - delta[i])
            ref, mag = c * (ds @ kk[:i + 1]), c * (ds.abs() @ kk[:i + 1].abs())
            noise = c * (p @ kk[:i + 1].abs())
            assert ((dq[77 + i, h].double() - ref).abs() <= u * (mag + ref.abs()) + 5e-4 * noise).all()
    for j in (0, 20001, 39990):  # a key: its sums run over both query heads
        ref = {n: torch.zeros(d, dtype=torch.float64, device=cuda_device) for n in ("dk", "dv", "mk", "mv", "nk")}
        for h in range(hq):
            qq, gg, oo = (t[77 + j:, h].double() for t in (q, dO, o))
            p = torch.exp(c * (qq @ kk[j]) - lse[h, 77 + j:].double())
            ds = p * (gg @ vv[j] - (gg * oo).sum(-1))
            for n, t in (("dk", c * (ds @ qq)), ("dv", p @ gg), ("mk", c * (ds.abs() @ qq.abs())), ("mv", p @ gg.abs()),
                         ("nk", c * (p @ qq.abs()))):
                ref[n] += t
        assert ((dk[77 + j, 0].double() - ref["dk"]).abs() <= u * (ref["mk"] + ref["dk"].abs()) + 5e-4 * ref["nk"]).all()
        assert ((dv[77 + j, 0].double() - ref["dv"]).abs() <= u * (ref["mv"] + ref["dv"].abs()) + 2e-4 * ref["mv"]).all()
