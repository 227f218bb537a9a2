"""Packed causal attention on the GPU where it can go wrong beside the
ordinary cases.  Helpers and the tolerances' derivation: test_gpu_packed.py.
"""

import numpy as np
import pytest
import torch

from oracle import packed
from test_gpu_packed import SUB, U, check, check_backward, check_forward, draw, f64, pa  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lengths,hq,hkv,d", [([3000, 1100, 77], 8, 8, 64), ([2500, 900], 8, 2, 32), ([4096], 4, 1, 64),
                                              ([700] * 20, 6, 2, 64), ([2000, 129], 8, 4, 128)])
def test_backward_under_memory_traffic(cuda_device, pa, lengths, hq, hkv, d, dtype):  # noqa: F811
    # Loads come late and the warps of a step drift apart while another stream keeps HBM busy.  No order of theirs may
    # change a result or run out of time: the same bits as on a quiet device.
    q, k, v, dO = (t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, dtype))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    want = pa.backward(q, k, v, o, lse, dO, lay)
    torch.cuda.synchronize()
    a, b = (torch.zeros(1 << 27, device=cuda_device) for _ in range(2))
    side = torch.cuda.Stream()
    ws = pa.workspace(hq, hkv, d, lay, cuda_device)
    got = []
    for i in range(16):
        with torch.cuda.stream(side):
            torch.add(a, 1.0, out=b) if i % 2 else a.copy_(b)
        got.append(pa.backward(q, k, v, o, lse, dO, lay, ws=ws))
    assert pa.packed_attn_status() == 0
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(want, g))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lengths,hq,hkv,first", [([500], 2, 2, 128), ([500], 1, 1, 256), ([390, 520] * 8, 8, 4, 256),
                                                  ([390, 131] * 8, 9, 9, 128)])
def test_first_key_tiles_without_weight(cuda_device, pa, lengths, hq, hkv, d, dtype, first):  # noqa: F811
    # Rows from `first` on score -inf on every key before `first`: their whole first key tiles have no weight, and the
    # result is that of the later keys alone.  Rows before `first` see nothing but -inf; they are not looked at.
    q, k, v, _ = draw(sum(lengths), hq, hkv, d, dtype)
    q[..., 0] = q[..., 0].abs() + 0.5
    at = 0
    for n in lengths:
        k[at:at + min(first, n), :, 0] = float("-inf")
        at += n
    lay = pa.Layout(lengths)
    q, k, v = (t.to(cuda_device) for t in (q, k, v))
    o, lse = pa.forward(q, k, v, lay)
    assert pa.packed_attn_status() == 0
    at = 0
    for n in lengths:
        if n > first:  # the later keys as a sequence of their own
            part = slice(at + first, at + n)
            check_forward(q[part], k[part], v[part], o[part], lse[:, part], [n - first])
        at += n


@pytest.mark.parametrize("d", [32, 64, 128])
def test_products_that_leave_float32(cuda_device, pa, d):  # noqa: F811
    # finite bf16 values, scores of -2^140 on the first 256 keys for the rows from 256 on: no weight, forward and backward
    lengths, hq, hkv = [700], 4, 2
    q, k, v, dO = draw(700, hq, hkv, d, torch.bfloat16)
    q[:256, :, 0], k[256:, :, 0] = 0.0, 0.0
    q[256:, :, 0], k[:256, :, 0] = 2.0 ** 70, -2.0 ** 70
    q, k, v, dO = (t.to(cuda_device) for t in (q, k, v, dO))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    check_forward(q, k, v, o, lse, lengths)
    check_backward(q, k, v, o, lse, dO, pa.backward(q, k, v, o, lse, dO, lay), lengths)
    assert pa.packed_attn_status() == 0


# sizes of dO, v, q, k
FP16_SIZES = [(2.0 ** -13, 1.0, 2.0 ** -4, 2.0 ** 4), (2.0 ** -13, 1.0, 2.0 ** 4, 2.0 ** -4),
              (2.0 ** -16, 1.0, 2.0 ** -4, 2.0 ** 4), (2.0 ** -16, 2.0 ** -5, 2.0 ** 5, 2.0 ** -5),
              (2.0 ** 8, 2.0 ** 8, 2.0 ** -3, 2.0 ** -3), (0.0, 1.0, 1.0, 1.0)]


@pytest.mark.parametrize("lengths,hq,hkv,d", [([1500, 40], 2, 2, 64), ([1999], 2, 1, 64), ([1300, 300], 4, 2, 128),
                                              ([1100], 2, 1, 32)])
@pytest.mark.parametrize("f,fv,fq,fk", FP16_SIZES)
def test_fp16_gradients_of_any_size(cuda_device, pa, lengths, hq, hkv, d, f, fv, fq, fk):  # noqa: F811
    # dS keeps its relative precision whatever the size of dO and v: the factor of a sequence and K/V head takes the
    # bound 2 max|dO_i| max|v_j| of |dS| to [2^14, 2^15), so a dS that rounds to a subnormal is off by at most
    # 2^-25 2 max|dO_i| max|v_j| / 2^14.  P is scaled by 2^12.  The other terms as at the head of test_gpu_packed.py, the
    # cancellation of dP - delta as 1e-5 of the largest term.
    q, k, v, dO = draw(sum(lengths), hq, hkv, d, torch.float16)
    q, k, v, dO = ((t.float() * s).half().to(cuda_device) for t, s in ((q, fq), (k, fk), (v, fv), (dO, f)))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    grads = pa.backward(q, k, v, o, lse, dO, lay)
    assert pa.packed_attn_status() == 0
    x = [f64(t) for t in (q, k, v, o, lse, dO)]
    *ref, m = packed.backward(*x, lengths)
    vv = np.repeat(x[2], hq // hkv, axis=1)
    term = max(float(np.abs(x[5][:, h] @ vv[:, h].T).max()) for h in range(hq))
    sub = 2.0 ** -38 * np.sqrt((x[5] ** 2).sum(-1)).max() * np.sqrt((x[2] ** 2).sum(-1)).max()
    u, tiny = U[torch.float16], 2.0 ** -25
    for name, got, r, ds, p, n in (("dq", grads[0], ref[0], "dq_ds", "dq_p", "dq_n"), ("dk", grads[1], ref[1], "dk_ds", "dk_p", "dk_n")):
        check(name, got, r, u * (m[ds] + np.abs(r)) + 1e-5 * term * m[p] + sub * m[n] + tiny)
    r = ref[2]
    check("dv", grads[2], r, u * (m["dv_p"] + np.abs(r)) + 2e-4 * m["dv_p"] + 2.0 ** -37 * m["dv_n"] + tiny)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 60000.0])
def test_fp16_factors_stay_in_their_sequence(cuda_device, pa, value):  # noqa: F811
    # small gradients beside a sequence of large ones, or of values that are not finite: the same bits as without it
    lengths, hq, hkv, d = [130, 70, 200], 4, 2, 64
    q, k, v, dO = draw(sum(lengths), hq, hkv, d, torch.float16)
    x = [t.to(cuda_device) for t in (q, k, v, dO * 2.0 ** -10)]
    lay = pa.Layout(lengths)
    o, lse = pa.forward(*x[:3], lay)
    ref = pa.backward(*x[:3], o, lse, x[3], lay)
    y = [t.clone() for t in x]
    for t in y[2:]:
        t[130:200] = value
    got = pa.backward(*y[:3], o, lse, y[3], lay)
    for a, b in zip(ref, got):
        for part in (slice(0, 130), slice(200, 400)):
            assert torch.equal(a[part], b[part])
    # a row of the same sequence that is not finite costs the others nothing either
    z = x[3].clone()
    z[399] = float("inf")
    late = pa.backward(*x[:3], o, lse, z, lay)
    assert torch.equal(late[0][:399], ref[0][:399])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_peaked_rows_backward(cuda_device, pa, d, dtype):  # noqa: F811
    # Scores up to about +-100: masked keys far above the row's lse, P of a row on one key.  A score is a float32 sum of d
    # products, off by at most a step of 2^-23 an addition of the sum of magnitudes, and P by that factor (and 1e-4 for
    # the exponential); dP - delta as at the head of test_gpu_packed.py, 1e-5 of the largest term.
    lengths = [300, 77, 500]
    q, k, v, dO = (t.to(cuda_device) for t in draw(sum(lengths), 4, 2, d, dtype, q_scale=16.0))
    lay = pa.Layout(lengths)
    o, lse = pa.forward(q, k, v, lay)
    grads = pa.backward(q, k, v, o, lse, dO, lay)
    assert pa.packed_attn_status() == 0
    x = [f64(t) for t in (q, k, v, o, lse, dO)]
    *ref, m = packed.backward(*x, lengths)
    qa, ka = np.abs(x[0]), np.repeat(np.abs(x[1]), 2, axis=1)
    size = max(float((qa[:, h] @ ka[:, h].T).max()) for h in range(4)) * d ** -0.5
    p_err = 2.0 ** -23 * d * size + 1e-4
    vv = np.repeat(x[2], 2, axis=1)
    term = max(float(np.abs(x[5][:, h] @ vv[:, h].T).max()) for h in range(4))
    u, s = U[dtype], SUB[dtype]
    for name, got, r, ds, p, n in (("dq", grads[0], ref[0], "dq_ds", "dq_p", "dq_n"), ("dk", grads[1], ref[1], "dk_ds", "dk_p", "dk_n")):
        check(name, got, r, u * (m[ds] + np.abs(r)) + p_err * m[ds] + 1e-5 * term * m[p] + s * m[n] + s + 1e-30)
    check("dv", grads[2], ref[2], u * (m["dv_p"] + np.abs(ref[2])) + p_err * m["dv_p"] + s * m["dv_n"] + s + 1e-30)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_causality_of_the_backward_pass(cuda_device, pa, d):  # noqa: F811
    # From the same o, lse and dO: keys and values from row 256 on reach no gradient before row 256, and queries and
    # upstream gradients before row 256 none from there on, whatever they hold.
    q, k, v, dO = (t.to(cuda_device) for t in draw(400, 4, 2, d, torch.bfloat16))
    lay = pa.Layout([400])
    o, lse = pa.forward(q, k, v, lay)
    want = pa.backward(q, k, v, o, lse, dO, lay)
    k2, v2, q2, g2 = k.clone(), v.clone(), q.clone(), dO.clone()
    k2[256:], v2[256:] = float("inf"), float("nan")
    q2[:256], g2[:256] = float("nan"), float("inf")
    late = pa.backward(q, k2, v2, o, lse, dO, lay)
    early = pa.backward(q2, k, v, o, lse, g2, lay)
    for name, a, b, c in zip(("dq", "dk", "dv"), want, late, early):
        assert torch.equal(a[:256], b[:256]), name
        assert torch.equal(a[256:], c[256:]), name


@pytest.mark.parametrize("lengths", [[], [0, 0]])
@pytest.mark.parametrize("T", [0, 5])
def test_packings_without_rows(cuda_device, pa, lengths, T):  # noqa: F811
    # nothing to do: rows behind the last sequence are zero, and a workspace is still given
    lay = pa.Layout(lengths)
    q, k, dO = (torch.full((T, h, 64), float("nan"), dtype=torch.bfloat16, device=cuda_device) for h in (4, 2, 4))
    o, lse = pa.forward(q, k, k, lay)
    assert o.shape == q.shape and lse.shape == (4, T) and not o.any() and not lse.any()
    grads = pa.backward(q, k, k, o, lse, dO, lay)
    assert [g.shape for g in grads] == [q.shape, k.shape, k.shape] and not any(g.any() for g in grads)
    assert pa.workspace(4, 2, 64, lay, cuda_device).numel() > 0 and pa.packed_attn_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_one_row_one_head_and_values_for_keys(cuda_device, pa, d, dtype):  # noqa: F811
    # strides of extents of 1 are not looked at, and one tensor may be k and v
    lay = pa.Layout([1])
    buf = torch.randn(1 + 3 * 1024, device=cuda_device).to(dtype)
    q = buf[:d].as_strided((1, 1, d), (3, 5, 1))
    k = buf[1024:1024 + d].as_strided((1, 1, d), (1, 7, 1))
    dO = torch.randn(1, 1, d, device=cuda_device).to(dtype)
    o, lse = pa.forward(q, k, k, lay)
    check_forward(q, k, k, o, lse, [1])
    check_backward(q, k, k, o, lse, dO, pa.backward(q, k, k, o, lse, dO, lay), [1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_two_graphs_of_one_workspace_in_turn(cuda_device, pa, dtype):  # noqa: F811
    # replayed one behind the other they may share it; each replay starts from whatever the other left there
    sets = [([700, 130], 8, 2, 64), ([2100], 2, 1, 64)]
    lays = [pa.Layout(s[0]) for s in sets]
    n = max(pa.workspace(*s[1:], lay, cuda_device).numel() for s, lay in zip(sets, lays))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=cuda_device)
    x, want, graphs = [], [], []
    for (lengths, hq, hkv, d), lay in zip(sets, lays):
        t = [t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, dtype)]
        o, lse = pa.forward(*t[:3], lay)
        x.append((t, o, lse))
        want.append(pa.backward(*t[:3], o, lse, t[3], lay))
    s = torch.cuda.Stream()
    for (t, o, lse), lay in zip(x, lays):
        g = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            out = pa.backward(*t[:3], o, lse, t[3], lay, ws=ws)
        graphs.append((g, out))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[i], graphs[i][1]))
    assert pa.packed_attn_status() == 0
