"""Packed causal attention on the GPU where it can go wrong beside the
ordinary cases.  Helpers and the tolerances' derivation: test_gpu_packed.py.
"""

import pytest
import torch

from test_gpu_packed import check_backward, check_forward, draw, pa  # noqa: F401

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
