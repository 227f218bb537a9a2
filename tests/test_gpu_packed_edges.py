"""Packed causal attention on the GPU where it can go wrong beside the
ordinary cases.  Helpers and the tolerances' derivation: test_gpu_packed.py.
"""

import pytest
import torch

from test_gpu_packed import draw, pa  # noqa: F401

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
