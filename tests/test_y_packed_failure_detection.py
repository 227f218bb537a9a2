"""Failure detection of the packed attention on the GPU, without a GPU fault.

As in test_y_failure_detection.py: every device-side wait is bounded, and one
that runs out records SA_ERR_TIMEOUT in the library's status word, lets what
is in flight land and returns.  The library's test build
(libpacked_attn_test.so, the same sources compiled with SA_TEST_HOOKS) gives up
after a few milliseconds and can withhold a producer's first load of one kind in
the CTA that takes the first item: it is never issued, so the roles that wait for
it run out of time, and with them those that wait for these.
"""

import time

import pytest
import torch

from factorized_block_sparse_b200 import build
from test_gpu_packed import draw

pytestmark = pytest.mark.gpu

# the load that stays away: forward Q, V; dK/dV part dO, K and V; dQ part V, Q and dO
FORWARD, BACKWARD = (1, 2), (3, 4, 5, 6)


@pytest.fixture()
def pt(monkeypatch):
    """The binding on the test build."""
    from factorized_block_sparse_b200 import packed_attn as pa

    monkeypatch.setattr(pa, "lib", pa.load_library(build.build_packed_test_lib()))
    yield pa
    pa.lib.packed_attn_test_withhold(0)


@pytest.mark.parametrize("what", FORWARD + BACKWARD)
@pytest.mark.parametrize("lengths,hq,hkv,d", [([700, 300, 129], 8, 4, 64), ([700, 300, 129], 4, 4, 32), ([600, 500], 16, 4, 128),
                                              ([4096], 4, 1, 64)])
def test_withheld_load_times_out_then_recovers(cuda_device, pt, lengths, hq, hkv, d, what):
    from factorized_block_sparse_b200 import sparse_attn as sa

    q, k, v, dO = (t.to(cuda_device) for t in draw(sum(lengths), hq, hkv, d, torch.bfloat16))
    lay = pt.Layout(lengths)
    ws = pt.workspace(hq, hkv, d, lay, cuda_device)

    def run(o, lse):
        return pt.forward(q, k, v, lay) if what in FORWARD else pt.backward(q, k, v, o, lse, dO, lay, ws=ws)

    o, lse = pt.forward(q, k, v, lay)
    want = run(o, lse)
    assert pt.packed_attn_status() == sa.SA_OK
    assert pt.lib.packed_attn_test_withhold(what) == sa.SA_OK
    t0 = time.perf_counter()
    run(o, lse)  # enqueued; the failure shows in the status word
    st = pt.packed_attn_status()
    elapsed = time.perf_counter() - t0
    assert pt.lib.packed_attn_test_withhold(0) == sa.SA_OK
    assert st == sa.SA_ERR_TIMEOUT, sa.strerror(st)
    assert elapsed < 2.0, f"the timeout took {elapsed:.2f} s"
    # reading the status word has cleared it, and the context is usable
    assert pt.packed_attn_status() == sa.SA_OK
    got = run(o, lse)
    assert pt.packed_attn_status() == sa.SA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    lay.close()
