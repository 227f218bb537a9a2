"""The norm of all gradients on the GPU where a float32 sum would lose some of it."""

import numpy as np
import pytest
import torch

from test_gpu_train import TYPES, f64, sb  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lead", range(8))
@pytest.mark.parametrize("n", [8, 4096, 100000])
def test_norm_of_one_large_element_among_small_ones(cuda_device, sb, n, lead, dtype):  # noqa: F811
    # One element of every eight is 1 and the others' squares lie just below half a step of float32 at 1: a running float32
    # sum would lose every one of them, 3.5 2^-24 of the norm.  The norm is good to 2^-23: two roundings of 2^-24 in the sum
    # of half a 16-byte word make one in the norm, and its own.
    small = torch.tensor(2.0 ** -12, dtype=dtype) * (1 - 2.0 ** -7)
    g = torch.full((n,), float(small), dtype=dtype)
    g[lead::8] = 1.0
    ref = np.sqrt((f64(g) ** 2).sum())
    assert abs(float(sb.grad_norm([g.to(cuda_device)]).double()) - ref) <= 2.0 ** -23 * ref
