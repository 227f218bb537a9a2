"""Layer norm and clipping on the GPU where a float32 sum or a 32-bit offset would lose something.
Helpers and the tolerances' derivation: test_gpu_train.py.
"""

import numpy as np
import pytest
import torch

from test_gpu_train import TYPES, check_bwd, check_fwd, f64, sb  # noqa: F401

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


@pytest.mark.parametrize("C,off", [(16384, 0), (16383, 0), (16384, 1)])
def test_layer_norm_beyond_32_bit_offsets(cuda_device, sb, C, off):  # noqa: F811
    # more than 2^31 elements: the first and last rows as on their own, and the rows' sums over all of them
    M = (1 << 31) // C + 3
    buf = torch.empty((M, C + off), dtype=torch.bfloat16, device=cuda_device).normal_()
    x = buf[:, off:]
    assert x.numel() > 1 << 31
    g, b = (torch.linspace(0.5, 1.5, C, device=cuda_device) for _ in range(2))
    y, mean, rstd = sb.layer_norm(x, g, b)
    dx, dg, db = sb.layer_norm_backward(x, g, y, mean, rstd)
    for rows in (slice(0, 3), slice(M - 3, M)):
        check_fwd(x[rows], g, b, y[rows], mean[rows], rstd[rows])
        few = sb.layer_norm_backward(x[rows], g, y[rows], mean[rows], rstd[rows])
        check_bwd(x[rows], g, y[rows], mean[rows], rstd[rows], *few)
        check_bwd(x[rows], g, y[rows], mean[rows], rstd[rows], dx[rows], few[1], few[2])
    # a channel's sum of M terms, by blocks: at most M / 296 + 400 roundings of 2^-24 of its magnitudes
    ref, mag = torch.zeros(C, dtype=torch.float64, device=cuda_device), torch.zeros(C, dtype=torch.float64, device=cuda_device)
    for part in y.split(4096):
        d = part.double()
        ref += d.sum(0)
        mag += d.abs().sum(0)
    assert ((db.double() - ref).abs() <= 2.0 ** -24 * (M / 296 + 400) * mag).all()


def test_clip_beyond_32_bit_counts(cuda_device, sb):  # noqa: F811
    # one gradient of more than 2^32 elements beside a small one; the norm by halves that are far from 32 bits each
    n = (1 << 32) + 12345
    g = [torch.full((n,), 0.5, dtype=torch.bfloat16, device=cuda_device), torch.full((7,), 3.0, device=cuda_device)]
    g[0][-5:] = 4096.0
    ref = np.sqrt((n - 5) * 0.25 + 5 * 4096.0 ** 2 + 7 * 9.0)
    assert abs(float(sb.grad_norm(g).double()) - ref) <= 2.0 ** -23 * ref
    norm = sb.clip_grads(g, ref / 4)
    assert abs(float(norm.double()) - ref) <= 2.0 ** -23 * ref
    assert (g[0][-5:] == 1024.0).all() and (g[0][:100] == 0.125).all() and (g[0][-105:-5] == 0.125).all()
    assert bool((g[0][:-5] == 0.125).all()) and (g[1] - 0.75).abs().max() <= 2.0 ** -22
