"""The gated product at gates whose exponential leaves binary32's range."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, device, host
from oracle.layer import gated, scaled_product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,k", [(1, 16), (20, 16), (40, 16), (40, 17)])
@pytest.mark.parametrize("up", [1.0, -(2.0 ** 60), 2.0 ** -20])
def test_gates_where_silu_is_tiny(gpu, m, k, up):
    """silu(g) for g down to -120: 2^-122 at -87, subnormal from about -92 on,
    2^-149 at -108. Half steps: the exponential 3, the sum, the reciprocal, two
    products and the two of up: 9, and silu's own last step where it is
    subnormal."""
    g = np.concatenate([np.linspace(-120, -60, 481), np.linspace(-64.5, -63.5, 33)]).astype(np.float32)
    n = len(g)
    a, b = np.zeros((m, k), np.int8), np.zeros((2 * n, k), np.int8)
    a[:, 0] = b[:, 0] = 1
    sa, sb = np.ones(m, np.float32), np.concatenate([g, np.full(n, up, np.float32)])
    out = torch.full((m, n), float("nan"), device="cuda")
    qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out, gated=True)
    want = gated(scaled_product(a, sa, b, sb))
    tol = np.abs(want) * 9 * STEP + 2.0 ** -149 * (abs(up) + 1)
    off = np.abs(host(out) - want) / tol
    assert np.all(off <= 1), (np.argwhere(off > 1)[:4], off.max())
