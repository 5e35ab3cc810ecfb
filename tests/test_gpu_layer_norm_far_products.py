"""GPU parity of the layer norm's gradients where weight * grad_y is beyond
binary32's range, above or below, and the gradients themselves are not."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import TORCH, device, host, values
from oracle.blocks import layer_norm_backward
from oracle.layer import round_to
from test_gpu_layer_norm import _tolerances

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("w_exp,dy_exp,s_exp", [(70, 70, 60), (100, 29, 40), (-80, -80, -45), (-60, -95, -49), (-75, -75, -20),
                                                (-70, -56, -30), (-20, -100, 0)])
@pytest.mark.parametrize("t,h", [(3, 100), (40, 1024), (300, 4096), (9, 8192), (3, 16384)])
def test_products_beyond_binary32(gpu, t, h, w_exp, dy_exp, s_exp, kind):
    """Rows of such products beside rows of ordinary ones and of zeros."""
    rng = np.random.default_rng([t, h, w_exp + 128])
    size = lambda n: np.float32(2.0 ** n)
    s, dy, w = (values(rng, shape, kind) * size(n) for shape, n in (((t, h), s_exp), ((t, h), dy_exp), (h, w_exp)))
    dy[1] = 0
    s[2] = s[2] * size(-s_exp)  # about one
    s, dy, w = (round_to(v, kind) for v in (s, dy, w))
    gx = torch.full((t, h), 7.0, dtype=TORCH[kind], device="cuda")
    gw, gb = torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    eps = 2.0 ** -126
    qrs.layer_norm_backward(device(dy, kind), device(s, kind), device(w, kind), eps, None, gx, gw, gb)
    want = layer_norm_backward(dy, s, w, eps)
    # What is past the type's largest value is infinite, and what it is subtracted from with it.
    near = np.abs(want[0]) < 2.0 ** 126
    for got, ref, tol, what in zip((gx, gw, gb), want, _tolerances(dy, s, w, np.zeros_like(s), kind, eps),
                                   ("x", "weight", "bias")):
        got = host(got)
        off = np.abs(got - ref)
        keep = near if what == "x" else np.ones_like(ref, bool)
        assert np.all(off[keep] <= tol[keep]), (what, np.max((off / tol)[keep]))
