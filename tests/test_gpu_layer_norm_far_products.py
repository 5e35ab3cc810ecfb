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


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["grad_y", "grad_sum"])
@pytest.mark.parametrize("t,h", [(600, 1024), (5, 101), (300, 4096), (40, 20000)])
def test_products_beyond_binary32_in_place(gpu, t, h, which, kind):
    """A wave reads its gradient a second time where its products left the range: before
    it is overwritten."""
    rng = np.random.default_rng([t, h])
    s, dy, gs = (values(rng, (t, h), kind) * np.float32(2.0 ** n) for n in (60, 70, 80))
    w = round_to(values(rng, h, kind) * np.float32(2.0 ** 70), kind)
    args = [device(round_to(dy, kind), kind), device(round_to(s, kind), kind), device(w, kind), 1e-5,
            device(round_to(gs, kind), kind)]
    want = torch.empty_like(args[0]), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(*args, *want)
    assert all(torch.isfinite(v).all() for v in want)
    ref = layer_norm_backward(host(args[0]), host(args[1]), w, 1e-5, host(args[4]))
    tol = _tolerances(host(args[0]), host(args[1]), w, host(args[4]), kind)
    assert np.all(np.abs(host(want[0]) - ref[0]) <= tol[0])
    gx, got = args[0 if which == "grad_y" else 4], [torch.empty(h, device="cuda") for _ in range(2)]
    qrs.layer_norm_backward(*args, gx, *got)
    assert torch.equal(gx, want[0]) and torch.equal(got[0], want[1]) and torch.equal(got[1], want[2])
