"""GPU parity of the layer norm and its gradients for rows whose values are all
equal, where 1 / h is not a binary64 number, and for rows that differ from that in
one element by the last place."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, TORCH, device, empty_codes, host, values
from oracle.blocks import layer_norm_backward
from oracle.layer import round_to
from oracle.quantize import quantize_values
from test_gpu_layer_norm import _check, _tolerances

pytestmark = pytest.mark.gpu

VALUES = [1.0, 1.7, -0.1, 3.3e4, -7e-5, 0.0]
WIDTHS = [1, 49, 98, 1000, 4104, 6272, 8201, 16391]  # on 16-byte boundaries and off them, each shape


def _rows(h, kind):
    v = VALUES + ([1.3e30, -3e-30] if kind != "f16" else [])
    return round_to(np.repeat(np.array(v, np.float32)[:, None], h, axis=1), kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("eps", [1e-5, 2.0 ** -126, 0.0])
@pytest.mark.parametrize("h", WIDTHS)
def test_rows_of_equal_values(gpu, h, eps, kind):
    """s - mean is zero: y is the bias bit for bit, or without eps 0 / 0."""
    rng = np.random.default_rng(h)
    x, w = _rows(h, kind), round_to(values(rng, h, kind) * np.float32(3), kind)
    b = values(rng, h, kind)
    t = len(x)
    for layout in ["f32_row"] + (["f32_group128", "e8m0_block32"] if h % 128 == 0 else []):
        codes, scales = empty_codes(t, h, layout)
        qrs.add_layer_norm_quantize(device(x, kind), None, device(w, kind), device(b, kind), eps, None, codes, scales,
                                    "e4m3fn", layout)
        if eps == 0:
            assert torch.all(scales == 255) if layout == "e8m0_block32" else torch.all(torch.isnan(scales))
            continue
        want, want_s = quantize_values(np.tile(b, (t, 1)), "e4m3fn", layout)
        assert np.array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s), layout
        got = codes.cpu().numpy()
        assert not ((got != want) & (((got | want) & 0x7F) != 0)).any(), layout  # zeros of either sign


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("eps", [1e-5, 2.0 ** -126, 0.0])
@pytest.mark.parametrize("h", WIDTHS)
def test_gradients_of_rows_of_equal_values(gpu, h, eps, kind):
    rng = np.random.default_rng([h, 1])
    s, w = _rows(h, kind), round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    t = len(s)
    dy = values(rng, (t, h), kind)
    gx = torch.full((t, h), 7.0, dtype=TORCH[kind], device="cuda")
    gw, gb = torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(device(dy, kind), device(s, kind), device(w, kind), eps, None, gx, gw, gb)
    if eps == 0:
        assert torch.isnan(gx).all() and torch.isnan(gw).all()
        assert np.all(np.abs(host(gb) - dy.astype(np.float64).sum(axis=0)) <= np.abs(dy).sum(axis=0) * t * STEP)
        return
    assert torch.all(gw == 0)
    want = layer_norm_backward(dy, s, w, eps)
    tol = _tolerances(dy, s, w, np.zeros_like(s), kind, eps)
    got = host(gx)
    near = np.abs(want[0]) < (65000 if kind == "f16" else np.inf)
    assert np.all(np.abs(got - want[0])[near] <= tol[0][near])
    assert np.all(np.abs(got[~near]) > 64000)  # infinite, or the type's largest
    assert np.all(np.abs(host(gb) - want[2]) <= tol[2])


def _one_off(h):
    """Rows of 1.7 but for one element, which is one unit of the last place above, and what
    they are above 1.7: exactly that much, where a mean near 1.7 would round."""
    s = np.full((6, h), 1.7, np.float32)
    for i, at in enumerate([0, 1, h // 2, h - 1, min(h - 1, 700), h // 3]):
        s[i, at] = np.nextafter(np.float32(1.7), np.float32(2))
    return s, s.astype(np.float64) - np.float64(np.float32(1.7))


@pytest.mark.parametrize("layout,x_format", [("f32_group128", "e4m3fn"), ("f32_row", "int8")])
@pytest.mark.parametrize("h", [1024, 5120, 6272, 7168, 16384])
def test_a_mean_millions_of_deviations_away(gpu, h, layout, x_format):
    """u is known as closely as for a mean of zero."""
    (s, about), w, b = _one_off(h), np.ones(h, np.float32), np.zeros(h, np.float32)
    codes, scales = empty_codes(len(s), h, layout)
    qrs.add_layer_norm_quantize(device(s), None, device(w), None, 2.0 ** -126, None, codes, scales, x_format, layout)
    _check(about, w, b, x_format, layout, codes, scales, "one off", 2.0 ** -126)


@pytest.mark.parametrize("h", [512, 1000, 5120, 6272, 16384])
def test_gradients_about_a_mean_millions_of_deviations_away(gpu, h):
    rng = np.random.default_rng([h, 2])
    (s, about), eps = _one_off(h), 2.0 ** -100
    t = len(s)
    dy, w = values(rng, (t, h), "f32"), values(rng, h, "f32", 0.1) + np.float32(1)
    gx, gw, gb = torch.empty(t, h, device="cuda"), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(device(dy), device(s), device(w), eps, None, gx, gw, gb)
    want = layer_norm_backward(dy, about, w, eps)
    for got, ref, bound, what in zip((gx, gw, gb), want, _tolerances(dy, about, w, np.zeros_like(s), "f32", eps),
                                     ("x", "weight", "bias")):
        off = np.abs(host(got) - ref)
        assert np.all(off <= bound), (what, np.max(off / bound))
