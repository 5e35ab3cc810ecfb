"""The norm's gradients on rows whose sums leave binary32's range, and on more
rows than work-groups at every width, against oracle/layer.py in 64 bits."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, TORCH, device, host, values
from oracle.layer import HALF_STEP, rms_norm_backward, round_to

pytestmark = pytest.mark.gpu


def check_gradients(dy, s, w, ds, eps, kind, check_weight=True):
    """Bounds from the kernel's roundings (u = 2^-24). ss: seven additions in a
    piece of eight (the squares of 16-bit values are exact; fp32: four of four),
    so r 3.5, and 1 more in binary32; s * r 5.5. d * s: two products and seven
    additions, 9; its mean 9 + 3.5 + 1 = 13.5. u * mean 20; d 1; their
    difference 1; times r 5.5; the sum with grad_sum 1; then the rounding to
    the type. grad_weight: a term 6.5, then the rows of a work-group (at least
    256 of them take the rows), sixteen parts a half wave, and 32 of those."""
    t, h = s.shape
    gx = torch.full((t, h), float("nan"), dtype=TORCH[kind], device="cuda")
    gw = torch.full((h,), float("nan"), device="cuda")
    qrs.rms_norm_backward(device(dy, kind), device(s, kind), device(w, kind), eps,
                          None if ds is None else device(ds, kind), gx, gw)
    want_x, want_w = rms_norm_backward(dy, s, w, eps, ds)
    s64, dy64 = s.astype(np.float64), dy.astype(np.float64)
    rms = np.sqrt(np.mean(s64 * s64, axis=1, keepdims=True) + eps)
    u = s64 / rms
    d = np.abs(dy64 * w.astype(np.float64))
    size = (d + np.abs(u) * np.mean(d * np.abs(u), axis=1, keepdims=True)) / rms
    whole = size if ds is None else size + np.abs(ds.astype(np.float64))
    tiny = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}[kind]  # a step of subnormal numbers
    tol = 28 * STEP * size + (STEP + 1.001 * HALF_STEP[kind]) * whole + tiny
    off = np.abs(host(gx) - want_x) / tol
    assert np.all(off <= 1), (np.argwhere(~(off <= 1))[:4], np.nanmax(off))
    if check_weight:
        tol = np.sum(np.abs(dy64 * u), axis=0) * (6.5 + -(-t // 256) + 16 + 32) * STEP
        off = np.abs(host(gw) - want_w) / (tol + 2.0 ** -149)
        assert np.all(off <= 1), (np.argwhere(~(off <= 1))[:4], np.nanmax(off))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t,h", [(1700, 1024), (1100, 5120), (700, 16384), (40, 1001)])
@pytest.mark.parametrize("with_sum", [True, False])
def test_gradient_of_rows_whose_squares_leave_binary32(gpu, t, h, kind, with_sum):
    """Rows of about 2^100, 2^62, 2^-62 and 2^-100 between rows of ordinary
    size, a row of zeros and one of zero gradients: the norm of all of them has
    a gradient, and grad_weight has their share."""
    rng = np.random.default_rng([t, h, 7])
    size = np.exp2(rng.choice([0, 0, 100, -100, 62, -62], t)).astype(np.float32)
    s = round_to(values(rng, (t, h), kind) * size[:, None], kind)
    dy, ds = values(rng, (t, h), kind, 0.1), values(rng, (t, h), kind, 0.1)
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    s[5], dy[7] = 0, 0
    check_gradients(dy, s, w, ds if with_sum else None, 2.0 ** -126, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("h", [1024, 5120])
def test_gradient_of_rows_whose_products_leave_binary32(gpu, h, kind):
    """Gradients and rows whose products pass 2^128 or fall below 2^-126, though
    grad_x itself is an ordinary number."""
    pairs = [(0, 0), (60, 90), (100, 100), (-40, -60), (0, -110), (-20, -100), (100, -20), (0, -90),
             (-20, -126)]
    t = 100 * len(pairs)
    rng = np.random.default_rng([h, 8])
    e = np.array(pairs * 100, dtype=np.float32)
    s = round_to(values(rng, (t, h), kind) * np.exp2(e[:, :1]), kind)
    dy = round_to(values(rng, (t, h), kind) * np.exp2(e[:, 1:]), kind)
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    check_gradients(dy, s, w, None, 2.0 ** -126, kind, check_weight=False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t,h", [(600, 1024), (40, 9000), (7, 100)])
def test_gradient_with_weights_of_any_size(gpu, t, h, kind):
    """Weights from 2^-100 to 2^100, whose products with the gradients pass
    2^64, beside rows of zero and of tiny gradients."""
    rng = np.random.default_rng([t, h, 11])
    s, dy = values(rng, (t, h), kind), values(rng, (t, h), kind, 0.1)
    w = round_to(values(rng, h, kind) * np.exp2(rng.choice([0, 0, 0, 59, 60, 100, -100], h)).astype(np.float32), kind)
    dy[1], dy[2] = 0, round_to(dy[2] * np.float32(2.0 ** -120), kind)
    check_gradients(dy, s, w, None, 1e-5, kind)


def test_gradient_of_a_row_that_is_not_finite_stays_in_its_row(gpu):
    rng = np.random.default_rng(9)
    s, dy = values(rng, (5, 1024), "bf16"), values(rng, (5, 1024), "bf16")
    w = values(rng, 1024, "bf16")
    ds, dw = device(s, "bf16"), device(w, "bf16")
    gx, gw, clean = torch.empty_like(ds), torch.empty(1024, device="cuda"), torch.empty_like(ds)
    qrs.rms_norm_backward(device(dy, "bf16"), ds, dw, 1e-5, None, clean, gw)
    ds[3, 700] = float("inf")
    qrs.rms_norm_backward(device(dy, "bf16"), ds, dw, 1e-5, None, gx, gw)
    keep = [0, 1, 2, 4]
    assert torch.equal(gx[keep], clean[keep]) and not torch.isfinite(gx[3]).any() and torch.isnan(gw[700])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t,h", [(2047, 2048), (2048, 2048), (2051, 1000), (2049, 1024), (1030, 4096), (600, 16384),
                                 (520, 9000), (530, 8201), (300, 40000), (5000, 8192)])
def test_gradient_of_more_rows_than_work_groups(gpu, t, h, kind):
    """Two work-groups a CU from 2048 narrow rows on; rows past 8192 elements;
    operands that are loaded as a stream."""
    rng = np.random.default_rng([t, h, 10])
    s, dy, ds = values(rng, (t, h), kind, 2), values(rng, (t, h), kind, 0.1), values(rng, (t, h), kind, 0.1)
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    check_gradients(dy, s, w, ds, 1e-5, kind)
