"""GPU parity of add_rms_norm_quantize, rms_norm_backward and quantize_rows
against oracle/layer.py in 64 bits."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, TORCH, assert_codes, device, empty_codes, host, norm_rel, padded, values
from oracle.layer import HALF_STEP, rms_norm, rms_norm_backward, round_to, rounded_sum
from oracle.quantize import quantize_values

pytestmark = pytest.mark.gpu

EPS = 1e-5
MODES = [("int8", "f32_row"), ("e4m3fn", "f32_row"), ("e5m2", "f32_row"), ("int8", "f32_group128"),
         ("e4m3fn", "f32_group128"), ("e5m2", "f32_group128"), ("e4m3fn", "e8m0_block32"), ("e5m2", "e8m0_block32")]
KINDS = ["bf16", "f16", "f32"]


def _norm_case(rng, t, h, kind):
    x = values(rng, (t, h), kind) * np.exp2(rng.integers(-6, 7, (t, 1))).astype(np.float32)
    r = values(rng, (t, h), kind) * np.float32(4)
    w = values(rng, h, kind, 0.1) + np.float32(1)
    x, r, w = (round_to(v, kind) for v in (x, r, w))
    if t > 2:
        x[1] = r[1] = 0  # a padded token
        x[2] = -r[2]  # a sum that cancels
    return x, r, w


def _check_norm(x, r, w, kind, x_format, layout, total, codes, scales, what):
    s = x if r is None else rounded_sum(x, r, kind)
    if r is not None:
        assert np.array_equal(host(total), s), f"{what}: sum"
    y = rms_norm(s, w, EPS)
    assert_codes(codes.cpu().numpy(), scales.cpu().numpy(), y, norm_rel(s.shape[1]), x_format, layout, what)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x_format,layout", MODES)
@pytest.mark.parametrize("t,h", [(1, 1024), (3, 128), (5, 1152), (130, 2048), (7, 4096), (2, 8192), (1, 8192),
                                 (3, 16384), (2, 33280), (1, 65536), (700, 8192), (300, 5120)])
def test_norm(gpu, t, h, x_format, layout, kind):
    rng = np.random.default_rng([t, h])
    x, r, w = _norm_case(rng, t, h, kind)
    codes, scales = empty_codes(t, h, layout)
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    qrs.add_rms_norm_quantize(device(x, kind), device(r, kind), device(w, kind), EPS, total, codes, scales, x_format,
                              layout)
    _check_norm(x, r, w, kind, x_format, layout, total, codes, scales, "norm")


@pytest.mark.parametrize("kind,x_format", [("f32", "e5m2"), ("f32", "e4m3fn"), ("bf16", "e4m3fn"), ("f16", "e5m2")])
def test_norm_rounds_once_to_codes_of_e8m0_scales(gpu, kind, x_format):
    """Of 2^22 values, none falls on the far side of a border between two
    codes: y is exact to far more than binary32 when its code is chosen."""
    t, h = 1024, 4096
    rng = np.random.default_rng([t, h, len(kind)])
    x, r, w = _norm_case(rng, t, h, kind)
    codes, scales = empty_codes(t, h, "e8m0_block32")
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    qrs.add_rms_norm_quantize(device(x, kind), device(r, kind), device(w, kind), EPS, total, codes, scales, x_format,
                              "e8m0_block32")
    y = rms_norm(rounded_sum(x, r, kind), w, EPS)
    assert_codes(codes.cpu().numpy(), scales.cpu().numpy(), y, 2.0 ** -40, x_format, "e8m0_block32")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("x_format,layout", [("int8", "f32_row"), ("e4m3fn", "f32_group128"), ("e5m2", "e8m0_block32")])
@pytest.mark.parametrize("h", [1024, 5120, 16384])
def test_norm_of_rows_whose_squares_leave_binary32(gpu, h, x_format, layout, kind):
    """Rows of about 2^100 and 2^-100 between rows of ordinary size."""
    t = 1700  # several rows a work-group at any width
    rng = np.random.default_rng([t, h, 3])
    x, r, w = values(rng, (t, h), kind), values(rng, (t, h), kind), values(rng, h, kind, 0.1) + np.float32(1)
    w = round_to(w, kind)
    size = np.exp2(rng.choice([0, 0, 100, -100, 62, -62], t)).astype(np.float32)
    x, r = (round_to(v * size[:, None], kind) for v in (x, r))
    x[5] = r[5] = 0
    codes, scales = empty_codes(t, h, layout)
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    eps = 2.0 ** -126
    qrs.add_rms_norm_quantize(device(x, kind), device(r, kind), device(w, kind), eps, total, codes, scales, x_format,
                              layout)
    s = rounded_sum(x, r, kind)
    assert np.array_equal(host(total), s)
    assert_codes(codes.cpu().numpy(), scales.cpu().numpy(), rms_norm(s, w, eps), norm_rel(h), x_format, layout)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,h", [(1, 1), (5, 7), (3, 100), (4, 1001), (2, 8200), (9, 4100), (2, 65535), (66, 33)])
def test_norm_with_row_scales_at_any_width(gpu, t, h, kind):
    rng = np.random.default_rng([t, h, 1])
    x, r, w = _norm_case(rng, t, h, kind)
    codes, scales = empty_codes(t, h, "f32_row")
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    qrs.add_rms_norm_quantize(device(x, kind), device(r, kind), device(w, kind), EPS, total, codes, scales, "int8",
                              "f32_row")
    _check_norm(x, r, w, kind, "int8", "f32_row", total, codes, scales, "odd width")


@pytest.mark.parametrize("layout,x_format", [("f32_row", "int8"), ("e8m0_block32", "e5m2"), ("f32_group128", "e4m3fn")])
@pytest.mark.parametrize("left,right", [(0, 8), (8, 0), (1, 2), (3, 5), (16, 16)])
def test_norm_of_strided_rows_writes_only_its_rows(gpu, left, right, layout, x_format):
    rng = np.random.default_rng([left, right])
    t, h, kind = 6, 1152, "bf16"
    x, r, w = _norm_case(rng, t, h, kind)
    _, dx = padded(device(x, kind), left, right, float("nan"))
    _, dr = padded(device(r, kind), right, left, float("nan"))
    tb, total = padded(torch.zeros(t, h, dtype=torch.bfloat16, device="cuda"), left, right, 7.0)
    codes, scales = empty_codes(t, h, layout)
    cb, codes = padded(codes, right, left, 0x5A)
    qrs.add_rms_norm_quantize(dx, dr, device(w, kind), EPS, total, codes, scales, x_format, layout)
    _check_norm(x, r, w, kind, x_format, layout, total, codes, scales, "strided")
    assert torch.all(tb[:, :left] == 7) and torch.all(tb[:, left + h:] == 7)
    assert torch.all(cb[:, :right] == 0x5A) and torch.all(cb[:, right + h:] == 0x5A)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("t,h", [(4, 1024), (3, 100)])
def test_norm_updates_the_residual_stream_in_place(gpu, which, t, h):
    rng = np.random.default_rng(5)
    x, r, w = _norm_case(rng, t, h, "bf16")
    dx, dr = device(x, "bf16"), device(r, "bf16")
    total = dx if which == "x" else dr
    codes, scales = empty_codes(t, h, "f32_row")
    qrs.add_rms_norm_quantize(dx, dr, device(w, "bf16"), EPS, total, codes, scales, "int8", "f32_row")
    _check_norm(x, r, w, "bf16", "int8", "f32_row", total, codes, scales, which)


def test_norm_without_a_residual(gpu):
    rng = np.random.default_rng(6)
    x, _, w = _norm_case(rng, 5, 2048, "f16")
    codes, scales = empty_codes(5, 2048, "f32_group128")
    qrs.add_rms_norm_quantize(device(x, "f16"), None, device(w, "f16"), EPS, None, codes, scales, "e4m3fn",
                              "f32_group128")
    _check_norm(x, None, w, "f16", "e4m3fn", "f32_group128", None, codes, scales, "no residual")


@pytest.mark.parametrize("layout,x_format", [("f32_row", "int8"), ("e8m0_block32", "e4m3fn"), ("f32_group128", "e5m2")])
def test_zero_rows_take_the_smallest_scale_and_zero_codes(gpu, layout, x_format):
    x = torch.zeros(3, 1024, dtype=torch.bfloat16, device="cuda")
    codes, scales = empty_codes(3, 1024, layout)
    qrs.add_rms_norm_quantize(x, x, torch.ones(1024, dtype=torch.bfloat16, device="cuda"), EPS, torch.empty_like(x),
                              codes, scales, x_format, layout)
    assert torch.all(codes == 0)
    want = 0 if layout == "e8m0_block32" else 2.0 ** -126
    assert torch.all(scales == want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("layout,x_format", [("f32_row", "int8"), ("e8m0_block32", "e4m3fn"), ("f32_group128", "e5m2")])
def test_a_row_that_is_not_finite_shows_in_its_scales_alone(gpu, layout, x_format, bad):
    rng = np.random.default_rng(8)
    x, r, w = _norm_case(rng, 5, 1024, "bf16")
    dx = device(x, "bf16")
    dx[3, 700] = bad
    codes, scales = empty_codes(5, 1024, layout)
    total = torch.empty_like(dx)
    qrs.add_rms_norm_quantize(dx, device(r, "bf16"), device(w, "bf16"), EPS, total, codes, scales, x_format, layout)
    s = scales.cpu().reshape(5, -1)
    g = 700 // {"f32_row": 1024, "e8m0_block32": 32, "f32_group128": 128}[layout]
    assert s[3, g] == 255 if layout == "e8m0_block32" else not torch.isfinite(s[3, g])
    keep = [0, 1, 2, 4]
    _check_norm(x[keep], r[keep], w, "bf16", x_format, layout, total[keep], codes[keep], s[keep], "other rows")


def test_quantize_rows_of_the_norms_own_scale_rule(gpu):
    """A weight of 1 and rows whose mean square is 1: y is s up to eps = 0."""
    s = np.array([[1.0, -1.0] * 64, [1.0, 1.0] * 64], dtype=np.float32)
    codes, scales = empty_codes(2, 128, "f32_row")
    qrs.add_rms_norm_quantize(device(s, "f32"), None, torch.ones(128, device="cuda"), 0.0, None, codes, scales, "int8",
                              "f32_row")
    c, sc = quantize_values(s, "int8", "f32_row")
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), sc[:, 0])


# ---- quantize_rows: every step is one binary32 operation, so bit for bit ------------------------------------


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x_format", ["int8", "e4m3fn", "e5m2"])
@pytest.mark.parametrize("t,h", [(1, 1), (3, 7), (130, 64), (5, 1000), (4, 1001), (300, 3584), (2, 8192), (3, 28672),
                                 (1, 65536), (2, 65535), (65, 512), (1025, 2048)])
def test_quantize_rows(gpu, t, h, x_format, kind):
    rng = np.random.default_rng([t, h, 2])
    v = values(rng, (t, h), kind) * np.exp2(rng.integers(-8, 9, (t, 1))).astype(np.float32)
    v = round_to(v, kind)
    if t > 2:
        v[1] = 0
    codes, scales = empty_codes(t, h, "f32_row")
    qrs.quantize_rows(device(v, kind), codes, scales, x_format)
    c, s = quantize_values(v, x_format, "f32_row")
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s[:, 0].view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), c)


@pytest.mark.parametrize("left,right", [(8, 8), (1, 0), (0, 3)])
def test_quantize_rows_strided(gpu, left, right):
    rng = np.random.default_rng(11)
    v = values(rng, (9, 1024), "bf16")
    _, x = padded(device(v, "bf16"), left, right, float("inf"))
    codes, scales = empty_codes(9, 1024, "f32_row")
    cb, codes = padded(codes, left, right, 0x33)
    qrs.quantize_rows(x, codes, scales)
    c, s = quantize_values(v, "int8", "f32_row")
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s[:, 0])
    assert torch.all(cb[:, :left] == 0x33) and torch.all(cb[:, left + 1024:] == 0x33)


def test_quantize_rows_of_tiny_and_extreme_values(gpu):
    v = np.zeros((4, 256), dtype=np.float32)
    v[0, 3] = 2.0 ** -140  # subnormal maximum: the scale stays at 2^-126
    v[1, :2] = [3.0e38, -1.0e38]
    v[2, 5] = 127 * 2.0 ** -126
    v[3] = -1.0
    codes, scales = empty_codes(4, 256, "f32_row")
    qrs.quantize_rows(device(v), codes, scales)
    c, s = quantize_values(v, "int8", "f32_row")
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s[:, 0])


# ---- backward -----------------------------------------------------------------------------------------------


def _backward_tolerances(dy, s, w, ds, kind):
    """Absolute bounds from the operation counts. r as in norm_rel; the mean
    of d * s sums products with the same depth; grad_weight adds at most
    ceil(t / parts) + parts rows of products of three roundings."""
    t, h = s.shape
    s, dy, w = s.astype(np.float64), dy.astype(np.float64), w.astype(np.float64)
    rms = np.sqrt(np.mean(s * s, axis=1, keepdims=True) + EPS)
    u = s / rms
    d = np.abs(dy * w)
    along = np.mean(d * np.abs(u), axis=1, keepdims=True)
    depth = min(h, 64) + 6 + 16 + 4
    rel = (depth + 8) * STEP
    size = (d + np.abs(u) * along) / rms
    gx = 3 * rel * size + 2 * STEP * np.abs(ds) + HALF_STEP[kind] * (size * (1 + 3 * rel) + np.abs(ds))
    gw = np.sum(np.abs(dy * u), axis=0) * (norm_rel(h) + (t + 3) * STEP)
    return gx, gw


BACK_SHAPES = [(1, 1), (1, 8192), (2, 7), (5, 100), (3, 1001), (17, 1024), (513, 256), (1030, 512), (700, 4096),
               (33, 7168), (530, 8192), (3, 16384), (2, 65536), (2, 65535), (20, 5160)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,h", BACK_SHAPES)
@pytest.mark.parametrize("with_sum", [True, False])
def test_backward(gpu, t, h, kind, with_sum):
    rng = np.random.default_rng([t, h, 3])
    s, dy, ds = values(rng, (t, h), kind, 2), values(rng, (t, h), kind, 0.1), values(rng, (t, h), kind, 0.1)
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    if t > 2:
        s[1] = 0
    gx = torch.full((t, h), float("nan"), dtype=TORCH[kind], device="cuda")
    gw = torch.full((h,), float("nan"), device="cuda")
    qrs.rms_norm_backward(device(dy, kind), device(s, kind), device(w, kind), EPS,
                          device(ds, kind) if with_sum else None, gx, gw)
    if not with_sum:
        ds = np.zeros_like(ds)
    want_x, want_w = rms_norm_backward(dy, s, w, EPS, ds)
    tol_x, tol_w = _backward_tolerances(dy, s, w, ds, kind)
    # f16 subnormals: half their fixed step.
    tol_x = tol_x + (2.0 ** -25 if kind == "f16" else 0)
    assert np.all(np.abs(host(gx) - want_x) <= tol_x), np.max(np.abs(host(gx) - want_x) / (tol_x + 1e-300))
    assert np.all(np.abs(host(gw) - want_w) <= tol_w), np.max(np.abs(host(gw) - want_w) / (tol_w + 1e-300))


@pytest.mark.parametrize("which", ["grad_y", "grad_sum"])
@pytest.mark.parametrize("t,h", [(600, 1024), (5, 101)])
def test_backward_in_place_is_the_same(gpu, which, t, h):
    rng = np.random.default_rng(12)
    s, dy, ds = (values(rng, (t, h), "bf16") for _ in range(3))
    w = values(rng, h, "bf16")
    args = [device(dy, "bf16"), device(s, "bf16"), device(w, "bf16"), EPS, device(ds, "bf16")]
    want_x, want_w = torch.empty_like(args[0]), torch.empty(h, device="cuda")
    qrs.rms_norm_backward(*args, want_x, want_w)
    gx, gw = args[0 if which == "grad_y" else 4], torch.empty(h, device="cuda")
    qrs.rms_norm_backward(*args, gx, gw)
    assert torch.equal(gx, want_x) and torch.equal(gw, want_w)


@pytest.mark.parametrize("left,right", [(8, 8), (1, 2), (0, 8)])
def test_backward_strided_is_the_same(gpu, left, right):
    rng = np.random.default_rng(13)
    t, h = 40, 1024
    s, dy, ds = (device(values(rng, (t, h), "f16"), "f16") for _ in range(3))
    w = device(values(rng, h, "f16"), "f16")
    want_x, want_w = torch.empty_like(s), torch.empty(h, device="cuda")
    qrs.rms_norm_backward(dy, s, w, EPS, ds, want_x, want_w)
    xb, gx = padded(torch.zeros_like(s), left, right, 3.0)
    gw = torch.empty(h, device="cuda")
    nan = float("nan")
    qrs.rms_norm_backward(padded(dy, left, right, nan)[1], padded(s, right, left, nan)[1], w, EPS,
                          padded(ds, left, right, nan)[1], gx, gw)
    # The same sums in the same order wherever the rows lie.
    assert torch.equal(gx, want_x) and torch.equal(gw, want_w)
    assert torch.all(xb[:, :left] == 3) and torch.all(xb[:, left + h:] == 3)


def test_backward_is_deterministic(gpu):
    rng = np.random.default_rng(14)
    s, dy, ds = (device(values(rng, (2000, 2048), "bf16"), "bf16") for _ in range(3))
    w = device(values(rng, 2048, "bf16"), "bf16")
    got = []
    for _ in range(3):
        gx, gw = torch.empty_like(s), torch.empty(2048, device="cuda")
        qrs.rms_norm_backward(dy, s, w, EPS, ds, gx, gw)
        got.append((gx, gw))
    for gx, gw in got[1:]:
        assert torch.equal(gx, got[0][0]) and torch.equal(gw, got[0][1])
