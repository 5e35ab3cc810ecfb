"""GPU parity of add_layer_norm_quantize and layer_norm_backward against
oracle/blocks.py in 64 bits."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import assert_codes_within
from layer_util import STEP, TORCH, device, empty_codes, host, padded, values
from oracle.blocks import layer_norm, layer_norm_backward
from oracle.layer import HALF_STEP, round_to, rounded_sum

pytestmark = pytest.mark.gpu

EPS = 1e-5
MODES = [("int8", "f32_row"), ("e4m3fn", "f32_row"), ("e5m2", "f32_row"), ("int8", "f32_group128"),
         ("e4m3fn", "f32_group128"), ("e5m2", "f32_group128"), ("e4m3fn", "e8m0_block32"), ("e5m2", "e8m0_block32")]
KINDS = ["bf16", "f16", "f32"]


def _case(rng, t, h, kind):
    x = values(rng, (t, h), kind) * np.exp2(rng.integers(-4, 5, (t, 1))).astype(np.float32)
    r = values(rng, (t, h), kind) * np.float32(4) + rng.standard_normal((t, 1)).astype(np.float32)
    w, b = values(rng, h, kind, 0.1) + np.float32(1), values(rng, h, kind, 0.5)
    x, r, w, b = (round_to(v, kind) for v in (x, r, w, b))
    if t > 2:
        x[1] = r[1] = 0  # a padded token: y is the bias
        x[2] = -r[2]  # a sum that cancels
    return x, r, w, b


def _y(s, w, b, eps=EPS):
    """y and its bound: s - mean off by two half steps, r, their product and the
    fused sum one each, the moments less than one."""
    y = layer_norm(s, w, b, eps)
    off = np.abs(y - np.asarray(b, np.float64)) * 4.1 * STEP + np.abs(y) * STEP
    return y, off + 2.0 ** -140


def _check(s, w, b, x_format, layout, codes, scales, what, eps=EPS):
    y, tol = _y(s, w, b, eps)
    assert_codes_within(codes.cpu().numpy(), scales.cpu().numpy(), y, tol, x_format, layout, what)


SHAPES = [(1, 1024), (3, 128), (5, 1152), (130, 2048), (7, 4096), (1, 8192), (3, 16384), (2, 33280), (1, 65536),
          (700, 8192), (300, 5120)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x_format,layout", MODES)
@pytest.mark.parametrize("t,h", SHAPES)
def test_norm(gpu, t, h, x_format, layout, kind):
    rng = np.random.default_rng([t, h])
    x, r, w, b = _case(rng, t, h, kind)
    codes, scales = empty_codes(t, h, layout)
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    qrs.add_layer_norm_quantize(device(x, kind), device(r, kind), device(w, kind), device(b, kind), EPS, total, codes,
                                scales, x_format, layout)
    s = rounded_sum(x, r, kind)
    assert np.array_equal(host(total), s)
    _check(s, w, b, x_format, layout, codes, scales, "norm")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,h", [(1, 1), (5, 2), (5, 7), (3, 100), (4, 1001), (2, 8200), (9, 4100), (2, 65535), (66, 33),
                                 (3, 4097), (2, 16391)])
def test_norm_with_row_scales_at_any_width(gpu, t, h, kind):
    rng = np.random.default_rng([t, h, 1])
    x, r, w, b = _case(rng, t, h, kind)
    codes, scales = empty_codes(t, h, "f32_row")
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    qrs.add_layer_norm_quantize(device(x, kind), device(r, kind), device(w, kind), device(b, kind), EPS, total, codes,
                                scales, "int8", "f32_row")
    s = rounded_sum(x, r, kind)
    assert np.array_equal(host(total), s)
    _check(s, w, b, "int8", "f32_row", codes, scales, "odd width")


@pytest.mark.parametrize("layout,x_format", [("f32_row", "int8"), ("e8m0_block32", "e5m2"), ("f32_group128", "e4m3fn")])
@pytest.mark.parametrize("left,right", [(0, 8), (8, 0), (1, 2), (16, 16)])
def test_norm_of_strided_rows_writes_only_its_rows(gpu, left, right, layout, x_format):
    rng = np.random.default_rng([left, right])
    t, h, kind = 6, 1152, "bf16"
    x, r, w, b = _case(rng, t, h, kind)
    _, dx = padded(device(x, kind), left, right, float("nan"))
    _, dr = padded(device(r, kind), right, left, float("nan"))
    tb, total = padded(torch.zeros(t, h, dtype=torch.bfloat16, device="cuda"), left, right, 7.0)
    codes, scales = empty_codes(t, h, layout)
    cb, codes = padded(codes, right, left, 0x5A)
    qrs.add_layer_norm_quantize(dx, dr, device(w, kind), device(b, kind), EPS, total, codes, scales, x_format, layout)
    _check(rounded_sum(x, r, kind), w, b, x_format, layout, codes, scales, "strided")
    assert torch.all(tb[:, :left] == 7) and torch.all(tb[:, left + h:] == 7)
    assert torch.all(cb[:, :right] == 0x5A) and torch.all(cb[:, right + h:] == 0x5A)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("t,h", [(4, 1024), (3, 100), (700, 8192)])
def test_norm_updates_the_residual_stream_in_place(gpu, which, t, h):
    rng = np.random.default_rng(5)
    x, r, w, b = _case(rng, t, h, "bf16")
    dx, dr = device(x, "bf16"), device(r, "bf16")
    total = dx if which == "x" else dr
    codes, scales = empty_codes(t, h, "f32_row")
    qrs.add_layer_norm_quantize(dx, dr, device(w, "bf16"), device(b, "bf16"), EPS, total, codes, scales, "int8", "f32_row")
    s = rounded_sum(x, r, "bf16")
    assert np.array_equal(host(total), s)
    _check(s, w, b, "int8", "f32_row", codes, scales, which)


@pytest.mark.parametrize("with_bias", [True, False])
def test_norm_without_a_residual_or_a_bias(gpu, with_bias):
    rng = np.random.default_rng(6)
    x, _, w, b = _case(rng, 5, 2048, "f16")
    codes, scales = empty_codes(5, 2048, "f32_group128")
    qrs.add_layer_norm_quantize(device(x, "f16"), None, device(w, "f16"), device(b, "f16") if with_bias else None, EPS,
                                None, codes, scales, "e4m3fn", "f32_group128")
    _check(x, w, b if with_bias else np.zeros_like(b), "e4m3fn", "f32_group128", codes, scales, "bare")


@pytest.mark.parametrize("h", [1024, 1000, 8192])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["mean", "first", "last", "wave"])
def test_norm_of_rows_far_from_zero(gpu, where, kind, h):
    """A mean that is thousands of deviations away, or one element that is (the
    first of the row, which the variance is taken about, or another)."""
    rng = np.random.default_rng([h, len(where)])
    x = values(rng, (9, h), kind)
    if where == "mean":
        x = x * np.float32(0.01) + np.float32(100.0 if kind == "bf16" else 20000.0)
    else:
        x[:, {"first": 0, "last": h - 1, "wave": min(h - 1, 512)}[where]] = np.exp2(np.arange(9) * 3.0)
    x = round_to(x, kind)
    w, b = np.ones(h, np.float32), np.zeros(h, np.float32)
    codes, scales = empty_codes(9, h, "f32_row")
    qrs.add_layer_norm_quantize(device(x, kind), None, device(w, kind), None, EPS, None, codes, scales, "int8", "f32_row")
    _check(x, w, b, "int8", "f32_row", codes, scales, where)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("x_format,layout", [("int8", "f32_row"), ("e4m3fn", "f32_group128"), ("e5m2", "e8m0_block32")])
@pytest.mark.parametrize("h", [1024, 5120, 16384])
def test_norm_of_rows_whose_squares_leave_binary32(gpu, h, x_format, layout, kind):
    t = 700
    rng = np.random.default_rng([t, h, 3])
    x, w, b = values(rng, (t, h), kind), values(rng, h, kind, 0.1) + np.float32(1), values(rng, h, kind)
    size = np.exp2(rng.choice([0, 0, 120, -100, 62, -62], t)).astype(np.float32)
    x, w = round_to(x * size[:, None], kind), round_to(w, kind)
    x[5] = 0
    codes, scales = empty_codes(t, h, layout)
    eps = 2.0 ** -126
    qrs.add_layer_norm_quantize(device(x, kind), None, device(w, kind), device(b, kind), eps, None, codes, scales,
                                x_format, layout)
    _check(x, w, b, x_format, layout, codes, scales, "far", eps)


@pytest.mark.parametrize("layout,x_format", [("f32_row", "int8"), ("e8m0_block32", "e4m3fn"), ("f32_group128", "e5m2")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("at", [0, 700])
def test_a_row_that_is_not_finite_shows_in_its_scales_alone(gpu, at, layout, x_format, bad):
    rng = np.random.default_rng(8)
    x, r, w, b = _case(rng, 5, 1024, "bf16")
    dx = device(x, "bf16")
    dx[3, at] = bad
    codes, scales = empty_codes(5, 1024, layout)
    total = torch.empty_like(dx)
    qrs.add_layer_norm_quantize(dx, device(r, "bf16"), device(w, "bf16"), device(b, "bf16"), EPS, total, codes, scales,
                                x_format, layout)
    s = scales.cpu().reshape(5, -1)
    assert torch.all(s[3] == 255) if layout == "e8m0_block32" else torch.all(torch.isnan(s[3]))
    keep = [0, 1, 2, 4]
    _check(rounded_sum(x, r, "bf16")[keep], w, b, x_format, layout, codes[keep], s[keep], "other rows")


def test_rows_of_equal_values(gpu):
    """With eps: the bias. Without: 0 / 0, which shows."""
    x = torch.full((2, 256), 3.0, device="cuda")
    w, b = torch.ones(256, device="cuda"), torch.full((256,), 0.5, device="cuda")
    codes, scales = empty_codes(2, 256, "f32_row")
    qrs.add_layer_norm_quantize(x, None, w, b, EPS, None, codes, scales, "int8", "f32_row")
    assert torch.all(codes == 127) and torch.all(scales == torch.tensor(0.5) / 127)
    qrs.add_layer_norm_quantize(x, None, w, b, 0.0, None, codes, scales, "int8", "f32_row")
    assert torch.all(torch.isnan(scales))


# ---- backward -----------------------------------------------------------------------------------------------


def _tolerances(dy, s, w, gs, kind, eps=EPS):
    """Absolute bounds from the operation counts: u is off by four half steps, d by
    one (and its mean by one more), d - mean(d) by one of itself and of what it is
    made of, the next fused operation one, the last one, then the output.
    grad_weight and grad_bias add at most t rows, one rounding each."""
    s, dy, w, gs = (np.asarray(v, np.float64) for v in (s, dy, w, gs))
    c = s - s.mean(axis=1, keepdims=True)
    std = np.sqrt(np.mean(c * c, axis=1, keepdims=True) + eps)
    u, d = c / std, dy * w
    md = np.mean(np.abs(d), axis=1, keepdims=True)
    mdu = np.mean(np.abs(d * u), axis=1, keepdims=True)
    size = (np.abs(d) + md + np.abs(u) * mdu) / std
    gx = size * 12 * STEP + np.abs(gs) * 2 * STEP + HALF_STEP[kind] * (size * (1 + 12 * STEP) + np.abs(gs))
    t = len(s)
    gw = np.sum(np.abs(dy * u), axis=0) * (5 + t) * STEP
    gb = np.sum(np.abs(dy), axis=0) * (1 + t) * STEP
    return gx + 2.0 ** -120 + (2.0 ** -25 if kind == "f16" else 0), gw + 2.0 ** -120, gb + 2.0 ** -120


BACK_SHAPES = [(1, 1), (1, 8192), (2, 7), (5, 100), (3, 1001), (17, 1024), (513, 256), (1030, 512), (2100, 1024),
               (700, 4096), (33, 7168), (530, 8192), (3, 16384), (300, 12288), (2, 65536), (2, 65535), (20, 5160)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,h", BACK_SHAPES)
@pytest.mark.parametrize("with_sum", [True, False])
def test_backward(gpu, t, h, kind, with_sum):
    rng = np.random.default_rng([t, h, 3])
    s, dy, gs = values(rng, (t, h), kind, 2), values(rng, (t, h), kind, 0.1), values(rng, (t, h), kind, 0.1)
    s = round_to(s + rng.standard_normal((t, 1)).astype(np.float32) * 3, kind)
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    if t > 2:
        s[1] = 0
    gx = torch.full((t, h), float("nan"), dtype=TORCH[kind], device="cuda")
    gw, gb = (torch.full((h,), float("nan"), device="cuda") for _ in range(2))
    qrs.layer_norm_backward(device(dy, kind), device(s, kind), device(w, kind), EPS,
                            device(gs, kind) if with_sum else None, gx, gw, gb)
    if not with_sum:
        gs = np.zeros_like(gs)
    want = layer_norm_backward(dy, s, w, EPS, gs)
    for got, ref, tol, what in zip((gx, gw, gb), want, _tolerances(dy, s, w, gs, kind), ("x", "weight", "bias")):
        off = np.abs(host(got) - ref)
        assert np.all(off <= tol), (what, np.max(off / tol))


@pytest.mark.parametrize("h", [512, 2048, 8192, 16384])
def test_backward_of_rows_far_from_zero_and_of_any_size(gpu, h):
    """Rows about 2^62, 2^-62 and 2^110, rows whose mean is thousands of
    deviations away, and rows whose first element is."""
    t = 300
    rng = np.random.default_rng(h)
    s, dy = values(rng, (t, h), "f32"), values(rng, (t, h), "f32", 0.1)
    s = (s * np.exp2(rng.choice([0, 62, -62, 110], (t, 1)))).astype(np.float32)
    s[::5] = values(rng, s[::5].shape, "f32") + np.float32(5000)
    s[1::5, 0] = s[1::5, 1] * 3000
    w = values(rng, h, "f32", 0.1) + np.float32(1)
    eps = 2.0 ** -126
    gx, gw, gb = torch.empty(t, h, device="cuda"), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(device(dy), device(s), device(w), eps, None, gx, gw, gb)
    want = layer_norm_backward(dy, s, w, eps)
    for got, ref, tol, what in zip((gx, gw, gb), want, _tolerances(dy, s, w, np.zeros_like(s), "f32", eps),
                                   ("x", "weight", "bias")):
        off = np.abs(host(got) - ref)
        assert np.all(off <= tol), (what, np.max(off / tol))


@pytest.mark.parametrize("which", ["grad_y", "grad_sum"])
@pytest.mark.parametrize("t,h", [(600, 1024), (5, 101), (300, 16384)])
def test_backward_in_place_is_the_same(gpu, which, t, h):
    rng = np.random.default_rng(12)
    s, dy, gs = (values(rng, (t, h), "bf16") for _ in range(3))
    w = values(rng, h, "bf16")
    args = [device(dy, "bf16"), device(s, "bf16"), device(w, "bf16"), EPS, device(gs, "bf16")]
    want_x, want_w, want_b = torch.empty_like(args[0]), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(*args, want_x, want_w, want_b)
    gx, gw = args[0 if which == "grad_y" else 4], torch.empty(h, device="cuda")
    qrs.layer_norm_backward(*args, gx, gw)  # without grad_bias
    assert torch.equal(gx, want_x) and torch.equal(gw, want_w)


@pytest.mark.parametrize("left,right", [(8, 8), (1, 2), (0, 8)])
def test_backward_strided_is_the_same(gpu, left, right):
    rng = np.random.default_rng(13)
    t, h = 40, 1024
    s, dy, gs = (device(values(rng, (t, h), "f16"), "f16") for _ in range(3))
    w = device(values(rng, h, "f16"), "f16")
    want = torch.empty_like(s), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(dy, s, w, EPS, gs, *want)
    xb, gx = padded(torch.zeros_like(s), left, right, 3.0)
    gw, gb = torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    nan = float("nan")
    qrs.layer_norm_backward(padded(dy, left, right, nan)[1], padded(s, right, left, nan)[1], w, EPS,
                            padded(gs, left, right, nan)[1], gx, gw, gb)
    tol = _tolerances(host(dy), host(s), host(w), host(gs), "f16")
    for got, ref, bound in zip((gx, gw, gb), want, tol):
        assert np.all(np.abs(host(got) - host(ref)) <= 2 * bound)
    assert torch.all(xb[:, :left] == 3) and torch.all(xb[:, left + h:] == 3)


def test_backward_is_deterministic(gpu):
    rng = np.random.default_rng(14)
    s, dy, gs = (device(values(rng, (2000, 2048), "bf16"), "bf16") for _ in range(3))
    w = device(values(rng, 2048, "bf16"), "bf16")
    got = []
    for _ in range(3):
        out = torch.empty_like(s), torch.empty(2048, device="cuda"), torch.empty(2048, device="cuda")
        qrs.layer_norm_backward(dy, s, w, EPS, gs, *out)
        got.append(out)
    for out in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out, got[0]))


def test_backward_against_differences(gpu):
    """The gradient of a weighted sum of y, by differences of the norm in 64 bits
    at the same point."""
    rng = np.random.default_rng(15)
    t, h = 3, 40
    s, dy = values(rng, (t, h), "f32"), values(rng, (t, h), "f32")
    w, b = values(rng, h, "f32"), np.zeros(h)
    gx, gw, gb = torch.empty(t, h, device="cuda"), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(device(dy), device(s), device(w), EPS, None, gx, gw, gb)
    step = 1e-6

    def slope(i, at):
        parts = [np.array(v, dtype=np.float64) for v in (s, w, b)]
        out = []
        for sign in (1, -1):
            moved = [v.copy() for v in parts]
            moved[i][at] += sign * step
            out.append(np.sum(layer_norm(*moved, EPS) * dy))
        return (out[0] - out[1]) / (2 * step)

    for i, got in enumerate((gx, gw, gb)):
        got = host(got)
        for at in list(np.ndindex(got.shape))[::7]:
            assert abs(slope(i, at) - got[at]) < 1e-4
