"""GPU parity of quantize_blocks and quantize_transposed: every step is one
binary32 operation, so codes and scales are the oracle's bit for bit."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import FP8, G, up
from layer_util import device, padded, values
from oracle.blocks import quantize_groups
from oracle.layer import round_to

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "f16", "f32"]
SIZES = [(1, 1), (1, 128), (128, 1), (3, 5), (128, 128), (129, 127), (127, 264), (200, 1000), (1000, 200), (256, 1024),
         (640, 384), (1021, 520), (77, 4104)]


def _values(rng, r, c, kind):
    v = values(rng, (r, c), kind) * np.exp2(rng.integers(-8, 9, (r, 1))).astype(np.float32)
    v *= np.exp2(rng.integers(-4, 5, c)).astype(np.float32)
    if r > 2:
        v[1] = 0
    return round_to(v, kind)


def _empty(rows, cols, scale_shape):
    codes = torch.full((rows, cols), 0xAA, dtype=torch.uint8, device="cuda")
    return codes, torch.full(scale_shape, float("nan"), device="cuda")


def _equal(codes, scales, want):
    c, s = want
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s.view(np.uint32))
    got = codes.contiguous().view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, c), np.argwhere(got != c)[:4]


def _padded_rows(n):
    """The widths a transpose of n rows may have: n, a multiple of 16, of 128."""
    return sorted({n, up(n, 16) * 16, up(n) * G})


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x_format", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("r,c", SIZES)
def test_blocks(gpu, r, c, x_format, kind):
    rng = np.random.default_rng([r, c])
    v = _values(rng, r, c, kind)
    codes, scales = quantize_groups(v, x_format, G, G)
    for rows_t in _padded_rows(r):
        got, got_s = _empty(r, c, (up(r), up(c)))
        got_t, got_ts = _empty(c, rows_t, (up(c), up(r)))
        qrs.quantize_blocks(device(v, kind), got.view(FP8[x_format]), got_s, x_format, got_t, got_ts)
        _equal(got, got_s, (codes, scales))
        want_t = np.zeros((c, rows_t), np.uint8)
        want_t[:, :r] = codes.T
        _equal(got_t, got_ts, (want_t, np.ascontiguousarray(scales.T)))
    got, got_s = _empty(r, c, (up(r), up(c)))
    qrs.quantize_blocks(device(v, kind), got, got_s, x_format)
    _equal(got, got_s, (codes, scales))
    got_t, got_ts = _empty(c, r, (up(c), up(r)))
    qrs.quantize_blocks(device(v, kind), None, None, x_format, got_t.view(FP8[x_format]), got_ts)
    _equal(got_t, got_ts, (np.ascontiguousarray(codes.T), np.ascontiguousarray(scales.T)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x_format", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("r,c", SIZES)
def test_transposed(gpu, r, c, x_format, kind):
    rng = np.random.default_rng([r, c, 1])
    v = _values(rng, r, c, kind)
    codes, scales = quantize_groups(np.ascontiguousarray(v.T), x_format, 1, G)
    rows = quantize_groups(v, x_format, 1, G)
    for rows_t in _padded_rows(r):
        got_t, got_ts = _empty(c, rows_t, (c, up(r)))
        got, got_s = _empty(r, c, (r, up(c)))
        qrs.quantize_transposed(device(v, kind), got_t, got_ts, x_format, got, got_s)
        want_t = np.zeros((c, rows_t), np.uint8)
        want_t[:, :r] = codes
        _equal(got_t, got_ts, (want_t, scales))
        _equal(got, got_s, rows)
    got_t, got_ts = _empty(c, r, (c, up(r)))
    qrs.quantize_transposed(device(v, kind), got_t.view(FP8[x_format]), got_ts, x_format)
    _equal(got_t, got_ts, (codes, scales))


@pytest.mark.parametrize("left,right", [(8, 8), (16, 16), (1, 2), (0, 3)])
@pytest.mark.parametrize("by_block", [True, False])
def test_strided_views_write_only_their_own(gpu, by_block, left, right):
    rng = np.random.default_rng([left, right])
    r, c = 150, 264
    v = _values(rng, r, c, "bf16")
    _, x = padded(device(v, "bf16"), left, right, float("inf"))
    call = qrs.quantize_blocks if by_block else qrs.quantize_transposed
    got, got_s = _empty(r, c, (up(r), up(c)) if by_block else (r, up(c)))
    got_t, got_ts = _empty(c, 160, (up(c), up(r)) if by_block else (c, up(r)))
    buf, got = padded(got, right, left, 0x33)
    buf_t, got_t = padded(got_t, left, right, 0x44)
    if by_block:
        call(x, got, got_s, "e4m3fn", got_t, got_ts)
        codes, scales = quantize_groups(v, "e4m3fn", G, G)
        codes_t, scales_t = codes.T, scales.T
    else:
        call(x, got_t, got_ts, "e4m3fn", got, got_s)
        codes, scales = quantize_groups(v, "e4m3fn", 1, G)
        codes_t, scales_t = quantize_groups(np.ascontiguousarray(v.T), "e4m3fn", 1, G)
    _equal(got, got_s, (codes, scales))
    want_t = np.zeros((c, 160), np.uint8)
    want_t[:, :r] = codes_t
    _equal(got_t, got_ts, (want_t, np.ascontiguousarray(scales_t)))
    assert torch.all(buf[:, :right] == 0x33) and torch.all(buf[:, right + c:] == 0x33)
    assert torch.all(buf_t[:, :left] == 0x44) and torch.all(buf_t[:, left + 160:] == 0x44)


@pytest.mark.parametrize("x_format", ["e4m3fn", "e5m2"])
def test_tiny_and_extreme_values(gpu, x_format):
    v = np.zeros((256, 256), dtype=np.float32)
    v[3, 4] = 2.0 ** -140  # a subnormal maximum: the scale stays at 2^-126
    v[200, 4], v[201, 5] = 3.0e38, -1.0e38
    v[5, 200] = 448 * 2.0 ** -126
    v[130:, 130:] = -1.0
    codes, scales = quantize_groups(v, x_format, G, G)
    got, got_s = _empty(256, 256, (2, 2))
    qrs.quantize_blocks(device(v), got, got_s, x_format)
    _equal(got, got_s, (codes, scales))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_finite_shows_in_its_own_scales(gpu, bad):
    rng = np.random.default_rng(3)
    v = _values(rng, 300, 300, "f32")
    x = device(v)
    x[140, 7] = bad
    (got, got_s), (got_t, got_ts) = _empty(300, 300, (3, 3)), _empty(300, 300, (3, 3))
    qrs.quantize_blocks(x, got, got_s, "e4m3fn", got_t, got_ts)
    want, scales = quantize_groups(v, "e4m3fn", G, G)
    ok = np.ones((3, 3), bool)
    ok[1, 0] = False
    assert np.array_equal(np.isfinite(got_s.cpu().numpy()), ok) and np.array_equal(np.isfinite(got_ts.cpu().numpy()), ok.T)
    assert np.array_equal(got_s.cpu().numpy()[ok], scales[ok])
    (got_t, got_ts), (got, got_s) = _empty(300, 300, (300, 3)), _empty(300, 300, (300, 3))
    qrs.quantize_transposed(x, got_t, got_ts, "e4m3fn", got, got_s)
    by_row, by_col = ~torch.isfinite(got_s), ~torch.isfinite(got_ts)
    assert by_row.sum() == 1 and by_row[140, 0] and by_col.sum() == 1 and by_col[7, 1]


def test_refusals_of_shapes_and_types(gpu):
    x = torch.zeros(200, 130, dtype=torch.bfloat16, device="cuda")
    codes, scales = _empty(200, 130, (2, 2))
    codes_t, scales_t = _empty(130, 208, (2, 2))
    qrs.quantize_blocks(x, codes, scales, "e4m3fn", codes_t, scales_t)
    bad = [
        (lambda: qrs.quantize_blocks(x, codes[:100], scales, "e4m3fn"), "codes"),
        (lambda: qrs.quantize_blocks(x, codes.view(torch.float8_e5m2), scales, "e4m3fn"), "codes"),
        (lambda: qrs.quantize_blocks(x, codes, scales.half(), "e4m3fn"), "scales"),
        (lambda: qrs.quantize_blocks(x, codes, scales[:1], "e4m3fn"), "scales"),
        (lambda: qrs.quantize_blocks(x, codes, None, "e4m3fn"), "scales"),
        (lambda: qrs.quantize_blocks(x, codes, scales, "int8"), "e4m3fn or e5m2"),
        (lambda: qrs.quantize_blocks(x, codes, scales, "e4m3fn", codes_t[:, :199], scales_t), "codes_t"),
        (lambda: qrs.quantize_blocks(x, codes, scales, "e4m3fn", codes_t, None), "scales"),
        (lambda: qrs.quantize_blocks(x.double(), codes, scales, "e4m3fn"), "float32, bfloat16 or float16"),
        (lambda: qrs.quantize_blocks(x.t(), codes, scales, "e4m3fn"), "adjacent"),
        (lambda: qrs.quantize_transposed(x, codes_t, scales_t, "e4m3fn"), "scales"),
    ]
    for call, text in bad:
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(qrs.QrsError, match="codes"):
        qrs.quantize_blocks(x, None, None, "e4m3fn")
