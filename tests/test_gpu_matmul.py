"""GPU parity of matmul_int8 and matmul_int8_quantize. The integer sums are
exact and each later step is one binary32 operation, so ungated results equal
the oracle's bit for bit; the gated form is held to its operation count."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from gpu_util import oracle_bits, out_bits
from layer_util import STEP, TORCH, device, empty_codes, host, padded
from oracle.layer import HALF_STEP, gated, scaled_product
from oracle.quantize import quantize_values
from oracle.reduce import fp32_to_bf16_bits, fp32_to_f16_bits

pytestmark = pytest.mark.gpu


def _operands(rng, m, n, k, full=True):
    lo = -128 if full else -127
    a = rng.integers(lo, 128, size=(m, k), dtype=np.int8)
    b = rng.integers(lo, 128, size=(n, k), dtype=np.int8)
    sa = np.exp2(rng.uniform(-8, 2, m)).astype(np.float32)
    sb = np.exp2(rng.uniform(-12, -4, n)).astype(np.float32)
    return a, sa, b, sb


def _bits(v, kind):
    return {"f32": lambda: v.view(np.uint32), "bf16": lambda: fp32_to_bf16_bits(v),
            "f16": lambda: fp32_to_f16_bits(v)}[kind]()


def _check(a, sa, b, sb, kind, da=None, db=None):
    out = torch.full((a.shape[0], b.shape[0]), float("nan"), dtype=TORCH[kind], device="cuda")
    qrs.matmul_int8(device(a) if da is None else da, device(sa), device(b) if db is None else db, device(sb), out)
    got, want = out_bits(out), _bits(scaled_product(a, sa, b, sb), kind)
    bad = np.argwhere(got != want)
    assert bad.size == 0, (len(bad), bad[:4])


SIZES = [
    # one token to a few, every row of a fragment
    (1, 8192, 512), (1, 1, 16), (1, 33, 48), (2, 100, 4096), (3, 640, 1040), (7, 64, 8192), (8, 2048, 2064),
    (15, 200, 272), (16, 1000, 1024), (17, 512, 640), (24, 96, 7168), (31, 77, 96), (32, 4096, 256), (33, 130, 1600),
    (48, 256, 4112), (63, 63, 64), (64, 640, 512),
    # tiles and their edges
    (65, 129, 128), (100, 1000, 1008), (127, 255, 144), (128, 128, 128), (129, 257, 272), (200, 520, 2048),
    (255, 511, 528), (256, 256, 256), (257, 640, 384), (333, 1280, 1792), (400, 2000, 80), (512, 512, 4096),
    (513, 769, 1152), (777, 1111, 336), (1024, 1024, 1024), (1100, 2304, 512), (2048, 1000, 208),
]


@pytest.mark.parametrize("m,n,k", SIZES, ids=lambda v: str(v))
def test_product(gpu, m, n, k):
    rng = np.random.default_rng([m, n, k])
    _check(*_operands(rng, m, n, k), kind=["bf16", "f16", "f32"][(m + n + k // 16) % 3])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 5, 3), (3, 7, 15), (2, 130, 17), (66, 65, 100), (130, 131, 1001),
                                   (5, 1000, 4095)])
def test_product_at_any_k(gpu, m, n, k, kind):
    rng = np.random.default_rng([m, n, k])
    _check(*_operands(rng, m, n, k), kind=kind)


@pytest.mark.parametrize("m,n", [(1, 300), (40, 70), (300, 300)])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_product_of_rows_off_their_lines(gpu, m, n, shift):
    """Operands that start off 16-byte boundaries, or whose row stride is no
    multiple of 16; what lies beside them is 127 and must not be added."""
    rng = np.random.default_rng([m, n, shift])
    a, sa, b, sb = _operands(rng, m, n, 256)
    _check(a, sa, b, sb, "f32", da=padded(device(a), shift, 16 - shift, 127)[1])
    _check(a, sa, b, sb, "f32", db=padded(device(b), 0, shift, 127)[1])


@pytest.mark.parametrize("m,n,k", [(1, 200, 528), (16, 128, 1040), (40, 300, 272), (300, 520, 176), (600, 900, 400)])
def test_product_of_column_ranges(gpu, m, n, k):
    rng = np.random.default_rng([m, n, k, 1])
    a, sa, b, sb = _operands(rng, m, n, k)
    da, db = padded(device(a), 16, 32, 127)[1], padded(device(b), 32, 16, -128)[1]
    for left, right in [(8, 8), (1, 2)]:
        buf, out = padded(torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), left, right, 5.0)
        qrs.matmul_int8(da, device(sa), db, device(sb), out)
        assert np.array_equal(out_bits(out.contiguous()), _bits(scaled_product(a, sa, b, sb), "bf16"))
        assert torch.all(buf[:, :left] == 5) and torch.all(buf[:, left + n:] == 5)


@pytest.mark.parametrize("m", [1, 20, 130, 300])
def test_product_at_the_largest_sums(gpu, m):
    """k = 131071 rounds of (-128)^2: just below 2^31; and k = 131056 of the
    same on the aligned path."""
    for k in (131071, 131056):
        a, b = np.full((m, k), -128, dtype=np.int8), np.full((3, k), -128, dtype=np.int8)
        _check(a, np.ones(m, np.float32), b, np.ones(3, np.float32), "f32")


@pytest.mark.parametrize("far", ["a", "b", "out"])
@pytest.mark.parametrize("m,n,k", [(12, 300, 80), (140, 200, 144)])
def test_product_of_far_rows(gpu, m, n, k, far):
    """Rows 4 MiB and more apart: a tile's rows span more than 2^30 bytes."""
    rng = np.random.default_rng([m, n, k, 5])
    a, sa, b, sb = _operands(rng, m, n, k)
    spread = lambda t, stride: torch.empty_strided(t.shape, (stride, 1), dtype=t.dtype, device="cuda").copy_(t)
    da, db = device(a), device(b)
    if far == "a":
        da = spread(da, (1 << 22) + 16)
    if far == "b":
        db = spread(db, (1 << 22) + 32)
    out = spread(torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda"), (1 << 22) + 8 if far == "out" else n)
    qrs.matmul_int8(da, device(sa), db, device(sb), out)
    assert np.array_equal(out_bits(out.contiguous()), _bits(scaled_product(a, sa, b, sb), "bf16"))


def test_whole_tiles_of_far_rows(gpu):
    """Whole tiles of the largest size, whose output rows lie 4 MiB apart."""
    rng = np.random.default_rng(6)
    m, n, k = 2048, 5120, 144
    a, sa, b, sb = _operands(rng, m, n, k)
    out = torch.empty_strided((m, n), ((1 << 21) + 8, 1), dtype=torch.bfloat16, device="cuda")
    qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out)
    assert np.array_equal(out_bits(out.contiguous()), _bits(scaled_product(a, sa, b, sb), "bf16"))


def test_scales_that_are_not_finite_propagate(gpu):
    rng = np.random.default_rng(2)
    a, sa, b, sb = _operands(rng, 40, 200, 64)
    sa[3], sb[7], sb[8] = np.nan, np.inf, 0
    out = torch.empty(40, 200, device="cuda")
    qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out)
    with np.errstate(invalid="ignore"):
        want = scaled_product(a, sa, b, sb)
    assert np.array_equal(host(out), want, equal_nan=True)


GATED = [(1, 1, 16), (1, 2048, 1024), (4, 100, 272), (16, 1792, 512), (17, 33, 64), (64, 256, 2048), (100, 130, 96),
         (128, 128, 256), (130, 1000, 528), (333, 640, 1024), (600, 700, 304), (1030, 1280, 512), (3, 9, 35)]


@pytest.mark.parametrize("m,n,k", GATED)
def test_gated(gpu, m, n, k):
    rng = np.random.default_rng([m, n, k, 2])
    a, sa, b, sb = _operands(rng, m, 2 * n, k, full=False)
    # Gates of a few units, both signs.
    sa, sb = np.full(m, 2.0 ** -6, np.float32), np.full(2 * n, np.float32(2.0 ** -6 / np.sqrt(k)))
    kind = ["bf16", "f16", "f32"][(m + n) % 3]
    out = torch.full((m, n), float("nan"), dtype=TORCH[kind], device="cuda")
    qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out, gated=True)
    want = gated(scaled_product(a, sa, b, sb))
    # exp within a step and a half, then a sum, a quotient and a product; the
    # output's rounding; and where exp(-g) overflows the quotient is 0
    # instead of less than 2^-120.
    tol = np.abs(want) * (6 * STEP * 2 + HALF_STEP[kind] * 1.001) + 2.0 ** -100
    tol = tol + (2.0 ** -25 if kind == "f16" else 0)
    assert np.all(np.abs(host(out) - want) <= tol)


def test_gated_at_large_gates(gpu):
    """Gates from -1000 to 1000: exp overflows and underflows."""
    n = 64
    a = np.ones((1, 16), np.int8)
    b = np.ones((2 * n, 16), np.int8)
    g = np.linspace(-1000, 1000, n)
    sb = np.concatenate([g / 16, np.full(n, 1.0 / 16)]).astype(np.float32)
    out = torch.empty(1, n, device="cuda")
    qrs.matmul_int8(device(a), device(np.ones(1, np.float32)), device(b), device(sb), out, gated=True)
    want = gated(scaled_product(a, np.ones(1, np.float32), b, sb))
    assert np.all(np.abs(host(out) - want) <= np.abs(want) * 16 * STEP + 2.0 ** -100)


def test_gated_at_gates_of_any_size(gpu):
    """silu(g) is 0 for large negative gates, however large, and g / (1 +
    exp(-g)) of an infinity or NaN is what the formula gives."""
    g = np.array([-3e38, -1e30, -1e4, -104, -89, -88, -87, 0, 1e30, 3e38, np.inf, -np.inf, np.nan], np.float32)
    n = len(g)
    a, b = np.zeros((40, 16), np.int8), np.zeros((2 * n, 16), np.int8)
    a[:, 0] = b[:, 0] = 1
    sb = np.concatenate([g, np.ones(n, np.float32)])
    with np.errstate(over="ignore", invalid="ignore"):
        want = g.astype(np.float64) / (1.0 + np.exp(-g.astype(np.float64)))
    bound = np.where(np.isfinite(want), np.abs(want) * 16 * STEP + 2.0 ** -100, 0.0)
    for m in (1, 20, 40):
        out = torch.empty(m, n, device="cuda")
        qrs.matmul_int8(device(a[:m]), device(np.ones(m, np.float32)), device(b), device(sb), out, gated=True)
        got = host(out)
        with np.errstate(invalid="ignore"):
            assert np.all((np.abs(got - want) <= bound) | (got == want) | (np.isnan(got) & np.isnan(want))), got[0]


MODES = [("int8", "f32_group128"), ("e4m3fn", "f32_group128"), ("e5m2", "f32_group128"), ("e4m3fn", "e8m0_block32"),
         ("e5m2", "e8m0_block32")]


@pytest.mark.parametrize("x_format,layout", MODES)
@pytest.mark.parametrize("m,n,k", [(1, 128, 16), (1, 4096, 1024), (5, 256, 3584), (16, 1024, 272), (33, 384, 64),
                                   (64, 2048, 512), (130, 640, 1040), (300, 1280, 256), (1030, 2048, 512),
                                   (7, 128, 37)])
def test_quantized_product(gpu, m, n, k, x_format, layout):
    rng = np.random.default_rng([m, n, k, 3])
    a, sa, b, sb = _operands(rng, m, n, k)
    if m > 2:
        sa[1] = 0  # a row of zeros
    codes, scales = empty_codes(m, n, layout)
    qrs.matmul_int8_quantize(device(a), device(sa), device(b), device(sb), codes, scales, x_format, layout)
    c, s = quantize_values(scaled_product(a, sa, b, sb), x_format, layout)
    assert np.array_equal(scales.cpu().numpy().reshape(s.shape), s)
    got = codes.cpu().numpy()
    # Zero rows may keep the sign of zero in floating codes.
    bad = (got != c) & ((got & 0x7F) != 0) if x_format != "int8" else got != c
    assert not bad.any(), np.argwhere(bad)[:4]


@pytest.mark.parametrize("m,n,k", [(3, 256, 64), (30, 256, 64), (200, 512, 128), (2048, 5120, 144), (3, 256, 17)])
@pytest.mark.parametrize("x_format,layout", [("int8", "f32_group128"), ("e4m3fn", "e8m0_block32")])
def test_quantized_product_that_is_not_finite(gpu, m, n, k, x_format, layout):
    """NaN and infinite scales, and sums that overflow, show in the scales of
    their groups; the other groups are the oracle's."""
    rng = np.random.default_rng([m, n, k, 4])
    a, sa, b, sb = _operands(rng, m, n, k)
    clean, clean_scales = quantize_values(scaled_product(a, sa, b, sb), x_format, layout)
    a[1], b[5], b[37] = 127, 127, 0
    a[m - 1] = b[n - 1] = b[70]
    sa[m - 1], sb[n - 1], sb[140] = np.nan, np.inf, np.nan
    # Row 1: infinite where a sum is not 0, NaN where its b scale is 0 then.
    sa[1], sb[5], sb[6] = 2.0 ** 127, 0, 2.0 ** -10
    # Channels 32 .. 63 of row 1: a NaN beside finite numbers.
    b[32:64] = 0
    b[40], sb[40] = 1, 0
    codes, scales = empty_codes(m, n, layout)
    qrs.matmul_int8_quantize(device(a), device(sa), device(b), device(sb), codes, scales, x_format, layout)
    with np.errstate(all="ignore"):
        v = scaled_product(a, sa, b, sb)
    g = 128 if layout == "f32_group128" else 32
    good = np.isfinite(v.reshape(m, n // g, g)).all(axis=2)
    if g == 32:
        assert not good[1, 1] and np.isnan(v[1, 40]) and np.isfinite(v[1, 41:64]).all()
    assert not good[m - 1].any() and not good[:, n // g - 1].all() and not good[:, 140 // g].any() and good.any()
    got = scales.cpu().numpy().reshape(good.shape)
    assert np.array_equal(got != 255 if layout == "e8m0_block32" else np.isfinite(got), good)
    c, s = quantize_values(np.where(np.repeat(good, g, axis=1), v, 0), x_format, layout)
    assert np.array_equal(got[good], s.reshape(good.shape)[good])
    where = np.repeat(good, g, axis=1) & (np.abs(v) > 0)
    assert np.array_equal(codes.cpu().numpy()[where], c[where])


def test_quantized_product_feeds_a_share(gpu):
    """Four ranks' partial products through run_all_shares: the oracle's bits."""
    import oracle

    rng = np.random.default_rng(9)
    w, bs, h, k = 4, 32, 1024, 256
    p = qrs.plan(w, bs, h, "e4m3fn", "e8m0_block32", "bf16")
    dx, ds, cx, cs = [], [], [], []
    for _ in range(w):
        a, sa, b, sb = _operands(rng, bs, h, k)
        codes, scales = empty_codes(bs, h, "e8m0_block32")
        qrs.matmul_int8_quantize(device(a), device(sa), device(b), device(sb), codes, scales, "e4m3fn", "e8m0_block32")
        dx.append(codes)
        ds.append(scales)
        c, s = quantize_values(scaled_product(a, sa, b, sb), "e4m3fn", "e8m0_block32")
        cx.append(c)
        cs.append(s)
    outs = [torch.empty(bs // w, h, dtype=torch.bfloat16, device="cuda") for _ in range(w)]
    qrs.run_all_shares(p, dx, ds, outs)
    want = oracle.all_shares(cx, cs, "e4m3fn", "e8m0_block32", "bf16")
    for got, ref in zip(outs, want):
        g, r = out_bits(got), oracle_bits(ref, "bf16")
        assert np.all((g == r) | (((g | r) & 0x7FFF) == 0))


def test_random_sizes(gpu):
    rng = np.random.default_rng(77)
    for case in range(60):
        m, n = (int(np.exp(rng.uniform(0, np.log(1200)))) for _ in range(2))
        k = int(np.exp(rng.uniform(0, np.log(4000))))
        k = k if case % 4 == 0 else -(-k // 16) * 16
        print(f"case {case}: m={m} n={n} k={k}", flush=True)
        _check(*_operands(rng, m, n, k), kind=["bf16", "f16", "f32"][case % 3])
