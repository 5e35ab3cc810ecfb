"""GPU parity of the 8-bit floating-point product at sizes that take the tiles of
many tokens, one and several of them a work-group, whole and ragged, against
float64 products on the device; and what 16-bit outputs, whose tiles multiply the
codes in 8-bit instructions, may be off by."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import Operands, assert_codes_within, up
from layer_util import STEP, TORCH, empty_codes
from oracle.layer import HALF_STEP
from oracle.quantize import quantize_values

pytestmark = pytest.mark.gpu

# Tokens, outputs (a gated product of half as many has as many tiles), k: one tile a
# work-group, several, one group of k, a part of one.
PIPE = [(4096, 4096, 160), (4100, 8200, 272), (4099, 4111, 128), (4352, 4096, 16), (2049, 8321, 1040),
        (4095, 4093, 144)]
MID = [(130, 900, 272), (333, 5003, 400), (700, 4096, 1040), (64, 256, 128), (1000, 8200, 144), (256, 4096, 528),
       (512, 4096, 272)]


def _want(o):
    """The product and the sum of the magnitudes that it adds, float64 on the device."""
    a, b = (torch.from_numpy(v).cuda() for v in o.values())
    return a @ b.t(), a.abs() @ b.abs().t()


def _kernel(o, **form):
    return qrs.matmul_fp8_launch_info(o.m, o.n, o.k, o.gated, b_scale_rows=1 if o.grouped else 128, **form)["kernel"]


def _silu(p):
    g, u = p.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _instruction_bound(size, kind, k):
    """What sums may be off by. Binary32 outputs: product_bound's. 16-bit ones: each
    eight products are added with a last place of 2^-14 of the largest's power of two,
    which is at most 2^-14 of the sum of their magnitudes, each of the eight off by
    less than one: 2^-11 of that sum."""
    eights = 0.0 if kind == "f32" else 2.0 ** -11
    return size * (eights + 127 * 2 * STEP + STEP + up(k) * STEP) * (1 + 2.0 ** -10)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("form", ["block", "group", "gated"])
@pytest.mark.parametrize("m,n,k", PIPE + MID, ids=lambda v: str(v))
def test_whole_numbers(gpu, m, n, k, form, kind):
    rng = np.random.default_rng([m, n, k])
    gated = form == "gated"
    o = Operands(rng, m, n // 2 if gated else n, k, ["e4m3fn", "e5m2"][m % 2], ["e4m3fn", "e5m2"][n % 2], gated=gated,
                 grouped=form == "group", whole=True)
    assert _kernel(o, out_dtype=kind) in ("pipe", "mid")
    if gated:
        o.sa *= np.float32(2.0 ** -np.round(np.log2(k) / 2 + 2))
    buf = torch.full((m, o.n + 16), 7.0, dtype=TORCH[kind], device="cuda")
    out = buf[:, 8:8 + o.n]
    qrs.matmul_fp8(*o.device(), out, gated=gated)
    p, _ = _want(o)
    if gated:
        want = _silu(p)
        # silu's five half units, the product's one, the output's.
        bound = want.abs() * (6 * 2 * STEP + HALF_STEP[kind] * 1.001) + 2.0 ** -100 + (2.0 ** -25 if kind == "f16" else 0)
        assert ((out.double() - want).abs() <= bound).all()
    else:
        assert torch.equal(out, p.float().to(TORCH[kind]))
    assert (buf[:, :8] == 7).all() and (buf[:, 8 + o.n:] == 7).all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("form", ["block", "group", "gated"])
@pytest.mark.parametrize("types", [("e4m3fn", "e4m3fn"), ("e5m2", "e4m3fn"), ("e4m3fn", "e5m2"), ("e5m2", "e5m2")],
                         ids=lambda t: "-".join(t))
@pytest.mark.parametrize("m,n,k", [(4100, 4352, 528), (1000, 8200, 400), (333, 2050, 1168), (130, 900, 272)])
def test_any_values(gpu, m, n, k, types, form, kind):
    rng = np.random.default_rng([m, n, k, 1])
    gated = form == "gated"
    o = Operands(rng, m, n // 2 if gated else n, k, *types, gated=gated, grouped=form == "group")
    # Results of about one, which half precision holds.
    rms = float(np.sqrt(np.mean(_want(Operands(rng, 64, 64, k, *types))[0].cpu().numpy() ** 2)))
    o.sb /= np.float32(2.0 ** np.round(np.log2(rms)))
    out = torch.full((m, o.n), float("nan"), dtype=TORCH[kind], device="cuda")
    qrs.matmul_fp8(*o.device(), out, gated=gated)
    p, size = _want(o)
    tol = _instruction_bound(size, kind, k)
    if gated:
        g, u = p.chunk(2, dim=1)
        tg, tu = tol.chunk(2, dim=1)
        p, s = _silu(p), 1 / (1 + torch.exp(-g))
        # silu's slope is at most 1.1, its arithmetic five half units, the product one.
        tol = 1.1 * tg * (u.abs() + tu) + (g * s).abs() * tu + p.abs() * 6 * STEP + 2.0 ** -100
    tol = tol * (1 + HALF_STEP[kind]) + p.abs() * HALF_STEP[kind] + (2.0 ** -25 if kind == "f16" else 0)
    off = (out.double() - p).abs()
    assert (off <= tol).all(), float((off / tol).max())


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(4100, 4352, 400), (1000, 8200, 400), (300, 900, 400)])
def test_codes_and_scales_that_are_not_finite(gpu, m, n, k, kind):
    rng = np.random.default_rng([m, n])
    o = Operands(rng, m, n, k, "e5m2", "e4m3fn", whole=True)
    o.b[7, 130], o.b[n - 1, 5], o.b[260:300] = 0x7F, 0xFF, 0  # NaN; rows of zeros
    o.a[0, 300], o.a[m - 1, 300] = 0x7C, 0xFC  # infinities
    o.sa[m - 3, 1], o.sa[5, up(k) - 1] = np.nan, np.inf
    out = torch.empty(m, n, dtype=TORCH[kind], device="cuda")
    qrs.matmul_fp8(*o.device(), out)
    # A group's sum first, then its scales, as the operation is defined.
    sa, o.sa = torch.from_numpy(o.sa.astype(np.float64)).cuda(), np.ones_like(o.sa)
    with np.errstate(invalid="ignore"):
        a, b = (torch.from_numpy(v).cuda() for v in o.values())
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for g in range(up(k)):
        part = slice(g * 128, min((g + 1) * 128, k))
        want = want + a[:, part] @ b[:, part].t() * sa[:, g:g + 1]
    want = want.float().to(TORCH[kind])
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    keep = ~torch.isnan(want)
    assert torch.equal(out[keep], want[keep])


MODES = [("int8", "f32_group128"), ("e4m3fn", "f32_group128"), ("e5m2", "e8m0_block32")]


@pytest.mark.parametrize("x_format,layout", MODES)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("m,n,k", [(4096, 4096, 160), (4100, 8192, 272), (300, 4096, 400), (1000, 1024, 400)])
def test_codes(gpu, m, n, k, gated, x_format, layout):
    rng = np.random.default_rng([m, n, k, 3])
    o = Operands(rng, m, n // 2 if gated else n, k, gated=gated, whole=not gated)
    codes, scales = empty_codes(m, o.n, layout)
    qrs.matmul_fp8_quantize(*o.device(), codes, scales, x_format, layout, gated=gated)
    rows = np.unique(np.concatenate([np.arange(0, m, 37), [0, 63, 64, 255, 256, m - 1]]) % m)
    got, got_s = codes[rows].cpu().numpy(), scales.reshape(m, -1)[rows].cpu().numpy()
    o.a, o.sa, o.m = o.a[rows], o.sa[rows], len(rows)
    want, tol = o.want()
    if gated:
        assert_codes_within(got, got_s, want, tol, x_format, layout)
        return
    c, s = quantize_values(want.astype(np.float32), x_format, layout)
    assert np.array_equal(got_s, s)
    bad = (got != c) & (((got | c) & 0x7F) != 0) if x_format != "int8" else got != c
    assert not bad.any(), np.argwhere(bad)[:4]


def test_rows_of_whole_tiles_far_apart(gpu):
    """Whole tiles of the largest size, whose output rows lie 4 MiB apart."""
    o = Operands(np.random.default_rng(6), 4096, 4096, 160, whole=True)
    out = torch.empty_strided((4096, 4096), ((1 << 21) + 8, 1), dtype=torch.bfloat16, device="cuda")
    qrs.matmul_fp8(*o.device(), out)
    assert torch.equal(out.contiguous(), _want(o)[0].float().bfloat16())
