"""Helpers of the GPU tests of the operators between two shares: seeded
device tensors, and how far codes may be from the oracle's values."""

import numpy as np
import torch

import oracle
from oracle.layer import round_to
from oracle.quantize import EMAX_ELEM, QMAX

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEP = 2.0 ** -24  # half a binary32 step, relative


def values(rng, shape, kind, scale=1.0):
    """Normal values that the type holds, as float32."""
    return round_to(rng.standard_normal(shape).astype(np.float32) * np.float32(scale), kind)


def device(v, kind=None):
    t = torch.from_numpy(np.ascontiguousarray(v)).cuda()
    return t if kind is None else t.to(TORCH[kind])


def padded(t, left, right, fill):
    """The same values as a column range of a wider buffer, the rest filled."""
    rows, cols = t.shape
    buf = torch.full((rows, left + cols + right), fill, dtype=t.dtype, device=t.device)
    view = buf[:, left:left + cols]
    view.copy_(t)
    return buf, view


def host(t):
    return t.float().cpu().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.cpu().numpy()


def group_size(layout, h):
    return {"f32_group128": 128, "e8m0_block32": 32, "f32_row": h}[layout]


def empty_codes(t, h, layout):
    n = h // group_size(layout, h)
    codes = torch.full((t, h), 0xAA, dtype=torch.uint8, device="cuda")
    if layout == "e8m0_block32":
        return codes, torch.full((t, n), 0xAA, dtype=torch.uint8, device="cuda")
    return codes, torch.full((t, n) if n > 1 or layout != "f32_row" else (t,), float("nan"), device="cuda")


def decode(codes, x_format):
    if x_format == "int8":
        return codes.view(np.int8).astype(np.float64)
    return oracle.decode_table(x_format)[codes].astype(np.float64)


def half_step(q, x_format):
    """Half the distance between neighbouring code values at |q|."""
    if x_format == "int8":
        return np.full(q.shape, 0.5)
    digits, low = (3, -6) if x_format == "e4m3fn" else (2, -14)
    _, e = np.frexp(np.abs(q))
    return np.exp2(np.maximum(e - 1, low).astype(np.float64) - digits) / 2


def assert_codes(codes, scales, y, rel, x_format, layout, what=""):
    """Codes and scales of float64 values y, each known to the kernel within
    `rel` of itself.

    fp32 scales: amax / qmax within rel and one rounding; E8M0: the exponent
    of some value within rel of amax, exactly. Codes: nearest to y / scale
    with the kernel's own scale, up to rel and the roundings of the
    multiplier and of the product, plus (fp32 scales: the multiplier is not
    1 / the stored scale) the scale's own rounding.
    """
    t, h = y.shape
    g = group_size(layout, h)
    blocks = y.reshape(t, h // g, g)
    amax = np.abs(blocks).max(axis=2)
    scales = scales.reshape(t, h // g)
    if layout == "e8m0_block32":
        def code(a):
            _, e = np.frexp(a)
            return np.where(a == 0, 0, np.clip(e - 1 - EMAX_ELEM[x_format], -127, 127) + 127)
        ok = (scales >= code(amax * (1 - rel))) & (scales <= code(amax * (1 + rel)))
        assert np.all(ok), f"{what}: {np.count_nonzero(~ok)} E8M0 scales"
        scale = np.exp2(scales.astype(np.float64) - 127)
        tol = rel
    else:
        want = np.maximum(amax / QMAX[x_format], 2.0 ** -126)
        bad = np.abs(scales - want) > want * (rel + 2 * STEP)
        assert not bad.any(), f"{what}: {np.count_nonzero(bad)} scales, {scales[bad][:3]} {want[bad][:3]}"
        scale = scales.astype(np.float64)
        tol = rel + 4 * STEP
    q = np.clip(blocks / scale[:, :, None], -QMAX[x_format], QMAX[x_format]).reshape(t, h)
    got = decode(codes, x_format)
    bad = np.abs(got - q) > half_step(q, x_format) * (1 + 1e-12) + np.abs(q) * tol
    assert not bad.any(), f"{what}: {np.count_nonzero(bad)} codes, {got[bad][:3]} {q[bad][:3]}"


def norm_rel(h):
    """How far the kernel's y = s * r * w may be from the exact one: at most
    64 squares a lane, then 6 lane and 16 wave additions, each square and sum
    off by half a step (half as much in r), then the mean, eps, square root,
    reciprocal and the two products."""
    return (0.5 * (min(h, 64) + 6 + 16 + 1) + 6) * STEP
