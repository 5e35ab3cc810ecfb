"""Helpers of the GPU tests of the 8-bit floating-point operators: seeded
operands, and how far results may be from the oracle's values."""

import numpy as np
import torch

import oracle
from layer_util import STEP, decode, device, group_size, half_step
from oracle.blocks import dequantize, product
from oracle.decode import decode_table
from oracle.quantize import EMAX_ELEM, QMAX, encode_fp8_rne

FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
G = 128


def up(n, step=G):
    return -(-n // step)


def fp8(codes, kind):
    return device(codes).view(FP8[kind])


class Operands:
    """Codes and scales of both operands, and what they stand for.

    ``whole``: small whole numbers and scales of powers of two, so that every
    product and every sum, in whatever order, is a binary32 number: results are
    the oracle's bit for bit."""

    def __init__(self, rng, m, n, k, a_kind="e4m3fn", b_kind="e4m3fn", gated=False, grouped=False, whole=False):
        self.m, self.n, self.k, self.gated = m, n, k, gated
        self.a_kind, self.b_kind = a_kind, b_kind
        wide = 2 * n if gated else n
        rows = wide if grouped else 2 * up(n) if gated else up(n)
        if whole:
            # |sum of a group| <= 9 * 128, times scales of 1 to 4 and 1/2 to 2: below 2^24 halves for k <= 2^17.
            draw = lambda kind, r: encode_fp8_rne(rng.integers(-3, 4, (r, k)).astype(np.float32), kind)
            self.sa = np.exp2(rng.integers(0, 3, (m, up(k)))).astype(np.float32)
            self.sb = np.exp2(rng.integers(-1, 2, (rows, up(k)))).astype(np.float32)
        else:
            draw = lambda kind, r: encode_fp8_rne(
                np.clip(rng.standard_normal((r, k)) * QMAX[kind] / 4.5, -QMAX[kind], QMAX[kind]).astype(np.float32), kind)
            self.sa = np.exp2(rng.uniform(-12, -8, (m, up(k)))).astype(np.float32)
            self.sb = np.exp2(rng.uniform(-14, -10, (rows, up(k)))).astype(np.float32)
        self.a, self.b = draw(a_kind, m), draw(b_kind, wide)
        self.grouped = grouped

    def device(self):
        return fp8(self.a, self.a_kind), device(self.sa), fp8(self.b, self.b_kind), device(self.sb)

    def values(self):
        """The dequantized operands in 64 bits."""
        a = dequantize(self.a, self.sa, self.a_kind, 1)
        if self.grouped:
            return a, dequantize(self.b, self.sb, self.b_kind, 1)
        if not self.gated:
            return a, dequantize(self.b, self.sb, self.b_kind, G)
        blocks = up(self.n)
        return a, np.concatenate([dequantize(self.b[:self.n], self.sb[:blocks], self.b_kind, G),
                                  dequantize(self.b[self.n:], self.sb[blocks:], self.b_kind, G)])

    def want(self):
        """(value, bound of the kernel's error) in binary32, before the output's rounding."""
        p, size = product(*self.values())
        tol = product_bound(size, self.k)
        if not self.gated:
            return p, tol
        n = self.n
        g, u = p[:, :n], p[:, n:]
        s = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
        # silu's slope is at most 1.1; its own arithmetic: five half units; the last product one.
        v = g * s * u
        return v, 1.1 * tol[:, :n] * (np.abs(u) + tol[:, n:]) + np.abs(g * s) * tol[:, n:] + np.abs(v) * 6 * STEP + 2.0 ** -100


def product_bound(size, k):
    """How far a product may be, size being the sum of the magnitudes that it
    adds. Within a group, 127 additions of exact products, each off by at most one
    unit of the last place (an instruction need not round to nearest); the scales'
    product half a unit; and a fused operation for each group, half a unit of
    partial sums each."""
    return size * (127 * 2 * STEP + STEP + up(k) * STEP) * (1 + 2.0 ** -10)


def assert_codes_within(codes, scales, y, tol, x_format, layout, what=""):
    """``assert_codes`` for values y that the kernel knows within ``tol`` each."""
    t, h = y.shape
    g = group_size(layout, h)
    blocks, tols = y.reshape(t, h // g, g), tol.reshape(t, h // g, g)
    low = np.maximum((np.abs(blocks) - tols).max(axis=2), 0)
    high = (np.abs(blocks) + tols).max(axis=2)
    scales = scales.reshape(t, h // g)
    if layout == "e8m0_block32":
        def code(a):
            _, e = np.frexp(a)
            return np.where(a == 0, 0, np.clip(e - 1 - EMAX_ELEM[x_format], -127, 127) + 127)
        bad = (scales < code(low)) | (scales > code(high))
        scale, rel = np.exp2(scales.astype(np.float64) - 127), 0.0
    else:
        floor = 2.0 ** -126
        top = QMAX[x_format]
        bad = (scales < np.maximum(low / top, floor) * (1 - 2 * STEP)) | (scales > np.maximum(high / top, floor) * (1 + 2 * STEP))
        scale, rel = scales.astype(np.float64), 4 * STEP
    assert not bad.any(), f"{what}: {np.count_nonzero(bad)} scales"
    q = np.clip(blocks / scale[:, :, None], -QMAX[x_format], QMAX[x_format])
    off = (tols / scale[:, :, None]).reshape(t, h)
    q = q.reshape(t, h)
    got = decode(codes, x_format)
    # The step is that of the larger of both where the tolerance crosses a border between steps.
    bad = np.abs(got - q) > half_step(np.maximum(np.abs(q), np.abs(got)), x_format) * (1 + 1e-12) + np.abs(q) * rel + off
    assert not bad.any(), f"{what}: {np.count_nonzero(bad)} codes, {got[bad][:3]} {q[bad][:3]}"


def float_bits(v, kind):
    """The type's bits of float64 values that round to it once (from binary32)."""
    v = np.asarray(v, dtype=np.float32)
    if kind == "f32":
        return v.view(np.uint32)
    return (oracle.reduce.fp32_to_bf16_bits if kind == "bf16" else oracle.reduce.fp32_to_f16_bits)(v)


__all__ = ["FP8", "G", "Operands", "assert_codes_within", "decode_table", "float_bits", "fp8", "product_bound", "up"]
