"""The operators between two shares, from their formulas.

TEST INFRASTRUCTURE (part of the CPU oracle; see ``oracle/__init__.py``).

* ``rounded_sum``: x + residual rounded once to the activations' type.
* ``rms_norm``: y = s / sqrt(mean(s^2) + eps) * w in 64 bits.
* ``rms_norm_backward``: the gradients of its s and w, in 64 bits, written as
  the derivative of the unit vector: with u = s / rms, dy/ds projects out
  the part of w * dy along u.
* ``scaled_product``: the integer product (exact in int64) as binary32 times
  the token's and then the channel's scale: one rounding each, so this is
  the definition bit for bit.
* ``gated``: silu(g) * u of two binary32 products, in 64 bits.
"""

import numpy as np

from .reduce import bf16_bits_to_fp32, fp32_to_bf16_bits, fp32_to_f16_bits

# Half a step, relative to the value: how far a rounding may move it.
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def round_to(v, kind):
    """Values rounded nearest-even to the type, as float32."""
    v = np.asarray(v, dtype=np.float32)
    if kind == "bf16":
        return bf16_bits_to_fp32(fp32_to_bf16_bits(v))
    if kind == "f16":
        return fp32_to_f16_bits(v).view(np.float16).astype(np.float32)
    return v


def rounded_sum(x, residual, kind):
    return round_to(np.asarray(x, dtype=np.float32) + np.asarray(residual, dtype=np.float32), kind)


def rms_norm(s, w, eps):
    s = np.asarray(s, dtype=np.float64)
    return s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def rms_norm_backward(grad_y, s, w, eps, grad_sum=None):
    """(grad of s, grad of w)."""
    s = np.asarray(s, dtype=np.float64)
    grad_y = np.asarray(grad_y, dtype=np.float64)
    rms = np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    unit = s / rms
    scaled = grad_y * np.asarray(w, dtype=np.float64)
    grad_s = (scaled - unit * np.mean(scaled * unit, axis=1, keepdims=True)) / rms
    if grad_sum is not None:
        grad_s = grad_s + np.asarray(grad_sum, dtype=np.float64)
    return grad_s, np.sum(grad_y * unit, axis=0)


def scaled_product(a, a_scales, b, b_scales):
    """int8 [m, k] and [n, k] -> float32 [m, n]."""
    # float64 holds every partial sum exactly: |sum| <= 2^14 * 131071 < 2^53.
    p = (a.astype(np.float64) @ b.astype(np.float64).T).astype(np.int64)
    v = p.astype(np.float32)  # nearest-even
    v = (v * np.asarray(a_scales, dtype=np.float32)[:, None]).astype(np.float32)
    return (v * np.asarray(b_scales, dtype=np.float32)[None, :]).astype(np.float32)


def gated(product):
    """binary32 [m, 2 n] (gate, then up) -> float64 [m, n]."""
    n = product.shape[1] // 2
    g, u = product[:, :n].astype(np.float64), product[:, n:].astype(np.float64)
    return g / (1.0 + np.exp(np.minimum(-g, 700.0))) * u
