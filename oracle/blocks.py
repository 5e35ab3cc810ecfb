"""Layer norm, and 8-bit floating-point codes with scales of 128 x 128 blocks
and their products, from their formulas.

TEST INFRASTRUCTURE (part of the CPU oracle; see ``oracle/__init__.py``).

* ``layer_norm``: y = (s - mean) / sqrt(var + eps) * w + b in 64 bits.
* ``layer_norm_backward``: the gradients of its s, w and b, in 64 bits: what is
  left of w * dy after its mean and its part along the normalized row.
* ``quantize_groups``: the per-group rule of ``quantize_values`` for groups of any
  height and width, the last ones of a matrix smaller.
* ``dequantize``: what codes and such scales stand for.
* ``product``: the dequantized operands' product in 64 bits, and the sum of the
  magnitudes that it adds.
"""

import numpy as np

from .decode import decode_table
from .quantize import quantize_values

GROUP = 128


def layer_norm(s, w, b, eps):
    s = np.asarray(s, dtype=np.float64)
    mean = np.mean(s, axis=1, keepdims=True)
    c = s - mean
    return c / np.sqrt(np.mean(c * c, axis=1, keepdims=True) + eps) * np.asarray(w, np.float64) + np.asarray(b, np.float64)


def layer_norm_backward(grad_y, s, w, eps, grad_sum=None):
    """(grad of s, grad of w, grad of b)."""
    s, grad_y = np.asarray(s, dtype=np.float64), np.asarray(grad_y, dtype=np.float64)
    c = s - np.mean(s, axis=1, keepdims=True)
    std = np.sqrt(np.mean(c * c, axis=1, keepdims=True) + eps)
    unit = c / std
    scaled = grad_y * np.asarray(w, dtype=np.float64)
    grad_s = (scaled - np.mean(scaled, axis=1, keepdims=True) - unit * np.mean(scaled * unit, axis=1, keepdims=True)) / std
    if grad_sum is not None:
        grad_s = grad_s + np.asarray(grad_sum, dtype=np.float64)
    return grad_s, np.sum(grad_y * unit, axis=0), np.sum(grad_y, axis=0)


def quantize_groups(v, x_format, height, width):
    """binary32 [r, c] -> (uint8 codes [r, c], float32 scales [ceil(r / height), ceil(c / width)])."""
    v = np.asarray(v, dtype=np.float32)
    r, c = v.shape
    rows, cols = -(-r // height), -(-c // width)
    padded = np.zeros((rows * height, cols * width), np.float32)
    padded[:r, :c] = v
    groups = padded.reshape(rows, height, cols, width).transpose(0, 2, 1, 3).reshape(rows * cols, height * width)
    codes, scales = quantize_values(groups, x_format, "f32_row")
    codes = codes.reshape(rows, cols, height, width).transpose(0, 2, 1, 3).reshape(padded.shape)
    return np.ascontiguousarray(codes[:r, :c]), scales.reshape(rows, cols)


def spread(scales, shape, height, width):
    """A scale for each element."""
    full = np.repeat(np.repeat(scales, height, axis=0), width, axis=1)
    return full[:shape[0], :shape[1]]


def dequantize(codes, scales, x_format, height, width=GROUP):
    values = decode_table(x_format)[codes].astype(np.float64)
    return values * spread(np.asarray(scales, np.float64), codes.shape, height, width)


def product(a, b):
    """Dequantized [m, k] and [n, k] -> (product, sum of magnitudes), in 64 bits."""
    return a @ b.T, np.abs(a) @ np.abs(b).T
