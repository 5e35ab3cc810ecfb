"""The oracle of layer norm and of block-scaled codes against closed forms,
differences and another way of writing the same."""

import numpy as np
import pytest

from oracle.blocks import dequantize, layer_norm, layer_norm_backward, product, quantize_groups
from oracle.quantize import quantize_values


def test_layer_norm_closed_forms():
    y = layer_norm([[1.0, 3.0], [5.0, 5.0]], [2.0, 1.0], [10.0, 0.0], 0.0 + 1e-300)
    assert np.allclose(y[0], [8.0, 1.0]) and np.allclose(y[1], [10.0, 0.0])
    s = np.random.default_rng(0).standard_normal((3, 50))
    far = layer_norm(s + 1e6, np.ones(50), np.zeros(50), 1e-5)
    assert np.allclose(far, layer_norm(s, np.ones(50), np.zeros(50), 1e-5), atol=1e-8)


@pytest.mark.parametrize("eps", [1e-5, 0.5])
def test_layer_norm_gradients_against_differences(eps):
    rng = np.random.default_rng(1)
    s, dy, gs = (rng.standard_normal((3, 7)) for _ in range(3))
    w, b = rng.standard_normal(7), rng.standard_normal(7)

    def loss(s, w, b):
        return np.sum(layer_norm(s, w, b, eps) * dy) + np.sum(s * gs)

    grads = layer_norm_backward(dy, s, w, eps, gs)
    for i, v in enumerate((s, w, b)):
        for at in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[at] = 1e-5
            args = [s, w, b]
            up, down = ([x + sign * d if j == i else x for j, x in enumerate(args)] for sign in (1, -1))
            assert abs((loss(*up) - loss(*down)) / 2e-5 - grads[i][at]) < 1e-7


@pytest.mark.parametrize("x_format", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("shape,height,width", [((3, 256), 1, 128), ((200, 130), 128, 128), ((130, 5), 128, 1)])
def test_groups_one_at_a_time(shape, height, width, x_format):
    v = np.random.default_rng(2).standard_normal(shape).astype(np.float32)
    codes, scales = quantize_groups(v, x_format, height, width)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = v[i * height:(i + 1) * height, j * width:(j + 1) * width]
            c, s = quantize_values(part.reshape(1, -1), x_format, "f32_row")
            assert s[0, 0] == scales[i, j]
            assert np.array_equal(codes[i * height:(i + 1) * height, j * width:(j + 1) * width], c.reshape(part.shape))
    off = np.abs(dequantize(codes, scales, x_format, height, width) - v)
    assert np.all(off <= np.abs(v) * (2.0 ** -4 if x_format == "e4m3fn" else 2.0 ** -3) * 1.01 + np.repeat(
        np.repeat(scales, height, 0), width, 1)[:shape[0], :shape[1]] * 2.0 ** -9)


def test_product_adds_what_it_says():
    a, b = np.array([[1.0, -2.0, 3.0]]), np.array([[4.0, 5.0, 6.0], [0.0, 1.0, 0.0]])
    p, size = product(a, b)
    assert p.tolist() == [[12.0, -2.0]] and size.tolist() == [[32.0, 2.0]]
