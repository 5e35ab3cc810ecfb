"""Pins of oracle/layer.py: gradients against differences, the scaled product
against Python integers, row scales against the per-group rule."""

import numpy as np
import pytest

from oracle.layer import HALF_STEP, gated, rms_norm, rms_norm_backward, round_to, rounded_sum, scaled_product
from oracle.quantize import quantize_values

EPS = 1e-5


def test_norm_of_a_constant_row_is_its_sign_times_the_weight():
    s = np.array([[3.0] * 8, [-0.5] * 8])
    w = np.arange(8, dtype=np.float64)
    y = rms_norm(s, w, 0.0)
    assert np.array_equal(y, np.sign(s) * w)


def test_norm_of_a_zero_row_is_zero():
    assert np.array_equal(rms_norm(np.zeros((1, 5)), np.ones(5), EPS), np.zeros((1, 5)))


@pytest.mark.parametrize("t,h", [(1, 1), (1, 7), (5, 16), (3, 33)])
def test_gradients_against_central_differences(t, h):
    rng = np.random.default_rng(t * 100 + h)
    s, w, dy, ds = (rng.standard_normal(shape) for shape in ((t, h), h, (t, h), (t, h)))

    def loss(s_, w_):
        return np.sum(rms_norm(s_, w_, EPS) * dy) + np.sum(s_ * ds)

    gs, gw = rms_norm_backward(dy, s, w, EPS, ds)
    # Central differences: an error of step^2 / 6 times the third derivative
    # (at most a few dozen / rms^3 here) plus 2^-52 * |loss| / step.
    step = 1e-5
    for i in range(t):
        for j in range(h):
            d = np.zeros_like(s)
            d[i, j] = step
            rms = np.sqrt(np.mean(s[i] ** 2) + EPS)
            tol = 100 * step * step / rms ** 3 + 1e-8
            assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * step) - gs[i, j]) < tol * (1 + np.abs(dy[i]).sum())
    for j in range(h):
        d = np.zeros_like(w)
        d[j] = step
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * step) - gw[j]) < 1e-8  # linear in w


def test_gradient_without_a_residual_gradient_is_with_zeros():
    rng = np.random.default_rng(3)
    s, dy, w = rng.standard_normal((4, 12)), rng.standard_normal((4, 12)), rng.standard_normal(12)
    a, b = rms_norm_backward(dy, s, w, EPS), rms_norm_backward(dy, s, w, EPS, np.zeros((4, 12)))
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_product_against_python_integers():
    rng = np.random.default_rng(1)
    a = rng.integers(-128, 128, size=(3, 300), dtype=np.int8)
    b = rng.integers(-128, 128, size=(5, 300), dtype=np.int8)
    sa, sb = rng.uniform(0.1, 2, 3).astype(np.float32), rng.uniform(0.1, 2, 5).astype(np.float32)
    got = scaled_product(a, sa, b, sb)
    for i in range(3):
        for j in range(5):
            p = sum(int(x) * int(y) for x, y in zip(a[i], b[j]))
            assert got[i, j] == np.float32(np.float32(np.float32(p) * sa[i]) * sb[j])


def test_product_at_the_largest_k_is_exact():
    k = 131071
    a = np.full((1, k), -128, dtype=np.int8)
    one = np.ones(1, dtype=np.float32)
    assert scaled_product(a, one, a, one)[0, 0] == np.float32(16384 * k)
    assert 16384 * k < 2 ** 31 <= 16384 * (k + 1)


def test_gated_is_silu_times_up():
    p = np.array([[0.0, 2.0, -1e4, 5.0, 7.0, 3.0]], dtype=np.float32)
    got = gated(p)
    assert got[0, 0] == 0.0
    assert got[0, 1] == pytest.approx(2.0 / (1 + np.exp(-2.0)) * 7.0, rel=1e-14)
    assert abs(got[0, 2]) < 1e-290


@pytest.mark.parametrize("x_format", ["int8", "e4m3fn", "e5m2"])
def test_row_scales_are_the_group_rule_on_whole_rows(x_format):
    v = np.random.default_rng(2).standard_normal((6, 128)).astype(np.float32)
    v[3] = 0
    c, s = quantize_values(v, x_format, "f32_row")
    gc, gs = quantize_values(v, x_format, "f32_group128")
    assert np.array_equal(c, gc) and np.array_equal(s, gs)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_rounding_moves_a_value_by_at_most_half_a_step(kind):
    rng = np.random.default_rng(4)
    x, r = (round_to(rng.standard_normal((8, 64)), kind) for _ in range(2))
    s = rounded_sum(x, r, kind)
    want = x.astype(np.float64) + r
    assert np.all(np.abs(s - want) <= HALF_STEP[kind] * np.abs(want))
    assert np.array_equal(round_to(s, kind), s)
