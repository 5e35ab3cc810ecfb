"""add_rms_norm_quantize to the accuracy that qrs.h states, and rows_kernel's
walk over many more rows than work-groups."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, TORCH, assert_codes, device, empty_codes, host, values
from oracle.layer import rms_norm, round_to, rounded_sum
from oracle.quantize import quantize_values

pytestmark = pytest.mark.gpu

EPS = 1e-5
# Half steps of binary32 that y may be off: three of its products, and in r half
# of what a piece's squares gather (binary64 throughout for E8M0 scales, whose
# codes are then the real number's).
REL = {"bf16": 6.5, "f16": 6.5, "f32": 5.0}


def _rel(kind, layout):
    return 2.0 ** -40 if layout == "e8m0_block32" else REL[kind] * STEP * (1 + 2.0 ** -20)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("x_format,layout", [("int8", "f32_row"), ("e4m3fn", "f32_group128"), ("e5m2", "f32_row"),
                                             ("e4m3fn", "e8m0_block32")])
@pytest.mark.parametrize("t,h", [(400, 1024), (300, 4096), (64, 8192), (20, 16384), (6, 65536)])
def test_norm_to_the_stated_accuracy(gpu, t, h, x_format, layout, kind):
    """Rows of one value repeated (every piece rounds the same way), rows of two
    values, and ordinary ones."""
    rng = np.random.default_rng([t, h, 21])
    s = values(rng, (t, h), kind)
    s[::3] = round_to(1 + rng.random((len(s[::3]), 1)).astype(np.float32), kind)
    s[1::3] = np.where(rng.random((len(s[1::3]), h)) < 0.5, s[1::3, :1], s[1::3, 1:2])
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    codes, scales = empty_codes(t, h, layout)
    qrs.add_rms_norm_quantize(device(s, kind), None, device(w, kind), EPS, None, codes, scales, x_format, layout)
    assert_codes(codes.cpu().numpy(), scales.cpu().numpy(), rms_norm(s, w, EPS), _rel(kind, layout), x_format, layout)


@pytest.mark.parametrize("kind,x_format,layout", [("bf16", "int8", "f32_row"), ("f32", "e4m3fn", "f32_group128"),
                                                  ("f16", "e5m2", "e8m0_block32")])
@pytest.mark.parametrize("t,h", [(9001, 1024), (13000, 128), (8200, 4096), (4097, 2048)])
def test_norm_of_more_rows_than_work_groups(gpu, t, h, x_format, layout, kind):
    rng = np.random.default_rng([t, h, 22])
    x = values(rng, (t, h), kind) * np.exp2(rng.integers(-6, 7, (t, 1))).astype(np.float32)
    x, r = round_to(x, kind), values(rng, (t, h), kind, 2)
    w = round_to(values(rng, h, kind, 0.1) + np.float32(1), kind)
    x[4096] = r[4096] = 0  # a second row of the first work-group, taken in binary64
    codes, scales = empty_codes(t, h, layout)
    total = torch.empty(t, h, dtype=TORCH[kind], device="cuda")
    qrs.add_rms_norm_quantize(device(x, kind), device(r, kind), device(w, kind), EPS, total, codes, scales, x_format,
                              layout)
    s = rounded_sum(x, r, kind)
    assert np.array_equal(host(total), s)
    assert_codes(codes.cpu().numpy(), scales.cpu().numpy(), rms_norm(s, w, EPS), _rel(kind, layout), x_format, layout)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("t,h", [(9001, 1024), (12500, 33), (8200, 4096), (4500, 8192), (4100, 10000), (4099, 16384),
                                 (20000, 8)])
def test_quantize_rows_of_more_rows_than_work_groups(gpu, t, h, kind):
    rng = np.random.default_rng([t, h, 23])
    v = values(rng, (t, h), kind)
    v[::7] *= np.float32(16)
    v[5::911] = 0
    codes, scales = empty_codes(t, h, "f32_row")
    qrs.quantize_rows(device(v, kind), codes, scales)
    c, s = quantize_values(v, "int8", "f32_row")
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), s[:, 0].view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), c)
