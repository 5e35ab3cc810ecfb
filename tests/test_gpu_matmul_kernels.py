"""Every kernel and tile of the products, in every form: the chosen kernel is
asserted with the whole output, so that another choice cannot leave one
untested. Sizes end inside tiles, and the pipelined kernel's work-groups walk
over several: whole ones after ragged ones and ragged ones after whole ones."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from gpu_util import out_bits
from layer_util import STEP, TORCH, device, empty_codes, host, padded
from oracle.layer import HALF_STEP, gated, scaled_product
from oracle.quantize import quantize_values
from oracle.reduce import fp32_to_bf16_bits, fp32_to_f16_bits

pytestmark = pytest.mark.gpu


def _operands(m, n, k, scale=2.0 ** -6):
    rng = np.random.default_rng([m, n, k])
    a = rng.integers(-127, 128, size=(m, k), dtype=np.int8)
    b = rng.integers(-127, 128, size=(n, k), dtype=np.int8)
    sa = (scale * np.exp2(rng.uniform(-1, 1, m))).astype(np.float32)
    sb = (scale / np.sqrt(k) * np.exp2(rng.uniform(-1, 1, n))).astype(np.float32)
    return a, sa, b, sb


def _chosen(m, n, k, kernel, tile, **form):
    info = qrs.matmul_launch_info(m, n, k, **form)
    assert (info["kernel"], info["tile"]) == (kernel, tile), info


def _bits(v, kind):
    return {"f32": lambda: v.view(np.uint32), "bf16": lambda: fp32_to_bf16_bits(v),
            "f16": lambda: fp32_to_f16_bits(v)}[kind]()


VALUES = [
    ("few_tokens", (16, 16), (9, 1000, 400)), ("few_tokens", (16, 32), (13, 5003, 272)),
    ("few_tokens", (32, 16), (31, 3320, 1040)), ("few_tokens", (32, 32), (17, 6648, 144)),
    ("mid", (64, 32), (33, 1000, 1040)), ("mid", (64, 32), (65, 40, 2064)), ("mid", (64, 64), (100, 6641, 272)),
    ("mid", (64, 128), (130, 6648, 1040)), ("mid", (128, 128), (333, 6648, 656)), ("mid", (128, 256), (700, 6648, 272)),
    ("mid", (128, 256), (2000, 4001, 1040)), ("mid", (128, 256), (4859, 5000, 112)),
    ("pipe", (256, 256), (2000, 6648, 400)), ("pipe", (256, 256), (4859, 6648, 144)),
    ("pipe", (256, 256), (4859, 6648, 272)), ("pipe", (256, 256), (4859, 6643, 400)), ("tiles", (64, 128), (200, 300, 401)),
]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kernel,tile,shape", VALUES, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_values(gpu, kernel, tile, shape, kind):
    m, n, k = shape
    _chosen(m, n, k, kernel, tile)
    a, sa, b, sb = _operands(m, n, k)
    out = torch.full((m, n), float("nan"), dtype=TORCH[kind], device="cuda")
    qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out)
    bad = np.argwhere(out_bits(out) != _bits(scaled_product(a, sa, b, sb), kind))
    assert bad.size == 0, (len(bad), bad[:4])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_values_beside_others_through_many_pipelined_tiles(gpu, kind):
    m, n, k = 4859, 6648, 272
    _chosen(m, n, k, "pipe", (256, 256))
    a, sa, b, sb = _operands(m, n, k)
    want = _bits(scaled_product(a, sa, b, sb), kind)
    for left, right in [(8, 8), (1, 3)]:
        buf, out = padded(torch.zeros(m, n, dtype=TORCH[kind], device="cuda"), left, right, 5.0)
        qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out)
        assert np.array_equal(out_bits(out.contiguous()), want)
        assert torch.all(buf[:, :left] == 5) and torch.all(buf[:, left + n:] == 5)


GATED = [
    ("few_tokens", (16, 16), (9, 1000, 400)), ("few_tokens", (16, 32), (13, 5003, 272)),
    ("few_tokens", (32, 16), (31, 2040, 1040)), ("few_tokens", (32, 32), (17, 4000, 144)),
    ("mid", (64, 32), (33, 1000, 1040)), ("mid", (64, 64), (40, 6641, 272)), ("mid", (64, 128), (100, 5000, 1040)),
    ("mid", (128, 128), (200, 5000, 656)), ("mid", (128, 256), (520, 3320, 272)), ("mid", (128, 256), (2000, 2001, 1040)),
    ("pipe", (256, 256), (1000, 5000, 400)), ("pipe", (256, 256), (4859, 3320, 144)),
    ("pipe", (256, 256), (4859, 3320, 272)), ("pipe", (256, 256), (4859, 3317, 400)), ("tiles", (64, 128), (200, 300, 401)),
]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kernel,tile,shape", GATED, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_gated(gpu, kernel, tile, shape, kind):
    m, n, k = shape
    _chosen(m, n, k, kernel, tile, gated=True)
    a, sa, b, sb = _operands(m, 2 * n, k)
    out = torch.full((m, n), float("nan"), dtype=TORCH[kind], device="cuda")
    qrs.matmul_int8(device(a), device(sa), device(b), device(sb), out, gated=True)
    want = gated(scaled_product(a, sa, b, sb))
    # silu within five half units, its product with up one more, and the type's rounding.
    tol = np.abs(want) * (6 * STEP + 1.001 * HALF_STEP[kind]) + (2.0 ** -24 if kind == "f16" else 2.0 ** -133)
    off = np.abs(host(out) - want) / tol
    assert np.all(off <= 1), (np.argwhere(~(off <= 1))[:4], np.nanmax(off))


CODES = {
    "f32_group128": [
        ("few_tokens", (16, 128), (9, 1920, 400)), ("few_tokens", (32, 128), (31, 3968, 272)),
        ("mid", (64, 128), (40, 6528, 1040)), ("mid", (64, 128), (130, 3968, 400)), ("mid", (128, 128), (520, 3968, 656)),
        ("mid", (128, 256), (1000, 6528, 272)), ("mid", (128, 256), (2000, 3968, 1040)),
        ("pipe", (256, 256), (4859, 6528, 144)), ("pipe", (256, 256), (4859, 6528, 272)),
        ("pipe", (256, 256), (4859, 6528, 400)), ("tiles", (64, 128), (200, 384, 401)),
    ],
    "e8m0_block32": [
        ("few_tokens", (16, 32), (9, 1920, 400)), ("few_tokens", (32, 32), (31, 3968, 272)),
        ("mid", (64, 32), (40, 896, 1040)), ("mid", (64, 64), (100, 6528, 400)), ("mid", (64, 128), (130, 6528, 656)),
        ("mid", (128, 128), (520, 3968, 656)), ("mid", (128, 256), (1000, 6528, 272)),
        ("mid", (128, 256), (2000, 3968, 1040)), ("pipe", (256, 256), (4859, 6528, 144)),
        ("pipe", (256, 256), (4859, 6528, 272)), ("pipe", (256, 256), (4859, 6528, 400)),
        ("tiles", (64, 128), (200, 384, 401)),
    ],
}
FORMATS = {"f32_group128": ["int8", "e4m3fn", "e5m2"], "e8m0_block32": ["e4m3fn", "e5m2"]}


@pytest.mark.parametrize("layout,kernel,tile,shape", [(layout, *c) for layout, cs in CODES.items() for c in cs],
                         ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else v)
def test_codes(gpu, layout, kernel, tile, shape):
    m, n, k = shape
    _chosen(m, n, k, kernel, tile, scale_layout=layout)
    a, sa, b, sb = _operands(m, n, k)
    # The largest ones in one format: the encodings themselves are the same code everywhere.
    formats = FORMATS[layout] if m * n < 1 << 23 else FORMATS[layout][k // 128 % 2:][:1]
    v = scaled_product(a, sa, b, sb)
    for x_format in formats:
        codes, scales = empty_codes(m, n, layout)
        qrs.matmul_int8_quantize(device(a), device(sa), device(b), device(sb), codes, scales, x_format, layout)
        c, s = quantize_values(v, x_format, layout)
        assert np.array_equal(scales.cpu().numpy().reshape(s.shape), s), x_format
        bad = np.argwhere(codes.cpu().numpy() != c)
        assert bad.size == 0, (x_format, len(bad), bad[:4])
