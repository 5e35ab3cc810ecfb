"""GPU parity of the block quantizations of matrices large enough that the transposed
codes pass the caches by, bit for bit on the device, and of those just below."""

import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import FP8, up
from layer_util import TORCH

pytestmark = pytest.mark.gpu

QMAX = {"e4m3fn": 448.0, "e5m2": 57344.0}


def _want(x, kind, height, width):
    """The rule in binary32: codes of x * (qmax / amax), and amax / qmax."""
    r, c = x.shape
    v = torch.zeros(up(r, height) * height, up(c, width) * width, device="cuda")
    v[:r, :c] = x.float()
    v = v.view(-1, height, v.shape[1] // width, width)
    amax = v.abs().amax((1, 3), keepdim=True)
    top = torch.full_like(amax, QMAX[kind])
    scale = amax / top
    small = scale < 2.0 ** -126
    mul = torch.where(small, torch.full_like(amax, 2.0 ** 126), top / amax)
    codes = (v * mul).clamp(-QMAX[kind], QMAX[kind]).reshape(-1, v.shape[2] * width)[:r, :c].to(FP8[kind])
    return codes.view(torch.uint8), scale.clamp_min(2.0 ** -126).view(v.shape[0], -1)


@pytest.mark.parametrize("kind,r,c", [("bf16", 4096, 8192), ("bf16", 4100, 8192), ("f16", 7168, 5128), ("f32", 4999, 5000),
                                      ("bf16", 20001, 1688)])
@pytest.mark.parametrize("x_format", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("by_block", [True, False])
def test_both_ways(gpu, by_block, x_format, kind, r, c):
    g = torch.Generator(device="cuda").manual_seed(r)
    x = torch.randn(r, c, device="cuda", generator=g) * torch.exp2(torch.randint(-6, 7, (r, 1), device="cuda", generator=g).float())
    x = x.to(TORCH[kind])
    x[7] = 0
    rows_t = up(r, 16) * 16
    codes = torch.full((r, c), 0xAA, dtype=torch.uint8, device="cuda")
    codes_t = torch.full((c, rows_t), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.empty(up(r) if by_block else r, up(c), device="cuda")
    scales_t = torch.empty(up(c) if by_block else c, up(r), device="cuda")
    if by_block:
        qrs.quantize_blocks(x, codes, scales, x_format, codes_t, scales_t)
    else:
        qrs.quantize_transposed(x, codes_t, scales_t, x_format, codes, scales)
    want, want_s = _want(x, x_format, 128 if by_block else 1, 128)
    assert torch.equal(scales, want_s) and torch.equal(codes, want)
    want, want_s = _want(x, x_format, 128, 128 if by_block else 1)
    assert torch.equal(scales_t, want_s.t()) and torch.equal(codes_t[:, :r], want.t())
    assert torch.all(codes_t[:, r:] == 0)
