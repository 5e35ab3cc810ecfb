"""The columns that a transpose of codes has beyond the rows it is of: zeros,
whatever the rows hold."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import FP8, up
from layer_util import TORCH, device, values
from oracle.layer import round_to

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("x_format", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("r,c", [(1, 1), (3, 40), (200, 264), (300, 300), (129, 128)])
def test_padding_beside_what_is_not_finite(gpu, r, c, bad, x_format, kind):
    """Both quantizations, alone and with the rows' codes, at every width that rows of
    16 bytes or a whole block need; the groups that are not finite show in their scales."""
    rng = np.random.default_rng([r, c])
    x = device(round_to(values(rng, (r, c), kind), kind), kind)
    x[r - 1, 0], x[0, c - 1] = bad, bad
    for rows_t in sorted({r, up(r, 16) * 16, up(r) * 128}):
        for by_block in (True, False):
            for beside in (True, False):
                codes_t = torch.full((c, rows_t), 0xAA, dtype=torch.uint8, device="cuda").view(FP8[x_format])
                scales_t = torch.empty(up(c) if by_block else c, up(r), device="cuda")
                codes = torch.empty(r, c, dtype=FP8[x_format], device="cuda") if beside else None
                scales = torch.empty(up(r) if by_block else r, up(c), device="cuda") if beside else None
                if by_block:
                    qrs.quantize_blocks(x, codes, scales, x_format, codes_t, scales_t)
                else:
                    qrs.quantize_transposed(x, codes_t, scales_t, x_format, codes, scales)
                pad = codes_t.view(torch.uint8)[:, r:]
                assert torch.all(pad == 0), (rows_t, by_block, beside, int((pad != 0).sum()))
                assert not torch.isfinite(scales_t[0, (r - 1) // 128])
                assert not torch.isfinite(scales_t[-1, 0])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_padding_of_rows_of_zeros_and_of_the_smallest_values(gpu, kind):
    x = torch.zeros(100, 200, dtype=TORCH[kind], device="cuda")
    x[7, 100:] = 2.0 ** -130
    for call, rows in ((qrs.quantize_blocks, 2), (qrs.quantize_transposed, 200)):
        codes_t = torch.full((200, 128), 0xAA, dtype=torch.uint8, device="cuda")
        scales_t = torch.empty(rows, 1, device="cuda")
        args = (x, None, None, "e4m3fn", codes_t, scales_t) if call is qrs.quantize_blocks else (x, codes_t, scales_t, "e4m3fn")
        call(*args)
        assert torch.all(codes_t[:, 100:] == 0)
