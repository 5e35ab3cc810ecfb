"""The 8-bit floating-point product with ``binary32_sums``: 16-bit outputs of products
that cancel, and bit for bit the float32 output's."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import FP8, Operands, fp8, up
from layer_util import TORCH, device
from oracle.quantize import encode_fp8_rne

pytestmark = pytest.mark.gpu

# Sizes of every kernel: few tokens, each tile of the middle ones, the largest, and
# rows off 16-byte boundaries.
SIZES = [(20, 640, 256), (48, 1024, 256), (130, 900, 272), (333, 5003, 256), (700, 4096, 1040), (1000, 8200, 144),
         (4100, 4352, 256), (66, 65, 100)]


def _cancelling(m, n, k, small):
    """Codes of whole numbers whose sums binary32 holds in any order: pairs of products of
    2^16 that cancel, six of 0 to 9 small * small beside each pair. The columns of
    the pairs move with their eight."""
    rng = np.random.default_rng([m, n, k])
    a = (rng.integers(-3, 4, (m, k)) * small).astype(np.float32)
    b = (rng.integers(-3, 4, (n, k)) * small).astype(np.float32)
    for i in range(0, k - 7, 8):
        one, other = i + i // 8 % 8, i + (i // 8 + 3) % 8
        a[:, one] = a[:, other] = 256.0
        b[:, one], b[:, other] = 256.0, -256.0
    return a, b


def _product(a, b, kind, **kw):
    (m, k), n = a.shape, b.shape[0]
    out = torch.full((m, n), float("nan"), dtype=TORCH[kind], device="cuda")
    codes = [fp8(encode_fp8_rne(v, "e4m3fn"), "e4m3fn") for v in (a, b)]
    qrs.matmul_fp8(codes[0], torch.ones(m, up(k), device="cuda"), codes[1], torch.ones(up(n), up(k), device="cuda"), out, **kw)
    return out


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES, ids=lambda v: str(v))
def test_binary32_sums_keep_what_cancelling_products_leave(gpu, m, n, k, kind):
    a, b = _cancelling(m, n, k, 1)
    want = (torch.from_numpy(a).cuda().double() @ torch.from_numpy(b).cuda().double().t()).float().to(TORCH[kind])
    assert torch.equal(_product(a, b, kind, binary32_sums=True), want)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("form", ["block", "group", "gated"])
@pytest.mark.parametrize("m,n,k", SIZES, ids=lambda v: str(v))
def test_binary32_sums_are_the_binary32_output_rounded(gpu, m, n, k, form, kind):
    rng = np.random.default_rng([m, n, k, 1])
    gated = form == "gated"
    o = Operands(rng, m, n // 2 if gated else n, k, ["e4m3fn", "e5m2"][m % 2], ["e4m3fn", "e5m2"][n % 2], gated=gated,
                 grouped=form == "group")
    operands = o.device()
    wide = torch.empty(m, o.n, device="cuda")
    out = torch.empty(m, o.n, dtype=TORCH[kind], device="cuda")
    qrs.matmul_fp8(*operands, wide, gated=gated)
    qrs.matmul_fp8(*operands, out, gated=gated, binary32_sums=True)
    assert torch.equal(out, wide.to(TORCH[kind]))


def test_codes_with_scales_of_powers_of_two_and_of_rows(gpu):
    """binary32_sums with every argument that matmul_fp8 takes."""
    a, b = _cancelling(40, 264, 256, 1)
    codes = [device(encode_fp8_rne(v, "e4m3fn")) for v in (a, b)]
    sa, sb = torch.full((40, 2), 0.5, device="cuda"), torch.full((264, 2), 4.0, device="cuda")
    out = torch.empty(40, 264, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    qrs.matmul_fp8(*[v for pair in zip(codes, (sa, sb)) for v in pair], out, a_dtype="e4m3fn", b_dtype="e4m3fn",
                   stream=stream, binary32_sums=True)
    stream.synchronize()
    want = 2 * (torch.from_numpy(a).double() @ torch.from_numpy(b).double().t())
    assert torch.equal(out.cpu(), want.float().bfloat16())
    assert codes[0].view(FP8["e4m3fn"]).shape == a.shape
