"""Products whose fastest kernel would need more work-items than a launch holds:
2^27 channels of one token, and 2^29 tokens of a few channels."""

import pytest
import torch

import quantized_collective_reduction_amd as qrs

pytestmark = pytest.mark.gpu


def _ints(g, rows, k):
    return torch.randint(-128, 128, (rows, k), dtype=torch.int8, device="cuda", generator=g)


def _scales(g, n):
    return torch.rand(n, device="cuda", generator=g) + 0.5


def _want(a, sa, b, sb):
    # k = 16: sums below 2^19, exact in float32.
    return ((a.float() @ b.float().t()) * sa[:, None] * sb).bfloat16()


def test_more_channels_than_narrow_work_groups_can_take(gpu):
    g = torch.Generator(device="cuda").manual_seed(1)
    n, k = (1 << 27) + 40, 16
    assert qrs.matmul_launch_info(1, n, k)["kernel"] == "tiles"
    a, sa, b, sb = _ints(g, 1, k), _scales(g, 1), _ints(g, n, k), _scales(g, n)
    out = torch.full((1, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    qrs.matmul_int8(a, sa, b, sb, out)
    for at in range(0, n, 1 << 25):
        assert torch.equal(out[:, at:at + (1 << 25)], _want(a, sa, b[at:at + (1 << 25)], sb[at:at + (1 << 25)])), at


def test_more_tokens_than_narrow_work_groups_can_take(gpu):
    g = torch.Generator(device="cuda").manual_seed(2)
    m, n, k = (1 << 29) + 70, 8, 16
    # The 64 x 32 tiles that fewer tokens of so few channels take.
    assert qrs.matmul_launch_info(m // 2, n, k)["tile"] == (64, 32)
    assert qrs.matmul_launch_info(m, n, k)["tile"] != (64, 32)
    a, sa, b, sb = _ints(g, m, k), _scales(g, m), _ints(g, n, k), _scales(g, n)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    qrs.matmul_int8(a, sa, b, sb, out)
    for at in range(0, m, 1 << 26):
        assert torch.equal(out[at:at + (1 << 26)], _want(a[at:at + (1 << 26)], sa[at:at + (1 << 26)], b, sb)), at
