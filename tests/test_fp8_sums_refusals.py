"""The product with binary32 sums refuses what the product refuses, on the host."""

import pytest

import quantized_collective_reduction_amd as qrs
from test_fp8_refusals import INVALID, MM, MM_BAD, lib  # noqa: F401


def test_refusals(lib):  # noqa: F811
    for kw, text in MM_BAD:
        d = {**MM, **kw}
        status = lib.qrs_matmul_float_single(d["m"], d["n"], d["k"], d["gated"], d["kind"], d["ad"], d["a"], d["lda"],
                                               d["sa"], d["bd"], d["bs"], d["b"], d["ldb"], d["sb"], d["o"], d["ldo"], None)
        assert status == INVALID, kw
        assert text in lib.qrs_last_error().decode(), (kw, lib.qrs_last_error())


def test_binding_refuses_before_it_calls():
    import torch

    c, s, x = torch.zeros(2, 128, dtype=torch.float8_e4m3fn), torch.zeros(2, 1), torch.zeros(2, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.matmul_fp8(c, s, c, s, x, binary32_sums=True)
