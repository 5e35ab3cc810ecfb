"""Arguments that the binding of the operators between two shares refuses with
a message of its own, with tensors that only say they are on the device."""

import pytest
import torch

import quantized_collective_reduction_amd as qrs


class _OnDevice(torch.Tensor):
    is_cuda = True


def _tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice)


def test_a_residual_needs_a_sum():
    x, w = _tensor(2, 128), _tensor(128)
    codes, scales = _tensor(2, 128, dtype=torch.int8), _tensor(2, dtype=torch.float32)
    with pytest.raises(ValueError, match="sum_out"):
        qrs.add_rms_norm_quantize(x, x, w, 1e-5, None, codes, scales, "int8", "f32_row")


def test_a_workspace_is_a_tensor():
    x, w, gw = _tensor(2, 128), _tensor(128), _tensor(128, dtype=torch.float32)
    with pytest.raises(ValueError, match="workspace"):
        qrs.rms_norm_backward(x, _tensor(2, 128), w, 1e-5, None, _tensor(2, 128), gw, workspace=1 << 32)
