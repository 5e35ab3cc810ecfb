"""The norm's gradient on streams given as handles, the default stream's among
them: the workspace is allocated under the stream that uses it."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import device, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inside", [False, True])
def test_gradient_on_the_default_stream_by_its_handle(gpu, monkeypatch, inside):
    rng = np.random.default_rng(1)
    s, dy = (device(values(rng, (300, 1024), "bf16"), "bf16") for _ in range(2))
    w = device(values(rng, 1024, "bf16"), "bf16")
    want_x, want_w = torch.empty_like(s), torch.empty(1024, device="cuda")
    qrs.rms_norm_backward(dy, s, w, 1e-5, None, want_x, want_w)
    gx, gw = torch.empty_like(s), torch.empty(1024, device="cuda")
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    under, empty = [], torch.empty

    def recording(*args, **kw):
        under.append(torch.cuda.current_stream().cuda_stream)
        return empty(*args, **kw)

    with torch.cuda.stream(other) if inside else torch.cuda.stream(None):
        current = torch.cuda.current_stream().cuda_stream
        monkeypatch.setattr(torch, "empty", recording)
        for handle in (0, other.cuda_stream):
            qrs.rms_norm_backward(dy, s, w, 1e-5, None, gx, gw, stream=handle)
            torch.cuda.synchronize()
            assert torch.equal(gx, want_x) and torch.equal(gw, want_w)
        qrs.rms_norm_backward(dy, s, w, 1e-5, None, gx, gw)
        monkeypatch.undo()
    torch.cuda.synchronize()
    assert under == [0, other.cuda_stream, current] and (current == other.cuda_stream) is inside
    assert torch.equal(gx, want_x) and torch.equal(gw, want_w)
