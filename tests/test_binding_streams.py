"""Streams of the operators between two shares in the binding, on the host:
torch's stream and allocation calls are replaced by ones that record."""

import contextlib
import types

import pytest
import torch

import quantized_collective_reduction_amd as qrs


class _Given:
    """A stream object of the caller."""

    cuda_stream = 77


@pytest.fixture
def recorded(monkeypatch):
    """The stream under which each torch.empty was called; None: the current one."""
    log, active = [], [None]

    @contextlib.contextmanager
    def stream(s):
        active.append(s)
        yield
        active.pop()

    def empty(n, dtype=None, device=None):
        log.append(active[-1])
        return torch.zeros(n, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    monkeypatch.setattr(torch, "empty", empty)
    return log


def test_the_workspace_is_allocated_under_the_stream_that_uses_it(recorded):
    like = types.SimpleNamespace(device="cuda:3")
    given = _Given()
    for s in (None, given, 0x7F00, 0):
        _, nbytes, ws = qrs._workspace(None, 64, like, s)
        assert nbytes == 64 and ws.numel() == 64
    # 0 is the handle of the default stream, not of a stream of its own.
    assert recorded == [None, given, ("external", 0x7F00, "cuda:3"), ("default", "cuda:3")]


@pytest.mark.parametrize("missing", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",)])
def test_the_current_stream_without_torchs_own_functions(monkeypatch, missing):
    given = {"_cuda_getCurrentRawStream": lambda device: 1000 + device, "_cuda_getDevice": lambda: 5}
    monkeypatch.setattr(torch, "_C", types.SimpleNamespace(**{k: f for k, f in given.items() if k not in missing}))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=1005))
    monkeypatch.setattr(qrs, "_current_stream_call", qrs._current_stream_call.__wrapped__)
    assert qrs._stream_handle(None) == 1005
    assert qrs._stream_handle(0) == 0 and qrs._stream_handle(_Given()) == 77
