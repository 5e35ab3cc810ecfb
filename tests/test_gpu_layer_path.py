"""The operators between two shares used together: the feed-forward example,
HIP graphs, other streams, several host threads, and tensors past 2^32 bytes."""

import os
import sys
import threading

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from gpu_util import out_bits
from layer_util import TORCH, assert_codes, device, empty_codes, host, norm_rel, values
from oracle.layer import rms_norm, rms_norm_backward, rounded_sum, scaled_product
from oracle.quantize import quantize_values
from oracle.reduce import fp32_to_bf16_bits

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import feed_forward_block  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.mark.parametrize("ranks,tokens", [(2, 2), (2, 16), (4, 64), (8, 256), (4, 1000)])
def test_feed_forward_example(gpu, ranks, tokens):
    """Four roundings to 8 bits on the way: int8 rows and weights (a maximum of
    about 4 sigma: errors of 4 / 127 / sqrt(12) = 0.9 % of a row's sigma each,
    six of them in quadrature: 2.3 %) and E4M3 partial sums (half a step is at most 2^-4,
    2^-4 / sqrt(3) = 3.6 % in the root mean square at most)."""
    error = feed_forward_block.main(["--ranks", str(ranks), "--tokens", str(tokens), "--hidden", "1024", "--inner",
                                     str(512 * ranks)])
    assert error < 0.06


class _Chain:
    """norm -> product -> rows -> quantized product on fixed buffers."""

    def __init__(self, t, h, n, seed):
        rng = np.random.default_rng(seed)
        dev = "cuda"
        self.rng = rng
        self.t, self.h, self.n = t, h, n
        self.x, self.r = (torch.empty(t, h, dtype=torch.bfloat16, device=dev) for _ in range(2))
        self.w = device(values(rng, h, "bf16"), "bf16")
        self.total = torch.empty_like(self.x)
        self.q, self.qs = torch.empty(t, h, dtype=torch.int8, device=dev), torch.empty(t, device=dev)
        self.b = device(rng.integers(-127, 128, (2 * n, h), dtype=np.int8))
        self.bs = device(np.full(2 * n, 2.0 ** -10, np.float32))
        self.mid = torch.empty(t, n, dtype=torch.bfloat16, device=dev)
        self.m8, self.ms = torch.empty(t, n, dtype=torch.int8, device=dev), torch.empty(t, device=dev)
        self.d = device(rng.integers(-127, 128, (h, n), dtype=np.int8))
        self.ds = device(np.full(h, 2.0 ** -10, np.float32))
        self.codes = torch.empty(t, h, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(t, h // 32, dtype=torch.uint8, device=dev)
        self.gx, self.gw = torch.empty_like(self.x), torch.empty(h, device=dev)
        self.fill()

    def fill(self):
        self.x.copy_(device(values(self.rng, (self.t, self.h), "bf16"), "bf16"))
        self.r.copy_(device(values(self.rng, (self.t, self.h), "bf16"), "bf16"))

    def run(self, stream=None):
        qrs.add_rms_norm_quantize(self.x, self.r, self.w, EPS, self.total, self.q, self.qs, "int8", "f32_row",
                                  stream=stream)
        qrs.matmul_int8(self.q, self.qs, self.b, self.bs, self.mid, gated=True, stream=stream)
        qrs.quantize_rows(self.mid, self.m8, self.ms, stream=stream)
        qrs.matmul_int8_quantize(self.m8, self.ms, self.d, self.ds, self.codes, self.scales, "e4m3fn", "e8m0_block32",
                                 stream=stream)
        qrs.rms_norm_backward(self.x, self.total, self.w, EPS, self.r, self.gx, self.gw, stream=stream)

    def outputs(self):
        return [t.clone() for t in (self.total, self.q, self.qs, self.mid, self.m8, self.ms, self.codes, self.scales,
                                    self.gx, self.gw)]

    def wipe(self):
        for t in (self.total, self.q, self.qs, self.mid, self.m8, self.ms, self.codes, self.scales, self.gx, self.gw):
            t.zero_()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [1, 20, 100, 700])
def test_chain_in_a_graph(gpu, t):
    """Captured once, replayed with new inputs and eager runs between replays:
    every replay equals the eager result bit for bit."""
    c = _Chain(t, 1024, 640, seed=t)
    c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c.run()
    for _ in range(3):
        c.fill()
        c.run()
        torch.cuda.synchronize()
        want = c.outputs()
        c.wipe()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(c.outputs(), want)


def test_chain_on_another_stream(gpu):
    c = _Chain(130, 2048, 512, seed=3)
    c.run()
    torch.cuda.synchronize()
    want = c.outputs()
    c.wipe()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        c.run(stream=stream)
        # The gradient's workspace belongs to that stream: what this one
        # allocates and writes meanwhile is other memory.
        for _ in range(4):
            torch.full((c.gw.numel() * 512,), 1.0, device="cuda")
        s.synchronize()
        torch.cuda.synchronize()
        assert _same(c.outputs(), want)
        c.wipe()
        torch.cuda.synchronize()


def test_chains_from_several_threads(gpu):
    chains = [_Chain(40 + 8 * i, 1024, 384, seed=i) for i in range(4)]
    want = []
    for c in chains:
        c.run()
        torch.cuda.synchronize()
        want.append(c.outputs())
        c.wipe()
    torch.cuda.synchronize()
    errors = []

    def work(c):
        try:
            s = torch.cuda.Stream()
            for _ in range(10):
                c.run(stream=s)
            s.synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in chains]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for c, w in zip(chains, want):
        assert _same(c.outputs(), w)


def test_caller_workspace_must_be_large_enough(gpu):
    c = _Chain(8, 1024, 128, seed=5)
    c.run()
    with pytest.raises(qrs.QrsError, match="workspace"):
        qrs.rms_norm_backward(c.x, c.total, c.w, EPS, c.r, c.gx, c.gw,
                              workspace=torch.empty(8 * 1024 * 4 - 16, dtype=torch.uint8, device="cuda"))
    want = c.outputs()
    ws = torch.empty(8 * 1024 * 4, dtype=torch.uint8, device="cuda")
    qrs.rms_norm_backward(c.x, c.total, c.w, EPS, c.r, c.gx, c.gw, workspace=ws)
    assert _same(c.outputs(), want)


def test_binding_refusals_on_the_device(gpu):
    c = _Chain(4, 1024, 128, seed=6)
    with pytest.raises(ValueError, match="sum_out"):
        qrs.add_rms_norm_quantize(c.x, c.r, c.w, EPS, c.total[:3], c.q, c.qs, "int8", "f32_row")
    with pytest.raises(ValueError, match="residual"):
        qrs.add_rms_norm_quantize(c.x, c.r.float(), c.w, EPS, c.total, c.q, c.qs, "int8", "f32_row")
    with pytest.raises(ValueError, match="weight"):
        qrs.add_rms_norm_quantize(c.x, c.r, c.w[:-1], EPS, c.total, c.q, c.qs, "int8", "f32_row")
    with pytest.raises(ValueError, match="scales"):
        qrs.add_rms_norm_quantize(c.x, c.r, c.w, EPS, c.total, c.q, c.qs[:2], "int8", "f32_row")
    with pytest.raises(ValueError, match="adjacent"):
        qrs.quantize_rows(c.x.t(), c.q.t(), c.qs)
    with pytest.raises(ValueError, match="b: expected"):
        qrs.matmul_int8(c.q, c.qs, c.d, c.ds, c.mid)
    with pytest.raises(ValueError, match="a_scales"):
        qrs.matmul_int8(c.q, c.qs[:2], c.b, c.bs, c.mid, gated=True)
    with pytest.raises(ValueError, match="out"):
        qrs.matmul_int8(c.q, c.qs, c.b, c.bs, c.mid)
    with pytest.raises(qrs.QrsError, match="multiple of 128"):
        qrs.matmul_int8_quantize(c.q, c.qs, c.b[:64], c.bs[:64], c.codes[:, :64], c.scales[:, :2].contiguous(), "e5m2",
                                 "e8m0_block32")
    with pytest.raises(qrs.QrsError, match="overlaps"):
        qrs.rms_norm_backward(c.x, c.total, c.w, EPS, c.r, c.total, c.gw)


def test_norm_past_2_to_the_32_bytes(gpu):
    """2^18 + 3 rows of 8192 bf16 elements: 4 GiB a tensor, the last rows past
    2^32 bytes and 2^31 elements; sampled rows against the oracle."""
    t, h, period = (1 << 18) + 3, 8192, 64
    rng = np.random.default_rng(21)
    x, r = values(rng, (period, h), "bf16"), values(rng, (period, h), "bf16", 3)
    w = values(rng, h, "bf16")
    dx, dr, dw = device(x, "bf16"), device(r, "bf16"), device(w, "bf16")
    at = torch.arange(t, device="cuda") % period
    bx, br = dx[at], dr[at]
    codes = torch.empty(t, h, dtype=torch.uint8, device="cuda")
    scales = torch.empty(t, device="cuda")
    qrs.add_rms_norm_quantize(bx, br, dw, EPS, br, codes, scales, "int8", "f32_row")
    for first in (0, t - period):
        rows = (np.arange(first, first + period)) % period
        s = rounded_sum(x, r, "bf16")[rows]
        assert np.array_equal(host(br[first:first + period]), s)
        assert_codes(codes[first:first + period].cpu().numpy(), scales[first:first + period].cpu().numpy(),
                     rms_norm(s, w, EPS), norm_rel(h), "int8", "f32_row", f"rows from {first}")
    # Every block of rows is the first one again.
    whole = t // period * period
    assert torch.equal(codes[:whole].view(-1, period, h).amax(0), codes[:whole].view(-1, period, h).amin(0))
    del codes
    gx, gw = bx, torch.empty(h, device="cuda")
    want_x, _ = rms_norm_backward(x[-4:], rounded_sum(x, r, "bf16")[-4:], w, EPS)
    last = (whole - 4, whole)
    qrs.rms_norm_backward(bx, br, dw, EPS, None, gx, gw)
    got = host(gx[last[0]:last[1]])
    assert np.all(np.abs(got - want_x) <= 2.0 ** -8 * np.abs(want_x) + 1e-4 * np.abs(want_x).max())
    assert torch.isfinite(gw).all()


def test_product_past_2_to_the_32_bytes(gpu):
    """2^18 + 5 tokens: a is 4 GiB of k = 16384, the output 2^32 + bytes."""
    m, n, k, period = (1 << 18) + 5, 8448, 16384, 128
    rng = np.random.default_rng(22)
    a = rng.integers(-128, 128, (period, k), dtype=np.int8)
    b = rng.integers(-128, 128, (n, k), dtype=np.int8)
    sa = np.exp2(rng.uniform(-4, 0, period)).astype(np.float32)
    sb = np.exp2(rng.uniform(-12, -8, n)).astype(np.float32)
    at = torch.arange(m, device="cuda") % period
    out = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    qrs.matmul_int8(device(a)[at], device(sa)[at], device(b), device(sb), out)
    want = fp32_to_bf16_bits(scaled_product(a, sa, b, sb))
    for first in (0, m // 2, m - period):
        rows = np.arange(first, first + period) % period
        assert np.array_equal(out_bits(out[first:first + period]), want[rows]), first
