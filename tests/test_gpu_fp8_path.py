"""Layer norm, block quantizations and the 8-bit floating-point product used
together: a feed-forward block between two shares, a linear layer's gradients, HIP
graphs, other streams, and tensors past 2^32 bytes."""

import numpy as np
import pytest
import torch

import quantized_collective_reduction_amd as qrs
from fp8_util import FP8, G, assert_codes_within, product_bound, up
from layer_util import device, values
from oracle.blocks import dequantize, layer_norm, quantize_groups
from oracle.layer import HALF_STEP

pytestmark = pytest.mark.gpu

EPS = 1e-5
E4M3, E5M2 = FP8["e4m3fn"], FP8["e5m2"]


def _blocks(w, transposed=False):
    n, k = w.shape
    codes, scales = torch.empty(n, k, dtype=E4M3, device="cuda"), torch.empty(up(n), up(k), device="cuda")
    if not transposed:
        qrs.quantize_blocks(w, codes, scales, "e4m3fn")
        return codes, scales
    codes_t, scales_t = torch.empty(k, n, dtype=E4M3, device="cuda"), torch.empty(up(k), up(n), device="cuda")
    qrs.quantize_blocks(w, codes, scales, "e4m3fn", codes_t, scales_t)
    return codes, scales, codes_t, scales_t


class _Block:
    """A rank's feed-forward block on fixed buffers."""

    def __init__(self, tokens, hidden, inner, gate, lift, down, weight, bias):
        dev = "cuda"
        gates, ups = _blocks(gate), _blocks(lift)
        self.up, self.up_scales = torch.cat([gates[0], ups[0]]), torch.cat([gates[1], ups[1]])
        self.down, self.down_scales = _blocks(down)
        self.weight, self.bias = weight, bias
        self.x8, self.x8_scales = torch.empty(tokens, hidden, dtype=E4M3, device=dev), torch.empty(tokens, up(hidden), device=dev)
        self.mid, self.mid_scales = torch.empty(tokens, inner, dtype=E4M3, device=dev), torch.empty(tokens, up(inner), device=dev)
        self.codes = torch.empty(tokens, hidden, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(tokens, hidden // 32, dtype=torch.uint8, device=dev)

    def step(self, x, stream_in, stream_out, stream=None):
        qrs.add_layer_norm_quantize(x, stream_in, self.weight, self.bias, EPS, stream_out, self.x8, self.x8_scales,
                                    "e4m3fn", "f32_group128", stream=stream)
        qrs.matmul_fp8_quantize(self.x8, self.x8_scales, self.up, self.up_scales, self.mid, self.mid_scales, "e4m3fn",
                                "f32_group128", gated=True, stream=stream)
        qrs.matmul_fp8_quantize(self.mid, self.mid_scales, self.down, self.down_scales, self.codes, self.scales,
                                "e4m3fn", "e8m0_block32", stream=stream)


def _normal(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape, scale=1.0: torch.randn(*shape, device="cuda", generator=g) * scale


def _make(tokens, hidden, inner, seed):
    normal = _normal(seed)
    args = [normal(inner, hidden, scale=hidden ** -0.5), normal(inner, hidden, scale=hidden ** -0.5),
            normal(hidden, inner, scale=inner ** -0.5), (1 + 0.1 * normal(hidden)).bfloat16(), normal(hidden, scale=0.1).bfloat16()]
    return normal, args, _Block(tokens, hidden, inner, *args)


@pytest.mark.parametrize("ranks,tokens", [(2, 2), (2, 16), (4, 64), (2, 1000)])
def test_feed_forward_blocks_between_shares(gpu, ranks, tokens):
    """Against float32. Eight roundings to E4M3 on the way (the norm's codes into gate
    and up, both weights, the product of both, the down projection's weights, the
    partial sums): half a step is at most 2^-4, 3.6 % in the root mean square at most,
    all of them in quadrature 10 %, and gates pass theirs on 1.1 times at most."""
    hidden, inner = 1024, 512
    normal, _, _ = _make(1, 128, 128, tokens)
    weight, bias = (1 + 0.1 * normal(hidden)).bfloat16(), normal(hidden, scale=0.1).bfloat16()
    x, residual = normal(tokens, hidden).bfloat16(), normal(tokens, hidden, scale=4.0).bfloat16()
    s = (x.float() + residual.float()).bfloat16().float()
    y = torch.nn.functional.layer_norm(s, (hidden,), weight.float(), bias.float(), EPS)
    want, blocks = torch.zeros(tokens, hidden, device="cuda"), []
    for _ in range(ranks):
        gate, lift = normal(inner, hidden, scale=hidden ** -0.5), normal(inner, hidden, scale=hidden ** -0.5)
        down = normal(hidden, inner, scale=(ranks * inner) ** -0.5)
        want += (torch.nn.functional.silu(y @ gate.t()) * (y @ lift.t())) @ down.t()
        blocks.append(_Block(tokens, hidden, inner, gate, lift, down, weight, bias))
    for b in blocks:
        total = torch.empty_like(x)
        b.step(x, residual, total)
        assert torch.equal(total.float(), s)
    plan = qrs.plan(ranks, tokens, hidden, "e4m3fn", "e8m0_block32", "bf16")
    shares = [torch.empty(tokens // ranks, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]
    qrs.run_all_shares(plan, [b.codes for b in blocks], [b.scales for b in blocks], shares)
    got = torch.cat(shares).float()
    assert float((got - want).norm() / want.norm()) < 0.11


@pytest.mark.parametrize("tokens", [1, 5, 40, 300])
def test_each_step_reads_what_the_one_before_wrote(gpu, tokens):
    """Every step's codes against the formula in 64 bits of its own inputs."""
    hidden, inner = 640, 384
    normal, _, b = _make(tokens, hidden, inner, tokens)
    x, residual = normal(tokens, hidden).bfloat16(), normal(tokens, hidden).bfloat16()
    total = torch.empty_like(x)
    b.step(x, residual, total)
    host = lambda t: t.float().cpu().numpy()
    raw = lambda t: t.view(torch.uint8).cpu().numpy()
    y = layer_norm(host(total), host(b.weight), host(b.bias), EPS)
    assert_codes_within(raw(b.x8), host(b.x8_scales), y, np.abs(y) * 2.0 ** -24 + 2.0 ** -140, "e4m3fn", "f32_group128")
    a, w = dequantize(raw(b.x8), host(b.x8_scales), "e4m3fn", 1), raw(b.up)
    blocks = up(inner)
    gate, lift = (dequantize(w[i * inner:(i + 1) * inner], host(b.up_scales)[i * blocks:(i + 1) * blocks], "e4m3fn", G)
                  for i in range(2))
    g, u = a @ gate.T, a @ lift.T
    tg, tu = (product_bound(np.abs(a) @ np.abs(v).T, hidden) for v in (gate, lift))
    s = 1 / (1 + np.exp(-g))
    v = g * s * u
    tol = 1.1 * tg * (np.abs(u) + tu) + np.abs(g * s) * tu + np.abs(v) * 6 * 2.0 ** -24 + 2.0 ** -100
    assert_codes_within(raw(b.mid), host(b.mid_scales), v, tol, "e4m3fn", "f32_group128")
    a, w = dequantize(raw(b.mid), host(b.mid_scales), "e4m3fn", 1), dequantize(raw(b.down), host(b.down_scales), "e4m3fn", G)
    assert_codes_within(raw(b.codes), raw(b.scales), a @ w.T, product_bound(np.abs(a) @ np.abs(w).T, inner), "e4m3fn",
                        "e8m0_block32")


class _Linear:
    """y = x W^T through codes, and its gradients."""

    def __init__(self, t, n, k, seed, kind=torch.bfloat16):
        normal = _normal(seed)
        self.x, self.grad, w = normal(t, k).to(kind), normal(t, n, scale=0.01).to(kind), normal(n, k, scale=k ** -0.5)
        self.w = w
        self.w8, self.ws, self.wt8, self.wts = _blocks(w, True)
        dev = "cuda"
        self.g8, self.gs = torch.empty(t, n, dtype=E5M2, device=dev), torch.empty(t, up(n), device=dev)
        wide = up(t, 16) * 16
        self.gt8, self.gts = torch.empty(n, wide, dtype=E5M2, device=dev), torch.empty(n, up(t), device=dev)
        self.xt8, self.xts = torch.empty(k, wide, dtype=E4M3, device=dev), torch.empty(k, up(t), device=dev)
        self.grad_x, self.grad_w = torch.empty(t, k, dtype=kind, device=dev), torch.empty(n, k, device=dev)

    def backward(self, stream=None):
        qrs.quantize_transposed(self.grad, self.gt8, self.gts, "e5m2", self.g8, self.gs, stream=stream)
        qrs.quantize_transposed(self.x, self.xt8, self.xts, "e4m3fn", stream=stream)
        qrs.matmul_fp8(self.g8, self.gs, self.wt8, self.wts, self.grad_x, stream=stream)
        qrs.matmul_fp8(self.gt8, self.gts, self.xt8, self.xts, self.grad_w, stream=stream)


@pytest.mark.parametrize("t,n,k", [(1, 128, 256), (37, 256, 384), (300, 640, 512), (1021, 512, 1024)])
def test_gradients_of_a_linear_layer(gpu, t, n, k):
    """Against the formula in 64 bits with the oracle's codes, and against differences
    of the loss that the dequantized operands stand for."""
    m = _Linear(t, n, k, t)
    m.backward()
    grad, x = m.grad.float().cpu().numpy(), m.x.float().cpu().numpy()
    g = dequantize(*quantize_groups(grad, "e5m2", 1, G), "e5m2", 1)
    gt = dequantize(*quantize_groups(np.ascontiguousarray(grad.T), "e5m2", 1, G), "e5m2", 1)
    xt = dequantize(*quantize_groups(np.ascontiguousarray(x.T), "e4m3fn", 1, G), "e4m3fn", 1)
    w = dequantize(*quantize_groups(m.w.cpu().numpy(), "e4m3fn", G, G), "e4m3fn", G)
    want, size = g @ w, np.abs(g) @ np.abs(w)
    got = m.grad_x.float().cpu().numpy()
    # 16-bit outputs of many tokens: eight products at a time, 2^-11 of their magnitudes.
    tol = size * 2.0 ** -11 * 1.01 + product_bound(size, n) + np.abs(want) * HALF_STEP["bf16"] * 1.01
    assert np.all(np.abs(got - want) <= tol)
    want, size = gt @ xt.T, np.abs(gt) @ np.abs(xt).T
    off = np.abs(m.grad_w.cpu().numpy() - want)
    assert np.all(off <= product_bound(size, up(t, 16) * 16) + np.abs(want) * 2.0 ** -24)
    # The loss sum(grad * x W^T) at a weight and at an input moved by one.
    loss = lambda x_, w_: np.sum(gt.T * (x_ @ w_.T))
    base, rng = loss(xt.T, w), np.random.default_rng(t)
    for _ in range(3):
        i, j = int(rng.integers(n)), int(rng.integers(k))
        moved = w.copy()
        moved[i, j] += 1.0
        assert abs(loss(xt.T, moved) - base - m.grad_w[i, j].item()) <= 1e-6 * (size[i, j] + abs(base))


def test_norm_gradients_reach_a_layers_input(gpu):
    """The linear layer's grad_x through the norm, against torch's in float64."""
    t, n, k = 64, 256, 512
    m = _Linear(t, n, k, 3, torch.float32)
    m.backward()
    normal = _normal(9)
    s, w, gs = normal(t, k), 1 + 0.1 * normal(k), normal(t, k)
    gx, gw, gb = torch.empty(t, k, device="cuda"), torch.empty(k, device="cuda"), torch.empty(k, device="cuda")
    qrs.layer_norm_backward(m.grad_x, s, w, EPS, gs, gx, gw, gb)
    leaf = [v.double().cpu().requires_grad_() for v in (s, w, torch.zeros(k))]
    y = torch.nn.functional.layer_norm(leaf[0], (k,), leaf[1], leaf[2], EPS)
    ((y * m.grad_x.double().cpu()).sum() + (leaf[0] * gs.double().cpu()).sum()).backward()
    for got, ref in zip((gx, gw, gb), leaf):
        assert torch.allclose(got.double().cpu(), ref.grad, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("tokens", [1, 24, 200, 600])
def test_graph_replays_are_the_eager_results(gpu, tokens):
    hidden, inner = 1024, 768
    normal, _, b = _make(tokens, hidden, inner, 5)
    m = _Linear(tokens, 512, hidden, 6)
    x, residual, total = normal(tokens, hidden).bfloat16(), normal(tokens, hidden).bfloat16(), None
    total = torch.empty_like(x)
    gy, gx, gw, gb = (normal(tokens, hidden).bfloat16(), torch.empty_like(x), torch.empty(hidden, device="cuda"),
                      torch.empty(hidden, device="cuda"))

    def step():
        b.step(x, residual, total)
        m.backward()
        qrs.layer_norm_backward(gy, total, b.weight, EPS, m.grad_x, gx, gw, gb)

    outs = [total, b.x8, b.x8_scales, b.mid, b.mid_scales, b.codes, b.scales, m.grad_x, m.grad_w, gx, gw, gb]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    with torch.cuda.graph(other):
        step()
    for i in range(4):
        x.copy_(normal(tokens, hidden).bfloat16())
        m.grad.copy_(normal(tokens, 512).bfloat16())
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.view(torch.uint8).fill_(0xFF)
        (graph if i % 2 else other).replay()
        torch.cuda.synchronize()
        for t, ref in zip(outs, want):
            assert torch.equal(t.view(torch.uint8), ref.view(torch.uint8))


def test_streams_by_object_and_by_handle(gpu):
    normal, _, b = _make(8, 512, 256, 7)
    x, residual = normal(8, 512).bfloat16(), normal(8, 512).bfloat16()
    total = torch.empty_like(x)
    b.step(x, residual, total)
    torch.cuda.synchronize()
    outs = [total, b.x8, b.x8_scales, b.mid, b.mid_scales, b.codes, b.scales]
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        for t in outs:
            t.view(torch.uint8).fill_(0xFF)
        torch.cuda.synchronize()
        b.step(x, residual, total, stream=stream)
        torch.cuda.synchronize()
        for t, ref in zip(outs, want):
            assert torch.equal(t.view(torch.uint8), ref.view(torch.uint8))


def test_two_blocks_at_once_on_two_streams(gpu):
    made = [_make(16, 512, 256, seed) for seed in (1, 2)]
    io = [(normal(16, 512).bfloat16(), normal(16, 512).bfloat16()) for normal, _, _ in made]
    totals = [torch.empty_like(x) for x, _ in io]
    want = []
    for (_, _, b), (x, r), total in zip(made, io, totals):
        b.step(x, r, total)
        torch.cuda.synchronize()
        want.append((b.codes.clone(), b.scales.clone()))
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for _ in range(20):
        for (_, _, b), (x, r), total, stream in zip(made, io, totals, streams):
            b.step(x, r, total, stream=stream)
    torch.cuda.synchronize()
    for (_, _, b), (codes, scales) in zip(made, want):
        assert torch.equal(b.codes, codes) and torch.equal(b.scales, scales)


def test_a_workspace_of_the_callers(gpu):
    normal, _, b = _make(4, 512, 256, 11)
    x, residual = normal(4, 512).bfloat16(), normal(4, 512).bfloat16()
    b.step(x, residual, torch.empty_like(x))
    want = b.mid.clone(), b.mid_scales.clone()
    args = (b.x8, b.x8_scales, b.up, b.up_scales, b.mid, b.mid_scales, "e4m3fn", "f32_group128")
    guard = torch.full((4 * 256 * 4 + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    qrs.matmul_fp8_quantize(*args, gated=True, workspace=guard[:4 * 256 * 4])
    assert torch.equal(b.mid.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(b.mid_scales, want[1])
    assert (guard[4 * 256 * 4:] == 0x5A).all()
    with pytest.raises(qrs.QrsError, match="workspace"):
        qrs.matmul_fp8_quantize(*args, gated=True, workspace=guard[:4 * 256 * 4 - 16])
    with pytest.raises(ValueError, match="tensor"):
        qrs.matmul_fp8_quantize(*args, gated=True, workspace=guard.data_ptr())


def test_tensors_past_2_to_the_32_bytes(gpu):
    """Rows, codes and their transposes past 2^32 elements; ends and middle checked."""
    rows, cols = 66000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    for at in range(0, rows, 8250):
        x[at:at + 8250] = _normal(at)(min(8250, rows - at), cols).bfloat16()
    codes = torch.empty(rows, cols, dtype=E4M3, device="cuda")
    codes_t = torch.empty(cols, rows, dtype=E4M3, device="cuda")
    scales, scales_t = torch.empty(up(rows), up(cols), device="cuda"), torch.empty(up(cols), up(rows), device="cuda")
    qrs.quantize_blocks(x, codes, scales, "e4m3fn", codes_t, scales_t)
    for r in (0, 32768, 65920):
        for c in (0, 65408):
            part = x[r:r + 128, c:c + 128].float().cpu().numpy()
            want, s = quantize_groups(part, "e4m3fn", G, G)
            h, w = part.shape
            assert np.array_equal(codes[r:r + h, c:c + w].view(torch.uint8).cpu().numpy(), want)
            assert np.array_equal(codes_t[c:c + w, r:r + h].view(torch.uint8).cpu().numpy(), want.T)
            assert scales[r // G, c // G].item() == s[0, 0] == scales_t[c // G, r // G].item()
    # The product of a few tokens, and of hundreds, with all of it.
    for m, kind in ((2, torch.float32), (200, torch.bfloat16)):
        a = torch.zeros(m, cols, device="cuda")
        a[:, 5], a[0, cols - 1] = 1.0, 2.0
        sa = torch.ones(m, up(cols), device="cuda")
        out = torch.empty(m, rows, dtype=kind, device="cuda")
        qrs.matmul_fp8(a.to(E4M3), sa, codes, scales, out)
        first = codes[:, 5].float() * scales[:, 0].repeat_interleave(G)[:rows]
        last = codes[:, cols - 1].float() * scales[:, -1].repeat_interleave(G)[:rows]
        assert torch.equal(out[1], first.to(kind))
        assert torch.allclose(out[0].double(), first.double() + 2 * last.double(), rtol=2.0 ** -7, atol=1e-6)
    total = x  # in place
    s8, w = torch.empty(rows, up(cols), device="cuda"), torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    keep = x[[0, rows - 1]].float()
    qrs.add_layer_norm_quantize(x, x, w, None, EPS, total, codes, s8, "e4m3fn", "f32_group128")
    assert torch.equal(x[[0, rows - 1]].float(), (2 * keep).bfloat16().float())
    for r in (0, rows - 1):
        y = layer_norm(x[r:r + 1].float().cpu().numpy(), np.ones(cols), np.zeros(cols), EPS)
        assert_codes_within(codes[r:r + 1].view(torch.uint8).cpu().numpy(), s8[r:r + 1].cpu().numpy(), y,
                            np.abs(y) * 2.0 ** -24, "e4m3fn", "f32_group128")


def test_device_helpers_hold_what_the_tests_need(gpu):
    """The oracle's codes and torch's float8 types agree on every finite code."""
    codes = np.arange(256, dtype=np.uint8)
    for name, kind in FP8.items():
        want = torch.from_numpy(codes).view(kind).float().numpy()
        got = dequantize(codes.reshape(1, -1), np.ones((1, 2), np.float32), name, 1)[0]
        keep = np.isfinite(want)
        assert np.array_equal(got[keep], want[keep].astype(np.float64))
    assert values(np.random.default_rng(0), (2, 2), "bf16").shape == (2, 2) and device(codes).is_cuda
