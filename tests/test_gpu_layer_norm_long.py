"""GPU parity of the layer norm's gradients of weight and bias over batches of so
many tokens that every work-group adds hundreds of rows: sums whose error does
not grow with them."""

import ctypes

import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, TORCH

pytestmark = pytest.mark.gpu

FOLD = 64  # rows that a work-group adds before it puts them with those of before


def _work_groups(t, h):
    n = ctypes.c_size_t()
    assert qrs.load_library().qrs_layer_norm_backward_workspace(t, h, ctypes.byref(n)) == 0
    return n.value // (8 * h)


def _chain(t, h, kind):
    """Additions, each off by half a step of its result, that a term goes through:
    with others of its work-group, with those of before, in the lanes and the
    row of the last kernel."""
    groups = min(_work_groups(t, h), 256) if kind == "f32" and h > 2048 else _work_groups(t, h)
    rows = -(-t // groups)
    return min(rows, FOLD) + -(-rows // FOLD) + -(-groups // 32) + 32


@pytest.mark.parametrize("kind,t,h", [("f32", 1 << 22, 8), ("f32", (1 << 21) + 77, 7), ("bf16", (1 << 20) + 5, 40),
                                      ("f32", 300001, 520), ("bf16", 120000, 2056), ("f32", 50021, 4096),
                                      ("f16", 20001, 8192), ("f32", 20000, 8200)])
def test_gradients_of_one_sign(gpu, kind, t, h):
    """Gradients of 0.7 everywhere, whose additions round to the same side again and
    again: 4096 in a row are off by 2^-14.6."""
    g = torch.Generator(device="cuda").manual_seed(t)
    s = torch.randn(t, h, device="cuda", generator=g).to(TORCH[kind])
    dy = torch.full((t, h), 0.7, device="cuda").to(TORCH[kind])
    w = torch.ones(h, device="cuda", dtype=TORCH[kind])
    gx, gw, gb = torch.empty_like(s), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    eps = 1e-5
    qrs.layer_norm_backward(dy, s, w, eps, None, gx, gw, gb)
    want_w, size_w = (torch.zeros(h, device="cuda", dtype=torch.float64) for _ in range(2))
    value = float(dy[0, 0])
    for part in s.split(max(1, (1 << 26) // h)):
        c = part.double()
        c -= c.mean(dim=1, keepdim=True)
        c *= value / torch.sqrt((c * c).mean(dim=1, keepdim=True) + eps)
        want_w += c.sum(dim=0)
        size_w += c.abs().sum(dim=0)
    chain = _chain(t, h, kind)
    off = (gb.double() - value * t).abs()
    assert (off <= value * t * chain * STEP).all(), float((off / (value * t)).max() / STEP)
    # u is off by four half steps, its product with grad_y goes into the sum as it is.
    off = (gw.double() - want_w).abs()
    assert (off <= size_w * (chain + 5) * STEP).all(), float((off / size_w).max() / STEP)


def test_folded_sums_are_the_same_every_time(gpu):
    g = torch.Generator(device="cuda").manual_seed(3)
    s, dy = (torch.randn(200003, 264, device="cuda", generator=g).bfloat16() for _ in range(2))
    w = torch.randn(264, device="cuda", generator=g).bfloat16()
    outs = []
    for _ in range(3):
        out = torch.empty_like(s), torch.empty(264, device="cuda"), torch.empty(264, device="cuda")
        workspace = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN from before
        qrs.layer_norm_backward(dy, s, w, 1e-5, dy, *out, workspace=workspace)
        outs.append(out)
    for out in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out, outs[0]))


def _case(t, h, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, dy, gs = (torch.randn(t, h, device="cuda", generator=g).bfloat16() for _ in range(3))
    return s, dy, gs, torch.randn(h, device="cuda", generator=g).bfloat16()


@pytest.mark.parametrize("which", ["grad_y", "grad_sum"])
def test_long_batches_in_place_and_strided(gpu, which):
    """Three launches, the last one of fewer rows than the others have work-groups."""
    t, h = 2 * 65536 + 300, 136
    s, dy, gs, w = _case(t, h, 5)
    want = torch.empty_like(s), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(dy, s, w, 1e-5, gs, *want)
    wide = torch.full((t, 2 * h), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, :h] = dy if which == "grad_y" else gs
    gx = wide[:, :h]
    got = torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    qrs.layer_norm_backward(gx if which == "grad_y" else dy, s, w, 1e-5, gs if which == "grad_y" else gx, gx, *got)
    assert torch.equal(gx, want[0]) and torch.equal(got[0], want[1]) and torch.equal(got[1], want[2])
    assert torch.isnan(wide[:, h:]).all()


def test_long_batches_in_a_graph(gpu):
    """Replayed over other inputs, with eager work between: each replay is the eager result."""
    t, h = 70000, 264
    s, dy, gs, w = _case(t, h, 6)
    out = torch.empty_like(s), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
    n = ctypes.c_size_t()
    assert qrs.load_library().qrs_layer_norm_backward_workspace(t, h, ctypes.byref(n)) == 0
    workspace = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        qrs.layer_norm_backward(dy, s, w, 1e-5, gs, *out, workspace=workspace)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qrs.layer_norm_backward(dy, s, w, 1e-5, gs, *out, workspace=workspace)
    for seed in (7, 8, 9):
        for to, v in zip((s, dy, gs, w), _case(t, h, seed)):
            to.copy_(v)
        want = torch.empty_like(s), torch.empty(h, device="cuda"), torch.empty(h, device="cuda")
        qrs.layer_norm_backward(dy, s, w, 1e-5, gs, *want)
        for v in out:
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), seed
