"""GPU parity of the layer norm and its gradients over batches of thousands of rows:
every shape of a work-group with operands that pass the Infinity Cache by, and every
number of work-groups that the gradient takes, against 64-bit values on the device."""

import pytest
import torch

import quantized_collective_reduction_amd as qrs
from layer_util import STEP, TORCH
from oracle.layer import HALF_STEP

pytestmark = pytest.mark.gpu

EPS = 1e-5
# Activations, tokens, h, scales.
FORWARD = [("bf16", 40000, 1024, "f32_group128"), ("f16", 20001, 2048, "f32_row"), ("bf16", 10000, 4096, "e8m0_block32"),
           ("bf16", 16384, 8192, "f32_group128"), ("f16", 2501, 16384, "f32_row"), ("bf16", 1200, 32768, "f32_group128"),
           ("f32", 21000, 1024, "f32_row"), ("f32", 10300, 2048, "f32_group128"), ("f32", 5200, 4096, "e8m0_block32"),
           ("f32", 8192, 5120, "f32_group128"), ("f32", 2701, 8192, "f32_row"), ("f32", 1301, 16384, "f32_group128"),
           ("f32", 701, 32768, "f32_row")]
BACKWARD = [(kind, t, h) for kind in ("bf16", "f16", "f32") for t, h in
            [(4100, 1024), (4100, 2048), (2100, 2048), (2600, 4096), (2600, 8192), (5000, 520), (2049, 1032)]]
BACKWARD += [("bf16", 33000, 1024), ("f16", 17000, 2048), ("bf16", 8300, 4096), ("bf16", 16384, 8192),
             ("f16", 2100, 16384), ("bf16", 1100, 32768), ("f32", 16500, 1024), ("f32", 8300, 2048), ("f32", 4200, 4096),
             ("f32", 8192, 5120), ("f32", 1040, 16384), ("f32", 530, 32768)]


def _rows(g, t, h, kind, scale):
    v = torch.randn(t, h, device="cuda", generator=g) * scale
    v *= torch.exp2(torch.randint(-3, 4, (t, 1), device="cuda", generator=g).float())
    v += torch.randn(t, 1, device="cuda", generator=g) * scale
    v[5::97] = 0  # padded tokens
    return v.to(TORCH[kind])


def _unit(s, eps=EPS):
    """u, and 1 / sqrt(var + eps), in 64 bits."""
    c = s.double()
    c = c - c.mean(dim=1, keepdim=True)
    r = torch.rsqrt((c * c).mean(dim=1, keepdim=True) + eps)
    return c * r, r


def _check_e4m3(codes, scales, y, tol, layout):
    """layer_util's assert_codes on the device."""
    t, h = y.shape
    g = {"f32_group128": 128, "e8m0_block32": 32, "f32_row": h}[layout]
    amax, off = y.abs().view(t, -1, g), tol.view(t, -1, g)
    low, high = (amax - off).amax(2).clamp_min(0), (amax + off).amax(2)
    scales = scales.view(t, -1)
    if layout == "e8m0_block32":
        code = lambda a: torch.where(a == 0, 0.0, (torch.frexp(a)[1] - 1 - 8).clamp(-127, 127) + 127.0)
        assert ((scales.double() >= code(low)) & (scales.double() <= code(high))).all()
        scale, rel = torch.exp2(scales.double() - 127), 0.0
    else:
        scale, rel = scales.double(), 4 * STEP
        assert (scale >= low.clamp_min(448 * 2.0 ** -126) / 448 * (1 - 2 * STEP)).all()
        assert (scale <= high.clamp_min(448 * 2.0 ** -126) / 448 * (1 + 2 * STEP)).all()
    q = (y.view(t, -1, g) / scale.unsqueeze(2)).clamp(-448, 448).view(t, h)
    off = (off / scale.unsqueeze(2)).view(t, h)
    got = codes.view(torch.float8_e4m3fn).double()
    e = torch.frexp(torch.maximum(q.abs(), got.abs()))[1].double() - 1
    half = torch.exp2(e.clamp_min(-6) - 3) / 2
    bad = (got - q).abs() > half * (1 + 1e-12) + q.abs() * rel + off
    assert not bad.any(), int(bad.sum())


@pytest.mark.parametrize("kind,t,h,layout", FORWARD, ids=lambda v: str(v))
def test_norm(gpu, kind, t, h, layout):
    g = torch.Generator(device="cuda").manual_seed(t)
    x, r = _rows(g, t, h, kind, 1.0), _rows(g, t, h, kind, 4.0)
    w = (1 + 0.1 * torch.randn(h, device="cuda", generator=g)).to(TORCH[kind])
    b = (0.5 * torch.randn(h, device="cuda", generator=g)).to(TORCH[kind])
    codes, total = torch.full((t, h), 0xAA, dtype=torch.uint8, device="cuda"), torch.empty_like(x)
    scales = {"f32_group128": lambda: torch.empty(t, h // 128, device="cuda"), "f32_row": lambda: torch.empty(t, device="cuda"),
              "e8m0_block32": lambda: torch.empty(t, h // 32, dtype=torch.uint8, device="cuda")}[layout]()
    qrs.add_layer_norm_quantize(x, r, w, b, EPS, total, codes, scales, "e4m3fn", layout)
    step = max(1, (1 << 24) // h)
    for i in range(0, t, step):
        part = slice(i, i + step)
        s = (x[part].double() + r[part].double()).to(TORCH[kind])
        assert torch.equal(total[part], s)
        y = _unit(s)[0] * w.double()
        # Rounded once, to binary32; what binary64 leaves is less.
        _check_e4m3(codes[part], scales[part], y + b.double(), (y.abs() + b.double().abs()) * 1.1 * STEP, layout)


@pytest.mark.parametrize("with_sum", [True, False])
@pytest.mark.parametrize("kind,t,h", BACKWARD, ids=lambda v: str(v))
def test_backward(gpu, kind, t, h, with_sum):
    """Bounds as in test_gpu_layer_norm, but for the sums over tokens: chains of at
    most 64 rows, and as many again of work-groups and launches."""
    g = torch.Generator(device="cuda").manual_seed(t + h)
    s, dy = _rows(g, t, h, kind, 2.0), _rows(g, t, h, kind, 0.1)
    gs = _rows(g, t, h, kind, 0.1) if with_sum else None
    w = (1 + 0.1 * torch.randn(h, device="cuda", generator=g)).to(TORCH[kind])
    gx = torch.full_like(s, float("nan"))
    gw, gb = torch.full((h,), float("nan"), device="cuda"), torch.full((h,), float("nan"), device="cuda")
    qrs.layer_norm_backward(dy, s, w, EPS, gs, gx, gw, gb)
    want_w, want_b, size_w, size_b = (torch.zeros(h, dtype=torch.float64, device="cuda") for _ in range(4))
    step = max(1, (1 << 24) // h)
    for i in range(0, t, step):
        part = slice(i, i + step)
        u, r = _unit(s[part])
        grad = dy[part].double()
        d = grad * w.double()
        md, mdu = d.mean(dim=1, keepdim=True), (d * u).mean(dim=1, keepdim=True)
        want = r * (d - md - u * mdu)
        size = (d.abs() + d.abs().mean(dim=1, keepdim=True) + u.abs() * (d * u).abs().mean(dim=1, keepdim=True)) * r
        far = size * 12 * STEP
        if with_sum:
            k = gs[part].double()
            want, size, far = want + k, size + k.abs(), far + k.abs() * 2 * STEP
        far += HALF_STEP[kind] * size * (1 + 12 * STEP) + (2.0 ** -25 if kind == "f16" else 0) + 2.0 ** -120
        off = (gx[part].double() - want).abs()
        assert (off <= far).all(), float((off / far).max())
        want_w += (grad * u).sum(dim=0)
        want_b += grad.sum(dim=0)
        size_w += (grad * u).abs().sum(dim=0)
        size_b += grad.abs().sum(dim=0)
    chain = 64 + 64 + 32
    for got, ref, size, extra in ((gw, want_w, size_w, 5), (gb, want_b, size_b, 0)):
        off = (got.double() - ref).abs()
        assert (off <= size * (chain + extra) * STEP).all(), float((off / size).max() / STEP)
