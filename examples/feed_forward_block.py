"""A tensor-parallel feed-forward block between two quantized reduce-scatters,
every rank of the group on one GPU.

    python examples/feed_forward_block.py [--ranks 4] [--tokens 512] [--hidden 4096] [--inner 14336]

Each rank holds the residual stream of all tokens of its batch [tokens, hidden]
and a slice of the block's 8-bit weights: inner / ranks gate and up channels,
and the same columns of the down projection. Per rank:

    add_rms_norm_quantize   the last share's rows + residual -> norm -> int8, a scale per token
    matmul_int8 (gated)     silu(gate) * up
    quantize_rows           int8, a scale per token
    matmul_int8_quantize    partial sums as E4M3 codes and E8M0 scales

The ranks' codes are then reduced by run_all_shares, and the next block's norm
starts from the shares. The result is compared with the same block in float32,
and so are the gradients of the norm in front of it (rms_norm_backward).
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_collective_reduction_amd as qrs  # noqa: E402

EPS = 1e-5


def quantized_weights(w):
    """[channels, k] as int8 codes and a scale for each channel."""
    codes = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    scales = torch.empty(w.shape[0], device=w.device)
    qrs.quantize_rows(w.contiguous(), codes, scales)
    return codes, scales


class Rank:
    """One rank's weights and buffers; ``step`` leaves its partial sums in
    ``codes`` and ``scales``."""

    def __init__(self, tokens, hidden, up, down, norm_weight):
        dev, bf = norm_weight.device, torch.bfloat16
        inner = down.shape[1]
        self.norm_weight = norm_weight
        self.up, self.up_scales = quantized_weights(up)
        self.down, self.down_scales = quantized_weights(down)
        self.x8 = torch.empty(tokens, hidden, dtype=torch.int8, device=dev)
        self.x8_scales = torch.empty(tokens, device=dev)
        self.mid = torch.empty(tokens, inner, dtype=bf, device=dev)
        self.mid8 = torch.empty(tokens, inner, dtype=torch.int8, device=dev)
        self.mid8_scales = torch.empty(tokens, device=dev)
        self.codes = torch.empty(tokens, hidden, dtype=torch.uint8, device=dev)
        self.scales = torch.empty(tokens, hidden // 32, dtype=torch.uint8, device=dev)

    def step(self, x, residual):
        """The residual stream is updated in place."""
        qrs.add_rms_norm_quantize(x, residual, self.norm_weight, EPS, residual, self.x8, self.x8_scales, "int8",
                                  "f32_row")
        qrs.matmul_int8(self.x8, self.x8_scales, self.up, self.up_scales, self.mid, gated=True)
        qrs.quantize_rows(self.mid, self.mid8, self.mid8_scales)
        qrs.matmul_int8_quantize(self.mid8, self.mid8_scales, self.down, self.down_scales, self.codes, self.scales,
                                 "e4m3fn", "e8m0_block32")


def norm_gradients(total, norm_weight, products, grad_out, grad_stream):
    """Gradients of the residual stream and of the norm's weight by
    rms_norm_backward, and the same by torch in float32.

    ``total`` is the stream that the norm read, ``products`` what follows the
    norm, in float32 (the products have no gradient here: what reaches the
    norm's output is torch's, with the quantization passed through), ``grad_out``
    the gradient of their result and ``grad_stream`` the stream's own."""
    s, w = total.float().requires_grad_(), norm_weight.float().requires_grad_()
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * w
    y.retain_grad()
    (products(y) * grad_out).sum().backward()
    grad_s, grad_w = torch.empty_like(total), torch.empty(total.shape[1], device=total.device)
    qrs.rms_norm_backward(y.grad.to(total.dtype), total, norm_weight, EPS, grad_stream, grad_s, grad_w)
    return (grad_s, grad_w), (s.grad + grad_stream.float(), w.grad)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--ranks", type=int, default=4, choices=[2, 4, 8])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    args = ap.parse_args(argv)
    w, t, h, inner = args.ranks, args.tokens, args.hidden, args.inner // args.ranks
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * scale

    norm_weight = (1 + 0.1 * normal(h)).bfloat16()
    x, residual = normal(t, h).bfloat16(), normal(t, h, scale=4.0).bfloat16()
    up = [normal(2 * inner, h, scale=h ** -0.5) for _ in range(w)]
    down = [normal(h, inner, scale=(w * inner) ** -0.5) for _ in range(w)]

    def products(y):
        out = torch.zeros(t, h, device="cuda")
        for u, d in zip(up, down):
            gate, lift = (y @ u.t()).chunk(2, dim=1)
            out = out + (torch.nn.functional.silu(gate) * lift) @ d.t()
        return out

    # The block in float32.
    s = (x.float() + residual.float()).bfloat16().float()
    want = products(s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * norm_weight.float())

    ranks = [Rank(t, h, u, d, norm_weight) for u, d in zip(up, down)]
    streams = [residual.clone() for _ in ranks]  # in a group, each rank's own copy of the residual stream
    plan = qrs.plan(w, t, h, "e4m3fn", "e8m0_block32", "bf16")
    shares = [torch.empty(t // w, h, dtype=torch.bfloat16, device="cuda") for _ in ranks]
    for r, stream in zip(ranks, streams):
        r.step(x, stream)
    qrs.run_all_shares(plan, [r.codes for r in ranks], [r.scales for r in ranks], shares)
    got = torch.cat(shares).float()
    error = float((got - want).norm() / want.norm())
    print(f"{w} ranks, {t} tokens, hidden {h}, inner {w * inner}: relative error {error:.4f} against float32")

    grads, want = norm_gradients(streams[0], norm_weight, products, normal(t, h), normal(t, h).bfloat16())
    errors = [float((g.float() - r).norm() / r.norm()) for g, r in zip(grads, want)]
    print(f"gradients of the stream and of the norm's weight: relative errors {errors[0]:.5f}, {errors[1]:.5f}")
    return error


if __name__ == "__main__":
    main()
