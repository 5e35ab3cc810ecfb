"""The feed-forward example's gradients against torch's in float32."""

import os
import sys

import pytest
import torch

import quantized_collective_reduction_amd as qrs  # noqa: F401

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import feed_forward_block  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,h,kind", [(64, 1024, torch.bfloat16), (300, 640, torch.float32)])
def test_gradients_of_the_example(gpu, t, h, kind):
    """Of the relative error, grad_y's rounding to the type and grad_s's are
    half a step each (2^-8 for bfloat16); float32 sums of h products are off by
    less than h * 2^-24, in torch's products and here."""
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    total, weight = normal(t, h).to(kind), (1 + 0.1 * normal(h)).to(kind)
    m = normal(h, h) * h ** -0.5
    (gs, gw), (want_s, want_w) = feed_forward_block.norm_gradients(
        total, weight, lambda y: torch.nn.functional.silu(y @ m), normal(t, h), normal(t, h).to(kind))
    step = torch.finfo(kind).eps / 2
    tol = 2.5 * step + 4 * h * 2.0 ** -24
    assert (gs.float() - want_s).norm() <= tol * want_s.norm()
    assert (gw - want_w).norm() <= tol * want_w.norm()
