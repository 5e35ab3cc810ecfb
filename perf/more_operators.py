"""Cases for the operators of a layer whose products are 8-bit floating point with a scale for each block of
128: layer norm to codes and its gradients, the quantizations that such a product reads, and the product.

  layer_norm       add_layer_norm_quantize: s = x + residual, y = (s - mean) / std * weight + bias, y as codes
                   and scales
  layer_norm_grad  layer_norm_backward: the gradients of s, of weight and of bias
  quantize         quantize_blocks: a scale for each 128 x 128 block, with the transpose beside it;
                   quantize_transposed: the transpose with a scale for each 128 rows of a column, and the rows
                   themselves with a scale for each 128 columns
  product          matmul_fp8: a scale for each row and 128 columns of a, for each 128 x 128 block (or each row
                   and 128 columns) of b; gated: two products joined as silu(gate) * up; codes:
                   matmul_fp8_quantize
  forward          a rank's feed-forward block: layer norm, gated product to codes, product to codes
  backward         a linear layer's gradients: the quantizations of its input and of the output's gradient, and
                   two products

``run`` computes each in elementary torch operations, or with ``own`` through this package. ``exact``
computes them in 64 bits.
"""

import math

import torch
import torch.nn.functional as F

own = False

EPS = 1e-5
G = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
EMAX = {"e4m3fn": 8, "e5m2": 15}
TINY = 2.0 ** -126  # the smallest fp32 scale


def listed():
    return [
        # One decoded token's residual stream: latency.
        dict(name="layer norm, one token", op="layer_norm", tokens=1, h=4096, type="bf16", codes="e4m3fn"),
        # The fp32 share of the W=8, BS=65536, H=5120 workload.
        dict(name="layer norm, fp32 share", op="layer_norm", tokens=8192, h=5120, type="f32", codes="e4m3fn"),
        # Training: the width of the W=8, BS=8192, H=7168 share, with a ragged last microbatch.
        dict(name="layer norm gradient, ragged", op="layer_norm_grad", tokens=1021, h=7168, type="bf16"),
        # Training: a rank's whole batch.
        dict(name="layer norm gradient, a batch", op="layer_norm_grad", tokens=16384, h=8192, type="bf16"),
        # Training: a weight matrix after its update, for the forward and for the backward product.
        dict(name="quantize, a weight", op="quantize", form="blocks", rows=7168, cols=8192, type="bf16",
             codes="e4m3fn"),
        # Training: the output's gradient of a ragged microbatch, for both of the backward products.
        dict(name="quantize, a gradient", op="quantize", form="transposed", rows=1021, cols=5120, type="bf16",
             codes="e5m2"),
        # One decoded token through a square projection: the weights' bytes bound it.
        dict(name="product, one token", op="product", m=1, n=8192, k=8192, type="bf16", gated=False, out="values",
             a="e4m3fn", b="e4m3fn", by="block"),
        # A few hundred tokens in flight and an output, such as a vocabulary's slice, that no block divides.
        dict(name="product, 333 tokens", op="product", m=333, n=5003, k=7168, type="f32", gated=False, out="values",
             a="e4m3fn", b="e4m3fn", by="block"),
        # A prompt through a projection.
        dict(name="product, a prompt", op="product", m=4096, n=8192, k=7168, type="bf16", gated=False, out="values",
             a="e4m3fn", b="e4m3fn", by="block"),
        # A prompt through one rank's gate and up projections, as what the down projection reads.
        dict(name="product, gated to codes", op="product", m=2048, n=3584, k=8192, type="f32", gated=True, out="codes",
             a="e4m3fn", b="e4m3fn", by="block"),
        # Sixteen decoded tokens through a rank's feed-forward block, as the codes that it sends. (E8M0 scales: codes
        # are rounded on the way, and a value next to a border between two of them moves what follows by more than
        # 32 bits resolve.)
        dict(name="forward, 16 tokens", op="forward", tokens=16, h=4096, inner=2048, type="bf16", codes="e4m3fn"),
        # A linear layer's gradients over a microbatch.
        dict(name="backward, a microbatch", op="backward", tokens=4096, n=3584, k=4096, type="bf16"),
    ]


MOST_PRODUCT = 4096 * 8192 * 7168


def _log_int(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, -(-lo // step) * step), hi // step * step)


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_grad", "quantize", "product", "product", "product", "forward",
                     "backward"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    code = rng.choice(["e4m3fn", "e4m3fn", "e5m2"])
    if op == "layer_norm":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), h=_log_int(rng, 1024, 8192, G), type=kind, codes=code)
    if op == "layer_norm_grad":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), h=_log_int(rng, 1024, 8192, rng.choice([8, G])), type=kind)
    if op == "quantize":
        return dict(op=op, form=rng.choice(["blocks", "transposed"]), rows=_log_int(rng, 64, 8192),
                    cols=_log_int(rng, 512, 8192, rng.choice([8, G])), type=kind, codes=code)
    if op == "product":
        out, by = rng.choice([("values", "block"), ("values", "block"), ("values", "group"), ("codes", "block")])
        gated = by == "block" and rng.choice([False, False, True])
        n = _log_int(rng, 512, 4096 if gated else 8192, G if out == "codes" else rng.choice([1, 8, G]))
        k = _log_int(rng, 512, 8192, rng.choice([16, G]))
        m = min(_log_int(rng, 1, 8192), MOST_PRODUCT // (n * k * (2 if gated else 1)))
        return dict(op=op, m=m, n=n, k=k, type=kind, gated=gated, out=out, a=code, b=rng.choice(["e4m3fn", "e4m3fn", "e5m2"]),
                    by=by)
    if op == "forward":
        return dict(op=op, tokens=_log_int(rng, 1, 4096), h=_log_int(rng, 1024, 8192, G),
                    inner=_log_int(rng, 512, 3584, G), type=rng.choice(["bf16", "f16"]), codes="e4m3fn")
    n, k = _log_int(rng, 512, 4096, G), _log_int(rng, 512, 8192, G)
    return dict(op=op, tokens=_log_int(rng, 128, 4096), n=n, k=k, type=rng.choice(["bf16", "f16"]))


# ---- inputs ---------------------------------------------------------------------------------------------


def _rows(g, t, h, kind, scale):
    """Activations: normal values, a size of its own for each token, some channels larger than the rest, and
    (in batches) the zero rows of padded tokens."""
    dev = g.device
    v = torch.randn(t, h, device=dev, generator=g)
    v *= torch.exp2(torch.randint(-2, 3, (t, 1), device=dev, generator=g).float()) * scale
    v *= 1 + 7 * (torch.rand(h, device=dev, generator=g) < 0.005)
    if t >= 64:
        v[torch.randperm(t, device=dev, generator=g)[: t // 64]] = 0
    return v.to(TYPES[kind])


def _weights(g, n, k):
    """Normal values of 1 / sqrt(k), rows of different size."""
    v = torch.randn(n, k, device=g.device, generator=g) / math.sqrt(k)
    return v * torch.exp2(torch.rand(n, 1, device=g.device, generator=g) * 2 - 1)


def _norm_weights(g, h, kind):
    w = 1 + 0.1 * torch.randn(h, device=g.device, generator=g)
    return w.to(TYPES[kind]), (0.1 * torch.randn(h, device=g.device, generator=g)).to(TYPES[kind])


def _up(n, step):
    return -(-n // step) * step


def _codes(dev, rows, cols, kind):
    return torch.empty(rows, cols, device=dev, dtype=FP8[kind]), torch.empty(rows, -(-cols // G), device=dev)


def _gated_blocks(w, kind):
    """The 128 x 128 blocks of the gates, then those of the ups."""
    parts = [_plain_blocks(v, kind) for v in w.chunk(2)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op in ("layer_norm", "forward"):
        t, h = c["tokens"], c["h"]
        s["x"], s["residual"] = _rows(g, t, h, c["type"], 1.0), _rows(g, t, h, c["type"], 4.0)
        s["weight"], s["bias"] = _norm_weights(g, h, c["type"])
        s["sum"] = torch.empty_like(s["x"])
        s["codes"], s["scales"] = _codes(dev, t, h, c["codes"])
        if op == "forward":
            s["scales"] = torch.empty(t, h // 32, device=dev, dtype=torch.float8_e8m0fnu)
    if op == "layer_norm_grad":
        t, h = c["tokens"], c["h"]
        s["sum"] = _rows(g, t, h, c["type"], 4.0)
        s["grad_y"], s["grad_sum"] = _rows(g, t, h, c["type"], 0.01), _rows(g, t, h, c["type"], 0.01)
        s["weight"], _ = _norm_weights(g, h, c["type"])
        s["grad_x"] = torch.empty_like(s["sum"])
        s["grad_weight"], s["grad_bias"] = torch.empty(h, device=dev), torch.empty(h, device=dev)
    elif op == "quantize":
        r, n = c["rows"], c["cols"]
        if c["form"] == "blocks":
            s["x"] = _weights(g, r, n).to(TYPES[c["type"]])
            s["scales"] = torch.empty(-(-r // G), -(-n // G), device=dev)
            s["scales_t"] = torch.empty(-(-n // G), -(-r // G), device=dev)
        else:
            s["x"] = _rows(g, r, n, c["type"], 0.01)
            s["scales"] = torch.empty(r, -(-n // G), device=dev)
            s["scales_t"] = torch.empty(n, -(-r // G), device=dev)
        s["codes"] = torch.empty(r, n, device=dev, dtype=FP8[c["codes"]])
        s["codes_t"] = torch.empty(n, _up(r, 16), device=dev, dtype=FP8[c["codes"]])
    elif op == "product":
        m, n, k = c["m"], c["n"], c["k"]
        s["a"], s["a_scales"] = _plain_groups(_rows(g, m, k, "f32", 1.0), c["a"])
        w = _weights(g, 2 * n if c["gated"] else n, k)
        make = _plain_groups if c["by"] == "group" else _gated_blocks if c["gated"] else _plain_blocks
        s["b"], s["b_scales"] = make(w, c["b"])
        if c["out"] == "values":
            s["out"] = torch.empty(m, n, device=dev, dtype=TYPES[c["type"]])
        else:
            s["codes"], s["scales"] = _codes(dev, m, n, c["a"])
    elif op == "forward":
        i = c["inner"]
        s["x8"], s["x8_scales"] = _codes(dev, t, h, "e4m3fn")
        s["up"], s["up_scales"] = _gated_blocks(_weights(g, 2 * i, h), "e4m3fn")
        s["mid"], s["mid_scales"] = _codes(dev, t, i, "e4m3fn")
        s["down"], s["down_scales"] = _plain_blocks(_weights(g, h, i), "e4m3fn")
    elif op == "backward":
        t, n, k = c["tokens"], c["n"], c["k"]
        s["x"], s["grad"] = _rows(g, t, k, c["type"], 1.0), _rows(g, t, n, c["type"], 0.01)
        # The weight [n, k], transposed: what its gradient's product reads.
        s["weight_t"], s["weight_t_scales"] = _plain_blocks(_weights(g, n, k).t(), "e4m3fn")
        s["g8"], s["g8_scales"] = _codes(dev, t, n, "e5m2")
        s["g8_t"], s["x8_t"] = (torch.empty(cols, _up(t, 16), device=dev, dtype=FP8[kind])
                                for cols, kind in ((n, "e5m2"), (k, "e4m3fn")))
        s["g8_t_scales"], s["x8_t_scales"] = (torch.empty(cols, -(-t // G), device=dev) for cols in (n, k))
        s["grad_x"] = torch.empty(t, k, device=dev, dtype=TYPES[c["type"]])
        s["grad_weight"] = torch.empty(n, k, device=dev)
    return s


# ---- the plain forms, in 32 bits ------------------------------------------------------------------------


def _plain_scaled(v, amax, kind):
    """Values as codes, and the scales: amax / qmax, multiplied by qmax / amax."""
    top = torch.full_like(amax, QMAX[kind])
    scale = (amax / top).clamp_min(TINY)
    mul = torch.where(amax / top < TINY, torch.full_like(amax, 1 / TINY), top / amax)
    return (v * mul).clamp(-QMAX[kind], QMAX[kind]), scale


def _plain_groups(v, kind):
    """[r, c] as codes with a scale for each row and 128 columns."""
    r, c = v.shape
    v = F.pad(v.float(), (0, _up(c, G) - c)).view(r, -1, G)
    q, scale = _plain_scaled(v, v.abs().amax(2, keepdim=True), kind)
    return q.view(r, -1)[:, :c].to(FP8[kind]).contiguous(), scale.view(r, -1)


def _plain_blocks(v, kind):
    """[r, c] as codes with a scale for each 128 rows and 128 columns."""
    r, c = v.shape
    v = F.pad(v.float(), (0, _up(c, G) - c, 0, _up(r, G) - r)).view(_up(r, G) // G, G, -1, G)
    q, scale = _plain_scaled(v, v.abs().amax((1, 3), keepdim=True), kind)
    return q.view(-1, _up(c, G))[:r, :c].to(FP8[kind]).contiguous(), scale.view(scale.shape[0], -1)


def _plain_mx(v, kind):
    """[r, c] as codes with an E8M0 scale for each row and 32 columns."""
    r, c = v.shape
    v = v.view(r, -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    e = torch.frexp(amax)[1] - 1 - EMAX[kind]
    e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    one = torch.ones_like(amax)
    q = (v * torch.ldexp(one, -e)).clamp(-QMAX[kind], QMAX[kind])
    return q.view(r, c).to(FP8[kind]), torch.ldexp(one, e).to(torch.float8_e8m0fnu).view(r, -1)


def _padded(codes):
    """Rows of codes, filled up to a multiple of 16."""
    return F.pad(codes.float(), (0, _up(codes.shape[1], 16) - codes.shape[1])).to(codes.dtype)


def _values(codes, scales):
    """What codes with a scale for each row, or 128 rows, and 128 columns stand for."""
    r, c = codes.shape
    if scales.shape[0] != r:
        scales = scales.repeat_interleave(G, 0)[:r]
    return codes.float() * scales.repeat_interleave(G, 1)[:, :c]


def _plain_product(a, a_scales, b, b_scales, gated=False):
    if gated:
        n, blocks = b.shape[0] // 2, b_scales.shape[0] // 2
        gate = _plain_product(a, a_scales, b[:n], b_scales[:blocks])
        return gate * torch.sigmoid(gate) * _plain_product(a, a_scales, b[n:], b_scales[blocks:])
    return _values(a, a_scales) @ _values(b, b_scales).t()


def _plain_norm(s):
    total = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    v = total.float()
    v = v - v.mean(-1, keepdim=True)
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float() + s["bias"].float()
    return total, y


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "layer_norm":
        total, y = _plain_norm(s)
        return (total, *_plain_groups(y, c["codes"]))
    if op == "layer_norm_grad":
        v, dy = s["sum"].float(), s["grad_y"].float()
        v = v - v.mean(-1, keepdim=True)
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        u, d = v * r, dy * s["weight"].float()
        dx = s["grad_sum"].float() + r * (d - d.mean(-1, keepdim=True) - u * (d * u).mean(-1, keepdim=True))
        return dx.to(s["sum"].dtype), (dy * u).sum(0), dy.sum(0)
    if op == "quantize":
        if c["form"] == "blocks":
            codes, scales = _plain_blocks(s["x"], c["codes"])
            return codes, scales, _padded(codes.t()), scales.t().contiguous()
        codes_t, scales_t = _plain_groups(s["x"].t(), c["codes"])
        return (*_plain_groups(s["x"], c["codes"]), _padded(codes_t), scales_t)
    if op == "product":
        p = _plain_product(s["a"], s["a_scales"], s["b"], s["b_scales"], c["gated"])
        return p.to(TYPES[c["type"]]) if c["out"] == "values" else _plain_groups(p, c["a"])
    if op == "forward":
        total, y = _plain_norm(s)
        q = _plain_groups(y, "e4m3fn")
        q = _plain_groups(_plain_product(*q, s["up"], s["up_scales"], True), "e4m3fn")
        return (total, *_plain_mx(_plain_product(*q, s["down"], s["down_scales"]), c["codes"]))
    grad_x = _plain_product(*_plain_groups(s["grad"], "e5m2"), s["weight_t"], s["weight_t_scales"])
    grad_w = _plain_product(*_plain_groups(s["grad"].t(), "e5m2"), *_plain_groups(s["x"].t(), "e4m3fn"))
    return grad_x.to(TYPES[c["type"]]), grad_w


# ---- the package's operators ----------------------------------------------------------------------------


def _run_own(s):
    import quantized_collective_reduction_amd as qrs

    c = s["case"]
    op = c["op"]
    if op == "layer_norm":
        qrs.add_layer_norm_quantize(s["x"], s["residual"], s["weight"], s["bias"], EPS, s["sum"], s["codes"],
                                    s["scales"], c["codes"], "f32_group128")
        return s["sum"], s["codes"], s["scales"]
    if op == "layer_norm_grad":
        qrs.layer_norm_backward(s["grad_y"], s["sum"], s["weight"], EPS, s["grad_sum"], s["grad_x"],
                                s["grad_weight"], s["grad_bias"])
        return s["grad_x"], s["grad_weight"], s["grad_bias"]
    if op == "quantize":
        if c["form"] == "blocks":
            qrs.quantize_blocks(s["x"], s["codes"], s["scales"], c["codes"], s["codes_t"], s["scales_t"])
        else:
            qrs.quantize_transposed(s["x"], s["codes_t"], s["scales_t"], c["codes"], s["codes"], s["scales"])
        return s["codes"], s["scales"], s["codes_t"], s["scales_t"]
    if op == "product":
        if c["out"] == "values":
            qrs.matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], gated=c["gated"])
            return s["out"]
        qrs.matmul_fp8_quantize(s["a"], s["a_scales"], s["b"], s["b_scales"], s["codes"], s["scales"], c["a"],
                                "f32_group128", gated=c["gated"])
        return s["codes"], s["scales"]
    if op == "forward":
        qrs.add_layer_norm_quantize(s["x"], s["residual"], s["weight"], s["bias"], EPS, s["sum"], s["x8"],
                                    s["x8_scales"], "e4m3fn", "f32_group128")
        qrs.matmul_fp8_quantize(s["x8"], s["x8_scales"], s["up"], s["up_scales"], s["mid"], s["mid_scales"],
                                "e4m3fn", "f32_group128", gated=True)
        qrs.matmul_fp8_quantize(s["mid"], s["mid_scales"], s["down"], s["down_scales"], s["codes"], s["scales"],
                                c["codes"], "e8m0_block32")
        return s["sum"], s["codes"], s["scales"]
    qrs.quantize_transposed(s["grad"], s["g8_t"], s["g8_t_scales"], "e5m2", s["g8"], s["g8_scales"])
    qrs.quantize_transposed(s["x"], s["x8_t"], s["x8_t_scales"], "e4m3fn")
    qrs.matmul_fp8(s["g8"], s["g8_scales"], s["weight_t"], s["weight_t_scales"], s["grad_x"])
    qrs.matmul_fp8(s["g8_t"], s["g8_t_scales"], s["x8_t"], s["x8_t_scales"], s["grad_weight"])
    return s["grad_x"], s["grad_weight"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------------------


def work(case):
    c = case
    op = c["op"]
    size = 4 if c["type"] == "f32" else 2
    if op == "layer_norm":  # x, residual in; sum, codes, scales out; weight, bias
        n = c["tokens"] * c["h"]
        return {"bytes": n * (3 * size + 1 + 4 / G) + 2 * c["h"] * size, "flops": 10 * n}
    if op == "layer_norm_grad":  # grad_y, sum, grad_sum in; grad_x out; weight, its gradient, the bias's
        n = c["tokens"] * c["h"]
        return {"bytes": n * 4 * size + c["h"] * (size + 8), "flops": 18 * n}
    if op == "quantize":
        n = c["rows"] * c["cols"]
        scales = 2 * 4 * n / (G * G if c["form"] == "blocks" else G)
        return {"bytes": n * (size + 2) + scales, "flops": 4 * n}
    if op == "product":
        m, n, k = c["m"], c["n"], c["k"]
        wide = 2 * n if c["gated"] else n
        scales = 4 * (m * k / G + wide * k / (G if c["by"] == "group" else G * G))
        out = m * n * (size if c["out"] == "values" else 1 + 4 / G)
        return {"bytes": m * k + wide * k + scales + out, "flops": 2 * m * wide * k}
    if op == "forward":
        t, h, i = c["tokens"], c["h"], c["inner"]
        return {"bytes": t * h * (3 * size + 1 + 4 / G) + 2 * h * size + 3 * i * h * (1 + 4 / (G * G)),
                "flops": 6 * t * i * h + 10 * t * h}
    t, n, k = c["tokens"], c["n"], c["k"]
    return {"bytes": t * (n + 2 * k) * size + n * k * (1 + 4 / (G * G)) + 4 * n * k, "flops": 4 * t * n * k}


# ---- the definitions in 64 bits -------------------------------------------------------------------------


def _grid(q, kind):
    """The format's value nearest each element of q, ties to even."""
    digits, low = (3, -6) if kind == "e4m3fn" else (2, -14)
    e = torch.frexp(q)[1].to(torch.float64) - 1
    step = torch.exp2(e.clamp_min(low) - digits)
    return torch.round(q / step) * step


def _f32(v):
    return v.float().double()


def _spread(scales, block, shape):
    """A scale for each element, of scales for each block."""
    at = [torch.arange(n, device=scales.device) // b for n, b in zip(shape, block)]
    return scales[at[0]][:, at[1]]


def _exact_codes(y, kind, block=(1, G)):
    """Binary32 values as codes and scales: the scale, its reciprocal and the product with that are rounded to
    binary32 by definition."""
    y = _f32(y)
    amax = F.max_pool2d(y.abs().unsqueeze(0), block, ceil_mode=True).squeeze(0)
    scale = _f32(amax / QMAX[kind])
    mul = torch.where(scale < TINY, torch.full_like(amax, 1 / TINY), _f32(QMAX[kind] / amax))
    q = _f32(y * _spread(mul, block, y.shape))
    return _grid(q.clamp(-QMAX[kind], QMAX[kind]), kind), scale.clamp_min(TINY)


def _exact_mx(y, kind):
    y = y.unflatten(1, (-1, 32))
    amax = y.abs().max(dim=2, keepdim=True).values
    e = torch.frexp(amax)[1].to(torch.float64) - 1 - EMAX[kind]
    scale = torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
    return _grid(torch.clamp(y / scale, -QMAX[kind], QMAX[kind]), kind).flatten(1), scale.squeeze(2)


def _exact_product(a, b, gated=False):
    """a, b: (codes, scales, the block of a scale)."""
    av, bv = (codes.double() * _spread(scales.double(), block, codes.shape) for codes, scales, block in (a, b))
    if not gated:
        return torch.mm(av, bv.t())
    n = bv.shape[0] // 2
    g, u = torch.mm(av, bv[:n].t()), torch.mm(av, bv[n:].t())
    return g / (1 + torch.exp(-g)) * u


def _gated_scales(scales, n):
    """Blocks of the gates and of the ups as a scale for each row of both."""
    row = torch.arange(2 * n, device=scales.device)
    return scales[torch.where(row < n, row // G, scales.shape[0] // 2 + (row - n) // G)]


def _exact_norm(s):
    total = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
    std, mean = torch.std_mean(total, dim=1, unbiased=False, keepdim=True)
    return total, (total - mean) / torch.sqrt(std * std + EPS) * s["weight"].double() + s["bias"].double()


def _transposed(codes):
    out = torch.zeros(codes.shape[1], _up(codes.shape[0], 16), device=codes.device, dtype=codes.dtype)
    out[:, :codes.shape[0]] = codes.t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    row, block = (1, G), (G, G)
    if op == "layer_norm":
        total, y = _exact_norm(s)
        return (total, *_exact_codes(y, c["codes"]))
    if op == "layer_norm_grad":
        v, dy = s["sum"].double(), s["grad_y"].double()
        std, mean = torch.std_mean(v, dim=1, unbiased=False, keepdim=True)
        std = torch.sqrt(std * std + EPS)
        unit, d = (v - mean) / std, dy * s["weight"].double()
        along = (d * unit).mean(dim=1, keepdim=True)
        return (s["grad_sum"].double() + (d - d.mean(dim=1, keepdim=True) - unit * along) / std, (dy * unit).sum(dim=0),
                dy.sum(dim=0))
    if op == "quantize":
        if c["form"] == "blocks":
            codes, scales = _exact_codes(s["x"], c["codes"], block)
            return codes, scales, _transposed(codes), scales.t()
        codes_t, scales_t = _exact_codes(s["x"], c["codes"], (G, 1))
        return (*_exact_codes(s["x"], c["codes"]), _transposed(codes_t), scales_t.t())
    if op == "product":
        b_scales, by = s["b_scales"], row if c["by"] == "group" else block
        if c["gated"]:
            b_scales, by = _gated_scales(b_scales, c["n"]), row
        p = _exact_product((s["a"], s["a_scales"], row), (s["b"], b_scales, by), c["gated"])
        return p if c["out"] == "values" else _exact_codes(p, c["a"])
    if op == "forward":
        total, y = _exact_norm(s)
        up_scales = _gated_scales(s["up_scales"], c["inner"])
        mid = _exact_product((*_exact_codes(y, "e4m3fn"), row), (s["up"], up_scales, row), True)
        out = _exact_product((*_exact_codes(mid, "e4m3fn"), row), (s["down"], s["down_scales"], block))
        return (total, *_exact_mx(out, c["codes"]))
    grad_x = _exact_product((*_exact_codes(s["grad"], "e5m2"), row), (s["weight_t"], s["weight_t_scales"], block))
    grad_w = _exact_product((*_exact_codes(s["grad"].t(), "e5m2"), row), (*_exact_codes(s["x"].t(), "e4m3fn"), row))
    return grad_x, grad_w
