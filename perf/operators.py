"""Cases for the operators between two quantized reduce-scatters of a tensor-parallel layer.

A share leaves the reduce-scatter as rows of partial-sum activations. What a layer does next with 8-bit
weights, and what is measured here:

  norm       add_rms_norm_quantize: s = x + residual, y = s / rms(s) * weight, y as 8-bit codes and scales
  norm_grad  rms_norm_backward: the gradients of s and of weight
  product    matmul_int8: 8-bit integers times 8-bit integers, a scale for each token and each channel;
             gated: two such products joined as silu(gate) * up
  partial    matmul_int8_quantize: the same product, written as the codes and scales the next share reads
  project    norm with a scale for each token, then product
  ffn        norm, gated product, quantize_rows, partial: a rank's whole feed-forward block

``run`` computes each in elementary torch operations, or with ``own`` through this package. ``exact``
computes them in 64 bits.
"""

import math

import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
GROUP = {"f32_group128": 128, "e8m0_block32": 32}
QMAX = {"int8": 127.0, "e4m3fn": 448.0, "e5m2": 57344.0}
EMAX = {"e4m3fn": 8, "e5m2": 15}
TINY = 2.0 ** -126  # the smallest fp32 scale


def listed():
    return [
        # One decoded token's residual stream: latency.
        dict(name="norm, one token", op="norm", tokens=1, h=4096, type="bf16", codes="e4m3fn", scales="e8m0_block32"),
        # The rows of one share of the W=8, BS=16384, H=8192 workload.
        dict(name="norm, a share's rows", op="norm", tokens=2048, h=8192, type="bf16", codes="e4m3fn",
             scales="f32_group128"),
        # The fp32 share of the W=8, BS=65536, H=5120 workload.
        dict(name="norm, fp32 share", op="norm", tokens=8192, h=5120, type="f32", codes="e5m2", scales="e8m0_block32"),
        # Training: the same width as the W=8, BS=8192, H=7168 share, with a ragged last microbatch.
        dict(name="norm gradient, ragged", op="norm_grad", tokens=1021, h=7168, type="bf16"),
        # Training: a rank's whole batch.
        dict(name="norm gradient, a batch", op="norm_grad", tokens=16384, h=8192, type="bf16"),
        # One decoded token through a square projection: the weights' bytes bound it.
        dict(name="product, one token", op="product", m=1, n=8192, k=8192, type="bf16", gated=False),
        # A few hundred tokens in flight, not a multiple of any tile.
        dict(name="product, 333 tokens", op="product", m=333, n=5120, k=7168, type="f16", gated=False),
        # A prompt through one rank's gate and up projections.
        dict(name="product, gated prompt", op="product", m=4096, n=3584, k=8192, type="bf16", gated=True),
        # A rank's down projection of a whole batch, as the codes that it sends.
        dict(name="partial, a batch", op="partial", m=16384, n=8192, k=3584, codes="e4m3fn", scales="e8m0_block32"),
        # Sixteen decoded tokens: norm, then a rank's query, key and value projection.
        dict(name="project, 16 tokens", op="project", tokens=16, h=5120, n=2560, type="bf16"),
        # Eight decoded tokens through a rank's feed-forward block.
        dict(name="ffn, 8 tokens", op="ffn", tokens=8, h=4096, inner=2048, type="bf16", codes="e4m3fn",
             scales="e8m0_block32"),
        # A prompt through the same block of a larger model.
        dict(name="ffn, a prompt", op="ffn", tokens=2048, h=8192, inner=3584, type="bf16", codes="e5m2",
             scales="e8m0_block32"),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, -(-lo // step) * step), hi // step * step)
    return v if v != 3072 else v + step


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "product", "product", "partial", "project", "ffn"])
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    mode = dict(codes=rng.choice(["e4m3fn", "e5m2"]), scales=rng.choice(["f32_group128", "e8m0_block32"]))
    tokens = _log_int(rng, 1, 8192)
    if op == "norm":
        return dict(op=op, tokens=tokens, h=_log_int(rng, 1024, 8192, 128), type=kind, **mode)
    if op == "norm_grad":
        return dict(op=op, tokens=tokens, h=_log_int(rng, 1024, 8192, rng.choice([8, 128])), type=kind)
    if op == "product":
        gated = rng.choice([False, False, True])
        return dict(op=op, m=tokens, n=_log_int(rng, 512, 4096 if gated else 8192, rng.choice([1, 8, 128])),
                    k=_log_int(rng, 512, 7168, rng.choice([16, 128])), type=kind, gated=gated)
    if op == "partial":
        return dict(op=op, m=tokens, n=_log_int(rng, 1024, 8192, 128), k=_log_int(rng, 512, 4096, 16), **mode)
    if op == "project":
        # 16-bit results here, and E8M0 scales below: codes are rounded on the way, and a value next to a border
        # between two codes moves what follows by more than 32 bits resolve.
        return dict(op=op, tokens=tokens, h=_log_int(rng, 1024, 8192, 128), n=_log_int(rng, 512, 7168, 8),
                    type=rng.choice(["bf16", "f16"]))
    return dict(op=op, tokens=_log_int(rng, 1, 4096), h=_log_int(rng, 1024, 8192, 128),
                inner=_log_int(rng, 512, 4096, 16), type=rng.choice(["bf16", "f16"]), codes=mode["codes"],
                scales="e8m0_block32")


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


def _int8(g, rows, cols):
    """What quantizing normal values with a maximum of about 4.5 sigma leaves."""
    v = torch.randn(rows, cols, device=g.device, generator=g) * (127 / 4.5)
    return v.round_().clamp_(-127, 127).to(torch.int8)


def _scales(g, n, typical):
    return typical * torch.exp2(torch.rand(n, device=g.device, generator=g) * 2 - 1)


def _weights(g, n, k):
    """8-bit weights [n, k] and their scales: values of about 1 / sqrt(k)."""
    return _int8(g, n, k), _scales(g, n, 4.5 / 127 / math.sqrt(k))


def _codes_out(dev, t, h, c):
    kind = torch.float32 if c["scales"] == "f32_group128" else torch.float8_e8m0fnu
    return (torch.empty(t, h, device=dev, dtype=FP8[c["codes"]]),
            torch.empty(t, h // GROUP[c["scales"]], device=dev, dtype=kind))


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": c}
    op = c["op"]
    if op in ("norm", "project", "ffn"):
        t, h = c["tokens"], c["h"]
        s["x"], s["residual"] = _rows(g, t, h, c["type"], 1.0), _rows(g, t, h, c["type"], 4.0)
        s["weight"] = (1 + 0.1 * torch.randn(h, device=dev, generator=g)).to(TYPES[c["type"]])
        s["sum"] = torch.empty_like(s["x"])
    if op == "norm":
        s["codes"], s["scales"] = _codes_out(dev, t, h, c)
    elif op == "norm_grad":
        t, h = c["tokens"], c["h"]
        s["sum"] = _rows(g, t, h, c["type"], 4.0)
        s["grad_y"], s["grad_sum"] = _rows(g, t, h, c["type"], 0.01), _rows(g, t, h, c["type"], 0.01)
        s["weight"] = (1 + 0.1 * torch.randn(h, device=dev, generator=g)).to(TYPES[c["type"]])
        s["grad_x"] = torch.empty_like(s["sum"])
        s["grad_weight"] = torch.empty(h, device=dev)
    elif op in ("product", "partial"):
        m, n, k = c["m"], c["n"], c["k"]
        s["a"], s["a_scales"] = _int8(g, m, k), _scales(g, m, 4.5 / 127)
        s["b"], s["b_scales"] = _weights(g, n * (2 if c.get("gated") else 1), k)
        if op == "product":
            s["out"] = torch.empty(m, n, device=dev, dtype=TYPES[c["type"]])
        else:
            s["codes"], s["scales"] = _codes_out(dev, m, n, c)
    elif op == "project":
        s["qa"], s["qs"] = torch.empty(t, h, device=dev, dtype=torch.int8), torch.empty(t, device=dev)
        s["b"], s["b_scales"] = _weights(g, c["n"], h)
        s["out"] = torch.empty(t, c["n"], device=dev, dtype=TYPES[c["type"]])
    elif op == "ffn":
        i = c["inner"]
        s["qa"], s["qs"] = torch.empty(t, h, device=dev, dtype=torch.int8), torch.empty(t, device=dev)
        s["up"], s["up_scales"] = _weights(g, 2 * i, h)
        s["down"], s["down_scales"] = _weights(g, h, i)
        s["mid"] = torch.empty(t, i, device=dev, dtype=TYPES[c["type"]])
        s["qm"], s["qms"] = torch.empty(t, i, device=dev, dtype=torch.int8), torch.empty(t, device=dev)
        s["codes"], s["scales"] = _codes_out(dev, t, h, c)
    return s


# ---- the plain forms, in 32 bits ------------------------------------------------------------------------


def _plain_row_codes(v):
    amax = v.abs().amax(-1, keepdim=True)
    top = torch.full_like(amax, 127.0)
    scale = (amax / top).clamp_min(TINY)
    mul = torch.where(amax / top < TINY, torch.full_like(amax, 1 / TINY), top / amax)
    return (v * mul).clamp(-127, 127).round(), scale


def _plain_codes(v, c):
    kind, layout = c["codes"], c["scales"]
    t, h = v.shape
    v = v.view(t, -1, GROUP[layout])
    amax = v.abs().amax(-1, keepdim=True)
    if layout == "f32_group128":
        top = torch.full_like(amax, QMAX[kind])
        scale = (amax / top).clamp_min(TINY)
        mul = torch.where(amax / top < TINY, torch.full_like(amax, 1 / TINY), top / amax)
        held = scale
    else:
        e = torch.frexp(amax)[1] - 1 - EMAX[kind]
        e = torch.where(amax == 0, torch.full_like(e, -127), e).clamp(-127, 127)
        held = torch.ldexp(torch.ones_like(amax), e).to(torch.float8_e8m0fnu)
        mul = torch.ldexp(torch.ones_like(amax), -e)
    q = (v * mul).clamp(-QMAX[kind], QMAX[kind]).to(FP8[kind])
    return q.view(t, h), held.view(t, -1)


def _plain_norm(s):
    total = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    v = total.float()
    return total, v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()


def _plain_product(a, a_scales, b, b_scales, gated=False):
    p = (a.float() @ b.float().t()) * a_scales.view(-1, 1) * b_scales
    if not gated:
        return p
    gate, up = p.chunk(2, dim=1)
    return gate * torch.sigmoid(gate) * up


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        total, y = _plain_norm(s)
        return (total, *_plain_codes(y, c))
    if op == "norm_grad":
        v, w, dy = s["sum"].float(), s["weight"].float(), s["grad_y"].float()
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        dn = dy * w
        dx = s["grad_sum"].float() + r * (dn - v * (r * r * (dn * v).mean(-1, keepdim=True)))
        return dx.to(s["sum"].dtype), (dy * v * r).sum(0)
    if op == "product":
        return _plain_product(s["a"], s["a_scales"], s["b"], s["b_scales"], c["gated"]).to(TYPES[c["type"]])
    if op == "partial":
        return _plain_codes(_plain_product(s["a"], s["a_scales"], s["b"], s["b_scales"]), c)
    total, y = _plain_norm(s)
    q, scale = _plain_row_codes(y)
    if op == "project":
        return total, _plain_product(q, scale, s["b"], s["b_scales"]).to(TYPES[c["type"]])
    mid = _plain_product(q, scale, s["up"], s["up_scales"], True).to(TYPES[c["type"]])
    q, scale = _plain_row_codes(mid.float())
    return (total, *_plain_codes(_plain_product(q, scale, s["down"], s["down_scales"]), c))


# ---- the package's operators ----------------------------------------------------------------------------


def _run_own(s):
    import quantized_collective_reduction_amd as qrs

    c = s["case"]
    op = c["op"]
    if op == "norm":
        qrs.add_rms_norm_quantize(s["x"], s["residual"], s["weight"], EPS, s["sum"], s["codes"], s["scales"],
                                  c["codes"], c["scales"])
        return s["sum"], s["codes"], s["scales"]
    if op == "norm_grad":
        qrs.rms_norm_backward(s["grad_y"], s["sum"], s["weight"], EPS, s["grad_sum"], s["grad_x"], s["grad_weight"])
        return s["grad_x"], s["grad_weight"]
    if op == "product":
        qrs.matmul_int8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], gated=c["gated"])
        return s["out"]
    if op == "partial":
        qrs.matmul_int8_quantize(s["a"], s["a_scales"], s["b"], s["b_scales"], s["codes"], s["scales"],
                                 c["codes"], c["scales"])
        return s["codes"], s["scales"]
    qrs.add_rms_norm_quantize(s["x"], s["residual"], s["weight"], EPS, s["sum"], s["qa"], s["qs"], "int8", "f32_row")
    if op == "project":
        qrs.matmul_int8(s["qa"], s["qs"], s["b"], s["b_scales"], s["out"])
        return s["sum"], s["out"]
    qrs.matmul_int8(s["qa"], s["qs"], s["up"], s["up_scales"], s["mid"], gated=True)
    qrs.quantize_rows(s["mid"], s["qm"], s["qms"], "int8")
    qrs.matmul_int8_quantize(s["qm"], s["qms"], s["down"], s["down_scales"], s["codes"], s["scales"],
                             c["codes"], c["scales"])
    return s["sum"], s["codes"], s["scales"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ----------------------------------------------------------------------


def work(case):
    c = case
    op = c["op"]
    size = 4 if c.get("type") == "f32" else 2
    if op == "norm":  # x, residual in; sum, codes, scales out; weight
        n = c["tokens"] * c["h"]
        return {"bytes": n * (3 * size + 1 + 1 / 32) + c["h"] * size, "flops": 8 * n}
    if op == "norm_grad":  # grad_y, sum, grad_sum in; grad_x out; weight, grad_weight
        n = c["tokens"] * c["h"]
        return {"bytes": n * 4 * size + c["h"] * (size + 4), "flops": 14 * n}
    if op in ("product", "partial"):
        m, n, k = c["m"], c["n"], c["k"]
        wide = 2 * n if c.get("gated") else n
        out = m * n * (size if op == "product" else 1 + 1 / 32)
        return {"bytes": m * k + wide * k + 4 * (m + wide) + out, "flops": 2 * m * wide * k}
    t, h = c["tokens"], c["h"]
    norm = t * h * 3 * size + h * size
    if op == "project":
        n = c["n"]
        return {"bytes": norm + n * h + 4 * n + t * n * size, "flops": 2 * t * n * h + 8 * t * h}
    i = c["inner"]
    return {"bytes": norm + 3 * i * h + 4 * (2 * i + h) + t * h * (1 + 1 / 32), "flops": 6 * t * i * h + 8 * t * h}


# ---- the definitions in 64 bits -------------------------------------------------------------------------


def _grid(q, kind):
    """The format's value nearest each element of q, ties to even."""
    digits, low = (3, -6) if kind == "e4m3fn" else (2, -14)
    e = torch.frexp(q)[1].to(torch.float64) - 1
    step = torch.exp2(e.clamp_min(low) - digits)
    return torch.round(q / step) * step


def _exact_codes(y, c):
    kind, layout = c["codes"], c["scales"]
    y = y.unflatten(1, (-1, GROUP[layout]))
    amax = y.abs().max(dim=2, keepdim=True).values
    if layout == "f32_group128":
        scale = torch.clamp(amax / QMAX[kind], min=TINY)
    else:
        e = torch.frexp(amax)[1].to(torch.float64) - 1 - EMAX[kind]
        scale = torch.exp2(torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127))
    q = _grid(torch.clamp(y / scale, -QMAX[kind], QMAX[kind]), kind)
    return q.flatten(1), scale.squeeze(2)


def _exact_rows(y):
    scale = torch.clamp(y.abs().max(dim=1, keepdim=True).values / 127, min=TINY)
    return torch.round(y / scale), scale.squeeze(1)


def _exact_product(a, a_scales, b, b_scales, gated=False):
    p = torch.einsum("mk,nk->mn", a.double(), b.double())
    p = p * a_scales.double().unsqueeze(1) * b_scales.double().unsqueeze(0)
    if gated:
        n = p.shape[1] // 2
        p = p[:, :n] / (1 + torch.exp(-p[:, :n])) * p[:, n:]
    return p


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "product":
        return _exact_product(s["a"], s["a_scales"], s["b"], s["b_scales"], c["gated"])
    if op == "partial":
        return _exact_codes(_exact_product(s["a"], s["a_scales"], s["b"], s["b_scales"]), c)
    if op == "norm_grad":
        v, w, dy = s["sum"].double(), s["weight"].double(), s["grad_y"].double()
        rms = torch.sqrt((v * v).mean(dim=1) + EPS).unsqueeze(1)
        unit = v / rms
        along = (dy * w * unit).mean(dim=1).unsqueeze(1)
        return s["grad_sum"].double() + (dy * w - unit * along) / rms, (dy * unit).sum(dim=0)
    total = (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
    v = total.double()
    y = v / torch.sqrt((v * v).mean(dim=1) + EPS).unsqueeze(1) * s["weight"].double()
    if op == "norm":
        return (v, *_exact_codes(y, c))
    q, scale = _exact_rows(y)
    if op == "project":
        return v, _exact_product(q, scale, s["b"], s["b_scales"])
    mid = _exact_product(q, scale, s["up"], s["up_scales"], True).to(TYPES[c["type"]])
    q, scale = _exact_rows(mid.double())
    return (v, *_exact_codes(_exact_product(q, scale, s["down"], s["down_scales"]), c))
