"""What layer norm, the block quantizations and the 8-bit floating-point product
refuse, on the host: every call here breaks one documented constraint, with
addresses that nothing dereferences."""

import ctypes

import pytest

import quantized_collective_reduction_amd as qrs

INVALID, UNSUPPORTED = int(qrs.Status.INVALID_ARG), int(qrs.Status.UNSUPPORTED)
F32, BF16 = 0, 1
INT8, E4M3, E5M2, HIF8 = 0, 1, 2, 3
GROUP, MX, ROW = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    import torch

    if torch.cuda.is_available():
        pytest.skip("fake-address checks run only without a GPU")
    return qrs.load_library()


def _at(i):
    """Addresses 4 GiB apart: no two of the small tensors below overlap."""
    return (i + 1) << 32


NORM = dict(tokens=4, h=1024, io=BF16, xd=E4M3, sl=GROUP, eps=1e-5, x=_at(0), ldx=1024, r=_at(1), ldr=1024, w=_at(2),
            b=_at(6), s=_at(3), lds=1024, c=_at(4), ldc=1024, sc=_at(5))
BACK = dict(tokens=4, h=1024, io=BF16, eps=1e-5, dy=_at(0), ldy=1024, s=_at(1), lds=1024, w=_at(2), g=_at(3), ldg=1024,
            dx=_at(4), ldx=1024, dw=_at(5), db=_at(7), ws=_at(6), wsb=1 << 20)
BLOCKS = dict(rows=300, cols=200, kind=BF16, xd=E4M3, x=_at(0), ldx=200, c=_at(1), ldc=200, sc=_at(2), ct=_at(3),
              rt=304, ldct=304, sct=_at(4))
MM = dict(m=4, n=256, k=512, gated=0, kind=BF16, ad=E4M3, a=_at(0), lda=512, sa=_at(1), bd=E4M3, bs=128, b=_at(2),
          ldb=512, sb=_at(3), o=_at(4), ldo=256)
MMQ = dict(m=4, n=256, k=512, gated=0, xd=E4M3, sl=MX, ad=E4M3, a=_at(0), lda=512, sa=_at(1), bd=E5M2, b=_at(2),
           ldb=512, sb=_at(3), c=_at(4), ldc=256, sc=_at(6), ws=_at(7), wsb=1 << 20)


def _norm(lib, **kw):
    d = {**NORM, **kw}
    return lib.qrs_add_layer_norm_quantize(d["tokens"], d["h"], d["io"], d["xd"], d["sl"], d["eps"], d["x"], d["ldx"],
                                           d["r"], d["ldr"], d["w"], d["b"], d["s"], d["lds"], d["c"], d["ldc"],
                                           d["sc"], None)


def _back(lib, **kw):
    d = {**BACK, **kw}
    return lib.qrs_layer_norm_backward(d["tokens"], d["h"], d["io"], d["eps"], d["dy"], d["ldy"], d["s"], d["lds"],
                                       d["w"], d["g"], d["ldg"], d["dx"], d["ldx"], d["dw"], d["db"], d["ws"], d["wsb"],
                                       None)


def _blocks(lib, **kw):
    d = {**BLOCKS, **kw}
    return lib.qrs_quantize_blocks(d["rows"], d["cols"], d["kind"], d["xd"], d["x"], d["ldx"], d["c"], d["ldc"],
                                   d["sc"], d["ct"], d["rt"], d["ldct"], d["sct"], None)


def _transposed(lib, **kw):
    d = {**BLOCKS, **kw}
    return lib.qrs_quantize_transposed(d["rows"], d["cols"], d["kind"], d["xd"], d["x"], d["ldx"], d["ct"], d["rt"],
                                       d["ldct"], d["sct"], d["c"], d["ldc"], d["sc"], None)


def _mm(lib, **kw):
    d = {**MM, **kw}
    return lib.qrs_matmul_float(d["m"], d["n"], d["k"], d["gated"], d["kind"], d["ad"], d["a"], d["lda"], d["sa"],
                                d["bd"], d["bs"], d["b"], d["ldb"], d["sb"], d["o"], d["ldo"], None)


def _mmq(lib, **kw):
    d = {**MMQ, **kw}
    return lib.qrs_matmul_float_quantize(d["m"], d["n"], d["k"], d["gated"], d["xd"], d["sl"], d["ad"], d["a"],
                                         d["lda"], d["sa"], d["bd"], d["b"], d["ldb"], d["sb"], d["c"], d["ldc"],
                                         d["sc"], d["ws"], d["wsb"], None)


NORM_BAD = [
    (dict(tokens=0), "must be positive"), (dict(tokens=1 << 50), "too many"), (dict(h=0), "must be in"),
    (dict(h=65664, ldx=65664), "must be in"), (dict(h=1040), "not a multiple"), (dict(sl=MX, h=1040), "not a multiple"),
    (dict(io=3), "io_dtype"), (dict(xd=7), "x_dtype"), (dict(sl=MX, xd=INT8), "INT8"), (dict(sl=3), "scale_layout"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(x=None), "x"), (dict(w=None), "weight"),
    (dict(c=None), "codes"), (dict(sc=None), "scales"), (dict(s=None), "sum_out"), (dict(x=_at(0) + 1), "aligned"),
    (dict(b=_at(6) + 1), "bias is not aligned"), (dict(ldx=1023), "row stride"), (dict(ldr=0), "row stride"),
    (dict(lds=-4), "row stride"), (dict(ldc=1 << 50), "too large"), (dict(s=_at(0) + 2048), "overlaps"),
    (dict(s=_at(0), lds=2048), "overlaps"), (dict(c=_at(0)), "overlaps"), (dict(sc=_at(4) + 4), "overlaps"),
    (dict(s=_at(2)), "overlaps"), (dict(s=_at(6)), "overlaps bias"), (dict(c=_at(6) + 100), "overlaps bias"),
]
BACK_BAD = [
    (dict(tokens=0), "must be positive"), (dict(h=65537), "must be in"), (dict(io=5), "io_dtype"),
    (dict(eps=-0.5), "eps"), (dict(ws=None), "workspace"), (dict(wsb=2 * 4 * 1024 * 4 - 1), "workspace"),
    (dict(ws=_at(6) + 8), "16-byte"), (dict(dy=None), "grad_y"), (dict(s=None), "sum"), (dict(w=None), "weight"),
    (dict(dx=None), "grad_x"), (dict(dw=None), "grad_weight"), (dict(ldg=1000), "row stride"),
    (dict(dx=_at(1)), "overlaps"), (dict(dx=_at(0), ldx=1032), "overlaps"), (dict(dw=_at(4) + 4), "overlaps"),
    (dict(ws=_at(3)), "overlaps"), (dict(db=_at(2)), "overlaps"), (dict(db=_at(5)), "overlaps grad_bias"),
    (dict(db=_at(7) + 2), "aligned"), (dict(db=_at(6) + 8192 * 4 - 4), "overlaps"),
]
BLOCKS_BAD = [
    (dict(rows=0), "must be positive"), (dict(cols=-1), "must be positive"), (dict(rows=1 << 31), "below 2^31"),
    (dict(rows=(1 << 31) - 1, cols=1 << 17), "too large"), (dict(kind=4), "in_dtype"), (dict(xd=INT8), "x_dtype"),
    (dict(xd=HIF8), "x_dtype"), (dict(x=None), "x"), (dict(sc=None), "scales"), (dict(sct=None), "scales_t"),
    (dict(ldx=199), "row stride"), (dict(ldc=199), "row stride"), (dict(ldct=303), "row stride"),
    (dict(rt=299), "rows_t"), (dict(rt=385, ldct=385), "rows_t"), (dict(x=_at(0) + 1), "aligned"),
    (dict(sc=_at(2) + 2), "aligned"), (dict(c=_at(0) + 300), "overlaps"), (dict(ct=_at(1) + 9), "overlaps"),
    (dict(sct=_at(2)), "overlaps"), (dict(sc=_at(3) + 304 * 199), "overlaps"), (dict(ct=_at(0)), "overlaps"),
]
MM_BAD = [
    (dict(m=0), "must be positive"), (dict(n=1 << 31), "below 2^31"), (dict(k=0), "k 0"),
    (dict(k=(1 << 24) + 1), "16777216"), (dict(gated=2), "gated"), (dict(m=(1 << 31) - 1, n=1 << 20), "too large"),
    (dict(kind=3), "out_dtype"), (dict(ad=INT8), "a_dtype"), (dict(bd=HIF8), "b_dtype"), (dict(bs=64), "b_scale_rows"),
    (dict(bs=1, gated=1), "128 rows"), (dict(a=None), "a"), (dict(b=None), "b"), (dict(sa=None), "a_scales"),
    (dict(sb=None), "b_scales"), (dict(o=None), "out"), (dict(lda=511), "row stride"), (dict(ldb=500), "row stride"),
    (dict(ldo=255), "row stride"), (dict(o=_at(4) + 1), "aligned"), (dict(sa=_at(1) + 2), "aligned"),
    (dict(o=_at(0) + 16), "overlaps"), (dict(o=_at(3) + 4 * 2 * 4 - 2), "overlaps"),
    (dict(bs=1, o=_at(3) + 4 * 256 * 4 - 2), "overlaps"), (dict(gated=1, o=_at(2) + 512 * 512 - 2), "overlaps"),
    (dict(gated=1, o=_at(3) + 4 * 4 * 4 - 2), "overlaps"),
]
MMQ_BAD = [
    (dict(n=200, ldc=208), "multiple of 128"), (dict(xd=INT8), "INT8"), (dict(sl=ROW), "scale_layout"),
    (dict(c=_at(4) + 8), "16-byte"), (dict(ldc=264), "16-byte"), (dict(sc=None), "scales"), (dict(c=None), "codes"),
    (dict(sc=_at(4) + 1), "overlaps"), (dict(sc=_at(2)), "overlaps"), (dict(sl=GROUP, sc=_at(6) + 1), "aligned"),
    (dict(m=0), "must be positive"), (dict(k=-3), "k -3"), (dict(ad=INT8), "a_dtype"), (dict(bd=INT8), "b_dtype"),
    (dict(sl=GROUP, ws=None), "workspace"), (dict(sl=GROUP, wsb=4 * 256 * 4 - 1), "workspace"),
    (dict(sl=GROUP, ws=_at(7) + 4), "16-byte"), (dict(sl=GROUP, ws=_at(4)), "overlaps"),
    (dict(sl=GROUP, ws=_at(2)), "overlaps b"), (dict(sl=GROUP, ws=_at(6)), "overlaps scales"),
]


@pytest.mark.parametrize("call,cases", [(_norm, NORM_BAD), (_back, BACK_BAD), (_blocks, BLOCKS_BAD),
                                        (_transposed, BLOCKS_BAD), (_mm, MM_BAD), (_mmq, MMQ_BAD)],
                         ids=lambda v: getattr(v, "__name__", ""))
def test_refusals(lib, call, cases):
    for kw, text in cases:
        assert call(lib, **kw) == INVALID, (call.__name__, kw)
        assert text in lib.qrs_last_error().decode(), (call.__name__, kw, lib.qrs_last_error())


def test_what_may_be_left_out(lib):
    assert _blocks(lib, c=None, ct=None) == INVALID
    assert _transposed(lib, ct=None) == INVALID
    assert "codes_t" in lib.qrs_last_error().decode()


@pytest.mark.parametrize("call", [_norm, _mmq])
def test_hifloat8_is_unsupported(lib, call):
    assert call(lib, xd=HIF8) == UNSUPPORTED


def test_workspace_query(lib):
    n = ctypes.c_size_t(7)
    assert lib.qrs_layer_norm_backward_workspace(4, 1024, ctypes.byref(n)) == 0
    assert n.value == 4 * 2 * 1024 * 4  # a row of both sums for each of the four rows
    assert lib.qrs_layer_norm_backward_workspace(1 << 20, 1024, ctypes.byref(n)) == 0
    assert 0 < n.value <= 1 << 24  # bounded whatever the number of tokens
    assert lib.qrs_layer_norm_backward_workspace(0, 1024, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.qrs_layer_norm_backward_workspace(4, 1024, None) == INVALID


def test_product_workspace_query(lib):
    n = ctypes.c_size_t(7)
    ask = lib.qrs_matmul_float_quantize_workspace
    for gated in (0, 1):
        assert ask(32, 256, gated, GROUP, ctypes.byref(n)) == 0 and n.value == 32 * 256 * 4
        assert ask(33, 256, gated, GROUP, ctypes.byref(n)) == 0 and n.value == 0
        assert ask(32, 256, gated, MX, ctypes.byref(n)) == 0 and n.value == 32 * 256 * 4 * gated
    assert ask(32, 200, 0, GROUP, ctypes.byref(n)) == INVALID and ask(32, 256, 2, GROUP, ctypes.byref(n)) == INVALID
    assert ask(32, 256, 0, ROW, ctypes.byref(n)) == INVALID and ask(32, 256, 0, GROUP, None) == INVALID


def test_launch_info_refusals(lib):
    info = qrs.MatmulInfo()
    ref = ctypes.byref(info)
    call = lib.qrs_matmul_float_launch_info
    assert call(4, 256, 512, 0, 128, 0, BF16, 0, ref) == 0 and info.blocks > 0
    for args in [(4, 256, 512, 0, 128, 2, BF16, 0, ref), (4, 200, 512, 0, 128, 1, BF16, 0, ref),
                 (4, 256, 512, 0, 1, 1, BF16, 0, ref), (4, 256, 512, 1, 1, 0, BF16, 0, ref),
                 (4, 256, 0, 0, 128, 0, BF16, 0, ref), (4, 256, 512, 0, 128, 1, BF16, ROW, ref),
                 (4, 256, 512, 0, 128, 0, 7, 0, ref), (4, 256, 512, 0, 128, 0, BF16, 0, None)]:
        assert call(*args) == INVALID, args


def test_binding_refuses_before_it_calls():
    """Host tensors, and formats and shapes that do not go together."""
    import torch

    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 128, dtype=torch.float8_e4m3fn), torch.zeros(2, 1)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.add_layer_norm_quantize(x, x, x[0], x[0], 1e-5, x, c, s, "e4m3fn", "f32_group128")
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.layer_norm_backward(x, x, x[0], 1e-5, None, x, s)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.quantize_blocks(x, c, s, "e4m3fn")
    with pytest.raises(ValueError, match="codes_t"):
        qrs.quantize_transposed(x, None, None, "e4m3fn", c, s)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.matmul_fp8(c, s, c, s, x)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.matmul_fp8_quantize(c, s, c, s, c, s, "e4m3fn", "f32_group128")
