"""What the operators between two shares refuse, on the host: every call here
breaks one documented constraint, with addresses that nothing dereferences."""

import ctypes

import pytest

import quantized_collective_reduction_amd as qrs

INVALID, UNSUPPORTED = int(qrs.Status.INVALID_ARG), int(qrs.Status.UNSUPPORTED)
F32, BF16 = 0, 1
INT8, E4M3, HIF8 = 0, 1, 3
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


NORM = dict(tokens=4, h=1024, io=BF16, xd=E4M3, sl=MX, eps=1e-5, x=_at(0), ldx=1024, r=_at(1), ldr=1024, w=_at(2),
            s=_at(3), lds=1024, c=_at(4), ldc=1024, sc=_at(5))
BACK = dict(tokens=4, h=1024, io=BF16, eps=1e-5, dy=_at(0), ldy=1024, s=_at(1), lds=1024, w=_at(2), g=_at(3), ldg=1024,
            dx=_at(4), ldx=1024, dw=_at(5), ws=_at(6), wsb=1 << 20)
QROWS = dict(rows=4, cols=1000, kind=BF16, xd=INT8, x=_at(0), ldx=1000, c=_at(1), ldc=1000, sc=_at(2))
MM = dict(m=4, n=256, k=512, gated=0, kind=BF16, a=_at(0), lda=512, sa=_at(1), b=_at(2), ldb=512, sb=_at(3), o=_at(4),
          ldo=256)
MMQ = dict(m=4, n=256, k=512, xd=E4M3, sl=MX, a=_at(0), lda=512, sa=_at(1), b=_at(2), ldb=512, sb=_at(3), c=_at(4),
           ldc=256, sc=_at(6))


def _norm(lib, **kw):
    d = {**NORM, **kw}
    return lib.qrs_add_rms_norm_quantize(d["tokens"], d["h"], d["io"], d["xd"], d["sl"], d["eps"], d["x"], d["ldx"],
                                         d["r"], d["ldr"], d["w"], d["s"], d["lds"], d["c"], d["ldc"], d["sc"], None)


def _back(lib, **kw):
    d = {**BACK, **kw}
    return lib.qrs_rms_norm_backward(d["tokens"], d["h"], d["io"], d["eps"], d["dy"], d["ldy"], d["s"], d["lds"],
                                     d["w"], d["g"], d["ldg"], d["dx"], d["ldx"], d["dw"], d["ws"], d["wsb"], None)


def _qrows(lib, **kw):
    d = {**QROWS, **kw}
    return lib.qrs_quantize_rows(d["rows"], d["cols"], d["kind"], d["xd"], d["x"], d["ldx"], d["c"], d["ldc"], d["sc"],
                                 None)


def _mm(lib, **kw):
    d = {**MM, **kw}
    return lib.qrs_matmul_int(d["m"], d["n"], d["k"], d["gated"], d["kind"], d["a"], d["lda"], d["sa"], d["b"],
                              d["ldb"], d["sb"], d["o"], d["ldo"], None)


def _mmq(lib, **kw):
    d = {**MMQ, **kw}
    return lib.qrs_matmul_int_quantize(d["m"], d["n"], d["k"], d["xd"], d["sl"], d["a"], d["lda"], d["sa"], d["b"],
                                       d["ldb"], d["sb"], d["c"], d["ldc"], d["sc"], None)


NORM_BAD = [
    (dict(tokens=0), "must be positive"), (dict(tokens=-1), "must be positive"), (dict(tokens=1 << 50), "too many"),
    (dict(h=0), "must be in"), (dict(h=65664, ldx=65664), "must be in"), (dict(h=1040), "not a multiple"),
    (dict(sl=GROUP, h=1056), "not a multiple"), (dict(io=3), "io_dtype"), (dict(io=-1), "io_dtype"),
    (dict(xd=7), "x_dtype"), (dict(xd=INT8), "INT8"), (dict(sl=3), "scale_layout"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(x=None), "x"), (dict(w=None), "weight"), (dict(c=None), "codes"), (dict(sc=None), "scales"),
    (dict(s=None), "sum_out"), (dict(x=_at(0) + 1), "aligned"), (dict(sl=GROUP, sc=_at(5) + 2), "aligned"),
    (dict(ldx=1023), "row stride"), (dict(ldr=0), "row stride"), (dict(lds=-4), "row stride"),
    (dict(ldc=1 << 50), "too large"),
    (dict(s=_at(0) + 2048), "overlaps"), (dict(s=_at(0), lds=2048), "overlaps"), (dict(c=_at(0)), "overlaps"),
    (dict(c=_at(1) + 100), "overlaps"), (dict(sc=_at(4) + 5), "overlaps"), (dict(s=_at(2)), "overlaps"),
    (dict(sc=_at(2) + 9), "overlaps"),
]
BACK_BAD = [
    (dict(tokens=0), "must be positive"), (dict(h=65537), "must be in"), (dict(io=5), "io_dtype"),
    (dict(eps=-0.5), "eps"), (dict(ws=None), "workspace"), (dict(wsb=4 * 1024 * 4 - 1), "workspace"),
    (dict(ws=_at(6) + 8), "16-byte"), (dict(dy=None), "grad_y"), (dict(s=None), "sum"), (dict(w=None), "weight"),
    (dict(dx=None), "grad_x"), (dict(dw=None), "grad_weight"), (dict(ldg=1000), "row stride"),
    (dict(dx=_at(1)), "overlaps"), (dict(dx=_at(0), ldx=1032), "overlaps"), (dict(dw=_at(4) + 4), "overlaps"),
    (dict(ws=_at(3)), "overlaps"), (dict(dw=_at(2)), "overlaps"), (dict(dw=_at(5) + 2), "aligned"),
]
QROWS_BAD = [
    (dict(rows=0), "must be positive"), (dict(cols=0), "must be in"), (dict(cols=70000, ldx=70000), "must be in"),
    (dict(kind=9), "in_dtype"), (dict(xd=4), "x_dtype"), (dict(x=None), "x"), (dict(c=None), "codes"),
    (dict(sc=None), "scales"), (dict(ldx=999), "row stride"), (dict(ldc=999), "row stride"),
    (dict(c=_at(0) + 7), "overlaps"), (dict(sc=_at(1) + 4), "overlaps"), (dict(sc=_at(2) + 1), "aligned"),
]
MM_BAD = [
    (dict(m=0), "must be positive"), (dict(n=0), "must be positive"), (dict(n=1 << 31), "below 2^31"),
    (dict(k=0), "k 0"), (dict(k=131072, lda=131072, ldb=131072), "131071"), (dict(gated=2), "gated"),
    (dict(m=(1 << 31) - 1, n=1 << 20), "too large"), (dict(kind=3), "out_dtype"), (dict(a=None), "a"),
    (dict(b=None), "b"), (dict(sa=None), "a_scales"), (dict(sb=None), "b_scales"), (dict(o=None), "out"),
    (dict(lda=511), "row stride"), (dict(ldb=500), "row stride"), (dict(ldo=255), "row stride"),
    (dict(o=_at(4) + 1), "aligned"), (dict(sa=_at(1) + 2), "aligned"), (dict(o=_at(0) + 16), "overlaps"),
    (dict(o=_at(3)), "overlaps"), (dict(o=_at(2) + 128 * 1024 - 2), "overlaps"),
    (dict(gated=1, o=_at(2) + 256 * 1024 - 2), "overlaps"),
]
MMQ_BAD = [
    (dict(n=200, ldc=208), "multiple of 128"), (dict(xd=INT8), "INT8"), (dict(sl=ROW), "scale_layout"),
    (dict(c=_at(4) + 8), "16-byte"), (dict(ldc=264), "16-byte"), (dict(sc=None), "scales"), (dict(c=None), "codes"),
    (dict(sc=_at(4) + 1), "overlaps"), (dict(sc=_at(2)), "overlaps"), (dict(sl=GROUP, sc=_at(6) + 1), "aligned"),
    (dict(m=0), "must be positive"), (dict(k=-3), "k -3"),
]


@pytest.mark.parametrize("call,cases", [(_norm, NORM_BAD), (_back, BACK_BAD), (_qrows, QROWS_BAD), (_mm, MM_BAD),
                                        (_mmq, MMQ_BAD)], ids=lambda v: getattr(v, "__name__", ""))
def test_refusals(lib, call, cases):
    for kw, text in cases:
        assert call(lib, **kw) == INVALID, (call.__name__, kw)
        assert text in lib.qrs_last_error().decode(), (call.__name__, kw, lib.qrs_last_error())


@pytest.mark.parametrize("call", [_norm, _qrows, _mmq])
def test_hifloat8_is_unsupported(lib, call):
    assert call(lib, xd=HIF8) == UNSUPPORTED


def test_workspace_query(lib):
    n = ctypes.c_size_t(7)
    assert lib.qrs_rms_norm_backward_workspace(4, 1024, ctypes.byref(n)) == 0
    assert n.value == 4 * 1024 * 4  # a row of sums for each of the four rows
    assert lib.qrs_rms_norm_backward_workspace(1 << 20, 1024, ctypes.byref(n)) == 0
    assert 0 < n.value <= 1 << 23  # bounded whatever the number of tokens
    assert lib.qrs_rms_norm_backward_workspace(0, 1024, ctypes.byref(n)) == INVALID and n.value == 0
    assert lib.qrs_rms_norm_backward_workspace(4, 1024, None) == INVALID


def test_row_scales_are_no_mode_of_the_reduce_scatter(lib):
    h, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert lib.qrs_plan(2, 32, 1024, INT8, ROW, F32, ctypes.byref(h), ctypes.byref(n)) == INVALID
    assert lib.qrs_quantize(4, 1024, INT8, ROW, _at(0), _at(1), _at(2), None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch

    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 128, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.quantize_rows(x, c, s)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        qrs.quantize_rows(c, c, s)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.add_rms_norm_quantize(x, x, x[0], 1e-5, x, c, s, "int8", "f32_row")
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.rms_norm_backward(x, x, x[0], 1e-5, None, x, s)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.matmul_int8(c, s, c, s, x)
    with pytest.raises(ValueError, match="device tensors only"):
        qrs.matmul_int8_quantize(c, s, c, s, c, s, "e4m3fn", "f32_group128")
