"""Python binding for libqrs: one GPU's share of a quantized reduce-scatter
on MI355X.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI (include/qrs.h). torch supplies device memory and
streams. If the built library is missing, loading fails with an error; there
is no CPU fallback.

    p = plan(world_size=8, bs=16384, h=8192, x_dtype="e4m3fn",
             scale_layout="e8m0_block32", out_dtype="bf16")
    run(p, x_slices, scale_slices, out)        # on torch's current stream

``x_slices`` / ``scale_slices`` are sequences of W device tensors (or raw
device pointers as ints); ``out`` is a ``[rows, H]`` device tensor.

What a layer computes between one share and the next, with 8-bit weights:

    add_rms_norm_quantize(x, residual, weight, eps, total, codes, scales, "int8", "f32_row")
    matmul_int8(codes, scales, w, w_scales, out)               # gated=True: silu(gate) * up
    quantize_rows(out, codes2, scales2, "int8")
    matmul_int8_quantize(codes2, scales2, w2, w2_scales, x_codes, x_scales, "e4m3fn", "e8m0_block32")
"""

import ctypes
import functools
import os
from enum import IntEnum

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqrs.so")

__all__ = [
    "Status",
    "XDtype",
    "ScaleLayout",
    "OutDtype",
    "QrsError",
    "Plan",
    "load_library",
    "plan",
    "run",
    "run_all_shares",
    "run_strided",
    "slice_pitch",
    "alloc_slices",
    "quantize",
    "Launch",
    "StridedLaunch",
    "AllSharesLaunch",
    "QuantizeLaunch",
    "add_rms_norm_quantize",
    "rms_norm_backward",
    "quantize_rows",
    "matmul_int8",
    "matmul_int8_quantize",
    "stream_copy",
    "run_launch_info",
    "LaunchInfo",
    "matmul_launch_info",
    "EXPORTED_SYMBOLS",
]


class Status(IntEnum):
    OK = 0
    INVALID_ARG = 1
    UNSUPPORTED = 2
    HIP = 3
    OUT_OF_MEMORY = 4


class XDtype(IntEnum):
    INT8 = 0
    FP8_E4M3FN = 1
    FP8_E5M2 = 2
    HIFLOAT8 = 3


class ScaleLayout(IntEnum):
    F32_GROUP128 = 0
    E8M0_BLOCK32 = 1
    F32_ROW = 2  # add_rms_norm_quantize only


class OutDtype(IntEnum):
    F32 = 0
    BF16 = 1
    F16 = 2


_X_NAMES = {"int8": XDtype.INT8, "e4m3fn": XDtype.FP8_E4M3FN, "e5m2": XDtype.FP8_E5M2, "hifloat8": XDtype.HIFLOAT8}
_SCALE_NAMES = {"f32_group128": ScaleLayout.F32_GROUP128, "e8m0_block32": ScaleLayout.E8M0_BLOCK32,
                "f32_row": ScaleLayout.F32_ROW}
_OUT_NAMES = {"f32": OutDtype.F32, "bf16": OutDtype.BF16, "f16": OutDtype.F16}

# Every function include/qrs.h declares.
EXPORTED_SYMBOLS = (
    "qrs_plan",
    "qrs_run",
    "qrs_run_all_shares",
    "qrs_run_strided",
    "qrs_quantize",
    "qrs_plan_destroy",
    "qrs_plan_shape",
    "qrs_slice_pitch",
    "qrs_status_string",
    "qrs_last_error",
    "qrs_stream_copy",
    "qrs_run_launch_info",
    "qrs_launch_create",
    "qrs_launch_enqueue",
    "qrs_launch_destroy",
    "qrs_add_rms_norm_quantize",
    "qrs_rms_norm_backward",
    "qrs_rms_norm_backward_workspace",
    "qrs_quantize_rows",
    "qrs_matmul_int",
    "qrs_matmul_int_quantize",
    "qrs_matmul_launch_info",
)


class LaunchInfo(ctypes.Structure):
    """qrs_launch_info: the launch qrs_run makes for a plan (see run_launch_info)."""

    _fields_ = [
        ("blocks", ctypes.c_uint64),
        ("threads_per_block", ctypes.c_uint32),
        ("dynamic_lds_bytes", ctypes.c_uint32),
        ("blocks_per_cu_cap", ctypes.c_uint32),
        ("device_cus", ctypes.c_uint32),
        ("device_lds_per_cu", ctypes.c_uint32),
        ("device_lds_per_block", ctypes.c_uint32),
        ("launches", ctypes.c_uint32),
    ]

    def as_dict(self):
        return {name: int(getattr(self, name)) for name, _ in self._fields_}


class MatmulInfo(ctypes.Structure):
    """qrs_matmul_info: the kernel a product takes (see matmul_launch_info)."""

    _fields_ = [
        ("blocks", ctypes.c_uint64),
        ("threads_per_block", ctypes.c_uint32),
        ("kernel", ctypes.c_uint32),
        ("tile_m", ctypes.c_uint32),
        ("tile_n", ctypes.c_uint32),
    ]


class QrsError(RuntimeError):
    def __init__(self, status, message):
        self.status = Status(status)
        super().__init__(f"{self.status.name}: {message}")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libqrs.so and declare its signatures. Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -m quantized_collective_reduction_amd._build` "
            "(there is no CPU fallback)"
        )
    lib = ctypes.CDLL(path)
    c_int, c_i64, c_sz, vp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
    lib.qrs_plan.argtypes = [c_int, c_i64, c_i64, c_int, c_int, c_int, ctypes.POINTER(vp), ctypes.POINTER(c_sz)]
    lib.qrs_plan.restype = c_int
    lib.qrs_run.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, vp, c_sz, vp]
    lib.qrs_run.restype = c_int
    lib.qrs_launch_create.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), vp, vp, ctypes.POINTER(vp)]
    lib.qrs_launch_create.restype = c_int
    lib.qrs_launch_enqueue.argtypes = [vp]
    lib.qrs_launch_enqueue.restype = c_int
    lib.qrs_launch_destroy.argtypes = [vp]
    lib.qrs_launch_destroy.restype = c_int
    lib.qrs_run_all_shares.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp), vp, c_sz, vp]
    lib.qrs_run_all_shares.restype = c_int
    lib.qrs_run_strided.argtypes = [vp, ctypes.POINTER(vp), c_i64, ctypes.POINTER(vp), c_i64, vp, c_i64, vp, c_sz, vp]
    lib.qrs_run_strided.restype = c_int
    lib.qrs_quantize.argtypes = [c_i64, c_i64, c_int, c_int, vp, vp, vp, vp]
    lib.qrs_quantize.restype = c_int
    lib.qrs_plan_destroy.argtypes = [vp]
    lib.qrs_plan_destroy.restype = c_int
    lib.qrs_plan_shape.argtypes = [vp, ctypes.POINTER(c_i64), ctypes.POINTER(c_i64)]
    lib.qrs_plan_shape.restype = c_int
    lib.qrs_slice_pitch.argtypes = [vp, c_int, ctypes.POINTER(c_sz), ctypes.POINTER(c_sz)]
    lib.qrs_slice_pitch.restype = c_int
    lib.qrs_status_string.argtypes = [c_int]
    lib.qrs_status_string.restype = ctypes.c_char_p
    lib.qrs_last_error.argtypes = []
    lib.qrs_last_error.restype = ctypes.c_char_p
    lib.qrs_stream_copy.argtypes = [vp, vp, c_sz, vp]
    lib.qrs_stream_copy.restype = c_int
    lib.qrs_run_launch_info.argtypes = [vp, vp, ctypes.POINTER(LaunchInfo)]
    lib.qrs_run_launch_info.restype = c_int
    c_f = ctypes.c_float
    lib.qrs_add_rms_norm_quantize.argtypes = [c_i64, c_i64, c_int, c_int, c_int, c_f, vp, c_i64, vp, c_i64, vp, vp,
                                              c_i64, vp, c_i64, vp, vp]
    lib.qrs_add_rms_norm_quantize.restype = c_int
    lib.qrs_rms_norm_backward_workspace.argtypes = [c_i64, c_i64, ctypes.POINTER(c_sz)]
    lib.qrs_rms_norm_backward_workspace.restype = c_int
    lib.qrs_rms_norm_backward.argtypes = [c_i64, c_i64, c_int, c_f, vp, c_i64, vp, c_i64, vp, vp, c_i64, vp, c_i64, vp,
                                          vp, c_sz, vp]
    lib.qrs_rms_norm_backward.restype = c_int
    lib.qrs_quantize_rows.argtypes = [c_i64, c_i64, c_int, c_int, vp, c_i64, vp, c_i64, vp, vp]
    lib.qrs_quantize_rows.restype = c_int
    lib.qrs_matmul_int.argtypes = [c_i64, c_i64, c_i64, c_int, c_int, vp, c_i64, vp, vp, c_i64, vp, vp, c_i64, vp]
    lib.qrs_matmul_int.restype = c_int
    lib.qrs_matmul_int_quantize.argtypes = [c_i64, c_i64, c_i64, c_int, c_int, vp, c_i64, vp, vp, c_i64, vp, vp,
                                            c_i64, vp, vp]
    lib.qrs_matmul_int_quantize.restype = c_int
    lib.qrs_matmul_launch_info.argtypes = [c_i64, c_i64, c_i64, c_int, c_int, c_int, ctypes.POINTER(MatmulInfo)]
    lib.qrs_matmul_launch_info.restype = c_int
    _lib = lib
    return lib


def _check(status):
    if status:  # Status.OK is 0
        msg = _lib.qrs_last_error().decode(errors="replace")
        raise QrsError(status, msg)


def _enum(value, names, enum_cls):
    if isinstance(value, str):
        key = value.lower()
        if key not in names:
            raise ValueError(f"unknown {enum_cls.__name__} {value!r}; expected one of {sorted(names)}")
        return names[key]
    return enum_cls(value) if value in enum_cls._value2member_map_ else int(value)


class Plan:
    """An immutable plan for one share shape and mode (phase 1 of the op)."""

    def __init__(self, world_size, bs, h, x_dtype, scale_layout, out_dtype):
        self._handle = None  # set first: __del__ runs even when a check below raises
        lib = load_library()
        self.world_size = int(world_size)
        self.bs = int(bs)
        self.h = int(h)
        self.x_dtype = _enum(x_dtype, _X_NAMES, XDtype)
        self.scale_layout = _enum(scale_layout, _SCALE_NAMES, ScaleLayout)
        self.out_dtype = _enum(out_dtype, _OUT_NAMES, OutDtype)
        handle = ctypes.c_void_p()
        ws = ctypes.c_size_t()
        _check(lib.qrs_plan(self.world_size, self.bs, self.h, int(self.x_dtype), int(self.scale_layout),
                            int(self.out_dtype), ctypes.byref(handle), ctypes.byref(ws)))
        self._handle = handle
        self.workspace_bytes = ws.value
        rows, hh = ctypes.c_int64(), ctypes.c_int64()
        _check(lib.qrs_plan_shape(handle, ctypes.byref(rows), ctypes.byref(hh)))
        self.rows = rows.value

    @property
    def handle(self):
        return self._handle

    @property
    def group(self):
        return 128 if self.scale_layout == ScaleLayout.F32_GROUP128 else 32

    def __del__(self):
        if getattr(self, "_handle", None) is not None and _lib is not None:
            _lib.qrs_plan_destroy(self._handle)
            self._handle = None


def plan(world_size, bs, h, x_dtype, scale_layout, out_dtype) -> Plan:
    return Plan(world_size, bs, h, x_dtype, scale_layout, out_dtype)


def slice_pitch(p: Plan, full_inputs=False):
    """Recommended byte distance between consecutive rank slices of x and of
    the scales when each kind shares one allocation (qrs_slice_pitch)."""
    lib = load_library()
    xp, sp = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.qrs_slice_pitch(p.handle, 1 if full_inputs else 0, ctypes.byref(xp), ctypes.byref(sp)))
    return xp.value, sp.value


def alloc_slices(p: Plan, device="cuda", full_inputs=False):
    """One x buffer and one scale buffer holding the W rank slices at the
    recommended pitch. Returns (x_views, scale_views): lists of W contiguous
    device views, ``[rows, H]`` uint8 and ``[rows, H/G]`` fp32 or uint8
    (``rows`` = BS with ``full_inputs``)."""
    import torch

    w = p.world_size
    rows = p.bs if full_inputs else p.rows
    xp, sp = slice_pitch(p, full_inputs)
    g = p.group
    x_buf = torch.empty(xp * w, dtype=torch.uint8, device=device)
    s_buf = torch.empty(sp * w, dtype=torch.uint8, device=device)
    xs = [x_buf[r * xp:r * xp + rows * p.h].view(rows, p.h) for r in range(w)]
    n_s = rows * p.h // g
    if p.scale_layout == ScaleLayout.F32_GROUP128:
        ss = [s_buf[r * sp:r * sp + 4 * n_s].view(torch.float32).view(rows, p.h // g) for r in range(w)]
    else:
        ss = [s_buf[r * sp:r * sp + n_s].view(rows, p.h // g) for r in range(w)]
    return xs, ss


@functools.lru_cache(maxsize=None)
def _element_dtypes():
    """torch element types of the codes, scales and outputs each mode names."""
    import torch

    return (
        {XDtype.INT8: torch.int8, XDtype.FP8_E4M3FN: torch.float8_e4m3fn, XDtype.FP8_E5M2: torch.float8_e5m2},
        {ScaleLayout.F32_GROUP128: torch.float32, ScaleLayout.E8M0_BLOCK32: torch.float8_e8m0fnu},
        {OutDtype.F32: torch.float32, OutDtype.BF16: torch.bfloat16, OutDtype.F16: torch.float16},
    )


def _check_dtype(t, want, what):
    """A tensor with a floating-point element type must have the one the mode
    names (a float16 tensor handed a bf16 result would hold wrong values);
    integer tensors are taken as raw bytes. Raw pointers are not checked, nor
    modes the library rejects anyway (want is None)."""
    if isinstance(t, int) or want is None or t.dtype == want:
        return
    if t.dtype.is_floating_point or t.dtype.is_complex:
        raise ValueError(f"{what}: dtype {t.dtype} does not match the mode's {want}")


def _check_plan_dtypes(p, xs, ss, outs, x_what, s_what, o_what):
    x_dt, s_dt, o_dt = _element_dtypes()
    for r, t in enumerate(xs):
        _check_dtype(t, x_dt.get(p.x_dtype), f"{x_what} {r}")
    for r, t in enumerate(ss):
        _check_dtype(t, s_dt.get(p.scale_layout), f"{s_what} {r}")
    for r, t in enumerate(outs):
        _check_dtype(t, o_dt.get(p.out_dtype), o_what if len(outs) == 1 else f"{o_what} {r}")


def _ptr(t):
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("device tensors only (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


@functools.lru_cache(maxsize=None)
def _current_stream_call():
    """What gives the current stream's handle. torch has it without the Stream
    object (2.7 us -> 0.2 us a call) in two functions that are not of its
    documented interface; where they are missing, the documented one is called."""
    import torch

    torch.cuda.current_device()  # initialises torch's device state, which the two need
    raw_stream, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw_stream is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw_stream(device())


def _stream_handle(stream):
    if stream is None:
        return _current_stream_call()()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensor(t, nbytes, what):
    if isinstance(t, int):
        return
    if t.numel() * t.element_size() != nbytes:
        raise ValueError(f"{what}: expected {nbytes} bytes, got {t.numel() * t.element_size()}")


def run(p: Plan, x_slices, scale_slices, out, stream=None):
    """Phase 2: enqueue the share on ``stream`` (torch's current stream by default)."""
    lib = load_library()
    w = p.world_size
    if len(x_slices) != w or len(scale_slices) != w:
        raise ValueError(f"need {w} x slices and {w} scale slices")
    n = p.rows * p.h
    scale_bytes = n // 128 * 4 if p.scale_layout == ScaleLayout.F32_GROUP128 else n // 32
    for r in range(w):
        _check_tensor(x_slices[r], n, f"x slice {r}")
        _check_tensor(scale_slices[r], scale_bytes, f"scale slice {r}")
    _check_tensor(out, n * (4 if p.out_dtype == OutDtype.F32 else 2), "out")
    _check_plan_dtypes(p, x_slices, scale_slices, [out], "x slice", "scale slice", "out")
    xs = (ctypes.c_void_p * w)(*[_ptr(t) for t in x_slices])
    ss = (ctypes.c_void_p * w)(*[_ptr(t) for t in scale_slices])
    _check(lib.qrs_run(p.handle, xs, ss, _ptr(out), None, 0, _stream_handle(stream)))


def _row_stride(tensors, rows, cols, what):
    """Common row stride (in elements) of 2-D device views [rows, cols] whose
    elements within a row are adjacent."""
    strides = set()
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("device tensors only (there is no CPU path)")
        if t.dim() != 2 or tuple(t.shape) != (rows, cols):
            raise ValueError(f"{what}: expected shape [{rows}, {cols}], got {list(t.shape)}")
        if t.stride(1) != 1 and cols > 1:
            raise ValueError(f"{what}: elements within a row must be adjacent")
        strides.add(t.stride(0) if rows > 1 else cols)
    if len(strides) != 1:
        raise ValueError(f"{what}: every slice must have the same row stride")
    return strides.pop()


def _strided_strides(p: Plan, x_slices, scale_slices, out):
    """Row strides of ``run_strided``'s views, in the units qrs_run_strided
    takes (bytes for x, scale elements, output elements). Each view's element
    must be the size of the mode's element, since the library counts its
    strides and row lengths in those."""
    ld_x = _row_stride(x_slices, p.rows, p.h, "x slices")
    ld_s = _row_stride(scale_slices, p.rows, p.h // p.group, "scale slices")
    ld_o = _row_stride([out], p.rows, p.h, "out")
    sizes = ((x_slices, 1, "x slices"),
             (scale_slices, 4 if p.scale_layout == ScaleLayout.F32_GROUP128 else 1, "scale slices"),
             ([out], 4 if p.out_dtype == OutDtype.F32 else 2, "out"))
    for tensors, size, what in sizes:
        for t in tensors:
            if t.element_size() != size:
                raise ValueError(f"{what}: {size}-byte elements expected for this plan, got {t.dtype}")
    return ld_x, ld_s, ld_o


def run_strided(p: Plan, x_slices, scale_slices, out, stream=None):
    """``run`` for 2-D views whose rows are not adjacent (row ranges of wider
    buffers, padded rows): x slices ``[rows, H]`` uint8, scale slices
    ``[rows, H/G]``, out ``[rows, H]``; each kind shares one row stride."""
    lib = load_library()
    w = p.world_size
    if len(x_slices) != w or len(scale_slices) != w:
        raise ValueError(f"need {w} x slices and {w} scale slices")
    ld_x, ld_s, ld_o = _strided_strides(p, x_slices, scale_slices, out)
    _check_plan_dtypes(p, x_slices, scale_slices, [out], "x slice", "scale slice", "out")
    xs = (ctypes.c_void_p * w)(*[t.data_ptr() for t in x_slices])
    ss = (ctypes.c_void_p * w)(*[t.data_ptr() for t in scale_slices])
    _check(lib.qrs_run_strided(p.handle, xs, ld_x, ss, ld_s, out.data_ptr(), ld_o, None, 0, _stream_handle(stream)))


def run_all_shares(p: Plan, x_full, scale_full, out_shares, stream=None):
    """Every rank's share from the ranks' inputs before the all-to-all.

    ``x_full[r]``: rank r's ``[BS, H]`` codes; ``scale_full[r]``: its scales
    for all BS rows; ``out_shares[j]``: share j's ``[BS/W, H]`` output.
    """
    lib = load_library()
    w = p.world_size
    if len(x_full) != w or len(scale_full) != w or len(out_shares) != w:
        raise ValueError(f"need {w} inputs, {w} scale tensors and {w} outputs")
    n = p.rows * p.h
    scale_bytes = n // 128 * 4 if p.scale_layout == ScaleLayout.F32_GROUP128 else n // 32
    for r in range(w):
        _check_tensor(x_full[r], n * w, f"x of rank {r}")
        _check_tensor(scale_full[r], scale_bytes * w, f"scales of rank {r}")
        _check_tensor(out_shares[r], n * (4 if p.out_dtype == OutDtype.F32 else 2), f"output of share {r}")
    _check_plan_dtypes(p, x_full, scale_full, out_shares, "x of rank", "scales of rank", "output of share")
    xs = (ctypes.c_void_p * w)(*[_ptr(t) for t in x_full])
    ss = (ctypes.c_void_p * w)(*[_ptr(t) for t in scale_full])
    os_ = (ctypes.c_void_p * w)(*[_ptr(t) for t in out_shares])
    _check(lib.qrs_run_all_shares(p.handle, xs, ss, os_, None, 0, _stream_handle(stream)))


def _check_quantize_dtypes(x_bf16, x_codes, scales, xd, sl):
    import torch

    x_dt, s_dt, _ = _element_dtypes()
    _check_dtype(x_bf16, torch.bfloat16, "x_bf16")
    _check_dtype(x_codes, x_dt.get(xd), "x_codes")
    _check_dtype(scales, s_dt.get(sl), "scales")


def quantize(x_bf16, x_codes, scales, x_dtype, scale_layout, stream=None):
    """Producer-side quantization of a bf16 ``[tokens, H]`` device tensor into
    ``x_codes`` (uint8 ``[tokens, H]``) and ``scales`` (fp32 ``[tokens, H/128]``
    or uint8 E8M0 ``[tokens, H/32]``)."""
    lib = load_library()
    if isinstance(x_bf16, int):
        raise ValueError("pass tensors (the shape is taken from x_bf16)")
    tokens, h = x_bf16.shape
    xd = _enum(x_dtype, _X_NAMES, XDtype)
    sl = _enum(scale_layout, _SCALE_NAMES, ScaleLayout)
    n = tokens * h
    _check_tensor(x_bf16, 2 * n, "x_bf16")
    _check_tensor(x_codes, n, "x_codes")
    _check_tensor(scales, n // 128 * 4 if sl == ScaleLayout.F32_GROUP128 else n // 32, "scales")
    _check_quantize_dtypes(x_bf16, x_codes, scales, xd, sl)
    _check(lib.qrs_quantize(tokens, h, int(xd), int(sl), _ptr(x_bf16), _ptr(x_codes), _ptr(scales),
                            _stream_handle(stream)))


class Launch:
    """``run`` prepared once (qrs_launch_create: the checks, the kernel, grid
    and residency cap), for repeated launches of one plan on fixed buffers
    and one stream: each call is one qrs_launch_enqueue with one argument."""

    def __init__(self, p: Plan, x_slices, scale_slices, out, stream=None):
        lib = load_library()
        w = p.world_size
        if len(x_slices) != w or len(scale_slices) != w:
            raise ValueError(f"need {w} x slices and {w} scale slices")
        n = p.rows * p.h
        scale_bytes = n // 128 * 4 if p.scale_layout == ScaleLayout.F32_GROUP128 else n // 32
        for r in range(w):
            _check_tensor(x_slices[r], n, f"x slice {r}")
            _check_tensor(scale_slices[r], scale_bytes, f"scale slice {r}")
        _check_tensor(out, n * (4 if p.out_dtype == OutDtype.F32 else 2), "out")
        _check_plan_dtypes(p, x_slices, scale_slices, [out], "x slice", "scale slice", "out")
        self._plan = p  # keeps the plan alive
        self._keep = (list(x_slices), list(scale_slices), out)  # keeps the buffers alive
        xs = (ctypes.c_void_p * w)(*[_ptr(t) for t in x_slices])
        ss = (ctypes.c_void_p * w)(*[_ptr(t) for t in scale_slices])
        h = ctypes.c_void_p()
        _check(lib.qrs_launch_create(p.handle, xs, ss, ctypes.c_void_p(_ptr(out)),
                                     ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(h)))
        self._h = h
        self._destroy = lib.qrs_launch_destroy
        self._fn = lib.qrs_launch_enqueue

    def on_stream(self, stream):
        """The same launch (plan and buffers) enqueued on another stream."""
        return Launch(self._plan, *self._keep, stream=stream)

    def __call__(self):
        status = self._fn(self._h)
        if status:
            _check(status)

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            self._destroy(h)
            self._h = None


class StridedLaunch:
    """``run_strided`` with its arguments marshalled once."""

    def __init__(self, p: Plan, x_slices, scale_slices, out, stream=None):
        lib = load_library()
        w = p.world_size
        if len(x_slices) != w or len(scale_slices) != w:
            raise ValueError(f"need {w} x slices and {w} scale slices")
        self._ld_x, self._ld_s, self._ld_o = _strided_strides(p, x_slices, scale_slices, out)
        _check_plan_dtypes(p, x_slices, scale_slices, [out], "x slice", "scale slice", "out")
        self._plan = p
        self._keep = (list(x_slices), list(scale_slices), out)
        self._xs = (ctypes.c_void_p * w)(*[t.data_ptr() for t in x_slices])
        self._ss = (ctypes.c_void_p * w)(*[t.data_ptr() for t in scale_slices])
        self._out = ctypes.c_void_p(out.data_ptr())
        self._stream = ctypes.c_void_p(_stream_handle(stream))
        self._fn = lib.qrs_run_strided
        self._handle = p.handle

    def on_stream(self, stream):
        """The same launch (plan and views) enqueued on another stream."""
        return StridedLaunch(self._plan, *self._keep, stream=stream)

    def __call__(self):
        status = self._fn(self._handle, self._xs, self._ld_x, self._ss, self._ld_s, self._out, self._ld_o, None, 0,
                          self._stream)
        if status:
            _check(status)


class AllSharesLaunch:
    """``run_all_shares`` with its arguments marshalled once."""

    def __init__(self, p: Plan, x_full, scale_full, out_shares, stream=None):
        lib = load_library()
        w = p.world_size
        if len(x_full) != w or len(scale_full) != w or len(out_shares) != w:
            raise ValueError(f"need {w} inputs, {w} scale tensors and {w} outputs")
        n = p.rows * p.h
        scale_bytes = n // 128 * 4 if p.scale_layout == ScaleLayout.F32_GROUP128 else n // 32
        for r in range(w):
            _check_tensor(x_full[r], n * w, f"x of rank {r}")
            _check_tensor(scale_full[r], scale_bytes * w, f"scales of rank {r}")
            _check_tensor(out_shares[r], n * (4 if p.out_dtype == OutDtype.F32 else 2), f"output of share {r}")
        _check_plan_dtypes(p, x_full, scale_full, out_shares, "x of rank", "scales of rank", "output of share")
        self._plan = p
        self._keep = (list(x_full), list(scale_full), list(out_shares))
        self._xs = (ctypes.c_void_p * w)(*[_ptr(t) for t in x_full])
        self._ss = (ctypes.c_void_p * w)(*[_ptr(t) for t in scale_full])
        self._os = (ctypes.c_void_p * w)(*[_ptr(t) for t in out_shares])
        self._stream = ctypes.c_void_p(_stream_handle(stream))
        self._fn = lib.qrs_run_all_shares
        self._handle = p.handle

    def on_stream(self, stream):
        """The same launch (plan and buffers) enqueued on another stream."""
        return AllSharesLaunch(self._plan, *self._keep, stream=stream)

    def __call__(self):
        status = self._fn(self._handle, self._xs, self._ss, self._os, None, 0, self._stream)
        if status:
            _check(status)


class QuantizeLaunch:
    """``quantize`` with its arguments marshalled once."""

    def __init__(self, x_bf16, x_codes, scales, x_dtype, scale_layout, stream=None):
        lib = load_library()
        tokens, h = x_bf16.shape
        self._xd = int(_enum(x_dtype, _X_NAMES, XDtype))
        self._sl = int(_enum(scale_layout, _SCALE_NAMES, ScaleLayout))
        n = tokens * h
        _check_tensor(x_bf16, 2 * n, "x_bf16")
        _check_tensor(x_codes, n, "x_codes")
        _check_tensor(scales, n // 128 * 4 if self._sl == ScaleLayout.F32_GROUP128 else n // 32, "scales")
        _check_quantize_dtypes(x_bf16, x_codes, scales, self._xd, self._sl)
        self._keep = (x_bf16, x_codes, scales)
        self._args = (tokens, h, self._xd, self._sl, _ptr(x_bf16), _ptr(x_codes), _ptr(scales),
                      ctypes.c_void_p(_stream_handle(stream)))
        self._fn = lib.qrs_quantize

    def on_stream(self, stream):
        """The same launch (mode and buffers) enqueued on another stream."""
        return QuantizeLaunch(*self._keep, self._xd, self._sl, stream=stream)

    def __call__(self):
        status = self._fn(*self._args)
        if status:
            _check(status)


# ---- between two shares -----------------------------------------------------


# The checks below run in front of kernels of a few microseconds: each tensor
# attribute is read once, and messages are made only for refusals.


@functools.lru_cache(maxsize=None)
def _activation_types():
    import torch

    return {torch.float32: int(OutDtype.F32), torch.bfloat16: int(OutDtype.BF16), torch.float16: int(OutDtype.F16)}


def _act_dtype(t, what):
    kind = _activation_types().get(t.dtype)
    if kind is None:
        raise ValueError(f"{what}: float32, bfloat16 or float16 expected, got {t.dtype}")
    return kind


def _matrix(t, what, shape=None, dtype=None):
    """Row stride of a 2-D device view whose elements within a row are
    adjacent, after checking its shape and element type."""
    if not t.is_cuda:
        raise ValueError(f"{what}: device tensors only (there is no CPU path)")
    got = t.shape
    if got != shape if shape is not None else len(got) != 2:
        want = "two dimensions" if shape is None else f"shape {list(shape)}"
        raise ValueError(f"{what}: expected {want}, got {list(got)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    ld, step = t.stride()
    if step != 1 and got[1] > 1:
        raise ValueError(f"{what}: elements within a row must be adjacent")
    return ld if got[0] > 1 else got[1]


def _vector(t, what, n, dtype):
    if not t.is_cuda:
        raise ValueError(f"{what}: device tensors only (there is no CPU path)")
    if t.numel() != n or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous {dtype} elements expected, got {list(t.shape)} {t.dtype}")


@functools.lru_cache(maxsize=None)
def _mode(x_dtype, scale_layout):
    """(x_dtype, scale_layout) as the library's ints, with the element types
    of codes and scales and the scales' group (0: the row)."""
    import torch

    xd, sl = _enum(x_dtype, _X_NAMES, XDtype), _enum(scale_layout, _SCALE_NAMES, ScaleLayout)
    x_dt, s_dt, _ = _element_dtypes()
    group = {ScaleLayout.F32_GROUP128: 128, ScaleLayout.E8M0_BLOCK32: 32}.get(sl, 0)
    return int(xd), int(sl), x_dt.get(xd), s_dt.get(sl, torch.float32), group


def _codes_and_scales(codes, scales, shape, mode):
    """Checks codes and scales of a mode; the codes' row stride."""
    _, _, x_dt, s_dt, group = mode
    ld = _matrix(codes, "codes", shape)
    if codes.dtype != x_dt:
        if codes.element_size() != 1:
            raise ValueError(f"codes: 1-byte elements expected, got {codes.dtype}")
        _check_dtype(codes, x_dt, "codes")
    rows, h = shape
    n = rows * h // group if group else rows
    if group == 32 and scales.dtype != s_dt:  # E8M0 codes also as raw bytes
        _check_tensor(scales, n, "scales")
        _check_dtype(scales, s_dt, "scales")
        _ptr(scales)
    else:
        _vector(scales, "scales", n, s_dt)
    return ld


def _workspace(workspace, nbytes, like, stream):
    """The caller's workspace, or one that torch's allocator gives ``stream``:
    memory that only work of that stream used before and will use next."""
    import torch

    if workspace is not None:
        if isinstance(workspace, int):
            raise ValueError("workspace: a tensor expected, whose size is known")
        return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace
    if stream is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    else:
        if isinstance(stream, int):
            # ExternalStream takes the default stream's handle, 0, for none given and answers with one of its own.
            stream = (torch.cuda.ExternalStream(stream, device=like.device) if stream
                      else torch.cuda.default_stream(like.device))
        with torch.cuda.stream(stream):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return ws.data_ptr(), nbytes, ws


def add_rms_norm_quantize(x, residual, weight, eps, sum_out, codes, scales, x_dtype, scale_layout, stream=None):
    """s = x + residual, y = s / sqrt(mean(s**2) + eps) * weight along each
    row, and y as codes and scales (qrs_add_rms_norm_quantize).

    ``x``, ``residual``, ``sum_out``: ``[tokens, h]`` of one type (float32,
    bfloat16 or float16); ``weight``: ``[h]`` of that type. ``sum_out`` receives
    s and may be ``x`` or ``residual`` itself. With ``residual=None``, s = x and
    ``sum_out`` is not used. ``scale_layout``: "f32_group128", "e8m0_block32",
    or "f32_row" (one scale per token, for ``matmul_int8``)."""
    lib = load_library()
    io = _act_dtype(x, "x")
    ld_x = _matrix(x, "x")
    tokens, h = x.shape
    _vector(weight, "weight", h, x.dtype)
    ld_r = ld_s = 0
    if residual is not None:
        if sum_out is None:
            raise ValueError("sum_out: needed with a residual")
        ld_r = _matrix(residual, "residual", x.shape, x.dtype)
        ld_s = _matrix(sum_out, "sum_out", x.shape, x.dtype)
    mode = _mode(x_dtype, scale_layout)
    ld_c = _codes_and_scales(codes, scales, x.shape, mode)
    _check(lib.qrs_add_rms_norm_quantize(
        tokens, h, io, mode[0], mode[1], eps, x.data_ptr(), ld_x, None if residual is None else residual.data_ptr(),
        ld_r, weight.data_ptr(), None if residual is None else sum_out.data_ptr(), ld_s, codes.data_ptr(), ld_c,
        scales.data_ptr(), _stream_handle(stream)))


def rms_norm_backward(grad_y, sum, weight, eps, grad_sum, grad_x, grad_weight, workspace=None, stream=None):
    """Gradients of ``add_rms_norm_quantize``'s y, with the quantization passed
    through (qrs_rms_norm_backward): ``grad_x`` of s (so of x and of residual
    alike), ``grad_weight`` (float32 ``[h]``).

    ``sum`` is s; ``grad_sum`` the gradient that reaches s by the residual
    stream (None = zero). ``grad_x`` may be ``grad_y`` or ``grad_sum`` itself.
    ``workspace``: device memory of ``rms_norm_backward_workspace`` bytes, by
    default taken from torch's allocator."""
    import torch

    lib = load_library()
    io = _act_dtype(sum, "sum")
    ld_s = _matrix(sum, "sum")
    tokens, h = sum.shape
    ld_y = _matrix(grad_y, "grad_y", sum.shape, sum.dtype)
    ld_g = 0 if grad_sum is None else _matrix(grad_sum, "grad_sum", sum.shape, sum.dtype)
    ld_x = _matrix(grad_x, "grad_x", sum.shape, sum.dtype)
    _vector(weight, "weight", h, sum.dtype)
    _vector(grad_weight, "grad_weight", h, torch.float32)
    need = ctypes.c_size_t()
    _check(lib.qrs_rms_norm_backward_workspace(tokens, h, ctypes.byref(need)))
    ws, nbytes, _keep = _workspace(workspace, need.value, sum, stream)  # _keep: until it is enqueued
    _check(lib.qrs_rms_norm_backward(
        tokens, h, io, eps, grad_y.data_ptr(), ld_y, sum.data_ptr(), ld_s, weight.data_ptr(),
        None if grad_sum is None else grad_sum.data_ptr(), ld_g, grad_x.data_ptr(), ld_x, grad_weight.data_ptr(), ws,
        nbytes, _stream_handle(stream)))


def quantize_rows(x, codes, scales, x_dtype="int8", stream=None):
    """Rows of activations or weights ``[rows, cols]`` (float32, bfloat16 or
    float16) as ``codes`` with one float32 scale per row (qrs_quantize_rows)."""
    lib = load_library()
    kind = _act_dtype(x, "x")
    ld_x = _matrix(x, "x")
    rows, cols = x.shape
    mode = _mode(x_dtype, "f32_row")
    ld_c = _codes_and_scales(codes, scales, x.shape, mode)
    _check(lib.qrs_quantize_rows(rows, cols, kind, mode[0], x.data_ptr(), ld_x, codes.data_ptr(), ld_c,
                                 scales.data_ptr(), _stream_handle(stream)))


@functools.lru_cache(maxsize=None)
def _operand_types():
    import torch

    return torch.int8, torch.float32


def _matmul_operands(a, a_scales, b, b_scales, gated):
    int8, float32 = _operand_types()
    ld_a = _matrix(a, "a", None, int8)
    ld_b = _matrix(b, "b", None, int8)
    m, k = a.shape
    wide, kb = b.shape
    if kb != k or (gated and wide % 2):
        raise ValueError(f"b: expected [{'2 n' if gated else 'n'}, {k}], got {list(b.shape)}")
    _vector(a_scales, "a_scales", m, float32)
    _vector(b_scales, "b_scales", wide, float32)
    return m, wide // 2 if gated else wide, k, ld_a, ld_b


def matmul_int8(a, a_scales, b, b_scales, out, gated=False, stream=None):
    """``out = (a @ b.T) * a_scales[:, None] * b_scales`` of int8 ``a [m, k]``
    (tokens) and ``b [n, k]`` (channels), float32 scales, summed exactly
    (qrs_matmul_int). ``out [m, n]``: float32, bfloat16 or float16.

    ``gated``: ``b`` is ``[2 n, k]``, n gate and then n up channels, and
    ``out = silu(gate product) * up product``."""
    lib = load_library()
    m, n, k, ld_a, ld_b = _matmul_operands(a, a_scales, b, b_scales, gated)
    kind = _act_dtype(out, "out")
    ld_o = _matrix(out, "out", (m, n))
    _check(lib.qrs_matmul_int(m, n, k, 1 if gated else 0, kind, a.data_ptr(), ld_a, a_scales.data_ptr(), b.data_ptr(),
                              ld_b, b_scales.data_ptr(), out.data_ptr(), ld_o, _stream_handle(stream)))


def matmul_int8_quantize(a, a_scales, b, b_scales, codes, scales, x_dtype, scale_layout, stream=None):
    """``matmul_int8``'s product, quantized in float32 into the codes
    ``[m, n]`` and scales that ``run`` and ``run_all_shares`` read
    (qrs_matmul_int_quantize): one rank's partial sums. n is a multiple of 128."""
    lib = load_library()
    m, n, k, ld_a, ld_b = _matmul_operands(a, a_scales, b, b_scales, False)
    mode = _mode(x_dtype, scale_layout)
    ld_c = _codes_and_scales(codes, scales, (m, n), mode)
    _check(lib.qrs_matmul_int_quantize(m, n, k, mode[0], mode[1], a.data_ptr(), ld_a, a_scales.data_ptr(),
                                       b.data_ptr(), ld_b, b_scales.data_ptr(), codes.data_ptr(), ld_c,
                                       scales.data_ptr(), _stream_handle(stream)))


def run_launch_info(p: Plan, stream=None) -> dict:
    """The grid, residency cap and device sizes of the launch ``run`` makes
    for ``p`` on ``stream``'s device (qrs_run_launch_info); launches nothing."""
    lib = load_library()
    info = LaunchInfo()
    _check(lib.qrs_run_launch_info(p.handle, _stream_handle(stream), ctypes.byref(info)))
    return info.as_dict()


def matmul_launch_info(m, n, k, gated=False, scale_layout=None) -> dict:
    """The kernel ("tiles", "few_tokens", "mid" or "pipe"), its tile and its
    grid that ``matmul_int8`` takes for contiguous operands of this shape, or
    ``matmul_int8_quantize`` with a ``scale_layout`` (qrs_matmul_launch_info);
    launches nothing."""
    lib = load_library()
    info = MatmulInfo()
    layout = ScaleLayout.F32_GROUP128 if scale_layout is None else _enum(scale_layout, _SCALE_NAMES, ScaleLayout)
    _check(lib.qrs_matmul_launch_info(m, n, k, 1 if gated else 0, 0 if scale_layout is None else 1, layout,
                                      ctypes.byref(info)))
    return {"kernel": ("tiles", "few_tokens", "mid", "pipe")[info.kernel], "tile": (info.tile_m, info.tile_n),
            "blocks": info.blocks, "threads_per_block": info.threads_per_block}


def stream_copy(src, dst, nbytes=None, stream=None):
    """Calibration copy of ``nbytes`` (default: all of src) from src to dst."""
    lib = load_library()
    if nbytes is None:
        nbytes = src.numel() * src.element_size()
    _check(lib.qrs_stream_copy(_ptr(src), _ptr(dst), int(nbytes), _stream_handle(stream)))
