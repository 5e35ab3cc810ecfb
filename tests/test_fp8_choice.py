"""Which kernel an 8-bit floating-point product takes, on the host: every accepted
shape has one whose grid a launch holds, and the shapes of the GPU tests reach all
of them."""

import pytest

import quantized_collective_reduction_amd as qrs

FORMS = [dict(), dict(out_dtype="bf16"), dict(gated=True), dict(gated=True, out_dtype="f16"), dict(b_scale_rows=1),
         dict(b_scale_rows=1, out_dtype="bf16"), dict(scale_layout="f32_group128"),
         dict(scale_layout="e8m0_block32"), dict(gated=True, scale_layout="f32_group128"),
         dict(gated=True, scale_layout="e8m0_block32")]


def _ids(form):
    return "-".join(f"{k}={v}" for k, v in form.items()) or "values"


@pytest.mark.parametrize("form", FORMS, ids=_ids)
@pytest.mark.parametrize("k", [16, 128, 144, 8192, 17, 1 << 20])
def test_every_accepted_shape_has_a_grid_that_a_launch_holds(form, k):
    step = 128 if "scale_layout" in form else 1
    limit = (1 << 24) - 1  # 64 x 64 tiles
    for m in sorted({min(max((1 << e) + d, 1), (1 << 30) - 64) for e in range(0, 31) for d in (-1, 0, 1)}):
        most = limit // -(-m // 64) * 64
        for n in {most, most // 2, most // 3, 4096, 33, 1}:
            n = n // step * step
            if n < 1 or -(-m // 64) * -(-n // 64) > limit:
                continue
            info = qrs.matmul_fp8_launch_info(m, n, k, **form)
            assert 0 < info["blocks"] * info["threads_per_block"] < 1 << 32, (m, n, info)
            tile_m, rows = info["tile"]
            outputs = rows // 2 if form.get("gated") else rows
            if info["kernel"] != "pipe":  # whose work-groups walk over the tiles
                assert info["blocks"] == -(-m // tile_m) * -(-n // outputs), (m, n, info)
            if form.get("scale_layout") == "f32_group128" and info["kernel"] != "few_tokens":
                assert outputs % 128 == 0
            if form.get("scale_layout") == "e8m0_block32" and not (info["kernel"] == "few_tokens" and form.get("gated")):
                assert outputs % 32 == 0


def test_the_gpu_tests_reach_every_kernel():
    from test_gpu_matmul_fp8 import CODE_SIZES, GATED, SIZES
    from test_gpu_matmul_fp8_tiles import MID, PIPE

    def kernels(sizes, **form):
        return {(info["kernel"], info["tile"]) for m, n, k in sizes
                for info in [qrs.matmul_fp8_launch_info(m, n, k, **form)]}

    few = {("few_tokens", t) for t in [(8, 16), (16, 16), (32, 32)]}
    pipe = ("pipe", (256, 256))
    mid = {("mid", t) for t in [(64, 32), (64, 64), (64, 128), (128, 128)]}
    wide = ("mid", (128, 256))  # of 16-bit outputs, with scales of 128 rows of b
    sizes = SIZES + MID + PIPE
    halves = GATED + [(m, n // 2, k) for m, n, k in MID + PIPE]
    for out in ("f32", "bf16", "f16"):
        more = {wide} if out != "f32" else set()
        assert few | mid | {pipe} | more <= kernels(sizes, out_dtype=out)
        assert few | mid | {pipe} <= kernels(sizes, b_scale_rows=1, out_dtype=out)
        assert few | mid | {pipe} | more <= kernels(halves, gated=True, out_dtype=out)
    assert kernels([(66, 65, 100)]) == {("tiles", (64, 128))}
    assert kernels([(66, 65, 100)], gated=True) == {("tiles", (64, 256))}
    large = CODE_SIZES + [(4096, 4096, 160), (4100, 8192, 272), (300, 4096, 400), (1000, 1024, 400)]
    assert few | {("mid", (64, 128)), ("mid", (128, 128)), pipe} <= kernels(large, scale_layout="f32_group128")
    few_codes = {("few_tokens", t) for t in [(8, 32), (16, 32), (32, 32)]}
    assert few_codes | mid | {pipe} <= kernels(large, scale_layout="e8m0_block32")
    large = CODE_SIZES + [(4096, 2048, 160), (4100, 4096, 272), (300, 2048, 400), (1000, 512, 400)]
    assert few | {("mid", (64, 256)), pipe} <= kernels(large, scale_layout="f32_group128", gated=True)
    assert few | mid - {("mid", (64, 32))} | {pipe} <= kernels(large, scale_layout="e8m0_block32", gated=True)
