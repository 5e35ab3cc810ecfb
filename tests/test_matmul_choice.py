"""Which kernel a product takes, on the host: every accepted shape has one whose
grid a launch holds, and the shapes of the GPU tests reach the kernels that they
are there for."""

import ctypes

import pytest

import quantized_collective_reduction_amd as qrs

FORMS = [dict(), dict(gated=True), dict(scale_layout="f32_group128"), dict(scale_layout="e8m0_block32")]


def _ids(form):
    return "-".join(f"{k}={v}" for k, v in form.items()) or "values"


@pytest.mark.parametrize("form", FORMS, ids=_ids)
@pytest.mark.parametrize("k", [16, 128, 144, 8192, 17])
def test_every_accepted_shape_has_a_grid_that_a_launch_holds(form, k):
    step = 128 if "scale_layout" in form else 1
    limit = (1 << 24) - 1  # 64 x 64 tiles
    sizes = sorted({min(max(v + d, 1), (1 << 30) - 64) for e in range(0, 31) for d in (-1, 0, 1) for v in (1 << e,)})
    seen = set()
    for m in sizes:
        # n at the edges of what is accepted beside this m, and below.
        most = limit // -(-m // 64) * 64
        for n in {most, most // 2, most // 3, 4096, 33, 1}:
            n = n // step * step
            if n < 1 or -(-m // 64) * -(-n // 64) > limit:
                continue
            info = qrs.matmul_launch_info(m, n, k, **form)
            assert 0 < info["blocks"] * info["threads_per_block"] < 1 << 32, (m, n, info)
            tile_m, tile_n = info["tile"]
            if form.get("gated"):
                tile_n //= 2
            if info["kernel"] == "pipe":
                assert info["blocks"] == 256  # work-groups walk over the tiles
            else:
                assert info["blocks"] == -(-m // tile_m) * -(-n // tile_n), (m, n, info)
            seen.add(info["kernel"])
    assert "tiles" in seen and (k % 16 != 0 or {"few_tokens", "mid"} <= seen)


def test_the_documented_limit_is_refused():
    for m, n in [(1 << 30, 1), (1, 1 << 30), (1 << 17, 1 << 19), ((1 << 24) * 64, 64)]:
        with pytest.raises(qrs.QrsError, match="too large"):
            qrs.matmul_launch_info(m, n, 16)
        assert qrs.matmul_launch_info(m - 64 if m > n else m, n if m > n else n - 64, 16)["blocks"] > 0


def test_refusals():
    lib = qrs.load_library()
    info = qrs.MatmulInfo()
    for args, text in [((0, 1, 16, 0, 0, 0), "positive"), ((1, 1, 16, 2, 0, 0), "gated"), ((1, 1, 16, 0, 2, 0), "quantize"),
                       ((1, 128, 16, 1, 1, 0), "gated"), ((1, 100, 16, 0, 1, 1), "multiple of 128"),
                       ((1, 128, 16, 0, 1, 2), "scale_layout"), ((1, 128, 131072, 0, 0, 0), "131071")]:
        assert lib.qrs_matmul_launch_info(*args, ctypes.byref(info)) == int(qrs.Status.INVALID_ARG), args
        assert text in lib.qrs_last_error().decode(), args
    assert lib.qrs_matmul_launch_info(1, 1, 16, 0, 0, 0, None) == int(qrs.Status.INVALID_ARG)
