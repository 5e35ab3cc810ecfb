"""The batches that the GPU tests of the layer norm run reach every number of
work-groups that its gradient takes, and every shape with operands beyond the
Infinity Cache as well as within it, on the host."""

import ctypes

import quantized_collective_reduction_amd as qrs

STREAMED = 256 << 20
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _work_groups(t, h):
    n = ctypes.c_size_t()
    assert qrs.load_library().qrs_layer_norm_backward_workspace(t, h, ctypes.byref(n)) == 0
    return n.value // (8 * h)


def _shape(kind, h, limits):
    """Which of the widths, in elements of a row, holds h."""
    return next(limit for limit in limits if h <= limit)


def test_forward_batches_reach_every_shape_streamed():
    from test_gpu_layer_norm_batches import FORWARD

    for wide in (False, True):
        limits = [1024, 2048, 4096, 6144, 8192, 16384, 65536] if wide else [1024, 2048, 4096, 8192, 16384, 65536]
        reached = {_shape(kind, h, limits) for kind, t, h, _ in FORWARD
                   if (kind == "f32") == wide and h % 8 == 0 and t * h * (3 * SIZE[kind] + 1) > STREAMED}
        assert reached == set(limits)


def test_backward_batches_reach_every_shape_and_number_of_work_groups():
    from test_gpu_layer_norm import BACK_SHAPES
    from test_gpu_layer_norm_batches import BACKWARD

    for wide in (False, True):
        limits = [1024, 2048, 4096, 8192, 16384, 65536]
        cases = [(kind, t, h) for kind, t, h in BACKWARD if (kind == "f32") == wide]
        streamed = {_shape(kind, h, limits) for kind, t, h in cases if h % 8 == 0 and t * h * 4 * SIZE[kind] > STREAMED}
        assert streamed == set(limits)
        assert {_work_groups(t, h) for _, t, h in cases} == {256, 512, 1024}
        # More than two thousand rows, of each width that has a rule of its own.
        for most, least in [(2048, 0), (8192, 2048), (65536, 8192)]:
            assert any(least < h <= most and t > 1000 for _, t, h in cases)
    assert {_work_groups(t, h) for t, h in BACK_SHAPES} >= {1, 256, 512}
    # Binary32 takes 256 where the workspace holds more.
    assert any(kind == "f32" and 2048 < h <= 8192 and _work_groups(t, h) == 512 for kind, t, h in BACKWARD)
