"""The built library holds no instance of a kernel that no call takes: the names of
its kernels, as it registers them, against the shapes and forms that the launches
choose from."""

import re

import quantized_collective_reduction_amd as qrs

F32, BF16, F16 = 0, 1, 2
PLAIN, GATED, GROUPED = 0, 1, 2


def _instances(kernel):
    """Template arguments of every instance: enums, numbers and truth values alike."""
    with open(qrs.LIB_PATH, "rb") as f:
        held = f.read()
    found = set()
    for args in re.findall(rb"_ZN3qrs12_GLOBAL__N_1%d%sI((?:L[A-Za-z0-9_]*?E)+)E" % (len(kernel), kernel.encode()), held):
        found.add(tuple(int(v.replace("n", "-")) for v in re.findall(r"(?:Lb|Li|LNS_7XFormatE|LS\d*_)(n?\d+)E", args.decode())))
    assert found
    return found


def test_tiles_of_the_8_bit_floating_point_product():
    both = {False, True}
    # Tokens, rows of b: the forms, and whether codes are widened.
    want = {(64, 32): ({PLAIN, GATED, GROUPED}, both), (64, 64): ({PLAIN, GATED, GROUPED}, both),
            (64, 128): ({PLAIN, GATED, GROUPED}, both), (128, 128): ({PLAIN, GATED, GROUPED}, both),
            (128, 256): ({PLAIN, GATED}, {False}),  # 16-bit outputs
            (64, 256): ({GATED}, {True})}  # codes with a scale for each 128 outputs
    want = {(a, b, *tile, form, wide) for tile, (forms, ways) in want.items() for form in forms for wide in ways
            for a in (1, 2) for b in (1, 2)}
    got = {(i[0], i[1], i[2], i[3], i[7], bool(i[8])) for i in _instances("mid_kernel") if len(i) == 9}
    assert got == want


def test_shapes_of_the_layer_norm():
    aligned = {(128, 1), (128, 2), (256, 2), (512, 2), (1024, 2), (1024, 8)}
    want = {(io, sl, *shape, True, stream) for io in (F32, BF16, F16) for sl in range(3) for stream in (False, True)
            for shape in aligned | ({(768, 1)} if io == F32 else set())}
    want |= {(io, sl, *shape, False, False) for io in (F32, BF16, F16) for sl in range(3) for shape in [(512, 2), (1024, 8)]}
    assert {(*i[:4], bool(i[4]), bool(i[5])) for i in _instances("layer_norm_kernel")} == want


def test_shapes_of_the_layer_norms_gradient():
    aligned = {(128, 1), (128, 2), (256, 2), (512, 4), (1024, 8)}
    want = {(io, *shape, True, stream) for io in (F32, BF16, F16) for stream in (False, True)
            for shape in aligned | ({(512, 2)} if io == F32 else {(256, 4)})}
    want |= {(io, *shape, False, False) for io in (F32, BF16, F16) for shape in [(256, 4), (1024, 8)]}
    assert {(*i[:3], bool(i[3]), bool(i[4])) for i in _instances("layer_norm_backward_kernel")} == want
