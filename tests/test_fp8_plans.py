"""What the 8-bit product is planned to do, on the host: every kernel shape is taken by sizes that the GPU
tests run, in one K slice and in several, with K a multiple of 128 and not. A change of the time model's
constants that moves a size to another shape shows here, and the list gets another size."""
import pytest

import decode_gemm_amd as uw

SKINNY = [(16, 16), (32, 16), (32, 32), (32, 64)]
TILES = {"f32": [(128, 32), (128, 64), (128, 128), (256, 128)], "bf16": [(128, 32), (128, 64), (128, 128), (256, 128), (256, 256)]}
TYPES = {"f32": uw.F32, "bf16": uw.BF16}

# type of Y, tile (rows of W, rows of X), K slices, M, N, K; cut where the whole workspace is given, else without any
PLANS = [
    ("f32", (16, 16), 1, 1, 1, 512),
    ("f32", (16, 16), 1, 1, 1, 386),
    ("f32", (16, 16), 16, 1, 1, 8192),
    ("f32", (16, 16), 16, 1, 1, 8076),
    ("f32", (32, 16), 1, 357, 343, 1664),
    ("f32", (32, 16), 1, 333, 380, 1561),
    ("f32", (32, 16), 6, 104, 191, 12928),
    ("f32", (32, 16), 6, 100, 183, 12518),
    ("f32", (32, 32), 1, 426, 451, 512),
    ("f32", (32, 32), 1, 438, 459, 390),
    ("f32", (32, 32), 8, 135, 164, 9984),
    ("f32", (32, 32), 12, 121, 152, 10670),
    ("f32", (32, 64), 1, 598, 424, 512),
    ("f32", (32, 64), 1, 407, 632, 385),
    ("f32", (32, 64), 16, 146, 136, 9600),
    ("f32", (32, 64), 16, 165, 115, 9381),
    ("f32", (128, 32), 1, 725, 677, 512),
    ("f32", (128, 32), 1, 629, 807, 389),
    ("f32", (128, 32), 12, 214, 331, 7424),
    ("f32", (128, 32), 12, 193, 332, 7450),
    ("f32", (128, 64), 1, 1097, 910, 512),
    ("f32", (128, 64), 1, 844, 1155, 389),
    ("f32", (128, 64), 16, 225, 323, 8192),
    ("f32", (128, 64), 16, 262, 281, 9468),
    ("f32", (128, 128), 1, 1412, 1414, 512),
    ("f32", (128, 128), 1, 1840, 1041, 393),
    ("f32", (128, 128), 8, 385, 772, 6912),
    ("f32", (128, 128), 8, 992, 264, 6676),
    ("f32", (256, 128), 1, 3269, 1798, 512),
    ("f32", (256, 128), 1, 2729, 2191, 387),
    ("f32", (256, 128), 3, 1808, 1054, 3712),
    ("f32", (256, 128), 3, 1696, 1178, 3767),
    ("bf16", (16, 16), 1, 1, 1, 512),
    ("bf16", (16, 16), 1, 1, 1, 389),
    ("bf16", (16, 16), 16, 1, 1, 8192),
    ("bf16", (16, 16), 16, 1, 1, 8082),
    ("bf16", (32, 16), 1, 326, 380, 1792),
    ("bf16", (32, 16), 1, 366, 341, 1539),
    ("bf16", (32, 16), 6, 97, 187, 11392),
    ("bf16", (32, 16), 6, 111, 189, 12943),
    ("bf16", (32, 32), 1, 423, 449, 512),
    ("bf16", (32, 32), 1, 644, 299, 385),
    ("bf16", (32, 32), 12, 114, 142, 12032),
    ("bf16", (32, 32), 12, 168, 83, 11742),
    ("bf16", (32, 64), 1, 564, 449, 512),
    ("bf16", (32, 64), 1, 646, 423, 386),
    ("bf16", (32, 64), 16, 133, 147, 9472),
    ("bf16", (32, 64), 16, 145, 130, 9776),
    ("bf16", (128, 32), 1, 592, 815, 512),
    ("bf16", (128, 32), 1, 844, 605, 400),
    ("bf16", (128, 32), 16, 148, 174, 9344),
    ("bf16", (128, 32), 16, 149, 168, 9518),
    ("bf16", (128, 64), 1, 812, 1167, 512),
    ("bf16", (128, 64), 1, 1185, 771, 394),
    ("bf16", (128, 64), 8, 475, 278, 4736),
    ("bf16", (128, 64), 8, 327, 407, 4846),
    ("bf16", (128, 128), 1, 1384, 1427, 512),
    ("bf16", (128, 128), 1, 1185, 1665, 391),
    ("bf16", (128, 128), 16, 1402, 35, 9472),
    ("bf16", (128, 128), 16, 1384, 35, 9271),
    ("bf16", (256, 128), 1, 2985, 1315, 896),
    ("bf16", (256, 128), 1, 2958, 1290, 778),
    ("bf16", (256, 128), 3, 2059, 924, 5760),
    ("bf16", (256, 128), 3, 2738, 663, 5749),
    ("bf16", (256, 256), 1, 3862, 3076, 512),
    ("bf16", (256, 256), 1, 1667, 7090, 428),
    ("bf16", (256, 256), 3, 2831, 1426, 8192),
    ("bf16", (256, 256), 3, 1654, 2485, 8348),
]


def plan_of(y, M, N, K, slices):
    return uw.fp8_gemm_plan(M, N, K, TYPES[y], uw.fp8_gemm_workspace(M, N, K) if slices > 1 else 0)


def test_every_shape_is_planned_in_every_way():
    """On a device of 256 compute units, which is what the library assumes where there is none."""
    for y, tile, slices, M, N, K in PLANS:
        p = plan_of(y, M, N, K, slices)
        assert ((p.tile_n, p.tile_m), p.slices) == (tile, slices), (y, M, N, K)
        assert p.exact == (y == "f32" or tile in SKINNY)
    have = {(y, tile, slices > 1, K % 128 > 0) for y, tile, slices, _, _, K in PLANS}
    want = {(y, t, cut, ragged) for y in TYPES for t in SKINNY + TILES[y] for cut in (False, True) for ragged in (False, True)}
    assert have == want


def test_workspace_and_plan_agree():
    """The workspace is what the slices' partial sums take; with fewer bytes fewer slices, and no more than fit."""
    for y, _, slices, M, N, K in PLANS:
        if slices == 1:
            continue
        need = uw.fp8_gemm_workspace(M, N, K)
        of = lambda s: s * M * ((N + 3) // 4 * 4) * 4 if s > 1 else 0
        assert need == max(of(uw.fp8_gemm_plan(M, N, K, t, 1 << 40).slices) for t in TYPES.values())
        for given in (0, need // 4, need // 2, need - 1, need):
            assert of(uw.fp8_gemm_plan(M, N, K, TYPES[y], given).slices) <= given
        assert uw.fp8_gemm_plan(M, N, K, TYPES[y], need).slices == uw.fp8_gemm_plan(M, N, K, TYPES[y], 1 << 40).slices == slices


def test_plan_refusals():
    for args, status in (((-1, 4, 4, 0), uw.ESHAPE), ((4, 0, 4, 0), uw.ESHAPE), ((4, 4, 0, 1), uw.ESHAPE), ((4, 4, 4, 2), uw.EINVAL),
                         ((1 << 31, 4, 4, 0), uw.EUNSUPPORTED), ((1 << 30, 16, 16, 0), uw.EUNSUPPORTED)):
        with pytest.raises(uw.UwError) as e:
            uw.fp8_gemm_plan(*args)
        assert e.value.status == status
    assert uw.lib.uw_fp8_gemm_plan(4, 4, 4, 0, 0, None) == uw.EINVAL
    p = uw.fp8_gemm_plan(0, 4, 4, uw.F32)
    assert (p.tile_n, p.tile_m, p.slices, p.exact) == (0, 0, 0, 0)
