"""uw_sample on the GPU at the ends of its ranges: long rows in one workgroup, rows of ties and infinities
longer than its list, temperatures that bring the lowest numbers into play. The oracle is that of
test_gpu_sample: a row on the host, masses as whole multiples of 2^-43 of the largest."""
import math

import numpy as np
import pytest

from tests.test_gpu_sample import _compare, _settings, _uw

pytestmark = pytest.mark.gpu

LOWEST = np.finfo(np.float32).min


@pytest.mark.parametrize("M", [4, 150])
def test_lowest_numbers_with_a_share_of_the_mass(M):
    """Temperatures of 10^37 and more, at which tokens of the type's lowest value weigh something, some of them so
    that the lowest value lies right below the upper end of its bin (46 bins per power of two)."""
    uw = _uw()
    rng = np.random.default_rng(17)
    hexes = ["0x1.fef3ep127", "0x1.557dbp127", "0x1.54a296p126", "0x1.543572p125", "0x1.fef3dcp127", "0x1.557daep127"]
    T = [float.fromhex(hexes[m % 6]) if m % 4 != 3 else [1e38, 3e37, math.inf][m % 3] for m in range(M)]
    for low in (3000, 6000):  # the lowest bin fits a list, or does not
        x = np.zeros((M, 13000), np.float32)
        for m in range(M):
            x[m, rng.choice(13000, low, replace=False)] = LOWEST
        for k, p, least in ((0, 1.0, 0.0), (9000, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.2), (0, 1.0, 0.01), (11000, 0.95, 0.04)):
            u = (1 - 0.3 * rng.random(M)).astype(np.float32)
            _compare(uw, x, u, f"{low} {k} {p} {least}", temperature=T, top_k=[k] * M, top_p=[p] * M, min_p=[least] * M)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", [(130, 131072), (200, 50257), (140, 33000)])
def test_long_rows_of_one_workgroup_each(M, V, dtype):
    """More rows than two workgroups each would serve: one workgroup reads a row in several turns, and every
    setting meets every kind of row: peaked, flat, masked to a twentieth, and ties that fill the list."""
    uw = _uw()
    assert uw.sample_workspace(M, V) == 0
    rng = np.random.default_rng(M + V)
    x = rng.standard_normal((M, V)).astype(np.float32)
    x[0::4] = 2 * x[0::4] + np.where(rng.random(x[0::4].shape) < 0.002, 4 + 6 * rng.random(x[0::4].shape), 0).astype(np.float32)
    x[2::4][rng.random(x[2::4].shape) < 0.95] = -np.inf
    x[3::4] = np.round(x[3::4])  # a dozen distinct logits, thousands of each
    u = rng.random(M).astype(np.float32).tolist()
    settings = _settings(rng, M)
    ks = [0, 890, 900, 5000, 1, 50, 0, V - 1, 895, 896, 897]
    settings["top_k"] = [ks[m % len(ks)] for m in range(M)]
    _compare(uw, x, u, f"{M}x{V}", dtype=dtype, **settings)


@pytest.mark.parametrize("M", [3, 140])
def test_lists_that_overflow(M):
    """More equal logits at the top than the list holds (4096): on the row's own histogram, then on the passes
    over the row, for rows shared by workgroups and not."""
    uw = _uw()
    rng = np.random.default_rng(M)
    V = 40000
    x = rng.standard_normal((M, V)).astype(np.float32)
    for m, n in zip(range(M), [4095, 4096, 4097, 5000, 30000] * M):
        x[m, rng.choice(V, n, replace=False)] = 3.0
    u = rng.random(M).astype(np.float32).tolist()
    for k, p, least in ((0, 1.0, 0.0), (300, 1.0, 0.0), (4096, 0.5, 0.0), (6000, 1.0, 0.0), (0, 0.9, 0.1), (0, 1.0, 0.9)):
        _compare(uw, x, u, f"{k} {p} {least}", top_k=[k] * M, top_p=[p] * M, min_p=[least] * M)


@pytest.mark.parametrize("M,V", [(4, 70000), (140, 20000)])
def test_more_infinities_than_the_list_holds(M, V):
    """They share the mass; every filter cuts among them, by index."""
    uw = _uw()
    rng = np.random.default_rng(V)
    x = rng.standard_normal((M, V)).astype(np.float32)
    for m in range(M):
        x[m, rng.choice(V, [5000, 4097, V // 2, V][m % 4], replace=False)] = np.inf
        if m % 4 < 3:
            x[m, rng.choice(V, 100, replace=False)] = np.nan
    u = rng.random(M).astype(np.float32).tolist()
    for T, k, p, least in ((1.0, 0, 1.0, 0.0), (0.5, 100, 0.9, 0.0), (2.0, 4500, 1.0, 0.3), (0.0, 0, 1.0, 0.0), (math.inf, 0, 0.3, 0.0),
                           (1.0, 0, 0.999, 1.0)):
        _compare(uw, x, u, f"{T} {k} {p} {least}", temperature=[T] * M, top_k=[k] * M, top_p=[p] * M, min_p=[least] * M)
