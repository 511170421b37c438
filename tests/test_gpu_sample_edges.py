"""uw_sample on the GPU at the ends of its ranges: long rows in one workgroup, rows of ties and infinities
longer than its list, temperatures that bring the lowest numbers into play. The oracle is that of
test_gpu_sample: a row on the host, masses as whole multiples of 2^-43 of the largest."""
import math

import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda
from tests.test_gpu_sample import _compare, _draw, _settings, _uw

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
