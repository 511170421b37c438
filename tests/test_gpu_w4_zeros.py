"""4-bit products: what has to come out exactly.

  zeros      a group whose codes are all its zero point stands for zeros and adds nothing: rows of W of such groups give 0, and
             beside others the outputs are, bit for bit, those of X with 0 in the group's places
  one value  a row of X with a single 1 makes every sum on the way exact (1 + q / 16, 1, their difference and its product with a
             scale of 20 bits), so Y is the plane's value as w4_expand gives it in fp32: a weight or scale rounded on
             the way would show. h of gate and up has exact products, so silu's and its product's 8 * 2^-24 and the rounding to
             bf16, 2^-8, are all that it is off by.
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda
from tests.test_gpu_w4 import _up, _weights, bf16, plane_of, put_plane, quantized, upload, values_of

pytestmark = pytest.mark.gpu

# every number of rows of X per workgroup (1, 4, 16, 32, 64), of row tiles (1, 2, 4), with and without K slices, K inside a tile
SIZES = [(1, 40, 1000), (3, 100, 520), (9, 64, 640), (16, 2500, 256), (12, 12400, 256), (20, 64, 700), (32, 5000, 300), (40, 3000, 256), (64, 12300, 128),
         (48, 96, 6200), (130, 1700, 256), (700, 1300, 200)]


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def _products(plane, up, d_x, M, N, K, group):
    """Y (fp32), with K slices where the size has them and without, and h of the two planes."""
    torch, uw = torch_cuda(), _uw()
    out = []
    for need in sorted({0, uw.w4_gemm_workspace(M, N, K)}):
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
        y = torch.full((M, N), 77.0, device="cuda")
        uw.w4_gemm(d_x, plane, y, M, N, K, group=group, ldx=d_x.stride(0), d_ws=ws, ws_bytes=need)
        out.append(y)
    h = torch.full((M, N), 77.0, dtype=torch.bfloat16, device="cuda")
    uw.w4_gate_up(d_x, plane, up, h, M, N, K, group=group, ldx=d_x.stride(0))
    return out, h


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (64, 5), (128, False), (128, True), (128, 15), (32, 16), (64, 16), (128, 16)])
@pytest.mark.parametrize("M,N,K", SIZES + [(1, 1, 1000), (64, 2, 4000), (5, 1, 6000)])
def test_groups_of_zeros_add_nothing(M, N, K, group, zeros):
    """zeros: whether w4_quantize's planes have zero points; in a caller's own plane the one zero point, or 16 for any."""
    torch = torch_cuda()
    rng = np.random.default_rng(M + N + K + group)
    x = bf16(rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 20, 1))
    w = 1e-3 * _weights(rng, N, K)
    w[::5] = 0  # rows of zeros
    G = -(-K // group)
    gone = rng.random(G) < 0.4
    gone[0] = True
    columns = np.repeat(gone, group)[:K]
    w[:, columns] = 0
    log(f"  zeros {M}x{N}x{K} group {group} zeros {zeros}")
    q, s, z = quantized(w, group, zeros is True)  # groups of zeros have the scale 1
    empty = (q == z[..., None]).all(2)
    assert empty[:, gone].all() and (s[empty] == 1).all()
    if zeros and zeros is not True:
        z[:] = zeros if zeros < 16 else rng.integers(0, 16, z.shape)
        q = np.where(empty[..., None], z[..., None], q)
        s[empty] = np.ldexp(1.0, rng.integers(-20, 20, empty.sum()))
        q.reshape(N, -1)[:, K:] = 0
    plane = put_plane(plane_of(q, s, z, N, K, group))
    ys, h = _products(plane, plane, upload(x, torch.bfloat16, _up(K, 8)), M, N, K, group)
    cleared, h_cleared = _products(plane, plane, upload(np.where(columns, 0, x), torch.bfloat16, _up(K, 8)), M, N, K, group)
    for y, c in zip(ys, cleared):
        assert (y[:, ::5] == 0).all()
        assert torch.equal(y, c)
    assert (h[:, ::5] == 0).all() and torch.equal(h, h_cleared)


@pytest.mark.parametrize("M", [3, 16, 64])
def test_groups_of_zeros_keep_what_is_not_finite(M):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M)
    N, K, group = 48, 512, 128
    w = _weights(rng, N, K)
    w[:, :256] = 0
    q, s, z = quantized(w, group, False)
    s[5, 1], s[20, 3] = np.nan, np.nan  # as of groups with a NaN, all codes alike
    q[[5, 20], [1, 3]], z[[5, 20], [1, 3]] = 0, 0
    w[7] = w[21] = 0
    q[[7, 21]], s[[7, 21]], z[[7, 21]] = 8, 1, 8
    x = bf16(rng.standard_normal((M, K)))
    x[1, 3], x[2, 200] = np.inf, np.nan
    y = torch.zeros(M, N, device="cuda")
    uw.w4_gemm(upload(x, torch.bfloat16), put_plane(plane_of(q, s, z, N, K, group)), y, M, N, K, group=group)
    bad = np.isnan(y.cpu().numpy())
    assert bad[1:3].all() and bad[:, [5, 20]].all() and bad.sum() == 2 * N + 2 * (M - 2)
    assert (y[0, [7, 21]] == 0).all() and (y[3:, [7, 21]] == 0).all()


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_one_value_gives_the_weight_itself(M, N, K, group, zeros):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M * 3 + N + K + group)
    x = np.zeros((M, K), np.float32)
    at = rng.integers(0, K, M)
    at[-1] = K - 1
    x[np.arange(M), at] = 1
    planes, values = [], []
    for _ in range(2):
        q, s, z = quantized(30 * _weights(rng, N, K), group, zeros)
        planes.append(put_plane(plane_of(q, s, z, N, K, group)))
        v = torch.zeros(N, _up(K, 8), device="cuda")
        uw.w4_expand(planes[-1], v, N, K, group=group, ldw=_up(K, 8))
        values.append(v.cpu().numpy()[:, at].T)
        assert (values[-1] == values_of(q, s, z, K)[:, at].T).all()
    log(f"  one value {M}x{N}x{K} group {group} zeros {zeros}")
    ys, h = _products(*planes, upload(x, torch.bfloat16, _up(K, 8)), M, N, K, group)
    for y in ys:
        assert (y.cpu().numpy() == values[0]).all()
    g, u = (v.astype(np.float64) for v in values)
    want = g / (1 + np.exp(-g)) * u
    assert (np.abs(h.double().cpu().numpy() - want) <= np.abs(want) * (2.0**-8 + 8 * 2.0**-24) + 2.0**-133).all()
