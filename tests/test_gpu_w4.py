"""4-bit weights on the GPU against their definition in 64 bits.

  plane    codes, scales and zero points by the definition in fp64, laid out as the header file says: equal
  values   s (q - z) is exact in fp32: equal; bf16 one rounding of it: equal
  product  where X and the scales are small whole numbers and powers of two every sum is exact: equal. Else, per
           output, the matrix unit's sums of a group may cut a whole step (2^-23) per addition, of terms that
           reach 2 |x| for D and, times 1 + z / 16 < 2, for S, all in units of 16 s: with A = sum of 16 s |x| it is
           (4 group + 2) 2^-23 A, and each addition of groups and waves half a step more: (groups + 20) 2^-24 A. bf16
           outputs add 2^-8 of the value. silu and its product add 8 * 2^-24 of the value to the products' own error, which
           silu passes on at most 1.1 times
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def _up(n, m):
    return (n + m - 1) // m * m


def round20(v):
    m, e = np.frexp(v)
    return np.ldexp(np.rint(m * 2.0**20), e - 20)


def quantized(w, group, zeros):
    """Codes [N][groups][group], scales and zero points [N][groups] of w (fp32), by the definition."""
    N, K = w.shape
    g = np.zeros((N, _up(K, group)))
    g[:, :K] = w
    g = g.reshape(N, -1, group)
    bad = ~np.isfinite(g).all(2)
    g = np.where(bad[..., None], 0.0, g)
    if zeros:
        lo, hi = np.minimum(g.min(2), 0), np.maximum(g.max(2), 0)
        s = np.where(hi > lo, np.maximum(round20((hi - lo) / 15.0), 2.0**-126), 1.0)
        z = np.minimum(np.rint(-lo / s), 15)
    else:
        a = np.abs(g).max(2)
        s = np.where(a > 0, np.maximum(round20(a / 7.0), 2.0**-126), 1.0)
        z = np.full_like(s, 8)
    q = np.clip(np.rint(g / s[..., None]) + z[..., None], 0, 15)
    q, z, s = np.where(bad[..., None], 0, q), np.where(bad, 0, z), np.where(bad, np.nan, s)
    return q.astype(np.int64), s.astype(np.float32), z.astype(np.int64)


def plane_of(q, s, z, N, K, group):
    """The plane's 32-bit words from codes, scales and zero points, value by value of the layout's words."""
    T, J, per = -(-N // 16), -(-K // 128), 128 // group
    codes = np.zeros((T * 16, J * 128), np.int64)
    flat = q.reshape(N, -1)[:, :K]
    codes[:N, :K] = flat
    words = np.zeros(T * J * 256, np.uint32)
    n, k = np.meshgrid(np.arange(T * 16), np.arange(J * 128), indexing="ij")
    at = (n // 16 * J + k // 128) * 256 + 4 * (16 * (k % 32 // 8) + n % 16) + k % 128 // 32
    np.bitwise_or.at(words, at, (codes << (4 * (k % 8 // 2) + 16 * (k % 2))).astype(np.uint32))
    meta = np.zeros((T, J, per, 16), np.uint32)
    for g in range(s.shape[1]):
        bits = np.where(np.isnan(s[:, g]), np.uint32(0x7FC00000), s[:, g].view(np.uint32)) | z[:, g].astype(np.uint32)
        for i in range(N):
            meta[i // 16, g // per, g % per, i % 16] = bits[i]
    return np.concatenate([words, meta.reshape(-1)])


def values_of(q, s, z, K):
    with np.errstate(invalid="ignore"):
        return ((q - z[..., None]) * s[..., None].astype(np.float64)).reshape(q.shape[0], -1)[:, :K]


def upload(a, dtype=None, ld=None, fill=float("nan")):
    """Rows of a on the GPU, ld apart, with `fill` behind them."""
    torch = torch_cuda()
    t = torch.full((a.shape[0], ld or a.shape[1]), fill, dtype=dtype or torch.float32, device="cuda")
    t[:, :a.shape[1]] = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return t


def put_plane(words):
    torch = torch_cuda()
    return torch.from_numpy(words.view(np.int32)).to("cuda")


def bf16(a):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).float().numpy()


def _weights(rng, N, K):
    w = 0.02 * rng.standard_normal((N, K)) * np.exp(0.3 * rng.standard_normal((N, 1)))
    w[rng.random((N, K)) < 0.03] = 0
    return w.astype(np.float32)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(1, 1), (16, 128), (17, 129), (5, 40), (33, 1000), (130, 333)])
def test_quantize_and_expand(group, zeros, dtype, N, K):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(N * 1000 + K + group + 7 * zeros)
    w = _weights(rng, N, K)
    # kinds of groups: zeros, one sign, tiny, huge, and exact ties between codes
    w[0, :] = np.abs(w[0, :])
    if N > 4:
        w[1, :] = 0
        w[2, :] = -np.abs(w[2, :]) * np.float32(1e30)
        w[3, :] = bf16(w[3, :] * np.float32(2.0**-125))
        w[4, :] = np.resize(np.array([7, -7, 0.5, 1.5, 2.5, -0.5, -3.5, 6.5], np.float32), K)
    if dtype == "bf16":
        w = bf16(w)
    log(f"  quantize {N}x{K} group {group} zeros {zeros} {dtype}")
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    ld = _up(K, 8) + 8
    plane = torch.full((uw.w4_plane_bytes(N, K, group) // 4 + 16,), -1, dtype=torch.int32, device="cuda")
    uw.w4_quantize(upload(w, td, ld), plane, N, K, group=group, zeros=zeros, ldw=ld)
    q, s, z = quantized(w, group, zeros)
    want = plane_of(q, s, z, N, K, group)
    got = plane.cpu().numpy().view(np.uint32)
    assert (got[-16:] == 0xFFFFFFFF).all(), "past the plane"
    assert (got[:-16] == want).all(), np.flatnonzero(got[:-16] != want)[:10]
    for out in (torch.float32, torch.bfloat16):
        back = torch.full((N, ld), 77.0, dtype=out, device="cuda")
        uw.w4_expand(plane, back, N, K, group=group, ldw=ld)
        assert (back[:, K:] == 77).all()
        v = torch.from_numpy(values_of(q, s, z, K)).to(out)
        assert torch.equal(back[:, :K].cpu(), v)


def test_quantize_what_is_not_finite():
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(5)
    N, K = 20, 300
    w = _weights(rng, N, K)
    w[3, 40], w[4, 299], w[19, 0] = np.nan, np.inf, -np.inf
    for group in (32, 128):
        for zeros in (False, True):
            plane = torch.zeros(uw.w4_plane_bytes(N, K, group) // 4, dtype=torch.int32, device="cuda")
            uw.w4_quantize(upload(w, ld=300), plane, N, K, group=group, zeros=zeros)
            back = torch.zeros(N, K, device="cuda")
            uw.w4_expand(plane, back, N, K, group=group)
            q, s, z = quantized(w, group, zeros)
            assert (plane.cpu().numpy().view(np.uint32) == plane_of(q, s, z, N, K, group)).all()
            v = values_of(q, s, z, K)
            b = back.cpu().numpy()
            assert (np.isnan(b) == np.isnan(v)).all() and np.isnan(b[3]).sum() == group
            assert (b[~np.isnan(v)] == v[~np.isnan(v)]).all()
            # and a product's outputs are NaN in those columns only
            x = torch.ones(2, _up(K, 8), dtype=torch.bfloat16, device="cuda")
            y = torch.zeros(2, N, device="cuda")
            uw.w4_gemm(x, plane, y, 2, N, K, group=group, ldx=_up(K, 8))
            bad = np.isnan(y.cpu().numpy())
            assert bad[:, [3, 4, 19]].all() and bad.sum() == 6


def _whole(rng, M, N, K, group, zeros):
    """X of whole numbers, codes, power-of-two scales: all sums are whole multiples of 2^-6 below 2^17."""
    x = rng.integers(-4, 5, (M, K)).astype(np.float32)
    G = -(-K // group)
    q = rng.integers(0, 16, (N, G, group))
    q.reshape(N, -1)[:, K:] = 0
    s = np.ldexp(np.float32(1), rng.integers(-2, 1, (N, G))).astype(np.float32)
    z = rng.integers(0, 16, (N, G)) if zeros else np.full((N, G), 8)
    return x, q, s, z


SIZES = [(1, 16, 128), (1, 1, 1), (2, 40, 72), (3, 333, 1000), (4, 96, 2048), (5, 17, 129), (16, 100, 640), (17, 48, 384),
         (31, 130, 1000), (33, 64, 256), (64, 200, 520), (65, 35, 300), (130, 50, 136), (1, 500, 4096), (7, 64, 5000)]


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gemm_of_whole_numbers_is_exact(M, N, K, group, zeros):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M * 7 + N * 3 + K + group)
    x, q, s, z = _whole(rng, M, N, K, group, zeros)
    want = x.astype(np.float64) @ values_of(q, s, z, K).T
    plane, ldx, ldy = put_plane(plane_of(q, s, z, N, K, group)), _up(K, 8) + 8, N + 3
    log(f"  gemm {M}x{N}x{K} group {group} zeros {zeros}")
    d_x = upload(x, torch.bfloat16, ldx)
    need = uw.w4_gemm_workspace(M, N, K)
    for ws_bytes in {0, need}:
        for out in (torch.float32, torch.bfloat16):
            ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
            y = torch.full((M + 1, ldy), 77.0, dtype=out, device="cuda")
            uw.w4_gemm(d_x, plane, y, M, N, K, group=group, ldx=ldx, ldy=ldy, d_ws=ws, ws_bytes=ws_bytes)
            assert (y[M:] == 77).all() and (y[:, N:] == 77).all(), "outside M x N"
            assert torch.equal(y[:M, :N].cpu(), torch.from_numpy(want).to(out))


@pytest.mark.parametrize("M,N,K,group", [(17, 40, 6144, 128), (33, 100, 6500, 32), (64, 96, 14336, 128), (64, 4096, 6300, 64), (130, 33, 25000, 128)])
def test_products_in_slices(M, N, K, group):
    """K cut among workgroups, in as many slices as the workspace given has room for, none past its end."""
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M + N + K)
    x = rng.integers(-2, 3, (M, K)).astype(np.float32)
    sides = []
    for _ in range(2):
        _, q, s, z = _whole(rng, 1, N, K, group, True)
        sides.append((put_plane(plane_of(q, s, z, N, K, group)), x.astype(np.float64) @ values_of(q, s, z, K).T))
    ldx = _up(K, 8)
    d_x = upload(x, torch.bfloat16, ldx)
    need = uw.w4_gemm_workspace(M, N, K)
    assert need > 0 and need % (4 * M * N) == 0
    for given in (need, need - 4, 8 * M * N, 0):
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        y = torch.full((M, N + 1), 77.0, device="cuda")
        log(f"  slices {M}x{N}x{K} workspace {given} of {need}")
        uw.w4_gemm(d_x, sides[0][0], y, M, N, K, group=group, ldx=ldx, ldy=N + 1, d_ws=ws, ws_bytes=given)
        assert torch.equal(y[:, :N].cpu().double(), torch.from_numpy(sides[0][1])) and (y[:, N] == 77).all()
        assert (ws[given:] == 255).all()
    two = uw.w4_gemm_workspace(M, 2 * N, K)
    g, u = sides[0][1] / 4096, sides[1][1] / 4096
    d_x = upload(x / 4096, torch.bfloat16, ldx)  # a power of two: the products stay exact
    want = g / (1 + np.exp(-g)) * u
    hs = []
    for given in (two, 0):
        ws = torch.full((two + 64,), 255, dtype=torch.uint8, device="cuda")
        h = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        uw.w4_gate_up(d_x, sides[0][0], sides[1][0], h, M, N, K, group=group, ldx=ldx, d_ws=ws, ws_bytes=given)
        assert (ws[given:] == 255).all()
        hs.append(h)
    assert torch.equal(*hs)
    err = np.abs(hs[0].double().cpu().numpy() - want)
    assert (err <= np.abs(want) * (2.0**-8 + 8 * 2.0**-24) + 2.0**-133).all()


def _tolerance(x, s, K, group):
    """A = sum of 16 s |x| per output, times the steps of its sums."""
    M, G = x.shape[0], s.shape[1]
    xs = np.zeros((M, G * group))
    xs[:, :K] = np.abs(x)
    A = 16 * xs.reshape(M, G, group).sum(2) @ s.astype(np.float64).T
    return A * ((4 * group + 2) * 2.0**-23 + (G + 20) * 2.0**-24)


@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False)])
@pytest.mark.parametrize("M,N,K", [(1, 272, 4096), (4, 100, 1000), (6, 333, 2000), (16, 64, 4096), (40, 130, 1536), (64, 96, 4096)])
def test_gemm(M, N, K, group, zeros):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M + N + K)
    x = bf16(rng.standard_normal((M, K)) * np.exp(0.5 * rng.standard_normal((M, 1))))
    q, s, z = quantized(_weights(rng, N, K), group, zeros)
    want = x.astype(np.float64) @ values_of(q, s, z, K).T
    plane = put_plane(plane_of(q, s, z, N, K, group))
    tol = _tolerance(x, s, K, group)
    for out in (torch.float32, torch.bfloat16):
        ys = []
        for _ in range(2):
            y = torch.empty(M, N, dtype=out, device="cuda")
            uw.w4_gemm(upload(x, torch.bfloat16), plane, y, M, N, K, group=group)
            ys.append(y)
        assert torch.equal(*ys), "differs from run to run"
        err = np.abs(ys[0].double().cpu().numpy() - want)
        bound = tol + (np.abs(want) * 2.0**-8 if out is torch.bfloat16 else 0)
        log(f"  gemm {M}x{N}x{K} {out}: worst {np.max(err / bound):.3f} of the bound")
        assert (err <= bound).all()


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 333, 1000), (3, 40, 2000), (9, 64, 640), (16, 100, 4096), (20, 33, 300), (64, 48, 1000), (70, 30, 256)])
def test_gate_up(M, N, K, group, zeros):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M + N + K + 1)
    x = bf16(rng.standard_normal((M, K)))
    sides = [quantized(5 * _weights(rng, N, K), group, zeros) for _ in range(2)]
    g, u = (x.astype(np.float64) @ values_of(*p, K).T for p in sides)
    tg, tu = (_tolerance(x, p[1], K, group) for p in sides)
    sig = 1 / (1 + np.exp(-g))
    want = g * sig * u
    planes = [put_plane(plane_of(*p, N, K, group)) for p in sides]
    ldx, ldh = _up(K, 8), N + 1
    h = torch.full((M + 1, ldh), 77.0, dtype=torch.bfloat16, device="cuda")
    log(f"  gate_up {M}x{N}x{K}")
    uw.w4_gate_up(upload(x, torch.bfloat16, ldx), *planes, h, M, N, K, group=group, ldx=ldx, ldh=ldh)
    assert (h[M:] == 77).all() and (h[:, N:] == 77).all()
    err = np.abs(h[:M, :N].double().cpu().numpy() - want)
    # an error e of g changes silu(g) by at most 1.1 e
    bound = 1.1 * tg * (np.abs(u) + tu) + np.abs(g * sig) * tu + np.abs(want) * (2.0**-8 + 8 * 2.0**-24) + 2.0**-133
    assert (err <= bound).all(), np.max(err / bound)


def test_rows_keep_what_is_not_finite():
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(8)
    for M in (4, 16, 64):
        N, K, group = 48, 512, 128
        x, q, s, z = _whole(rng, M, N, K, group, True)
        want = x.astype(np.float64) @ values_of(q, s, z, K).T
        x[1, 5], x[3, 500] = np.nan, np.inf
        y = torch.zeros(M, N, device="cuda")
        uw.w4_gemm(upload(x, torch.bfloat16), put_plane(plane_of(q, s, z, N, K, group)), y, M, N, K, group=group)
        y = y.cpu().numpy()
        assert np.isnan(y[[1, 3]]).all()
        keep = [m for m in range(M) if m not in (1, 3)]
        assert (y[keep] == want[keep]).all()


def test_large_values_do_not_overflow_on_the_way():
    """x of 2^120 and scales of 2^-100: the products fit easily, and so must what leads to them."""
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(9)
    M, N, K, group = 2, 32, 256, 64
    x, q, s, z = _whole(rng, M, N, K, group, True)
    want = x.astype(np.float64) @ values_of(q, s, z, K).T
    big = np.ldexp(x, 115)
    for xs, ss, k in ((big, np.ldexp(s, -100), 15), (np.ldexp(x, -60), np.ldexp(s, 120), 60)):
        y = torch.zeros(M, N, device="cuda")
        uw.w4_gemm(upload(xs, torch.bfloat16), put_plane(plane_of(q, ss, z, N, K, group)), y, M, N, K, group=group)
        assert (y.cpu().numpy().astype(np.float64) == np.ldexp(want, k)).all()


def test_streams_and_graphs():
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(10)
    M, N, K, group = 3, 512, 2048, 128
    x, q, s, z = _whole(rng, M, N, K, group, False)
    want = torch.from_numpy(x.astype(np.float64) @ values_of(q, s, z, K).T).float()
    d_x, plane = upload(x, torch.bfloat16), put_plane(plane_of(q, s, z, N, K, group))
    need = max(1, uw.w4_gemm_workspace(M, N, K), uw.w4_gemm_workspace(M, 2 * N, K))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    y, h = torch.zeros(M, N, device="cuda"), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        uw.w4_gemm(d_x, plane, y, M, N, K, d_ws=ws, ws_bytes=need)
        uw.w4_gate_up(d_x, plane, plane, h, M, N, K, d_ws=ws, ws_bytes=need)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y.cpu(), want)
    h0 = h.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        uw.w4_gemm(d_x, plane, y, M, N, K, d_ws=ws, ws_bytes=need)
        uw.w4_gate_up(d_x, plane, plane, h, M, N, K, d_ws=ws, ws_bytes=need)
    for i in range(3):
        y.zero_()
        h.zero_()
        ws.fill_(255)
        d_x.neg_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want if i % 2 else -want)
        if i % 2:
            assert torch.equal(h, h0)


def test_rows_of_x_far_apart():
    """64 rows of X at the largest leading dimension: the last one begins 4.2 GB behind the first."""
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(11)
    N, K, group, ldx = 48, 300, 64, 1 << 25
    for M in (4, 16, 64):
        x, q, s, z = _whole(rng, M, N, K, group, True)
        want = torch.from_numpy(x.astype(np.float64) @ values_of(q, s, z, K).T).float()
        far = torch.empty((M - 1) * ldx + K, dtype=torch.bfloat16, device="cuda")
        for m in range(M):
            far[m * ldx:m * ldx + K] = torch.from_numpy(x[m]).to("cuda")
        y = torch.zeros(M, N, device="cuda")
        uw.w4_gemm(far, put_plane(plane_of(q, s, z, N, K, group)), y, M, N, K, group=group, ldx=ldx)
        assert torch.equal(y.cpu(), want)


def test_planes_past_four_gigabytes():
    """The last rows of a plane of 4.4 GB are those of a plane of their own."""
    torch, uw = torch_cuda(), _uw()
    K, N, group = 16384, 520_016, 128
    need = uw.w4_plane_bytes(N, K, group)
    assert need > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")
    w.normal_(generator=g)
    plane = torch.empty(need, dtype=torch.uint8, device="cuda")
    uw.w4_quantize(w, plane, N, K, group=group, zeros=True)
    few = 32
    tail = torch.empty(uw.w4_plane_bytes(few, K, group), dtype=torch.uint8, device="cuda")
    uw.w4_quantize(w[N - few:], tail, few, K, group=group, zeros=True)
    codes, codes_few = N * K // 2, few * K // 2
    assert torch.equal(plane[codes - codes_few:codes], tail[:codes_few])
    assert torch.equal(plane[need - (tail.numel() - codes_few):], tail[codes_few:])
    back = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    uw.w4_expand(plane, back, N, K, group=group)
    few_back = torch.zeros(few, K, dtype=torch.bfloat16, device="cuda")
    uw.w4_expand(tail, few_back, few, K, group=group)
    assert torch.equal(back[N - few:], few_back)
    del back, w
    x = torch.randint(-4, 5, (2, K), generator=g, device="cuda").to(torch.bfloat16)
    y, y_few = torch.zeros(2, N, device="cuda"), torch.zeros(2, few, device="cuda")
    uw.w4_gemm(x, plane, y, 2, N, K, group=group)
    uw.w4_gemm(x, tail, y_few, 2, few, K, group=group)
    want = x.double() @ few_back.double().t()
    assert torch.allclose(y[:, N - few:].double(), want, rtol=0, atol=2e-2 * float(want.abs().max()))
    err = (y[:, N - few:] - y_few).abs().max()
    assert float(err) <= 1e-5 * float(want.abs().max())
