"""The 8-bit path on the GPU where its sizes, values and kernels' shapes reach their ends, against its
definition in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda
from tests.test_fp8_plans import PLANS, SKINNY, plan_of
from tests.test_gpu_fp8 import _e4m3, _scales, _spread

pytestmark = pytest.mark.gpu


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def test_swiglu_down_to_where_silu_ends():
    """From g = -86 down e^g leaves the normal range (-87.3), silu itself (-91.9), and then fp32 (-108). One
    value per row, so that the scales tell |h| in fp32. silu is within 2.5 steps of 2^-23 and, subnormal,
    half of 2^-149; u = 2^60 is exact; the scale rounds by half a step, and so does the product: 3.5 * 2^-23."""
    uw, torch = _uw(), torch_cuda()
    rng = np.random.default_rng(87)
    g = np.concatenate([np.linspace(-112, -86, 20001), rng.uniform(-104, -87, 20000), -np.logspace(1.9, 38, 500)]).astype(np.float32)
    M = g.size
    y = np.zeros((M, 8), np.float32)
    y[:, 0], y[:, 4] = g, 2.0**60
    d = torch.from_numpy(y).cuda()
    q = torch.zeros(M, 16, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, M, device="cuda")
    uw.fp8_swiglu(d, d[:, 4:], q, s, M, 1, ldg=8, ldu=8, ldq=16)
    sh, qh = s[0].cpu().numpy().astype(np.float64), q[:, 0].cpu().numpy()
    g64 = g.astype(np.float64)
    silu = -g64 * np.exp(np.maximum(g64, -700)) / (1 + np.exp(np.maximum(g64, -700)))  # its absolute value
    tol = 3.5 * 2.0**-23 * silu + 2.0**-150
    none = qh & 0x7F == 0  # h is 0: scale 1
    assert (silu[none] <= tol[none]).all() and (sh[none] == 1).all()
    off = np.abs(sh * 448 * 2.0**-60 - silu)[~none] / tol[~none]
    log(f"  worst {off.max():.3g} of the tolerance, {int(none.sum())} of {M} are 0")
    assert (off <= 1).all()
    assert (qh[~none] == 0xFE).all()  # -448 at the scale
    assert none[g < -110].all() and not none[g > -107].any()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zeros_keep_their_sign(dtype, rows):
    """-0 / s is -0, code 0x80, beside other values and in a group of zeros alone."""
    uw, torch = _uw(), torch_cuda()
    K = 384
    x = np.random.default_rng(1).standard_normal((5, K)).astype(np.float32)
    x[:, 3::7] = -0.0
    x[:, 4::7] = 0.0
    x[:, 128:256:2], x[:, 129:256:2] = 0.0, -0.0
    d = torch.from_numpy(x).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)
    q = torch.full((5, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.zeros((3, 5) if rows == 1 else (1, 3), device="cuda")
    uw.fp8_quantize(d, q, s, 5, K, block_rows=rows)
    zero = x == 0
    assert (q.cpu().numpy()[zero] == np.where(np.signbit(x[zero]), 0x80, 0)).all()


def test_swiglu_zeros_keep_their_sign():
    """silu(-0) is -0, and so is silu of what underflows; the product's sign is that of both."""
    uw, torch = _uw(), torch_cuda()
    g = np.tile(np.array([0.0, -0.0, -300.0, 1.0, -1.0, 2.0, 0.0, -0.0], np.float32), 16)
    u = np.tile(np.array([1.0, 1.0, 1.0, -0.0, -0.0, 3.0, -1.0, -1.0], np.float32), 16)
    d = [torch.from_numpy(v).cuda().reshape(1, 128) for v in (g, u)]
    q = torch.full((1, 128), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, 1, device="cuda")
    uw.fp8_swiglu(d[0], d[1], q, s, 1, 128)
    assert (q[0].cpu().numpy() == np.tile(np.array([0, 0x80, 0x80, 0x80, 0, 0x7E, 0x80, 0], np.uint8), 16)).all()


def _up(n, m):
    return (n + m - 1) // m * m


def _exact_operands(M, N, K, seed):
    """Codes of which every group sum is exact in the matrix unit whichever product it takes, and scales of
    all sizes. The codes' values are 0 or 1 to 15/8 in steps of 1/8 with either sign: products are multiples of
    1/64 below 4, so 128 of them need 15 bits and no bit lies below 2^-8 of the largest product. Padding holds
    NaN codes. Returns ld and (codes, scales, values [n][K] in 64 bits without scales) of X and W."""
    torch = torch_cuda()
    gen = torch.Generator("cuda").manual_seed(seed)
    G, ld = -(-K // 128), _up(K, 16)
    out = []
    for n, rows in ((M, 1), (N, 128)):
        v = 1 + torch.randint(0, 8, (n, K), device="cuda", generator=gen) / 8.0
        v *= torch.randint(-1, 2, (n, K), device="cuda", generator=gen)
        q = torch.full((n, ld), 0x7F, dtype=torch.uint8, device="cuda")
        q[:, :K] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        s = torch.exp(torch.randn((G, n) if rows == 1 else (-(-n // 128), G), device="cuda", generator=gen))
        out.append((q, s, v.double()))
    return ld, out[0], out[1]


def _exact_product(M, N, K, x, w):
    """Y in 64 bits, and the sum of the magnitudes of the groups' terms."""
    torch = torch_cuda()
    (_, sx, xv), (_, sw, wv) = x, w
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for g in range(-(-K // 128)):
        k = slice(128 * g, min(K, 128 * g + 128))
        t = xv[:, k] @ wv[:, k].t().contiguous()
        t *= sx[g].double()[:, None]
        t *= sw[:, g].double().repeat_interleave(128)[:N][None, :]
        y += t
        mag += t.abs_()
    return y, mag


def _check_exact(y, ref, mag, K, slices, what):
    """The group sums being exact, what is left is the product of the scales, a group's fma and the waves'
    and slices' additions (16 of each at most), half a step of 2^-23 each and counted whole, and for bf16 the
    one rounding, 2^-8."""
    torch = torch_cuda()
    tol = (2 + -(-K // 128) + 16 + slices) * 2.0**-23 * mag
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0**-8 * (ref.abs() + tol)
    off = (y.double() - ref).abs()
    worst = float((off / tol.clamp(min=1e-300)).max())
    log(f"  {what}: worst {worst:.3g} of the tolerance")
    assert worst <= 1.0, what


@pytest.mark.parametrize("M,N,K", [(64, 4096, 14336), (100, 183, 12518), (2050, 257, 9000)])
def test_gemm_with_part_of_the_workspace(M, N, K):
    """Less workspace than uw_fp8_gemm_workspace gives fewer slices: right results, the same for every call, and
    nothing written past the bytes given."""
    uw, torch = _uw(), torch_cuda()
    need = uw.fp8_gemm_workspace(M, N, K)
    assert need > 0
    ld, x, w = _exact_operands(M, N, K, 5)
    ref, mag = _exact_product(M, N, K, x, w)
    for dt in (torch.float32, torch.bfloat16):
        for given in sorted({0, 15, need // 16, need // 4, 3 * need // 8, need // 2, 5 * need // 8, need - 1, need, need + 4096}):
            ws = torch.full((_up(given, 16) + 4096,), 0xEE, dtype=torch.uint8, device="cuda")
            y = [torch.zeros(M, N, dtype=dt, device="cuda") for _ in range(2)]
            for i in range(2):
                uw.fp8_gemm(x[0], x[1], w[0], w[1], y[i], M, N, K, ldx=ld, ldw=ld, d_ws=ws, ws_bytes=given)
            assert bool((ws[given:] == 0xEE).all()), f"{given} of {need} bytes given, written past them"
            assert torch.equal(y[0], y[1])
            _check_exact(y[0], ref, mag, K, 16, f"{M}x{N}x{K} {dt} {given} of {need}")


def _run_plan(uw, y, slices, M, N, K, ld, x, w, ldx=None, ldw=None):
    """Y [M][N] by the plan, with rows of Y a little further apart than N, which stay as they are behind it."""
    torch = torch_cuda()
    need = uw.fp8_gemm_workspace(M, N, K) if slices > 1 else 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
    out = torch.full((M + 1, N + 3), -77.0, dtype=torch.float32 if y == "f32" else torch.bfloat16, device="cuda")
    uw.fp8_gemm(x[0], x[1], w[0], w[1], out, M, N, K, ldx=ldx or ld, ldw=ldw or ld, ldy=N + 3, d_ws=ws, ws_bytes=need)
    assert bool((out[:M, N:] == -77).all()) and bool((out[M] == -77).all()), "outside the matrix"
    return out[:M, :N]


@pytest.mark.parametrize("y,tile,slices,M,N,K", PLANS + [("bf16", (128, 64), 1, 333, 5003, 2000), ("bf16", (256, 256), 1, 2048, 14336, 4096)])
def test_gemm_of_every_shape(y, tile, slices, M, N, K):
    """Every kernel shape, in one K slice and in several, K whole groups or not, with operands whose group sums
    are exact: a scale or a group that is off by more than the output's rounding shows. Then NaN codes
    and scales, which reach the outputs that they stand for and change no bit of the others."""
    uw, torch = _uw(), torch_cuda()
    p = plan_of(y, M, N, K, slices)
    assert ((p.tile_n, p.tile_m), p.slices) == (tile, slices)
    ld, x, w = _exact_operands(M, N, K, M + N + K)
    ref, mag = _exact_product(M, N, K, x, w)
    clean = _run_plan(uw, y, slices, M, N, K, ld, x, w)
    _check_exact(clean, ref, mag, K, slices, f"{y} {tile} / {slices}, {M}x{N}x{K}")
    m, n, G = M // 2, N - 1, -(-K // 128)
    x[0][m, K - 1] = 0xFF
    w[0][n, min(K - 1, 7)] = 0x7F
    x[1][G - 1, M - 1] = float("nan")
    w[1][0, G // 2] = float("nan")  # the first 128 columns
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[m], hit[M - 1], hit[:, n], hit[:, :128] = True, True, True, True
    got = _run_plan(uw, y, slices, M, N, K, ld, x, w)
    assert torch.equal(torch.isnan(got), hit)
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("y,tile,slices,M,N,K", [p for p in PLANS if p[1] not in SKINNY and p[5] % 128 and p[3] + p[4] < 6000])
def test_tiles_of_rows_past_32_bits(y, tile, slices, M, N, K):
    """The tile kernels take a row's place in its tile in 32 bits: rows of X and of W as far apart as they may
    be (255 of them are just under 2^32 bytes) give the bits that rows side by side give."""
    uw, torch = _uw(), torch_cuda()
    ld, x, w = _exact_operands(M, N, K, M)
    far = (1 << 24) - 16
    near = _run_plan(uw, y, slices, M, N, K, ld, x, w)
    for both in (False, True):
        fx = torch.empty(M, far, dtype=torch.uint8, device="cuda")
        fx[:, :ld] = x[0]
        fw, ldw = w[0], ld
        if both:
            fw, ldw = torch.empty(N, far, dtype=torch.uint8, device="cuda"), far
            fw[:, :ld] = w[0]
        assert torch.equal(_run_plan(uw, y, slices, M, N, K, ld, (fx, x[1]), (fw, w[1]), far, ldw), near)
        del fx, fw
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_of_tiny_values(dtype):
    """Every bf16 value over ten binades beside every largest value of its group, for groups whose scales go from
    2^-126 to 2^-103: the codes are those of the correctly rounded fp32 quotient, where x is subnormal or the
    quotient's residual would be, too."""
    uw, torch = _uw(), torch_cuda()
    man = np.arange(128, 256) / 128.0
    e = np.arange(-121, -95)
    x = np.zeros((128, 10, 2, e.size, 128))  # the group's largest, binades below it, halves of the others, binade of the largest
    x[..., 0] = (man[:, None] * 2.0**e)[:, None, None, :]
    v = (man.reshape(2, 64)[None, :, :] * 2.0 ** -np.arange(10)[:, None, None])[None, :, :, None, :] * (2.0**e)[:, None]
    x[..., 1:65] = np.where(v <= x[..., :1], v, 0)
    x[..., 65:] = -x[..., 1:64]
    M, K = 128 * 20, 128 * e.size
    x = x.reshape(M, K).astype(np.float32)
    d = torch.from_numpy(x).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)
    x = d.float().cpu().numpy()  # bf16 holds fewer bits of the smallest
    q = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    s = torch.zeros(K // 128, M, device="cuda")
    uw.fp8_quantize(d, q, s, M, K)
    ref = _scales(x, 1)
    assert (s.cpu().numpy().T == ref).all()
    off = q.cpu().numpy() != _e4m3(x / _spread(ref, 1, M, K))
    assert not off.any(), f"{int(off.sum())} of {off.size} codes"
