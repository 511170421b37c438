"""The 8-bit path on the GPU against its definition in 64 bits.

Tolerances, from the definition (half a step of a type: fp32 2^-24, bf16 2^-8, e4m3 2^-4
relative, 2^-10 of the scale below the normal range):
  scales   a / 448 is one fp32 division: equal to NumPy's
  codes    those of the correctly rounded fp32 quotient x / s: equal
  swiglu   h goes through exp, sum, quotient, product in fp32, each off by at most two halves of a
           step: 8 * 2^-24 of h; a code adds its own rounding
  gemm     per output, of sum |sx sw x w|: 128 additions in the matrix unit, which may cut instead
           of round (a whole step each), G fmas and the product of scales: (128 + G + 2) 2^-23;
           bf16 outputs add 2^-8 of the value, and 2^-10 of every group's largest product (the 8-bit
           matrix product lines 128 products up to the largest and drops their bits below 2^-17 of it
           or so, 128 * 2^-17 together)
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

TINY = np.float32(2.0**-126)


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def _up(n, m):
    return (n + m - 1) // m * m


def _values(rng, M, K):
    """Rows of different norms, some large channels, zeros, and groups of one size only."""
    x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))
    x[:, rng.random(K) < 0.02] *= 30
    x[rng.random((M, K)) < 0.05] = 0
    return x.astype(np.float32)


def _scales(x, rows):
    """Group scales in fp32 by the definition, [row groups][K groups], of finite-only maxima."""
    M, K = x.shape
    mb, kb = -(-M // rows), -(-K // 128)
    p = np.zeros((mb * rows, kb * 128), np.float32)
    p[:M, :K] = np.where(np.isfinite(x), np.abs(x), 0)
    a = p.reshape(mb, rows, kb, 128).max(axis=(1, 3))
    with np.errstate(under="ignore"):
        s = np.maximum(a / np.float32(448), TINY)
    return np.where(a == 0, np.float32(1), s).astype(np.float32)


def _spread(s, rows, M, K):
    return np.repeat(np.repeat(s, rows, 0)[:M], 128, 1)[:, :K]


def _e4m3(v):
    """e4m3 codes of fp32 v, nearest even, held at 448; non-finite -> 0x7F."""
    torch = torch_cuda()
    c = torch.from_numpy(np.clip(np.where(np.isfinite(v), v, 0), -448, 448).astype(np.float32)).to(torch.float8_e4m3fn)
    c = c.view(torch.uint8).numpy().copy()
    c[~np.isfinite(v)] = 0x7F
    return c


def _decode(codes):
    torch = torch_cuda()
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def _padded(x, ld, fill, dtype):
    torch = torch_cuda()
    t = torch.full((x.shape[0], ld), fill, dtype=dtype, device="cuda")
    t[:, : x.shape[1]] = torch.from_numpy(x).to("cuda").to(dtype)
    return t


SHAPES = [(1, 1), (1, 128), (1, 4096), (3, 129), (15, 100), (16, 640), (17, 127), (40, 1000), (128, 256), (129, 513),
          (300, 2056)]


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize(M, K, dtype, rows):
    uw, torch = _uw(), torch_cuda()
    rng = np.random.default_rng(1000 * M + K + rows)
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    ld = _up(K, 8) + 24
    x = _padded(_values(rng, M, K), ld, float("nan"), td)  # what lies behind a row is not looked at
    xs = x[:, :K].float().cpu().numpy()
    kb, mb = -(-K // 128), -(-M // rows)
    ldq = _up(K, 16) + 16
    q = torch.full((M + 1, ldq), 0xA5, dtype=torch.uint8, device="cuda")
    lds = (M if rows == 1 else kb) + 3
    s = torch.full((kb if rows == 1 else mb, lds), -7.0, device="cuda")
    uw.fp8_quantize(x, q, s, M, K, block_rows=rows, ldx=ld, ldq=ldq, lds=lds)
    torch.cuda.synchronize()
    sh, qh = s.cpu().numpy(), q.cpu().numpy()
    got = sh[:, :M].T if rows == 1 else sh[:, :kb]
    ref = _scales(xs, rows)
    assert (got == ref).all()
    assert (qh[:M, :K] == _e4m3(xs / _spread(ref, rows, M, K))).all()
    assert (qh[:M, K:] == 0xA5).all() and (qh[M] == 0xA5).all(), "codes outside the matrix were written"
    assert (sh[:, M if rows == 1 else kb:] == -7.0).all()


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize_extremes(rows):
    """Zero groups, one value, tiny and huge maxima, NaN and infinities beside finite values."""
    uw, torch = _uw(), torch_cuda()
    K = 128 * 8
    x = np.zeros((20, K), np.float32)
    rng = np.random.default_rng(5)
    x[:, 128:256] = rng.standard_normal((20, 128))
    x[:, 256] = -3.0
    x[:, 384:512] = rng.standard_normal((20, 128)) * np.float32(1e-40)   # subnormal
    x[:, 512:640] = rng.standard_normal((20, 128)) * np.float32(3e37)
    x[0, 512] = np.finfo(np.float32).max
    x[:, 640:768] = rng.standard_normal((20, 128))
    x[3, 640], x[4, 641], x[5, 642] = np.nan, np.inf, -np.inf
    x[:, 768:896] = np.nan
    x[:, 896:] = rng.standard_normal((20, 128)) * np.float32(2.0**-118)  # a / 448 just above 2^-126
    d = torch.from_numpy(x).cuda()
    q = torch.zeros(20, K, dtype=torch.uint8, device="cuda")
    s = torch.zeros((8, 20) if rows == 1 else (1, 8), device="cuda")
    uw.fp8_quantize(d, q, s, 20, K, block_rows=rows)
    got = s.cpu().numpy()
    got = got.T if rows == 1 else got
    ref = _scales(x, rows)
    assert (got == ref).all()
    assert (got[:, 0] == 1).all() and (got[:, 3] == TINY).all() and (got[:, 6] == 1).all()
    sp = _spread(ref, rows, 20, K)
    qh = q.cpu().numpy()
    fine = np.isfinite(x)
    assert ((qh[~fine] & 0x7F) == 0x7F).all()
    v = _decode(qh)
    err = np.abs(v * sp.astype(np.float64) - x)[fine]
    # half a step of e4m3, and half a subnormal step of the scale; 2^-22: the fp32 quotient
    assert (err <= (np.abs(x[fine].astype(np.float64)) * (2.0**-4 + 2.0**-22) + sp[fine].astype(np.float64) * 2.0**-10)).all()


@pytest.mark.parametrize("M,K", [(1, 1), (1, 14336), (7, 130), (16, 128), (33, 1000), (200, 640)])
def test_swiglu(M, K):
    uw, torch = _uw(), torch_cuda()
    rng = np.random.default_rng(M + K)
    half = _up(K, 4) + 4
    y = np.full((M, 2 * half), np.nan, np.float32)
    y[:, :K] = _values(rng, M, K)
    y[:, half:half + K] = _values(rng, M, K)
    y[0, 0] = -200.0  # silu underflows
    d = torch.from_numpy(y).cuda()
    ldq = _up(K, 16)
    q = torch.full((M, ldq), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.zeros(-(-K // 128), M, device="cuda")
    uw.fp8_swiglu(d, d[:, half:], q, s, M, K, ldg=2 * half, ldu=2 * half, ldq=ldq)
    g, u = y[:, :K].astype(np.float64), y[:, half:half + K].astype(np.float64)
    # the formula is an fp32 one: e^-g is past its largest number (e^88.72) there, and silu 0, which is
    # off by 88.73 e^-88.72 < 2.7e-37 of u at most; no input lies between -88.5 and -89
    h = np.where(g < -88.72, 0.0, g / (1 + np.exp(np.minimum(-g, 700)))) * u
    sg = s.cpu().numpy().T.astype(np.float64)
    p = np.zeros((M, _up(K, 128)))
    p[:, :K] = np.abs(h)
    a = p.reshape(M, -1, 128).max(2)
    ref = np.where(a == 0, 1, np.maximum(a / 448, 2.0**-126))
    assert (np.abs(sg - ref) <= 9 * 2.0**-24 * ref).all()
    qh = q.cpu().numpy()
    sp = _spread(sg, 1, M, K)
    v = _decode(qh[:, :K]) * sp
    assert (np.abs(v - h) <= np.abs(h) * (2.0**-4 + 2.0**-19) + sp * 2.0**-10).all()
    assert (qh[:, K:] == 0xA5).all()


def _operands(uw, rng, M, N, K, pad=0):
    """Codes and scales of X and W in padded rows whose padding holds NaN codes, and their values in 64 bits."""
    torch = torch_cuda()
    ld = _up(K, 16) + pad
    out = []
    for n, rows in ((M, 1), (N, 128)):
        v = _values(rng, n, K)
        s = _scales(v, rows)
        c = _e4m3(v / _spread(s, rows, n, K))
        q = np.full((n, ld), 0x7F, np.uint8)
        q[:, :K] = c
        st = np.ascontiguousarray(s.T if rows == 1 else s)
        out.append((torch.from_numpy(q).cuda(), torch.from_numpy(st).cuda(), _decode(c) * _spread(s, rows, n, K).astype(np.float64)))
    return ld, out[0], out[1]


def _check(y, x, w, K, bf16, what):
    ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = (128 + -(-K // 128) + 2) * 2.0**-23 * mag
    if bf16:
        for k in range(0, K, 128):  # at least the largest product of the group
            tol = tol + 2.0**-10 * np.minimum(np.abs(x[:, k:k + 128]).max(1)[:, None] * np.abs(w[:, k:k + 128]).max(1)[None, :],
                                              np.abs(x[:, k:k + 128]) @ np.abs(w[:, k:k + 128]).T)
        tol = tol + 2.0**-8 * (np.abs(ref) + tol)
    err = np.abs(y - ref)
    assert np.isfinite(y).all(), what
    assert (err <= tol).all(), f"{what}: worst {np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


GEMMS = [(1, 1, 1), (1, 16, 128), (1, 4096, 512), (1, 1000, 4096), (2, 130, 127), (5, 257, 129), (16, 128, 1000),
         (17, 300, 384), (33, 100, 2000), (64, 512, 1024), (64, 5, 14336), (65, 129, 256), (100, 1000, 640),
         (128, 256, 128), (200, 333, 1408), (257, 511, 272), (333, 1003, 2000), (600, 260, 100), (1024, 1024, 512),
         (1100, 770, 1296), (2049, 257, 384)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm(M, N, K, out):
    uw, torch = _uw(), torch_cuda()
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    ld, (qx, sx, x), (qw, sw, w) = _operands(uw, rng, M, N, K, pad=16 * (M % 3))
    dt = torch.float32 if out == "f32" else torch.bfloat16
    need = uw.fp8_gemm_workspace(M, N, K)
    for ldy, ws in ((N, True), (N + 3, False), (_up(N, 4) + 4, True)):
        y = torch.full((M + 1, ldy), -77.0, dtype=dt, device="cuda")
        d_ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda") if ws else None
        uw.fp8_gemm(qx, sx, qw, sw, y, M, N, K, ldx=ld, ldw=ld, ldy=ldy, d_ws=d_ws, ws_bytes=need if ws else 0)
        yh = y.double().cpu().numpy()
        _check(yh[:M, :N], x, w, K, out == "bf16", f"M={M} N={N} K={K} {out} ldy={ldy} ws={ws}")
        assert (yh[:M, N:] == -77).all() and (yh[M] == -77).all(), "outside the matrix"
        if ws:
            again = torch.empty_like(y)
            uw.fp8_gemm(qx, sx, qw, sw, again, M, N, K, ldx=ld, ldw=ld, ldy=ldy, d_ws=d_ws, ws_bytes=need)
            assert torch.equal(again[:M, :N], y[:M, :N]), "two runs differ"


def test_gemm_nan_stays_in_its_row_and_column():
    uw, torch = _uw(), torch_cuda()
    for M, N, K in ((5, 130, 300), (200, 270, 300)):
        ld, (qx, sx, x), (qw, sw, w) = _operands(uw, np.random.default_rng(3), M, N, K)
        qx[2, 17] = 0x7F
        qw[129, 299] = 0xFF
        y = torch.zeros(M, N, device="cuda")
        uw.fp8_gemm(qx, sx, qw, sw, y, M, N, K, ldx=ld, ldw=ld)
        bad = torch.isnan(y).cpu().numpy()
        ref = np.zeros((M, N), bool)
        ref[2] = True
        ref[:, 129] = True
        assert (bad == ref).all()


def test_mlp_from_a_blob_end_to_end():
    """A user's run: weights out of a compressed blob, quantized in blocks; hidden states quantized by
    rows; gate and up as one stacked product; the activation into codes; down. Against the same
    steps in 64 bits from the GPU's own codes at each step, and the whole against bf16 weights."""
    import synth

    uw, torch = _uw(), torch_cuda()
    M, K, F = 24, 256, 512
    rng = np.random.default_rng(11)
    mats = {}
    for name, (n, k) in (("gate", (F, K)), ("up", (F, K)), ("down", (K, F))):
        wb = synth.f32_to_bf16_bits((rng.standard_normal((n, k)) * 0.05).astype(np.float32))
        blob = uw.encode(wb)
        h = uw.inspect(blob)
        d_blob = torch.from_numpy(blob).cuda()
        d_w = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
        uw.decode_full(h, d_blob, d_w)
        mats[name] = d_w
    gu = torch.cat([mats["gate"], mats["up"]])

    def blocks(w):
        n, k = w.shape
        q = torch.empty(n, k, dtype=torch.uint8, device="cuda")
        s = torch.empty(-(-n // 128), -(-k // 128), device="cuda")
        uw.fp8_quantize(w, q, s, n, k, block_rows=128)
        return q, s

    qgu, sgu = blocks(gu)
    qd, sd = blocks(mats["down"])
    x = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()

    def step():
        qx = torch.empty(M, K, dtype=torch.uint8, device="cuda")
        sx = torch.empty(K // 128, M, device="cuda")
        uw.fp8_quantize(x, qx, sx, M, K)
        y = torch.empty(M, 2 * F, device="cuda")
        uw.fp8_gemm(qx, sx, qgu, sgu, y, M, 2 * F, K)
        qh = torch.empty(M, F, dtype=torch.uint8, device="cuda")
        sh = torch.empty(F // 128, M, device="cuda")
        uw.fp8_swiglu(y, y[:, F:], qh, sh, M, F, ldg=2 * F, ldu=2 * F)
        out = torch.empty(M, K, device="cuda")
        uw.fp8_gemm(qh, sh, qd, sd, out, M, K, F)
        return y, qh, sh, out

    y, qh, sh, out = step()
    hv = _decode(qh.cpu().numpy()) * _spread(sh.cpu().numpy().T, 1, M, F)
    dv = _decode(qd.cpu().numpy()) * _spread(sd.cpu().numpy(), 128, K, F)
    _check(out.double().cpu().numpy(), hv, dv, F, False, "down")
    g, u = (x.double() @ w.double().t() for w in (mats["gate"], mats["up"]))
    ref = (g / (1 + torch.exp(-g)) * u) @ mats["down"].double().t()
    rel = float((out.double() - ref).norm() / ref.norm())
    log(f"  8-bit MLP against bf16 weights: {rel:.4f} of the norm")
    # every code is off by at most 2^-4 of its value, two operands a product, two products in a row; the
    # activation's slope is at most 1.1 and enters once for g and once for u: 2 * 2^-4 * (1 + 2.1)
    assert rel < 0.39

    # the same in a captured graph, replayed on other hidden states, with eager work in between
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()[3]
    for seed in range(3):
        x.copy_(torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, step()[3])


def _far(x, ld, dtype):
    """x in the first columns of rows ld elements apart; the rest is never written."""
    torch = torch_cuda()
    t = torch.empty(x.shape[0], ld, dtype=dtype, device="cuda")
    t[:, : x.shape[1]] = x
    return t


def test_rows_past_32_bits():
    """Strides that put the last rows more than 2^32 bytes behind the first, in every operand."""
    uw, torch = _uw(), torch_cuda()
    K = 200
    rng = np.random.default_rng(21)
    for M, N in ((300, 290), (20, 290)):
        ld0, (qx, sx, x), (qw, sw, w) = _operands(uw, rng, M, N, K)
        ld = (1 << 24) - 16
        fx, fw = _far(qx, ld, torch.uint8), _far(qw, ld, torch.uint8)
        for dt in (torch.float32, torch.bfloat16):
            ldy = (1 << 24) + 5
            y = torch.empty(M, ldy, dtype=dt, device="cuda")
            uw.fp8_gemm(fx, sx, fw, sw, y, M, N, K, ldx=ld, ldw=ld, ldy=ldy)
            _check(y[:, :N].double().cpu().numpy(), x, w, K, dt == torch.bfloat16, f"M={M} {dt}")
        del fx, fw, y
    M = 300
    for dt, ld in ((torch.float32, (1 << 22) + 4), (torch.bfloat16, (1 << 23) + 8)):
        v = torch.from_numpy(_values(rng, M, K)).cuda().to(dt)
        fv = _far(v, ld, dt)
        for rows in (1, 128):
            q, qf = torch.zeros(M, 208, dtype=torch.uint8, device="cuda"), torch.empty(M, 1 << 24, dtype=torch.uint8, device="cuda")
            s, sf = torch.zeros(2, 3, M, device="cuda")
            lds = M if rows == 1 else 2
            uw.fp8_quantize(v, q, s, M, K, block_rows=rows, ldq=208, lds=lds)
            uw.fp8_quantize(fv, qf, sf, M, K, block_rows=rows, ldx=ld, ldq=1 << 24, lds=lds)
            assert torch.equal(q[:, :K], qf[:, :K]) and torch.equal(s, sf)
        del fv, qf
    g, u = (torch.from_numpy(_values(rng, M, K)).cuda() for _ in range(2))
    fg = _far(torch.cat([g, u], 1), (1 << 22) + 4, torch.float32)
    s, sf = torch.zeros(2, 2, M, device="cuda")
    uw.fp8_swiglu(g, u, q, s, M, K, ldq=208)
    q2 = torch.zeros_like(q)
    uw.fp8_swiglu(fg, fg[:, K:], q2, sf, M, K, ldg=(1 << 22) + 4, ldu=(1 << 22) + 4, ldq=208)
    assert torch.equal(q[:, :K], q2[:, :K]) and torch.equal(s, sf)


def test_gemm_slices_in_two_graphs_at_once():
    """Two captured products replayed on two streams, each with a workspace of its own; of the two sizes
    the longer one is cut into K slices."""
    uw, torch = _uw(), torch_cuda()
    sizes = ((40, 512, 8192), (64, 2048, 14336))
    assert max(uw.fp8_gemm_workspace(*size) for size in sizes) > 0
    for size in sizes:
        _two_graphs(uw, torch, *size)


def _two_graphs(uw, torch, M, N, K):
    need = uw.fp8_gemm_workspace(M, N, K)
    runs = []
    for i in range(2):
        ld, (qx, sx, x), (qw, sw, w) = _operands(uw, np.random.default_rng(30 + i), M, N, K)
        y, ws = torch.zeros(M, N, device="cuda"), torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        call = lambda: uw.fp8_gemm(qx, sx, qw, sw, y, M, N, K, ldx=ld, ldw=ld, d_ws=ws, ws_bytes=need)
        call()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
        runs.append((graph, stream, y, x, w, (qx, sx, qw, sw, ws)))
    for _ in range(4):
        for graph, stream, y, *_ in runs:
            y.zero_()
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, y, x, w, _ in runs:
            _check(y.double().cpu().numpy(), x, w, K, False, "replay")


# Sizes that each of the kernel's shapes takes, in one slice and in several where it is cut at all
LARGER = [(40, 6000, 144), (100, 4100, 144), (24, 4100, 4112), (1030, 1003, 144), (2050, 1003, 144), (130, 515, 9000),
          (40, 4100, 4112), (520, 8010, 400), (2050, 257, 4112), (2050, 257, 9000), (2050, 6000, 272), (2050, 1003, 4112),
          (2050, 1003, 9000), (2050, 6000, 1296), (700, 6000, 9000)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", LARGER)
def test_gemm_larger(M, N, K, out):
    """The tolerance of the small ones, with operands and reference made on the GPU."""
    uw, torch = _uw(), torch_cuda()
    gen = torch.Generator("cuda").manual_seed(M + N + K)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen)
    G, ld = -(-K // 128), _up(K, 16)
    qx, qw = (torch.full((n, ld), 0x7F, dtype=torch.uint8, device="cuda") for n in (M, N))
    sx, sw = torch.exp(rand(G, M)), torch.exp(rand(-(-N // 128), G))
    spread = lambda s, n: s.repeat_interleave(128, 1)[:n, :K].double()
    vals = []
    for q, s in ((qx, sx.t()), (qw, sw.repeat_interleave(128, 0)[:N])):
        c = (rand(q.shape[0], K) * 40).to(torch.float8_e4m3fn)
        q[:, :K] = c.view(torch.uint8)
        vals.append(c.double() * spread(s, q.shape[0]))
    x, w = vals
    bf16 = out == "bf16"
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    tol = (128 + G + 2) * 2.0**-23 * mag
    if bf16:
        for k in range(0, K, 128):
            a, b = x[:, k:k + 128].abs(), w[:, k:k + 128].abs()
            tol += 2.0**-10 * torch.minimum(a.amax(1)[:, None] * b.amax(1)[None, :], a @ b.t())
        tol += 2.0**-8 * (ref.abs() + tol)
    need = uw.fp8_gemm_workspace(M, N, K)
    for ws in (None, torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")):
        ldy = N + 1 if ws is None else _up(N, 4)
        y = torch.full((M + 1, ldy), -77.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
        uw.fp8_gemm(qx, sx, qw, sw, y, M, N, K, ldx=ld, ldw=ld, ldy=ldy, d_ws=ws, ws_bytes=need if ws is not None else 0)
        err = (y[:M, :N].double() - ref).abs()
        worst = float((err / tol).max())
        log(f"  M={M} N={N} K={K} {out} workspace {0 if ws is None else need}: worst {worst:.3g} of the tolerance")
        assert worst <= 1.0
        assert bool((y[:M, N:] == -77).all()) and bool((y[M] == -77).all()), "outside the matrix"


def test_swiglu_over_the_range_of_g():
    """One value per row, so that the scales tell |h| in fp32. silu is within 2.5 steps of 2^-23, product
    and scale round by half a step each: 3.5 * 2^-23."""
    uw, torch = _uw(), torch_cuda()
    g = np.concatenate([np.linspace(-87, 90, 5000), -np.logspace(-30, 1, 500), np.logspace(-30, 30, 500)]).astype(np.float32)
    odd = np.array([0.0, -0.0, -100.0, -1e4, -3e38, np.inf, -np.inf, np.nan], np.float32)
    y = np.zeros((g.size + odd.size, 8), np.float32)
    y[:, 0], y[:, 4] = np.concatenate([g, odd]), 2.0**30
    M = y.shape[0]
    d = torch.from_numpy(y).cuda()
    q = torch.zeros(M, 16, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, M, device="cuda")
    uw.fp8_swiglu(d, d[:, 4:], q, s, M, 1, ldg=8, ldu=8, ldq=16)
    sh, qh = s[0].cpu().numpy().astype(np.float64), q[:, 0].cpu().numpy()
    g64 = g.astype(np.float64)
    with np.errstate(over="ignore"):
        h = g64 / (1 + np.exp(-g64)) * 2.0**30
    fits = np.abs(h) <= np.finfo(np.float32).max  # 10^30 * 2^30 is infinite in fp32: a NaN code, scale 1
    assert (sh[: g.size][~fits] == 1).all() and (qh[: g.size][~fits] & 0x7F == 0x7F).all()
    ref = np.maximum(np.abs(h) / 448, 2.0**-126)
    assert (np.abs(sh[: g.size] - ref) <= 3.5 * 2.0**-23 * ref)[fits].all()
    big = fits & (np.abs(h) / 448 > 2.0**-125)
    assert (qh[: g.size][big] == np.where(h[big] < 0, 0xFE, 0x7E)).all()  # +-448 at the scale
    assert (qh[g.size + np.array([0, 1, 3, 4])] & 0x7F == 0).all() and (qh[g.size + 5 :] & 0x7F == 0x7F).all()
    # e^-100 is 26.5 of the smallest fp32 steps, known to one of them: a value all the same, and not 0
    tiny = 100 * np.exp(-100.0) * 2.0**30
    assert qh[g.size + 2] == 0xFE and abs(sh[g.size + 2] * 448 - tiny) <= tiny / 26
    assert (sh[g.size + 5 :] == 1).all()
