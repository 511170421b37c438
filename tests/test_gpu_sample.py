"""uw_sample on the GPU against its definition, row by row on the host.

The masses are whole multiples of 2^-43 of the largest token's, so the oracle's sums are exact
integers too and tokens have to be equal. The kernel's exponential is within 2.2e-12 of the value
and the oracle's is NumPy's, so borders between tokens may differ by 2^-38 of the row's mass; the
random numbers are multiples of 2^-24, and no seed here puts one that near a border.
Probabilities: one fp32 rounding, 2^-24, and the kept mass's 2^-30.
"""
import math

import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

ONE = 1 << 43


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def _draw(l, u, T=1.0, k=0, p=1.0, least=0.0):
    """(token, probability) of one row of float64 logits."""
    ids = np.flatnonzero(l > -math.inf)
    if not ids.size:
        return -1, 0.0
    ids = ids[np.lexsort((ids, -l[ids]))]
    top = l[ids[0]]
    if not T > 0:
        return int(ids[0]), 1.0
    with np.errstate(over="ignore", invalid="ignore"):
        if top == math.inf:
            w = np.where(l[ids] == top, 1.0, 0.0)
        else:
            d = l[ids] - top
            w = np.exp(np.where(d == 0, 0.0, d / T))
    if 0 < k < ids.size:
        w = w[:k]
    mass = np.rint(w * ONE).astype(np.uint64)  # 2^20 tokens of 2^43 are 2^63
    if p < 1:
        before = np.cumsum(mass) - mass
        mass = mass[: max(1, int(np.count_nonzero(before < np.uint64(max(1, math.ceil(max(float(p), 0.0) * float(mass.sum())))))))]
    if least > 0:
        mass = mass[: max(1, int(np.count_nonzero(w[: mass.size] >= least)))]
    c = np.cumsum(mass)
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0**-24)
    j = int(np.searchsorted(c, np.uint64(int(u * float(c[-1]))), side="right"))
    return int(ids[j]), float(w[j] * ONE / float(c[-1]))


def _run(uw, x, u, dtype="f32", ld=None, offset=0, **settings):
    """tokens and probabilities; x [M][V] float32, settings as lists or None."""
    torch = torch_cuda()
    M, V = x.shape
    ld = V if ld is None else ld
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    buf = torch.full((M * ld + offset,), float("inf"), dtype=td, device="cuda")  # what lies between rows is not looked at
    rows = buf[offset:].view(M, ld)
    rows[:, :V] = torch.from_numpy(x).cuda().to(td)
    dev = {}
    for n, v in settings.items():
        dev["d_" + n] = None if v is None else torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32, device="cuda")
    token = torch.full((M + 2,), -99, dtype=torch.int32, device="cuda")
    prob = torch.full((M + 2,), -99.0, device="cuda")
    need = uw.sample_workspace(M, V)
    ws = torch.full((max(16, need),), 0xEE, dtype=torch.uint8, device="cuda")
    du = torch.tensor(u, dtype=torch.float32, device="cuda")
    uw.sample(rows, du, token, M, V, ld=ld, d_prob=prob, d_ws=ws, ws_bytes=need, **dev)
    t, q = token.cpu().numpy(), prob.cpu().numpy()
    assert (t[M:] == -99).all() and (q[M:] == -99).all()
    again = torch.full_like(token, -99)
    uw.sample(rows, du, again, M, V, ld=ld, d_ws=ws, ws_bytes=need, **dev)  # no probabilities, workspace as left
    assert torch.equal(again, token)
    return t[:M], q[:M], rows[:, :V].double().cpu().numpy()


def _compare(uw, x, u, what="", **k):
    settings = {n: k.pop(n, None) for n in ("temperature", "top_k", "top_p", "min_p")}
    t, q, l = _run(uw, x, u, **k, **settings)
    for m in range(x.shape[0]):
        at = {n: np.float32(v[m]) if n != "top_k" else v[m] for n, v in settings.items() if v is not None}
        tok, pr = _draw(l[m], np.float32(u[m]), float(at.get("temperature", 1.0)), int(at.get("top_k", 0)),
                        float(at.get("top_p", 1.0)), float(at.get("min_p", 0.0)))
        assert t[m] == tok, f"{what} row {m} {at} u={u[m]}: {t[m]}, not {tok}"
        assert abs(q[m] - pr) <= 2.0**-23 * pr + 2.0**-30, f"{what} row {m} {at}: probability {q[m]}, not {pr}"


def _settings(rng, M):
    pick = lambda v: [v[i] for i in rng.integers(0, len(v), M)]  # noqa: E731
    return dict(temperature=pick([0.0, 0.3, 0.7, 1.0, 1.0, 1.5, 4.0]), top_k=pick([0, 0, 1, 2, 7, 50, 500, 5000]),
                top_p=pick([1.0, 1.0, 0.1, 0.5, 0.9, 0.99]), min_p=pick([0.0, 0.0, 0.001, 0.05, 0.5]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", [(1, 1), (3, 2), (5, 63), (4, 1000), (1, 32000), (7, 50257), (2, 131072), (33, 4099), (70, 20000),
                                 (300, 1111)])
def test_settings_and_sizes(M, V, dtype):
    uw = _uw()
    rng = np.random.default_rng(M * 31 + V)
    x = (rng.standard_normal((M, V)) * 2 + np.where(rng.random((M, V)) < 0.002, 6, 0)).astype(np.float32)
    _compare(uw, x, rng.random(M).astype(np.float32).tolist(), f"{M}x{V}", dtype=dtype, **_settings(rng, M))


@pytest.mark.parametrize("offset,pad", [(1, 0), (2, 1), (3, 7), (0, 5)])
def test_strides_and_alignment(offset, pad):
    uw = _uw()
    rng = np.random.default_rng(offset * 10 + pad)
    for dtype in ("f32", "bf16"):
        x = rng.standard_normal((6, 3001)).astype(np.float32) * 3
        _compare(uw, x, rng.random(6).tolist(), dtype=dtype, ld=3001 + pad, offset=offset, **_settings(rng, 6))


def test_no_settings_is_the_plain_softmax():
    uw = _uw()
    rng = np.random.default_rng(2)
    x = rng.standard_normal((16, 5000)).astype(np.float32)
    _compare(uw, x, rng.random(16).tolist())


@pytest.mark.parametrize("V", [40, 5000, 70001])
def test_ties(V):
    """Equal logits, few distinct ones, signed zeros: equal logits go by index, also where a filter cuts
    between them."""
    uw = _uw()
    rng = np.random.default_rng(V)
    u = [0.0, 0.1, 0.5, 0.75, 0.999, 1 - 2.0**-24]
    for x in (np.zeros((6, V)), np.full((6, V), -3.5), rng.choice([1.0, 0.0, -0.0, -1.0], (6, V)), rng.choice([5.0, 4.999], (6, V))):
        x = x.astype(np.float32)
        _compare(uw, x, u, "plain")
        _compare(uw, x, u, "k", top_k=[1, 2, V // 2, V - 1, V, V + 1])
        _compare(uw, x, u, "p", top_p=[0.0, 0.25, 0.5, 0.75, 0.999, 1.0])
        _compare(uw, x, u, "k p m", top_k=[V // 2 + 1] * 6, top_p=[0.5] * 6, min_p=[0.0, 0.1, 0.367, 0.5, 1.0, 2.0])
        _compare(uw, x, u, "greedy", temperature=[0.0] * 6)


def test_masks_and_special_values():
    uw = _uw()
    rng = np.random.default_rng(9)
    inf, nan = math.inf, math.nan
    x = rng.standard_normal((12, 3000)).astype(np.float32)
    low = np.finfo(np.float32).min
    x[0] = -inf                      # nothing left
    x[1] = nan
    x[2] = -inf
    x[2, 2999] = -1e30               # one left
    x[3, ::2] = -inf
    x[4, 5:100] = nan
    x[5, [7, 9]] = inf               # share the mass
    x[6] = low                       # masked by the type's lowest value throughout: equal logits
    x[7, 1:] = low
    x[8] = np.float32(-1e38) * rng.random(3000).astype(np.float32)
    x[9, 1500:] = -inf
    x[10] = 0
    x[10, 17] = 80.0                 # everything else below 2^-43
    x[11] = inf
    u = rng.random(12).astype(np.float32)
    u[5] = 0.7
    for kw in ({}, {"top_k": [3] * 12}, {"top_p": [0.9] * 12}, {"min_p": [0.2] * 12}, {"temperature": [0.0] * 12},
               {"temperature": [inf] * 12}, {"temperature": [1e-30] * 12}, {"temperature": [1e30] * 12},
               {"top_k": [100] * 12, "top_p": [0.5] * 12, "min_p": [0.01] * 12, "temperature": [0.8] * 12}):
        _compare(uw, x, u.tolist(), str(kw), **kw)


def test_settings_outside_their_range():
    uw = _uw()
    rng = np.random.default_rng(12)
    x = rng.standard_normal((8, 500)).astype(np.float32)
    u = rng.random(8).tolist()
    nan, inf = math.nan, math.inf
    _compare(uw, x, u, temperature=[-1.0, nan, 0.0, -inf, inf, 1e-45, 1e38, 1.0])
    _compare(uw, x, u, top_k=[-5, 0, 500, 501, 2**31 - 1, -(2**31), 1, 499])
    _compare(uw, x, u, top_p=[0.0, -1.0, 1.0, 2.0, nan, inf, -inf, 1e-30])
    _compare(uw, x, u, min_p=[0.0, -1.0, 1.0, 2.0, nan, inf, -inf, 1e-30])
    _compare(uw, x, [-1.0, nan, 1.0, 2.0, inf, -inf, 1 - 2.0**-24, 2.0**-24])


def test_long_runs_of_ties_beside_a_peak():
    """Vocabularies whose body is one value: the bins that the filters cut hold more tokens than fit a
    list, so the passes over the row answer."""
    uw = _uw()
    rng = np.random.default_rng(21)
    x = np.full((10, 100000), 1.0, np.float32)
    x[:, 500:520] = 9.0 + rng.standard_normal((10, 20)).astype(np.float32)
    x[5:, 1000:60000] = 1.0 + 1e-4 * rng.random((5, 59000)).astype(np.float32)
    u = rng.random(10).tolist()
    _compare(uw, x, u)
    _compare(uw, x, u, top_k=[5000, 20, 21, 60000, 99999] * 2)
    _compare(uw, x, u, top_p=[0.1, 0.5, 0.9, 0.99, 0.2] * 2)
    _compare(uw, x, u, min_p=[1e-3, 1e-4, 1e-5, 0.5, 1e-6] * 2)
    _compare(uw, x, u, top_k=[70000] * 10, top_p=[0.95] * 10, min_p=[1e-5] * 10, temperature=[0.9, 1.0] * 5)


def test_frequencies_follow_the_softmax():
    """Evenly spread numbers draw every token as often as its probability says, within one draw."""
    uw = _uw()
    rng = np.random.default_rng(6)
    l = rng.standard_normal(50).astype(np.float32) * 2
    n = 4096
    x = np.broadcast_to(l, (n, 50)).copy()
    t, _, _ = _run(uw, x, ((np.arange(n) + 0.5) / n).tolist(), temperature=None, top_k=None, top_p=None, min_p=None)
    p = np.exp(l.astype(np.float64) - l.max())
    p /= p.sum()
    assert (np.abs(np.bincount(t, minlength=50) - n * p) <= 1 + 1e-6).all()


def test_after_the_output_projection_in_a_graph():
    """A user's last steps of a token: 8-bit output projection, then the draw from its fp32 logits; the
    same after the lossless projection; captured, replayed with other numbers and settings."""
    import synth

    uw, torch = _uw(), torch_cuda()
    M, K, V = 8, 256, 1003
    rng = np.random.default_rng(8)
    wb = synth.f32_to_bf16_bits((rng.standard_normal((V, K)) * 0.2).astype(np.float32))
    blob = uw.encode(wb)
    h = uw.inspect(blob)
    d_blob = torch.from_numpy(blob).cuda()
    direct = torch.empty(uw.direct_plane_bytes(h), dtype=torch.uint8, device="cuda")
    uw.prepare_direct(h, d_blob, direct)
    d_w = torch.empty(V, K, dtype=torch.bfloat16, device="cuda")
    uw.decode_full(h, d_blob, d_w)
    qw = torch.empty(V, K, dtype=torch.uint8, device="cuda")
    sw = torch.empty(-(-V // 128), K // 128, device="cuda")
    uw.fp8_quantize(d_w, qw, sw, V, K, block_rows=128)
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda().bfloat16()
    u = torch.rand(M, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    T = torch.full((M,), 0.8, device="cuda")
    k = torch.full((M,), 40, dtype=torch.int32, device="cuda")
    need = uw.sample_workspace(M, V)
    logits = torch.zeros(2, M, V, device="cuda")
    token = torch.zeros(2, M, dtype=torch.int32, device="cuda")
    prob = torch.zeros(2, M, device="cuda")
    ws = torch.zeros(2, max(16, need), dtype=torch.uint8, device="cuda")
    qx = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    sx = torch.empty(K // 128, M, device="cuda")

    def step():
        uw.fp8_quantize(x, qx, sx, M, K)
        uw.fp8_gemm(qx, sx, qw, sw, logits[0], M, V, K)
        uw.run_pipeline(uw.PIPE_DIRECT, h, d_blob, x, logits[1].view(-1), M, d_direct=direct)
        for i in range(2):
            uw.sample(logits[i], u, token[i], M, V, d_temperature=T, d_top_k=k, d_prob=prob[i], d_ws=ws[i], ws_bytes=need)

    def check():
        for i in range(2):
            l = logits[i].double().cpu().numpy()
            for m in range(M):
                t, p = _draw(l[m], float(u[m]), float(T[m]), int(k[m]))
                assert int(token[i, m]) == t and abs(float(prob[i, m]) - p) <= 2.0**-23 * p + 2.0**-30

    step()
    check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        u.copy_(torch.rand(M, device="cuda", generator=torch.Generator("cuda").manual_seed(10 + i)))
        T.fill_(0.5 + 0.3 * i)
        k.fill_(3 + 40 * i)
        token.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        check()


def test_two_streams_at_once():
    uw, torch = _uw(), torch_cuda()
    M, V = 5, 30011
    rng = np.random.default_rng(14)
    xs = [torch.from_numpy(rng.standard_normal((M, V)).astype(np.float32) * 3).cuda() for _ in range(2)]
    us = [torch.rand(M, device="cuda") for _ in range(2)]
    toks = [torch.zeros(20, M, dtype=torch.int32, device="cuda") for _ in range(2)]
    need = uw.sample_workspace(M, V)
    wss = [torch.zeros(max(16, need), dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for x, u, t, ws, s in zip(xs, us, toks, wss, streams):
            with torch.cuda.stream(s):
                uw.sample(x, u, t[i], M, V, d_ws=ws, ws_bytes=need)
    torch.cuda.synchronize()
    for x, u, t in zip(xs, us, toks):
        ref = [_draw(l, float(v))[0] for l, v in zip(x.double().cpu().numpy(), u)]
        assert (t.cpu().numpy() == np.array(ref)).all()
    log("  20 calls on each of two streams")


@pytest.mark.parametrize("M,V,ld", [(300, 1001, (1 << 23) + 1), (100, 9001, (1 << 25) + 3)])
def test_rows_past_32_bits(M, V, ld):
    uw, torch = _uw(), torch_cuda()
    x = np.random.default_rng(V).standard_normal((M, V)).astype(np.float32) * 3
    near = torch.from_numpy(x).cuda().bfloat16()
    far = torch.empty(M, ld, dtype=torch.bfloat16, device="cuda")
    far[:, :V] = near
    u = torch.rand(M, device="cuda")
    tok = torch.zeros(2, M, dtype=torch.int32, device="cuda")
    need = uw.sample_workspace(M, V)
    ws = torch.zeros(max(16, need), dtype=torch.uint8, device="cuda")
    uw.sample(far, u, tok[0], M, V, ld=ld, d_ws=ws, ws_bytes=need)
    ref = [_draw(l, float(v))[0] for l, v in zip(near.double().cpu().numpy(), u)]
    assert (tok[0].cpu().numpy() == np.array(ref)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V", [(2, 40000), (3, 3000), (40, 9000)])
def test_large_k_and_wide_distributions(M, V, dtype):
    """k past what is gathered, alone and with the other steps, and distributions whose answers lie deep."""
    uw = _uw()
    rng = np.random.default_rng(M + V)
    u = rng.random(M).astype(np.float32)
    for spread, T in ((3.0, 1.0), (1.0, 1.0), (2.0, 3.0), (0.05, 1.0), (0.0, 1.0)):
        x = (rng.standard_normal((M, V)) * spread).astype(np.float32)
        for k, p, least in ((600, 1.0, 0.0), (890, 0.9, 0.0), (900, 1.0, 0.001), (2000, 0.95, 0.0), (2500, 0.7, 0.0), (V - 1, 0.999, 1e-3), (0, 0.9, 0.0), (0, 1.0, 1e-3), (0, 0.6, 0.02)):
            _compare(uw, x, u, f"spread {spread}", dtype=dtype, temperature=[T] * M, top_k=[k] * M, top_p=[p] * M, min_p=[least] * M)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_largest_vocabulary(dtype):
    """2^20 logits: all equal, all at the type's lowest value, flat, masked to a few, an infinite one among them."""
    uw = _uw()
    V = 1 << 20
    rng = np.random.default_rng(20)
    x = np.zeros((5, V), np.float32)
    x[1] = np.finfo(np.float32).min if dtype == "f32" else -float.fromhex("0x1.fep127")
    x[2] = rng.standard_normal(V)
    x[3] = -np.inf
    x[3, rng.integers(0, V, 30)] = rng.standard_normal(30)
    x[4] = rng.standard_normal(V)
    x[4, [7, V - 1]] = np.inf
    for k, p, least, T in ((0, 1.0, 0.0, 1.0), (0, 0.9, 0.0, 1.0), (100000, 0.5, 0.01, 2.0), (0, 1.0, 0.3, 1.0), (400, 0.9, 0.0, 1.0)):
        u = rng.random(5).astype(np.float32)
        _compare(uw, x, u, dtype=dtype, temperature=[T] * 5, top_k=[k] * 5, top_p=[p] * 5, min_p=[least] * 5)


def test_large_logits():
    """Logits far from 0 against their spread, and temperatures that make up for it."""
    uw = _uw()
    rng = np.random.default_rng(22)
    M, V = 6, 30000
    x = (rng.standard_normal((M, V)) * np.array([[1e6], [3e30], [1e-30], [1.0], [100.0], [1e-3]])).astype(np.float32)
    x[3] += np.float32(2e5)
    T = [1e6, 1e30, 1e-30, 1.0, 0.01, 1e-3]
    for k, p, least in ((0, 1.0, 0.0), (0, 0.9, 0.001), (700, 0.99, 0.0), (50, 0.9, 0.0)):
        _compare(uw, x, rng.random(M).astype(np.float32), temperature=T, top_k=[k] * M, top_p=[p] * M, min_p=[least] * M)


def test_rows_in_parts_in_a_graph():
    """Several workgroups per row, captured once and replayed on other logits, numbers and settings, on a
    stream of its own, with eager calls through another workspace in between."""
    uw, torch = _uw(), torch_cuda()
    M, V = 4, 50257
    need = uw.sample_workspace(M, V)
    assert need > 0
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.zeros(M, V, device="cuda")
    u, T, p, least = (torch.zeros(M, device="cuda") for _ in range(4))
    k = torch.zeros(M, dtype=torch.int32, device="cuda")
    token, again = (torch.zeros(M, dtype=torch.int32, device="cuda") for _ in range(2))
    prob = torch.zeros(M, device="cuda")
    ws = torch.full((2, need), 0xFF, dtype=torch.uint8, device="cuda")

    def call(tok, w):
        uw.sample(x, u, tok, M, V, d_temperature=T, d_top_k=k, d_top_p=p, d_min_p=least, d_prob=prob, d_ws=w, ws_bytes=need)

    call(token, ws[0])
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(token, ws[0])
    for spread, kk, pp, mm in ((3.0, 0, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (4.0, 60, 0.95, 0.0), (1.0, 3000, 0.8, 0.001), (2.0, 0, 1.0, 0.02)):
        x.copy_(torch.randn(M, V, device="cuda", generator=gen) * spread)
        u.copy_(torch.rand(M, device="cuda", generator=gen))
        T.copy_(torch.tensor([0.0, 0.7, 1.0, 1.6]))
        k.fill_(kk)
        p.fill_(pp)
        least.fill_(mm)
        token.fill_(-7)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
            graph.replay()
        torch.cuda.synchronize()
        call(again, ws[1])
        l = x.double().cpu().numpy()
        for m in range(M):
            t, q = _draw(l[m], float(u[m]), float(T[m]), kk, float(p[m]), float(least[m]))
            assert int(token[m]) == t and int(again[m]) == t and abs(float(prob[m]) - q) <= 2.0**-23 * q + 2.0**-30
