"""Log probabilities on the GPU against their definition in 64 bits.

Ranks and top tokens are comparisons: equal. With u = 2^-24 and y = (l - max) log2(e) / T, a term 2^y is off by 3 u |y| (its three
roundings; log(2) < 1) + 2 u (the exponential), the sums of a thread by one u per addition: 16 in a step, and one and two for a
grown maximum in each of V / 4096 + 1 steps; the mean of these over the row's mass is what log S may be off by:
  e_S = u (3 E|y| + 20 + 3 (V / 4096 + 1)),
a log probability by that and half a step of fp32, the entropy by e_S and, for H / S, by (2 e_S + u) E|y| and, where y is large and the mass
small, 3 u E(y^2); outputs are rounded once.
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0**-24


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def reference(x, token, T, n):
    """(logprob, its tolerance, rank, entropy, its tolerance, top tokens, top logprobs) of one row (float32 values)."""
    V = x.size
    l = x.astype(np.float64)
    placed = np.flatnonzero(l > -np.inf)
    order = placed[np.lexsort((placed, -l[placed]))]
    lp = np.full(V, -np.inf)
    ent = tol = tol_ent = 0.0
    if order.size:
        if not T > 0:
            lp[order[0]] = 0.0
        else:
            top = l[order[0]]
            if top == np.inf:
                y = np.where(l[placed] == top, 0.0, -np.inf)
            else:
                with np.errstate(over="ignore"):
                    y = (l[placed] - top) / T
            e = np.exp(y)
            S = e.sum()
            some = e > 0
            lp[placed] = y - np.log1p(S - 1)
            ent = np.log1p(S - 1) - (e[some] * y[some]).sum() / S
            E1 = (e[some] * -y[some]).sum() / S * 1.4427
            E2 = (e[some] * y[some]**2).sum() / S * 2.0814
            tol = U * (3 * E1 + 20 + 3 * (V / 4096 + 1))
            tol_ent = tol + (2 * tol + U) * E1 + 3 * U * E2
    rank, p = -1, -np.inf
    if 0 <= token < V and l[token] > -np.inf:
        rank, p = int(np.flatnonzero(order == token)[0]), lp[token]
    tt = np.full(n, -1)
    tl = np.full(n, -np.inf)
    tt[:order.size] = order[:n]
    tl[:order.size] = lp[order[:n]]
    return p, tol, rank, ent, tol_ent, tt, tl


def near(got, want, tol, what):
    if want < -(2.0**128 - 2.0**103):  # past fp32's range, the rounding of an output is -inf
        want = -np.inf
    if not np.isfinite(want):
        assert got == want, f"{what}: {got} for {want}"
    else:
        assert abs(got - want) <= tol + U * abs(want) + 2.0**-149, f"{what}: {got} for {want}, off by {abs(got - want):.3g}, allowed {tol:.3g}"


def run(x, token, n=0, T=None, bf16=False, pad=0, shift=0):
    """logprobs() of rows x (float32 NumPy), checked row by row. pad: elements behind a row; shift: the first row starts that
    many elements into its buffer."""
    torch, uw = torch_cuda(), _uw()
    M, V = x.shape
    dtype = torch.bfloat16 if bf16 else torch.float32
    if bf16:
        x = torch.from_numpy(x).to(dtype).float().numpy()
    ld = V + pad
    buf = torch.full((shift + M * ld,), 1e9, dtype=dtype, device="cuda")  # what is not of a row would win every maximum
    rows = buf[shift:].view(M, ld)
    rows[:, :V] = torch.from_numpy(x).to("cuda", dtype)
    t = torch.tensor(token, dtype=torch.int32, device="cuda")
    temp = None if T is None else torch.tensor(np.broadcast_to(np.asarray(T, np.float32), (M,)).copy(), device="cuda")
    lp, ent = torch.full((M + 1,), 77.0, device="cuda"), torch.full((M + 1,), 77.0, device="cuda")
    rank = torch.full((M + 1,), 77, dtype=torch.int32, device="cuda")
    tt, tl = torch.full((M + 1, max(1, n)), 77, dtype=torch.int32, device="cuda"), torch.full((M + 1, max(1, n)), 77.0, device="cuda")
    need = uw.logprobs_workspace(M, V, n)
    ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device="cuda")
    log(f"  logprobs {M}x{V} top {n} {'bf16' if bf16 else 'f32'} workspace {need}")
    uw.logprobs(rows, M, V, d_token=t, d_logprob=lp[:M], d_rank=rank[:M], d_entropy=ent[:M], n_top=n, d_top_token=tt[:M] if n else None, d_top_logprob=tl[:M] if n else None,
                d_temperature=temp, ld=ld, d_ws=ws, ws_bytes=need)
    lp, ent, rank, tt, tl = (v.cpu().numpy() for v in (lp, ent, rank, tt, tl))
    assert lp[M] == 77 and ent[M] == 77 and rank[M] == 77 and (tt[M] == 77).all() and (tl[M] == 77).all()
    for m in range(M):
        f = 1.0 if T is None else float(np.broadcast_to(np.asarray(T, np.float32), (M,))[m])
        p, tol, k, e, tol_e, wt, wl = reference(x[m], int(token[m]), f, n)
        assert rank[m] == k, f"row {m}: rank {rank[m]} for {k}"
        near(lp[m], p, tol, f"row {m}: log probability")
        near(ent[m], e, tol_e, f"row {m}: entropy")
        if n:
            assert (tt[m] == wt).all(), f"row {m}: top tokens {tt[m][:8]} for {wt[:8]}"
            for i in range(n):
                near(tl[m][i], wl[i], tol, f"row {m}: top {i}")


def _logits(rng, M, V, kind):
    x = 2 * rng.standard_normal((M, V))
    if kind == "peaked":
        x += np.where(rng.random((M, V)) < 0.002, 4 + 6 * rng.random((M, V)), 0)
    if kind == "masked":
        x[rng.random((M, V)) >= 0.05] = -np.inf
    if kind == "sure":  # one token has nearly all of the mass
        x[np.arange(M), rng.integers(0, V, M)] += 25
    return x.astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 255, 256, 257, 1000, 4095, 4096, 4097, 8200, 32000, 50257, 131072])
@pytest.mark.parametrize("bf16", [False, True])
def test_row_lengths(V, bf16):
    rng = np.random.default_rng(V)
    for M, kind, n, pad, shift in ((1, "peaked", 20, 0, 0), (3, "flat", 5, 3, 1), (2, "masked", 64, 1, 3)):
        run(_logits(rng, M, V, kind), rng.integers(0, V, M), n, bf16=bf16, pad=pad, shift=shift)


@pytest.mark.parametrize("M", [7, 64, 300, 1100])
def test_many_rows(M):
    rng = np.random.default_rng(M)
    run(_logits(rng, M, 5003, "peaked"), rng.integers(0, 5003, M), 3, T=rng.choice([0.6, 1.0, 1.3], M), pad=1)
    run(_logits(rng, M, 700, "masked"), rng.integers(0, 700, M), 128, bf16=True)


@pytest.mark.parametrize("M,V", [(3, 47999), (3, 48000), (127, 50001), (128, 50001), (320, 100000), (321, 100000), (767, 5000), (768, 5000)])
def test_where_launch_shapes_change(M, V):
    """Every number of threads and of slices, a few rows of each checked (the others are copies of them)."""
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M + V)
    few = _logits(rng, 3, V, "peaked")
    tok, n = rng.integers(0, V, 3), 20
    rows = torch.from_numpy(few).to("cuda").repeat(-(-M // 3), 1)[:M]
    t = torch.tensor(np.tile(tok, -(-M // 3))[:M].astype(np.int32), device="cuda")
    lp, ent, rank = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")
    tt, tl = torch.zeros(M, n, dtype=torch.int32, device="cuda"), torch.zeros(M, n, device="cuda")
    need = uw.logprobs_workspace(M, V, n)
    ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device="cuda")
    uw.logprobs(rows, M, V, d_token=t, d_logprob=lp, d_rank=rank, d_entropy=ent, n_top=n, d_top_token=tt, d_top_logprob=tl, d_ws=ws, ws_bytes=need)
    for m in range(min(3, M)):
        p, tol, k, e, tol_e, wt, wl = reference(few[m], int(tok[m]), 1.0, n)
        assert (rank[m::3] == k).all() and (tt[m::3].cpu().numpy() == wt).all()
        near(float(lp[m]), p, tol, "log probability")
        near(float(ent[m]), e, tol_e, "entropy")
        # rows that lie elsewhere in memory may begin at another place in a word, and sum up in another order
        assert (lp[m::3] - lp[m]).abs().max() <= 2 * tol + 2 * U * abs(p) and (tl[m::3] - tl[m]).abs().max() <= 2 * tol + 2 * U * abs(wl[-1])


def test_longest_row():
    rng = np.random.default_rng(4)
    V = 1 << 20
    run(_logits(rng, 2, V, "flat"), [V - 1, 12345], 128)


@pytest.mark.parametrize("n", [0, 1, 2, 20, 64, 127, 128])
def test_list_lengths(n):
    rng = np.random.default_rng(n)
    for V in (20, 3000, 70001):
        run(_logits(rng, 2, V, "peaked"), rng.integers(0, V, 2), n)


def test_temperatures():
    rng = np.random.default_rng(6)
    T = np.array([0.0, -1.0, np.nan, np.inf, 1e-3, 1e-38, 1e-42, 1e6, 3e38, 0.7, 1.0, 2.0], np.float32)
    x = np.repeat(_logits(rng, 1, 9000, "peaked"), T.size, 0)
    best = int(x[0].argmax())
    run(x, [best] * T.size, 4, T=T)
    run(x, rng.integers(0, 9000, T.size), 4, T=T)
    m = _logits(rng, T.size, 9000, "masked")
    run(m, [int(r.argmax()) for r in m], 4, T=T)


@pytest.mark.parametrize("V", [500, 40000])
def test_nearly_certain(V):
    rng = np.random.default_rng(7)
    x = _logits(rng, 6, V, "sure")
    run(x, x.argmax(1), 5)


def test_masks_infinities_nan_and_tokens_outside():
    V = 10000
    rng = np.random.default_rng(8)
    x = _logits(rng, 12, V, "flat")
    tok = rng.integers(0, V, 12)
    x[0] = -np.inf                         # nothing left
    x[1] = -np.inf
    x[1, 77] = -3.0                        # one left
    tok[1] = 77
    x[2, 5] = np.inf
    x[2, 9000] = np.inf                    # shared by two
    tok[2] = 9000
    x[3, 100] = np.inf
    tok[3] = 4                             # finite beside an infinity
    x[4, ::2] = np.nan
    tok[4] = 2                             # NaN has no place
    x[5] = np.finfo(np.float32).min        # a mask of the type's lowest value
    x[5, 3], x[5, 4] = 1.0, 2.0
    tok[5] = 9
    x[6] = np.finfo(np.float32).min        # nothing but that
    tok[7], tok[8], tok[9] = -1, V, 2**31 - 1
    x[10] = np.nan
    x[11, 0], x[11, 1] = 3e38, -3e38
    tok[11] = 1
    for n in (0, 3, 128):
        run(x, tok, n)
        run(x, tok, n, T=np.float32(np.inf))
        run(x[:, :300], np.minimum(tok, 300), n, T=0.5)


def test_ties():
    rng = np.random.default_rng(9)
    V = 30000
    rows = [np.zeros(V), np.repeat(np.arange(V // 100), 100)[:V], rng.integers(0, 3, V), np.sort(rng.standard_normal(V)),
            np.sort(rng.standard_normal(V))[::-1], np.where(np.arange(V) % 4096 < 16, 1.0, -np.inf), np.where(np.arange(V) < 5000, -0.0, 0.0)]
    x = np.stack(rows).astype(np.float32)
    for n in (1, 20, 128):
        run(x, rng.integers(0, V, len(rows)), n)
        run(x, rng.integers(0, V, len(rows)), n, bf16=True)
    # places that all fall into a few threads' shares, in long rows
    V = 200000
    x = np.full((3, V), -np.inf, np.float32)
    x[0, ::4096] = 1
    x[1, np.arange(V) % 4096 < 512] = rng.integers(0, 2, (np.arange(V) % 4096 < 512).sum())
    x[2, np.arange(V) % 1024 < 256] = 5
    run(x, [4096, 8192, 0], 128)


def test_outputs_may_be_left_out():
    torch, uw = torch_cuda(), _uw()
    M, V, n = 5, 9999, 7
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, V, generator=g, device="cuda")
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    need = uw.logprobs_workspace(M, V, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    f, i = (lambda *s: torch.zeros(*s, device="cuda")), (lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda"))
    outs = {"d_logprob": f(M), "d_rank": i(M), "d_entropy": f(M), "d_top_token": i(M, n), "d_top_logprob": f(M, n)}
    uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws, ws_bytes=need, **outs)
    for name, whole in outs.items():
        alone = torch.zeros_like(whole)
        top = n if "top" in name else 0
        uw.logprobs(x, M, V, d_token=t if name in ("d_logprob", "d_rank") else None, n_top=top, d_ws=ws, ws_bytes=need, **{name: alone})
        assert torch.equal(alone, whole), name


def test_streams_graphs_and_runs():
    torch, uw = torch_cuda(), _uw()
    M, V, n = 4, 32003, 20
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, V, generator=g, device="cuda")
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    need = uw.logprobs_workspace(M, V, n)

    def make():
        return dict(d_logprob=torch.zeros(M, device="cuda"), d_rank=torch.zeros(M, dtype=torch.int32, device="cuda"),
                    d_entropy=torch.zeros(M, device="cuda"), d_top_token=torch.zeros(M, n, dtype=torch.int32, device="cuda"),
                    d_top_logprob=torch.zeros(M, n, device="cuda"))

    a, b = make(), make()
    ws, ws2 = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws, ws_bytes=need, **a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws2, ws_bytes=need, **b)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a[k], b[k]) for k in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws2, ws_bytes=need, **b)
    for _ in range(3):
        x.normal_(generator=g)
        for v in b.values():
            v.zero_()
        ws2.fill_(255)
        uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws, ws_bytes=need, **a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_offsets_past_four_gigabytes():
    torch, uw = torch_cuda(), _uw()
    M, V = 1300, 1 << 20  # 5.5 GB
    x = torch.empty(M, V, device="cuda").normal_()
    t = torch.arange(M, dtype=torch.int32, device="cuda") * 700
    lp, top = torch.zeros(M, device="cuda"), torch.zeros(M, 1, dtype=torch.int32, device="cuda")
    need = uw.logprobs_workspace(M, V, 1)
    ws = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    uw.logprobs(x, M, V, d_token=t, d_logprob=lp, n_top=1, d_top_token=top, d_ws=ws, ws_bytes=need)
    for m in (0, 1023, 1024, M - 1):
        row = x[m].double()
        assert abs(float(row[t[m]] - torch.logsumexp(row, 0)) - float(lp[m])) < 1e-5
        assert int(row.argmax()) == int(top[m])
