"""The 8-bit block-scaled path and token sampling: the calls that are timed, and their plain forms.

Operators (entry points of decode_gemm_amd):
  quantize  fp8_quantize: bf16 / fp32 to e4m3 codes with one fp32 scale per 128 values of a row
            (activations) or per 128 x 128 block (weights)
  swiglu    fp8_swiglu: silu(g) * u of a gate/up product, written as e4m3 codes and scales
  gemm      fp8_gemm: Y = X W^T from codes and scales
  sample    sample: one token per row of logits, with temperature, top-k, top-p and min-p, from
            given uniform numbers

Scales of rows are stored group-major ([K / 128][M]), those of weights block-row-major
([N / 128][K / 128]).
"""
import math

import numpy as np
import torch

own = False

G = 128         # values per scale
TOP = 448.0     # largest e4m3 value
TINY = 2.0**-126
WORKSPACE = 64 << 20  # bytes of scratch memory that a serving program keeps for these calls


def listed():
    return [
        # one token's hidden state before a projection: latency
        {"name": "quantize_1x4096", "op": "quantize", "M": 1, "K": 4096, "rows": 1, "dtype": "bf16"},
        # hidden states of a prefill
        {"name": "quantize_4096x4096", "op": "quantize", "M": 4096, "K": 4096, "rows": 1, "dtype": "bf16"},
        # the gate matrix of an MLP, decoded to bf16, at load time
        {"name": "quantize_weight_14336x4096", "op": "quantize", "M": 14336, "K": 4096, "rows": 128, "dtype": "bf16"},
        # the activation of a decode batch between up and down
        {"name": "swiglu_64x14336", "op": "swiglu", "M": 64, "K": 14336},
        # the same of a prefill
        {"name": "swiglu_4096x14336", "op": "swiglu", "M": 4096, "K": 14336},
        # one token through the gate projection
        {"name": "gemm_1_gate", "op": "gemm", "M": 1, "N": 14336, "K": 4096, "out": "f32"},
        # a decode batch through the down projection (long K)
        {"name": "gemm_64_down", "op": "gemm", "M": 64, "N": 4096, "K": 14336, "out": "f32"},
        # odd sizes everywhere: a short prefill of an unpadded model, K ends inside a block
        {"name": "gemm_333_ragged", "op": "gemm", "M": 333, "N": 5003, "K": 2000, "out": "bf16"},
        # a prefill through the gate projection
        {"name": "gemm_4096_gate", "op": "gemm", "M": 4096, "N": 14336, "K": 4096, "out": "bf16"},
        # the next token of one request
        {"name": "sample_1", "op": "sample", "M": 1, "V": 131072, "dtype": "f32", "shape": "peaked"},
        # a decode batch over a vocabulary of odd size
        {"name": "sample_64_odd", "op": "sample", "M": 64, "V": 50257, "dtype": "f32", "shape": "flat"},
        # many requests, a large vocabulary, every kind of setting among the rows
        {"name": "sample_256", "op": "sample", "M": 256, "V": 131072, "dtype": "f32", "shape": "peaked"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "swiglu", "gemm", "gemm", "sample", "sample"])
    if op == "quantize":
        rows = rng.choice([1, 1, 128])
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 64, 14336), "rows": rows,
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "swiglu":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 64, 14336)}
    if op == "gemm":
        while True:
            c = {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 28672), "K": _log(rng, 64, 14336),
                 "out": rng.choice(["f32", "bf16"])}
            if c["N"] * c["K"] <= 14336 * 4096:
                return c
    return {"op": op, "M": _log(rng, 1, 256), "V": _log(rng, 1000, 131072), "dtype": rng.choice(["f32", "bf16"]),
            "shape": rng.choice(["peaked", "flat", "masked"])}


def _up(n, m):
    return (n + m - 1) // m * m


def _codes(x, s):
    """e4m3 codes of x / s, rounded to nearest even, held at the largest value."""
    return (x / s).clamp(-TOP, TOP).to(torch.float8_e4m3fn)


def _scale(a):
    return torch.where(a == 0, torch.ones_like(a), (a / TOP).clamp(min=TINY))


def _quantize_plain(x, rows):
    """Codes [M][K] and scales ([K / 128][M] for rows, [M / 128][K / 128] for blocks) of x in fp32."""
    M, K = x.shape
    mb, kb = _up(M, rows) // rows, _up(K, G) // G
    p = torch.nn.functional.pad(x, (0, kb * G - K, 0, mb * rows - M)).view(mb, rows, kb, G)
    s = _scale(p.abs().amax(dim=(1, 3)))
    q = _codes(p, s[:, None, :, None]).view(mb * rows, kb * G)[:M, :K]
    return q, s.t().contiguous() if rows == 1 else s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    op, M = case["op"], case["M"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def activations(m, k):
        # token norms that differ, and a few channels that carry far more than the others
        x = randn(m, k) * torch.exp(0.5 * randn(m, 1))
        return x * torch.where(rand(1, k) < 0.01, 20.0, 1.0)

    st = dict(case)
    if op == "quantize":
        K, rows = case["K"], case["rows"]
        x = activations(M, K) if rows == 1 else 0.02 * randn(M, K)
        ld = _up(K, 16)  # rows start at 16-byte boundaries
        st["x"] = torch.zeros(M, ld, device=dev, dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        st["x"][:, :K] = x
        st["q"] = torch.zeros(M, ld, device=dev, dtype=torch.uint8)
        kb = _up(K, G) // G
        st["s"] = torch.zeros((kb, M) if rows == 1 else (_up(M, G) // G, kb), device=dev)
    elif op == "swiglu":
        K = case["K"]
        ld = _up(K, 16)
        st["y"] = randn(M, 2 * ld) * torch.exp(0.5 * randn(M, 1))  # gate and up, side by side as one product leaves them
        st["q"] = torch.zeros(M, ld, device=dev, dtype=torch.uint8)
        st["s"] = torch.zeros(_up(K, G) // G, M, device=dev)
    elif op == "gemm":
        N, K = case["N"], case["K"]
        ld = _up(K, 16)
        for n, v, rows in (("x", activations(M, K), 1), ("w", 0.02 * randn(N, K), G)):
            q, s = _quantize_plain(v, rows)
            st[n] = torch.zeros(q.shape[0], ld, device=dev, dtype=torch.uint8)
            st[n][:, :K] = q.view(torch.uint8)
            st["s" + n] = s
        st["out"] = torch.zeros(M, N, device=dev, dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
        st["ws"] = torch.empty(WORKSPACE, device=dev, dtype=torch.uint8)
    else:
        V = case["V"]
        if case["shape"] == "flat":
            x = 1.5 * randn(M, V)
        else:
            # a wide body of unlikely tokens, and about one in 500 that the text makes likely
            x = 2.0 * randn(M, V) + torch.where(rand(M, V) < 0.002, 4.0 + 6.0 * rand(M, V), 0.0)
        if case["shape"] == "masked":
            # a grammar leaves one token in twenty
            x = torch.where(rand(M, V) < 0.05, x, -math.inf)
        st["x"] = x.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        one = M == 1
        # the settings that requests come with; 0, 0, 1 and 0 leave the four steps out
        def choice(values):
            v = torch.tensor(values, device=dev)
            return v[torch.randint(0, len(values), (M,), generator=g, device=dev)]
        st["temperature"] = choice([0.7] if one else [0.0, 0.6, 0.7, 1.0, 1.0, 1.3])
        st["top_k"] = choice([50] if one else [0, 0, 1, 20, 50, 200]).to(torch.int32)
        st["top_p"] = choice([0.95] if one else [1.0, 1.0, 0.8, 0.9, 0.95])
        st["min_p"] = choice([0.0, 0.0, 0.02, 0.1])
        st["u"] = rand(M)
        st["token"] = torch.zeros(M, device=dev, dtype=torch.int32)
        st["prob"] = torch.zeros(M, device=dev)
        st["ws"] = torch.empty(WORKSPACE, device=dev, dtype=torch.uint8)
    return st


def _floats(q):
    return q.view(torch.float8_e4m3fn)


def _spread(s, rows, cols, m, k):
    """Scales repeated over the rows x cols values that each stands for, cut to m x k."""
    return s.repeat_interleave(rows, 0)[:m].repeat_interleave(cols, 1)[:, :k]


def _run_quantize(st):
    M, K = st["M"], st["K"]
    if own:
        import decode_gemm_amd as uw

        uw.fp8_quantize(st["x"], st["q"], st["s"], M, K, block_rows=st["rows"], ldx=st["x"].stride(0), ldq=st["q"].stride(0))
        return _floats(st["q"])[:, :K], st["s"]
    return _quantize_plain(st["x"][:, :K].float(), st["rows"])


def _run_swiglu(st):
    M, K = st["M"], st["K"]
    half = st["y"].shape[1] // 2
    if own:
        import decode_gemm_amd as uw

        uw.fp8_swiglu(st["y"], st["y"][:, half:], st["q"], st["s"], M, K, ldg=2 * half, ldu=2 * half, ldq=st["q"].stride(0))
        return _floats(st["q"])[:, :K], st["s"]
    gate, up = st["y"][:, :K], st["y"][:, half:half + K]
    return _quantize_plain(gate / (1 + torch.exp(-gate)) * up, 1)


def _run_gemm(st):
    M, N, K = st["M"], st["N"], st["K"]
    if own:
        import decode_gemm_amd as uw

        uw.fp8_gemm(st["x"], st["sx"], st["w"], st["sw"], st["out"], M, N, K, ldx=st["x"].stride(0), ldw=st["w"].stride(0),
                    d_ws=st["ws"], ws_bytes=WORKSPACE)
        return st["out"]
    x = _floats(st["x"])[:, :K].float() * _spread(st["sx"].t(), 1, G, M, K)
    w = _floats(st["w"])[:, :K].float() * _spread(st["sw"], G, G, N, K)
    return (x @ w.t()).to(st["out"].dtype)


def _run_sample(st):
    M, V = st["x"].shape
    if own:
        import decode_gemm_amd as uw

        uw.sample(st["x"], st["u"], st["token"], M, V, d_temperature=st["temperature"], d_top_k=st["top_k"],
                  d_top_p=st["top_p"], d_min_p=st["min_p"], d_prob=st["prob"], d_ws=st["ws"], ws_bytes=WORKSPACE)
        return st["token"], st["prob"]
    # in 64 bits: the sums over a vocabulary decide which token a number falls on
    v, at = torch.sort(st["x"].double(), dim=1, descending=True, stable=True)
    t = st["temperature"].double()[:, None]
    d = v - v[:, :1]
    w = torch.where(v == -math.inf, 0.0, torch.exp(d / torch.where(t > 0, t, 1.0)))
    first = torch.arange(V, device=v.device)[None, :]
    k = torch.where(st["temperature"] > 0, st["top_k"], 1)[:, None]
    w = torch.where((k > 0) & (first >= k), 0.0, w)
    p = st["top_p"].double()[:, None]
    c = torch.cumsum(w, 1)
    w = torch.where((p < 1) & (first > 0) & (c - w >= p * c[:, -1:]), 0.0, w)
    w = torch.where(w < st["min_p"].double()[:, None], 0.0, w)
    c = torch.cumsum(w, 1)
    total = c[:, -1:]
    j = (c <= st["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    some = total[:, 0] > 0
    token = torch.where(some, at.gather(1, j)[:, 0], -1).to(torch.int32)
    prob = torch.where(some, (w.gather(1, j) / total)[:, 0], 0.0).float()
    return token, prob


def run(state):
    return {"quantize": _run_quantize, "swiglu": _run_swiglu, "gemm": _run_gemm, "sample": _run_sample}[state["op"]](state)


def work(case):
    op, M = case["op"], case["M"]
    if op == "quantize":
        n = M * case["K"]
        s = (_up(M, case["rows"]) // case["rows"]) * (_up(case["K"], G) // G)
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + 4 * s, "flops": 4 * n}
    if op == "swiglu":
        n = M * case["K"]
        return {"bytes": 9 * n + 4 * M * (_up(case["K"], G) // G), "flops": 10 * n}
    if op == "gemm":
        N, K = case["N"], case["K"]
        kb = _up(K, G) // G
        y = 4 if case["out"] == "f32" else 2
        return {"bytes": M * K + N * K + y * M * N + 4 * kb * (M + _up(N, G) // G), "flops": 2 * M * N * K}
    return {"bytes": M * (case["V"] * (4 if case["dtype"] == "f32" else 2) + 28), "flops": 4 * M * case["V"]}


def _round_e4m3(v):
    """v (float64, |v| <= 448) rounded to the e4m3 grid, ties to even: steps of 2^(e - 3), e from -6 up."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0**-9))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_codes(x, rows):
    M, K = x.shape
    kb = -(-K // G)
    mb = -(-M // rows)
    a = torch.zeros(mb, kb, dtype=torch.float64, device=x.device)
    for j in range(kb):
        part = x[:, j * G:(j + 1) * G].abs().amax(1)
        full = torch.zeros(mb * rows, dtype=torch.float64, device=x.device)
        full[:M] = part
        a[:, j] = full.view(mb, rows).amax(1)
    s = torch.where(a > 0, torch.maximum(a / TOP, torch.full_like(a, TINY)), torch.ones_like(a))
    q = torch.empty_like(x)
    for j in range(kb):
        sj = s[:, j].repeat_interleave(rows)[:M, None]
        q[:, j * G:(j + 1) * G] = _round_e4m3(x[:, j * G:(j + 1) * G] / sj)
    return q, s.t().contiguous() if rows == 1 else s


def _exact_gemm(st):
    M, N, K = st["M"], st["N"], st["K"]
    x, w = _floats(st["x"]).double(), _floats(st["w"]).double()
    y = torch.zeros(M, N, dtype=torch.float64, device=x.device)
    for b in range(-(-K // G)):
        k0, k1 = b * G, min(K, (b + 1) * G)
        sw = st["sw"][:, b].double().repeat_interleave(G)[:N]
        y += (x[:, k0:k1] @ w[:, k0:k1].t()) * st["sx"][b].double()[:, None] * sw[None, :]
    return y


def _exact_sample(st):
    """The probabilities of the tokens drawn, row by row on the host; tokens are whole numbers and stand in run()."""
    x = st["x"].double().cpu().numpy()
    rows = {n: st[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "u")}
    prob = np.zeros(x.shape[0])
    for m, l in enumerate(x):
        T, k, p, least, u = (float(rows[n][m]) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        ids = np.flatnonzero(l > -math.inf)
        if not ids.size:
            continue
        ids = ids[np.lexsort((ids, -l[ids]))]
        if T <= 0:
            prob[m] = 1.0
            continue
        if 0 < k < ids.size:
            ids = ids[:int(k)]
        w = np.exp((l[ids] - l[ids[0]]) / T)
        if p < 1:
            before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
            w = w[:max(1, int(np.count_nonzero(before < p * w.sum())))]
        w = w[w >= least]
        c = np.cumsum(w)
        prob[m] = w[min(int(np.searchsorted(c, u * c[-1], side="right")), w.size - 1)] / c[-1]
    return prob


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_codes(st["x"][:, :case["K"]].double(), case["rows"])
    if op == "swiglu":
        K, half = case["K"], st["y"].shape[1] // 2
        a, b = st["y"][:, :K].double(), st["y"][:, half:half + K].double()
        return _exact_codes(a * torch.sigmoid(a) * b, 1)
    if op == "gemm":
        return _exact_gemm(st)
    return None, _exact_sample(st)
