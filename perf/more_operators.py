"""4-bit weights, norms around a block, and log probabilities: the calls that are timed, and their plain forms.

Operators (entry points of decode_gemm_amd):
  quantize  w4_quantize and w4_expand: bf16 / fp32 weights to a plane of 4-bit codes with a scale and a
            zero point per group of 32, 64 or 128 values of a row, and back to the values that it stands for
  gemm      w4_gemm: Y = X W^T from such a plane
  gate_up   w4_gate_up: silu(X Wg^T) * (X Wu^T) from two planes
  norm      block_norm: the norm after a block, its gate, the residual and the norm before the next block
  logprobs  logprobs: log probability and rank of a given token per row of logits, the row's entropy and
            its likeliest tokens

A plane: N rows in tiles of 16, K in tiles of 128. First the codes, 1024 bytes for each (row tile, K tile), in that
order: 32-bit word 4 * (16 * q + r) + s holds row r, values 32 * s + 8 * q + (0..7), value e in bits 4 * (e / 2) +
16 * (e % 2). Then a 32-bit word for each (row tile, K tile, group in it, row): an fp32 scale of 20 significant
bits, and in the 4 bits below them the zero point. What lies past N or K is 0.
"""
import math

import numpy as np
import torch

own = False

TINY = 2.0**-126
WORKSPACE = 64 << 20  # bytes of scratch memory that a serving program keeps for these calls


def listed():
    return [
        # the gate matrix of an MLP at load time: codes, and the bf16 weights that a prefill multiplies by
        {"name": "quantize_14336x4096", "op": "quantize", "N": 14336, "K": 4096, "group": 128, "zeros": False, "dtype": "bf16"},
        # a small odd matrix with zero points, checked against its fp32 original
        {"name": "quantize_ragged", "op": "quantize", "N": 1003, "K": 2000, "group": 32, "zeros": True, "dtype": "f32"},
        # one token through the down projection (long K)
        {"name": "gemm_1_down", "op": "gemm", "M": 1, "N": 4096, "K": 14336, "group": 128, "zeros": False, "out": "f32"},
        # odd sizes everywhere, K ends inside a group, small groups with zero points
        {"name": "gemm_5_ragged", "op": "gemm", "M": 5, "N": 5003, "K": 2000, "group": 32, "zeros": True, "out": "bf16"},
        # a decode batch through the gate projection
        {"name": "gemm_64_gate", "op": "gemm", "M": 64, "N": 14336, "K": 4096, "group": 128, "zeros": False, "out": "f32"},
        # one token through gate, up and the activation
        {"name": "gate_up_1", "op": "gate_up", "M": 1, "N": 14336, "K": 4096, "group": 128, "zeros": False},
        # a small decode batch through them, with zero points
        {"name": "gate_up_16", "op": "gate_up", "M": 16, "N": 14336, "K": 4096, "group": 64, "zeros": True},
        # one token's hidden state between two blocks: latency
        {"name": "norm_1x4096", "op": "norm", "M": 1, "K": 4096, "y": "f32", "r": "bf16", "post": "rms", "pre": "rms", "gate": 0, "out": "bf16"},
        # a prefill's, gated per sequence, ending in 8-bit codes for the next product
        {"name": "norm_4096x4096_codes", "op": "norm", "M": 4096, "K": 4096, "y": "f32", "r": "bf16", "post": "rms", "pre": "rms", "gate": 512,
         "out": "codes"},
        # the token just drawn, with the alternatives that an API returns
        {"name": "logprobs_1", "op": "logprobs", "M": 1, "V": 131072, "dtype": "f32", "top": 20, "shape": "peaked"},
        # a decode batch over a vocabulary of odd size
        {"name": "logprobs_64_odd", "op": "logprobs", "M": 64, "V": 50257, "dtype": "bf16", "top": 5, "shape": "flat"},
        # a prompt being scored
        {"name": "logprobs_1024", "op": "logprobs", "M": 1024, "V": 131072, "dtype": "f32", "top": 1, "shape": "peaked"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "gate_up", "norm", "norm", "logprobs", "logprobs"])
    if op in ("quantize", "gemm", "gate_up"):
        while True:
            N, K = _log(rng, 64, 28672), _log(rng, 64, 14336)
            if N * K <= 14336 * 4096:
                break
        c = {"op": op, "N": N, "K": K, "group": rng.choice([32, 64, 128, 128]), "zeros": rng.random() < 0.5}
        if op == "quantize":
            c["dtype"] = rng.choice(["bf16", "f32"])
        else:
            c["M"] = _log(rng, 1, 64)
            if op == "gemm":
                c["out"] = rng.choice(["f32", "bf16"])
        return c
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 64, 8192), "y": rng.choice(["f32", "bf16"]),
                "r": rng.choice(["f32", "bf16"]), "post": rng.choice(["none", "rms", "rms", "layer"]),
                "pre": rng.choice(["none", "rms", "rms", "layer"]), "gate": rng.choice([0, 0, 1, 7, 512]),
                "out": rng.choice(["bf16", "f32", "codes"])}
    return {"op": op, "M": _log(rng, 1, 1024), "V": _log(rng, 1000, 131072), "dtype": rng.choice(["f32", "bf16"]),
            "top": rng.choice([0, 1, 5, 20, 64]), "shape": rng.choice(["peaked", "flat", "masked"])}


def _up(n, m):
    return (n + m - 1) // m * m


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _scale20(v):
    """The nearest number of 20 significant bits, at least 2^-126, of v >= 0 (float64)."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 2.0**20), e - 20).clamp(min=TINY)


def _quantized(w, group, zeros):
    """Codes [N][K / group][group], scales and zero points [N][K / group] of w [N][K]. In 64 bits: quotients next
    to a border between two codes."""
    N, K = w.shape
    g = torch.nn.functional.pad(w.double(), (0, _up(K, group) - K)).view(N, -1, group)
    if zeros:
        lo, hi = g.amin(2).clamp(max=0), g.amax(2).clamp(min=0)
        s = torch.where(hi > lo, _scale20((hi - lo) / 15), 1.0)
        z = torch.round(-lo / s).clamp(0, 15)
    else:
        a = g.abs().amax(2)
        s = torch.where(a > 0, _scale20(a / 7), 1.0)
        z = torch.full_like(s, 8)
    return (torch.round(g / s[..., None]) + z[..., None]).clamp(0, 15).to(torch.int32), s, z


def _plane(q, s, z, N, K, group):
    """The plane of codes, scales and zero points."""
    T, J, per = _up(N, 16) // 16, _up(K, 128) // 128, 128 // group
    pad = torch.nn.functional.pad
    q = torch.where(torch.arange(q.shape[1] * group, device=q.device) < K, q.view(N, -1), 0)
    q = pad(q, (0, J * 128 - q.shape[1], 0, T * 16 - N)).view(T, 16, J, 4, 4, 4, 2)  # t r j s q e/2 e%2
    shift = torch.tensor([[0, 16], [4, 20], [8, 24], [12, 28]], device=q.device)
    word = (q.long() << shift).sum((5, 6)).permute(0, 2, 4, 1, 3)  # t j q r s
    meta = (s.float().view(torch.int32) | z.to(torch.int32)).long()
    meta = pad(meta, (0, J * per - meta.shape[1], 0, T * 16 - N)).view(T, 16, J, per).permute(0, 2, 3, 1)
    both = torch.cat([word.reshape(-1), meta.reshape(-1)])
    return torch.where(both >= 2**31, both - 2**32, both).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)
    op = case["op"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def activations(m, k):
        # token norms that differ, and a few channels that carry far more than the others
        x = randn(m, k) * torch.exp(0.5 * randn(m, 1))
        return x * torch.where(rand(1, k) < 0.01, 20.0, 1.0)

    def rows(x, dtype):
        ld = _up(x.shape[1], 16)  # rows start at 16-byte boundaries
        t = torch.zeros(x.shape[0], ld, device=dev, dtype=dtype)
        t[:, :x.shape[1]] = x
        return t

    def weights(n, k):
        # rows of different sizes, as trained matrices have them
        return 0.02 * randn(n, k) * torch.exp(0.3 * randn(n, 1))

    st = dict(case)
    if op == "quantize":
        N, K = case["N"], case["K"]
        st["x"] = rows(weights(N, K), _dtype(case["dtype"]))
        T, J, per = _up(N, 16) // 16, _up(K, 128) // 128, 128 // case["group"]
        st["plane"] = torch.zeros(T * J * (256 + 16 * per), device=dev, dtype=torch.int32)
        st["back"] = torch.zeros_like(st["x"])
    elif op in ("gemm", "gate_up"):
        M, N, K = case["M"], case["N"], case["K"]
        st["x"] = rows(activations(M, K), torch.bfloat16)
        for n in ("w",) if op == "gemm" else ("wg", "wu"):
            st[n] = _plane(*_quantized(weights(N, K), case["group"], case["zeros"]), N, K, case["group"])
        st["y"] = torch.zeros(M, _up(N, 16), device=dev, dtype=_dtype(case.get("out", "bf16")))
        st["ws"] = torch.empty(WORKSPACE, device=dev, dtype=torch.uint8)
    elif op == "norm":
        M, K = case["M"], case["K"]
        st["y"] = rows(3 * activations(M, K), _dtype(case["y"]))
        st["r"] = rows(activations(M, K), _dtype(case["r"]))
        st["r2"] = torch.zeros_like(st["r"])
        vec = lambda n, base: rows(base + 0.2 * randn(n, K), torch.bfloat16)  # noqa: E731
        for n in ("post", "pre"):
            st[n + "_w"] = vec(1, 1.0) if case[n] != "none" else None
            st[n + "_b"] = vec(1, 0.0) if case[n] == "layer" else None
        st["gates"] = vec(-(-M // case["gate"]), 1.0) if case["gate"] else None  # one row per sequence of `gate` tokens
        if case["out"] == "codes":
            st["q"] = torch.zeros(M, _up(K, 16), device=dev, dtype=torch.uint8)
            st["s"] = torch.zeros(_up(K, 128) // 128, M, device=dev)
        else:
            st["h"] = torch.zeros(M, _up(K, 16), device=dev, dtype=_dtype(case["out"]))
    else:
        M, V = case["M"], case["V"]
        if case["shape"] == "flat":
            x = 1.5 * randn(M, V)
        else:
            # a wide body of unlikely tokens, and about one in 500 that the text makes likely
            x = 2.0 * randn(M, V) + torch.where(rand(M, V) < 0.002, 4.0 + 6.0 * rand(M, V), 0.0)
        if case["shape"] == "masked":
            # a grammar leaves one token in twenty
            x = torch.where(rand(M, V) < 0.05, x, -math.inf)
        st["x"] = x.to(_dtype(case["dtype"]))
        # the token: mostly one that the row makes likely, sometimes any (a prompt's)
        likely = (x - torch.log(-torch.log(rand(M, V).clamp(min=1e-30, max=1 - 1e-7)))).argmax(1)
        st["token"] = torch.where(rand(M) < 0.8, likely, (rand(M) * V).long().clamp(max=V - 1)).to(torch.int32)
        t = torch.tensor([1.0] if M == 1 else [0.6, 1.0, 1.0, 1.3], device=dev)
        st["temperature"] = t[torch.randint(0, len(t), (M,), generator=g, device=dev)]
        st["logprob"], st["entropy"] = torch.zeros(M, device=dev), torch.zeros(M, device=dev)
        st["rank"] = torch.zeros(M, device=dev, dtype=torch.int32)
        st["top_token"] = torch.zeros(M, case["top"], device=dev, dtype=torch.int32)
        st["top_logprob"] = torch.zeros(M, case["top"], device=dev)
        st["ws"] = torch.empty(WORKSPACE, device=dev, dtype=torch.uint8)
    return st


def _values(plane, N, K, group):
    """The values [N][K] that a plane stands for, in 32 bits (exact)."""
    T, J, per = _up(N, 16) // 16, _up(K, 128) // 128, 128 // group
    word, meta = plane[:T * J * 256].view(T, J, 4, 16, 4), plane[T * J * 256:].view(T, J, per, 16)
    q = torch.stack([(word >> b) & 15 for b in (0, 16, 4, 20, 8, 24, 12, 28)], 5)  # t j q r s e
    q = q.permute(0, 3, 1, 4, 2, 5).reshape(T * 16, J * per, group)
    m = meta.permute(0, 3, 1, 2).reshape(T * 16, J * per)
    s, z = (m & ~15).view(torch.float32), m & 15
    return ((q - z[..., None]).float() * s[..., None]).view(T * 16, J * 128)[:N, :K]


def _run_quantize(st):
    N, K, ld = st["N"], st["K"], st["x"].stride(0)
    if own:
        import decode_gemm_amd as uw

        uw.w4_quantize(st["x"], st["plane"], N, K, group=st["group"], zeros=st["zeros"], ldw=ld)
        uw.w4_expand(st["plane"], st["back"], N, K, group=st["group"], ldw=ld)
        return st["back"][:, :K]
    q, s, z = _quantized(st["x"][:, :K], st["group"], st["zeros"])
    v = (q - z[..., None]) * s[..., None]
    return v.view(N, -1)[:, :K].to(st["x"].dtype)


def _run_gemm(st):
    M, N, K = st["M"], st["N"], st["K"]
    if own:
        import decode_gemm_amd as uw

        uw.w4_gemm(st["x"], st["w"], st["y"], M, N, K, group=st["group"], ldx=st["x"].stride(0), ldy=st["y"].stride(0),
                   d_ws=st["ws"], ws_bytes=WORKSPACE)
        return st["y"][:, :N]
    return (st["x"][:, :K].float() @ _values(st["w"], N, K, st["group"]).t()).to(st["y"].dtype)


def _run_gate_up(st):
    M, N, K = st["M"], st["N"], st["K"]
    if own:
        import decode_gemm_amd as uw

        uw.w4_gate_up(st["x"], st["wg"], st["wu"], st["y"], M, N, K, group=st["group"], ldx=st["x"].stride(0),
                      ldh=st["y"].stride(0), d_ws=st["ws"], ws_bytes=WORKSPACE)
        return st["y"][:, :N]
    x = st["x"][:, :K].float()
    a, b = (x @ _values(st[n], N, K, st["group"]).t() for n in ("wg", "wu"))
    return (a / (1 + torch.exp(-a)) * b).to(st["y"].dtype)


EPS = 1e-6
KEEP = 0.9  # what stays of the residual stream where a block is added
ADD = 0.5   # of the block


def _normed(v, kind, w, b, K):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w[:, :K].float() + b[:, :K].float()
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w[:, :K].float()


def _run_norm(st):
    M, K = st["M"], st["K"]
    if own:
        import decode_gemm_amd as uw

        kinds = {"none": uw.NORM_NONE, "rms": uw.NORM_RMS, "layer": uw.NORM_LAYER}
        uw.block_norm(st["y"], st["r"], st["r2"], M, K, d_h=st.get("h"), d_q=st.get("q"), d_s=st.get("s"),
                      post=kinds[st["post"]], d_post_w=st["post_w"], d_post_b=st["post_b"], pre=kinds[st["pre"]],
                      d_pre_w=st["pre_w"], d_pre_b=st["pre_b"], d_gate=st["gates"], gate_rows=st["gate"],
                      ldgate=_up(K, 16), scale_y=ADD, scale_r=KEEP, eps=EPS, ldy=_up(K, 16), ldr=_up(K, 16),
                      ldr_out=_up(K, 16), ldh=_up(K, 16))
        if st["out"] == "codes":
            return st["r2"][:, :K], st["q"].view(torch.float8_e4m3fn)[:, :K], st["s"]
        return st["r2"][:, :K], st["h"][:, :K]
    v = _normed(st["y"][:, :K].float(), st["post"], st["post_w"], st["post_b"], K)
    if st["gate"]:
        v = v * st["gates"][:, :K].float().repeat_interleave(st["gate"], 0)[:M]
    r = KEEP * st["r"][:, :K].float() + ADD * v
    h = _normed(r, st["pre"], st["pre_w"], st["pre_b"], K)
    if st["out"] != "codes":
        return r.to(st["r"].dtype), h.to(st["h"].dtype)
    p = torch.nn.functional.pad(h, (0, _up(K, 128) - K)).view(M, -1, 128)
    a = p.abs().amax(2)
    s = torch.where(a == 0, 1.0, (a / 448).clamp(min=TINY))
    q = (p / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(M, -1)[:, :K]
    return r.to(st["r"].dtype), q, s.t().contiguous()


def _run_logprobs(st):
    M, V = st["x"].shape
    n = st["top"]
    if own:
        import decode_gemm_amd as uw

        uw.logprobs(st["x"], M, V, d_token=st["token"], d_logprob=st["logprob"], d_rank=st["rank"], d_entropy=st["entropy"],
                    n_top=n, d_top_token=st["top_token"], d_top_logprob=st["top_logprob"], d_temperature=st["temperature"],
                    d_ws=st["ws"], ws_bytes=WORKSPACE)
        return st["logprob"], st["rank"], st["entropy"], st["top_token"], st["top_logprob"]
    x, t = st["x"], st["token"].long()[:, None]
    # in 64 bits: long sums, and differences of a logarithm and what is next to it
    y = x.double() / st["temperature"].double()[:, None]
    y = y - y.amax(1, keepdim=True)
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    lse = torch.log(total)
    entropy = lse - torch.where(e > 0, y * e, 0.0).sum(1, keepdim=True) / total
    l = x.gather(1, t)
    before = ((x > l) | ((x == l) & (torch.arange(V, device=x.device) < t))).sum(1, keepdim=True)
    rank = torch.where(l > -math.inf, before, -1)[:, 0].to(torch.int32)
    if n == 0:
        top, at = y[:, :0], t[:, :0]
    elif n == 1:
        top, at = y.max(1, keepdim=True)[0], (x == x.amax(1, keepdim=True)).int().argmax(1, keepdim=True)
    else:
        at = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :n]
        top = y.gather(1, at)
    at = torch.where(top > -math.inf, at, -1)
    return ((y.gather(1, t) - lse)[:, 0].float(), rank, entropy[:, 0].float(), at.to(torch.int32), (top - lse).float())


def run(state):
    return {"quantize": _run_quantize, "gemm": _run_gemm, "gate_up": _run_gate_up, "norm": _run_norm,
            "logprobs": _run_logprobs}[state["op"]](state)


def work(case):
    op = case["op"]
    size = lambda name: {"f32": 4, "bf16": 2, "codes": 1}[name]  # noqa: E731
    if op in ("quantize", "gemm", "gate_up"):
        N, K = case["N"], case["K"]
        plane = N * K // 2 + 4 * N * (_up(K, case["group"]) // case["group"])
        if op == "quantize":
            # the weights read, the plane written and read, the values written
            return {"bytes": 2 * N * K * size(case["dtype"]) + 2 * plane, "flops": 6 * N * K}
        M, two = case["M"], 2 if op == "gate_up" else 1
        return {"bytes": two * plane + 2 * M * K + M * N * size(case.get("out", "bf16")), "flops": 2 * two * M * N * K}
    if op == "norm":
        M, K = case["M"], case["K"]
        n = size(case["y"]) + 2 * size(case["r"]) + size(case["out"])
        return {"bytes": M * K * n + (4 * M * (_up(K, 128) // 128) if case["out"] == "codes" else 0), "flops": 12 * M * K}
    M, V = case["M"], case["V"]
    return {"bytes": M * (V * size(case["dtype"]) + 20 + 8 * case["top"]), "flops": 6 * M * V}


def _exact_quantize(st):
    x, group = st["x"][:, :st["K"]].double(), st["group"]
    out = torch.empty_like(x)

    def short(v):  # to 20 significant bits
        unit = torch.exp2(torch.floor(torch.log2(v.clamp(min=1e-300))) - 19)
        return (torch.round(v / unit) * unit).clamp(min=2.0**-126)

    for k in range(0, st["K"], group):
        w = x[:, k:k + group]
        if st["zeros"]:
            top, low = w.max(1, keepdim=True)[0].clamp(min=0), w.min(1, keepdim=True)[0].clamp(max=0)
            s = short((top - low) / 15)
            z = torch.round(-low / s)
            q = torch.minimum(torch.maximum(torch.round(w / s), -z), 15 - z)
        else:
            s = short(w.abs().max(1, keepdim=True)[0] / 7)
            q = torch.round(w / s).clamp(-8, 7)
        out[:, k:k + group] = q * s
    return out


def _exact_weights(plane, N, K, group):
    """Value by value from its place in the plane."""
    n, k = torch.arange(N, device=plane.device)[:, None], torch.arange(K, device=plane.device)[None, :]
    J, per = -(-K // 128), 128 // group
    tile = torch.div(n, 16, rounding_mode="floor") * J + torch.div(k, 128, rounding_mode="floor")
    in_tile = k % 128
    word = plane[tile * 256 + 4 * (16 * torch.div(in_tile % 32, 8, rounding_mode="floor") + n % 16)
                 + torch.div(in_tile, 32, rounding_mode="floor")]
    e = k % 8
    q = (word >> (4 * torch.div(e, 2, rounding_mode="floor") + 16 * (e % 2))) & 15
    meta = plane[-(-N // 16) * J * 256 + (tile * per + torch.div(in_tile, group, rounding_mode="floor")) * 16 + n % 16]
    return (meta & -16).view(torch.float32).double() * (q - (meta & 15)).double()


def _exact_norm(st):
    M, K, f = st["M"], st["K"], torch.float64

    def norm(v, kind, w, b):
        if kind == "none":
            return v
        if kind == "rms":
            return w[0, :K].to(f) * v * torch.rsqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True)**2 / K + EPS)
        mean = v.sum(1, keepdim=True) / K
        var = ((v - mean)**2).sum(1, keepdim=True) / K
        return w[0, :K].to(f) * (v - mean) * torch.rsqrt(var + EPS) + b[0, :K].to(f)

    branch = norm(st["y"][:, :K].to(f), st["post"], st["post_w"], st["post_b"])
    if st["gate"]:
        branch = branch * st["gates"][torch.arange(M, device=branch.device) // st["gate"], :K].to(f)
    r = st["r"][:, :K].to(f) * KEEP + branch * ADD
    h = norm(r, st["pre"], st["pre_w"], st["pre_b"])
    if st["out"] != "codes":
        return r, h
    q, scales = torch.empty_like(h), []
    for k in range(0, K, 128):
        part = h[:, k:k + 128]
        a = part.abs().amax(1)
        s = torch.where(a > 0, torch.maximum(a / 448.0, torch.full_like(a, 2.0**-126)), torch.ones_like(a))
        v = part / s[:, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0**-9))).clamp(min=-6) - 3)
        q[:, k:k + 128] = torch.round(v / step) * step
        scales.append(s)
    return r, q, torch.stack(scales)


def _exact_logprobs(st):
    """Row by row; ranks and tokens are whole numbers and stand in run()."""
    n, M = st["top"], st["x"].shape[0]
    T, token = st["temperature"].double().cpu().numpy(), st["token"].cpu().numpy()
    lp, ent, top = np.zeros(M), np.zeros(M), np.full((M, n), -math.inf)
    for m in range(M):
        l = st["x"][m].double() / float(T[m])
        l = torch.sort(l[l > -math.inf])[0]
        peak = l[-1]
        p = torch.exp(l - peak)
        total = p.sum()
        log_total = peak + torch.log1p(total - 1)
        lp[m] = float(st["x"][m, int(token[m])].double() / float(T[m]) - log_total)
        ent[m] = float(((log_total - l) * p).sum() / total)
        best = (l[-n:].flip(0) if n else l[:0]) - log_total
        top[m, :best.numel()] = best.cpu().numpy()
    return lp, None, ent, None, top


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(st)
    if op == "norm":
        return _exact_norm(st)
    if op == "logprobs":
        return _exact_logprobs(st)
    N, K, x = case["N"], case["K"], st["x"][:, :case["K"]].double()
    if op == "gemm":
        return x @ _exact_weights(st["w"], N, K, case["group"]).t()
    a = x @ _exact_weights(st["wg"], N, K, case["group"]).t()
    return a * torch.sigmoid(a) * (x @ _exact_weights(st["wu"], N, K, case["group"]).t())
