"""One decoding step through 4-bit weights, as the calls are used together: norm, gate and up with SwiGLU, down, the norm after the
block with the residual and the norm before the next, the output projection, a token drawn and its log probability; and the
prompt's way, the weights expanded to bf16 for the plain GEMM.

Each stage is checked on what the stage before it gave (its inputs read back), so tolerances are those of single calls: norms
and log probabilities as in their own tests (bounds of 64 and 200 half steps of fp32 here, of what is summed), products a
bf16 rounding or, in fp32, (4 group + groups + 22) 2^-23 of 16 s |x| summed. The drawn token's probability comes from a 64-bit sum (within 1e-12) and the log
probability within 1e-5 of it.
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda
from tests.test_gpu_w4 import _tolerance, plane_of, put_plane, quantized, values_of

pytestmark = pytest.mark.gpu

U = 2.0**-24


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


class Model:
    """A block and an output projection with 4-bit weights, their planes and their values in 64 bits."""

    def __init__(self, rng, K, F, V, group, zeros):
        self.K, self.F, self.V, self.group = K, F, V, group
        self.w, self.s, self.plane = {}, {}, {}
        for name, n, k in (("gate", F, K), ("up", F, K), ("down", K, F), ("head", V, K)):
            q, s, z = quantized((rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float32), group, zeros)
            self.w[name], self.s[name], self.plane[name] = values_of(q, s, z, k), s, put_plane(plane_of(q, s, z, n, k, group))


def _f64(t):
    return t.double().cpu().numpy()


def _rms(v, w):
    return v / np.sqrt((v * v).mean(1, keepdims=True) + 1e-6) * w


@pytest.mark.parametrize("M,K,F,V,group,zeros", [(1, 512, 1536, 5003, 128, False), (5, 512, 1000, 5003, 32, True), (33, 256, 768, 1999, 64, True)])
def test_step(M, K, F, V, group, zeros):
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M + K)
    model = Model(rng, K, F, V, group, zeros)
    b16 = torch.bfloat16
    w1, w2, w3 = (torch.from_numpy(1 + 0.2 * rng.standard_normal(K)).to("cuda", b16) for _ in range(3))
    res = torch.from_numpy(rng.standard_normal((M, K))).to("cuda", b16)
    u = torch.from_numpy(rng.random(M).astype(np.float32)).to("cuda")
    x, h2 = torch.zeros(M, K, dtype=b16, device="cuda"), torch.zeros(M, K, dtype=b16, device="cuda")
    res2 = torch.zeros_like(res)
    ldf = (F + 7) // 8 * 8
    h = torch.zeros(M, ldf, dtype=b16, device="cuda")
    y, logits = torch.zeros(M, K, device="cuda"), torch.zeros(M, V, device="cuda")
    token, rank = (torch.zeros(M, dtype=torch.int32, device="cuda") for _ in range(2))
    prob, lp, ent = (torch.zeros(M, device="cuda") for _ in range(3))
    tops, top_lp = torch.zeros(M, 4, dtype=torch.int32, device="cuda"), torch.zeros(M, 4, device="cuda")
    need = max(16, uw.w4_gemm_workspace(M, K, F), uw.w4_gemm_workspace(M, 2 * F, K), uw.w4_gemm_workspace(M, V, K), uw.sample_workspace(M, V),
               uw.logprobs_workspace(M, V, 4))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    space = dict(d_ws=ws, ws_bytes=need)

    def step():
        uw.block_norm(None, res, None, M, K, d_h=x, d_pre_w=w1)
        uw.w4_gate_up(x, model.plane["gate"], model.plane["up"], h, M, F, K, group=group, ldh=ldf, **space)
        uw.w4_gemm(h, model.plane["down"], y, M, K, F, group=group, ldx=ldf, **space)
        uw.block_norm(y, res, res2, M, K, d_h=h2, d_post_w=w2, d_pre_w=w3, scale_y=0.5)
        uw.w4_gemm(h2, model.plane["head"], logits, M, V, K, group=group, **space)
        uw.sample(logits, u, token, M, V, d_prob=prob, **space)
        uw.logprobs(logits, M, V, d_token=token, d_logprob=lp, d_rank=rank, d_entropy=ent, n_top=4, d_top_token=tops, d_top_logprob=top_lp, **space)

    step()
    torch.cuda.synchronize()
    log(f"  step of {M} rows, {K} / {F} / {V}, group {group}")

    def close(got, want, tol, what):
        bad = np.abs(_f64(got) - want) > tol + 2.0**-133
        assert not bad.any(), f"{what}: {bad.sum()} off"

    want = _rms(_f64(res), _f64(w1))
    close(x, want, np.abs(want) * (2.0**-8 + 64 * U), "first norm")
    g, p = (_f64(x) @ model.w[n].T for n in ("gate", "up"))
    tg, tp = (_tolerance(_f64(x), model.s[n], K, group) for n in ("gate", "up"))
    sig = 1 / (1 + np.exp(-g))
    close(h[:, :F], g * sig * p, np.abs(g * sig * p) * (2.0**-8 + 8 * U) + 1.1 * tg * (np.abs(p) + tp) + np.abs(g * sig) * tp, "gate and up")
    close(y, _f64(h[:, :F]) @ model.w["down"].T, _tolerance(_f64(h[:, :F]), model.s["down"], F, group), "down")
    r = _f64(res) + 0.5 * _rms(_f64(y), _f64(w2))
    near = 64 * U * (np.abs(_f64(res)) + np.abs(r - _f64(res)))
    close(res2, r, near + np.abs(r) * 2.0**-8, "residual")
    want = _rms(r, _f64(w3))
    close(h2, want, np.abs(want) * (2.0**-8 + 200 * U) + near * np.abs(want / r), "second norm")
    close(logits, _f64(h2) @ model.w["head"].T, _tolerance(_f64(h2), model.s["head"], K, group), "logits")
    l = _f64(logits)
    at = token.cpu().numpy()
    share = l - np.log(np.exp(l - l.max(1, keepdims=True)).sum(1, keepdims=True)) - l.max(1, keepdims=True)
    assert np.abs(_f64(lp) - share[np.arange(M), at]).max() < 1e-5
    assert np.abs(np.exp(_f64(lp)) - _f64(prob)).max() < 1e-5
    order = np.argsort(-l, axis=1, kind="stable")
    assert (rank.cpu().numpy() == [int(np.flatnonzero(order[m] == at[m])[0]) for m in range(M)]).all()
    assert (tops.cpu().numpy() == order[:, :4]).all()

    # captured and replayed, the step gives what it gave
    first = [t.clone() for t in (x, h, y, res2, h2, logits, token, prob, lp, rank, ent, tops, top_lp)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (x, h2, y, res2, logits, token, prob, lp, rank, ent, tops, top_lp):
            t.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (x, h, y, res2, h2, logits, token, prob, lp, rank, ent, tops, top_lp)))


@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (200, 320, 1024)])
def test_the_way_of_a_prompt(M, N, K):
    """Expanded weights through the plain GEMM give the product of the same values, each rounded to bf16 (half a step, 2^-8 of
    |x w| at most), within the plain GEMM's 1e-3 of sum |x w|."""
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(M)
    q, s, z = quantized((0.02 * rng.standard_normal((N, K))).astype(np.float32), 128, True)
    plane, w = put_plane(plane_of(q, s, z, N, K, 128)), values_of(q, s, z, K)
    x = torch.from_numpy(rng.standard_normal((M, K))).to("cuda", torch.bfloat16)
    wide, y, y4 = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, N, device="cuda"), torch.zeros(M, N, device="cuda")
    uw.w4_expand(plane, wide, N, K)
    uw.recon_gemm(uw.Header(N=N, K=K), None, uw.W_BF16, wide, x, y, M)
    uw.w4_gemm(x, plane, y4, M, N, K)
    total = np.abs(_f64(x)) @ np.abs(w).T
    assert (np.abs(_f64(y) - _f64(x) @ w.T) <= (2.0**-8 + 1e-3) * total).all()
    assert (np.abs(_f64(y4) - _f64(x) @ w.T) <= _tolerance(_f64(x), s, K, 128)).all()


def test_calls_side_by_side_on_two_streams():
    """Two products of many slices and two rows of log probabilities at once, each with a workspace of its own."""
    torch, uw = torch_cuda(), _uw()
    M, N, K, V = 48, 256, 14336, 100_000
    g = torch.Generator(device="cuda").manual_seed(5)
    plane = torch.zeros(uw.w4_plane_bytes(N, K), dtype=torch.uint8, device="cuda")
    uw.w4_quantize(torch.randn(N, K, generator=g, device="cuda"), plane, N, K)
    need = max(uw.w4_gemm_workspace(M, N, K), uw.logprobs_workspace(1, V, 20))
    sides = []
    for _ in range(2):
        sides.append(dict(x=torch.randn(M, K, generator=g, device="cuda").bfloat16(), y=torch.zeros(M, N, device="cuda"),
                          l=torch.randn(1, V, generator=g, device="cuda"), top=torch.zeros(1, 20, dtype=torch.int32, device="cuda"),
                          ws=torch.empty(need, dtype=torch.uint8, device="cuda"), stream=torch.cuda.Stream()))

    def run(s):
        for _ in range(5):
            uw.w4_gemm(s["x"], plane, s["y"], M, N, K, d_ws=s["ws"], ws_bytes=need)
            uw.logprobs(s["l"], 1, V, n_top=20, d_top_token=s["top"], d_ws=s["ws"], ws_bytes=need)

    for s in sides:
        run(s)
        torch.cuda.synchronize()
        s["want"] = (s["y"].clone(), s["top"].clone())
        s["y"].zero_()
    torch.cuda.synchronize()
    for s in sides:
        with torch.cuda.stream(s["stream"]):
            run(s)
    torch.cuda.synchronize()
    for s in sides:
        assert torch.equal(s["y"], s["want"][0]) and torch.equal(s["top"], s["want"][1])
