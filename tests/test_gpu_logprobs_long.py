"""Log probabilities of long rows, of tiny temperatures, and of rows that several workgroups share.

Long rows: one token l_0 and V - 1 tokens of one lower logit, whose weights round the same way in every addition. With u =
2^-24, y = (l - l_0) log2(e) and p the share of the equal tokens: a term is off by 3 u |y| log(2) (three roundings) and 2 u (the exponential), 16 of
them in a step by u (1 + 2 + .. + 16) / 16 = 8.5 u of their sum, 8 steps likewise by 4.5 u, and the rest is fp64: a row's maximum that
a thread has not met changes its fp64 sums alone. Log probabilities are off by that,
  e = p u (2.1 |y| + 15),
and half a step of the output, entropies by e and, through H / S, by (2 e + u) p |y|.
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda
from tests.test_gpu_logprobs import _logits, near, run

pytestmark = pytest.mark.gpu

U = 2.0**-24


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


@pytest.mark.parametrize("M,bf16", [(800, False), (800, True), (400, False), (130, True), (2, False)])
def test_sums_of_long_rows(M, bf16):
    """Every launch shape of rows of 2^20 tokens, one workgroup's to eight's."""
    torch, uw = torch_cuda(), _uw()
    V = 1 << 20
    low = np.resize(np.array([-12.986236, -12.944946, -12.72473, -1.505, -1.637, -1.043, -0.185, -0.086, -0.251, -1.274, -12.917419, -0.713], np.float32), M)
    x = torch.from_numpy(low).to("cuda", torch.bfloat16 if bf16 else torch.float32)
    low = x.double().cpu().numpy()
    x = x[:, None].repeat(1, V)
    x[:, 5] = 0
    token = torch.full((M,), 9, dtype=torch.int32, device="cuda")
    token[::3] = 5
    lp, ent, top = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, 2, device="cuda")
    need = uw.logprobs_workspace(M, V, 2)
    ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device="cuda")
    log(f"  sums of {M} rows, workspace {need}")
    uw.logprobs(x, M, V, d_token=token, d_logprob=lp, d_entropy=ent, n_top=2, d_top_logprob=top, d_ws=ws, ws_bytes=need)
    lp, ent, top = lp.cpu().numpy(), ent.cpu().numpy(), top.cpu().numpy()
    for m in range(min(M, 24)):
        logS = np.log1p((V - 1) * np.exp(low[m]))
        p = -np.expm1(-logS)
        tol = p * U * (2.1 * abs(low[m]) * 1.4427 + 15)
        near(lp[m], (0 if m % 3 == 0 else low[m]) - logS, tol, f"row {m}: log probability")
        near(top[m][0], -logS, tol, f"row {m}: first")
        near(top[m][1], low[m] - logS, tol, f"row {m}: second")
        near(ent[m], logS - p * low[m], tol + (2 * tol + U) * p * abs(low[m]) * 1.4427, f"row {m}: entropy")


def _calls(M, V, n):
    torch = torch_cuda()
    return dict(d_logprob=torch.zeros(M, device="cuda"), d_rank=torch.zeros(M, dtype=torch.int32, device="cuda"), d_entropy=torch.zeros(M, device="cuda"),
                d_top_token=torch.zeros(M, n, dtype=torch.int32, device="cuda"), d_top_logprob=torch.zeros(M, n, device="cuda"))


@pytest.mark.parametrize("M,V,n", [(2, 100_000, 20), (5, 60_001, 128)])
def test_slices_captured_and_replayed(M, V, n):
    torch, uw = torch_cuda(), _uw()
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(M, V, generator=g, device="cuda")
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    need = uw.logprobs_workspace(M, V, n)
    assert need > 0
    a, b = _calls(M, V, n), _calls(M, V, n)
    ws, ws2 = (torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws2, ws_bytes=need, **b)
    for i in range(3):
        x.normal_(generator=g)
        for v in b.values():
            v.zero_()
        ws2.fill_(255 if i else 0)
        uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws, ws_bytes=need, **a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], b[k]) for k in a)
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    assert torch.equal(b["d_top_token"].long(), order[:, :n])


def test_slices_with_outputs_left_out():
    torch, uw = torch_cuda(), _uw()
    M, V, n = 3, 70_001, 7
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, V, generator=g, device="cuda")
    t = torch.randint(0, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    need = uw.logprobs_workspace(M, V, n)
    assert need > uw.logprobs_workspace(M, V, 0) > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = _calls(M, V, n)
    uw.logprobs(x, M, V, d_token=t, n_top=n, d_ws=ws, ws_bytes=need, **outs)
    for name, whole in outs.items():
        alone = torch.zeros_like(whole)
        uw.logprobs(x, M, V, d_token=t if name in ("d_logprob", "d_rank") else None, n_top=n if "top" in name else 0, d_ws=ws, ws_bytes=need, **{name: alone})
        assert torch.equal(alone, whole), name


@pytest.mark.parametrize("V", [300, 9000, 60_000])
def test_temperatures_below_the_normal_numbers(V):
    """Logits that lie a few such temperatures apart, and others far off, of either sign and up to fp32's ends."""
    rng = np.random.default_rng(V)
    T = np.resize(np.array([2.0**-149, 1e-44, 1e-41, 1e-39, 1.17e-38, 1.2e-38, 1e-37], np.float32), 14)
    x = (rng.standard_normal((14, V)) * 8 * T[:, None]).astype(np.float32)
    x[:, ::7] = -np.inf
    x[1, 3], x[2, 5], x[3, 8], x[4, 9] = -3e38, -1.0, 1e-30, 0.75
    x[5, 4], x[5, 6] = 2.0, 2.0
    x[6, 10], x[6, 11] = 3e38, np.inf
    x[7] += np.float32(1.5)
    x[8, 2], x[8, 1] = 1.0, np.nextafter(np.float32(1), np.float32(0))
    run(x, np.where(np.arange(14) % 2, rng.integers(0, V, 14), 3), 6, T=T)
