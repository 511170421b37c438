"""The norms around a block on the GPU against their formulas in 64 bits.

Tolerances, u = 2^-24 (half a step of fp32), n = additions that one sum's longest chain has (8 or 64 per thread, 6 over
lanes, 16 over waves: 90 at most):
  sums        off by n u of the sum of magnitudes
  post(y)     its factor 1 / sqrt(mean square + eps) by (n / 2 + 4) u, two more products: (n / 2 + 6) u of |v - b|, 1 u of |v|; a layer
              norm's differences from the mean (n + 1) u mean|y| + u |y - mean| more, times the factor and weight
  r'          three more roundings of its terms
  h           the same of r', and what r' was off by: its own share times factor and weight, and through the factor
              (the relative change of the root mean square is at most that of the error)
Outputs add half a step of their type: bf16 2^-8 of the value, fp32 u. Codes are those that fp8_quantize makes of the
fp32 h: equal.
"""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu

U = 2.0**-24
CHAIN = 90


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def _up(n, m):
    return (n + m - 1) // m * m


def rows(a, dtype, ld):
    torch = torch_cuda()
    t = torch.full((a.shape[0], ld), float("nan"), dtype=dtype, device="cuda")
    t[:, :a.shape[1]] = torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    return t


def norm64(v, err, kind, w, b, add, eps):
    """The norm of v in 64 bits, and how far fp32's may be off when v is off by err."""
    if kind == 0:
        return v, err
    w = add + (w if w is not None else 1 - add)
    b = 0.0 if b is None else b
    K = v.shape[1]
    if kind == 2:
        mean = v.mean(1, keepdims=True)
        d = v - mean
        err = err + err.mean(1, keepdims=True) + (CHAIN + 1) * U * np.abs(v).mean(1, keepdims=True) + U * np.abs(d)
    else:
        d = v
    ms = (d * d).mean(1, keepdims=True) + eps
    f = 1 / np.sqrt(ms)
    n = d * f * w
    # of the factor: its own roundings, and the error's share of the root mean square
    rel = (CHAIN / 2 + 6) * U + np.sqrt((err * err).mean(1, keepdims=True)) * f
    return n + b, np.abs(n) * rel + err * f * np.abs(w) + U * np.abs(n + b) + U * np.abs(w) * np.abs(d * f)


def formula(y, r, post, pw, pb, gate, pre, qw, qb, sy, sr, add, eps):
    v, e = (None, 0) if y is None else norm64(y, np.zeros_like(y), post, pw, pb, add, eps)
    if y is not None and gate is not None:
        v, e = v * gate, e * np.abs(gate) + U * np.abs(v * gate)
    out = (0 if v is None else sy * v) + (0 if r is None else sr * r)
    e = abs(sy) * e + 3 * U * ((0 if v is None else np.abs(sy * v)) + (0 if r is None else np.abs(sr * r)))
    h, eh = norm64(out, e, pre, qw, qb, add, eps)
    return out, e, h, eh


def close(got, want, tol, dtype, what):
    torch = torch_cuda()
    g = got.double().cpu().numpy()
    bound = tol + np.abs(want) * (2.0**-8 if dtype is torch.bfloat16 else U) + 2.0**-149
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} outside, worst {np.max(np.abs(g - want) / bound):.3g} of the bound"


def case(M, K, seed, y=True, r=True, y_type="f32", r_type="bf16", w_type="bf16", out="f32", post=1, pre=1, weights=True, gate=0,
         sy=0.5, sr=0.9, add=0.0, eps=1e-6, offset=0.0, extra=8):
    """One call on random rows, checked."""
    torch, uw = torch_cuda(), _uw()
    rng = np.random.default_rng(seed)
    types = {"f32": torch.float32, "bf16": torch.bfloat16}

    def exactly(a, t):
        return torch.from_numpy(np.asarray(a, np.float32)).to(types[t]).double().numpy()

    Y = exactly(offset + 3 * rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1))), y_type) if y else None
    R = exactly(offset + rng.standard_normal((M, K)), r_type) if r else None
    vec = lambda base: exactly(base + 0.2 * rng.standard_normal(K), w_type) if weights else None  # noqa: E731
    pw, qw = vec(1.0 - add), vec(1.0 - add)
    pb, qb = (vec(0.0) if post == 2 else None), (vec(0.0) if pre == 2 else None)
    g = exactly(1 + 0.3 * rng.standard_normal((-(-M // gate), K)), w_type) if gate else None
    per_row = None if g is None else g[np.arange(M) // gate]
    if post == 0:
        pw = None
    ldy, ldr, ldo, ldh = (_up(K, 16) + extra for _ in range(4))
    if out == "codes":
        ldh = _up(K, 16)
    want = formula(Y, R, post, pw, pb, per_row, pre, qw if pre else None, qb, np.float64(np.float32(sy)), np.float64(np.float32(sr)),
                   np.float64(np.float32(add)), np.float64(np.float32(eps)))
    dv = lambda v: None if v is None else rows(v[None], types[w_type], _up(K, 8))[0]  # noqa: E731
    r_out = torch.full((M + 1, ldo), 77.0, dtype=types[r_type], device="cuda")
    args = dict(post=post, d_post_w=dv(pw), d_post_b=dv(pb), pre=pre, d_pre_w=dv(qw), d_pre_b=dv(qb),
                d_gate=None if g is None else rows(g, types[w_type], _up(K, 8)), gate_rows=gate, ldgate=_up(K, 8), scale_y=sy, scale_r=sr,
                w_add=add, eps=eps, ldy=ldy, ldr=ldr, ldr_out=ldo)
    d_y = None if Y is None else rows(Y, types[y_type], ldy)
    d_r = None if R is None else rows(R, types[r_type], ldr)
    h = torch.full((M + 1, ldh), 77.0, dtype=types.get(out, torch.float32), device="cuda")
    log(f"  norm {M}x{K} y {y_type if y else None} r {r_type if r else None} post {post} pre {pre} gate {gate} out {out}")
    uw.block_norm(d_y, d_r, r_out, M, K, d_h=h, ldh=ldh, **args)
    assert (r_out[M:] == 77).all() and (r_out[:, K:] == 77).all() and (h[M:] == 77).all() and (h[:, K:] == 77).all()
    close(r_out[:M, :K], want[0], want[1], types[r_type], "r'")
    close(h[:M, :K], want[2], want[3], h.dtype, "h")
    if out == "codes":
        q, s = torch.full((M + 1, ldh), 77, dtype=torch.uint8, device="cuda"), torch.full((_up(K, 128) // 128, M + 1), 77.0, device="cuda")
        q2, s2 = q.clone(), s.clone()
        uw.block_norm(d_y, d_r, r_out, M, K, d_q=q, d_s=s, ldh=ldh, lds=M + 1, **args)
        uw.fp8_quantize(h, q2, s2, M, K, ldx=ldh, ldq=ldh, lds=M + 1)
        assert torch.equal(q, q2) and torch.equal(s, s2)


EDGES = [1, 7, 8, 9, 64, 127, 511, 512, 513, 1024, 1025, 2048, 2049, 4095, 4096, 4097, 8192, 8193, 16384, 16385, 32768, 32777, 65536]


@pytest.mark.parametrize("K", EDGES)
def test_row_lengths(K):
    case(5, K, K, out="codes", gate=2)
    if K > 1:
        case(1, K, K + 1, post=2, pre=2, y_type="bf16", r_type="f32", out="bf16")


@pytest.mark.parametrize("K", [2049, 4096, 4097, 6144, 6145, 8192, 8200, 16384, 16399])
def test_row_lengths_of_many_rows(K):
    case(515, K, K, out="codes", gate=100)
    case(512, K, K + 1, post=2, pre=2, y_type="bf16", r_type="f32", w_type="f32", out="bf16", weights=K % 2 == 0)


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("out", ["f32", "bf16", "codes"])
def test_kinds(post, pre, out):
    for M, K, gate, weights in ((9, 333, 0, True), (9, 2000, 4, False), (2, 5003, 1, True)):
        case(M, K, M + K, post=post, pre=pre, out=out, gate=gate, weights=weights, w_type="f32" if M == 2 else "bf16")


@pytest.mark.parametrize("y_type,r_type,w_type", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
def test_types(y_type, r_type, w_type):
    case(33, 1000, 1, y_type=y_type, r_type=r_type, w_type=w_type, out="bf16", gate=33, add=1.0)
    case(700, 4096, 2, y_type=y_type, r_type=r_type, w_type=w_type, out="f32", gate=7, extra=0)


def test_what_may_be_left_out():
    case(6, 1000, 1, y=False)
    case(6, 1000, 2, y=False, sr=1.0, pre=2)
    case(6, 1000, 3, r=False, gate=3)
    case(6, 1000, 4, r=False, post=0, pre=1, sy=1.0)


def test_a_large_mean_keeps_the_variance():
    case(4, 4096, 5, post=2, pre=2, y_type="f32", r_type="f32", offset=1000.0, w_type="f32")


def test_zero_rows_and_rows_that_are_not_finite():
    torch, uw = torch_cuda(), _uw()
    M, K = 7, 1500
    rng = np.random.default_rng(1)
    y = rng.standard_normal((M, K)).astype(np.float32)
    y[2] = 0
    base = y.copy()
    y[4, 77], y[5, 1499] = np.nan, np.inf
    r = rng.standard_normal((M, K)).astype(np.float32)
    r[2] = 0
    outs = []
    for v in (base, y):
        ro, h = torch.zeros(M, K, device="cuda"), torch.zeros(M, K, device="cuda")
        uw.block_norm(rows(v, torch.float32, K), rows(r, torch.float32, K), ro, M, K, d_h=h)
        outs.append((ro.cpu().numpy(), h.cpu().numpy()))
    good = [0, 1, 2, 3, 6]
    for a, b in zip(*outs):
        assert (a[good] == b[good]).all() and (b[2] == 0).all()
        assert np.isnan(b[4]).all() and np.isnan(b[5, 1499])


def test_in_place():
    torch, uw = torch_cuda(), _uw()
    M, K = 50, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    y, r = (torch.randn(M, K, generator=g, device="cuda") for _ in range(2))
    w = torch.rand(K, generator=g, device="cuda")
    r1, h1 = torch.empty_like(r), torch.empty_like(y)
    uw.block_norm(y, r, r1, M, K, d_h=h1, d_post_w=w, d_pre_w=w)
    uw.block_norm(y, r, r, M, K, d_h=y, d_post_w=w, d_pre_w=w)
    assert torch.equal(r, r1) and torch.equal(y, h1)


def test_streams_and_graphs():
    torch, uw = torch_cuda(), _uw()
    M, K = 3, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    y, r = torch.randn(M, K, generator=g, device="cuda"), torch.randn(M, K, generator=g, device="cuda").bfloat16()
    r1, h1, r2, h2 = torch.zeros_like(r), torch.zeros_like(r), torch.zeros_like(r), torch.zeros_like(r)
    uw.block_norm(y, r, r1, M, K, d_h=h1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        uw.block_norm(y, r, r2, M, K, d_h=h2)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r1, r2) and torch.equal(h1, h2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uw.block_norm(y, r, r2, M, K, d_h=h2)
    for _ in range(3):
        y.mul_(-1.5)
        uw.block_norm(y, r, r1, M, K, d_h=h1)
        r2.zero_()
        h2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(r1, r2) and torch.equal(h1, h2)


def test_offsets_past_four_gigabytes():
    torch, uw = torch_cuda(), _uw()
    M, K = 270_000, 4096  # fp32 rows of 4.4 GB
    y = torch.empty(M, K, device="cuda").normal_()
    h = torch.empty(M, K, device="cuda")
    uw.block_norm(y, None, None, M, K, d_h=h, post=uw.NORM_NONE)
    few = torch.empty(600, K, device="cuda")  # as many rows as are summed up in the same order (512 and more)
    uw.block_norm(y[M - 600:], None, None, 600, K, d_h=few, post=uw.NORM_NONE)
    assert torch.equal(h[M - 600:], few)
