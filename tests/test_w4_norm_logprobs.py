"""CPU tests of the host side of 4-bit weights, block norms and log probabilities: every refusal comes back as its
status before any device call, empty batches are no-ops, the binding's defaults and type rules. No device call is made
here; 0x10000 and the like stand for device addresses."""
import pytest
import torch

import decode_gemm_amd as uw

P = 0x10000


def _status(call, *a, **k):
    with pytest.raises(uw.UwError) as e:
        call(*a, **k)
    assert str(e.value)
    return e.value.status


def test_plane_bytes():
    assert uw.w4_plane_bytes(16, 128, 128) == 1024 + 64
    assert uw.w4_plane_bytes(17, 129, 32) == 4 * (1024 + 256)
    assert uw.w4_plane_bytes(1, 1, 64) == 1024 + 128
    for bad in ((0, 128, 128), (16, 0, 128), (16, 128, 16), (16, 128, 256), (1 << 25, 128, 128), (16, 1 << 25, 128), (-1, 5, 32),
                (1 << 24, 1 << 24, 128)):
        assert uw.w4_plane_bytes(*bad) == 0


def test_quantize_and_expand_refusals():
    def q(**k):
        d = dict(d_w=P, d_plane=P, N=32, K=256, group=128, w_type=uw.BF16, stream=0)
        d.update(k)
        return _status(uw.w4_quantize, **d)

    def e(**k):
        d = dict(d_plane=P, d_w=P, N=32, K=256, group=128, w_type=uw.BF16, stream=0)
        d.update(k)
        return _status(uw.w4_expand, **d)

    for f in (q, e):
        assert f(N=0) == uw.ESHAPE
        assert f(K=0) == uw.ESHAPE
        assert f(group=16) == uw.EINVAL
        assert f(w_type=uw.E4M3) == uw.EINVAL
        assert f(d_w=None) == uw.EINVAL
        assert f(d_plane=None) == uw.EINVAL
        assert f(d_w=P + 8) == uw.EINVAL
        assert f(d_plane=P + 8) == uw.EINVAL
        assert f(ldw=248) == uw.EINVAL
        assert f(ldw=260) == uw.EINVAL
        assert f(w_type=uw.F32, ldw=258) == uw.EINVAL
        assert f(N=1 << 25) == uw.EUNSUPPORTED
        assert f(N=1 << 24, K=1 << 16) == uw.EUNSUPPORTED
    assert q(zeros=2) == uw.EINVAL


@pytest.mark.parametrize("up", [False, True])
def test_product_refusals(up):
    def f(**k):
        d = dict(d_x=P, M=4, N=64, K=256, group=64, stream=0)
        d.update({"d_gate": P, "d_up": P, "d_h": P} if up else {"d_plane": P, "d_y": P, "y_type": uw.F32})
        d.update(k)
        return _status(uw.w4_gate_up if up else uw.w4_gemm, **d)

    out = "d_h" if up else "d_y"
    assert f(M=-1) == uw.ESHAPE
    assert f(N=0) == uw.ESHAPE
    assert f(K=0) == uw.ESHAPE
    assert f(group=0) == uw.EINVAL
    for name in ("d_x", out) + (("d_gate", "d_up") if up else ("d_plane",)):
        assert f(**{name: None}) == uw.EINVAL
        assert f(**{name: P + 1}) == uw.EINVAL
    assert f(d_x=P + 8) == uw.EINVAL
    assert f(d_ws=P + 8, ws_bytes=100) == uw.EINVAL
    assert f(ldx=250) == uw.EINVAL
    assert f(ldx=260) == uw.EINVAL
    assert f(**{"ldh" if up else "ldy": 63}) == uw.EINVAL
    assert f(M=1 << 31) == uw.EUNSUPPORTED
    assert f(M=(1 << 31) - 1, N=1 << 20) == uw.EUNSUPPORTED
    assert f(ldx=(1 << 25) + 8) == uw.EUNSUPPORTED
    assert f(N=1 << 25) == uw.EUNSUPPORTED
    if not up:
        assert f(y_type=uw.E4M3) == uw.EINVAL


def test_gate_up_is_bf16():
    a = uw.W4Args(1, 16, 128, 128, P, 128, P, P, P, 16, uw.F32, None, 0)
    import ctypes

    assert uw.lib.uw_w4_gate_up(ctypes.byref(a), None) == uw.EINVAL


def _norm(**k):
    d = dict(d_y=P, d_r=P << 1, d_r_out=P << 2, M=4, K=256, d_h=P << 3, y_type=uw.F32, r_type=uw.BF16, w_type=uw.BF16, h_type=uw.BF16, stream=0)
    d.update(k)
    return _status(uw.block_norm, **d)


def test_norm_refusals():
    assert _norm(M=-1) == uw.ESHAPE
    assert _norm(K=0) == uw.ESHAPE
    assert _norm(K=65537) == uw.EUNSUPPORTED
    assert _norm(M=1 << 31) == uw.EUNSUPPORTED
    assert _norm(M=1 << 30, K=4096) == uw.EUNSUPPORTED  # more threads than a launch has
    for name in ("post", "pre"):
        assert _norm(**{name: 3}) == uw.EINVAL
        assert _norm(**{name: -1}) == uw.EINVAL
    for name in ("y_type", "r_type", "w_type", "h_type"):
        assert _norm(**{name: 3}) == uw.EINVAL
    assert _norm(y_type=uw.E4M3) == uw.EINVAL
    assert _norm(d_y=None, d_r=None) == uw.EINVAL
    assert _norm(d_r_out=None, d_h=None) == uw.EINVAL
    for name in ("d_y", "d_r", "d_r_out", "d_h", "d_post_w", "d_pre_w", "d_gate"):
        assert _norm(**{name: (P << 4) + 8}) == uw.EINVAL
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _norm(eps=eps) == uw.EINVAL
    assert _norm(gate_rows=-1) == uw.EINVAL
    assert _norm(d_post_b=P) == uw.EINVAL  # biases belong to layer norms
    assert _norm(d_pre_b=P) == uw.EINVAL
    assert _norm(post=uw.NORM_LAYER, d_post_b=P + 8) == uw.EINVAL
    for name in ("ldy", "ldr", "ldr_out", "ldh"):
        assert _norm(**{name: 248}) == uw.EINVAL
        assert _norm(**{name: 258}) == uw.EINVAL
    assert _norm(d_gate=P, ldgate=250) == uw.EINVAL


def test_norm_refuses_wrong_places():
    assert _norm(d_h=P) == uw.EINVAL                       # bf16 over fp32
    assert _norm(d_h=P << 1, ldh=264) == uw.EINVAL         # another leading dimension
    assert _norm(d_r_out=P) == uw.EINVAL
    assert _norm(d_r_out=P << 3) == uw.EINVAL              # both outputs in one place
    codes = dict(d_h=None, d_q=P << 3, h_type=None)
    assert _norm(**codes) == uw.EINVAL                     # no scales
    assert _norm(d_s=P + 2, **codes) == uw.EINVAL
    assert _norm(d_s=P, lds=3, **codes) == uw.EINVAL
    assert _norm(d_s=P, ldh=264, **codes) == uw.EINVAL
    assert _norm(d_s=P, **{**codes, "d_q": P << 1}) == uw.EINVAL


def _lp(**k):
    d = dict(d_logits=P, M=4, V=1000, d_token=P, d_logprob=P, n_top=0, type=uw.F32, d_ws=P, ws_bytes=1 << 30, stream=0)
    d.update(k)
    return _status(uw.logprobs, **d)


def test_logprobs_refusals():
    assert _lp(M=-1) == uw.ESHAPE
    assert _lp(V=0) == uw.ESHAPE
    assert _lp(n_top=-1) == uw.EINVAL
    assert _lp(n_top=129, d_top_token=P) == uw.EUNSUPPORTED
    assert _lp(V=(1 << 20) + 1) == uw.EUNSUPPORTED
    assert _lp(M=1 << 22) == uw.EUNSUPPORTED
    assert _lp(type=uw.E4M3) == uw.EINVAL
    assert _lp(d_logits=None) == uw.EINVAL
    assert _lp(d_logits=P + 2) == uw.EINVAL
    assert _lp(type=uw.BF16, d_logits=P + 1) == uw.EINVAL
    assert _lp(ld=999) == uw.EINVAL
    for name in ("d_token", "d_temperature", "d_logprob", "d_rank", "d_entropy"):
        assert _lp(**{name: P + 2}) == uw.EINVAL
    assert _lp(d_token=None) == uw.EINVAL
    assert _lp(d_token=None, d_logprob=None, d_rank=P) == uw.EINVAL
    assert _lp(d_logprob=None) == uw.EINVAL              # no output
    assert _lp(n_top=3) == uw.EINVAL                     # nowhere to put them
    assert _lp(d_top_token=P) == uw.EINVAL               # a list of nothing
    assert _lp(n_top=3, d_top_token=P + 2) == uw.EINVAL
    need = uw.logprobs_workspace(4, 100000, 3)
    assert need > 0
    assert _lp(V=100000, n_top=3, d_top_token=P, ws_bytes=need - 1) == uw.ENOSPACE
    assert _lp(V=100000, n_top=3, d_top_token=P, d_ws=None, ws_bytes=need) == uw.ENOSPACE
    assert _lp(V=100000, n_top=3, d_top_token=P, d_ws=P + 8) == uw.EINVAL


def test_workspaces():
    assert uw.logprobs_workspace(0, 1000) == 0
    assert uw.logprobs_workspace(4, 0) == 0
    assert uw.logprobs_workspace(1 << 22, 1000) == 0
    assert uw.logprobs_workspace(4, 1000, 129) == 0
    assert uw.logprobs_workspace(1, 1000, 20) == 0       # one workgroup has the row
    assert uw.logprobs_workspace(1024, 131072, 20) == 0
    assert uw.logprobs_workspace(4, 100000, 20) > uw.logprobs_workspace(4, 100000, 0) > 0
    assert uw.w4_gemm_workspace(0, 16, 128) == 0
    assert uw.w4_gemm_workspace(1, 0, 128) == 0
    assert uw.w4_gemm_workspace(1, 1 << 25, 128) == 0


def test_empty_batches():
    uw.w4_gemm(None, None, None, 0, 64, 256, y_type=uw.F32, stream=0)
    uw.w4_gate_up(None, None, None, None, 0, 64, 256, stream=0)
    uw.block_norm(None, None, None, 0, 256, stream=0)
    uw.logprobs(None, 0, 1000, type=uw.F32, stream=0)


def test_binding_types():
    f32, b16, i32 = torch.ones(4), torch.ones(4, dtype=torch.bfloat16), torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="type"):
        uw.w4_quantize(P, P, 16, 128, stream=0)
    with pytest.raises(ValueError, match="d_x must be bf16"):
        uw.w4_gemm(f32, P, f32, 1, 16, 128, stream=0)
    with pytest.raises(ValueError, match="d_h must be bf16"):
        uw.w4_gate_up(b16, P, P, f32, 1, 16, 128, stream=0)
    with pytest.raises(ValueError, match="d_plane"):
        uw.w4_gemm(b16, torch.zeros(100, dtype=torch.uint8), f32, 1, 16, 128, stream=0)
    with pytest.raises(ValueError, match="d_plane"):
        uw.w4_quantize(f32, torch.zeros(4000, dtype=torch.uint8)[::2], 16, 128, stream=0)
    with pytest.raises(ValueError, match="different types"):
        uw.block_norm(f32, f32, b16, 1, 4, stream=0)
    with pytest.raises(ValueError, match="different types"):
        uw.block_norm(f32, f32, f32, 1, 4, d_post_w=f32, d_pre_w=b16, stream=0)
    with pytest.raises(ValueError, match="type"):
        uw.block_norm(P, None, None, 1, 4, d_h=f32, stream=0)
    with pytest.raises(ValueError, match="values or codes"):
        uw.block_norm(f32, None, None, 1, 4, d_h=f32, d_q=P, stream=0)
    with pytest.raises(ValueError, match="d_q"):
        uw.block_norm(f32, None, None, 1, 4, d_q=f32, d_s=f32, stream=0)
    with pytest.raises(ValueError, match="one after another"):
        uw.block_norm(f32, None, None, 1, 4, d_h=f32, d_post_w=torch.ones(4, 2)[:, 0], stream=0)
    for name, wrong in (("d_token", f32), ("d_logprob", i32), ("d_rank", f32), ("d_entropy", b16), ("d_temperature", i32),
                        ("d_token", torch.ones(4, dtype=torch.int64))):
        kw = dict(d_token=P, d_logprob=P)
        kw[name] = wrong
        with pytest.raises(ValueError, match=name):
            uw.logprobs(P, 4, 1000, type=uw.F32, stream=0, **kw)
    with pytest.raises(ValueError, match="d_top_token"):
        uw.logprobs(P, 4, 1000, type=uw.F32, n_top=2, d_top_token=torch.ones(4, 4, dtype=torch.int32)[:, :2], stream=0)


def test_host_memory_is_refused():
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 256)
    plane = torch.zeros(uw.w4_plane_bytes(64, 256), dtype=torch.uint8)
    for call in (lambda: uw.w4_quantize(w, P, 4, 256, stream=0), lambda: uw.w4_expand(P, w, 4, 256, stream=0),
                 lambda: uw.w4_gemm(x, plane, torch.zeros(4, 64), 4, 64, 256, stream=0),
                 lambda: uw.w4_gate_up(x, plane, plane, x, 4, 64, 256, stream=0),
                 lambda: uw.block_norm(w, None, None, 4, 256, d_h=w, stream=0),
                 lambda: uw.logprobs(w, 4, 256, d_entropy=torch.zeros(4), stream=0)):
        with pytest.raises(ValueError, match="host memory"):
            call()


def test_scales_of_codes_are_fp32():
    f32, q = torch.ones(4), torch.zeros(4, dtype=torch.uint8)
    for wrong in (torch.ones(4, dtype=torch.bfloat16), torch.ones(4, dtype=torch.float64)):
        with pytest.raises(ValueError, match="d_s"):
            uw.block_norm(f32, None, None, 1, 4, d_q=q, d_s=wrong, stream=0)
