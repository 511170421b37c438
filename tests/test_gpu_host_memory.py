"""A tensor left in host memory is refused wherever it stands among a call's arguments, beside tensors on the GPU: no kernel is
launched."""
import pytest

from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


def _each_in_host_memory(call, **tensors):
    for name, t in tensors.items():
        with pytest.raises(ValueError, match="host memory"):
            call(**{**tensors, name: t.cpu()})


def test_every_argument():
    torch = torch_cuda()
    import decode_gemm_amd as uw

    def f(*s):
        return torch.zeros(*s, device="cuda")

    def b(*s):
        return torch.zeros(*s, dtype=torch.bfloat16, device="cuda")

    def i(*s):
        return torch.zeros(*s, dtype=torch.int32, device="cuda")

    def u(*s):
        return torch.zeros(*s, dtype=torch.uint8, device="cuda")

    M, N, K = 4, 64, 256
    plane, ws = u(uw.w4_plane_bytes(N, K)), u(1 << 16)
    _each_in_host_memory(lambda **t: uw.w4_quantize(N=N, K=K, **t), d_w=f(N, K), d_plane=plane)
    _each_in_host_memory(lambda **t: uw.w4_expand(N=N, K=K, **t), d_w=f(N, K), d_plane=plane)
    _each_in_host_memory(lambda **t: uw.w4_gemm(M=M, N=N, K=K, ws_bytes=1 << 16, **t), d_x=b(M, K), d_plane=plane, d_y=f(M, N), d_ws=ws)
    _each_in_host_memory(lambda **t: uw.w4_gate_up(M=M, N=N, K=K, ws_bytes=1 << 16, **t), d_x=b(M, K), d_gate=plane, d_up=plane.clone(), d_h=b(M, N), d_ws=ws)
    rows = dict(d_y=f(M, K), d_r=b(M, K), d_r_out=b(M, K), d_post_w=f(K), d_post_b=f(K), d_pre_w=f(K), d_pre_b=f(K), d_gate=f(1, K))
    layer = dict(M=M, K=K, post=uw.NORM_LAYER, pre=uw.NORM_LAYER)
    _each_in_host_memory(lambda **t: uw.block_norm(**layer, **t), d_h=f(M, K), **rows)
    _each_in_host_memory(lambda **t: uw.block_norm(**layer, **t), d_q=u(M, K), d_s=f(2, M), **rows)
    _each_in_host_memory(lambda **t: uw.logprobs(M=M, V=1000, n_top=2, ws_bytes=1 << 16, **t), d_logits=f(M, 1000), d_token=i(M), d_temperature=f(M), d_logprob=f(M),
                         d_rank=i(M), d_entropy=f(M), d_top_token=i(M, 2), d_top_logprob=f(M, 2), d_ws=ws)
    _each_in_host_memory(lambda **t: uw.sample(M=M, V=1000, ws_bytes=1 << 16, **t), d_logits=f(M, 1000), d_u=f(M), d_token=i(M), d_temperature=f(M), d_top_k=i(M),
                         d_top_p=f(M), d_min_p=f(M), d_prob=f(M), d_ws=ws)
    q, s = u(M, K), f(2, M)
    _each_in_host_memory(lambda **t: uw.fp8_quantize(M=M, K=K, **t), d_x=f(M, K), d_q=q, d_s=s)
    _each_in_host_memory(lambda **t: uw.fp8_swiglu(M=M, K=K, **t), d_g=f(M, K), d_u=f(M, K), d_q=q, d_s=s)
    _each_in_host_memory(lambda **t: uw.fp8_gemm(M=M, N=N, K=K, ws_bytes=1 << 16, **t), d_x=q, d_sx=s, d_w=u(N, K), d_sw=f(1, 2), d_y=f(M, N), d_ws=ws)
