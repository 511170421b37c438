"""CPU tests of the 8-bit path's and the sampler's host side: every refusal comes back as its
status before any device call, empty batches are no-ops, and the binding's defaults and type
rules. No device call is made here; 0x1000 and the like stand for device addresses."""
import numpy as np
import pytest
import torch

import decode_gemm_amd as uw

P = 0x10000


def _status(call, *a, **k):
    with pytest.raises(uw.UwError) as e:
        call(*a, **k)
    assert str(e.value)
    return e.value.status


def _quantize(**k):
    d = dict(d_x=P, d_q=P, d_s=P, M=4, K=256, x_type=uw.BF16, stream=0)
    d.update(k)
    return _status(uw.fp8_quantize, **d)


def test_quantize_refusals():
    assert _quantize(M=-1) == uw.ESHAPE
    assert _quantize(K=0) == uw.ESHAPE
    assert _quantize(x_type=2) == uw.EINVAL
    assert _quantize(x_type=-1) == uw.EINVAL
    assert _quantize(block_rows=64) == uw.EINVAL
    for name in ("d_x", "d_q", "d_s"):
        assert _quantize(**{name: None}) == uw.EINVAL
    assert _quantize(d_x=P + 8) == uw.EINVAL
    assert _quantize(d_q=P + 4) == uw.EINVAL
    assert _quantize(d_s=P + 2) == uw.EINVAL
    assert _quantize(ldx=255) == uw.EINVAL            # below K
    assert _quantize(ldx=260) == uw.EINVAL            # bf16 rows off 16-byte boundaries
    assert _quantize(x_type=uw.F32, ldx=258) == uw.EINVAL
    assert _quantize(ldq=264) == uw.EINVAL
    assert _quantize(ldq=240) == uw.EINVAL
    assert _quantize(K=100, ldx=104) == uw.EINVAL     # ldq defaults to K, no multiple of 16
    assert _quantize(lds=3) == uw.EINVAL              # rows: lds >= M
    assert _quantize(block_rows=128, lds=1) == uw.EINVAL  # blocks: lds >= ceil(K / 128)
    # more threads than a launch has along an axis (2^32)
    assert _quantize(M=1 << 28, K=2048) == uw.EUNSUPPORTED
    assert _quantize(M=2, K=1 << 36) == uw.EUNSUPPORTED
    assert _quantize(M=1 << 30, K=128, block_rows=128) == uw.EUNSUPPORTED


def test_swiglu_refusals():
    def f(**k):
        d = dict(d_g=P, d_u=P, d_q=P, d_s=P, M=4, K=256, stream=0)
        d.update(k)
        return _status(uw.fp8_swiglu, **d)

    assert f(M=-1) == uw.ESHAPE
    assert f(K=0) == uw.ESHAPE
    for name in ("d_g", "d_u", "d_q", "d_s"):
        assert f(**{name: None}) == uw.EINVAL
    assert f(d_g=P + 4) == uw.EINVAL
    assert f(d_u=P + 8) == uw.EINVAL
    assert f(ldg=255) == uw.EINVAL
    assert f(ldg=258) == uw.EINVAL
    assert f(ldu=252) == uw.EINVAL
    assert f(ldu=257) == uw.EINVAL
    assert f(ldq=250) == uw.EINVAL
    assert f(lds=2) == uw.EINVAL
    assert f(M=1 << 28, K=2048) == uw.EUNSUPPORTED


def test_gemm_refusals():
    def f(**k):
        d = dict(d_x=P, d_sx=P, d_w=P, d_sw=P, d_y=P, M=4, N=64, K=256, y_type=uw.F32, stream=0)
        d.update(k)
        return _status(uw.fp8_gemm, **d)

    assert f(M=-1) == uw.ESHAPE
    assert f(N=0) == uw.ESHAPE
    assert f(K=0) == uw.ESHAPE
    assert f(M=1 << 31, ldsx=1 << 31) == uw.EUNSUPPORTED
    assert f(N=1 << 31) == uw.EUNSUPPORTED
    assert f(M=1 << 30, N=16, K=16, ldsx=1 << 30) == uw.EUNSUPPORTED  # more threads than a launch has
    assert f(M=1 << 30, N=1 << 12, ldsx=1 << 30) == uw.EUNSUPPORTED
    assert uw.fp8_gemm_workspace(1 << 30, 16, 16) == 0
    assert f(y_type=5) == uw.EINVAL
    for name in ("d_x", "d_sx", "d_w", "d_sw", "d_y"):
        assert f(**{name: None}) == uw.EINVAL
    for name in ("d_x", "d_w", "d_y"):
        assert f(**{name: P + 8}) == uw.EINVAL
    for name in ("d_sx", "d_sw"):
        assert f(**{name: P + 2}) == uw.EINVAL
    assert f(ldx=240) == uw.EINVAL
    assert f(ldx=264) == uw.EINVAL
    assert f(ldw=250) == uw.EINVAL
    assert f(ldw=1 << 24) == uw.EUNSUPPORTED
    assert f(ldx=1 << 24) == uw.EUNSUPPORTED
    assert f(ldsx=3) == uw.EINVAL
    assert f(ldsw=1) == uw.EINVAL
    assert f(ldy=63) == uw.EINVAL
    assert f(d_ws=P + 4, ws_bytes=1 << 20) == uw.EINVAL
    assert uw.lib.uw_fp8_gemm(None, None) == uw.EINVAL


def test_sample_refusals():
    def f(**k):
        d = dict(d_logits=P, d_u=P, d_token=P, M=4, V=100000, type=uw.F32, d_ws=P, ws_bytes=1 << 30, stream=0)
        d.update(k)
        return _status(uw.sample, **d)

    assert f(M=-1) == uw.ESHAPE
    assert f(V=0) == uw.ESHAPE
    assert f(type=3) == uw.EINVAL
    assert f(V=(1 << 20) + 1) == uw.EUNSUPPORTED
    assert f(M=1 << 24) == uw.EUNSUPPORTED
    assert f(M=1 << 22) == uw.EUNSUPPORTED
    for name in ("d_logits", "d_u", "d_token"):
        assert f(**{name: None}) == uw.EINVAL
        assert f(**{name: P + 2}) == uw.EINVAL
    assert f(type=uw.BF16, d_logits=P + 1) == uw.EINVAL
    for name in ("d_temperature", "d_top_k", "d_top_p", "d_min_p", "d_prob"):
        assert f(**{name: P + 1}) == uw.EINVAL
    assert f(ld=99999) == uw.EINVAL
    need = uw.sample_workspace(4, 100000)
    assert need > 0
    assert f(d_ws=None) == uw.EINVAL
    assert f(d_ws=P + 8) == uw.EINVAL
    assert f(ws_bytes=need - 1) == uw.ENOSPACE
    assert uw.lib.uw_sample(None, None) == uw.EINVAL


def test_empty_batches_are_no_ops():
    uw.fp8_quantize(None, None, None, 0, 256, x_type=uw.BF16, stream=0)
    uw.fp8_swiglu(0, None, None, None, 0, 256, stream=0)
    uw.fp8_gemm(0, None, None, None, None, 0, 64, 256, y_type=uw.F32, stream=0)
    uw.sample(0, None, None, 0, 1000, type=uw.F32, stream=0)


def test_workspace_sizes():
    for M, N, K in ((0, 64, 64), (-1, 64, 64), (4, 0, 64), (4, 64, 0), (1 << 31, 64, 64)):
        assert uw.fp8_gemm_workspace(M, N, K) == 0
    for M, V in ((0, 100), (-1, 100), (4, 0), (4, (1 << 20) + 1), (1 << 24, 10)):
        assert uw.sample_workspace(M, V) == 0


    assert uw.sample_workspace(1, 131072) > 0
    assert uw.sample_workspace(2000, 131072) == 0  # one workgroup per row, which does all of it
    assert uw.sample_workspace(1, 2000) == 0


def test_types_follow_the_tensor():
    assert uw._type(torch.zeros(1), None) == uw.F32
    assert uw._type(torch.zeros(1, dtype=torch.bfloat16), None) == uw.BF16
    assert uw._type(torch.zeros(1, dtype=torch.int16), None) == uw.BF16
    assert uw._type(torch.zeros(1), uw.BF16) == uw.BF16
    for t in (torch.zeros(1, dtype=torch.float16), torch.zeros(1, dtype=torch.float64), P, np.zeros(1)):
        with pytest.raises(ValueError):
            uw._type(t, None)
