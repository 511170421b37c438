"""The binding's refusals of tensors that the kernels of the 8-bit path and the sampler would misread. On the
CPU: every one is raised before any device call."""
import pytest
import torch

import decode_gemm_amd as uw

P = 0x10000


def _sample(**k):
    d = dict(d_logits=P, d_u=P, d_token=P, M=4, V=1000, type=uw.F32, d_ws=P, ws_bytes=1 << 30, stream=0)
    d.update(k)
    return uw.sample(**d)


FLOATS = ["d_u", "d_temperature", "d_top_p", "d_min_p", "d_prob"]


@pytest.mark.parametrize("name", FLOATS + ["d_top_k", "d_token"])
def test_sample_refuses_other_types(name):
    right = torch.float32 if name in FLOATS else torch.int32
    for dtype in (torch.int64, torch.int32, torch.float64, torch.float32, torch.float16, torch.bfloat16, torch.uint8):
        if dtype is not right:
            with pytest.raises(ValueError, match=name):
                _sample(**{name: torch.ones(4, dtype=dtype)})


@pytest.mark.parametrize("name", FLOATS + ["d_top_k", "d_token"])
def test_sample_refuses_strided_arrays(name):
    right = torch.float32 if name in FLOATS else torch.int32
    with pytest.raises(ValueError, match=name):
        _sample(**{name: torch.ones(4, 2, dtype=right)[:, 0]})


def test_what_fits_reaches_the_library():
    """The library's own check comes next: here a logits pointer off its alignment."""
    kw = {n: torch.ones(4) for n in FLOATS}
    kw.update({n: torch.ones(4, dtype=torch.int32) for n in ("d_top_k", "d_token")})
    with pytest.raises(uw.UwError) as e:
        _sample(d_logits=P + 2, **kw)
    assert e.value.status == uw.EINVAL


def test_host_memory_is_refused():
    x, q, s = torch.zeros(4, 256), torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 4)
    y = torch.zeros(4, 128)
    for call in (lambda: uw.fp8_quantize(x, q, s, 4, 256, stream=0), lambda: uw.fp8_swiglu(x, x, q, s, 4, 256, stream=0),
                 lambda: uw.fp8_gemm(q, s, q, s, y, 4, 128, 256, stream=0),
                 lambda: _sample(d_logits=torch.zeros(4, 1000), type=None)):
        with pytest.raises(ValueError, match="host memory"):
            call()
