"""The quantizer's scale for every mantissa that a group's largest value can have: the nearest number of 20 bits, ties to even, as the
definition in 64 bits gives it."""
import pytest

from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [127, 128, 100, 26, 1])
def test_every_mantissa(exponent):
    """2^23 groups, each with one value of this exponent (26: scales below 2^-100 and above, 1: at the least scale)."""
    torch = torch_cuda()
    import decode_gemm_amd as uw

    N, group, per_row = 2048, 32, 4096
    bits = torch.arange(1 << 23, dtype=torch.int32, device="cuda") | exponent << 23
    top = bits.view(torch.float32)
    w = torch.zeros(N, per_row, group, device="cuda")
    w[:, :, 3] = top.view(N, per_row)
    K = per_row * group
    plane = torch.zeros(uw.w4_plane_bytes(N, K, group) // 4, dtype=torch.int32, device="cuda")
    uw.w4_quantize(w, plane, N, K, group=group)
    meta = plane[N * K // 8:].view(N // 16, K // 128, 4, 16).permute(0, 3, 1, 2).reshape(-1)  # t j g r -> t r j g
    m, e = torch.frexp(top.double() / 7)
    s = torch.ldexp(torch.round(m * 2.0**20), e - 20).clamp(min=2.0**-126)
    assert ((meta & 15) == 8).all()
    off = (meta & ~15).view(torch.float32).double() != s
    assert not off.any(), f"{int(off.sum())} scales, the first of {top[off][0].item().hex()}"
