"""The 8-bit path on the GPU where its sizes, values and kernels' shapes reach their ends, against its
definition in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import log, torch_cuda

pytestmark = pytest.mark.gpu


def _uw():
    torch_cuda()
    import decode_gemm_amd as uw

    return uw


def test_swiglu_down_to_where_silu_ends():
    """From g = -86 down e^g leaves the normal range (-87.3), silu itself (-91.9), and then fp32 (-108). One
    value per row, so that the scales tell |h| in fp32. silu is within 2.5 steps of 2^-23 and, subnormal,
    half of 2^-149; u = 2^60 is exact; the scale rounds by half a step, and so does the product: 3.5 * 2^-23."""
    uw, torch = _uw(), torch_cuda()
    rng = np.random.default_rng(87)
    g = np.concatenate([np.linspace(-112, -86, 20001), rng.uniform(-104, -87, 20000), -np.logspace(1.9, 38, 500)]).astype(np.float32)
    M = g.size
    y = np.zeros((M, 8), np.float32)
    y[:, 0], y[:, 4] = g, 2.0**60
    d = torch.from_numpy(y).cuda()
    q = torch.zeros(M, 16, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, M, device="cuda")
    uw.fp8_swiglu(d, d[:, 4:], q, s, M, 1, ldg=8, ldu=8, ldq=16)
    sh, qh = s[0].cpu().numpy().astype(np.float64), q[:, 0].cpu().numpy()
    g64 = g.astype(np.float64)
    silu = -g64 * np.exp(np.maximum(g64, -700)) / (1 + np.exp(np.maximum(g64, -700)))  # its absolute value
    tol = 3.5 * 2.0**-23 * silu + 2.0**-150
    none = qh & 0x7F == 0  # h is 0: scale 1
    assert (silu[none] <= tol[none]).all() and (sh[none] == 1).all()
    off = np.abs(sh * 448 * 2.0**-60 - silu)[~none] / tol[~none]
    log(f"  worst {off.max():.3g} of the tolerance, {int(none.sum())} of {M} are 0")
    assert (off <= 1).all()
    assert (qh[~none] == 0xFE).all()  # -448 at the scale
    assert none[g < -110].all() and not none[g > -107].any()


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zeros_keep_their_sign(dtype, rows):
    """-0 / s is -0, code 0x80, beside other values and in a group of zeros alone."""
    uw, torch = _uw(), torch_cuda()
    K = 384
    x = np.random.default_rng(1).standard_normal((5, K)).astype(np.float32)
    x[:, 3::7] = -0.0
    x[:, 4::7] = 0.0
    x[:, 128:256:2], x[:, 129:256:2] = 0.0, -0.0
    d = torch.from_numpy(x).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)
    q = torch.full((5, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.zeros((3, 5) if rows == 1 else (1, 3), device="cuda")
    uw.fp8_quantize(d, q, s, 5, K, block_rows=rows)
    zero = x == 0
    assert (q.cpu().numpy()[zero] == np.where(np.signbit(x[zero]), 0x80, 0)).all()


def test_swiglu_zeros_keep_their_sign():
    """silu(-0) is -0, and so is silu of what underflows; the product's sign is that of both."""
    uw, torch = _uw(), torch_cuda()
    g = np.tile(np.array([0.0, -0.0, -300.0, 1.0, -1.0, 2.0, 0.0, -0.0], np.float32), 16)
    u = np.tile(np.array([1.0, 1.0, 1.0, -0.0, -0.0, 3.0, -1.0, -1.0], np.float32), 16)
    d = [torch.from_numpy(v).cuda().reshape(1, 128) for v in (g, u)]
    q = torch.full((1, 128), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, 1, device="cuda")
    uw.fp8_swiglu(d[0], d[1], q, s, 1, 128)
    assert (q[0].cpu().numpy() == np.tile(np.array([0, 0x80, 0x80, 0x80, 0, 0x7E, 0x80, 0], np.uint8), 16)).all()
