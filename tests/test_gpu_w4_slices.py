"""4-bit products whose K is cut among workgroups, captured and replayed: the joined sums are those of the eager call, whatever the
workspace holds before."""
import pytest

from tests.gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,group", [(48, 256, 14336, 128), (17, 100, 6500, 32)])
def test_captured_and_replayed(M, N, K, group):
    torch = torch_cuda()
    import decode_gemm_amd as uw

    g = torch.Generator(device="cuda").manual_seed(M)
    planes = []
    for _ in range(2):
        planes.append(torch.zeros(uw.w4_plane_bytes(N, K, group), dtype=torch.uint8, device="cuda"))
        uw.w4_quantize(torch.randn(N, K, generator=g, device="cuda").mul_(0.02), planes[-1], N, K, group=group, ldw=K)
    ldx = (K + 7) // 8 * 8
    x = torch.randn(M, ldx, generator=g, device="cuda").bfloat16()
    one, two = uw.w4_gemm_workspace(M, N, K), uw.w4_gemm_workspace(M, 2 * N, K)
    assert one > 0 and two > 0
    need = max(one, two)
    sides = [(torch.zeros(M, N, device="cuda"), torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(need, dtype=torch.uint8, device="cuda")) for _ in range(2)]

    def run(y, h, ws):
        uw.w4_gemm(x, planes[0], y, M, N, K, group=group, ldx=ldx, d_ws=ws, ws_bytes=need)
        uw.w4_gate_up(x, *planes, h, M, N, K, group=group, ldx=ldx, d_ws=ws, ws_bytes=need)

    run(*sides[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*sides[1])
    for i in range(3):
        x.copy_(torch.randn(M, ldx, generator=g, device="cuda"))
        run(*sides[0])
        for t in sides[1]:
            t.fill_(255 if i else 0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sides[0][0], sides[1][0]) and torch.equal(sides[0][1], sides[1][1])
        assert float(sides[0][0].abs().max()) > 0 and float(sides[0][1].float().abs().max()) > 0
