"""The tensor-core forward and input gradient beside other kernels on CTA pairs and in CUDA graphs: results are those of
the calls alone, bit for bit."""
import pytest
import torch

from tests.test_gpu_graph_fp4 import _replays

pytestmark = pytest.mark.gpu


def _layer(nv, N, K, r, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    q = nv.quantize((torch.randn(N, K, device="cuda", generator=g) * 0.02).bfloat16())
    a = (torch.randn(r, K, device="cuda", generator=g) * 0.05).bfloat16()
    b = (torch.randn(N, r, device="cuda", generator=g) * 0.05).bfloat16()
    z = 1 + 1e-3 * torch.randn(K, device="cuda", generator=g)
    return q, a, b, z


@pytest.mark.parametrize("M,N,K", [(64, 320, 256), (700, 1024, 512), (2100, 2048, 1024)])
def test_three_streams(nv, M, N, K):
    g = torch.Generator("cuda").manual_seed(M)
    q, a, b, z = _layer(nv, N, K, 16, 1)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    dy = torch.randn(M, N, device="cuda", generator=g).bfloat16()
    mx = nv.mx_quantize(torch.randn(N, K, device="cuda", generator=g).bfloat16()).row
    w8 = nv.int8_quantize(torch.randn(N, K, device="cuda", generator=g))
    ws = [nv.new_workspace(n) for n in (nv.nvfp4_workspace_bytes(M, N, K, 16), nv.nvfp4_dgrad_workspace_bytes(M, N, K, 16),
                                        max(nv.nvfp4_mx_linear_workspace_bytes(M, N, K),
                                            nv.nvfp4_int8_linear_workspace_bytes(M, N, K)))]
    calls = [lambda: [nv.gemm(x, q, a, b, 2.0, z, workspace=ws[0])],
             lambda: [nv.gemm_dgrad(dy, q, a, b, 2.0, z, workspace=ws[1])],
             lambda: [nv.mx_linear(x, mx, workspace=ws[2]), nv.int8_linear(x, w8, workspace=ws[2])]]
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(25):
        for c, s, out in zip(calls, streams, got):
            with torch.cuda.stream(s):
                out.append(c())
    torch.cuda.synchronize()
    for want, outs in zip(alone, got):
        for ys in outs:
            for y, w in zip(ys, want):
                assert torch.equal(y, w)
    assert all(nv.nvfp4_get_device_status(w) == nv.OK for w in ws)


@pytest.mark.parametrize("M", [65, 300, 1111])
def test_captured(nv, M):
    N, K = 520, 448
    q, a, b, z = _layer(nv, N, K, 8, 2)
    g = torch.Generator("cuda").manual_seed(M)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    ws = nv.new_workspace(nv.nvfp4_workspace_bytes(M, N, K, 8))
    _replays(lambda: (nv.gemm(x, q, a, b, 2.0, z, workspace=ws), nv.gemm(x, q, workspace=ws, out_dtype=torch.bfloat16)),
             [x], lambda i: [torch.randn(M, K, device="cuda", generator=g).bfloat16()])
    assert nv.nvfp4_get_device_status(ws) == nv.OK
