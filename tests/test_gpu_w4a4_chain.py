"""Layers that follow one another in two buffers: each call's tokens are what the call before has just written, and its
output goes where the call before read.  Launches overlap, so an input must not be read before it is complete."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 512), (4, 1024), (16, 2048), (48, 512), (200, 768)])
def test_chain_in_two_buffers(nv, M, K, dtype):
    g = torch.Generator().manual_seed(M)
    ws_ = [nv.mx_quantize((torch.randn(K, K, generator=g) / K ** 0.5).cuda()).row for _ in range(3)]
    x = torch.randn(M, K, generator=g).to(dtype).cuda()
    space = nv.new_workspace(nv.nvfp4_mx_linear_workspace_bytes(M, K, K))
    want, t = [], x
    for i in range(24):
        t = nv.mx_linear(t, ws_[i % 3], out_dtype=dtype)
        torch.cuda.synchronize()
        want.append(t)
    code = nv.OUT_FP32 if dtype == torch.float32 else nv.OUT_BF16
    for _ in range(5):
        buf = [x.clone(), torch.empty_like(x)]
        torch.cuda.synchronize()
        got = []
        for i in range(24):
            a, b = buf[i % 2], buf[1 - i % 2]
            nv._call("nvfp4_mx_linear", a.data_ptr(), code, K, M, K, K, *ws_[i % 3].addresses(), b.data_ptr(), code,
                     space.data_ptr(), space.numel(), nv._raw_stream())
            if i % 8 == 7:
                got.append((i, b.clone()))
        for i, y in got:
            assert torch.equal(y, want[i])
    assert nv.nvfp4_get_device_status(space) == nv.OK
