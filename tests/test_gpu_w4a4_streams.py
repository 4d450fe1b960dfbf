"""W4A4 layers on several streams at once: the projections of one layer side by side."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 3, 16, 48])
def test_projections_on_three_streams(nv, M):
    """Clusters of eight CTAs of several launches share the SMs; each result is the one of the call alone."""
    g = torch.Generator().manual_seed(M)
    K = 3584
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    ws_ = [nv.mx_quantize((torch.randn(n, K, generator=g) * 0.05).cuda()).row for n in (3584, 512, 3584)]
    alone = [nv.mx_linear(x, w) for w in ws_]
    streams = [torch.cuda.Stream() for _ in ws_]
    spaces = [nv.new_workspace(nv.nvfp4_mx_linear_workspace_bytes(M, w.rows, K)) for w in ws_]
    torch.cuda.synchronize()
    got = [[] for _ in ws_]
    for _ in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(nv.mx_linear(x, ws_[i], workspace=spaces[i]))
    torch.cuda.synchronize()
    for i, want in enumerate(alone):
        assert nv.nvfp4_get_device_status(spaces[i]) == nv.OK
        for y in got[i]:
            assert torch.equal(y, want)
