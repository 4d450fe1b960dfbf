"""The distillation kernel for many long rows (more rows than SMs, above 96 KB each) over the types, temperatures and
incoming gradients that the few-row kernel is tested with, against the 64-bit definition; tolerances as derived in
test_gpu_distill.py."""
import pytest
import torch

from tests.test_gpu_distill import _case, _check

pytestmark = pytest.mark.gpu

T = 160


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [0.7, 2.0])
@pytest.mark.parametrize("tdtype,itype", [(torch.bfloat16, torch.int32), (torch.float32, torch.int64)])
@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 50003), (torch.float32, 25001)])
def test_types_temperature_and_gradients(nv, dtype, V, tdtype, itype, tau, tail):
    z, idx, val = _case(T, V, 40, dtype, 11, tail, tau, tdtype)
    w = torch.linspace(-1, 2, T, device="cuda")
    w[::9] = 0.0
    g = torch.linspace(-1, 2, T, device="cuda")
    _check(nv, z, idx.to(itype), val, tau, tail, w, g)
    _check(nv, z, idx.to(itype), val, tau, tail, w, torch.tensor([0.125], device="cuda"))
    _check(nv, z, idx.to(itype), val, tau, tail, None, None)


@pytest.mark.parametrize("tail", [False, True])
def test_indices_beyond_the_vocabulary(nv, tail):
    V = 50003
    z, idx, val = _case(T, V, 12, torch.bfloat16, 3, tail)
    w = torch.ones(T, device="cuda")
    w[7] = 0.0
    idx[7, 3] = V                             # weight 0: not looked at
    ws = nv.new_workspace(256)
    nv.distill_topk_loss_grad(z, idx, val, tail=tail, row_weight=w, workspace=ws)
    assert nv.nvfp4_get_device_status(ws) == nv.OK
    idx[90, 0] = V
    idx[155, 5] = 1 << 40
    _check(nv, z, idx, val, 1.0, tail, w)
    for call in (lambda: nv.distill_topk_loss(z, idx, val, tail=tail, row_weight=w, workspace=ws),
                 lambda: nv.distill_topk_grad(z, idx, val, tail=tail, row_weight=w, workspace=ws)):
        call()
        assert nv.nvfp4_get_device_status(ws) == nv.ERR_INDEX
        assert nv.nvfp4_get_device_status(ws) == nv.OK
