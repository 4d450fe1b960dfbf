"""Waits of the distillation kernels that give up: no row keeps what shared memory happened to hold.

The self-check entry gives up at once on every wait for a copy; nothing faults or hangs, and the next call is right.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

# rows in a cluster of one and of several CTAs, four entries a thread; the stream, its ring larger and smaller than a row
SIZES = [(7, 300, 4, torch.bfloat16), (5, 40001, 8, torch.float32), (3, 131072, 600, torch.bfloat16),
         (400, 60001, 16, torch.bfloat16), (400, 30000, 16, torch.float32), (700, 140001, 40, torch.bfloat16)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,V,k,dtype", SIZES)
def test_rows_whose_wait_gave_up_are_nan(nv, T, V, k, dtype, tail):
    g = torch.Generator("cuda").manual_seed(T + V)
    z = torch.randn(T, V, device="cuda", generator=g).to(dtype)
    val, idx = torch.topk(torch.randn(T, min(V, 4096), device="cuda", generator=g), k, dim=1)
    if tail:
        val = torch.log_softmax(val, 1) - 1.0
    idx = idx.int()
    idx[1] = -1                                    # no entry: 0 whatever the logits are
    w = torch.ones(T, device="cuda")
    w[2] = 0.0                                     # weight 0: the logits are not looked at
    before = nv.distill_topk_loss_grad(z, idx, val, tail=tail, row_weight=w)
    zero = torch.zeros(T, dtype=torch.bool, device="cuda")
    zero[1:3] = True
    assert not before[0][zero].any() and not before[1][zero].any()
    for ws in (None, nv.new_workspace(256)):
        for both in (True, False):
            loss = torch.full((T,), 7.0, device="cuda")
            dz = torch.full((T, V), 7.0, dtype=dtype, device="cuda") if both else None
            nv.nvfp4_distill_wait_selftest(z, idx, val, tail=tail, row_weight=w, loss=loss, dz=dz, workspace=ws)
            assert torch.isnan(loss[~zero]).all() and not loss[zero].any()
            if both:
                assert torch.isnan(dz[~zero]).all() and not dz[zero].any()
            if ws is not None:
                assert nv.nvfp4_get_device_status(ws) == nv.ERR_TIMEOUT
                assert nv.nvfp4_get_device_status(ws) == nv.OK
    after = nv.distill_topk_loss_grad(z, idx, val, tail=tail, row_weight=w, workspace=ws)
    assert torch.equal(after[0], before[0]) and torch.equal(after[1], before[1])
    assert nv.nvfp4_get_device_status(ws) == nv.OK
