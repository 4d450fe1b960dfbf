"""The 4-bit and distillation calls captured in a CUDA graph: replays on new inputs give what the calls give."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _replays(make, inputs, fresh):
    """make() -> outputs of the calls on `inputs` (static tensors); fresh(i): their values for replay i."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        make()                                  # kernels loaded before the capture
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = make()
    for i in range(3):
        for t, v in zip(inputs, fresh(i)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        want = make()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 9, 40, 300])
def test_layers_in_a_row(nv, M):
    """Decode and prefill layers behind one another: few tokens in one kernel, with a quantiser, and tiles."""
    g = torch.Generator("cuda").manual_seed(M)
    K = 2048
    w1 = nv.mx_quantize(torch.randn(K, K, device="cuda", generator=g) / 45).row
    w2 = nv.mx_quantize(torch.randn(1000, K, device="cuda", generator=g) / 45).row
    ws = nv.new_workspace(nv.nvfp4_mx_linear_workspace_bytes(M, K, K))
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)

    def make():
        h = nv.mx_linear(x, w1, out_dtype=torch.bfloat16, workspace=ws)
        return h, nv.mx_linear(h, w2, workspace=ws)

    _replays(make, [x], lambda i: [torch.randn(M, K, device="cuda", generator=g).bfloat16()])
    assert nv.nvfp4_get_device_status(ws) == nv.OK


@pytest.mark.parametrize("M,V", [(40, 1024), (200, 50016)])
def test_a_training_step(nv, M, V):
    g = torch.Generator("cuda").manual_seed(V)
    K, k = 512, 16
    x = torch.randn(M, K, device="cuda", generator=g)
    w = torch.randn(V, K, device="cuda", generator=g) / 20
    val, idx = torch.topk(torch.randn(M, V, device="cuda", generator=g), k)
    ws = nv.new_workspace(max(nv.nvfp4_w4a4_workspace_bytes(M, V, K),
                              nv.nvfp4_mx_linear_backward_workspace_bytes(M, V, K)))

    def make():
        xq, wq = nv.mx_quantize(x, colwise=True), nv.mx_quantize(w, colwise=True)
        z = nv.w4a4_gemm(xq.row, wq.row, out_dtype=torch.bfloat16, workspace=ws)
        loss, dz = nv.distill_topk_loss_grad(z, idx, val, temperature=1.5, out=z, workspace=ws)
        return (loss, dz) + nv.mx_linear_backward(dz, xq.col, wq.col, workspace=ws)

    _replays(make, [x, w], lambda i: [torch.randn(M, K, device="cuda", generator=g),
                                      torch.randn(V, K, device="cuda", generator=g) / 20])
    assert nv.nvfp4_get_device_status(ws) == nv.OK
