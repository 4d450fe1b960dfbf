"""W4A4 products whose rows of Y end inside a warp's lanes or columns: the stores part the warp between two reads of
the accumulator.  Every element against an FP64 product on the device of the operands' values."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [256, 544])
@pytest.mark.parametrize("M,N", [(33, 130), (50, 77), (64, 19841), (47, 20001),     # streamed, 64 tokens a tile
                                 (129, 255), (300, 1001), (777, 5003), (1025, 2311)])  # tiles, no row on 16 bytes
def test_ragged_rows(nv, M, N, K):
    g = torch.Generator("cuda").manual_seed(M + N)
    a = nv.mx_quantize(torch.randn(M, K, device="cuda", generator=g)).row
    w = nv.mx_quantize(torch.randn(N, K, device="cuda", generator=g)).row
    a64, w64 = a.dequantize().double(), w.dequantize().double()
    want, bound = a64 @ w64.t(), (K + 64) * 2.0 ** -23 * (a64.abs() @ w64.abs().t()) + 1e-38
    y = nv.w4a4_gemm(a, w)
    assert ((y.double() - want).abs() <= bound).all()
    assert torch.equal(nv.w4a4_gemm(a, w, out_dtype=torch.bfloat16), y.bfloat16())
