"""MXFP4 quantiser on the GPU against the 64-bit definition, bit for bit.

The scale is a power of two, so scaling is exact and every code is one rounding: codes, scale bytes and values are
compared for equality.
"""
import numpy as np
import pytest
import torch

from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32), (1, 3584), (8, 3584), (31, 64), (32, 128), (33, 160), (127, 96), (128, 256), (129, 288),
          (200, 1056), (777, 2048), (1000, 4096 + 32)]
DTYPES = [torch.bfloat16, torch.float32]


def _x(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp2(torch.randint(-20, 20, (rows, (cols + 31) // 32), generator=g).float()).repeat_interleave(32, 1)[:, :cols]
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    return x.to(dtype).cuda()


def _check_dir(op, values, x64, transpose_back):
    codes, byte = ref.mx_encode(x64)
    assert np.array_equal(op.codes.cpu().numpy(), ref.pack(codes))
    assert np.array_equal(op.scales.cpu().numpy(), ref.tile(byte))
    want = ref.mx_values(codes, byte)
    if values is not None:
        got = ref.to64(values)
        got = ref.pad_rows(got).T if transpose_back else got
        assert np.array_equal(got, want, equal_nan=True)
    for dt in (torch.float32, torch.bfloat16):
        assert np.array_equal(ref.to64(op.dequantize(dt)), want, equal_nan=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_both_directions(nv, rows, cols, dtype):
    x = _x(rows, cols, dtype, rows + cols)
    q = nv.mx_quantize(x, colwise=True, values=True)
    _check_dir(q.row, q.values, ref.to64(x), False)
    _check_dir(q.col, q.values_t, np.ascontiguousarray(ref.pad_rows(ref.to64(x)).T), True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_each_output_alone(nv, dtype):
    x = _x(161, 224, dtype, 5)
    full = nv.mx_quantize(x, colwise=True, values=True)
    row = nv.mx_quantize(x)
    col = nv.mx_quantize(x, rowwise=False, colwise=True)
    fake = nv.mx_quantize(x, codes=False, values=True)
    fake_t = nv.mx_quantize(x, rowwise=False, colwise=True, codes=False, values=True)
    assert row.col is None and row.values is None and col.row is None and fake.row is None
    for a, b in ((row.row, full.row), (col.col, full.col)):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert torch.equal(fake.values, full.values) and torch.equal(fake_t.values_t, full.values_t)


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_tie_and_exponent(nv, dtype):
    # every midpoint of the grid and its neighbours, at every exponent a block can have
    mid = (ref.GRID[1:] + ref.GRID[:-1]) / 2
    rows = []
    for e in range(-140, 128):
        vals = np.concatenate([[4.0], mid, mid * (1 + 2.0 ** -7), mid * (1 - 2.0 ** -8), [6.0, 7.0, 7.9375, 0.0]])
        vals = vals * 2.0 ** (e - 2)
        vals = np.resize(vals, 32) * np.resize([1, -1], 32)
        rows.append(vals)
    x = torch.from_numpy(np.array(rows)).to(dtype).cuda()
    q = nv.mx_quantize(x, colwise=True, values=True)
    _check_dir(q.row, q.values, ref.to64(x), False)
    _check_dir(q.col, q.values_t, np.ascontiguousarray(ref.pad_rows(ref.to64(x)).T), True)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_nonfinite_element_marks_its_block_only(nv, dtype, bad):
    x = _x(70, 128, dtype, 9)
    x[37, 50] = bad
    q = nv.mx_quantize(x, colwise=True, values=True)
    _check_dir(q.row, q.values, ref.to64(x), False)
    _check_dir(q.col, q.values_t, np.ascontiguousarray(ref.pad_rows(ref.to64(x)).T), True)
    assert torch.isnan(q.values[37, 32:64]).all() and int(torch.isnan(q.values).sum()) == 32
    assert torch.isnan(q.values_t[32:64, 50]).all() and int(torch.isnan(q.values_t).sum()) == 32


def test_zeros_subnormals_and_largest(nv):
    tiny = torch.tensor([[2.0 ** -149, -(2.0 ** -140), 0.0, -0.0] * 8, [3.0e38, -3.4028234e38, 1.0, 0.0] * 8,
                         [0.0] * 32], dtype=torch.float32).cuda()
    q = nv.mx_quantize(tiny, values=True)
    _check_dir(q.row, q.values, ref.to64(tiny), False)
    assert not q.values[2].any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_row_stride_and_side_stream(nv, dtype):
    big = _x(150, 512, dtype, 3)
    x = big[:, 64:64 + 160]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q = nv.mx_quantize(x, colwise=True, values=True)
    s.synchronize()
    _check_dir(q.row, q.values, ref.to64(x), False)
    _check_dir(q.col, q.values_t, np.ascontiguousarray(ref.pad_rows(ref.to64(x)).T), True)


def test_offsets_beyond_32_bits(nv):
    # 70000 x 65536 elements: the last rows against the definition
    rows, cols = 70000, 65536
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-40:] = torch.randn(40, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    q = nv.mx_quantize(x, colwise=True, values=True)
    codes, byte = ref.mx_encode(ref.to64(x[-40:]))
    assert np.array_equal(q.row.codes[-40:].cpu().numpy(), ref.pack(codes))
    assert np.array_equal(ref.to64(q.values[-40:]), ref.mx_values(codes, byte))
    r0 = (rows - 40) // 32 * 32
    want = ref.mx_round(np.ascontiguousarray(ref.pad_rows(ref.to64(x[r0:])).T))
    assert np.array_equal(ref.to64(q.values_t[r0:]), want.T[:rows - r0])
    assert np.array_equal(q.col.codes[:, r0 // 2:].cpu().numpy(),
                          ref.pack(ref.mx_encode(np.ascontiguousarray(ref.pad_rows(ref.to64(x[r0:])).T))[0]))


@pytest.mark.parametrize("fmt,block", [("mx", 32), ("nv", 16)])
@pytest.mark.parametrize("rows,cols", [(1, 32), (130, 96), (257, 2080)])
def test_tile_scales(nv, rows, cols, fmt, block):
    g = torch.Generator().manual_seed(rows)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g).cuda()
    sc = torch.randint(0, 127, (rows, cols // block), dtype=torch.uint8, generator=g).cuda()
    op = nv.MxOperand.from_row_major(codes, sc) if fmt == "mx" else nv.Nvfp4Operand.from_row_major(codes, sc, None)
    assert np.array_equal(op.scales.cpu().numpy(), ref.tile(sc.cpu().numpy()))


def test_refusals(nv):
    x = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        nv.mx_quantize(x.half())
    with pytest.raises(ValueError):
        nv.mx_quantize(x.t()[:, :32])
    with pytest.raises(ValueError):
        nv.mx_quantize(x.cpu())
    with pytest.raises(ValueError):
        nv.mx_quantize(x[0])
    for bad in (x[:, :48], x[:, :0]):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.mx_quantize(bad)
        assert e.value.status == nv.ERR_SHAPE
    with pytest.raises(nv.NVFP4Error) as e:
        nv.mx_quantize(x[:, 1:33])
    assert e.value.status == nv.ERR_ALIGNMENT
    with pytest.raises(nv.NVFP4Error) as e:
        nv.mx_quantize(x, rowwise=False)
    assert e.value.status == nv.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        nv.MxOperand(torch.zeros(4, 16, dtype=torch.uint8, device="cuda"),
                     torch.zeros(4, dtype=torch.uint8, device="cuda"))
