"""Addresses that the current device must not be given: tensors of the host or of another device are refused before
anything is launched (CPU: stand-ins for tensors; the C library is not called)."""
import pytest
import torch

from nvfp4_weight_only_02_gb300 import binding as nv

bf16, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class Fake:
    """What the binding asks of a contiguous tensor; device -1 is the host."""

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self._dev, self.is_cuda = torch.Size(shape), dtype, device, device >= 0
        self.device = torch.device("cpu" if device < 0 else f"cuda:{device}")

    def get_device(self):
        return self._dev

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def device_zero(monkeypatch):
    """Device 0 is current; whatever gets as far as an allocation or the library raises Reached."""
    def reached(*a, **k):
        raise Reached

    monkeypatch.setattr(nv, "_current", lambda: 0)
    monkeypatch.setattr(nv, "_call", reached)
    monkeypatch.setattr(nv, "_raw", lambda device: 0)
    monkeypatch.setattr(nv, "_stream", lambda: 0)
    monkeypatch.setattr(nv, "load", reached)
    monkeypatch.setattr(nv, "_lib", None)
    monkeypatch.setattr(nv.torch, "empty", lambda shape, dtype=None, device=None: Fake(
        shape if isinstance(shape, tuple) else (shape,), dtype, 0))


def mx(rows, cols, device=0):
    return nv.MxOperand(Fake((rows, cols // 2), u8, device), Fake((512 * -(-rows // 128) * -(-cols // 128),), u8, device))


space = Fake((1 << 20,), u8)
elsewhere = [Fake((1 << 20,), u8, -1), Fake((1 << 20,), u8, 1), Fake((1 << 20,), i32)]


def calls(x_dev=0, w_dev=0, workspace=space):
    x = Fake((16, 64), bf16, x_dev)
    w = mx(32, 64, w_dev)
    dy = Fake((32, 32), f32, x_dev)
    yield lambda: nv.w4a4_gemm(mx(16, 64, x_dev), w, workspace=workspace)
    yield lambda: nv.mx_linear(x, w, workspace=workspace)
    yield lambda: nv.mx_linear_backward(dy, mx(64, 32, w_dev), None, workspace=workspace)
    yield lambda: nv.mx_linear_backward(dy, None, mx(64, 32, w_dev), workspace=workspace)


def distill(workspace=None, **dev):
    d = lambda n: dev.get(n, 0)  # noqa: E731
    return nv.nvfp4_distill_topk(Fake((4, 100), f32, d("z")), Fake((4, 8), i32, d("index")), Fake((4, 8), f32, d("teacher")),
                                 1.0, False, Fake((4,), f32, d("row_weight")), Fake((1,), f32, d("grad_loss")),
                                 Fake((4,), f32, d("loss")), Fake((4, 100), f32, d("dz")), workspace)


def test_calls_on_one_device_reach_the_library():
    for call in calls():
        with pytest.raises(Reached):
            call()
    for ws in (None, space):
        with pytest.raises(Reached):
            distill(ws)
    with pytest.raises(Reached):
        nv.mx_quantize(Fake((16, 64), bf16))


@pytest.mark.parametrize("which", range(3))
def test_workspace_elsewhere_or_of_another_type(which):
    for call in calls(workspace=elsewhere[which]):
        with pytest.raises(ValueError, match="workspace"):
            call()
    with pytest.raises(ValueError, match="workspace"):
        distill(elsewhere[which])
    with pytest.raises(ValueError, match="workspace"):
        nv.nvfp4_distill_wait_selftest(Fake((4, 100), f32), Fake((4, 8), i32), Fake((4, 8), f32), loss=Fake((4,), f32),
                                       workspace=elsewhere[which])


@pytest.mark.parametrize("x_dev,w_dev", [(1, 0), (0, 1), (1, 1)])
def test_operands_on_another_device(x_dev, w_dev):
    for call in calls(x_dev, w_dev):
        with pytest.raises(ValueError, match="device"):
            call()


@pytest.mark.parametrize("name", ["z", "index", "teacher", "row_weight", "grad_loss", "loss", "dz"])
@pytest.mark.parametrize("device", [-1, 1])
def test_distillation_tensors_elsewhere(name, device):
    with pytest.raises(ValueError, match=name):
        distill(**{name: device})


@pytest.mark.parametrize("device", [-1, 1])
def test_quantiser_and_operands_elsewhere(device):
    with pytest.raises(ValueError, match="x must be"):
        nv.mx_quantize(Fake((16, 64), bf16, device))
    with pytest.raises(ValueError):
        nv.MxOperand(Fake((16, 32), u8), Fake((512,), u8, device))
    with pytest.raises(ValueError):
        nv.Nvfp4Operand(Fake((16, 32), u8), Fake((512,), u8), Fake((1,), f32, device))
    if device > 0:
        with pytest.raises(ValueError, match="operand"):
            mx(16, 64, device).dequantize()


@pytest.mark.parametrize("device", [-1, 1])
def test_weight_only_calls_with_a_workspace_elsewhere(device):
    ws = Fake((1 << 20,), u8, device)
    w = Fake((32, 64), bf16)
    codes, scales, ts = Fake((32, 32), u8), Fake((32, 4), u8), Fake((1,), f32)
    x, y = Fake((4, 64), bf16), Fake((4, 32), f32)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(nv, "load", lambda: type("L", (), {"__getattr__": lambda self, n: None})())
        for call in (lambda: nv.nvfp4_quantize(w, codes, scales, ts, False, ws),
                     lambda: nv.nvfp4_w4a16_lora_gemm(x, codes, scales, ts, None, None, 0.0, None, y, ws),
                     lambda: nv.nvfp4_round_scales(Fake((32, 4), f32), ts, scales, ws),
                     lambda: nv.nvfp4_get_device_status(ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
