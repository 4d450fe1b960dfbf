"""Refusals of the mixture-of-experts and 8-bit calls of the binding before anything is launched: tensors of the host or
of another device, wrong types, shapes and layouts (CPU: stand-ins for tensors; the C library is not called)."""
import pytest
import torch

from nvfp4_weight_only_02_gb300 import binding as nv
from tests.test_binding_devices import Fake, Reached, device_zero, elsewhere, space  # noqa: F401  (device_zero: autouse)

bf16, f32, u8, i32, i8 = torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int8
T, k, E, N, K = 6, 2, 4, 64, 96


@pytest.fixture(autouse=True)
def plan_sizes(monkeypatch):
    monkeypatch.setattr(nv, "_moe_sizes", lambda T, k, E: (4096, 16, 32, 64, 128 * (T * k // 128 + min(T * k, E))))
    for name in ("gemm", "linear", "linear_backward"):
        monkeypatch.setattr(nv, f"nvfp4_moe_{name}_workspace_bytes", lambda *a: 1024)
    monkeypatch.setattr(nv, "nvfp4_int8_linear_workspace_bytes", lambda *a: 1024)
    monkeypatch.setattr(nv.torch, "zeros", lambda n, dtype=None, device=None: Fake((n,), dtype, 0))


def plan(index=0):
    p = nv.MoePlan.__new__(nv.MoePlan)
    p._sizes = nv._moe_sizes(T, k, E)
    p.nbytes, p.padded_rows = p._sizes[0], p._sizes[4]
    p.T, p.k, p.E, p.rows, p.index, p.buffer = T, k, E, T * k, index, Fake((1024,), i32, index)
    return p


def experts(rows, cols, device=0, count=E):
    nbytes = -(-rows // 128) * -(-cols // 128) * 512
    return nv.MxExperts(Fake((count, rows, cols // 2), u8, device), Fake((count, nbytes), u8, device))


def col(rows, cols, device=0):
    return nv.MxOperand(Fake((rows, cols // 2), u8, device), Fake((512 * -(-rows // 128) * -(-cols // 128),), u8, device))


def routing(p, weights=None, chosen=None):
    return nv.MoeRouting(weights or Fake((T, k), f32), chosen or Fake((T, k), i32), p, "softmax", True, 1.0)


def calls(dev=0, plan_dev=0, w_dev=0, ws=space):
    p = plan(plan_dev)
    x = Fake((T, K), bf16, dev)
    dy = Fake((T * k, N), f32, dev)
    P = p.padded_rows
    yield lambda: nv.moe_linear(x, experts(N, K, w_dev), p, workspace=ws)
    yield lambda: nv.moe_linear_backward(dy, col(K, P, w_dev), experts(K, N, w_dev), p, workspace=ws)


def others(dev=0, plan_dev=0):
    p = plan(plan_dev)
    yield lambda: nv.moe_combine(Fake((T * k, N), bf16, dev), Fake((T, k), f32, dev), p)
    yield lambda: nv.moe_combine_backward(Fake((T, N), bf16, dev), Fake((T * k, N), bf16, dev), Fake((T, k), f32, dev), p)
    yield lambda: nv.moe_quantize(Fake((T, K), bf16, dev), p)


def test_calls_on_one_device_reach_the_library():
    for call in list(calls()) + list(others()) + list(calls(ws=None)):
        with pytest.raises(Reached):
            call()
    for call in (lambda: nv.moe_route(Fake((T, E), f32), k), lambda: nv.moe_plan(Fake((T, k), i32), E),
                 lambda: nv.moe_route_backward(Fake((T, k), f32), Fake((T, E), f32), routing(plan())),
                 lambda: nv.moe_quantize_weights(Fake((E, N, K), f32)), lambda: nv.int8_quantize(Fake((T, K), f32)),
                 lambda: nv.int8_linear(Fake((T, K), f32), int8()), lambda: nv.int8_gemm(int8(T), int8())):
        with pytest.raises(Reached):
            call()


def int8(rows=N, device=0):
    return nv.Int8Matrix(Fake((rows, K), i8, device), Fake((rows,), f32, device))


@pytest.mark.parametrize("which", range(3))
def test_workspace_elsewhere_or_of_another_type(which):
    for call in list(calls(ws=elsewhere[which])) + [lambda: nv.int8_linear(Fake((T, K), f32), int8(), workspace=elsewhere[which]),
                                                    lambda: nv.int8_gemm(int8(T), int8(), workspace=elsewhere[which]),
                                                    lambda: nv.moe_plan(Fake((T, k), i32), E, workspace=elsewhere[which])]:
        with pytest.raises(ValueError, match="workspace"):
            call()


@pytest.mark.parametrize("dev,plan_dev,w_dev", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (-1, 0, 0), (1, 1, 1)])
def test_tensors_elsewhere(dev, plan_dev, w_dev):
    for call in list(calls(dev, plan_dev, w_dev)) + (list(others(dev, plan_dev)) if dev or plan_dev else []):
        with pytest.raises(ValueError):
            call()
    if dev:
        for call in (lambda: nv.moe_route(Fake((T, E), f32, dev), k), lambda: nv.moe_plan(Fake((T, k), i32, dev), E),
                     lambda: nv.moe_quantize_weights(Fake((E, N, K), f32, dev)), lambda: nv.int8_quantize(Fake((T, K), f32, dev)),
                     lambda: nv.int8_linear(Fake((T, K), f32, dev), int8()),
                     lambda: nv.moe_route(Fake((T, E), f32), k, bias=Fake((E,), f32, dev)),
                     lambda: nv.moe_route_backward(Fake((T, k), f32, dev), Fake((T, E), f32), routing(plan())),
                     lambda: nv.moe_route_backward(Fake((T, k), f32), Fake((T, E), f32), routing(plan(), Fake((T, k), f32, dev))),
                     lambda: nv.moe_combine(Fake((T * k, N), bf16), Fake((T, k), f32, dev), plan()),
                     lambda: nv.moe_combine(Fake((T * k, N), bf16), None, plan(), base=Fake((T, N), bf16, dev))):
            with pytest.raises(ValueError):
                call()
    if w_dev:
        with pytest.raises(ValueError, match="operand"):
            nv.int8_linear(Fake((T, K), f32), int8(device=1))
        with pytest.raises(ValueError, match="operand"):
            nv.int8_gemm(int8(T, 1), int8())


def test_wrong_types_and_shapes():
    p = plan()
    P = p.padded_rows
    x, y = Fake((T, K), bf16), Fake((T * k, N), bf16)
    for call in (
            lambda: nv.moe_route(Fake((T, E), i32), k), lambda: nv.moe_route(Fake((T, E), f32), 0),
            lambda: nv.moe_route(Fake((T, E), f32), E + 1), lambda: nv.moe_route(Fake((T, E), f32), k, scoring="other"),
            lambda: nv.moe_route(Fake((T, E), f32), k, bias=Fake((E + 1,), f32)),
            lambda: nv.moe_route_backward(Fake((T, k + 1), f32), Fake((T, E), f32), routing(p)),
            lambda: nv.moe_route_backward(Fake((T, k), f32), Fake((T, E + 1), f32), routing(p)),
            lambda: nv.moe_plan(Fake((T, k), torch.int64), E), lambda: nv.moe_plan(Fake((T,), i32), E),
            lambda: nv.moe_combine(Fake((T * k - 1, N), bf16), None, p), lambda: nv.moe_combine(Fake((T * k, N), i32), None, p),
            lambda: nv.moe_combine(y, Fake((T, k), bf16), p), lambda: nv.moe_combine(y, None, p, base=Fake((T, N), f32)),
            lambda: nv.moe_combine(y, None, p, out_dtype=i32), lambda: nv.moe_combine(y, None, None),
            lambda: nv.moe_combine_backward(Fake((T, N), f32), y, Fake((T, k), f32), p),
            lambda: nv.moe_combine_backward(Fake((T, N), bf16), None, Fake((T, k), f32), p),
            lambda: nv.moe_combine_backward(Fake((T, N), bf16), y, Fake((T, k), f32), p, need_dy=False, need_dweights=False),
            lambda: nv.moe_quantize(Fake((T + 1, K), bf16), p), lambda: nv.moe_quantize(x, p, sorted_rows=True),
            lambda: nv.moe_quantize_weights(Fake((N, K), bf16)), lambda: nv.moe_quantize_weights(Fake((E, N, K), i8)),
            lambda: nv.moe_linear(x, experts(N, K, count=E + 1), p), lambda: nv.moe_linear(x, experts(N, K + 32), p),
            lambda: nv.moe_linear(x, col(N, K), p), lambda: nv.moe_linear(x, experts(N, K), p, out_dtype=i32),
            lambda: nv.moe_gemm(col(P + 128, K), experts(N, K), p), lambda: nv.moe_gemm(col(P, K + 32), experts(N, K), p),
            lambda: nv.moe_linear_backward(y, None, None, p), lambda: nv.moe_linear_backward(y, col(K, P + 128), None, p),
            lambda: nv.moe_linear_backward(y, None, experts(K, N + 32), p),
            lambda: nv.MxExperts(Fake((E, N, K // 2), u8), Fake((E, 100), u8)),
            lambda: nv.MxExperts(Fake((E, N, 20), u8), Fake((E, 512), u8)),
            lambda: nv.Int8Matrix(Fake((N, K), u8), Fake((N,), f32)), lambda: nv.Int8Matrix(Fake((N, K), i8), Fake((K,), f32)),
            lambda: nv.int8_linear(Fake((T, K + 16), f32), int8()), lambda: nv.int8_linear(Fake((T, K), f32), int8(), out_dtype=i8),
            lambda: nv.int8_linear(Fake((T, K), f32), Fake((N, K), i8)), lambda: nv.int8_quantize(Fake((T, K), i32))):
        with pytest.raises(ValueError):
            call()

