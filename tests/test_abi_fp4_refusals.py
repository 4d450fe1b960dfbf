"""Further host-side refusals of the 4-bit and distillation entry points (CPU): nothing is launched, with or without
a GPU."""
import ctypes

import pytest

from nvfp4_weight_only_02_gb300 import binding, build

P = ctypes.c_void_p
good, bad = P(4096), P(4096 + 4)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_distill_wait_selftest(lib):
    f = lambda z=good, dt=0, T=2, V=100, i=good, t=good, k=4, w=None, loss=good, dz=good, ws=None, n=0: \
        lib.nvfp4_distill_wait_selftest(z, dt, T, V, i, t, k, 0, w, loss, dz, ws, n, None)  # noqa: E731
    for kw in (dict(z=None), dict(i=None), dict(t=None), dict(loss=None, dz=None), dict(dt=2)):
        assert f(**kw) == binding.ERR_INVALID_ARG, kw
    for kw in (dict(T=0), dict(V=0), dict(k=0), dict(k=1025)):
        assert f(**kw) == binding.ERR_SHAPE, kw
    for kw in (dict(z=bad), dict(i=bad), dict(t=bad), dict(w=bad), dict(loss=bad), dict(dz=bad)):
        assert f(**kw) == binding.ERR_ALIGNMENT, kw
    assert f(ws=good, n=255) == binding.ERR_WORKSPACE


def test_distill_temperature_whose_reciprocal_leaves_fp32(lib):
    """The kernels scale by log2(e) / temperature: below 4.24e-39 that is beyond FP32 although 1 / temperature is not."""
    f = lambda tau: lib.nvfp4_distill_topk(good, 0, 2, 100, 100, good, 4, good, 0, 4, tau, 0, None, None, 0, good, good,  # noqa: E731
                                           100, good, 255, None)
    for tau in (3e-39, 4.2e-39):
        assert f(tau) == binding.ERR_INVALID_ARG, tau
    for tau in (4.3e-39, 1.0, 3e38):
        assert f(tau) == binding.ERR_WORKSPACE, tau    # the argument passes
