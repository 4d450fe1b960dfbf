"""Host-side checks of the mixture-of-experts and 8-bit entry points, and the plan's sizes (CPU).

Every call here is refused: nothing is launched, with or without a GPU.
"""
import ctypes
import os
import shutil
import subprocess

import pytest

from nvfp4_weight_only_02_gb300 import binding, build

P = ctypes.c_void_p
good, bad = P(4096), P(4096 + 4)   # never dereferenced
BIG = 1 << 40                      # bytes of a plan or workspace


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _refused(f, invalid=(), shape=(), alignment=(), workspace=()):
    for code, cases in ((binding.ERR_INVALID_ARG, invalid), (binding.ERR_SHAPE, shape),
                        (binding.ERR_ALIGNMENT, alignment), (binding.ERR_WORKSPACE, workspace)):
        for kw in cases:
            assert f(**kw) == code, (kw, f(**kw))


NO_PLAN = [dict(T=0), dict(k=0), dict(k=33), dict(E=0), dict(E=1025), dict(T=(1 << 24) + 1), dict(T=1 << 23, k=4), dict(T=-1)]


def test_plan_sizes(lib):
    assert lib.nvfp4_moe_plan_bytes(1, 1, 1) > 0 and lib.nvfp4_moe_padded_rows(1, 1, 1) == 128
    assert lib.nvfp4_moe_padded_rows(1000, 4, 3) == (4000 // 128 + 3) * 128
    for kw in NO_PLAN:
        a = dict(T=4, k=2, E=8)
        a.update(kw)
        assert lib.nvfp4_moe_plan_bytes(a["T"], a["k"], a["E"]) == 0
        assert lib.nvfp4_moe_padded_rows(a["T"], a["k"], a["E"]) == 0
        assert lib.nvfp4_moe_plan_part(a["T"], a["k"], a["E"], 0) == 0
        assert lib.nvfp4_moe_linear_workspace_bytes(a["T"], a["k"], a["E"], 64, 64) == 0
    parts = [lib.nvfp4_moe_plan_part(100, 3, 7, p) for p in range(3)]
    assert len(set(parts)) == 3 and all(p % 16 == 0 and 0 < p < lib.nvfp4_moe_plan_bytes(100, 3, 7) for p in parts)
    for f in (lib.nvfp4_moe_gemm_workspace_bytes, lib.nvfp4_moe_linear_workspace_bytes,
              lib.nvfp4_moe_linear_backward_workspace_bytes):
        assert f(100, 3, 7, 96, 64) > 0
        for N, K in ((0, 64), (96, 0), (96, 48), ((1 << 24) + 1, 64), (96, (1 << 24) + 32)):
            assert f(100, 3, 7, N, K) == 0, (N, K)
    # the backward pass contracts over N
    assert lib.nvfp4_moe_gemm_workspace_bytes(100, 3, 7, 100, 64) > 0
    assert lib.nvfp4_moe_linear_backward_workspace_bytes(100, 3, 7, 100, 64) == 0
    assert lib.nvfp4_moe_linear_backward_workspace_bytes(1, 1, 1, 1 << 24, 1 << 24) == 0


def test_route(lib):
    f = lambda z=good, dt=0, T=4, E=8, ld=8, k=2, how=0, b=None, scale=1.0, w=good, e=good, p=good, n=BIG: \
        lib.nvfp4_moe_route(z, dt, T, E, ld, k, how, 1, b, scale, w, e, p, n, None)  # noqa: E731
    _refused(f, [dict(z=None), dict(w=None), dict(e=None), dict(p=None), dict(dt=2), dict(how=2), dict(scale=float("nan")),
                 dict(scale=float("inf"))],
             [dict(ld=7), dict(k=9)] + [dict(kw, ld=2000) for kw in NO_PLAN],
             [dict(z=bad), dict(b=bad), dict(w=bad), dict(e=bad), dict(p=bad)], [dict(n=64), dict(n=0)])
    g = lambda d=good, z=good, dt=0, T=4, E=8, ld=8, k=2, how=0, scale=1.0, w=good, e=good, o=good, lo=8: \
        lib.nvfp4_moe_route_backward(d, z, dt, T, E, ld, k, how, 1, scale, w, e, o, lo, None)  # noqa: E731
    _refused(g, [dict(d=None), dict(z=None), dict(w=None), dict(e=None), dict(o=None), dict(dt=2), dict(how=-1),
                 dict(scale=float("nan"))], [dict(ld=7), dict(lo=7), dict(k=9)] + [dict(kw, ld=2000, lo=2000) for kw in NO_PLAN],
             [dict(d=bad), dict(z=bad), dict(w=bad), dict(e=bad), dict(o=bad)])


def test_plan(lib):
    f = lambda e=good, T=4, k=2, E=8, p=good, n=BIG, ws=None, wn=0: \
        lib.nvfp4_moe_plan(e, T, k, E, p, n, ws, wn, None)  # noqa: E731
    _refused(f, [dict(e=None), dict(p=None)], NO_PLAN, [dict(e=bad), dict(p=bad), dict(ws=bad)],
             [dict(n=64), dict(ws=good, wn=255)])


def test_combine(lib):
    f = lambda y=good, dt=0, w=good, p=good, n=BIG, T=4, k=2, E=8, N=64, b=None, o=good, odt=0: \
        lib.nvfp4_moe_combine(y, dt, w, p, n, T, k, E, N, b, o, odt, None)  # noqa: E731
    _refused(f, [dict(y=None), dict(o=None), dict(p=None), dict(dt=2), dict(odt=3)],
             NO_PLAN + [dict(N=0), dict(N=(1 << 24) + 1), dict(T=1 << 20, N=1 << 20)],
             [dict(y=bad), dict(w=bad), dict(p=bad), dict(b=bad), dict(o=bad)], [dict(n=64)])
    g = lambda d=good, y=good, dt=0, w=good, p=good, n=BIG, T=4, k=2, E=8, N=64, dy=good, dw=good: \
        lib.nvfp4_moe_combine_backward(d, y, dt, w, p, n, T, k, E, N, dy, dw, None)  # noqa: E731
    _refused(g, [dict(d=None), dict(w=None), dict(p=None), dict(dy=None, dw=None), dict(y=None), dict(dt=2)],
             NO_PLAN + [dict(N=0)], [dict(d=bad), dict(y=bad), dict(w=bad), dict(p=bad), dict(dy=bad), dict(dw=bad)],
             [dict(n=64)])


def test_quantisers(lib):
    f = lambda x=good, dt=0, ld=64, so=0, p=good, n=BIG, T=4, k=2, E=8, K=64, c=good, s=good, ct=None, st=None: \
        lib.nvfp4_moe_quantize(x, dt, ld, so, p, n, T, k, E, K, c, s, ct, st, None)  # noqa: E731
    _refused(f, [dict(x=None), dict(p=None), dict(dt=2), dict(c=None, s=None), dict(s=None), dict(ct=good)],
             NO_PLAN + [dict(K=0, ld=0), dict(K=48), dict(ld=32), dict(K=(1 << 24) + 32, ld=1 << 26)],
             [dict(x=bad), dict(ld=68), dict(dt=1, ld=66), dict(p=bad), dict(c=bad), dict(s=bad), dict(ct=bad, st=good),
              dict(ct=good, st=bad)], [dict(n=64)])
    g = lambda w=good, dt=0, E=4, N=64, K=64, c=good, s=good, ct=None, st=None: \
        lib.nvfp4_mx_quantize_experts(w, dt, E, N, K, c, s, ct, st, None)  # noqa: E731
    _refused(g, [dict(w=None), dict(dt=2), dict(c=None, s=None), dict(c=None), dict(st=good)],
             [dict(E=0), dict(E=1025), dict(N=0), dict(K=0), dict(K=40), dict(N=1 << 24, K=1 << 24)],
             [dict(w=bad), dict(c=bad), dict(s=bad), dict(ct=bad, st=good), dict(ct=good, st=bad)])


def test_products(lib):
    f = lambda a=good, b=good, c=good, d=good, p=good, n=BIG, T=4, k=2, E=8, N=64, K=64, y=good, dt=0, ws=good, wn=BIG: \
        lib.nvfp4_moe_gemm(a, b, c, d, p, n, T, k, E, N, K, y, dt, ws, wn, None)  # noqa: E731
    wrong = NO_PLAN + [dict(N=0), dict(K=48)]
    _refused(f, [dict(a=None), dict(b=None), dict(c=None), dict(d=None), dict(p=None), dict(y=None), dict(ws=None), dict(dt=2)],
             wrong, [dict(a=bad), dict(b=bad), dict(c=bad), dict(d=bad), dict(p=bad), dict(y=bad), dict(ws=bad)],
             [dict(n=64), dict(wn=256)])
    g = lambda x=good, xdt=0, ld=64, c=good, d=good, p=good, n=BIG, T=4, k=2, E=8, N=64, K=64, y=good, dt=0, ws=good, wn=BIG: \
        lib.nvfp4_moe_linear(x, xdt, ld, 0, c, d, p, n, T, k, E, N, K, y, dt, ws, wn, None)  # noqa: E731
    _refused(g, [dict(x=None), dict(c=None), dict(d=None), dict(p=None), dict(y=None), dict(ws=None), dict(dt=2), dict(xdt=2)],
             wrong + [dict(ld=32)], [dict(x=bad), dict(ld=68), dict(c=bad), dict(d=bad), dict(p=bad), dict(y=bad), dict(ws=bad)],
             [dict(n=64), dict(wn=1024)])
    h = lambda dy=good, ydt=0, ld=64, a=good, b=good, c=good, d=good, p=good, n=BIG, T=4, k=2, E=8, N=64, K=64, dx=good, xdt=0, \
        dw=good, wdt=0, ws=good, wn=BIG: lib.nvfp4_moe_linear_backward(dy, ydt, ld, a, b, c, d, p, n, T, k, E, N, K, dx, xdt,  # noqa: E731
                                                                      dw, wdt, ws, wn, None)
    _refused(h, [dict(dy=None), dict(p=None), dict(ws=None), dict(ydt=2), dict(xdt=2), dict(wdt=2), dict(dx=None, dw=None),
                 dict(c=None), dict(d=None), dict(a=None), dict(b=None)],
             wrong + [dict(ld=32), dict(N=40, ld=64)],
             [dict(dy=bad), dict(ld=68), dict(a=bad), dict(b=bad), dict(c=bad), dict(d=bad), dict(p=bad), dict(dx=bad),
              dict(dw=bad), dict(ws=bad)], [dict(n=64), dict(wn=1024)])


def test_int8(lib):
    f = lambda x=good, dt=0, M=4, K=64, ld=64, c=good, s=good: lib.nvfp4_int8_quantize(x, dt, M, K, ld, c, s, None)  # noqa: E731
    _refused(f, [dict(x=None), dict(c=None), dict(s=None), dict(dt=2)],
             [dict(M=0), dict(K=0), dict(K=40), dict(K=131088, ld=131088), dict(ld=48), dict(M=1 << 30, K=131072, ld=131072)],
             [dict(x=bad), dict(ld=68), dict(dt=1, ld=66), dict(c=bad), dict(s=bad)])
    need = lib.nvfp4_int8_linear_workspace_bytes
    assert need(4, 64, 64) > 0
    for a in ((0, 64, 64), (4, 0, 64), (4, 64, 40), (4, 64, 131088), (1 << 30, 1 << 30, 64)):
        assert need(*a) == 0
    g = lambda a=good, s=good, w=good, v=good, M=4, N=64, K=64, y=good, dt=0, ws=good, wn=BIG: \
        lib.nvfp4_int8_gemm(a, s, w, v, M, N, K, y, dt, ws, wn, None)  # noqa: E731
    _refused(g, [dict(a=None), dict(s=None), dict(w=None), dict(v=None), dict(y=None), dict(ws=None), dict(dt=2)],
             [dict(M=0), dict(N=0), dict(K=24)],
             [dict(a=bad), dict(s=bad), dict(w=bad), dict(v=bad), dict(y=bad), dict(ws=bad)], [dict(wn=need(4, 64, 64) - 1)])
    h = lambda x=good, xdt=0, ld=64, M=4, N=64, K=64, w=good, v=good, y=good, dt=0, ws=good, wn=BIG: \
        lib.nvfp4_int8_linear(x, xdt, ld, M, N, K, w, v, y, dt, ws, wn, None)  # noqa: E731
    _refused(h, [dict(x=None), dict(w=None), dict(v=None), dict(y=None), dict(ws=None), dict(dt=2), dict(xdt=2)],
             [dict(M=0), dict(N=0), dict(K=24), dict(ld=48)],
             [dict(x=bad), dict(ld=68), dict(w=bad), dict(v=bad), dict(y=bad), dict(ws=bad)], [dict(wn=need(4, 64, 64) - 1)])


def test_plan_layout_holds_every_distribution(tmp_path):
    """The lists are as long as the worst distribution of rows needs, and the parts do not overlap."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    csrc = os.path.join(os.path.dirname(os.path.abspath(build.__file__)), "csrc")
    src = tmp_path / "plan.cpp"
    src.write_text(r'''
#include <cstdio>
#include <vector>
#include "moe_plan.h"
using namespace nvfp4;
int main()
{
    for (int64_t T : {1, 2, 3, 31, 64, 100, 127, 128, 129, 500, 1000, 4096, 70000})
        for (int k : {1, 2, 5, 8, 32})
            for (int E : {1, 2, 7, 60, 128, 1000, 1024}) {
                const MoeLayout l(T, k, E);
                const int64_t R = T * k;
                if (l.tile_rows % 64 || l.tile_rows > 256) return 1;
                for (int size : {kMoeBlock, l.tile_rows}) {
                    // worst: as many experts as possible with one row more than whole pieces
                    int64_t best = 0;
                    for (int64_t used = 1; used <= std::min<int64_t>(R, E); used++) {
                        int64_t left = R - used, pieces = used;
                        pieces += left / size;
                        best = std::max(best, pieces);
                    }
                    if ((size == kMoeBlock ? l.max_blocks : l.max_tiles) < best) return 2;
                    if (size == l.tile_rows && l.max_tiles < best) return 3;
                }
                const int64_t at[] = {kMoeHeader, l.offsets, l.first_block, l.position, l.order, l.padded, l.blocks, l.tiles,
                                      l.counts, l.total};
                const int64_t size[] = {0, E + 1, E + 1, R, R, R, 4 * l.max_blocks, 4 * l.max_tiles,
                                        l.ctas > 1 ? (int64_t)l.ctas * E : 0};
                for (int i = 0; i < 9; i++)
                    if (at[i] % 4 || at[i] + size[i] > at[i + 1]) return 4;
                // 16-bit counters of a CTA's slots
                if ((T + l.ctas - 1) / l.ctas * k > 65535) return 5;
            }
    puts("ok");
    return 0;
}
''')
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "ok"
