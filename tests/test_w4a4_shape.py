"""Shared memory of the W4A4 kernel for few tokens against the TMEM of an SM (CPU: the host arithmetic compiled alone)."""
import itertools
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_weight_only_02_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "w4a4_shape.h"
using namespace nvfp4;
template <bool kNv, int NT, Tokens kTok> void all(const char *name)
{
    using S = WsShape<kNv, NT, kTok>;
    for (int nk = 1; nk <= 4096; nk++) {
        const int stages = S::stages(nk);
        if (stages > 0)
            std::printf("%s %d %d %d %zu\n", name, nk, stages, S::kTmemCols, S::smem(nk, stages));
    }
}
int main()
{
    all<false, 16, kBf16>("tokens_bf16");
    all<false, 16, kFp32>("tokens_fp32");
    all<false, 16, kCodes>("mx16"); all<false, 32, kCodes>("mx32"); all<false, 64, kCodes>("mx64"); all<false, 128, kCodes>("mx128");
    all<true, 16, kCodes>("nv16"); all<true, 32, kCodes>("nv32"); all<true, 64, kCodes>("nv64"); all<true, 128, kCodes>("nv128");
}
"""

CHOICE = r"""
#include <cstdio>
#include "w4a4_shape.h"
int main()
{
    long M, N, K;
    int fp32;
    while (std::scanf("%ld %ld %ld %d", &M, &N, &K, &fp32) == 4)
        std::printf("%d\n", nvfp4::ws_takes_tokens(M, N, K, fp32 != 0, 152) ? 1 : 0);
}
"""

SM_BYTES, CTA_BYTES, SM_COLUMNS = 228 * 1024, 1024, 512   # shared memory of an SM, of it reserved for each CTA; TMEM


def _run(d, source, text=""):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    (d / "shape.cpp").write_text(source)
    subprocess.run([gxx, "-std=c++17", "-I", CSRC, str(d / "shape.cpp"), "-o", str(d / "shape")], check=True)
    return subprocess.run([str(d / "shape")], check=True, input=text, capture_output=True, text=True).stdout


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    out = _run(tmp_path_factory.mktemp("shape"), PROGRAM)
    rows = [line.split() for line in out.splitlines()]
    return [(r[0], int(r[1]), int(r[2]), int(r[3]), int(r[4])) for r in rows]


def test_ctas_that_fit_an_sm_never_want_more_tmem_than_it_has(launches):
    """tcgen05.alloc waits without a limit, and a CTA of a cluster keeps its columns until its peers on other SMs arrive:
    CTAs of any variants that shared memory lets run together must find their columns free."""
    least = {}
    for _, _, _, cols, smem in launches:
        least[cols] = min(least.get(cols, smem), smem)
    assert set(least) <= {128, 256, 512}
    least[512] = 199 * 1024            # the tile kernels of the library
    for counts in itertools.product(*(range(SM_COLUMNS // c + 2) for c in least)):
        columns = sum(n * c for n, c in zip(counts, least))
        smem = sum(n * (least[c] + CTA_BYTES) for n, c in zip(counts, least))
        assert columns <= SM_COLUMNS or smem > SM_BYTES, dict(zip(least, counts))


def test_two_ctas_share_an_sm(launches):
    for name, nk, stages, _, smem in launches:
        assert smem <= 113 * 1024, (name, nk, stages)


# tokens, N, K, FP32, whether one kernel was the faster one (GPU time, by more than 0.2 us)
MEASURED = [
    (4, 3584, 18944, 0, 1), (6, 3584, 18944, 0, 0), (3, 3584, 18944, 0, 1), (4, 3584, 18944, 1, 1),
    (5, 3584, 18944, 1, 0), (1, 18944, 3584, 0, 1), (4, 18944, 3584, 0, 1), (6, 18944, 3584, 0, 1),
    (7, 18944, 3584, 0, 0), (5, 18944, 3584, 1, 1), (6, 18944, 3584, 1, 0), (6, 8192, 8192, 0, 1),
    (7, 8192, 8192, 0, 0), (4, 8192, 8192, 1, 1), (6, 8192, 8192, 1, 0), (8, 12288, 4096, 0, 1),
    (8, 12288, 4096, 1, 0), (6, 1024, 8192, 0, 1), (7, 1024, 8192, 0, 0), (7, 1024, 8192, 1, 0),
    (10, 1024, 10240, 0, 0), (6, 1024, 12288, 0, 1), (9, 1024, 12288, 0, 0), (12, 3584, 3584, 0, 1),
    (1, 27648, 5120, 0, 1), (2, 27648, 5120, 0, 1), (3, 27648, 5120, 0, 0), (2, 27648, 5120, 1, 0),
    (1, 76032, 3584, 0, 1), (2, 76032, 3584, 0, 0), (1, 76032, 3584, 1, 1), (3, 40000, 2048, 0, 1),
    (4, 40000, 2048, 0, 0), (2, 40000, 2048, 1, 0), (16, 2048, 2048, 0, 1), (17, 512, 512, 0, 0),
]


def test_one_kernel_or_two_as_measured(tmp_path):
    text = "".join("%d %d %d %d\n" % m[:4] for m in MEASURED)
    got = _run(tmp_path, CHOICE, text).split()
    assert [m[:4] for m, g in zip(MEASURED, got) if m[4] != int(g)] == [] and len(got) == len(MEASURED)
