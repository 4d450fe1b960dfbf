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

SM_BYTES, CTA_BYTES, SM_COLUMNS = 228 * 1024, 1024, 512   # shared memory of an SM, of it reserved for each CTA; TMEM


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("shape")
    (d / "shape.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-I", CSRC, str(d / "shape.cpp"), "-o", str(d / "shape")], check=True)
    out = subprocess.run([str(d / "shape")], check=True, capture_output=True, text=True).stdout
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
