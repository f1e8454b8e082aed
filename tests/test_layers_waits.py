"""Leaving a ring of copies, without a GPU: before a block uses a ring's memory again or
ends, its producer waits for the copies that may still be on their way.  last_copies says
which barriers at which parity; here it runs on the host against a model of the barriers,
for every ring size and number of copies.  (No wait is made to run out on a GPU.)"""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_rasterizer_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "tc_common.cuh"

// Copy j fills stage j % N: phase j / N of that stage's barrier, complete when it lands.
template <uint32_t N>
int check()
{
    int wrong = 0;
    for (uint32_t issued = 0; issued <= 4 * N + 1; ++issued) {
        const uint32_t safe = issued > N ? issued - N : 0;   // landed: their stages were filled again
        for (uint32_t late = safe; late <= issued; ++late) {  // the one copy that has not landed; issued: none
            std::vector<uint32_t> phase(N, 0);
            for (uint32_t j = 0; j < issued; ++j) phase[j % N] += j != late;
            bool waits = false;
            uint32_t visited = 0;
            gs::tc::last_copies<N>(issued, [&](uint32_t s, uint32_t parity) {
                ++visited;
                waits = waits || (phase[s] & 1) == parity;   // the phase of that parity is not complete
            });
            wrong += waits != (late < issued) || visited != issued - safe;
        }
    }
    return wrong;
}

int main()
{
    const int wrong = check<1>() + check<3>() + check<4>() + check<5>() + check<6>() + check<8>() + check<10>();
    std::printf("%d\n", wrong);
    return wrong != 0;
}
"""


def test_last_copies_are_waited_for(tmp_path):
    from differentiable_rasterizer_gb300 import build
    src, out = tmp_path / "ring.cu", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.run([build._nvcc(), "-std=c++17", "--extended-lambda", "-I", CSRC, *build.ARCH, str(src), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("name,rings", [("gemm.cu", 2), ("glu_narrow.cu", 2)])
def test_every_ring_is_left_so(name, rings):
    """Each producer ends with that wait, whether its loop ended or gave up, and without looking at the block's flag."""
    text = open(os.path.join(CSRC, name)).read()
    assert len(re.findall(r"last_copies<[\w:]+>\(.*mbar_wait_alone\(", text)) == rings


def test_few_rows_products_end_before_the_ring_is_used_again():
    """The issuer itself waits for its products: the others' wait ends at once when the block has given up."""
    text = open(os.path.join(CSRC, "gemm.cu")).read()
    assert re.search(r"mma_commit<false>\(bar_acc\);[^\n]*\n\s*if \(!mbar_wait_alone\(bar_acc, 0\)\)", text)


def test_contractions_past_the_bound_are_refused():
    """A product so deep that the wait for it would run out is refused, the deepest that is not answers.
    Size queries alone, which check all but the workspace and queue nothing: the pointers are none."""
    import ctypes

    from differentiable_rasterizer_gb300 import abi, build
    build.build()

    def query(name, args):
        return getattr(abi.lib(), name)(args, None, ctypes.byref(ctypes.c_size_t(0)), None)

    def linear(rows, k, type_, bias=4096):
        return query("gs_linear", abi.linear_args(rows, k, 8, 4096, k, 4096, k, 0, 0, bias, 0, 0, 4096, 8, 0, 0, type_, 1, 1, 0))

    def glu(k):
        return query("gs_glu", abi.glu_args(100, k, 8, 4096, k, 4096, k, 4096, k, 0, 0, 0, 4096, 8, 0, 0, 0, 0, 1, 1, 2))

    deep, ok, bad = 1 << 27, abi.GS_OK, abi.GS_ERR_INVALID_ARG
    assert linear(100, deep, abi.GS_BF16) == ok and linear(100, deep + 64, abi.GS_BF16) == bad
    assert linear(100, 2 * deep, abi.GS_E4M3) == ok and linear(100, 2 * deep + 128, abi.GS_E4M3) == bad
    assert linear(4, 8 * deep, abi.GS_BF16) == ok and linear(4, 8 * deep + 1024, abi.GS_BF16) == bad   # eight CTAs share k
    assert linear(100, 8 * deep, abi.GS_BF16, bias=0) == ok   # split over the SMs
    assert glu(deep) == ok and glu(deep + 64) == bad
