"""How the attention kernels find a row's sequence and what of a tile counts for a key, run on the host."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_rasterizer_gb300", "csrc")

SEQUENCE_OF = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attention.cuh"

using namespace gs::attn;

int main()
{
    int wrong = sequence_of(nullptr, 1, 17) != 0;
    std::srand(1);
    for (int trial = 0; trial < 3000; ++trial) {
        const int n = std::rand() % 20;
        std::vector<int32_t> starts(1, std::rand() % 5);
        for (int s = 0; s < n; ++s) starts.push_back(starts.back() + (std::rand() % 2 ? std::rand() % 9 : 0));
        for (int64_t row = 0; row < starts.back() + 4; ++row) {
            uint32_t want = (uint32_t)n;
            for (int s = 0; s < n; ++s)
                if (starts[s] <= row && row < starts[s + 1]) want = (uint32_t)s;
            wrong += sequence_of(starts.data(), (uint32_t)n, row) != want;
        }
        // starts in any order: a number within the array, or count
        for (auto& s : starts) s = std::rand() % 100 - 50;
        for (int64_t row = 0; row < 60; ++row) {
            const uint32_t s = sequence_of(starts.data(), (uint32_t)n, row);
            wrong += s > (uint32_t)n || (s < (uint32_t)n && !(starts[s] <= row && row < starts[s + 1]));
        }
    }
    std::printf("%d\n", wrong);
    return wrong != 0;
}
"""


def run_on_host(program, tmp_path):
    from differentiable_rasterizer_gb300 import build
    src, out = tmp_path / "program.cu", tmp_path / "program"
    src.write_text(program)
    subprocess.run([build._nvcc(), "-std=c++17", "--extended-lambda", "-I", CSRC, *build.ARCH, str(src), "-o", str(out)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_sequence_of_a_row(tmp_path):
    run_on_host(SEQUENCE_OF, tmp_path)
