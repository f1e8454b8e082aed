"""How the attention kernels find a row's sequence and what of a tile counts for a key, run on the host."""
import os
import subprocess

import pytest

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


COLUMNS = r"""
#include <cstdio>
#include <cstdlib>
#include "attention.cuh"

using namespace gs::attn;

int main()
{
    int wrong = 0;
    const int lengths[] = {1, 5, 127, 128, 1000, 1 << 24, (1 << 24) + 1000, 20000001, 0x7fffffff - 1024};
    const int groups[] = {1, 2, 3, 7, 16, 71, 128};
    std::srand(1);
    for (int lq : lengths)
        for (int lk : lengths)
            for (int group : groups)
                for (int trial = 0; trial < 300; ++trial) {
                    const int tokens = 128 / group, key = trial % 3 ? std::rand() % lk : (lk - 1 < trial ? lk - 1 : trial);
                    const Sequence s = {0, lq, 0, lk, 0};
                    const bool causal = trial % 2;
                    // a tile anywhere: the first, the last, around the first query that sees the key
                    const int64_t tiles = ((int64_t)lq + tokens - 1) / tokens;
                    int64_t tile = trial % 5 == 0 ? 0 : (trial % 5 == 1 ? tiles - 1 : std::rand() % tiles);
                    if (trial % 5 == 2 && first_query(s, key, causal) < lq) tile = first_query(s, key, causal) / tokens;
                    const int t0 = (int)(tile * tokens);
                    const Columns c = columns_of(s, key, t0, tokens, group, causal);
                    for (int e = 0; e < tokens * group; ++e) {
                        const int64_t token = (int64_t)t0 + e / group;
                        const bool counts = token < lq && (!causal || key <= token + lk - (int64_t)lq);
                        wrong += counts != (e >= c.from && e < c.to);
                    }
                    wrong += c.to > 128;
                    const int64_t seen = causal ? (int64_t)t0 + 1 + lk - lq : lk;
                    wrong += keys_seen(s, t0, causal) != (seen < 0 ? 0 : (seen < lk ? seen : lk));
                }
    // what f16's terms lose, keys 2^-25 each, below 2^-13 up to 2^24 keys; no more than asks for
    for (int keys : {0, 1, 4096, 4097, 8192, 8193, 1000000, 1 << 24, (1 << 24) + 1, 0x7fffffff - 1024}) {
        const int up = held_up(keys);
        wrong += up < 0 || up > 12 || (keys <= 1 << 24 && keys > 4096ll << up) || (up > 0 && keys <= 4096ll << (up - 1));
    }
    std::printf("%d\n", wrong);
    return wrong != 0;
}
"""


def test_rows_of_a_tile_that_count_for_a_key(tmp_path):
    """Against the definition, up to the longest sequences and past 2^31 packed rows."""
    run_on_host(COLUMNS, tmp_path)


@pytest.mark.parametrize("name", ["gs_attention", "gs_attention_bwd"])
def test_scale_whose_product_is_infinite(name):
    """The scores are taken times scale log2(e): finite for every scale that is taken."""
    from differentiable_rasterizer_gb300 import abi, build
    build.build()
    tensors = dict(q=4096, q_row=256, q_head=64, k=4096, k_row=128, k_head=64, v=4096, v_row=128, v_head=64)
    sizes = dict(q_rows=40, k_rows=50, sequences=1, q_starts=0, k_starts=0, heads=4, kv_heads=2, dim=64, type_=1, causal=0, fill=0)
    more = dict(k_lengths=0, o=4096, o_row=256, o_head=64, lse=0) if name == "gs_attention" else dict(
        d_o=4096, do_row=256, do_head=64, lse=4096, dq=4096, dq_row=256, dq_head=64, dk=4096, dk_row=128, dk_head=64, dv=4096, dv_row=128, dv_head=64)
    for scale, good in ((2.0 ** 127, True), (2.0 ** 127 * 1.001, False), (3.4e38, False), (2.0 ** -149, True)):
        args = getattr(abi, name[3:] + "_args")(**tensors, **sizes, **more, scale=scale)
        if good:
            assert abi.layer_ws_bytes(name, args) >= 0
        else:
            with pytest.raises(abi.GsError):
                abi.layer_ws_bytes(name, args)
