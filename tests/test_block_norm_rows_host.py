"""Which rows the block norm reads in pieces of eight columns, run on the host: no piece reaches beyond the matrix."""
from test_attention_host import run_on_host

PROGRAM = r"""
#include <cstdio>
#include "rows.cuh"

int main()
{
    int wrong = 0, pieces = 0;
    const void* const base = (const void*)4096;
    for (int type : {GS_F32, GS_BF16})
        for (int64_t cols = 1; cols <= 40; ++cols)
            for (int64_t ld = cols; ld <= cols + 20; ++ld)
                for (int64_t rows = 1; rows <= 4; ++rows)
                    for (int64_t row = 0; row < rows; ++row)
                        for (int64_t col = 0; col < cols; col += 8) {
                            const bool inside = row > 0 && row + 1 < rows;   // as fetch asks
                            if (!gs::rows::piece_rows(base, ld, type) || !(inside || cols % 8 == 0)) continue;
                            ++pieces;
                            wrong += row * ld + col + 8 > (rows - 1) * ld + cols;
                        }
    std::printf("%d of %d\n", wrong, pieces);
    return wrong != 0 || pieces == 0;
}
"""


def test_pieces_lie_in_the_matrix(tmp_path):
    run_on_host(PROGRAM, tmp_path)
