"""Two tiles of queries a CTA: heads of more than 64 columns with rows enough to fill the multiprocessors, and for the forward
4096 keys a sequence in the mean.  Sequences of different lengths, empty and short ones whose second tile has no row, keys
that end within a tile.  Bounds as in test_gpu_attention.py."""
import pytest
import torch

from test_gpu_attention import BF, HF, layers, no_wait_expired, run   # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

CASES = [([4097, 1, 300, 0, 3000], [9000, 5000, 4100, 17, 4095], 8, 8, 128, BF, False),
         ([5000, 77, 2500], [5000, 4000, 3900], 8, 8, 96, HF, True),
         ([3001, 2049], [6000, 3000], 24, 8, 127, BF, True),
         ([5003], [4099], 8, 4, 72, HF, True),
         ([900, 1, 2500, 33, 1500], [900, 700, 2500, 1, 1600], 8, 8, 128, HF, True),
         ([1300, 0, 129], [100, 8, 3], 40, 8, 80, BF, False)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_two_tiles(layers, i):
    q_lens, k_lens, heads, kv, dim, dt, causal = CASES[i]
    run(layers, q_lens, k_lens, heads, kv, dim, dt, causal, seed=i)
    torch.cuda.empty_cache()
