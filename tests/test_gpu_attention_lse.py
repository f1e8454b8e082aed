"""lse's rows of no sequence beside a given output."""
import pytest
import torch

from test_gpu_attention import layers, rnd, starts   # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 40])
def test_lse_of_rows_of_no_sequence(layers, tokens):
    lens, first, behind = [tokens, tokens], 3, 5
    n = first + sum(lens) + behind
    q, k = rnd((n, 4, 64), 0, torch.bfloat16), rnd((n, 2, 64), 1, torch.bfloat16)
    st = starts(lens, first)
    torch.cuda.empty_cache()
    junk = torch.full((1 << 20,), float("nan"), device="cuda")   # what the next allocation finds
    del junk
    out = torch.full_like(q, 7.0)
    a = layers.attention(q, k, k, q_starts=st, need_backward=True, out=out)
    b = layers.attention(q, k, k, q_starts=st, need_backward=True)
    assert torch.equal(a.lse, b.lse) and (a.lse[:first] == 0).all() and (a.lse[first + sum(lens):] == 0).all()
    assert (out[:first] == 7).all() and (out[first + sum(lens):] == 7).all()
