"""Packed query rows (tokens times the query heads of a key head) past 2^31 of them."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("causal", [0, 1])
def test_gradients_of_keys_past_32_bits(causal):
    """2^24 + 1000 tokens of 128 heads against one key head.  q is 0 and lse ln(keys), so that every p is 1 / keys but for
    its rounding, and dv the sum of do over all rows over keys: within the result's rounding (2^-8), p's (2^-8) and the
    exponential's argument (7 2^-24, one rounding of each factor).  q and do are one short buffer, rows and heads 8 columns
    apart; do is 1 in its first and last 500 places only.  (Causal: key j is seen by
    the last keys - j tokens.)"""
    from differentiable_rasterizer_gb300 import abi, build
    build.build()
    tokens, heads, keys, dim = 2 ** 24 + 1000, 128, 128, 8
    places = tokens + heads - 1
    q = torch.zeros((places, dim), dtype=BF, device="cuda")
    do = torch.zeros((places, dim), dtype=BF, device="cuda")
    do[:500], do[-500:] = 1, 1
    lse = torch.full((tokens, heads), math.log(keys), device="cuda")
    k = torch.zeros((keys, 1, dim), dtype=BF, device="cuda")
    v = torch.ones((keys, 1, dim), dtype=BF, device="cuda")
    dk, dv = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    args = abi.attention_bwd_args(tokens, keys, 1, q.data_ptr(), dim, dim, k.data_ptr(), dim, dim, v.data_ptr(), dim, dim, do.data_ptr(), dim, dim,
                                  lse.data_ptr(), 0, 0, 0, 0, 0, dk.data_ptr(), dim, dim, dv.data_ptr(), dim, dim, 1.0, heads, 1, dim, abi.GS_BF16,
                                  causal, 0)
    n = abi.layer_ws_bytes("gs_attention_bwd", args)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    abi.gs_attention_bwd(args, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert not abi.gs_wait_report()

    # do of (token, head) is 1 where token + head is among the first or last 500 places
    def ones(from_token):   # over the tokens from there on
        t = torch.arange(from_token, tokens, dtype=torch.int64, device="cuda")
        first = (500 - t).clamp(0, heads)
        last = (t + heads - (places - 500)).clamp(0, heads)
        return int(first.sum() + last.sum())
    for j in range(keys):
        want = ones(tokens - keys + j if causal else 0) / keys
        got = dv[j].double()
        assert ((got - want).abs() <= (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -20) * want).all(), (j, got[0, 0].item(), want)
    assert torch.isfinite(dk.float()).all()
