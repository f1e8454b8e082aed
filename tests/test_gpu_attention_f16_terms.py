"""Attention in f16 over long contexts: keys whose terms are below f16's smallest numbers count together.

Bounds as in test_gpu_attention.py, and 2^-13 of the row's largest term for what all terms below f16's
normal numbers lose together (half of its smallest step, 2^-25, each, terms being held times 2^-12 of the keys).
"""
import pytest
import torch

from test_gpu_attention import check_forward, layers, no_wait_expired   # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

HF = torch.float16
LOST = 2.0 ** -13


def inputs(rows, heads, keys, dim, first, score):
    """One key, `first`, takes most of the weight and has no value; each of the others has a value of 1 and the score."""
    q = torch.zeros((rows, heads, dim), dtype=HF, device="cuda")
    q[..., 0] = 1
    k = torch.zeros((keys, 1, dim), dtype=HF, device="cuda")
    k[:, 0, 0] = score
    k[first, 0, 0] = 0
    v = torch.ones((keys, 1, dim), dtype=HF, device="cuda")
    v[first] = 0
    return q, k, v


def check(a, k, keys):
    p = torch.exp(k[:, 0, 0].double())
    want = p[p < 0.5].sum() / p.sum()
    score = float(k[:, 0, 0].abs().max())
    rel = 2.0 ** -11 + 2.2 * 2.0 ** -21 * score + 2.0 ** -20 + keys * 2.0 ** -23
    assert ((a.o.double() - want).abs() <= (2.0 ** -11 + rel) * want + LOST).all(), (a.o.flatten()[0].item(), float(want))
    lse = torch.logsumexp(k[:, 0, 0].double(), 0)
    assert ((a.lse.double() - lse).abs() <= 2.0 ** -21 * score + 2.0 ** -20 + keys * 2.0 ** -23).all()


@pytest.mark.parametrize("keys", [40000, 131072])
@pytest.mark.parametrize("rows", [1, 5, 300])
@pytest.mark.parametrize("first", [0, 130, -1])
def test_few_rows(layers, rows, keys, first):
    """Keys in parts: 2^-25.5 of the largest term each."""
    q, k, v = inputs(rows, 2, keys, 64, first, -17.7)
    a = layers.attention(q, k, v, scale=1.0, need_backward=True)
    check(a, k, keys)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("first,score", [(0, -17.7), (130, -17.7), (-1, -17.7), (0, -20.0)])
def test_many_rows(layers, dim, first, score):
    """Enough rows that no keys are in parts, one and two tiles a CTA."""
    keys = 131072
    q, k, v = inputs(20011, 2, keys, dim, first, score)
    check(layers.attention(q, k, v, scale=1.0, need_backward=True), k, keys)


@pytest.mark.parametrize("rows", [3, 3000])
def test_rising_scores(layers, rows):
    """Scores that rise from tile to tile by less and by more than what raises the maximum, and fall again."""
    keys = 5000
    g = torch.Generator().manual_seed(3)
    step = torch.arange(keys) // 128
    for by in (0.3, 1.0, 2.0, 3.0, 3.6, 5.0, 8.0, 10.5, 12.0, 40.0):
        q = torch.zeros((rows, 2, 64), dtype=HF, device="cuda")
        q[..., 0] = 1
        k = torch.zeros((keys, 1, 64), dtype=HF, device="cuda")
        k[:, 0, 0] = (by * (step % 20) + torch.randn(keys, generator=g)).to(HF).cuda()
        v = torch.randn((keys, 1, 64), generator=g).to(HF).cuda()
        a = layers.attention(q, k, v, scale=1.0, need_backward=True)
        check_forward(a.o[-70:], a.lse[-70:], q[-70:], k, v, [min(rows, 70)], [keys], False, 1.0)
        assert torch.equal(a.o[0], a.o[-1])
