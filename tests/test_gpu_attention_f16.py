"""Gradients of attention in f16: what a sequence's gradients go by is its own.

ds enters its products as f16 times a power of two.  That power may depend on the row (dq) or on
the sequence (dk), not on rows of no sequence nor on other sequences: with other values there the
same bits come out, and each sequence is as close to the formulas as by itself.
"""
import pytest
import torch

from test_gpu_attention import check_backward, layers, no_wait_expired, rnd, starts   # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

HF = torch.float16


def gradients(layers, q, k, v, do, qs, ks, causal=False):
    a = layers.attention(q, k, v, q_starts=qs, k_starts=ks, causal=causal, need_backward=True)
    return a, layers.attention_backward(do, q, k, v, a.o, a.lse, q_starts=qs, k_starts=ks, causal=causal)


@pytest.mark.parametrize("dim", [64, 72, 33])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 6e4])
def test_rows_of_no_sequence(layers, bad, dim):
    """Rows before the first and behind the last sequence, whatever they hold."""
    q_lens, k_lens, first, behind = [90, 300], [170, 130], 3, 5
    nq, nk = first + sum(q_lens) + behind, first + sum(k_lens) + behind
    q, k, v, do = (rnd((n, h, dim), i, HF, std) for i, (n, h, std) in enumerate([(nq, 4, 1), (nk, 2, 1), (nk, 2, 1), (nq, 4, 1e-5)]))
    qs, ks = starts(q_lens, first), starts(k_lens, first)
    used = {nq: slice(first, first + sum(q_lens)), nk: slice(first, first + sum(k_lens))}
    clean = []
    for t in (q, k, v, do):
        c = torch.zeros_like(t)
        c[used[t.shape[0]]] = t[used[t.shape[0]]]
        clean.append(c)
    a, g = gradients(layers, *clean, qs, ks)
    check_backward(g, clean[3], a, *clean[:3], q_lens, k_lens, False, dim ** -0.5, first, first)
    for t in (q, k, v, do):
        keep = t[used[t.shape[0]]].clone()
        t.fill_(bad)
        t[used[t.shape[0]]] = keep
    b, h = gradients(layers, q, k, v, do, qs, ks)
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)
    for x, y, name in zip(g, h, ("dq", "dk", "dv")):
        assert torch.equal(x, y), name
    assert g.dq.abs().sum() > 0 and g.dk.abs().sum() > 0


@pytest.mark.parametrize("big", [100.0, 6e4, float("inf"), float("nan")])
def test_other_sequences(layers, big):
    """One sequence with large gradients and values beside others with small ones."""
    q_lens, k_lens = [130, 0, 200, 1, 77], [100, 9, 300, 33, 140]
    n, m = sum(q_lens), sum(k_lens)
    q, k, v, do = (rnd((r, h, 64), i, HF, std) for i, (r, h, std) in enumerate([(n, 6, 1), (m, 2, 1), (m, 2, 1), (n, 6, 1e-5)]))
    qs, ks = starts(q_lens), starts(k_lens)
    a, g = gradients(layers, q, k, v, do, qs, ks)
    check_backward(g, do, a, q, k, v, q_lens, k_lens, False, 0.125)
    do2, v2 = do.clone(), v.clone()
    do2[130:330], v2[109:409] = big, big     # the third sequence's
    b, h = gradients(layers, q, k, v2, do2, qs, ks)
    for rows in (slice(0, 130), slice(330, None)):
        assert torch.equal(a.o[rows], b.o[rows]) and torch.equal(g.dq[rows], h.dq[rows])
    for rows in (slice(0, 109), slice(409, None)):
        assert torch.equal(g.dk[rows], h.dk[rows]) and torch.equal(g.dv[rows], h.dv[rows])


@pytest.mark.parametrize("big", [6e4, float("inf")])
def test_other_rows(layers, big):
    """A row of large gradients leaves the dq of the others, and other key heads' gradients, as they are."""
    q, k, v, do = (rnd((300, h, 64), i, HF, std) for i, (h, std) in enumerate([(4, 1), (2, 1), (2, 1), (4, 1e-5)]))
    _, g = gradients(layers, q, k, v, do, None, None, causal=True)
    do[40, 1] = big
    _, h = gradients(layers, q, k, v, do, None, None, causal=True)
    keep = torch.ones((300, 4), dtype=torch.bool, device="cuda")
    keep[40, 1] = False
    assert torch.equal(g.dq[keep], h.dq[keep])
    assert torch.equal(g.dk[:, 1], h.dk[:, 1]) and torch.equal(g.dv[:, 1], h.dv[:, 1])
    if big == float("inf"):     # hidden from the keys behind its row; the power goes by finite values
        assert torch.equal(g.dk[40 + 256:], h.dk[40 + 256:])


@pytest.mark.parametrize("group,kv", [(1, 3), (5, 2)])
def test_many_short_sequences(layers, group, kv):
    """More sequences than rows of a block's share, empty ones among them, each of its own size of gradients."""
    lens = [(i * 7) % 5 for i in range(700)]
    n = sum(lens)
    q, k, v, do = (rnd((n, h, 40), i, HF) for i, h in enumerate((group * kv, kv, kv, group * kv)))
    at, size = 0, torch.ones(n, device="cuda")
    for i, m in enumerate(lens):
        size[at:at + m] = 2.0 ** -(i % 17)
        at += m
    do = (do.float() * size[:, None, None]).to(HF)
    st = starts(lens)
    a, g = gradients(layers, q, k, v, do, st, None, causal=True)
    at = 0
    for i in range(0, 700, 23):     # by themselves, each within its own bounds
        rows = slice(sum(lens[:i]), sum(lens[:i + 1]))
        one = type(a)(a.o[rows], a.lse[rows])
        part = type(g)(*(t[rows] for t in g))
        check_backward(part, do[rows], one, q[rows], k[rows], v[rows], [lens[i]], [lens[i]], True, 40 ** -0.5)


def test_a_captured_step(layers):
    """Replayed with values of another size, at every replay from the values at hand."""
    lens = [100, 0, 77, 130]
    n, st = sum(lens), starts(lens)
    q, k, v, do = (rnd((n, h, 64), i, HF) for i, h in enumerate((4, 2, 2, 4)))
    gradients(layers, q, k, v, do, st, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, out = gradients(layers, q, k, v, do, st, st)
    for by in (1.0, 2.0 ** -15, 2.0 ** 4, 2.0 ** -8):
        do.copy_((rnd(do.shape, 9, torch.float32) * by).to(HF))
        graph.replay()
        _, want = gradients(layers, q, k, v, do, st, st)
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("big", [6e4, float("inf"), float("nan")])
def test_rows_that_see_no_key(layers, big):
    """More queries than keys under the causal mask: the first ones' do changes nothing, whatever it holds."""
    q_lens, k_lens = [300, 50, 1], [130, 50, 40]
    q, k, v, do = (rnd((sum(n), h, 64), i, HF, std) for i, (n, h, std) in enumerate([(q_lens, 6, 1), (k_lens, 2, 1), (k_lens, 2, 1), (q_lens, 6, 1e-5)]))
    qs, ks = starts(q_lens), starts(k_lens)
    do[:170] = 0
    a, g = gradients(layers, q, k, v, do, qs, ks, causal=True)
    assert (a.lse[:170] == -float("inf")).all() and g.dk[:130].abs().sum() > 0
    check_backward(g, do, a, q, k, v, q_lens, k_lens, True, 0.125)
    do[:44] = big      # whole tiles of queries: a NaN or an infinity reaches keys within 256 tokens of what sees them
    if big == 6e4:
        do[44:170] = big
    _, h = gradients(layers, q, k, v, do, qs, ks, causal=True)
    assert (h.dq[:170] == 0).all()
    for x, y, name in zip(g, h, ("dq", "dk", "dv")):
        assert torch.equal(x, y), name
