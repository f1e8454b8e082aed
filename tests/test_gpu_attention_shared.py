"""Outputs of attention that lie where its inputs do."""
import pytest
import torch

from test_gpu_attention import layers, no_wait_expired, rnd, starts   # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
LENS = [70, 1, 130, 300]
N = sum(LENS)


def inputs(dim, dt):
    return tuple(rnd((N, h, dim), i, dt) for i, h in enumerate((4, 2, 2, 4)))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128, 33])
def test_what_may_be_shared(layers, dim, dt):
    """o in q's place, dq in q's or do's: the same bits."""
    q, k, v, do = inputs(dim, dt)
    seq = dict(q_starts=starts(LENS), causal=True)
    a = layers.attention(q, k, v, need_backward=True, **seq)
    g = layers.attention_backward(do, q, k, v, a.o, a.lse, **seq)
    q2, d2, q3 = q.clone(), do.clone(), q.clone()
    b = layers.attention(q2, k, v, out=q2, **seq)
    assert b.o.data_ptr() == q2.data_ptr() and torch.equal(q2, a.o)
    for do2, qq, dq in ((do, q3, q3), (d2, q, d2)):
        h = layers.attention_backward(do2, qq, k, v, None, a.lse, out=(dq, torch.empty_like(k), torch.empty_like(v)), **seq)
        assert torch.equal(dq, g.dq) and torch.equal(h.dk, g.dk) and torch.equal(h.dv, g.dv)


def test_single_tokens_in_place(layers):
    """Keys in parts, joined into q's place."""
    q, k, v = rnd((5, 8, 128), 0, BF), rnd((20000, 2, 128), 1, BF), rnd((20000, 2, 128), 2, BF)
    a = layers.attention(q, k, v)
    layers.attention(q, k, v, out=q)
    assert torch.equal(q, a.o)


def test_shared_memory_is_refused(layers):
    q, k, v, do = inputs(64, BF)
    same = rnd((N, 2, 64), 9, BF)
    for kk, vv, match in ((same, v, "out: shares memory with k"), (k, same, "out: shares memory with v")):
        with pytest.raises(ValueError, match=match):
            layers.attention(rnd((N, 2, 64), 0, BF), kk, vv, out=same)
    a = layers.attention(q, k, v, need_backward=True)
    new = [torch.empty_like(t) for t in (q, k, v)]
    for out, match in (((new[0], k, new[2]), "dk: shares memory with k"), ((new[0], new[1], v), "dv: shares memory with v"),
                       ((new[0], v, new[2]), "dk: shares memory with v"), ((new[0], new[1], k), "dv: shares memory with k"),
                       ((new[0], new[1], new[1]), "dk: shares memory with dv"), ((new[0], new[0][:, :2], new[2]), "dq: shares memory with dk"),
                       ((new[0], new[1], new[0][:, 2:]), "dq: shares memory with dv"), ((new[0], q[:, 1:3], new[2]), "dk: shares memory with q"),
                       ((new[0], new[1], do[:, :2]), "dv: shares memory with do")):
        with pytest.raises(ValueError, match=match):
            layers.attention_backward(do, q, k, v, a.o, a.lse, out=out)
    square = layers.attention(same, same, same, need_backward=True)
    with pytest.raises(ValueError, match="dq: shares memory with k"):
        layers.attention_backward(same, same, same, same, square.o, square.lse, out=(same, torch.empty_like(same), torch.empty_like(same)))


@pytest.mark.parametrize("rows", [1, 40])
def test_neighbours_are_not_refused(layers, rows):
    """Columns of one buffer, heads one behind the other or interleaved, rows behind rows."""
    h, d = 4, 64
    for pad in (0, 8, 200):
        for layout in ("blocks", "interleaved"):
            buf = rnd((rows, 4 * h * d + pad), 1, BF)
            body = buf[:, pad // 2:pad // 2 + 4 * h * d]
            if layout == "blocks":
                q, k, v, o = (body[:, i * h * d:(i + 1) * h * d].unflatten(1, (h, d)) for i in range(4))
            else:
                q, k, v, o = body.unflatten(1, (h, 4, d)).unbind(2)
            want = layers.attention(q.clone(), k.clone(), v.clone(), need_backward=True)
            got = layers.attention(q, k, v, need_backward=True, out=o)
            assert torch.equal(got.o, want.o) and torch.equal(got.lse, want.lse)
            grads = rnd((rows, 3 * h * d + pad), 2, BF)[:, :3 * h * d]
            out = [grads[:, i * h * d:(i + 1) * h * d].unflatten(1, (h, d)) for i in range(3)] if layout == "blocks" else grads.unflatten(1, (h, 3, d)).unbind(2)
            do = rnd((rows, h, d), 3, BF)
            g = layers.attention_backward(do, q, k, v, o, got.lse, out=out)
            w = layers.attention_backward(do, q.clone(), k.clone(), v.clone(), o, got.lse)
            assert all(torch.equal(x, y) for x, y in zip(g, w))
    whole = rnd((4 * rows, h, d), 5, BF)
    q, k, v, o = whole.split(rows)
    assert torch.equal(layers.attention(q, k, v).o, layers.attention(q, k, v, out=o).o)
