"""Attention over packed sequences on the GPU against the formulas in 64 bits.

Bounds, per element, from the formulas and the stated roundings (derived before the first
run; no case has its own).  With u(T) half a step of type T relative to the value:
  score   dt = scale (dim 2^-23 sum |q| |k|) + 2^-21 |t|: a product of dim terms added in fp32,
          each step truncating, then scaled and taken from a maximum in fp32
  p       e^dt - 1 <= 1.1 dt relative (dt < 0.1), the exponential's 2^-21, its rounding u
  o       (u + 2.2 dt + 2^-20 + keys 2^-23) sum p |v|, u |o| for o's own rounding: the sum
          of p is off by dt as well, and p v adds in fp32, truncating
  lse     dt + 2^-20 + 2^-22 |lse| + keys 2^-23
The gradients are compared with the formulas at the forward's stored lse:
  p       1.1 dt + 2^-20 + 2^-22 |lse| relative (the difference t - lse in fp32)
  r       dr = dim 2^-23 sum |do| |v|
  delta   sum of p (dp |r| + dr), keys 2^-23 sum p |r|
  ds      dds = p (dp |r - delta| + dr + ddelta) + u |ds|
  dv      (u + dp + rows 2^-23) sum p |do|;  dq: scale (sum dds |k| + keys 2^-23 sum |ds| |k|);
  dk      the same over the rows, with q
F16 holds p times 2^12 and ds times 2^e, 2 dim max|do| max|v| 2^e <= 2^15 (so at least 2^14):
below its normal numbers a factor is off by half its smallest step, 2^-25.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 2.0 ** -126, HF: 2.0 ** -24, F32: 2.0 ** -126}
TYPES = [BF, HF]


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


@pytest.fixture(autouse=True)
def no_wait_expired():
    """No bounded wait of a kernel may run out."""
    yield
    from differentiable_rasterizer_gb300 import abi
    assert not abi.gs_wait_report()


def rnd(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def starts(lengths, first=0):
    return torch.tensor([first] + list(lengths)).cumsum(0).to(torch.int32).cuda()


def visible(lq, lk, causal):
    m = torch.ones(lq, lk, dtype=torch.bool, device="cuda")
    return m.tril(lk - lq) if causal else m


class Sequence64:
    """One sequence and key head in 64 bits: q [group, lq, dim], k, v [lk, dim]."""

    def __init__(self, q, k, v, causal, scale):
        self.q, self.k, self.v, self.scale = q, k, v, scale
        lq, lk = q.shape[1], k.shape[0]
        self.see = visible(lq, lk, causal)
        t = (q @ k.t()) * scale
        dt = scale * q.shape[2] * 2.0 ** -23 * (q.abs() @ k.abs().t()) + 2.0 ** -21 * t.abs()
        self.dt = (dt * self.see).amax(-1) if lk else torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")   # [group, lq]
        t = t.masked_fill(~self.see, float("-inf"))
        self.lse = torch.logsumexp(t, -1) if lk else torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
        self.p = torch.exp(t - self.lse.clamp_min(-1e300)[..., None])
        self.o = self.p @ v


def close(got, want, slack, name):
    """|got - want| <= u(T) |want| + slack; infinities equal; no NaN."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    t = got.dtype
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), name
    err = torch.where(inf, 0.0, (got - torch.where(inf, 0.0, want)).abs())
    bound = U[t] * torch.where(inf, 0.0, want).abs() + slack * (1 + U[t]) + LEAST[t]
    bad = ~(torch.where(inf, 0.0, err) <= bound)
    if bad.any():
        i = int((err / bound).nan_to_num(1e30).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i} of {tuple(got.shape)}: got {got.flatten()[i].item()} "
                             f"want {want.flatten()[i].item()} bound {bound.expand_as(err).flatten()[i].item()}")


def check_forward(o, lse, q, k, v, q_lens, k_lens, causal, scale, q_first=0, k_first=0, k_slots=None):
    """o (and lse, if there) against the formulas, sequence by sequence and head by head."""
    heads, kv = q.shape[1], k.shape[1]
    g, u = heads // kv, U[q.dtype]
    q0, k0 = q_first, k_first
    for s, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        for h in range(kv):
            hs = slice(h * g, h * g + g)
            x = Sequence64(q[q0:q0 + lq, hs].double().transpose(0, 1), k[k0:k0 + lk, h].double(), v[k0:k0 + lk, h].double(), causal, scale)
            mass = x.p @ x.v.abs()
            slack = (u + 2.2 * x.dt + 2.0 ** -20 + lk * 2.0 ** -23)[..., None] * mass
            close(o[q0:q0 + lq, hs], x.o.transpose(0, 1), slack.transpose(0, 1), f"o of sequence {s}, key head {h}")
            if lse is not None:
                ls = x.dt + 2.0 ** -20 + 2.0 ** -22 * x.lse.abs().nan_to_num(posinf=0.0) + lk * 2.0 ** -23
                close(lse[q0:q0 + lq, hs], x.lse.t(), ls.t(), f"lse of sequence {s}, key head {h}")
        q0, k0 = q0 + lq, k0 + (k_slots[s] if k_slots else lk)


def check_backward(g, do, a, q, k, v, q_lens, k_lens, causal, scale, q_first=0, k_first=0):
    heads, kv = q.shape[1], k.shape[1]
    n, u, dim = heads // kv, U[q.dtype], q.shape[2]
    f16 = q.dtype == HF
    floor_p = 2.0 ** -37 if f16 else 0.0
    floor_ds = 2.0 ** -25 * 2 * dim * float(do.abs().max()) * float(v.abs().max()) * 2.0 ** -14 if f16 and do.numel() and v.numel() else 0.0
    q0, k0 = q_first, k_first
    for s, (lq, lk) in enumerate(zip(q_lens, k_lens)):
        for h in range(kv):
            hs, rows, keys = slice(h * n, h * n + n), slice(q0, q0 + lq), slice(k0, k0 + lk)
            qq, dd = (t[rows, hs].double().transpose(0, 1) for t in (q, do))
            kk, vv = k[keys, h].double(), v[keys, h].double()
            x = Sequence64(qq, kk, vv, causal, scale)
            lse = a.lse[rows, hs].double().t()
            t = ((qq @ kk.t()) * scale).masked_fill(~x.see, float("-inf"))
            p = torch.exp(t - lse.clamp_min(-1e300)[..., None])
            dp = (1.1 * x.dt + 2.0 ** -20 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0))[..., None]
            r = dd @ vv.t()
            delta = (p * r).sum(-1, keepdim=True)
            ds = p * (r - delta)
            dr = dim * 2.0 ** -23 * (dd.abs() @ vv.abs().t())
            ddelta = (p * ((dp + lk * 2.0 ** -23) * r.abs() + dr)).sum(-1, keepdim=True)
            dds = p * (dp * (r - delta).abs() + dr + ddelta) + u * ds.abs() + floor_ds * x.see
            total = n * lq
            close(g.dv[keys, h], (p.transpose(1, 2) @ dd).sum(0),
                  (((u + dp + total * 2.0 ** -23) * p + floor_p * x.see).transpose(1, 2) @ dd.abs()).sum(0), f"dv of sequence {s}, key head {h}")
            close(g.dk[keys, h], scale * (ds.transpose(1, 2) @ qq).sum(0),
                  scale * ((dds + total * 2.0 ** -23 * ds.abs()).transpose(1, 2) @ qq.abs()).sum(0), f"dk of sequence {s}, key head {h}")
            close(g.dq[rows, hs], scale * (ds @ kk).transpose(0, 1),
                  scale * ((dds + lk * 2.0 ** -23 * ds.abs()) @ kk.abs()).transpose(0, 1), f"dq of sequence {s}, key head {h}")
        q0, k0 = q0 + lq, k0 + lk


def run(layers, q_lens, k_lens, heads, kv, dim, dt, causal, seed=0, scale=None, std=1.0, need_backward=True,
        do_std=1.0):
    q, k, v = (rnd((sum(n), h, dim), seed + i, dt, std if i < 2 else 1.0) for i, (n, h) in enumerate([(q_lens, heads), (k_lens, kv), (k_lens, kv)]))
    one = len(q_lens) == 1
    a = layers.attention(q, k, v, q_starts=None if one else starts(q_lens), k_starts=None if one else starts(k_lens), causal=causal,
                         scale=scale, need_backward=need_backward)
    assert (a.lse is not None) == need_backward
    check_forward(a.o, a.lse, q, k, v, q_lens, k_lens, causal, scale or dim ** -0.5)
    if need_backward:
        do = rnd(q.shape, seed + 3, dt, do_std)
        g = layers.attention_backward(do, q, k, v, a.o, a.lse, q_starts=None if one else starts(q_lens),
                                      k_starts=None if one else starts(k_lens), causal=causal, scale=scale)
        check_backward(g, do, a, q, k, v, q_lens, k_lens, causal, scale or dim ** -0.5)
    return a


# one sequence: query and key lengths, heads, key heads, dim
ONE = [(1, 1, 1, 1, 64), (1, 1, 1, 1, 1), (2, 3, 2, 1, 8), (17, 17, 4, 4, 16), (127, 128, 2, 2, 32), (128, 128, 1, 1, 128),
       (129, 129, 3, 1, 40), (255, 257, 6, 2, 72), (256, 256, 4, 2, 64), (300, 512, 5, 5, 80), (1, 1000, 8, 2, 128),
       (7, 4097, 16, 4, 64), (64, 700, 7, 1, 33), (31, 999, 71, 1, 64), (5, 300, 128, 1, 127), (1000, 1, 2, 2, 64),
       (1111, 1111, 8, 8, 96), (2049, 2049, 2, 1, 128), (513, 100, 4, 1, 64), (3, 20000, 2, 2, 128)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lq,lk,heads,kv,dim", ONE)
def test_one_sequence(layers, lq, lk, heads, kv, dim, causal):
    """Lengths of one to many, odd ones, groups that do not divide a tile, causal rows that see nothing (more queries than keys)."""
    run(layers, [lq], [lk], heads, kv, dim, BF, causal, seed=lq)


@pytest.mark.parametrize("lq,lk,heads,kv,dim", [ONE[i] for i in (0, 2, 6, 9, 11, 16)])
def test_f16(layers, lq, lk, heads, kv, dim):
    run(layers, [lq], [lk], heads, kv, dim, HF, True, seed=lq + 1)


@pytest.mark.parametrize("std,do_std", [(4.0, 1.0), (0.01, 1e-4), (1.0, 1e-6), (1.0, 1e4)])
@pytest.mark.parametrize("dt", TYPES)
def test_sizes_of_values(layers, dt, std, do_std):
    """Scores that one key wins, and gradients of a type's smallest and largest sizes (f16's below its normal numbers)."""
    if dt == HF and do_std == 1e4:
        do_std = 100.0   # a sum of do v would leave f16
    run(layers, [300], [300], 4, 2, 64, dt, True, seed=5, std=std, do_std=do_std)


PACKS = [([5, 1, 130, 64], [5, 1, 130, 64], True), ([1] * 40, [3, 700, 1, 129, 128] * 8, True), ([17, 300, 2], [200, 1, 513], False),
         ([0, 7, 0, 0, 129, 1], [3, 0, 0, 5, 40, 1], False), ([9, 0, 4], [2, 8, 300], True), ([1, 1], [0, 0], True),
         ([33] * 70, [33] * 70, True), ([2, 1500, 3], [2, 1500, 3], True)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("i", range(len(PACKS)))
def test_packed_sequences(layers, i, dt):
    """Different lengths, empty sequences, sequences without keys, more than a warp's 32 of them."""
    q_lens, k_lens, causal = PACKS[i]
    run(layers, q_lens, k_lens, 6, 2, [64, 128, 40][i % 3], dt, causal, seed=i)


@pytest.mark.parametrize("need_backward", [False, True])
def test_single_tokens_split_over_blocks(layers, need_backward):
    """Few rows against many keys: parts of the keys, some of them empty for short sequences; the same with the statistics asked for."""
    run(layers, [1] * 5, [9000, 1, 128, 4097, 300], 8, 2, 128, BF, True, need_backward=need_backward)
    run(layers, [3] * 4, [2, 1000, 3, 257], 4, 4, 64, HF, True, need_backward=need_backward)
    run(layers, [200], [6000], 2, 1, 64, BF, True, need_backward=need_backward)


def lay(t, how):
    """t with the same values in another layout: of NaN between them."""
    r, h, d = t.shape
    if how == "slice":        # columns of wider rows, as of one projection
        wide = torch.full((r, h * d + 64), float("nan"), dtype=t.dtype, device="cuda")
        v = wide[:, 32:32 + h * d].view(r, h, d)
    elif how == "heads":      # heads first
        v = torch.full((h, r, d), float("nan"), dtype=t.dtype, device="cuda").transpose(0, 1)
    elif how == "odd":        # neither base nor pitch on 16 bytes
        wide = torch.full((r * (h * d + 3) + 1,), float("nan"), dtype=t.dtype, device="cuda")
        v = wide[1:].as_strided((r, h, d), (h * d + 3, d, 1), 1)
    else:
        return t.clone()
    v.copy_(t)
    return v


@pytest.mark.parametrize("dim", [64, 72, 33])
@pytest.mark.parametrize("how", ["slice", "heads", "odd"])
def test_layouts(layers, how, dim):
    """Inputs and outputs of any strides give the same bits as contiguous ones, and nothing beside them is written."""
    lens = [70, 1, 130]
    n = sum(lens)
    q, k, v, do = (rnd((n, h, dim), i, BF) for i, h in enumerate((4, 2, 2, 4)))
    st = starts(lens)
    a = layers.attention(q, k, v, q_starts=st, causal=True, need_backward=True)
    g = layers.attention_backward(do, q, k, v, a.o, a.lse, q_starts=st, causal=True)
    q2, k2, v2, do2 = (lay(t, how) for t in (q, k, v, do))
    o2 = lay(torch.zeros_like(q), how)
    b = layers.attention(q2, k2, v2, q_starts=st, causal=True, need_backward=True, out=o2)
    assert b.o.data_ptr() == o2.data_ptr() and torch.equal(b.o, a.o) and torch.equal(b.lse, a.lse)
    out = [lay(torch.zeros_like(t), how) for t in (q, k, v)]
    h = layers.attention_backward(do2, q2, k2, v2, o2, b.lse, q_starts=st, causal=True, out=out)
    for x, y, z in zip(h, g, out):
        assert torch.equal(x, y) and x.data_ptr() == z.data_ptr()
    if how == "odd":
        for t in [o2, *out]:
            whole = t.as_strided(((n * (t.shape[1] * dim + 3)) + 1,), (1,), 0)
            assert torch.isnan(whole[0]) and int(torch.isnan(whole).sum()) == 1 + 3 * n


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_rows_of_no_sequence(layers, bad):
    """Rows before, behind and of other sequences have no influence, whatever they hold; rows of no sequence are left as they
    are in given outputs and are zero in allocated ones."""
    q_lens, k_lens, first, behind = [9, 100], [70, 130], 3, 5
    nq, nk = first + sum(q_lens) + behind, first + sum(k_lens) + behind
    q, k, v, do = (rnd((n, h, 64), i, HF) for i, (n, h) in enumerate([(nq, 4), (nk, 2), (nk, 2), (nq, 4)]))
    qs, ks = starts(q_lens, first), starts(k_lens, first)
    used_q, used_k = slice(first, first + sum(q_lens)), slice(first, first + sum(k_lens))
    a = layers.attention(q, k, v, q_starts=qs, k_starts=ks, need_backward=True)
    check_forward(a.o, a.lse, q, k, v, q_lens, k_lens, False, 0.125, first, first)
    g = layers.attention_backward(do, q, k, v, a.o, a.lse, q_starts=qs, k_starts=ks)
    check_backward(g, do, a, q, k, v, q_lens, k_lens, False, 0.125, first, first)
    for t, used in ((a.o, used_q), (a.lse, used_q), (g.dq, used_q), (g.dk, used_k), (g.dv, used_k)):
        rest = torch.ones(t.shape[0], dtype=torch.bool, device="cuda")
        rest[used] = False
        assert (t[rest] == 0).all()
    outside = [t.clone() for t in (q, k, v)]
    for t, used in zip(outside, (used_q, used_k, used_k)):
        keep = t[used].clone()
        t.fill_(bad)
        t[used] = keep
    # the second sequence's values are the first's neighbours: bad there, the first stays as it was
    outside[1][used_k][k_lens[0]:], outside[2][used_k][k_lens[0]:] = bad, bad
    o = torch.full_like(q, 7.0)
    b = layers.attention(*outside, q_starts=qs, k_starts=ks, need_backward=True, out=o)
    mine = slice(first, first + q_lens[0])
    assert torch.equal(b.o[mine], a.o[mine]) and (o[:first] == 7).all() and (o[first + sum(q_lens):] == 7).all()
    out = [torch.full_like(t, 7.0) for t in (q, k, v)]
    d2 = torch.full_like(do, bad)
    d2[used_q] = do[used_q]
    only = starts(q_lens[:1], first), starts(k_lens[:1], first)
    h = layers.attention_backward(d2, *outside, b.o, b.lse, q_starts=only[0], k_starts=only[1], out=out)
    if math.isnan(bad):   # f16's power of two goes by all of do and v: finite ones change no more than roundings
        assert torch.equal(h.dv[first:first + k_lens[0]], g.dv[first:first + k_lens[0]])
    assert torch.isfinite(h.dq[mine]).all() and torch.isfinite(h.dk[first:first + k_lens[0]]).all()
    for t, used in zip(out, (q_lens[0], k_lens[0], k_lens[0])):
        assert (t[:first] == 7).all() and (t[first + used:] == 7).all()


def test_keys_in_use(layers):
    """k_lengths: slots of a cache that are filled in part, NaN behind; lengths beyond the slot are held to it."""
    slots, used, q_lens = [512, 300, 64, 128], [500, 0, 64, 1], [1, 2, 3, 1]
    q, k, v = rnd((7, 8, 128), 0, BF), rnd((sum(slots), 2, 128), 1, BF), rnd((sum(slots), 2, 128), 2, BF)
    at = 0
    for s, n in zip(slots, used):
        k[at + n:at + s] = float("nan")
        v[at + n:at + s] = float("nan")
        at += s
    lengths = torch.tensor(used, dtype=torch.int32, device="cuda")
    a = layers.attention(q, k, v, q_starts=starts(q_lens), k_starts=starts(slots), k_lengths=lengths, causal=True)
    check_forward(a.o, None, q, k, v, q_lens, used, True, 128 ** -0.5, k_slots=slots)
    lengths[2] = 2 ** 31 - 1
    b = layers.attention(q, k, v, q_starts=starts(q_lens), k_starts=starts(slots), k_lengths=lengths, causal=True)
    assert torch.equal(a.o, b.o)


def test_starts_are_held_within_the_rows(layers):
    """Starts beyond the rows are taken for their number; what is read stays inside, and the first sequence is as it should be."""
    q, k, v = rnd((40, 2, 64), 0, BF), rnd((50, 2, 64), 1, BF), rnd((50, 2, 64), 2, BF)
    st = torch.tensor([0, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    a = layers.attention(q, k, v, q_starts=st, k_starts=st, need_backward=True)
    check_forward(a.o, a.lse, q, k, v, [10, 30], [10, 40], False, 0.125)
    st = torch.tensor([-5, 10, 40], dtype=torch.int32, device="cuda")
    b = layers.attention(q, k, v, q_starts=st, k_starts=st, need_backward=True)
    assert torch.equal(a.o[:10], b.o[:10])


def test_offsets_past_32_bits(layers):
    """A cache whose last slot starts beyond 2^32 elements."""
    rows = 2 ** 32 // 256 + 1000
    k = torch.zeros((rows, 2, 128), dtype=BF, device="cuda")
    v = torch.zeros((rows, 2, 128), dtype=BF, device="cuda")
    k[-300:], v[-300:] = rnd((300, 2, 128), 1, BF), rnd((300, 2, 128), 2, BF)
    q = rnd((2, 4, 128), 3, BF)
    ks = torch.tensor([0, 100, rows - 300, rows], dtype=torch.int32, device="cuda")
    qs = torch.tensor([0, 1, 1, 2], dtype=torch.int32, device="cuda")
    a = layers.attention(q, k, v, q_starts=qs, k_starts=ks)
    check_forward(a.o[1:], None, q[1:], k[-300:], v[-300:], [1], [300], False, 128 ** -0.5)
    assert (a.o[0] == 0).all()
    big = torch.zeros((2 ** 31 // 512 + 700, 4, 128), dtype=BF, device="cuda")      # outputs there too
    big[-200:] = rnd((200, 4, 128), 4, BF)
    st = torch.tensor([big.shape[0] - 200, big.shape[0]], dtype=torch.int32, device="cuda")
    kk, vv = rnd((200, 2, 128), 5, BF), rnd((200, 2, 128), 6, BF)
    ks = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    out = torch.empty_like(big)
    layers.attention(big, kk, vv, q_starts=st, k_starts=ks, out=out)
    check_forward(out[-200:], None, big[-200:], kk, vv, [200], [200], False, 128 ** -0.5)


def test_nothing_to_do(layers):
    empty, k = torch.empty((0, 4, 64), dtype=BF, device="cuda"), rnd((9, 2, 64), 0, BF)
    a = layers.attention(empty, k, k, need_backward=True)
    assert a.o.shape == (0, 4, 64) and a.lse.shape == (0, 4)
    g = layers.attention_backward(empty, empty, k, k, a.o, a.lse)
    assert g.dq.shape == (0, 4, 64) and (g.dk == 0).all() and (g.dv == 0).all()
    q, none = rnd((9, 4, 64), 1, BF), torch.empty((0, 2, 64), dtype=BF, device="cuda")
    a = layers.attention(q, none, none, need_backward=True)
    assert (a.o == 0).all() and (a.lse == -math.inf).all()
    g = layers.attention_backward(q, q, none, none, a.o, a.lse)
    assert (g.dq == 0).all() and g.dk.shape == (0, 2, 64)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")     # no sequence at all
    a = layers.attention(q, k, k, q_starts=st, need_backward=True)
    assert (a.o == 0).all()
    g = layers.attention_backward(q, q, k, k, a.o, a.lse, q_starts=st)
    assert (g.dq == 0).all() and (g.dk == 0).all() and (g.dv == 0).all()


def test_nan_stays_in_its_row(layers):
    """A NaN in a query reaches that query's head alone, and all keys' gradients."""
    q, k, v = rnd((200, 2, 64), 0, BF), rnd((200, 2, 64), 1, BF), rnd((200, 2, 64), 2, BF)
    a = layers.attention(q, k, v, causal=True)
    q[50, 1, 3] = float("nan")
    b = layers.attention(q, k, v, causal=True, need_backward=True)
    assert torch.isnan(b.o[50, 1]).all() and torch.isnan(b.lse[50, 1])
    b.o[50, 1] = a.o[50, 1]
    assert torch.equal(a.o, b.o)
    k[199] = float("nan")     # hidden from all rows but the last
    c = layers.attention(rnd((200, 2, 64), 0, BF), k, v, causal=True)
    assert torch.equal(c.o[:199], a.o[:199]) and torch.isnan(c.o[199]).all()


def test_infinite_scores(layers):
    """Scores of minus infinity have no weight."""
    q, k, v = rnd((1, 1, 64), 0, BF).abs(), rnd((3, 1, 64), 1, BF), rnd((3, 1, 64), 2, BF)
    k[1] = -float("inf")
    a = layers.attention(q, k, v)
    b = layers.attention(q, k[[0, 2]].contiguous(), v[[0, 2]].contiguous())
    assert torch.allclose(a.o.float(), b.o.float(), rtol=2 ** -7, atol=1e-6)


def test_runs_give_the_same_bits(layers):
    lens = [400, 33, 900, 1]
    n, st = sum(lens), starts(lens)
    for dt in TYPES:
        q, k, v, do = (rnd((n, h, 80), i, dt) for i, h in enumerate((6, 2, 2, 6)))
        first = None
        for _ in range(5):
            a = layers.attention(q, k, v, q_starts=st, causal=True, need_backward=True)
            now = (*a, *layers.attention_backward(do, q, k, v, a.o, a.lse, q_starts=st, causal=True))
            first = first or now
            assert all(torch.equal(x, y) for x, y in zip(first, now))


def test_streams_and_graphs(layers):
    """On a stream of its own beside another call, and captured and replayed with new values; two graphs share a pool."""
    lens = [100, 1, 77]
    n, st = sum(lens), starts(lens)
    q, k, v, do = (rnd((n, h, 64), i, BF) for i, h in enumerate((4, 2, 2, 4)))

    def step():
        a = layers.attention(q, k, v, q_starts=st, causal=True, need_backward=True)
        return (*a, *layers.attention_backward(do, q, k, v, a.o, a.lse, q_starts=st, causal=True))

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    for t in got:
        assert all(torch.equal(x, y) for x, y in zip(t, want))
    pool = torch.cuda.graph_pool_handle()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            out = step()
        graphs.append((g, out))
    for t in (q, k, v, do):
        t.copy_(t.flip(0))
    want = step()
    for g, out in graphs:
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_against_differences(layers):
    """The change of the loss sum(do o) along a direction, by the formulas in 64 bits at two points either side, is the gradients'
    product with it: within the gradients' 16-bit roundings (2^-8 of each term)."""
    n, heads, kv, dim = 96, 4, 2, 32
    q, k, v, do = (rnd((n, h, dim), 20 + i, BF) for i, h in enumerate((heads, kv, kv, heads)))
    a = layers.attention(q, k, v, causal=True, need_backward=True)
    g = layers.attention_backward(do, q, k, v, a.o, a.lse, causal=True)

    def loss(q, k, v):
        total = 0.0
        for h in range(heads):
            x = Sequence64(q[:, h][None], k[:, h // 2], v[:, h // 2], True, dim ** -0.5)
            total = total + (x.o[0] * do[:, h].double()).sum()
        return total

    point = [t.double() for t in (q, k, v)]
    for i in range(3):
        step = [torch.zeros_like(t) for t in point]
        step[i] = rnd(point[i].shape, 40 + i, F32).double()
        eps = 1e-5
        up, down = (loss(*(p + f * eps * s for p, s in zip(point, step))) for f in (1, -1))
        terms = g[i].double() * step[i]
        want = (up - down) / (2 * eps)
        # independent roundings of the terms (o's in delta among them): six deviations of their root sum of squares
        assert abs(terms.sum() - want) <= 6 * 2.0 ** -8 * terms.square().sum().sqrt() + 1e-6 * abs(want), i


def test_refusals(layers):
    from differentiable_rasterizer_gb300 import abi
    q, k = rnd((8, 4, 64), 0, BF), rnd((8, 2, 64), 1, BF)
    st = starts([3, 5])
    lse = torch.zeros((8, 4), device="cuda")
    for bad, match in ((dict(k=rnd((8, 3, 64), 1, BF), v=rnd((8, 3, 64), 1, BF)), "do not divide"), (dict(v=rnd((7, 2, 64), 1, BF)), "expected"),
                       (dict(k=k.half()), "expected BFloat16"), (dict(q=q[:, 0]), "rows, heads, dim"), (dict(k_starts=st), "q_starts: required"),
                       (dict(q_starts=st.long()), "int32"), (dict(q_starts=st.cpu()), "on cpu"), (dict(q_starts=st, k_starts=st[:2]), "expected 3"),
                       (dict(q_starts=st[:0]), "no value"), (dict(q_starts=st, k_lengths=st), "expected 2"), (dict(out=q[:7]), "out: expected"),
                       (dict(out=q.float()), "out: expected"), (dict(scale="x"), "scale"), (dict(q=q.expand(8, 4, 64).transpose(1, 2)), "contiguous"),
                       (dict(q_starts=st, k_lengths=st[:2], need_backward=True), "k_lengths"), (dict(q=rnd((8, 4, 129), 0, BF)), "columns a head"),
                       (dict(q=q.requires_grad_(False).clone().requires_grad_(True)), "requires grad")):
        with pytest.raises(ValueError, match=match):
            layers.attention(**{**dict(q=q, k=k, v=k), **bad})
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(abi.GsError):
            layers.attention(q, k, k, scale=scale)
    for bad, match in ((dict(lse=None), "lse"), (dict(lse=lse[:7]), "lse"), (dict(do=q[:7]), "do: expected"), (dict(do=q.float()), "do: expected"),
                       (dict(out=(q.clone(), None, k.clone())), "expected dq, dk and dv")):
        with pytest.raises(ValueError, match=match):
            layers.attention_backward(**{**dict(do=q, q=q, k=k, v=k, o=q, lse=lse), **bad})
    wide = torch.empty((8, 4, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        layers.attention(q, k, k, out=wide.as_strided((8, 4, 64), (64, 32, 1)))
    with pytest.raises(abi.GsError):      # heads and rows share places
        layers.attention(q, k, k, out=wide.as_strided((8, 4, 64), (128, 64, 1)))
