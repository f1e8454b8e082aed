"""Attention over packed sequences on the GPU against the formulas in 64 bits.

Bounds, per element, from the formulas and the stated roundings (derived before the first
run; no case has its own).  With u(T) half a step of type T relative to the value:
  score   dt = scale (dim 2^-23 sum |q| |k|) + 2^-21 |t|: a product of dim terms added in fp32,
          each step truncating, then scaled and taken from a maximum in fp32
  p       e^dt - 1 <= 1.1 dt relative (dt < 0.1), the exponential's 2^-21, its rounding u
  o       (u + 2.2 dt + 2^-20 + keys 2^-23) sum p |v|, u |o| for o's own rounding: the sum
          of p is off by dt as well, and p v adds in fp32, truncating
  lse     dt + 2^-20 + 2^-22 |lse| + keys 2^-23
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


def run(layers, q_lens, k_lens, heads, kv, dim, dt, causal, seed=0, scale=None, std=1.0, need_backward=True):
    q, k, v = (rnd((sum(n), h, dim), seed + i, dt, std if i < 2 else 1.0) for i, (n, h) in enumerate([(q_lens, heads), (k_lens, kv), (k_lens, kv)]))
    one = len(q_lens) == 1
    a = layers.attention(q, k, v, q_starts=None if one else starts(q_lens), k_starts=None if one else starts(k_lens), causal=causal,
                         scale=scale, need_backward=need_backward)
    assert (a.lse is not None) == need_backward
    check_forward(a.o, a.lse, q, k, v, q_lens, k_lens, causal, scale or dim ** -0.5)
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
