"""The layers' activations at exact pre-activations: one input feature of value 1, so that
the sum is the weight itself and only the activation and the last rounding are left.
From -10 to 10, where GELU's negative tail falls to 8e-23, in every kernel that holds an
activation, which must agree to the bit: few rows, tiles, aligned rows and not.

Bounds (derived from the instructions: ex2.approx 2 ulp, rcp.approx 1 ulp, one rounding an
operation; relative to the result):
  Phi(v)    2^-20 + v^2 2^-23, the latter from rounding v^2 in the exponent; 2^-17 in place of
            2^-20 where the result is rounded to 16 bits (fewer terms)
  sigma(v)  2^-21 + |v| 2^-23
  value     that of Phi or sigma, and one rounding
  slope     the sum of its two terms' errors
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 2.0 ** -126, HF: 2.0 ** -24, F32: 2.0 ** -126}


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


@pytest.fixture(autouse=True)
def no_wait_expired():
    yield
    from differentiable_rasterizer_gb300 import abi
    assert not abi.gs_wait_report()


def points(n, dt):
    return torch.linspace(-10, 10, n, dtype=torch.float64).to(dt)


def value_and_slope(v, act, fine):
    """act(v), act'(v) and their bounds, in 64 bits; fine: not rounded to 16 bits."""
    if act == "silu":
        p, r = torch.sigmoid(v), 2.0 ** -21 + v.abs() * 2.0 ** -23
        slope = p * (1 + v * torch.sigmoid(-v))
        eslope = p * r * (1 + v.abs()) + 2.0 ** -22 * p * (1 + v.abs())
    else:
        # erfc, not ndtr: on the GPU that one subtracts in the tail (0 below -8.3)
        p, r = torch.erfc(v * -math.sqrt(0.5)) / 2, 2.0 ** (-20 if fine else -17) + v * v * 2.0 ** -23
        phi = torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        slope = p + v * phi
        eslope = (p + (v * phi).abs()) * (r + 2.0 ** -22)
    return v * p, (v * p).abs() * (r + 2.0 ** -23), slope, eslope


def check(got, want, slack, what):
    err, bound = (got.double() - want).abs(), U[got.dtype] * want.abs() + slack * (1 + U[got.dtype]) + LEAST[got.dtype]
    bad = ~(err <= bound)
    if bad.any():
        i = int((err / bound).nan_to_num(1e30).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i}: got {got.flatten()[i].item()!r} "
                             f"want {want.expand_as(got).flatten()[i].item()!r}")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("out", [F32, BF, HF])
def test_values(layers, act, dt, out):
    """1 to 64 rows run the few-rows kernel, 65 and 300 tiles; 4001 columns end inside a piece."""
    v = points(4001, dt).cuda()
    v[0], v[1] = 0.0, -0.0
    want, slack, _, _ = value_and_slope(v.double(), act, out == F32)
    rows = []
    for n in (4001, 4000, 72):
        for m in (1, 64, 65, 300):
            x = torch.ones((m, 1), dtype=dt, device="cuda")
            y = layers.linear(x, v[:n, None].contiguous(), act=act, out_dtype=out).y
            check(y, want[:n].expand(m, n), slack[:n], f"{m} x {n}")
            wide = torch.empty((m, n + 3), dtype=out, device="cuda")[:, 1:1 + n]   # rows of odd pitch and base
            layers.linear(x, v[:n, None].contiguous(), act=act, out=wide)
            rows += [y[0], y[-1], wide[0], wide[-1]]
    for r in rows:   # one value a point, whichever kernel made it
        assert torch.equal(r, rows[0][:len(r)])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_slopes(layers, act, dt):
    """The bias's gradient of one row is the unrounded slope: eight columns a thread and one."""
    v = points(4001, dt).cuda()
    v[0], v[1] = 0.0, -0.0
    _, _, want, slack = value_and_slope(v.double(), act, True)
    got = []
    for n in (4001, 4000):
        x, w = torch.ones((1, 1), dtype=dt, device="cuda"), torch.ones((n, 1), dtype=dt, device="cuda")
        g = layers.linear_backward(torch.ones((1, n), device="cuda"), x, w, z=v[None, :n].contiguous(), act=act, bias=True,
                                   db_dtype=F32, dw_dtype=F32)
        check(g.db, want[:n], slack[:n], f"db {n}")
        check(g.dw[:, 0], want[:n], slack[:n] + U[dt] * want[:n].abs() + LEAST[dt], f"dw {n}")   # dz in 16 bits
        got.append(g.db)
    assert torch.equal(got[0][:4000], got[1])


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", [BF, HF])
def test_gated(layers, act, dt):
    """Gated layers: few rows and tiles forward; gradients in one pass, as products, and from saved projections."""
    for f in (128, 127, 504, 501):
        v = points(f, dt).cuda()
        val, ev, slope, es = value_and_slope(v.double(), act, False)
        wg, wu = v[:, None].contiguous(), torch.ones((f, 1), dtype=dt, device="cuda")
        for m in (1, 64, 65):
            x = torch.ones((m, 1), dtype=dt, device="cuda")
            h = layers.glu(x, wg, wu, act=act).h
            check(h, val.expand(m, f), ev + 2.0 ** -24 * val.abs(), f"h {m} x {f}")
        x = torch.ones((1, 1), dtype=dt, device="cuda")
        dh = torch.ones((1, f), dtype=dt, device="cuda")
        for saved in ((None, None), (v[None].contiguous(), wu.t().contiguous())):
            g = layers.glu_backward(dh, x, wg, wu, *saved, act=act, dw_dtype=F32)
            check(g.dw_up[:, 0], val, ev + U[dt] * val.abs() + LEAST[dt], f"dw_up {f}")
            check(g.dw_gate[:, 0], slope, es + U[dt] * slope.abs() + LEAST[dt], f"dw_gate {f}")
