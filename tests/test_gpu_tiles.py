"""Every tile shape of the products' kernel (single CTAs and pairs, all factor orders, splits
of k, epilogues, gated layers and their gradients) at sizes that the choice by size would
give to another, ragged in every dimension, with one and with several tiles a CTA.

Inputs are small whole numbers, so that every sum is exact in fp32 whatever its order and
every factor exact in 16 bits (asserted): outputs must equal the 64-bit ones rounded once,
to the bit.  A lost or doubled row, k-block, split or tile cannot hide in a tolerance.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
WHOLE = {BF: 256, HF: 2048}   # whole numbers up to here are exact


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


@pytest.fixture(params=[0, 1, 2, 3])
def tile(request, layers):
    from differentiable_rasterizer_gb300 import abi
    abi.gs_layer_tile(request.param)
    yield request.param
    abi.gs_layer_tile(-1)
    assert not abi.gs_wait_report()


def whole(shape, seed, dtype, most):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype).cuda()


def wide(t, pad, off):
    """t as a slice of wider rows of other values."""
    w = torch.full((t.shape[0], t.shape[1] + pad), 99.0, device="cuda").to(t.dtype)[:, off:off + t.shape[1]]
    w.copy_(t)
    return w


def same(got, want, name):
    """got is the 64-bit value, rounded once to its type."""
    assert want.abs().max() < 2 ** 24, name   # exact in fp32 in any order
    want = want.float().to(got.dtype)
    if not torch.equal(got, want):
        bad = (got.float() != want.float())
        r, c = (int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} differ, first at ({r}, {c}): "
                             f"{got[r, c].item()} for {want[r, c].item()}")


SIZES = [(1, 64, 40), (65, 33, 24), (257, 130, 513), (700, 200, 300), (300, 5000, 200), (11000, 72, 520), (1000, 96, 512)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_linear(layers, tile, m, k, n, dt):
    x, w = whole((m, k), 0, dt, 2), whole((n, k), 1, dt, 1)
    b, r = whole((n,), 2, F32, 9), whole((m, n), 3, dt, 200)
    z = x.double() @ w.double().t()
    same(layers.linear(x, w).y, z, "plain")
    same(layers.linear(x, w, out_dtype=F32).y, z, "fp32")
    zb = z + b.double()
    relu = zb.clamp_min(0)
    o = layers.linear(x, w, b, act="relu", residual=r, need_backward=True)
    same(o.y, relu + r.double(), "bias, relu, residual")
    same(o.z, zb, "z")
    same(layers.linear(x, w, b, act="relu").y, relu, "bias, relu")
    r32 = r.float()
    same(layers.linear(x, w, b, act="relu", residual=r32).y, relu + r.double(), "fp32 residual")
    for pad, off in ((8, 0), (24, 16), (7, 3)):   # rows of 16- and 32-byte steps, and of neither
        for res in (r, r32):
            out = wide(res, pad, off)
            layers.linear(x, w, b, residual=wide(res, pad + 2, off), out=out)
            same(out, zb + r.double(), f"rows of {n} + {pad} from {off}")
            got = out.as_strided((m, n + pad), out.stride(), out.storage_offset() - off)
            assert (got[:, :off] == 99).all() and (got[:, off + n:] == 99).all()
    # a smooth activation: its own error beside the rounding (z exact)
    s = layers.linear(x, w, b, act="silu").y
    want = zb * torch.sigmoid(zb)
    u = 2.0 ** -8 if dt == BF else 2.0 ** -11
    assert ((s.double() - want).abs() <= want.abs() * (u + 2.0 ** -20 + zb.abs() * 2.0 ** -22) + 2.0 ** -24).all()


@pytest.mark.parametrize("m,k,n", SIZES)
def test_linear_e4m3(layers, tile, m, k, n):
    x, w = whole((m, k), 0, F32, 2).to(E4), whole((n, k), 1, F32, 1).to(E4)
    xs, ws = 2.0 ** (torch.arange(m, device="cuda") % 5).float(), 2.0 ** -(torch.arange(n, device="cuda") % 3).float()
    r = whole((m, n), 3, F32, 200)
    z = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    same(layers.linear(x, w, x_scale=xs, w_scale=ws, out_dtype=F32).y, z, "fp32")
    same(layers.linear(x, w, x_scale=xs, w_scale=ws, residual=r.to(BF)).y, z + r.double(), "residual")
    same(layers.linear(x, w, out_dtype=F32).y, x.double() @ w.double().t(), "unscaled")


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_linear_gradients(layers, tile, m, k, n, dt):
    x, w, dy = whole((m, k), 0, dt, 2), whole((n, k), 1, dt, 1), whole((m, n), 4, dt, 2)
    for gt in (dt, F32):
        g = layers.linear_backward(dy, x, w, bias=True, dw_dtype=gt, db_dtype=F32)
        same(g.dx, dy.double() @ w.double(), "dx")
        same(g.dw, dy.double().t() @ x.double(), "dw")
        same(g.db[None], dy.double().sum(0)[None], "db")
    z = whole((m, n), 5, dt, 3)
    g = layers.linear_backward(dy.float(), x, w, z=z, act="relu", dw_dtype=F32)
    dz = dy.double() * (z > 0)
    same(g.dx, dz @ w.double(), "dx, relu")
    same(g.dw, dz.t() @ x.double(), "dw, relu")


GLU_SIZES = [(1, 130, 40), (65, 70, 24), (257, 130, 137), (700, 200, 300), (11000, 72, 260), (1000, 96, 256)]


@pytest.mark.parametrize("m,k,f", GLU_SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("act", ["relu", "none"])
def test_glu_and_gradients(layers, tile, m, k, f, dt, act):
    x, wg, wu = whole((m, k), 0, dt, 1), whole((f, k), 1, dt, 1), whole((f, k), 2, dt, 1)
    dh = whole((m, f), 3, dt, 2)
    x64, wg64, wu64, d = x.double(), wg.double(), wu.double(), dh.double()
    g, u = x64 @ wg64.t(), x64 @ wu64.t()
    a, s = (g.clamp_min(0), (g > 0).double()) if act == "relu" else (g, torch.ones_like(g))
    same(layers.glu(x, wg, wu, act=act).h, a * u, "h")
    o = layers.glu(x, wg, wu, act=act, need_backward=True, save=True)
    for got, want, name in ((o.h, a * u, "h"), (o.g, g, "g"), (o.u, u, "u")):
        same(got, want, name + " saved")
    dg, du = d * u * s, d * a
    assert max(float(t.abs().max()) for t in (g, u, dg, du)) <= WHOLE[dt]
    dx, dwg, dwu = dg @ wg64 + du @ wu64, dg.t() @ x64, du.t() @ x64
    for saved in ((), (o.g, o.u)):
        for gt in (dt, F32):
            gr = layers.glu_backward(dh, x, wg, wu, *saved, act=act, dw_dtype=gt)
            for got, want, name in ((gr.dx, dx, "dx"), (gr.dw_gate, dwg, "dw_gate"), (gr.dw_up, dwu, "dw_up")):
                same(got, want, f"{name}, {'saved' if saved else 'again'}")
    odd = layers.glu_backward(wide(dh, 5, 3), wide(x, 9, 1), wide(wg, 7, 2), wide(wu, 8, 8), act=act)
    same(odd.dx, dx, "dx, rows of any pitch")
    same(odd.dw_up, dwu, "dw_up, rows of any pitch")


@pytest.mark.parametrize("m,k,f", GLU_SIZES)
@pytest.mark.parametrize("out", [BF, HF])
def test_glu_e4m3(layers, tile, m, k, f, out):
    x, wg, wu = (whole((r, k), i, F32, 1).to(E4) for i, r in enumerate((m, f, f)))
    xs = 2.0 ** -(torch.arange(m, device="cuda") % 3).float()
    gs, us = 2.0 ** (torch.arange(f, device="cuda") % 2).float(), 2.0 ** -(torch.arange(f, device="cuda") % 3).float()
    g = (x.double() @ wg.double().t()) * xs.double()[:, None] * gs.double()
    u = (x.double() @ wu.double().t()) * xs.double()[:, None] * us.double()
    h = layers.glu(x, wg, wu, x_scale=xs, gate_scale=gs, up_scale=us, act="relu", out_dtype=out).h
    same(h, g.clamp_min(0) * u, "h")
    same(layers.glu(x, wg, wu, act="none", out_dtype=out).h, (x.double() @ wg.double().t()) * (x.double() @ wu.double().t()), "unscaled")


def test_tile_numbers(layers):
    from differentiable_rasterizer_gb300 import abi
    for bad in (-2, 4):
        with pytest.raises(abi.GsError):
            abi.gs_layer_tile(bad)
