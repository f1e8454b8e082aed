"""Weights' gradients over many rows, exactly: a bound that grows with the rows passes
whatever is lost, so the inputs here are whole numbers whose sums are exact in fp32 in any
order, and the gradients equal the 64-bit ones to the bit.  The values are such that no
piece of work can be missing unseen: without any one tile of 128 rows, or any one part of a
split, most elements would differ (checked on the oracle)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


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


def whole(shape, seed, dtype, most):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(dtype)


def check_pieces(d, x, rows=128):
    """Every 128 rows' part of d^T x is zero in few elements: a missing one would show."""
    m = d.shape[0]
    for first in (0, m // 2 // rows * rows, (m - 1) // rows * rows):
        part = d[first:first + rows].t() @ x[first:first + rows]
        assert (part != 0).double().mean() > 0.5, first


@pytest.mark.parametrize("m,k,n", [(300_001, 24, 59), (300_001, 128, 59), (100_000, 256, 256), (1_000_003, 64, 14), (20_000, 1000, 330)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_linear(layers, m, k, n, dt):
    x, dy, w = whole((m, k), 0, dt, 2), whole((m, n), 1, dt, 2), whole((n, k), 2, dt, 1)
    z = whole((m, n), 3, dt, 2)
    x64 = x.double()
    for act in ("none", "relu"):
        dz = dy.double() * (z > 0) if act == "relu" else dy.double()
        want, db = dz.t() @ x64, dz.sum(0)
        assert (dz.abs().t() @ x64.abs()).max() < 2 ** 24   # any partial sum is exact
        check_pieces(dz, x64)
        for dyt in (dt, F32):
            g = layers.linear_backward(dy.to(dyt), x, w, z=z, act=act, bias=True, dw_dtype=F32, db_dtype=F32)
            assert torch.equal(g.dw, want.float()) and torch.equal(g.db, db.float()), (act, dyt)
        assert torch.equal(layers.linear_backward(dy, x, w, z=z, act=act, need_dx=False).dw, want.float().to(dt)), act


@pytest.mark.parametrize("m,k,f", [(20_000, 57, 100), (70_001, 64, 128), (70_001, 40, 24), (300_007, 64, 64), (50_003, 96, 72),
                                   (30_001, 64, 200)])
@pytest.mark.parametrize("dt,act", [(BF, "none"), (HF, "relu"), (BF, "relu")])
def test_glu(layers, m, k, f, dt, act):
    """In one pass (up to 64 features and 128 hidden columns) and as products."""
    x, wg, wu, dh = whole((m, k), 0, dt, 1), whole((f, k), 1, dt, 1), whole((f, k), 2, dt, 1), whole((m, f), 3, dt, 2)
    x64 = x.double()
    g, u = x64 @ wg.double().t(), x64 @ wu.double().t()
    a, s = (g.clamp_min(0), (g > 0).double()) if act == "relu" else (g, torch.ones_like(g))
    dg, du = dh.double() * u * s, dh.double() * a
    assert max(float(t.abs().max()) for t in (dg, du)) <= 256   # exact factors
    wants = []
    for d in (dg, du):
        assert (d.abs().t() @ x64.abs()).max() < 2 ** 24
        check_pieces(d, x64)
        wants.append((d.t() @ x64).float())
    gr = layers.glu_backward(dh, x, wg, wu, act=act, dw_dtype=F32)
    assert torch.equal(gr.dw_gate, wants[0]) and torch.equal(gr.dw_up, wants[1])
    assert torch.equal(gr.dx, (dg @ wg.double() + du @ wu.double()).float().to(dt))
    gr = layers.glu_backward(dh, x, wg, wu, act=act, need_dx=False)
    assert torch.equal(gr.dw_gate, wants[0].to(dt)) and torch.equal(gr.dw_up, wants[1].to(dt))


@pytest.mark.parametrize("m,d", [(300_001, 64), (100_000, 256), (70_001, 331), (20_000, 2048)])
def test_norm_weight(layers, m, d):
    """dweight with rstd given as powers of two: dy s rstd is exact."""
    dy, s = whole((m, d), 0, BF, 2), whole((m, d), 1, BF, 2)
    rstd = 2.0 ** (torch.arange(m, device="cuda") % 3).float()
    want = (dy.double() * s.double() * rstd.double()[:, None]).sum(0)
    assert (dy.double().abs() * s.double().abs() * rstd.double()[:, None]).sum(0).max() < 2 ** 24
    _, dw = layers.rms_norm_backward(dy, s, torch.ones(d, device="cuda"), rstd)
    assert torch.equal(dw, want.float())
    for first in (0, m // 2, m - 64):   # no 64 rows are missing
        part = (dy[first:first + 64].double() * s[first:first + 64].double() * rstd[first:first + 64, None].double()).sum(0)
        assert (part != 0).double().mean() > 0.5
