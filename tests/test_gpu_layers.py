"""Decoder layers on the GPU against the formulas in 64 bits, at the sizes, types,
strides and values where they can go wrong.

Bounds, per element, from the formulas and the stated roundings (derived before the
first run; no case has its own):
  u(T)   half a unit in the last place of type T, relative: bf16 2^-8, f16 2^-11, f32 2^-24
         (and T's smallest subnormal, absolute)
  sums   a product of K terms accumulated in fp32 in any order, each step truncating:
         K 2^-23 S with S the sum of the terms' magnitudes
  act    slope at most 1.13; hardware exponential and quotient 2^-20 relative
  dz     rounded to 16 bits before the gradients' products (u |dz|)
Gradients are compared with the formulas' at the forward's stored outputs (z, g, u, s,
rstd), which are themselves compared with the forward's formulas.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 2.0 ** -126, HF: 2.0 ** -24, F32: 2.0 ** -126}
ACTS = ["none", "relu", "silu", "gelu"]


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


@pytest.fixture(autouse=True)
def no_wait_expired():
    """No bounded wait of a layer kernel may run out."""
    yield
    from differentiable_rasterizer_gb300 import abi
    assert not abi.gs_wait_report()


def rnd(shape, seed, dtype, std=1.0, pitch=None, offset=0):
    """Seeded normal values on the GPU; pitch: columns of the wider rows it is a slice of."""
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(shape, generator=g) * std).to(dtype)
    if pitch is None:
        return t.cuda()
    wide = torch.full((shape[0], pitch), float("nan"), dtype=F32).to(dtype).cuda()
    v = wide[:, offset:offset + shape[1]]
    v.copy_(t)
    return v


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def check(got, want, slack, name=""):
    """|got - want| <= u(T) |want| + slack, T got's type; equal shapes; no NaN."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    t = got.dtype
    err = (got.double() - want).abs()
    bound = U[t] * want.abs() + slack * (1 + U[t]) + LEAST[t]
    bad = ~(err <= bound)
    if bad.any():
        i = int((err / bound).nan_to_num(1e30).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{got.double().flatten()[i].item()} want {want.flatten()[i].item()} "
                             f"bound {bound.expand_as(err).flatten()[i].item()}")


SIZES = [  # rows, in, out
    (1, 1, 1), (1, 8, 16), (1, 1024, 4096), (2, 33, 59), (3, 16, 8), (7, 100, 14), (8, 2048, 72), (17, 129, 65),
    (31, 64, 64), (33, 4096, 40), (64, 72, 128), (65, 257, 256), (127, 63, 130), (128, 128, 128), (129, 40, 257),
    (200, 1031, 333), (300, 520, 1032), (1000, 96, 59), (1111, 64, 512), (4099, 48, 24),
]
TYPES = [BF, HF]


def linear_case(m, k, n, dt, seed=0):
    return rnd((m, k), seed, dt), rnd((n, k), seed + 1, dt, k ** -0.5)


def pre64(x, w, b=None, xs=None, ws=None):
    x, w = x.double(), w.double()
    if xs is not None:
        x = x * xs.double()[:, None]
    if ws is not None:
        w = w * ws.double()[:, None]
    z = x @ w.t()
    mag = (x.abs() @ w.abs().t()) * (x.shape[1] + 4) * 2.0 ** -23
    if b is not None:
        z = z + b.double()
        mag = mag + 2.0 ** -23 * b.double().abs()
    return z, mag


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dt", TYPES)
def test_linear_sizes(layers, m, k, n, dt):
    x, w = linear_case(m, k, n, dt)
    z, mag = pre64(x, w)
    o = layers.linear(x, w)
    assert o.z is None and o.y.dtype == dt
    check(o.y, z, mag, "y")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k,n", [(1, 96, 200), (9, 64, 59), (150, 72, 333), (513, 200, 96)])
@pytest.mark.parametrize("dt,out", [(BF, BF), (HF, HF), (BF, F32), (HF, F32), (BF, HF)])
def test_linear_epilogue(layers, m, k, n, dt, out, act):
    """Bias, activation, residual and saved pre-activations, in every output type."""
    x, w = linear_case(m, k, n, dt)
    for bdt in (F32, dt):
        b = rnd((n,), 5, bdt)
        r = rnd((m, n), 6, out)
        z, mag = pre64(x, w, b)
        o = layers.linear(x, w, b, act=act, residual=r, out_dtype=out, need_backward=True)
        a = act64(z, act)
        check(o.y, a + r.double(), 1.13 * mag + 2.0 ** -20 * a.abs() + 2.0 ** -23 * r.double().abs(), "y")
        assert (o.z is None) == (act == "none")
        if o.z is not None:
            check(o.z, z, mag, "z")


@pytest.mark.parametrize("m,k,n", [(1, 64, 48), (5, 77, 59), (130, 200, 70), (260, 96, 264)])
@pytest.mark.parametrize("pitch_k,off", [(256, 0), (264, 8), (259, 3), (257, 0)])
def test_linear_strides(layers, m, k, n, pitch_k, off):
    """Slices of wider rows: aligned and unaligned bases and pitches of every matrix."""
    x = rnd((m, k), 0, BF, pitch=pitch_k, offset=off)
    w = rnd((n, k), 1, BF, k ** -0.5, pitch=pitch_k, offset=off)
    z, mag = pre64(x, w)
    for out, pitch in ((BF, 512), (BF, 517), (F32, 280), (F32, 283)):
        r = rnd((m, n), 2, out, pitch=pitch, offset=off)
        wide = torch.full((m, pitch), 7.0, dtype=out, device="cuda")
        y = wide[:, off:off + n]
        o = layers.linear(x, w, residual=r, out=y)
        assert o.y is y
        check(y, z + r.double(), mag + 2.0 ** -23 * r.double().abs(), f"{out} {pitch}")
        assert (wide[:, :off] == 7).all() and (wide[:, off + n:] == 7).all()   # nothing beside the slice is written
        # in place: the output is the residual
        r2 = r.clone() if r.is_contiguous() else r
        want = z + r2.double()
        slack = mag + 2.0 ** -23 * r2.double().abs()
        layers.linear(x, w, residual=r2, out=r2)
        check(r2, want, slack, "in place")


@pytest.mark.parametrize("m,k,n", [(1, 16, 8), (1, 1024, 512), (3, 100, 59), (40, 1040, 72), (129, 48, 257),
                                   (515, 200, 130), (700, 1031, 96)])
@pytest.mark.parametrize("out", [BF, HF, F32])
def test_linear_e4m3(layers, m, k, n, out):
    x, xs = layers.quantize_rows(rnd((m, k), 0, F32))
    w, ws = layers.quantize_rows(rnd((n, k), 1, F32, k ** -0.5))
    b, r = rnd((n,), 3, F32), rnd((m, n), 4, out)
    z, mag = pre64(x, w, b, xs, ws)
    y = layers.linear(x, w, b, x_scale=xs, w_scale=ws, act="silu", residual=r, out_dtype=out).y
    a = act64(z, "silu")
    check(y, a + r.double(), 1.13 * mag + 2.0 ** -20 * a.abs() + 2.0 ** -22 * r.double().abs(), "scaled")
    z, mag = pre64(x, w)
    check(layers.linear(x, w, out_dtype=F32).y, z, mag, "unscaled")


def linear_grads64(x, w, z, dy, act, ut, b):
    """Formula gradients and their bounds; ut: u of the operands' type; b: dz is dy, unrounded."""
    x, w, dy = x.double(), w.double(), dy.double()
    dz = dy * slope64(z, act)
    least = LEAST[HF] if ut == U[HF] else 0.0
    edz = ut * dz.abs() + 2.0 ** -19 * dy.abs() + least
    if b:   # dz is dy
        edz = edz * 0
    m, n = dz.shape
    dx = dz @ w
    ex = edz @ w.abs() + (n + 4) * 2.0 ** -23 * (dz.abs() @ w.abs())
    dw = dz.t() @ x
    ew = edz.t() @ x.abs() + (m + 4) * 2.0 ** -23 * (dz.abs().t() @ x.abs())
    db = dz.sum(0)
    eb = edz.sum(0) + (m + 4) * 2.0 ** -23 * dz.abs().sum(0)
    return dx, ex, dw, ew, db, eb


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dt", TYPES)
def test_linear_gradients_sizes(layers, m, k, n, dt):
    x, w = linear_case(m, k, n, dt)
    dy = rnd((m, n), 9, dt)
    g = layers.linear_backward(dy, x, w, bias=True)
    dx, ex, dw, ew, db, eb = linear_grads64(x, w, torch.zeros(m, n, device="cuda").double(), dy, "none", 0.0, True)
    check(g.dx, dx, ex, "dx")
    check(g.dw, dw, ew, "dw")
    check(g.db, db, eb, "db")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,k,n", [(1, 40, 24), (37, 59, 131), (700, 72, 264)])
@pytest.mark.parametrize("dt,dyt,gt", [(BF, BF, BF), (HF, HF, F32), (BF, F32, F32), (HF, F32, HF)])
def test_linear_gradients(layers, m, k, n, dt, dyt, gt, act):
    x, w = linear_case(m, k, n, dt)
    b = rnd((n,), 5, F32)
    dy = rnd((m, n), 9, dyt)
    z, _ = pre64(x, w, b)
    o = layers.linear(x, w, b, act=act, need_backward=True)
    g = layers.linear_backward(dy, x, w, z=o.z, act=act, bias=True, dw_dtype=gt, db_dtype=F32)
    z = z if o.z is None else o.z.double()
    dx, ex, dw, ew, db, eb = linear_grads64(x, w, z, dy, act, U[dt], False)
    assert g.dw.dtype == gt and g.db.dtype == F32
    check(g.dx, dx, ex, "dx")
    check(g.dw, dw, ew, "dw")
    check(g.db, db, eb, "db")
    # each alone
    only = layers.linear_backward(dy, x, w, z=o.z, act=act, need_dx=False, dw_dtype=gt)
    assert only.dx is None and only.db is None and torch.equal(only.dw, g.dw)
    only = layers.linear_backward(dy, x, w, z=o.z, act=act, need_dw=False)
    assert only.dw is None and torch.equal(only.dx, g.dx)
    only = layers.linear_backward(dy, x, w, z=o.z, act=act, need_dw=False, need_dx=False, bias=True, db_dtype=F32)
    assert torch.equal(only.db, g.db)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_linear_gradients_against_differences(layers, act):
    """Central differences of the formula's loss sum(dy * y) in 64 bits, step 1e-4: its
    truncation error is below 1e-7 here, far inside the 16-bit bounds."""
    m, k, n = 6, 10, 5
    x, w = linear_case(m, k, n, HF)
    b, dy = rnd((n,), 5, HF), rnd((m, n), 9, HF)
    o = layers.linear(x, w, b, act=act, need_backward=True)
    g = layers.linear_backward(dy, x, w, z=o.z, act=act, bias=True)
    args = [x.double(), w.double(), b.double()]

    def loss(x, w, b):
        return (act64(x @ w.t() + b, act) * dy.double()).sum()

    z, _ = pre64(x, w, b)
    _, ex, _, ew, _, eb = linear_grads64(x, w, z, dy, act, U[HF], False)
    # z is stored in 16 bits: act'' is at most 0.8
    off = 0.8 * (U[HF] * z.abs() + LEAST[HF]) * dy.double().abs()
    ex, ew, eb = ex + off @ w.double().abs(), ew + off.t() @ x.double().abs(), eb + off.sum(0)
    for i, (got, slack) in enumerate(((g.dx, ex), (g.dw, ew), (g.db, eb))):
        want = torch.zeros_like(args[i])
        for j in range(args[i].numel()):
            d = torch.zeros_like(args[i])
            d.view(-1)[j] = 1e-4
            up = [a + d if q == i else a for q, a in enumerate(args)]
            dn = [a - d if q == i else a for q, a in enumerate(args)]
            want.view(-1)[j] = (loss(*up) - loss(*dn)) / 2e-4
        check(got, want, slack + 1e-6, f"argument {i}")


def test_linear_many_rows(layers):
    """A contraction over many rows (the weights' gradient of a small layer) and
    outputs past 2^31 bytes."""
    m, k, n = 300_001, 24, 59
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((m, k), generator=g, device="cuda").to(BF)
    dy = torch.randn((m, n), generator=g, device="cuda").to(BF)
    w = rnd((n, k), 1, BF)
    gr = layers.linear_backward(dy, x, w, bias=True, dw_dtype=F32, db_dtype=F32)
    dx, ex, dw, ew, db, eb = linear_grads64(x, w, torch.zeros((m, n), device="cuda").double(), dy, "none", 0.0, True)
    check(gr.dx, dx, ex, "dx")
    check(gr.dw, dw, ew, "dw")
    check(gr.db, db, eb, "db")


def test_linear_offsets_past_32_bits(layers):
    """Rows whose offsets exceed 2^32 elements in the input and in the output."""
    m, k, n, pitch = 70_000, 16, 24, 65_536   # 4.6e9 elements, 9.2 GB each
    wide = torch.empty((m, pitch), dtype=BF, device="cuda")
    x = wide[:, 8:8 + k]
    x.copy_(rnd((m, k), 0, BF))
    out = wide[:, 4096:4096 + n]
    w = rnd((n, k), 1, BF, 0.25)
    layers.linear(x, w, out=out)
    z, mag = pre64(x, w)
    check(out, z, mag, "aligned")
    x2 = wide[:, 11:11 + k]
    x2.copy_(rnd((m, k), 2, BF))
    out2 = wide[:, 5001:5001 + n]
    layers.linear(x2, w, out=out2)
    z, mag = pre64(x2, w)
    check(out2, z, mag, "unaligned")


@pytest.mark.parametrize("m,k,f", [(1, 8, 8), (1, 1024, 2048), (2, 31, 45), (9, 200, 64), (33, 64, 129), (64, 72, 128),
                                   (130, 96, 72), (257, 331, 200), (1025, 64, 344)])
@pytest.mark.parametrize("dt,act", [(BF, "silu"), (HF, "gelu"), (BF, "relu"), (HF, "none")])
def test_glu_and_gradients(layers, m, k, f, dt, act):
    x = rnd((m, k), 0, dt)
    wg, wu = rnd((f, k), 1, dt, k ** -0.5), rnd((f, k), 2, dt, k ** -0.5)
    g, mg = pre64(x, wg)
    u, mu = pre64(x, wu)
    o = layers.glu(x, wg, wu, act=act, need_backward=True, save=True)
    a = act64(g, act)
    ea = 1.13 * mg + 2.0 ** -20 * a.abs()
    check(o.h, a * u, ea * u.abs() + mu * a.abs() + ea * mu + 2.0 ** -23 * (a * u).abs(), "h")
    check(o.g, g, mg, "g")
    check(o.u, u, mu, "u")
    plain = layers.glu(x, wg, wu, act=act)
    assert plain.g is None and plain.u is None and torch.equal(plain.h, o.h)
    dh = rnd((m, f), 7, dt)
    gr = layers.glu_backward(dh, x, wg, wu, o.g, o.u, act=act)
    g, u = o.g.double(), o.u.double()
    d, s, ut = dh.double(), slope64(g, act), U[dt]
    dg, du = d * u * s, d * act64(g, act)
    least = LEAST[dt]   # dg and du rounded to 16 bits
    eg = ut * dg.abs() + 2.0 ** -18 * (d * u).abs() + least
    eu = ut * du.abs() + 2.0 ** -18 * (d * g).abs() + least
    x64, wg64, wu64 = x.double(), wg.double(), wu.double()
    mag = dg.abs() @ wg64.abs() + du.abs() @ wu64.abs()
    check(gr.dx, dg @ wg64 + du @ wu64, eg @ wg64.abs() + eu @ wu64.abs() + (2 * f + 4) * 2.0 ** -23 * mag, "dx")
    for got, dd, ee, name in ((gr.dw_gate, dg, eg, "dw_gate"), (gr.dw_up, du, eu, "dw_up")):
        check(got, dd.t() @ x64, ee.t() @ x64.abs() + (m + 4) * 2.0 ** -23 * (dd.abs().t() @ x64.abs()), name)
    f32 = layers.glu_backward(dh, x, wg, wu, o.g, o.u, act=act, need_dx=False, dw_dtype=F32)
    assert f32.dx is None and torch.equal(f32.dw_gate.to(dt), gr.dw_gate) and torch.equal(f32.dw_up.to(dt), gr.dw_up)
    only = layers.glu_backward(dh, x, wg, wu, o.g, o.u, act=act, need_dw=False)
    assert only.dw_up is None and torch.equal(only.dx, gr.dx)


@pytest.mark.parametrize("m,k,f", [(1, 8, 8), (2, 31, 45), (33, 64, 129), (64, 72, 128), (130, 96, 72), (257, 331, 200),
                                   (1025, 64, 344), (5000, 40, 24), (700, 600, 520)])
@pytest.mark.parametrize("dt,act", [(BF, "silu"), (HF, "gelu"), (BF, "relu"), (HF, "none"), (BF, "gelu")])
def test_glu_gradients_again(layers, m, k, f, dt, act):
    """The gradients that compute the projections again, against the formula's at the exact ones."""
    x = rnd((m, k), 0, dt)
    wg, wu = rnd((f, k), 1, dt, k ** -0.5), rnd((f, k), 2, dt, k ** -0.5)
    g, mg = pre64(x, wg)
    u, mu = pre64(x, wu)
    dh = rnd((m, f), 7, dt)
    gr = layers.glu_backward(dh, x, wg, wu, act=act)
    d, s, a, ut = dh.double(), slope64(g, act), act64(g, act), U[dt]
    dg, du = d * u * s, d * a
    # act' is at most 1.13 and its slope at most 0.8 (relu's jumps at 0: where |g| is within its sum's error)
    jump = (g.abs() <= mg).double() if act == "relu" else 0.0
    eg = ut * dg.abs() + 2.0 ** -18 * (d * u).abs() + LEAST[dt] + d.abs() * (1.13 * mu + (0.8 * mg + jump) * (u.abs() + mu))
    eu = ut * du.abs() + 2.0 ** -18 * (d * g).abs() + LEAST[dt] + 1.13 * d.abs() * mg
    x64, wg64, wu64 = x.double(), wg.double(), wu.double()
    mag = dg.abs() @ wg64.abs() + du.abs() @ wu64.abs()
    check(gr.dx, dg @ wg64 + du @ wu64, eg @ wg64.abs() + eu @ wu64.abs() + (2 * f + 4) * 2.0 ** -23 * mag, "dx")
    for got, dd, ee, name in ((gr.dw_gate, dg, eg, "dw_gate"), (gr.dw_up, du, eu, "dw_up")):
        check(got, dd.t() @ x64, ee.t() @ x64.abs() + (m + 4) * 2.0 ** -23 * (dd.abs().t() @ x64.abs()), name)


@pytest.mark.parametrize("m,k,f", [(1, 64, 128), (127, 64, 128), (128, 16, 64), (129, 33, 65), (257, 64, 64), (5000, 1, 1),
                                   (20000, 57, 100), (70001, 64, 128), (70001, 40, 24)])
@pytest.mark.parametrize("dt,act", [(BF, "silu"), (HF, "gelu"), (BF, "relu"), (HF, "none")])
def test_glu_gradients_narrow(layers, m, k, f, dt, act):
    """The one-pass gradients of a narrow layer: tiles of 128 rows, several a multiprocessor, halves of 64 hidden columns."""
    x = rnd((m, k), 0, dt)
    wg, wu = rnd((f, k), 1, dt, k ** -0.5), rnd((f, k), 2, dt, k ** -0.5)
    g, mg = pre64(x, wg)
    u, mu = pre64(x, wu)
    dh = rnd((m, f), 7, dt)
    gr = layers.glu_backward(dh, x, wg, wu, act=act)
    d, s, a, ut = dh.double(), slope64(g, act), act64(g, act), U[dt]
    dg, du = d * u * s, d * a
    jump = (g.abs() <= mg).double() if act == "relu" else 0.0
    eg = ut * dg.abs() + 2.0 ** -18 * (d * u).abs() + LEAST[dt] + d.abs() * (1.13 * mu + (0.8 * mg + jump) * (u.abs() + mu))
    eu = ut * du.abs() + 2.0 ** -18 * (d * g).abs() + LEAST[dt] + 1.13 * d.abs() * mg
    x64, wg64, wu64 = x.double(), wg.double(), wu.double()
    mag = dg.abs() @ wg64.abs() + du.abs() @ wu64.abs()
    check(gr.dx, dg @ wg64 + du @ wu64, eg @ wg64.abs() + eu @ wu64.abs() + (2 * f + 4) * 2.0 ** -23 * mag, "dx")
    for got, dd, ee, name in ((gr.dw_gate, dg, eg, "dw_gate"), (gr.dw_up, du, eu, "dw_up")):
        check(got, dd.t() @ x64, ee.t() @ x64.abs() + (m + 4) * 2.0 ** -23 * (dd.abs().t() @ x64.abs()), name)
    twice = layers.glu_backward(dh, x, wg, wu, act=act)
    assert all(torch.equal(p, q) for p, q in ((gr.dx, twice.dx), (gr.dw_gate, twice.dw_gate), (gr.dw_up, twice.dw_up)))
    f32 = layers.glu_backward(dh, x, wg, wu, act=act, need_dx=False, dw_dtype=F32)
    assert f32.dx is None and torch.equal(f32.dw_gate.to(dt), gr.dw_gate) and torch.equal(f32.dw_up.to(dt), gr.dw_up)
    only = layers.glu_backward(dh, x, wg, wu, act=act, need_dw=False)
    assert only.dw_up is None and torch.equal(only.dx, gr.dx)
    # rows of other pitches and bases, the same values
    def wide(t, off):
        w = torch.full((t.shape[0], t.shape[1] + 11), float("nan"), dtype=dt, device="cuda")[:, off:off + t.shape[1]]
        w.copy_(t)
        return w
    odd = layers.glu_backward(wide(dh, 3), wide(x, 5), wide(wg, 1), wide(wu, 8), act=act)
    assert torch.equal(odd.dx, gr.dx) and torch.equal(odd.dw_gate, gr.dw_gate) and torch.equal(odd.dw_up, gr.dw_up)


def test_glu_gradients_narrow_bad_rows(layers):
    """A row with an infinity or a NaN spoils its own dx and no other row's."""
    m, k, f = 400, 40, 100
    x, wg, wu, dh = rnd((m, k), 0, BF), rnd((f, k), 1, BF), rnd((f, k), 2, BF), rnd((m, f), 3, BF)
    want = layers.glu_backward(dh, x, wg, wu).dx
    x[130, 7], dh[250, 99] = float("inf"), float("nan")
    got = layers.glu_backward(dh, x, wg, wu).dx
    same = torch.ones(m, dtype=torch.bool, device="cuda")
    same[[130, 250]] = False
    assert torch.equal(got[same], want[same]) and not got[130].isfinite().any() and got[250].isnan().all()


def test_glu_saves_for_wide_inputs_only(layers):
    for k, saved in ((512, False), (520, True)):
        o = layers.glu(rnd((3, k), 0, BF), rnd((16, k), 1, BF), rnd((16, k), 2, BF), need_backward=True)
        assert (o.g is not None) == (o.u is not None) == saved


@pytest.mark.parametrize("m,k,f", [(1, 512, 256), (5, 100, 59), (200, 1040, 136), (600, 96, 300)])
@pytest.mark.parametrize("out", [BF, HF])
def test_glu_e4m3(layers, m, k, f, out):
    x, xs = layers.quantize_rows(rnd((m, k), 0, F32))
    wg, gs = layers.quantize_rows(rnd((f, k), 1, F32, k ** -0.5))
    wu, us = layers.quantize_rows(rnd((f, k), 2, F32, k ** -0.5))
    g, mg = pre64(x, wg, None, xs, gs)
    u, mu = pre64(x, wu, None, xs, us)
    h = layers.glu(x, wg, wu, x_scale=xs, gate_scale=gs, up_scale=us, out_dtype=out).h
    a = act64(g, "silu")
    ea = 1.13 * mg + 2.0 ** -20 * a.abs()
    check(h, a * u, ea * u.abs() + mu * a.abs() + ea * mu + 2.0 ** -23 * (a * u).abs(), "h")


@pytest.mark.parametrize("pitch,off", [(280, 8), (277, 3)])
def test_glu_strides(layers, pitch, off):
    m, k, f = 140, 72, 200
    mats = [rnd((r, c), i, BF, c ** -0.5 if i else 1.0, pitch=pitch, offset=off)
            for i, (r, c) in enumerate(((m, k), (f, k), (f, k)))]
    dense = [t.contiguous() for t in mats]
    a = layers.glu(*mats, need_backward=True, save=True)
    b = layers.glu(*dense, need_backward=True, save=True)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    dh = rnd((m, f), 7, BF)
    wide = [rnd((m, f), 7, BF, pitch=pitch, offset=off)]
    for t in (a.g, a.u):
        v = torch.zeros((m, pitch), dtype=BF, device="cuda")[:, off:off + f]
        v.copy_(t)
        wide.append(v)
    p = layers.glu_backward(wide[0], *mats, wide[1], wide[2])
    q = layers.glu_backward(dh, *dense, b.g, b.u)
    for s, t in zip(p, q):
        assert torch.equal(s, t)
    for s, t in zip(layers.glu_backward(wide[0], *mats), layers.glu_backward(dh, *dense)):
        assert torch.equal(s, t)


# ------------------------------------------------------------------------------ norm
NORM_SIZES = [(1, 1), (1, 1024), (3, 7), (5, 8), (2, 16384), (4, 16383), (9, 33), (100, 256), (1, 8192), (33, 331),
              (1000, 64), (257, 2048), (17, 5000), (4097, 24), (65, 1000)]


def norm64(x, r, w, eps):
    s = x.double() + (r.double() if r is not None else 0)
    rstd = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return s, rstd, s * rstd * w.double()


@pytest.mark.parametrize("m,d", NORM_SIZES)
@pytest.mark.parametrize("dt,wt,ot", [(BF, BF, BF), (HF, F32, HF), (F32, F32, F32), (F32, BF, BF), (BF, F32, F32)])
def test_norm_and_gradients(layers, m, d, dt, wt, ot):
    x, r, w = rnd((m, d), 0, dt), rnd((m, d), 1, dt, 3.0), rnd((d,), 2, wt)
    for res in (r, None):
        o = layers.rms_norm(x, w, residual=res, eps=1e-5, out_dtype=ot, need_backward=True)
        s, rstd, y = norm64(x, res, w, 1e-5)
        e = (d + 16) * 2.0 ** -24   # sum of squares, its root, three products
        check(o.y, y, e * y.abs() + 2.0 ** -24 * 4 * (rstd * w.double().abs() * (x.double().abs() + 3 * r.double().abs())), "y")
        check(o.rstd, rstd[:, 0], e * rstd[:, 0] * 3, "rstd")
        if res is None:
            assert o.s is x
        else:
            check(o.s, s, 0.0, "s")
        dy, ds = rnd((m, d), 3, ot), rnd((m, d), 4, dt)
        # the gradients are those at the stored (rounded) sum and the forward's rstd
        s16, rs, w64, dy64 = o.s.double(), o.rstd.double()[:, None], w.double(), dy.double()
        p = dy64 * w64
        c = (p * s16).mean(-1, keepdim=True) * rs * rs
        mag = rs * (p.abs() + s16.abs() * (p * s16).abs().mean(-1, keepdim=True) * rs * rs)
        for extra in (ds, None):
            dx, dw = layers.rms_norm_backward(dy, o.s, w, o.rstd, ds=extra)
            want = rs * (p - s16 * c) + (extra.double() if extra is not None else 0)
            check(dx, want, (d + 16) * 2.0 ** -24 * mag + 2.0 ** -22 * want.abs(), "dx")
            terms = dy64 * s16 * rs
            check(dw, terms.sum(0), (m + 16) * 2.0 ** -24 * terms.abs().sum(0), "dw")


def test_norm_gradient_against_differences(layers):
    m, d = 3, 6
    x, r, w, dy, ds = (rnd((m, d) if i != 2 else (d,), i, F32) for i in range(5))
    o = layers.rms_norm(x, w, residual=r, need_backward=True)
    dx, dw = layers.rms_norm_backward(dy, o.s, w, o.rstd, ds=ds)

    def loss(x, w):
        s, _, y = norm64(x, r, w, 1e-6)
        return (y * dy.double()).sum() + (s * ds.double()).sum()

    for got, i in ((dx, 0), (dw, 1)):
        base = [x.double(), w.double()]
        for j in range(base[i].numel()):
            d1 = torch.zeros_like(base[i])
            d1.view(-1)[j] = 1e-4
            up = [b + d1 if q == i else b for q, b in enumerate(base)]
            dn = [b - d1 if q == i else b for q, b in enumerate(base)]
            want = (loss(*up) - loss(*dn)) / 2e-4
            assert abs(got.reshape(-1)[j].item() - want.item()) <= 1e-5 * (1 + abs(want.item()))


def e4m3_rows(t):
    """The 8-bit rows of fp32 values, from the definition, in fp32."""
    a = t.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -100)
    top = torch.full_like(a, 448.0)   # tensor / tensor: one rounding each
    return (t * (top / a)).to(E4), (a / top)[:, 0]


@pytest.mark.parametrize("m,d", NORM_SIZES)
@pytest.mark.parametrize("dt,wt", [(BF, BF), (F32, F32), (HF, F32)])
def test_norm_e4m3_bits(layers, m, d, dt, wt):
    """The 8-bit values follow the definition bit for bit, the scales to the norm's error."""
    x, r, w = rnd((m, d), 0, dt), rnd((m, d), 1, dt, 3.0), rnd((d,), 2, wt)
    o = layers.rms_norm(x, w, residual=r, out_dtype=E4)
    q, a = e4m3_rows((x.float() + r.float()) * w.float())
    assert torch.equal(o.y.float(), q.float())
    _, rstd, _ = norm64(x, r, w, 1e-6)
    check(o.scale, a.double() * rstd[:, 0], (d + 16) * 2.0 ** -24 * 3 * a.double() * rstd[:, 0], "scale")
    q1, s1 = layers.quantize_rows(x)
    q2, s2 = e4m3_rows(x.float())
    assert torch.equal(q1.float(), q2.float()) and torch.equal(s1, s2)


def test_norm_special_rows(layers):
    """Rows of zeros, tiny and huge values, infinities and NaN stay in their rows."""
    d = 40
    x = rnd((7, d), 0, F32)
    x[1] = 0
    x[2] *= 1e-38
    x[3, 5] = float("nan")
    x[4, 5] = float("inf")
    x[5] *= 1e18
    w = rnd((d,), 1, F32).abs() + 0.5
    o = layers.rms_norm(x, w, eps=1e-6, need_backward=True)
    ref = layers.rms_norm(x[[0, 6]].contiguous(), w, eps=1e-6)
    assert torch.equal(o.y[[0, 6]], ref.y)
    assert (o.y[1] == 0).all() and torch.isfinite(o.y[2]).all() and torch.isnan(o.y[3]).all()
    _, _, y5 = norm64(x[5:6], None, w, 1e-6)
    check(o.y[5:6], y5, 1e-4 * y5.abs(), "large")
    q = layers.rms_norm(x, w, eps=1e-6, out_dtype=E4)
    qr = layers.rms_norm(x[[0, 6]].contiguous(), w, eps=1e-6, out_dtype=E4)
    assert torch.equal(q.y[[0, 6]].float(), qr.y.float()) and torch.equal(q.scale[[0, 6]], qr.scale)
    assert (q.y[1].float() == 0).all() and torch.isfinite(q.scale[1])
    assert torch.isnan(q.y[3].float()).all() and torch.isnan(q.scale[3])
    k, s = layers.quantize_rows(x)
    assert torch.isnan(k[3].float()).all() and (k[1].float() == 0).all() and torch.isfinite(s[[0, 1, 2, 5, 6]]).all()


@pytest.mark.parametrize("pitch,off", [(352, 16), (345, 3), (339, 0)])
def test_norm_strides_and_aliases(layers, pitch, off):
    m, d = 70, 320
    x, r = (rnd((m, d), i, BF, pitch=pitch, offset=off) for i in range(2))
    w = rnd((d,), 2, BF)
    a = layers.rms_norm(x, w, residual=r, need_backward=True)
    b = layers.rms_norm(x.contiguous(), w, residual=r.contiguous(), need_backward=True)
    assert torch.equal(a.s, b.s)
    _, _, y = norm64(x, r, w, 1e-6)
    for o in (a, b):
        check(o.y, y, (d + 16) * 2.0 ** -24 * 4 * y.abs() + 2.0 ** -20, "y")
    # the sum written over the residual, through the C ABI
    from differentiable_rasterizer_gb300 import abi
    r2, y2 = r.contiguous().clone(), torch.empty((m, d), dtype=BF, device="cuda")
    xc = x.contiguous()
    abi.gs_rms_norm(m, d, xc.data_ptr(), d, r2.data_ptr(), d, w.data_ptr(), y2.data_ptr(), d, 0, r2.data_ptr(), d, 0,
                    1e-6, abi.GS_BF16, abi.GS_BF16, abi.GS_BF16, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(r2, b.s) and torch.equal(y2, b.y)


# ------------------------------------------------------------------------------ shared
def test_no_rows(layers):
    """Zero rows: empty outputs, zero gradients of the weights."""
    k, n = 24, 40
    x, w = torch.empty((0, k), dtype=BF, device="cuda"), rnd((n, k), 1, BF)
    assert layers.linear(x, w, act="silu", need_backward=True).y.shape == (0, n)
    g = layers.linear_backward(torch.empty((0, n), dtype=BF, device="cuda"), x, w, bias=True)
    assert g.dx.shape == (0, k) and (g.dw == 0).all() and (g.db == 0).all()
    o = layers.glu(x, w, w, need_backward=True)
    assert o.h.shape == (0, n)
    g = layers.glu_backward(o.h, x, w, w, o.g, o.u)
    assert g.dx.shape == (0, k) and (g.dw_gate == 0).all() and (g.dw_up == 0).all()
    wt = rnd((k,), 2, BF)
    o = layers.rms_norm(x, wt, residual=x, need_backward=True)
    dx, dw = layers.rms_norm_backward(x, o.s, wt, o.rstd)
    assert o.y.shape == (0, k) and dx.shape == (0, k) and (dw == 0).all()
    assert layers.quantize_rows(x)[0].shape == (0, k)


def test_leading_dimensions(layers):
    x, w = rnd((4, 5 * 16), 0, BF).view(4, 5, 16), rnd((24, 16), 1, BF)
    y = layers.linear(x, w).y
    assert y.shape == (4, 5, 24) and torch.equal(y.view(20, 24), layers.linear(x.view(20, 16), w).y)
    q, s = layers.quantize_rows(x)
    assert q.shape == (4, 5, 16) and s.shape == (4, 5)
    assert torch.equal(layers.linear(x[0, 0], w).y, layers.linear(x[0, :1], w).y[0])   # one dimension: one row


def test_nonfinite_values_stay_in_their_rows(layers):
    """A NaN or an infinity in one row of x reaches that row of y only; in one row of w, one column."""
    m, k, n = 200, 96, 136
    x, w = linear_case(m, k, n, BF)
    good = layers.linear(x, w, act="gelu").y
    xb = x.clone()
    xb[7, 3], xb[150, 60] = float("nan"), float("inf")
    y = layers.linear(xb, w, act="gelu").y
    keep = torch.ones(m, dtype=torch.bool)
    keep[[7, 150]] = False
    assert torch.equal(y[keep], good[keep]) and torch.isnan(y[7]).all()
    wb = w.clone()
    wb[133, 0] = float("nan")
    y = layers.linear(x, wb, act="gelu").y
    assert torch.equal(y[:, :133], good[:, :133]) and torch.isnan(y[:, 133]).all()
    assert torch.equal(y[:, 134:], good[:, 134:])


def test_runs_are_bit_identical(layers):
    m, k, n = 3001, 200, 136
    x, w = linear_case(m, k, n, BF)
    dy, b = rnd((m, n), 3, BF), rnd((n,), 4, BF)
    runs = []
    for _ in range(3):
        o = layers.linear(x, w, b, act="silu", need_backward=True)
        g = layers.linear_backward(dy, x, w, z=o.z, act="silu", bias=True)
        u = layers.glu(x, w, w, need_backward=True)
        h = layers.glu_backward(dy, x, w, w, u.g, u.u)
        nrm = layers.rms_norm(x, rnd((k,), 7, BF), need_backward=True)
        d = layers.rms_norm_backward(x, nrm.s, rnd((k,), 7, BF), nrm.rstd)
        s = layers.glu(x, w, w, need_backward=True, save=True)
        runs.append([*o, *g, u.h, *s, *h, *layers.glu_backward(dy, x, w, w, s.g, s.u), nrm.y, *d])
    for other in runs[1:]:
        for a, b_ in zip(runs[0], other):
            assert torch.equal(a, b_)


def test_other_stream(layers):
    """Calls queue on the current stream: inputs written there before are seen, in order."""
    s = torch.cuda.Stream()
    m, k, n = 2000, 256, 128
    x, w = linear_case(m, k, n, BF)
    want = layers.linear(x, w).y
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.empty((8192, 8192), device="cuda")
        for _ in range(4):
            big.normal_()
        x2 = torch.empty_like(x)
        x2.copy_(x)
        y = layers.linear(x2, w).y
        x2.zero_()
    s.synchronize()
    assert torch.equal(y, want)


def test_graph_capture(layers):
    """The calls can be captured: they allocate through torch and never synchronise."""
    m, k, n = 64, 128, 96
    x, w = linear_case(m, k, n, BF)
    dy = rnd((m, n), 5, BF)
    o = layers.linear(x, w, act="silu", need_backward=True)
    ref = layers.linear_backward(dy, x, w, z=o.z, act="silu", bias=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oc = layers.linear(x, w, act="silu", need_backward=True)
        gc = layers.linear_backward(dy, x, w, z=oc.z, act="silu", bias=True)
    for t in (oc.y, gc.dx, gc.dw, gc.db):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oc.y, o.y)
    for a, b in zip(gc, ref):
        assert torch.equal(a, b)


def test_refusals(layers):
    """What the torch layer cannot take, named; the device stays usable."""
    from differentiable_rasterizer_gb300 import abi
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")   # noqa: E731
    x, w, b = z(6, 16), z(8, 16), z(8)
    lin, back = layers.linear, layers.linear_backward
    cases = [
        ("expected BFloat16", lambda: lin(x, w.half())), ("expected", lambda: lin(x.float(), w)),
        ("expected", lambda: lin(x.to(torch.int32), w)), ("columns", lambda: lin(x, z(8, 15))),
        ("on cpu", lambda: lin(x, w.cpu())), ("not contiguous", lambda: lin(z(16, 6).t(), w)),
        ("overlap", lambda: lin(z(16).expand(6, 16), w)), ("do not merge", lambda: lin(z(2, 3, 16).transpose(0, 1), w)),
        ("one dimension", lambda: lin(z(), w)), ("contiguous values", lambda: lin(x, w, z(16)[::2])),
        ("contiguous values", lambda: lin(x, w, z(9))), ("rows, expected", lambda: lin(x, w, residual=z(5, 8))),
        ("expected", lambda: lin(x, w, residual=z(6, 8), out_dtype=F32)), ("out_dtype", lambda: lin(x, w, out_dtype=E4)),
        ("torch.dtype", lambda: lin(x, w, out_dtype="bfloat16")), ("rows, expected", lambda: lin(x, w, out=z(7, 8))),
        ("8-bit", lambda: lin(x.to(E4), w.to(E4), act="silu", need_backward=True)),
        ("x_scale", lambda: lin(x.to(E4), w.to(E4), x_scale=z(5, dt=F32))), ("x_scale", lambda: lin(x, w, x_scale=z(6))),
        ("z: required", lambda: back(z(6, 8), x, w, act="silu")), ("dw_dtype", lambda: back(z(6, 8), x, w, dw_dtype=HF)),
        ("db_dtype", lambda: back(z(6, 8), x, w, db_dtype=E4)), ("columns", lambda: back(z(6, 9), x, w)),
        ("rows, expected", lambda: layers.glu(x, w, z(9, 16))), ("out_dtype", lambda: layers.glu(x, w, w, out_dtype=HF)),
        ("8-bit", lambda: layers.glu(x.to(E4), w.to(E4), w.to(E4), need_backward=True)),
        ("u: expected a tensor", lambda: layers.glu_backward(z(6, 8), x, w, w, z(6, 8))),
        ("weight: required", lambda: layers.rms_norm(x, None)), ("contiguous values", lambda: layers.rms_norm(x, z(15))),
        ("residual", lambda: layers.rms_norm(x, z(16), residual=x.float())),
        ("rstd", lambda: layers.rms_norm_backward(x, x, z(16), None)),
        ("expected", lambda: layers.quantize_rows(x.to(E4))),
    ]
    for what, call in cases:
        with pytest.raises(ValueError, match=what):
            call()
    with pytest.raises(abi.GsError) as e:   # the library's own refusals: scales without 8-bit operands, too wide rows
        lin(x, w, x_scale=z(6, dt=F32))
    assert e.value.status == abi.GS_ERR_INVALID_ARG
    with pytest.raises(abi.GsError):
        layers.rms_norm(z(1, 16385), z(16385))
    with pytest.raises(abi.GsError):
        layers.rms_norm(x, z(16), eps=-1.0)
    assert (lin(x, w, b).y == 0).all()
