"""The norm after a block with its gate, the residual scale and the norm before the next block on
the GPU against the formulas in 64 bits.

Bounds, per element, from the formulas and the stated roundings (derived before the first run;
no case has its own).  u(T): half a step of type T relative to the value.
  mean    a sum of cols terms in fp32, any order: cols 2^-24 relative, half of it in the root
  s       es = (cols 2^-24 + 2^-21) |gate a| + 2^-22 |scale x|, and u |s|
  y       |weight| rstd (es + |s| (cols 2^-24 + 2^-20 + ||es|| / ||s||)), and u |y|
  grads   at the forward's stored s and factors: each sum over a row is off by cols 2^-23 of its
          terms' magnitudes, over rows by rows 2^-23 of theirs, each step by 2^-20
8-bit y: y_scale's bound is the norm's; y within half a step (2^-4, or 2^-10 absolute: e4m3's
subnormals) of the exact value times the scale's error.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
U = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
LEAST = {BF: 2.0 ** -126, HF: 2.0 ** -24, F32: 2.0 ** -126}
EPS = 1e-6


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


def rnd(shape, seed, dtype, std=1.0, pitch=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn(shape, generator=g) * std).to(dtype).cuda()
    if not pitch:
        return t
    v = torch.full((shape[0], pitch), float("nan"), dtype=dtype, device="cuda")[:, offset:offset + shape[1]]
    v.copy_(t)
    return v


def close(got, want, slack, name):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    t = got.dtype
    err = (got.double() - want).abs()
    bound = U[t] * want.abs() + slack * (1 + U[t]) + LEAST[t]
    bad = ~(err <= bound)
    if bad.any():
        i = int((err / bound).nan_to_num(1e30).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got {got.double().flatten()[i].item()} want "
                             f"{want.flatten()[i].item()} bound {bound.expand_as(err).flatten()[i].item()}")


def inputs(rows, cols, dt, gate, post, seed=0, pitch=0, offset=0, wt=None):
    wt = wt or dt
    h, x = (rnd((rows, cols), seed + i, dt, 1 + i, pitch, offset) for i in (0, 1))
    w, p = 1 + rnd((cols,), seed + 2, wt, 0.2), (1 + rnd((cols,), seed + 3, wt, 0.2) if post else None)
    g = None if gate == "none" else rnd((cols,), seed + 4, wt, 0.5) if gate == "vector" else rnd((rows, cols), seed + 5, dt, 0.5, pitch, offset)
    return h, x, w, p, g


def forward64(h, x, w, p, g, scale):
    cols = h.shape[1]
    h, x, w = h.double(), x.double(), w.double()
    gate = g.double() if g is not None else torch.ones((), dtype=torch.float64, device="cuda")
    rp = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) if p is not None else None
    a = h * rp * p.double() if p is not None else h
    s = scale * x + gate * a
    es = (cols * 2.0 ** -24 + 2.0 ** -21) * (gate * a).abs() + 2.0 ** -22 * (scale * x).abs()
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)
    rel = cols * 2.0 ** -24 + 2.0 ** -20 + es.norm(dim=1, keepdim=True) / s.norm(dim=1, keepdim=True).clamp_min(1e-300)
    return rp, s, es, r, s * r * w, w.abs() * r * (es + s.abs() * rel), rel


def check_backward(layers, h, x, w, p, g, scale, b, dy, ds):
    rows, cols = h.shape
    out = layers.block_norm_backward(dy, h, b.s if dy is not None else None, w if dy is not None else None, b.rstd if dy is not None else None,
                                     post_weight=p, rstd_post=b.rstd_post, gate=g, scale=scale, ds=ds)
    H, one = h.double(), torch.ones((), dtype=torch.float64, device="cuda")
    gate = one if g is None else g.double()
    P = one if p is None else p.double()
    rp = one if p is None else b.rstd_post.double()[:, None]
    a = H * rp * P
    k, up = cols * 2.0 ** -23 + 2.0 ** -20, rows * 2.0 ** -23 + 2.0 ** -20
    G, A = (torch.zeros_like(H),) * 2
    if dy is not None:
        S, r, t = b.s.double(), b.rstd.double()[:, None], dy.double() * w.double()
        G = r * (t - S * r * r * (t * S).mean(1, keepdim=True))
        A = r * (t.abs() + S.abs() * r * r * (t * S).abs().mean(1, keepdim=True))
        terms = dy.double() * S * r
        close(out.dweight, terms.sum(0), up * terms.abs().sum(0), "dweight")
    if ds is not None:
        G, A = G + ds.double(), A + ds.double().abs()
    close(out.dx, scale * G, k * abs(scale) * A, "dx")
    if g is not None:
        t, m = G * a, A * a.abs()
        if g.dim() == 2:
            close(out.dgate, t, k * m, "dgate")
        else:
            close(out.dgate, t.sum(0), (up + k) * m.sum(0), "dgate")
    else:
        assert out.dgate is None
    D, M = G * gate, A * gate.abs()
    if p is None:
        assert out.dpost_weight is None
        close(out.dh, D, k * M, "dh")
        return out
    close(out.dpost_weight, (D * H * rp).sum(0), (up + k) * (M * (H * rp).abs()).sum(0), "dpost_weight")
    t, m = D * P, M * P.abs()
    close(out.dh, rp * (t - H * rp * rp * (t * H).mean(1, keepdim=True)), 2 * k * rp * (m + H.abs() * rp * rp * (m * H.abs()).mean(1, keepdim=True)), "dh")
    return out


def run(layers, rows, cols, dt, gate, post, scale=0.75, need_ds=True, dy_type=None, **how):
    h, x, w, p, g = inputs(rows, cols, dt, gate, post, **how)
    b = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=scale, eps=EPS, need_backward=True)
    rp, s, es, r, y, ey, rel = forward64(h, x, w, p, g, scale)
    close(b.s, s, es, "s")
    close(b.y, y, ey, "y")
    close(b.rstd, r[:, 0], rel[:, 0] * r[:, 0], "rstd")
    if post:
        close(b.rstd_post, rp[:, 0], (cols * 2.0 ** -24 + 2.0 ** -21) * rp[:, 0], "rstd_post")
    else:
        assert b.rstd_post is None
    dy = rnd((rows, cols), 50, dy_type or dt)
    ds = rnd((rows, cols), 51, dt) if need_ds else None
    return b, check_backward(layers, h, x, w, p, g, scale, b, dy, ds)


SIZES = [(1, 1), (1, 8), (2, 7), (3, 16), (33, 59), (1, 1024), (1000, 64), (777, 128), (300, 256), (65, 331), (129, 520), (17, 1000),
         (40, 1024), (9, 2049), (7, 4096), (5, 5003), (3, 8192), (2, 12345), (2, 16384), (5000, 40), (1, 16383)]


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(layers, rows, cols, dt):
    run(layers, rows, cols, dt, "vector", True, seed=rows)


@pytest.mark.parametrize("need_ds", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "vector", "rows"])
@pytest.mark.parametrize("rows,cols", [(70, 72), (33, 65), (3, 3000)])
def test_what_may_be_absent(layers, rows, cols, gate, post, need_ds):
    run(layers, rows, cols, BF, gate, post, need_ds=need_ds)


@pytest.mark.parametrize("wt", [BF, HF, F32])
@pytest.mark.parametrize("dy_type", [BF, HF, F32])
def test_types_mixed(layers, wt, dy_type):
    run(layers, 50, 200, BF, "vector", True, wt=wt, dy_type=dy_type)
    run(layers, 50, 77, HF, "rows", True, wt=wt, dy_type=dy_type)


@pytest.mark.parametrize("pitch,offset", [(80, 0), (96, 8), (79, 3), (73, 0)])
@pytest.mark.parametrize("gate", ["vector", "rows"])
def test_strided_rows(layers, pitch, offset, gate):
    run(layers, 100, 72, HF, gate, True, pitch=pitch, offset=offset)


def test_without_the_next_norm(layers):
    """The last block's: no weight, no y; the gradient starts from s alone."""
    h, x, _, p, g = inputs(90, 100, BF, "vector", True)
    b = layers.block_norm(h, x, post_weight=p, gate=g, scale=2.0, eps=EPS, need_backward=True)
    assert b.y is None and b.rstd is None
    _, s, es, *_ = forward64(h, x, torch.ones(100, device="cuda"), p, g, 2.0)
    close(b.s, s, es, "s")
    check_backward(layers, h, x, None, p, g, 2.0, b, None, rnd((90, 100), 51, BF))


@pytest.mark.parametrize("rows,cols,gate", [(1, 1024, "vector"), (200, 256, "rows"), (33, 331, "none"), (4, 9000, "vector")])
def test_8_bits(layers, rows, cols, gate):
    h, x, w, p, g = inputs(rows, cols, BF, gate, True)
    b = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=0.75, eps=EPS, out_dtype=E4)
    _, s, es, r, y, ey, rel = forward64(h, x, w, p, g, 0.75)
    close(b.s, s, es, "s")
    t = (s * w.double()).abs()
    top = t.max(1, keepdim=True).values
    etop = (es * w.double().abs()).max(1, keepdim=True).values + 2.0 ** -22 * top
    close(b.y_scale, (top * r / 448)[:, 0], ((etop + top * rel) * r / 448)[:, 0], "y_scale")
    q, want = b.y.double(), s * w.double() * 448 / top
    slack = (es * w.double().abs() + 2.0 ** -22 * t) * 448 / top + want.abs() * etop / top
    assert ((q - want).abs() <= 2.0 ** -4 * (want.abs() + slack) + 2.0 ** -10 + slack).all()


def test_one_dimension_and_more(layers):
    """Rows of several leading dimensions, and a single row without one (its gate a vector)."""
    h, x, w, p, g = inputs(24, 64, BF, "rows", True)
    a = layers.block_norm(h, x, w, post_weight=p, gate=g)
    b = layers.block_norm(h.view(2, 3, 4, 64), x.view(2, 3, 4, 64), w, post_weight=p, gate=g.view(2, 3, 4, 64))
    assert b.y.shape == (2, 3, 4, 64) and torch.equal(b.y.view(24, 64), a.y) and torch.equal(b.s.view(24, 64), a.s)
    c = layers.block_norm(h[0], x[0], w, post_weight=p, gate=g[0])
    assert c.y.shape == (64,) and torch.equal(c.y, a.y[0])


def test_rows_do_not_mix(layers):
    """NaN and infinities stay in their row; a row of zeros gives zeros."""
    h, x, w, p, g = inputs(40, 72, BF, "vector", True)
    a = layers.block_norm(h, x, w, post_weight=p, gate=g)
    h[3, 5], x[7, 0], x[9], h[9] = float("nan"), float("inf"), 0, 0
    b = layers.block_norm(h, x, w, post_weight=p, gate=g)
    assert torch.isnan(b.y[3]).all() and not torch.isfinite(b.s[7, 0]) and (b.y[9] == 0).all()
    keep = [i for i in range(40) if i not in (3, 7, 9)]
    assert torch.equal(a.y[keep], b.y[keep])


def test_offsets_past_32_bits(layers):
    rows, cols = 2 ** 32 // 1024 + 3, 1024
    h = torch.zeros((rows, cols), dtype=BF, device="cuda")
    x = torch.zeros((rows, cols), dtype=BF, device="cuda")
    h[-2:], x[-2:] = rnd((2, cols), 0, BF), rnd((2, cols), 1, BF)
    w, p, g = rnd((cols,), 2, BF), rnd((cols,), 3, BF), rnd((cols,), 4, BF)
    b = layers.block_norm(h, x, w, post_weight=p, gate=g, need_backward=True)
    c = layers.block_norm(h[-2:].clone(), x[-2:].clone(), w, post_weight=p, gate=g)
    assert torch.equal(b.y[-2:], c.y) and torch.equal(b.s[-2:], c.s)
    out = layers.block_norm_backward(x, h, b.s, w, b.rstd, post_weight=p, rstd_post=b.rstd_post, gate=g)
    assert (out.dx[:5] == 0).all() and out.dx[-2:].abs().sum() > 0


@pytest.mark.parametrize("cols,ld", [(256, 256), (77, 80), (77, 77)])
@pytest.mark.parametrize("over", ["x", "h"])
def test_sum_in_place(layers, over, cols, ld):
    """s may be the array of x or of h (through the C ABI; the torch layer allocates s)."""
    from differentiable_rasterizer_gb300 import abi
    rows = 3001
    h, x, w, p, g = inputs(rows, cols, BF, "vector", True, pitch=ld)
    want = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=0.75)
    s, y = (x if over == "x" else h), torch.empty((rows, cols), dtype=BF, device="cuda")
    abi.gs_block_norm(rows, cols, h.data_ptr(), ld, x.data_ptr(), ld, p.data_ptr(), g.data_ptr(), 0, w.data_ptr(), s.data_ptr(), ld,
                      y.data_ptr(), cols, 0, 0, 0, 0.75, EPS, 1, 1, 1, 0, 1, 1, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(y, want.y) and torch.equal(s, want.s)


def test_no_rows(layers):
    e, w = torch.empty((0, 32), dtype=BF, device="cuda"), rnd((32,), 0, BF)
    b = layers.block_norm(e, e, w, post_weight=w, gate=w, need_backward=True)
    assert b.y.shape == (0, 32)
    g = layers.block_norm_backward(e, e, b.s, w, b.rstd, post_weight=w, rstd_post=b.rstd_post, gate=w)
    assert all((t == 0).all() for t in (g.dweight, g.dpost_weight, g.dgate)) and g.dh.shape == (0, 32)


def test_bits_streams_and_graphs(layers):
    h, x, w, p, g = inputs(3001, 256, BF, "vector", True)
    dy = rnd((3001, 256), 9, BF)

    def step():
        b = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=0.5, need_backward=True)
        return (*b[:1], *b[2:], *layers.block_norm_backward(dy, h, b.s, w, b.rstd, post_weight=p, rstd_post=b.rstd_post, gate=g, scale=0.5))

    want = step()
    assert all(torch.equal(u, v) for u, v in zip(want, step()))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, got))
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            out = step()
        graphs.append((graph, out))
    for t in (h, x, dy):
        t.copy_(t.flip(0))
    want = step()
    for graph, out in graphs:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, out))


def test_against_differences(layers):
    """Along a direction, the change of sum(dy y) + sum(ds s) by the formulas in 64 bits is the fp32 gradients' product with it."""
    rows, cols, scale = 20, 48, 0.6
    h, x, w, p, g = inputs(rows, cols, F32, "rows", True)
    dy, ds = rnd((rows, cols), 7, F32), rnd((rows, cols), 8, F32)
    b = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=scale, eps=EPS, need_backward=True)
    out = layers.block_norm_backward(dy, h, b.s, w, b.rstd, post_weight=p, rstd_post=b.rstd_post, gate=g, scale=scale, ds=ds)

    def loss(h, x, w, p, g):
        _, s, _, _, y, _, _ = forward64(h, x, w, p, g, scale)
        return (dy.double() * y).sum() + (ds.double() * s).sum()

    point = [t.double() for t in (h, x, w, p, g)]
    for i, grad in enumerate((out.dh, out.dx, out.dweight, out.dpost_weight, out.dgate)):
        step = [torch.zeros_like(t) for t in point]
        step[i] = rnd(tuple(point[i].shape), 60 + i, F32).double()
        e = 1e-6
        up, down = (loss(*(t + f * e * d for t, d in zip(point, step))) for f in (1, -1))
        terms = grad.double() * step[i]
        assert abs(terms.sum() - (up - down) / (2 * e)) <= 2.0 ** -18 * terms.abs().sum() + 1e-6, i


def test_refusals(layers):
    from differentiable_rasterizer_gb300 import abi
    h, x, w, p, g = inputs(6, 32, BF, "vector", True)
    r = torch.ones(6, device="cuda")
    for bad, match in ((dict(x=x[:5]), "x: 5 rows"), (dict(x=x.half()), "expected BFloat16"), (dict(weight=w[:31]), "weight"),
                       (dict(gate=g[:31]), "gate"), (dict(gate=rnd((5, 32), 0, BF)), "gate: 5 rows"), (dict(gate=rnd((6, 32), 0, F32)), "gate"),
                       (dict(scale=None), "scale"), (dict(out_dtype=torch.int8), "out_dtype"), (dict(weight=None, out_dtype=BF), "out_dtype"),
                       (dict(h=h.t()), "contiguous"), (dict(post_weight=p.cpu()), "on cpu")):
        with pytest.raises(ValueError, match=match):
            layers.block_norm(**{**dict(h=h, x=x, weight=w, post_weight=p, gate=g), **bad})
    for bad in (dict(scale=float("nan")), dict(scale=float("inf")), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(abi.GsError):
            layers.block_norm(h, x, w, **bad)
    full = dict(dy=h, h=h, s=x, weight=w, rstd=r, post_weight=p, rstd_post=r, gate=g)
    for bad, match in ((dict(rstd=None), "rstd"), (dict(rstd_post=None), "rstd_post"), (dict(dy=None), "dy: required"), (dict(s=x[:5]), "s: 5 rows"),
                       (dict(dy=None, weight=None), "ds: required"), (dict(weight=None), "weight: required")):
        with pytest.raises(ValueError, match=match):
            layers.block_norm_backward(**{**full, **bad})
    assert math.isfinite(float(layers.block_norm_backward(**full).dx.float().sum()))
