"""The norm over many tensors and clipping on the GPU.

Bounds (derived before the first run): squares are added in fp32 for at most 32 values, then in
fp64: 2^-20 relative of the sum, half of it in the root, 2^-24 for the result's rounding: the norm
within 2^-20.  The scaled values follow from the returned norm to the bit: factor =
fp32(max_norm / norm), out = v * factor rounded once (v * factor in fp32 first, where out is narrower)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
NP = {BF: "bf16", HF: "f16", F32: "f32"}


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


def rnd(n, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def norm64(tensors):
    return math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in tensors))


def check(layers, tensors, max_norm, out_types=None, in_place=False):
    before = [t.clone() for t in tensors]
    outs = None if in_place else [torch.full_like(t, 7, dtype=o) for t, o in zip(tensors, out_types or [t.dtype for t in tensors])]
    norm = layers.clip_norm(tensors, max_norm, out=outs)
    assert norm.shape == () and norm.dtype == F32
    want = norm64(before)
    assert abs(float(norm) - want) <= 2.0 ** -20 * want, (float(norm), want)
    factor = torch.where(norm > max_norm, torch.full_like(norm, max_norm) / norm, torch.ones_like(norm))
    for t, b, o in zip(tensors, before, tensors if in_place else outs):
        assert torch.equal(o, (b.float() * factor).to(o.dtype))
        if not in_place:
            assert torch.equal(t, b)
    return norm


SIZES = [[1], [8], [1, 2, 3], [8191, 8192, 8193], [0, 5, 0, 100000, 0], [64 * 128] * 7, [1000003], [3] * 1024, [16384 * 300 + 5, 1, 777],
         [i * 37 + 1 for i in range(200)], [0, 0]]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("over", [False, True])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_sizes(layers, i, over, in_place):
    tensors = [rnd(n, j, F32, 0.1) for j, n in enumerate(SIZES[i])]
    check(layers, tensors, 0.5 * norm64(tensors) if over else 2 * norm64(tensors) + 1, in_place=in_place)


@pytest.mark.parametrize("out", [BF, HF, F32])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_types(layers, dt, out):
    for most in (0.3, 1e6):
        check(layers, [rnd(n, n, dt, 0.3) for n in (5, 1024, 30000)], most, [out] * 3)
    check(layers, [rnd(3000, 1, BF), rnd(2001, 2, F32), rnd(999, 3, HF)], 1.0, [F32, out, BF])


@pytest.mark.parametrize("offset", [1, 3, 4])
def test_unaligned(layers, offset):
    """Slices of one buffer that start anywhere, inputs and outputs apart."""
    flat, to = rnd(50000, 0, BF), torch.zeros(50000, device="cuda")
    cuts = [(offset, 9000), (9000 + offset, 9001), (20000 + offset, 17000)]
    tensors, outs = [flat[a:a + n] for a, n in cuts], [to[a + 1:a + 1 + n] for a, n in cuts]
    norm = layers.clip_norm(tensors, 1.0, out=outs)
    factor = torch.full_like(norm, 1.0) / norm
    for t, o in zip(tensors, outs):
        assert torch.equal(o, t.float() * factor)
    covered = torch.zeros(50000, dtype=torch.bool, device="cuda")
    for a, n in cuts:
        covered[a + 1:a + 1 + n] = True
    assert (to[~covered] == 0).all()


@pytest.mark.parametrize("value", [2.0 ** 127, 2.0 ** 100, 2.0 ** 61, 2.0 ** 59, 2.0 ** -59, 2.0 ** -61, 2.0 ** -100, 2.0 ** -126, 2.0 ** -149])
def test_no_overflow_on_the_way(layers, value):
    """Values whose squares fp32 does not hold, beside zeros and beside far smaller ones."""
    for tensors in ([torch.full((1,), value, device="cuda")], [torch.tensor([0, value, 0, -value * 2 ** -8] * 5000, device="cuda")[:2] * 1.0,
                                                               torch.zeros(10000, device="cuda")]):
        got, want = float(layers.clip_norm(tensors, 1e38 if value < 1 else 0.0, out=[torch.empty_like(t) for t in tensors])), norm64(tensors)
        if want < 3.4e38:
            assert abs(got - want) <= 2.0 ** -20 * want + 2.0 ** -149, (got, want)


def test_norm_beyond_the_type(layers):
    """A finite norm that fp32 does not hold is infinite: nothing is scaled."""
    t = torch.full((100,), 3e38, device="cuda")
    norm = layers.clip_norm([t], 1.0)
    assert math.isinf(float(norm)) and (t == 3e38).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite(layers, bad):
    tensors = [rnd(100, 0, F32), rnd(20000, 1, BF)]
    tensors[1][777] = bad
    before = [t.clone() for t in tensors]
    outs = [torch.zeros_like(t, dtype=F32) for t in tensors]
    norm = layers.clip_norm(tensors, 1.0, out=outs)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    for b, o in zip(before, outs):
        assert torch.equal(b.float().nan_to_num(123.0), o.nan_to_num(123.0))
    layers.clip_norm(tensors, 1.0)
    assert all(torch.equal(b.nan_to_num(1.0), t.nan_to_num(1.0)) for b, t in zip(before, tensors))


def test_zeros_and_zero_norm(layers):
    check(layers, [torch.zeros(1000, device="cuda")], 0.0, in_place=True)
    t = rnd(1000, 0, F32)
    layers.clip_norm([t], 0.0)
    assert (t == 0).all()


def test_large(layers):
    """More values than the caches hold, and more than 2^32 of them."""
    tensors = [rnd(50_000_017, 0, BF, 0.01), rnd(31_000_001, 1, F32, 0.02)]
    check(layers, tensors, 0.7, [F32, F32])
    n = 2 ** 32 + 12345
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[-5:] = 3.0
    norm = layers.clip_norm([t], 1.0)
    assert abs(float(norm) - math.sqrt(45)) < 1e-5
    want = (torch.tensor(3.0) * (torch.tensor(1.0) / norm.cpu())).to(BF)
    assert (t[-5:].cpu() == want).all() and (t[:1000] == 0).all()


def test_bits_streams_and_graphs(layers):
    tensors = [rnd(n, n, BF, 0.1) for n in (100000, 3, 8193, 777777)]
    outs = [torch.empty(t.shape, device="cuda") for t in tensors]

    def step():
        return layers.clip_norm(tensors, 1.0, out=outs)

    norm, want = step().clone(), [o.clone() for o in outs]
    for _ in range(3):
        assert torch.equal(step(), norm) and all(torch.equal(a, b) for a, b in zip(outs, want))
    torch.cuda.synchronize()
    s, other = torch.cuda.Stream(), [torch.empty_like(o) for o in outs]
    with torch.cuda.stream(s):   # beside the same call on the current stream
        n2 = layers.clip_norm(tensors, 1.0, out=other)
    step()
    torch.cuda.synchronize()
    assert torch.equal(n2, norm) and all(torch.equal(a, b) for a, b in zip(other, want))
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            n = step()
        graphs.append((g, n))
    for t in tensors:
        t.mul_(0.5)
    norm, want = step().clone(), [o.clone() for o in outs]
    for g, n in graphs:
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, norm) and all(torch.equal(a, b) for a, b in zip(outs, want))


def test_written_tensors_are_seen_by_autograd(layers):
    t = rnd(100, 0, F32)
    v = t._version
    layers.clip_norm([t], 0.1)
    assert t._version > v


def test_refusals(layers):
    from differentiable_rasterizer_gb300 import abi
    a, b = rnd(100, 0, F32), rnd(100, 1, F32)
    for args, kw, match in ((([], 1.0), {}, "1 to 1024"), ((a, 1.0), {}, "expected a list"), (([a], None), {}, "max_norm"),
                            (([a] * 1025, 1.0), {}, "1 to 1024"), (([a.double()], 1.0), {}, "tensors\\[0\\]"), (([a, b.cpu()], 1.0), {}, "tensors\\[1\\]"),
                            (([a[::2]], 1.0), {}, "not contiguous"), (([a, None], 1.0), {}, "tensors\\[1\\]"), (([a], 1.0), dict(out=[]), "out"),
                            (([a], 1.0), dict(out=[b[:50]]), "out\\[0\\]"), (([a], 1.0), dict(out=b), "out"),
                            (([a.clone().requires_grad_(True)], 1.0), {}, "requires grad")):
        with pytest.raises(ValueError, match=match):
            layers.clip_norm(*args, **kw)
    for args, kw in ((([a], -1.0), {}), (([a], float("nan")), {}), (([a, a], 1.0), {}), (([a, a[50:]], 1.0), {}),
                     (([a, b], 1.0), dict(out=[b, a])), (([a[:50]], 1.0), dict(out=[a[20:70]])), (([a[:50], a[50:]], 1.0), dict(out=[b[:50], b[49:99]]))):
        with pytest.raises(abi.GsError):
            layers.clip_norm(*args, **kw)
    layers.clip_norm([a[:50], a[50:]], 1.0)   # neighbours do not overlap
