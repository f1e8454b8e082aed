"""The decoder network with attention: its outputs and gradients against the same network in
64 bits, its 8-bit serving form, and a clipped step through the rasterizer.

Tolerances as for the network without it: every intermediate is rounded to bfloat16 (RMS
2^-9), about twenty of them in a row on the longest path; 2^-9 sqrt(20) < 1 % in the norm of
each tensor, bounded by 2 %.  8 bits: two factors of 2.6 % in each of two projections: 6 % of
the decoded part.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import decoder, layers, pipeline, scenes
    return decoder, layers, pipeline, scenes


def net64(x, w, base, heads, kv_heads, dim, groups, scale):
    def norm(v, g):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * g

    qkv = norm(x, w["norm0"]) @ w["w_qkv"].t()
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], dim=1))
    k, v = (t.repeat_interleave(heads // kv_heads, dim=1) for t in (k, v))
    o, at = [], 0
    for n in groups:
        rows = slice(at, at + n)
        t = torch.einsum("qhd,khd->hqk", q[rows], k[rows]) * dim ** -0.5
        o.append(torch.einsum("hqk,khd->qhd", torch.softmax(t, -1), v[rows]).flatten(1))
        at += n
    o.append(torch.zeros((x.shape[0] - at, heads * dim), dtype=x.dtype, device=x.device))
    s1 = scale * x + w["gate1"] * norm(torch.cat(o) @ w["w_out"].t(), w["post1"])
    n1 = norm(s1, w["norm1"])
    h = torch.nn.functional.silu(n1 @ w["w_gate"].t()) * (n1 @ w["w_up"].t())
    s2 = scale * s1 + w["gate2"] * norm(h @ w["w_down"].t(), w["post2"])
    return norm(s2, w["norm2"]) @ w["w_head"].t() + w["b_head"] + base


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("n,features,hidden,sh,heads,kv_heads,groups,scale", [
    (1000, 64, 128, 0, 4, 4, [256, 256, 256, 232], 1.0), (333, 40, 72, 3, 4, 1, [100, 1, 200], 0.9),
    (700, 512, 1100, 3, 8, 2, [700], 0.8)])
def test_against_64_bits(mods, n, features, hidden, sh, heads, kv_heads, groups, scale):
    decoder = mods[0]
    stride = 16 if sh == 0 else 64
    g = torch.Generator().manual_seed(3)
    base = torch.randn((n, stride), generator=g).cuda()
    dec = decoder.GaussianDecoder(features, hidden, sh, base, heads=heads, kv_heads=kv_heads, groups=groups, residual_scale=scale)
    dec.masters["w_head"] *= 50
    for k in ("gate1", "gate2", "post1", "post2", "norm0"):
        dec.masters[k] += 0.3 * torch.randn(features, generator=g).cuda()
    dec.refresh()
    x = torch.randn((n, features), generator=g).cuda().to(torch.bfloat16)
    params = torch.full((n, stride), 7.0, device="cuda")
    saved = dec.decode(x, params)
    assert (params[:, dec.P:] == 7).all()
    x64 = x.double().requires_grad_(True)
    w64 = {k: v.double().requires_grad_(True) for k, v in dec.w.items()}
    out = net64(x64, w64, base[:, :dec.P].double(), heads, kv_heads, dec.head_dim, groups, scale)
    decoded = out.detach() - base[:, :dec.P].double()
    assert rel(params[:, :dec.P] - base[:, :dec.P], decoded) < 0.02
    dp = torch.zeros((n, stride), device="cuda")
    dp[:, :dec.P] = torch.randn((n, dec.P), generator=g).cuda() * 1e-6   # the size of an image loss's gradients
    grads = dec.backward(dp, saved)
    out.backward(dp[:, :dec.P].double())
    assert rel(grads["x"], x64.grad) < 0.02
    for k in dec.WEIGHTS + dec.ATTENTION_WEIGHTS:
        assert rel(grads[k], w64[k].grad) < 0.02, k
    q = torch.zeros((n, stride), device="cuda")
    dec.decode_e4m3(x, q)
    assert rel(q[:, :dec.P] - base[:, :dec.P], decoded) < 0.06


def test_a_clipped_step_through_the_rasterizer(mods):
    """Gradients of all weights arrive through the rasterizer, and clipping brings their norm to the largest allowed, in fp32."""
    decoder, layers, pipeline, scenes = mods
    sc = scenes.make_scene("tiny")
    trainer = pipeline.GaussianTrainer(sc.params, sc.sh_degree, sc.cameras, sc.opts, sc.lr)
    target = trainer.render().clone()
    base = trainer.params.clone()
    base[:, 11:trainer.P] = 0
    dec = decoder.GaussianDecoder(64, 128, sc.sh_degree, base, heads=4, kv_heads=2, groups=[256] * (trainer.n // 256))
    x = torch.randn((trainer.n, 64), generator=torch.Generator().manual_seed(1)).cuda().to(torch.bfloat16)
    grads = dec.grads(trainer, x, target)
    assert set(grads) == {"x", *dec.WEIGHTS, *dec.ATTENTION_WEIGHTS}
    assert all(torch.isfinite(t).all() and t.abs().sum() > 0 for t in grads.values())
    norm = sum(float(t.double().square().sum()) for t in grads.values()) ** 0.5
    out = [torch.empty(t.shape, device="cuda") for t in grads.values()]
    got = layers.clip_norm([t.contiguous() for t in grads.values()], norm / 4, out=out)
    assert abs(float(got) - norm) < 1e-5 * norm
    assert abs(sum(float(t.double().square().sum()) for t in out) ** 0.5 - norm / 4) < 1e-4 * norm


def test_the_command_runs(mods):
    losses = mods[0].main(["--steps", "3", "--heads", "4", "--kv-heads", "2", "--group", "100", "--clip", "1e-3"])
    assert len(losses) == 3 and all(x == x for x in losses)
