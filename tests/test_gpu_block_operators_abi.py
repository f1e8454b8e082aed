"""Attention, block norm and clipping through the ctypes calls, which the torch layer does not go
through: the same bits as the torch layer's, outputs not asked for left out, and the operators in a run
as a block's training step uses them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mods():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import abi, layers
    return abi, layers


def rnd(shape, seed, dtype=BF, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def scratch(abi, name, args):
    n = abi.layer_ws_bytes(name, args)
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"), n


def stream():
    return torch.cuda.current_stream().cuda_stream


def test_attention(mods):
    abi, layers = mods
    q_lens, k_lens = [70, 1, 200], [300, 9, 200]
    qs, ks = (torch.tensor([0, *n]).cumsum(0).to(torch.int32).cuda() for n in (q_lens, k_lens))
    q, k, v, do = rnd((280, 4, 72), 0), rnd((520, 2, 72), 1), rnd((520, 2, 72), 2), rnd((280, 4, 72), 3)
    want = layers.attention(q, k, v, q_starts=qs, k_starts=ks, causal=True, need_backward=True, scale=0.2)
    grads = layers.attention_backward(do, q, k, v, want.o, want.lse, q_starts=qs, k_starts=ks, causal=True, scale=0.2)
    o, lse = torch.full_like(q, 5.0), torch.full((280, 4), 5.0, device="cuda")
    sizes = (280, 520, 3)
    kv = (q.data_ptr(), 288, 72, k.data_ptr(), 144, 72, v.data_ptr(), 144, 72)
    args = abi.attention_args(*sizes, *kv, qs.data_ptr(), ks.data_ptr(), 0, o.data_ptr(), 288, 72, lse.data_ptr(), 0.2, 4, 2, 72,
                              abi.GS_BF16, 1, 0)
    ws, n = scratch(abi, "gs_attention", args)
    abi.gs_attention(args, ws.data_ptr(), n, stream())
    used = slice(0, 271)
    assert torch.equal(o[used], want.o[used]) and torch.equal(lse[used], want.lse[used])
    assert (o[271:] == 5).all() and (lse[271:] == 5).all() and (want.o[271:] == 0).all()
    dq, dk, dv = (torch.full_like(t, 5.0) for t in (q, k, v))

    def backward(dq, dk, dv, fill):
        args = abi.attention_bwd_args(*sizes, *kv, do.data_ptr(), 288, 72, want.lse.data_ptr(), qs.data_ptr(), ks.data_ptr(), dq, 288, 72, dk,
                                      144, 72, dv, 144, 72, 0.2, 4, 2, 72, abi.GS_BF16, 1, fill)
        ws, n = scratch(abi, "gs_attention_bwd", args)
        abi.gs_attention_bwd(args, ws.data_ptr(), n, stream())

    backward(dq.data_ptr(), 0, 0, 0)                       # dq alone
    assert torch.equal(dq[used], grads.dq[used]) and (dq[271:] == 5).all() and (dk == 5).all()
    backward(0, dk.data_ptr(), dv.data_ptr(), 1)           # dk and dv alone, rows of no sequence filled
    assert torch.equal(dk, grads.dk) and torch.equal(dv, grads.dv) and (dk[509:] == 0).all()


def test_block_norm_gradients_one_by_one(mods):
    abi, layers = mods
    rows, cols = 400, 96
    h, x, dy, ds = (rnd((rows, cols), i) for i in range(4))
    w, p, g = rnd((cols,), 4), rnd((cols,), 5), rnd((cols,), 6)
    b = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=0.5, need_backward=True)
    want = layers.block_norm_backward(dy, h, b.s, w, b.rstd, post_weight=p, rstd_post=b.rstd_post, gate=g, scale=0.5, ds=ds)
    for which in ("dh", "dx", "dgate", "dweight", "dpost"):
        out = torch.full_like(want.dpost_weight if which == "dpost" else getattr(want, which), 7.0)
        to = {k: 0 for k in ("dh", "dx", "dgate", "dweight", "dpost")}
        to[which] = out.data_ptr()
        args = abi.block_norm_bwd_args(rows, cols, dy.data_ptr(), cols, ds.data_ptr(), cols, h.data_ptr(), cols, b.s.data_ptr(), cols, p.data_ptr(),
                                       g.data_ptr(), 0, w.data_ptr(), b.rstd_post.data_ptr(), b.rstd.data_ptr(), to["dh"], cols, to["dx"], cols,
                                       to["dgate"], 0, to["dweight"], to["dpost"], 0.5, 1, 1, 1, 1, 0, 1)
        ws, n = scratch(abi, "gs_block_norm_bwd", args)
        abi.gs_block_norm_bwd(args, ws.data_ptr() if n else None, n if n else None, stream())
        assert torch.equal(out, want.dpost_weight if which == "dpost" else getattr(want, which)), which


def test_clip(mods):
    abi, layers = mods
    tensors = [rnd((n,), n, F32) for n in (5, 20000, 300)]
    outs = [torch.empty_like(t, dtype=BF) for t in tensors]
    norm = torch.empty((), device="cuda")
    args, table = abi.clip_norm_args([(t.data_ptr(), o.data_ptr(), t.numel(), abi.GS_F32, abi.GS_BF16) for t, o in zip(tensors, outs)],
                                     norm.data_ptr(), 3.0)
    ws, n = scratch(abi, "gs_clip_norm", args)
    abi.gs_clip_norm(args, ws.data_ptr(), n, stream())
    del table
    other = [torch.empty_like(t, dtype=BF) for t in tensors]
    assert torch.equal(layers.clip_norm(tensors, 3.0, out=other), norm) and all(torch.equal(a, b) for a, b in zip(outs, other))


def test_a_block_in_training(mods):
    """Attention, block norm and clipping as a block's step uses them, each on the others' outputs, against 64-bit autograd of the
    whole.  Every stored tensor is rounded to bfloat16 (RMS 2^-9 of its norm), eight in a row: below 2^-9 sqrt(8) 3 = 1.7 %."""
    abi, layers = mods
    n, heads, kv, dim = 300, 4, 2, 32
    width, lens = heads * dim, [100, 56, 144]
    starts = torch.tensor([0, *lens]).cumsum(0).to(torch.int32).cuda()
    x, dy = rnd((n, width), 0), rnd((n, width), 1)
    w = {"qkv": rnd((width + 2 * kv * dim, width), 2, std=width ** -0.5), "out": rnd((width, width), 3, std=width ** -0.5),
         "post": 1 + rnd((width,), 4, std=0.2), "gate": rnd((width,), 5, std=0.5), "norm": 1 + rnd((width,), 6, std=0.2)}
    cut = [heads * dim, kv * dim, kv * dim]
    qkv = layers.linear(x, w["qkv"]).y
    q, k, v = (t.unflatten(1, (-1, dim)) for t in qkv.split(cut, dim=1))
    a = layers.attention(q, k, v, q_starts=starts, causal=True, need_backward=True)
    p = layers.linear(a.o.flatten(1), w["out"]).y
    b = layers.block_norm(p, x, w["norm"], post_weight=w["post"], gate=w["gate"], scale=0.9, need_backward=True)
    g = layers.block_norm_backward(dy, p, b.s, w["norm"], b.rstd, post_weight=w["post"], rstd_post=b.rstd_post, gate=w["gate"], scale=0.9)
    out = layers.linear_backward(g.dh, a.o.flatten(1), w["out"])
    dqkv = torch.empty_like(qkv)
    layers.attention_backward(out.dx.unflatten(1, (heads, dim)), q, k, v, a.o, a.lse, q_starts=starts, causal=True,
                              out=[t.unflatten(1, (-1, dim)) for t in dqkv.split(cut, dim=1)])
    proj = layers.linear_backward(dqkv, x, w["qkv"])
    grads = [proj.dw, out.dw, g.dpost_weight, g.dgate, g.dweight]
    clipped = [torch.empty(t.shape, device="cuda") for t in grads]
    norm = layers.clip_norm(grads, 1.0, out=clipped)

    x64 = x.double()
    w64 = {name: t.double().requires_grad_(True) for name, t in w.items()}

    def rms(t):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6)

    q, k, v = (t.unflatten(1, (-1, dim)) for t in (x64 @ w64["qkv"].t()).split(cut, dim=1))
    k, v = (t.repeat_interleave(heads // kv, dim=1) for t in (k, v))
    o, at = [], 0
    for m in lens:
        rows = slice(at, at + m)
        t = torch.einsum("qhd,khd->hqk", q[rows], k[rows]) * dim ** -0.5
        t = t.masked_fill(~torch.ones(m, m, dtype=torch.bool, device="cuda").tril(), float("-inf"))
        o.append(torch.einsum("hqk,khd->qhd", torch.softmax(t, -1), v[rows]).flatten(1))
        at += m
    s = 0.9 * x64 + w64["gate"] * rms(torch.cat(o) @ w64["out"].t()) * w64["post"]
    (rms(s) * w64["norm"] * dy.double()).sum().backward()
    want = [w64[name].grad for name in ("qkv", "out", "post", "gate", "norm")]
    total = sum(float(t.square().sum()) for t in want) ** 0.5
    assert abs(float(norm) - total) < 0.01 * total
    for name, got, t in zip(("qkv", "out", "post", "gate", "norm"), clipped, want):
        assert float((got.double() * float(norm) - t).norm() / t.norm()) < 0.017, name
    assert not abi.gs_wait_report()
