"""The decoder network through the layers and the rasterizer: its outputs and gradients
against the same network in 64 bits, its 8-bit serving form, and training through the
rasterizer.

Tolerances: every intermediate is rounded to bfloat16 (2^-8 half a unit, so 2^-9 RMS),
about ten of them in a row on the longest path; a relative error of 2^-9 sqrt(10) < 1 %
in the norm of each tensor, bounded here by 2 %.  8 bits: e4m3's half unit is 2^-4, its
RMS error about 2.6 % a factor; two factors in each of two projections, 4 % in h, which
reaches the output through the head beside the exact residual stream: 6 % of the decoded
part.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mods():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import decoder, pipeline, scenes
    return decoder, pipeline, scenes


def net64(x, w, base):
    def norm(v, g):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * g
    n = norm(x, w["norm1"])
    h = torch.nn.functional.silu(n @ w["w_gate"].t()) * (n @ w["w_up"].t())
    y = norm(x + h @ w["w_down"].t(), w["norm2"])
    return y @ w["w_head"].t() + w["b_head"] + base


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("n,features,hidden,sh", [(1000, 64, 128, 0), (333, 40, 72, 3), (5, 600, 1100, 3)])
def test_decoder_against_64_bits(mods, n, features, hidden, sh):
    decoder, _, _ = mods
    stride = 16 if sh == 0 else 64
    g = torch.Generator().manual_seed(3)
    base = torch.randn((n, stride), generator=g).cuda()
    dec = decoder.GaussianDecoder(features, hidden, sh, base)
    dec.masters["w_head"] *= 50
    dec.refresh()
    x = torch.randn((n, features), generator=g).cuda().to(torch.bfloat16)
    params = torch.full((n, stride), 7.0, device="cuda")
    saved = dec.decode(x, params)
    assert (params[:, dec.P:] == 7).all()   # the blocks' padding is left alone
    x64 = x.double().requires_grad_(True)
    w64 = {k: v.double().requires_grad_(True) for k, v in dec.w.items()}
    out = net64(x64, w64, base[:, :dec.P].double())
    decoded = out.detach() - base[:, :dec.P].double()
    assert rel(params[:, :dec.P] - base[:, :dec.P], decoded) < 0.02
    dp = torch.zeros((n, stride), device="cuda")
    dp[:, :dec.P] = torch.randn((n, dec.P), generator=g).cuda() * 1e-6   # the size of an image loss's gradients
    grads = dec.backward(dp, saved)
    out.backward(dp[:, :dec.P].double())
    assert rel(grads["x"], x64.grad) < 0.02
    for k in dec.WEIGHTS:
        assert rel(grads[k], w64[k].grad) < 0.02, k
    q = torch.zeros((n, stride), device="cuda")
    dec.decode_e4m3(x, q)
    assert rel(q[:, :dec.P] - base[:, :dec.P], decoded) < 0.06


def test_training_through_the_rasterizer(mods):
    """The command's run on the tiny scene, 60 steps: the L1 loss falls below half its start."""
    decoder, pipeline, scenes = mods
    losses = decoder.main(["--steps", "60"])
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
