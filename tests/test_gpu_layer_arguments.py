"""Arguments of the layers on torch tensors: what is of the wrong kind raises ValueError and
names the argument, also with no rows, and leaves no error behind; a tensor whose gradient would be lost is
refused; writes to a given output are seen by autograd."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def layers():
    from differentiable_rasterizer_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from differentiable_rasterizer_gb300 import layers as L
    return L


def zeros(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt, device="cuda")


@pytest.mark.parametrize("rows", [0, 6])
def test_wrong_kinds(layers, rows):
    x, w, v, dy = zeros(rows, 16), zeros(8, 16), zeros(16), zeros(rows, 8)
    two = torch.tensor([1, 2])   # has no truth value
    cases = [
        ("eps: expected a number, got str", lambda: layers.rms_norm(x, v, eps="small")),
        ("eps: expected a number, got NoneType", lambda: layers.rms_norm(x, v, eps=None)),
        ("need_backward: expected a truth value", lambda: layers.rms_norm(x, v, need_backward=two)),
        ("need_backward: expected a truth value", lambda: layers.linear(x, w, act="relu", need_backward=two)),
        ("bias: expected a truth value", lambda: layers.linear_backward(dy, x, w, bias=two)),
        ("need_dx: expected a truth value", lambda: layers.linear_backward(dy, x, w, need_dx=two)),
        ("need_dw: expected a truth value", lambda: layers.linear_backward(dy, x, w, need_dw=two)),
        ("save: expected a truth value", lambda: layers.glu(x, w, w, need_backward=True, save=two)),
        ("need_dx: expected a truth value", lambda: layers.glu_backward(dy, x, w, w, need_dx=two)),
        ("need_dw: expected a truth value", lambda: layers.glu_backward(dy, x, w, w, need_dw=two)),
        ("act: .* is not one of", lambda: layers.linear(x, w, act=["silu"])),
        ("x: expected a tensor, got NoneType", lambda: layers.glu(None, w, w, need_backward=True)),
        ("x: needs at least one dimension", lambda: layers.glu(zeros(), w, w, need_backward=True)),
    ]
    for what, call in cases:
        with pytest.raises(ValueError, match=what):
            call()
        assert (layers.linear(zeros(1, 16), w).y == 0).all()   # and the next call is as ever
    assert layers.rms_norm(x, v, eps=1).y.shape == (rows, 16)   # any number is one


def test_tensors_that_require_grad(layers):
    """Refused while gradients are recorded, by name, wherever they come in; taken detached or without recording."""
    x, w, v, dy, b = zeros(6, 16), zeros(8, 16), zeros(16), zeros(6, 8), zeros(8)
    rstd, s8 = zeros(6, dt=F32), zeros(6, dt=F32)
    r = lambda t: t.clone().requires_grad_(True)   # noqa: E731
    calls = {
        "x": [lambda g: layers.rms_norm(g(x), v), lambda g: layers.linear(g(x), w), lambda g: layers.quantize_rows(g(x)),
              lambda g: layers.glu(g(x), w, w, need_backward=True), lambda g: layers.linear_backward(dy, g(x), w)],
        "w": [lambda g: layers.linear(x, g(w)), lambda g: layers.linear_backward(dy, x, g(w))],
        "weight": [lambda g: layers.rms_norm(x, g(v)), lambda g: layers.rms_norm_backward(x, x, g(v), rstd)],
        "bias": [lambda g: layers.linear(x, w, g(b))],
        "residual": [lambda g: layers.rms_norm(x, v, residual=g(x)), lambda g: layers.linear(x, w, residual=g(dy))],
        "out": [lambda g: layers.linear(x, w, out=g(dy))],
        "w_gate": [lambda g: layers.glu(x, g(w), w), lambda g: layers.glu_backward(dy, x, g(w), w)],
        "w_up": [lambda g: layers.glu(x, w, g(w)), lambda g: layers.glu_backward(dy, x, w, g(w))],
        "x_scale": [lambda g: layers.linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), x_scale=g(s8))],
        "dy": [lambda g: layers.linear_backward(g(dy), x, w), lambda g: layers.rms_norm_backward(g(x), x, v, rstd)],
        "dh": [lambda g: layers.glu_backward(g(dy), x, w, w)],
        "z": [lambda g: layers.linear_backward(dy, x, w, z=g(dy), act="silu")],
        "rstd": [lambda g: layers.rms_norm_backward(x, x, v, g(rstd))],
        "ds": [lambda g: layers.rms_norm_backward(x, x, v, rstd, ds=g(x))],
    }
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(ValueError, match=f"^{name}: requires grad"):
                f(r)
            f(lambda t: r(t).detach())
            with torch.no_grad():
                f(r)


def test_decoder_takes_its_own_masters(layers):
    """Masters that an optimizer trains require grad; the network's working weights do not."""
    from differentiable_rasterizer_gb300 import decoder
    dec = decoder.GaussianDecoder(16, 24, 0)
    for v in dec.masters.values():
        v.requires_grad_(True)
    dec.refresh()
    params = torch.zeros((10, 16), device="cuda")
    saved = dec.decode(torch.randn((10, 16), device="cuda").to(BF), params)
    assert dec.backward(torch.ones_like(params), saved)["w_head"].shape == dec.masters["w_head"].shape


def test_writes_to_out_are_seen(layers):
    """A tensor that autograd has saved and a layer overwrites: its backward says so, as after any write in place."""
    x, w = zeros(6, 16), zeros(8, 16)
    y = torch.ones((6, 12), device="cuda")
    leaf = torch.ones((6, 12), device="cuda", requires_grad=True)
    loss = (leaf * y).sum()
    before = y._version
    layers.linear(x, w, out=y[:, 2:10], out_dtype=F32)
    assert y._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        layers.linear(x, w, out=torch.ones((6, 8), dtype=BF, device="cuda"))
