"""Arguments of the layers on torch tensors: what is of the wrong kind raises ValueError and
names the argument, also with no rows, and leaves no error behind."""
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
