"""A single row without a dimension of rows, and a gate of another type than its own."""
import pytest
import torch

from test_gpu_block_norm import BF, F32, HF, close, forward64, layers, rnd   # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate_type", [BF, HF, F32])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("cols", [64, 331])
def test_gate_of_a_single_row(layers, cols, dt, gate_type):
    """The same as the row of a matrix with one, forward and gradients."""
    h, x, dy = (rnd((1, cols), i, dt) for i in range(3))
    w, p, g = rnd((cols,), 3, dt), rnd((cols,), 4, dt), rnd((cols,), 5, gate_type)
    b = layers.block_norm(h[0], x[0], w, post_weight=p, gate=g, scale=0.75, need_backward=True)
    _, s, es, _, y, ey, _ = forward64(h, x, w, p, g, 0.75)
    close(b.s[None], s, es, "s")
    close(b.y[None], y, ey, "y")
    c = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=0.75, need_backward=True)
    if dt != gate_type:
        assert torch.equal(b.y, c.y[0]) and torch.equal(b.s, c.s[0])
    d = layers.block_norm_backward(dy[0], h[0], c.s[0], w, c.rstd, post_weight=p, rstd_post=c.rstd_post, gate=g, scale=0.75)
    e = layers.block_norm_backward(dy, h, c.s, w, c.rstd, post_weight=p, rstd_post=c.rstd_post, gate=g, scale=0.75)
    assert d.dgate.shape == (cols,) and d.dgate.dtype == gate_type
    for name in ("dh", "dx", "dweight", "dpost_weight", "dgate"):
        m, n = getattr(d, name).double().flatten(), getattr(e, name).double().flatten()
        # both forms are the same number but for the order of two products, rounded to the type
        u = {BF: 2.0 ** -7, HF: 2.0 ** -10, F32: 2.0 ** -20}[getattr(d, name).dtype]
        assert ((m - n).abs() <= u * torch.maximum(m.abs(), n.abs()) + 2.0 ** -18 * n.abs().max()).all(), name
