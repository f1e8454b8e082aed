"""fp32 rows of a few columns at pitches of four, eight and twelve, the matrix's last row at the end of its memory."""
import pytest
import torch

from test_gpu_block_norm import F32, check_backward, close, forward64, layers, rnd   # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pitch", [4, 8, 12])
@pytest.mark.parametrize("cols", [1, 2, 3, 4, 5, 9, 11, 12])
@pytest.mark.parametrize("rows", [1, 2, 3, 50])
def test_narrow_rows(layers, rows, cols, pitch):
    if cols > pitch:
        return

    def at_end(seed):
        t = rnd((rows, cols), seed, F32)
        flat = torch.full(((rows - 1) * pitch + cols,), float("nan"), device="cuda")
        v = flat.as_strided((rows, cols), (pitch, 1))
        v.copy_(t)
        return v

    h, x, g, dy, ds = (at_end(i) for i in range(5))
    w, p = 1 + rnd((cols,), 5, F32, 0.2), 1 + rnd((cols,), 6, F32, 0.2)
    b = layers.block_norm(h, x, w, post_weight=p, gate=g, scale=0.75, eps=1e-6, need_backward=True)
    _, s, es, _, y, ey, _ = forward64(h, x, w, p, g, 0.75)
    close(b.s, s, es, "s")
    close(b.y, y, ey, "y")
    check_backward(layers, h, x, w, p, g, 0.75, b, dy, ds)
