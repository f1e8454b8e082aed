"""The ctypes calls of the layers' gradients, which the torch layer does not go through: no rows
and no weights' gradients asked for, so nothing is queued and no scratch is needed (no GPU)."""
import pytest


@pytest.fixture(scope="module")
def abi():
    from differentiable_rasterizer_gb300 import abi as A
    from differentiable_rasterizer_gb300 import build
    build.build()
    A.lib()
    return A


def calls(abi, rows):
    bf = abi.GS_BF16
    return [
        (abi.gs_rms_norm_bwd, abi.rms_norm_bwd_args(rows, 32, 0, 32, 0, 32, 4096, 0, 0, 0, 0, 32, 0, bf, bf, bf)),
        (abi.gs_linear_bwd, abi.linear_bwd_args(rows, 32, 16, 0, 16, 0, 32, 0, 32, 0, 0, 0, 32, 0, 32, 0, bf, bf, bf, bf, 0)),
        (abi.gs_glu_bwd, abi.glu_bwd_args(rows, 32, 16, 0, 16, 0, 32, 0, 32, 0, 32, 0, 16, 0, 16, 0, 32, 0, 32, 0, 32, bf, bf, 2)),
    ]


def test_gradient_calls_without_rows(abi):
    for call, args in calls(abi, 0):
        assert call(args, None, None, None) is None


def test_gradient_calls_raise_the_status(abi):
    for call, args in calls(abi, -1):
        with pytest.raises(abi.GsError) as e:
            call(args, None, None, None)
        assert e.value.status == abi.GS_ERR_INVALID_ARG
