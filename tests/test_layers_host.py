"""Refusals of the decoder layers, without a GPU: the library's argument checks answer
before any device work, and the torch layer names what it cannot take."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def abi():
    from differentiable_rasterizer_gb300 import abi as A
    from differentiable_rasterizer_gb300 import build
    build.build()
    A.lib()
    return A


LINEAR = dict(rows=4, in_features=32, out_features=16, x=4096, ldx=32, w=4096, ldw=32, x_scale=0, w_scale=0, bias=0,
              residual=0, ldr=0, y=4096, ldy=16, z=0, ldz=0, type_=1, bias_type=1, out_type=1, act=0)
LINEAR_BWD = dict(rows=4, in_features=32, out_features=16, dy=4096, lddy=16, x=4096, ldx=32, w=4096, ldw=32, z=0, ldz=0,
                  dx=4096, lddx=32, dw=4096, lddw=32, db=0, type_=1, dy_type=1, dw_type=1, db_type=1, act=0)
GLU = dict(rows=4, in_features=32, hidden=16, x=4096, ldx=32, w_gate=4096, ldwg=32, w_up=4096, ldwu=32, x_scale=0,
           gate_scale=0, up_scale=0, h=4096, ldh=16, g=0, ldg=0, u=0, ldu=0, type_=1, out_type=1, act=2)
GLU_BWD = dict(rows=4, in_features=32, hidden=16, dh=4096, lddh=16, x=4096, ldx=32, w_gate=4096, ldwg=32, w_up=4096,
               ldwu=32, g=4096, ldg=16, u=4096, ldu=16, dx=4096, lddx=32, dw_gate=4096, lddwg=32, dw_up=4096, lddwu=32,
               type_=1, dw_type=1, act=2)
NORM_BWD = dict(rows=4, cols=32, dy=4096, lddy=32, sum_=4096, lds=32, weight=4096, rstd=4096, dsum=0, ldds=0, dx=4096,
                lddx=32, dweight=4096, type_=1, dy_type=1, weight_type=1)

BAD = {
    "gs_linear": [dict(rows=-1), dict(in_features=0), dict(out_features=0), dict(rows=2 ** 31), dict(x=0), dict(w=0),
                  dict(y=0), dict(ldx=31), dict(ldw=31), dict(ldy=15), dict(x=4097), dict(y=4097), dict(type_=0),
                  dict(type_=4), dict(out_type=3), dict(act=4), dict(act=-1), dict(x_scale=4096),
                  dict(type_=3, x_scale=4098), dict(bias=4096, bias_type=3), dict(bias=4097), dict(residual=4096, ldr=15),
                  dict(z=4096, ldz=15), dict(type_=3, z=4096, ldz=16), dict(ldy=2 ** 31)],
    "gs_linear_bwd": [dict(rows=-1), dict(in_features=0), dict(dy=0), dict(lddy=15), dict(x=0), dict(w=0), dict(type_=3),
                      dict(type_=0), dict(dy_type=3), dict(act=1), dict(act=1, z=4096, ldz=15), dict(act=9), dict(dw_type=2),
                      dict(dw_type=3), dict(lddx=31), dict(lddw=31), dict(db=4097), dict(db=4096, db_type=3)],
    "gs_glu": [dict(rows=-1), dict(hidden=0), dict(x=0), dict(w_gate=0), dict(w_up=0), dict(h=0), dict(ldh=15),
               dict(ldwu=31), dict(type_=0), dict(out_type=0), dict(out_type=2), dict(gate_scale=4096), dict(act=7),
               dict(g=4096, ldg=16), dict(u=4096, ldu=16), dict(g=4096, ldg=15, u=4096, ldu=16)],
    "gs_glu_bwd": [dict(rows=-1), dict(dh=0), dict(g=0), dict(u=0), dict(x=0), dict(w_gate=0), dict(w_up=0),
                   dict(g=0, u=0, x=0, dw_gate=0, dw_up=0), dict(g=0, u=0, w_up=0, dx=0),
                   dict(dw_gate=0), dict(dw_type=2), dict(type_=3), dict(lddwu=31), dict(lddx=31), dict(ldg=15),
                   dict(act=4)],
    "gs_rms_norm_bwd": [dict(rows=-1), dict(cols=0), dict(cols=16385), dict(dy=0), dict(sum_=0), dict(weight=0),
                        dict(rstd=0), dict(lds=31), dict(lddx=31), dict(type_=3), dict(dy_type=3), dict(weight_type=4),
                        dict(dsum=4096, ldds=31), dict(dweight=4097)],
}
BASE = {"gs_linear": LINEAR, "gs_linear_bwd": LINEAR_BWD, "gs_glu": GLU, "gs_glu_bwd": GLU_BWD,
        "gs_rms_norm_bwd": NORM_BWD}


def _pack(abi, name, args):
    return getattr(abi, name[3:] + "_args")(**args)


@pytest.mark.parametrize("name", sorted(BAD))
def test_bad_arguments(abi, name):
    for change in BAD[name]:
        args = _pack(abi, name, dict(BASE[name], **change))
        big = ctypes.c_size_t(1 << 40)
        # with a workspace of any size: the arguments themselves are refused
        st = getattr(abi.lib(), name)(args, 4096, ctypes.byref(big), None)
        assert st == abi.GS_ERR_INVALID_ARG, change
    assert getattr(abi.lib(), name)(None, None, None, None) == abi.GS_ERR_INVALID_ARG


def test_bad_norm_arguments(abi):
    ok = dict(rows=4, cols=32, x=4096, ldx=32, residual=0, ldr=0, weight=4096, y=4096, ldy=32, y_scale=0, sum_=0, lds=0,
              rstd=0, eps=1e-6, type_=1, weight_type=1, y_type=1, stream=None)
    for change in (dict(rows=-1), dict(cols=0), dict(cols=16385), dict(x=0), dict(weight=0), dict(y=0), dict(ldx=31),
                   dict(ldy=31), dict(residual=4096, ldr=31), dict(sum_=4096, lds=31), dict(type_=3), dict(weight_type=3),
                   dict(y_type=4), dict(y_type=3), dict(y_scale=4096), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(eps=float("inf")), dict(x=4097), dict(rstd=4098)):
        with pytest.raises(abi.GsError) as e:
            abi.gs_rms_norm(**dict(ok, **change))
        assert e.value.status == abi.GS_ERR_INVALID_ARG, change
    ok = dict(rows=4, cols=32, x=4096, ldx=32, q=4096, ldq=32, scale=4096, type_=1, stream=None)
    for change in (dict(rows=-1), dict(cols=0), dict(cols=16385), dict(x=0), dict(q=0), dict(scale=0), dict(ldx=31),
                   dict(ldq=31), dict(type_=3), dict(scale=4097)):
        with pytest.raises(abi.GsError) as e:
            abi.gs_quantize_rows(**dict(ok, **change))
        assert e.value.status == abi.GS_ERR_INVALID_ARG, change


def test_workspaces(abi):
    """Queries answer without device work; too small, misaligned or missing scratch is refused."""
    for name, change in (("gs_linear_bwd", dict(db=4096)), ("gs_glu_bwd", {}), ("gs_rms_norm_bwd", {})):
        args = _pack(abi, name, dict(BASE[name], **change))
        need = abi.layer_ws_bytes(name, args)
        assert need > 0 and need % 256 == 0
        f = getattr(abi.lib(), name)
        for ws, size in ((4096, need - 1), (4096 + 16, need), (4096, 0)):
            assert f(args, ws, ctypes.byref(ctypes.c_size_t(size)), None) == abi.GS_ERR_INVALID_ARG, (name, ws, size)
        assert f(args, None, None, None) == abi.GS_ERR_INVALID_ARG
    small, large = (abi.layer_ws_bytes("gs_glu_bwd", _pack(abi, "gs_glu_bwd", dict(GLU_BWD, rows=r))) for r in (4, 400000))
    assert large > small


def test_zero_rows_do_no_device_work(abi):
    assert abi.gs_linear(_pack(abi, "gs_linear", dict(LINEAR, rows=0, x=0, y=0)), None, None, None) is None
    assert abi.gs_glu(_pack(abi, "gs_glu", dict(GLU, rows=0, x=0, h=0)), None, None, None) is None


def test_tensor_refusals(abi):
    from differentiable_rasterizer_gb300 import layers
    x, w = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros((4, 8), dtype=torch.bfloat16)
    for call in (lambda: layers.linear(x, w), lambda: layers.glu(x, w, w), lambda: layers.rms_norm(x, w[0]),
                 lambda: layers.quantize_rows(x), lambda: layers.linear_backward(x, x, w),
                 lambda: layers.glu_backward(x, x, w, w), lambda: layers.rms_norm_backward(x, x, w[0], w[0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="expected a tensor, got NoneType"):
        layers.linear(None, w)
    with pytest.raises(ValueError, match="expected a tensor, got list"):
        layers.rms_norm([1.0], w[0])
    with pytest.raises(ValueError, match="not one of"):
        layers.linear(x, w, act="tanh")


def test_missing_module_raises(abi, tmp_path, monkeypatch):
    from differentiable_rasterizer_gb300 import layers
    monkeypatch.setattr(abi, "LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="layer module missing"):
        layers._Native().linear
