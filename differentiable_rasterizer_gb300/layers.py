"""Decoder layers on torch tensors: the norm, the matrix product with its epilogue, the
gated feed-forward and their gradients, through the C ABI (``gs_rms_norm``,
``gs_linear``, ``gs_glu`` ... in ``include/gs.h``, which states the formulas).

    o = rms_norm(x, weight, residual=r)                      # o.y, o.s = x + r
    q = rms_norm(x, weight, residual=r, out_dtype=torch.float8_e4m3fn)   # q.y, q.scale
    y = linear(x, w, bias, act="gelu", residual=r).y         # act(x w^T + b) + r
    h = glu(x, w_gate, w_up, act="silu").h                   # act(x Wg^T) * (x Wu^T)
    y = linear(h, w_down, residual=r).y                      # ... and its down projection

Tensors are CUDA tensors whose last dimension is contiguous; leading dimensions are
rows and must merge into one stride (a slice of wider rows is fine).  Rows whose base
and pitch are multiples of 16 bytes need no copy.  Work is queued on the current
stream of the tensors' device, and outputs and scratch are allocated there, so a
tensor made on another stream needs the usual wait before the call.  Nothing is kept
between calls.  Arguments that the call cannot take raise ValueError (here) or
``abi.GsError`` (the library's status); there is no fallback.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import abi

_TYPES = {torch.float32: abi.GS_F32, torch.bfloat16: abi.GS_BF16, torch.float16: abi.GS_F16,
          torch.float8_e4m3fn: abi.GS_E4M3}
_ACTS = {None: abi.GS_ACT_NONE, "none": abi.GS_ACT_NONE, "relu": abi.GS_ACT_RELU, "silu": abi.GS_ACT_SILU,
         "gelu": abi.GS_ACT_GELU}
_HALF = (torch.bfloat16, torch.float16)
_FLOAT = (torch.float32, torch.bfloat16, torch.float16)


class NormOut(NamedTuple):
    y: torch.Tensor
    scale: Optional[torch.Tensor]   # [rows], 8-bit y only
    s: torch.Tensor                 # x + residual (x itself without one)
    rstd: Optional[torch.Tensor]    # [rows], for the gradients


class LinearOut(NamedTuple):
    y: torch.Tensor
    z: Optional[torch.Tensor]       # pre-activations, for the gradients


class GluOut(NamedTuple):
    h: torch.Tensor
    g: Optional[torch.Tensor]       # projections, for the gradients
    u: Optional[torch.Tensor]


class LinearGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]
    db: Optional[torch.Tensor]


class GluGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw_gate: Optional[torch.Tensor]
    dw_up: Optional[torch.Tensor]


# ------------------------------------------------------------------ argument checks
def _bad(what):
    raise ValueError(what)


def _wrong(t, name, dtypes, dev):
    """Raises for a tensor of another type or device (the slow path of the checks)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        _bad(f"{name}: expected a tensor of {[str(d) for d in dtypes]}, got {getattr(t, 'dtype', type(t))}")
    _bad(f"{name}: on {t.device}, expected cuda:{dev}")


def _matrix(t, name, dtypes, dev, cols=None, rows=None):
    """(pointer, leading dimension, rows, columns) of a tensor seen as rows."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.get_device() != dev:
        _wrong(t, name, dtypes, dev)
    shape = t.shape
    if len(shape) != 2:
        if not shape:
            _bad(f"{name}: needs at least one dimension")
        try:
            t = t.view(-1, shape[-1]) if shape[-1] else t.reshape(0, 0)
        except RuntimeError:
            _bad(f"{name}: leading dimensions do not merge into one stride {tuple(t.shape)} {t.stride()}")
        shape = t.shape
    n, c = shape
    if cols is not None and c != cols:
        _bad(f"{name}: {c} columns, expected {cols}")
    if rows is not None and n != rows:
        _bad(f"{name}: {n} rows, expected {rows}")
    ld, unit = t.stride()
    if unit != 1 and c > 1:
        _bad(f"{name}: the last dimension is not contiguous {t.stride()}")
    if n <= 1:   # the pitch of a single row is never used: one that keeps the row aligned
        ld = (c + 15) & ~15
    elif ld < c:
        _bad(f"{name}: rows overlap (stride {ld}, {c} columns)")
    return t.data_ptr(), ld, n, c


def _vector(t, name, dtypes, dev, size):
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.get_device() != dev:
        _wrong(t, name, dtypes, dev)
    if t.numel() != size or (size > 1 and not t.is_contiguous()):
        _bad(f"{name}: expected {size} contiguous values, got {tuple(t.shape)} {t.stride()}")
    return t.data_ptr()


def _device(t, name):
    """Index of the CUDA device that a call's first tensor is on."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad(f"{name}: expected a CUDA tensor, got {t.device if isinstance(t, torch.Tensor) else type(t)}")
    return t.get_device()


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        _bad(f"act: {act!r} is not one of {[a for a in _ACTS if a]}")
    return code


_PER_16 = {torch.float32: 4, torch.bfloat16: 8, torch.float16: 8, torch.float8_e4m3fn: 16}


def _output(like, lead, cols, dtype):
    """An uninitialised [*lead, cols] on like's device whose rows are 16-byte aligned, its pointer
    and leading dimension."""
    pad = -cols % _PER_16[dtype]
    t = torch.empty(lead + (cols + pad,), dtype=dtype, device=like.device)
    p = t.data_ptr()
    return (t[..., :cols] if pad else t), p, cols + pad


_current_device = torch._C._cuda_getDevice              # torch.cuda.current_device without its checks
_stream = torch._C._cuda_getCurrentRawStream            # torch.cuda.current_stream(dev).cuda_stream


def _run(f, dev, *args):
    """f(*args, stream) with the tensors' device current."""
    if dev == _current_device():
        f(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            f(*args, _stream(dev))


def _call(name, args, like, dev, try_first=False):
    """A layer call with the scratch that it asks for, on the current stream; try_first: it
    mostly needs none."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call(name, args, like, dev, try_first)
    stream = _stream(dev)
    if try_first and abi.layer_call(name, args, stream):
        return
    n = abi.layer_ws_bytes(name, args)
    if n:
        ws = torch.empty(n, dtype=torch.uint8, device=like.device)
        abi.layer_run(name, args, ws.data_ptr(), n, stream)
    else:
        abi.layer_run(name, args, None, None, stream)


# ------------------------------------------------------------------ norm
def rms_norm(x, weight, *, residual=None, eps=1e-6, out_dtype=None, need_backward=False) -> NormOut:
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last dimension.

    x, residual: float32, bfloat16 or float16 (one type); weight: any of them.  y has
    out_dtype (default: x's); float8_e4m3fn gives 8-bit rows with a float32 scale each,
    y * scale being the norm.  s is the sum rounded to x's type."""
    dev = _device(x, "x")
    px, ldx, rows, cols = _matrix(x, "x", _FLOAT, dev)
    pr = ldr = ps = lds = pscale = prstd = 0
    pw = _vector(weight, "weight", _FLOAT, dev, cols)
    if not pw:
        _bad("weight: required")
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _TYPES:
        _bad(f"out_dtype: {out_dtype}")
    lead = x.shape[:-1]
    s = x
    if residual is not None:
        pr, ldr, _, _ = _matrix(residual, "residual", (x.dtype,), dev, cols, rows)
        s, ps, lds = _output(x, lead, cols, x.dtype)
    y, py, ldy = _output(x, lead, cols, out_dtype)
    scale = rstd = None
    if out_dtype == torch.float8_e4m3fn:
        scale = torch.empty(lead, dtype=torch.float32, device=x.device)
        pscale = scale.data_ptr()
    if need_backward:
        rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
        prstd = rstd.data_ptr()
    if rows:
        _run(abi.gs_rms_norm, dev, rows, cols, px, ldx, pr, ldr, pw, py, ldy, pscale, ps, lds, prstd, eps,
             _TYPES[x.dtype], _TYPES[weight.dtype], _TYPES[out_dtype])
    return NormOut(y, scale, s, rstd)


def rms_norm_backward(dy, s, weight, rstd, *, ds=None):
    """(dx, dweight) of rms_norm from the gradient of y and (ds, optional) of s.

    dx, of s's type, is the gradient of x and of residual alike; dweight has weight's type."""
    dev = _device(s, "s")
    ps, lds, rows, cols = _matrix(s, "s", _FLOAT, dev)
    pdy, lddy, _, _ = _matrix(dy, "dy", _FLOAT, dev, cols, rows)
    pw = _vector(weight, "weight", _FLOAT, dev, cols)
    prstd = _vector(rstd, "rstd", (torch.float32,), dev, rows)
    if not pw or (not prstd and rows):
        _bad("weight and rstd (rms_norm's with need_backward) are required")
    pds = ldds = 0
    if ds is not None:
        pds, ldds, _, _ = _matrix(ds, "ds", (s.dtype,), dev, cols, rows)
    dx, pdx, lddx = _output(s, s.shape[:-1], cols, s.dtype)
    dw = torch.empty(weight.shape, dtype=weight.dtype, device=s.device)
    _call("gs_rms_norm_bwd", abi.rms_norm_bwd_args(rows, cols, pdy, lddy, ps, lds, pw, prstd, pds, ldds, pdx, lddx,
                                                   dw.data_ptr(), _TYPES[s.dtype], _TYPES[dy.dtype],
                                                   _TYPES[weight.dtype]), s, dev)
    return dx, dw


def quantize_rows(x):
    """(q, scale): rows of x in float8_e4m3fn, the largest magnitude of each at 448, and
    the float32 scale that restores it: x ~ q * scale[..., None]."""
    dev = _device(x, "x")
    px, ldx, rows, cols = _matrix(x, "x", _FLOAT, dev)
    q, pq, ldq = _output(x, x.shape[:-1], cols, torch.float8_e4m3fn)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    if rows:
        _run(abi.gs_quantize_rows, dev, rows, cols, px, ldx, pq, ldq, scale.data_ptr(), _TYPES[x.dtype])
    return q, scale


# ------------------------------------------------------------------ linear
def linear(x, w, bias=None, *, x_scale=None, w_scale=None, act=None, residual=None, out=None, out_dtype=None,
           need_backward=False) -> LinearOut:
    """y = act((x w^T) * x_scale * w_scale + bias) + residual.

    x [..., in], w [out, in]: bfloat16, float16, or float8_e4m3fn with float32 scales per
    row of x and per row of w.  y, residual: out_dtype (default: out's, residual's, x's,
    or bfloat16 for 8-bit x); `out` may be given, with rows of any pitch (a column range
    of the parameter buffer, or residual itself).  need_backward also returns the
    pre-activations z in x's type where an activation needs them."""
    dev = _device(x, "x")
    px, ldx, rows, k = _matrix(x, "x", (*_HALF, torch.float8_e4m3fn), dev)
    pw, ldw, n, _ = _matrix(w, "w", (x.dtype,), dev, k)
    code = _act(act)
    pb = _vector(bias, "bias", _FLOAT, dev, n)
    pxs = _vector(x_scale, "x_scale", (torch.float32,), dev, rows)
    pws = _vector(w_scale, "w_scale", (torch.float32,), dev, n)
    if out_dtype is None:
        out_dtype = (out.dtype if out is not None else residual.dtype if residual is not None else
                     x.dtype if x.dtype in _HALF else torch.bfloat16)
    if out_dtype not in _FLOAT:
        _bad(f"out_dtype: {out_dtype}")
    lead = x.shape[:-1]
    pr = ldr = pz = ldz = 0
    if residual is not None:
        pr, ldr, _, _ = _matrix(residual, "residual", (out_dtype,), dev, n, rows)
    if out is None:
        y, py, ldy = _output(x, lead, n, out_dtype)
    else:
        y = out
        py, ldy, _, _ = _matrix(y, "out", (out_dtype,), dev, n, rows)
    z = None
    if need_backward and code != abi.GS_ACT_NONE:
        if x.dtype not in _HALF:
            _bad("need_backward: 8-bit operands have no gradients")
        z, pz, ldz = _output(x, lead, n, x.dtype)
    _call("gs_linear", abi.linear_args(rows, k, n, px, ldx, pw, ldw, pxs, pws, pb, pr, ldr, py, ldy, pz, ldz,
                                       _TYPES[x.dtype], _TYPES[bias.dtype] if bias is not None else 0,
                                       _TYPES[out_dtype], code), x, dev, True)
    return LinearOut(y, z)


def linear_backward(dy, x, w, *, z=None, act=None, bias=False, need_dx=True, need_dw=True, dw_dtype=None,
                    db_dtype=None) -> LinearGrads:
    """Gradients of linear from dy (float32, bfloat16 or float16; the residual's gradient
    is dy itself).  z: linear's with need_backward, where act is one.  dx has x's type, dw
    dw_dtype (default x's; float32 also), db (with bias=True) db_dtype (default x's)."""
    dev = _device(x, "x")
    px, ldx, rows, k = _matrix(x, "x", _HALF, dev)
    pw, ldw, n, _ = _matrix(w, "w", (x.dtype,), dev, k)
    pdy, lddy, _, _ = _matrix(dy, "dy", _FLOAT, dev, n, rows)
    code = _act(act)
    pz = ldz = pdx = lddx = pdw = lddw = pdb = 0
    if code != abi.GS_ACT_NONE:
        if z is None:
            _bad("z: required with an activation")
        pz, ldz, _, _ = _matrix(z, "z", (x.dtype,), dev, n, rows)
    dw_dtype = x.dtype if dw_dtype is None else dw_dtype
    db_dtype = x.dtype if db_dtype is None else db_dtype
    if dw_dtype not in (x.dtype, torch.float32):
        _bad(f"dw_dtype: {dw_dtype}")
    if db_dtype not in _FLOAT:
        _bad(f"db_dtype: {db_dtype}")
    dx = dw = db = None
    if need_dx:
        dx, pdx, lddx = _output(x, x.shape[:-1], k, x.dtype)
    if need_dw:
        dw = torch.empty((n, k), dtype=dw_dtype, device=x.device)
        pdw, lddw = dw.data_ptr(), k
    if bias:
        db = torch.empty(n, dtype=db_dtype, device=x.device)
        pdb = db.data_ptr()
    _call("gs_linear_bwd", abi.linear_bwd_args(rows, k, n, pdy, lddy, px, ldx, pw, ldw, pz, ldz, pdx, lddx, pdw, lddw,
                                               pdb, _TYPES[x.dtype], _TYPES[dy.dtype], _TYPES[dw_dtype],
                                               _TYPES[db_dtype], code), x, dev)
    return LinearGrads(dx, dw, db)


# ------------------------------------------------------------------ gated feed-forward
# Up to this many input features glu's gradients compute the projections again rather than
# read them: two more products of that depth against 8 bytes a value written and read.
_AGAIN_FEATURES = 512


def glu(x, w_gate, w_up, *, x_scale=None, gate_scale=None, up_scale=None, act="silu", out_dtype=None,
        need_backward=False, save=None) -> GluOut:
    """h = act(x Wg^T) * (x Wu^T), both projections in one kernel.

    x [..., in], w_gate, w_up [hidden, in]: bfloat16, float16, or float8_e4m3fn with
    float32 scales per row.  h: x's type, or out_dtype (16 bits, default bfloat16) for
    8-bit x.  need_backward also returns the projections g and u where glu_backward is
    better off reading them (wide inputs; save=True or False decides instead), else None."""
    dev = _device(x, "x")
    px, ldx, rows, k = _matrix(x, "x", (*_HALF, torch.float8_e4m3fn), dev)
    pg_, ldwg, f, _ = _matrix(w_gate, "w_gate", (x.dtype,), dev, k)
    pu_, ldwu, _, _ = _matrix(w_up, "w_up", (x.dtype,), dev, k, f)
    pxs = _vector(x_scale, "x_scale", (torch.float32,), dev, rows)
    pgs = _vector(gate_scale, "gate_scale", (torch.float32,), dev, f)
    pus = _vector(up_scale, "up_scale", (torch.float32,), dev, f)
    if out_dtype is None:
        out_dtype = x.dtype if x.dtype in _HALF else torch.bfloat16
    if out_dtype not in _HALF:
        _bad(f"out_dtype: {out_dtype}")
    lead = x.shape[:-1]
    h, ph, ldh = _output(x, lead, f, out_dtype)
    g = u = None
    pg = ldg = pu = ldu = 0
    if need_backward:
        if x.dtype not in _HALF:
            _bad("need_backward: 8-bit operands have no gradients")
        if k > _AGAIN_FEATURES if save is None else save:
            g, pg, ldg = _output(x, lead, f, out_dtype)
            u, pu, ldu = _output(x, lead, f, out_dtype)
    _call("gs_glu", abi.glu_args(rows, k, f, px, ldx, pg_, ldwg, pu_, ldwu, pxs, pgs, pus, ph, ldh, pg, ldg, pu, ldu,
                                 _TYPES[x.dtype], _TYPES[out_dtype], _act(act)), x, dev, True)
    return GluOut(h, g, u)


def glu_backward(dh, x, w_gate, w_up, g=None, u=None, *, act="silu", need_dx=True, need_dw=True,
                 dw_dtype=None) -> GluGrads:
    """Gradients of glu from dh; g, u: glu's with need_backward (None: computed again)."""
    dev = _device(x, "x")
    px, ldx, rows, k = _matrix(x, "x", _HALF, dev)
    pwg, ldwg, f, _ = _matrix(w_gate, "w_gate", (x.dtype,), dev, k)
    pwu, ldwu, _, _ = _matrix(w_up, "w_up", (x.dtype,), dev, k, f)
    pdh, lddh, _, _ = _matrix(dh, "dh", (x.dtype,), dev, f, rows)
    pg = ldg = pu = ldu = 0
    if g is not None or u is not None:
        pg, ldg, _, _ = _matrix(g, "g", (x.dtype,), dev, f, rows)
        pu, ldu, _, _ = _matrix(u, "u", (x.dtype,), dev, f, rows)
    dw_dtype = x.dtype if dw_dtype is None else dw_dtype
    if dw_dtype not in (x.dtype, torch.float32):
        _bad(f"dw_dtype: {dw_dtype}")
    dx = dwg = dwu = None
    pdx = lddx = pdwg = lddwg = pdwu = lddwu = 0
    if need_dx:
        dx, pdx, lddx = _output(x, x.shape[:-1], k, x.dtype)
    if need_dw:
        dwg, dwu = (torch.empty((f, k), dtype=dw_dtype, device=x.device) for _ in range(2))
        pdwg, lddwg, pdwu, lddwu = dwg.data_ptr(), k, dwu.data_ptr(), k
    _call("gs_glu_bwd", abi.glu_bwd_args(rows, k, f, pdh, lddh, px, ldx, pwg, ldwg, pwu, ldwu, pg, ldg, pu, ldu, pdx,
                                         lddx, pdwg, lddwg, pdwu, lddwu, _TYPES[x.dtype], _TYPES[dw_dtype], _act(act)),
          x, dev)
    return GluGrads(dx, dwg, dwu)
