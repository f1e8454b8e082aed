"""Decoder layers on torch tensors: the norm, the matrix product with its epilogue, the
gated feed-forward and their gradients, through the C ABI (``gs_rms_norm``,
``gs_linear``, ``gs_glu``, ``gs_attention`` ... in ``include/gs.h``, which states the formulas).

    o = rms_norm(x, weight, residual=r)                      # o.y, o.s = x + r
    q = rms_norm(x, weight, residual=r, out_dtype=torch.float8_e4m3fn)   # q.y, q.scale
    y = linear(x, w, bias, act="gelu", residual=r).y         # act(x w^T + b) + r
    h = glu(x, w_gate, w_up, act="silu").h                   # act(x Wg^T) * (x Wu^T)
    y = linear(h, w_down, residual=r).y                      # ... and its down projection
    a = attention(q, k, v, q_starts=starts, causal=True).o   # over packed sequences
    b = block_norm(h, x, w, post_weight=p, gate=g, scale=c)  # b.s = c x + g norm(h), b.y = norm(b.s)
    n = clip_norm(grads, 1.0, out=grads_fp32)                # the norm over all, and all scaled to 1

Tensors are CUDA tensors whose last dimension is contiguous; leading dimensions are
rows and must merge into one stride (a slice of wider rows is fine).  Rows whose base
and pitch are multiples of 16 bytes need no copy; outputs that the functions allocate
have such rows (for other widths they are views of padded rows).  Work is queued on the
current stream of the tensors' device, and outputs and scratch are allocated there, so a
tensor made on another stream needs the usual wait before the call.  Nothing is kept
between calls.  Arguments that a call cannot take raise ValueError, or ``abi.GsError``
with the library's status; there is no fallback.

Kernels wait for their own copies and products within a bound of about two seconds; one that
runs out of it (a device fault, or a process stopped for that long) leaves its outputs
undefined, which ``abi.gs_wait_report()`` tells.

The layers are outside autograd: their gradients are the *_backward functions, called
explicitly.  A tensor that requires grad is refused while gradients are recorded (its
gradient would be lost without a word); pass ``t.detach()`` or call under
``torch.no_grad()``.

The checks, the allocations and the calls are native (``csrc/layers_torch.cpp``).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import abi

_ACTS = {None: abi.GS_ACT_NONE, "none": abi.GS_ACT_NONE, "relu": abi.GS_ACT_RELU, "silu": abi.GS_ACT_SILU,
         "gelu": abi.GS_ACT_GELU}


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


class AttentionOut(NamedTuple):
    o: torch.Tensor
    lse: Optional[torch.Tensor]     # [rows, heads], for the gradients


class AttentionGrads(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor


class BlockNormOut(NamedTuple):
    y: Optional[torch.Tensor]
    y_scale: Optional[torch.Tensor]    # [rows], 8-bit y only
    s: torch.Tensor
    rstd_post: Optional[torch.Tensor]  # [rows], both for the gradients
    rstd: Optional[torch.Tensor]


class BlockNormGrads(NamedTuple):
    dh: torch.Tensor
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


class LinearGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]
    db: Optional[torch.Tensor]


class GluGrads(NamedTuple):
    dx: Optional[torch.Tensor]
    dw_gate: Optional[torch.Tensor]
    dw_up: Optional[torch.Tensor]


class _Native:
    """The extension module, loaded and bound to the library that abi loads on first use."""

    def __getattr__(self, name):
        path = os.path.join(os.path.dirname(abi.LIB_PATH), "_layers_torch.so")
        if not os.path.exists(path):
            raise RuntimeError(f"layer module missing: {path}; build it with "
                               "`python -m differentiable_rasterizer_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_layers_torch", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_layers_torch", loader))
        loader.exec_module(module)
        L = abi.lib()
        module.bind(abi.GsError, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "gs_rms_norm", "gs_rms_norm_bwd", "gs_quantize_rows", "gs_linear", "gs_linear_bwd", "gs_glu", "gs_glu_bwd",
            "gs_attention", "gs_attention_bwd", "gs_block_norm", "gs_block_norm_bwd", "gs_clip_norm")))
        for f in ("rms_norm", "rms_norm_backward", "quantize_rows", "linear", "linear_backward", "glu", "glu_backward",
                  "attention", "attention_backward", "block_norm", "block_norm_backward", "clip_norm"):
            setattr(self, f, getattr(module, f))
        return self.__dict__[name]


_native = _Native()


def _act(act):
    code = _ACTS.get(act) if act is None or isinstance(act, str) else None
    if code is None:
        raise ValueError(f"act: {act!r} is not one of {[a for a in _ACTS if a]}")
    return code


# ------------------------------------------------------------------ norm
def rms_norm(x, weight, *, residual=None, eps=1e-6, out_dtype=None, need_backward=False) -> NormOut:
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last dimension.

    x, residual: float32, bfloat16 or float16 (one type); weight: any of them.  y has
    out_dtype (default: x's); float8_e4m3fn gives 8-bit rows with a float32 scale each,
    y * scale being the norm.  s is the sum rounded to x's type."""
    return NormOut(*_native.rms_norm(x, weight, residual, eps, out_dtype, need_backward))


def rms_norm_backward(dy, s, weight, rstd, *, ds=None):
    """(dx, dweight) of rms_norm from the gradient of y and (ds, optional) of s.

    dx, of s's type, is the gradient of x and of residual alike; dweight has weight's type."""
    return _native.rms_norm_backward(dy, s, weight, rstd, ds)


def quantize_rows(x):
    """(q, scale): rows of x in float8_e4m3fn, the largest magnitude of each at 448, and
    the float32 scale that restores it: x ~ q * scale[..., None]."""
    return _native.quantize_rows(x)


# ------------------------------------------------------------------ linear
def linear(x, w, bias=None, *, x_scale=None, w_scale=None, act=None, residual=None, out=None, out_dtype=None,
           need_backward=False) -> LinearOut:
    """y = act((x w^T) * x_scale * w_scale + bias) + residual.

    x [..., in], w [out, in]: bfloat16, float16, or float8_e4m3fn with float32 scales per
    row of x and per row of w.  y, residual: out_dtype (default: out's, residual's, x's,
    or bfloat16 for 8-bit x); `out` may be given, with rows of any pitch (a column range
    of the parameter buffer, or residual itself).  need_backward also returns the
    pre-activations z in x's type where an activation needs them."""
    return LinearOut(*_native.linear(x, w, bias, x_scale, w_scale, _act(act), residual, out, out_dtype, need_backward))


def linear_backward(dy, x, w, *, z=None, act=None, bias=False, need_dx=True, need_dw=True, dw_dtype=None,
                    db_dtype=None) -> LinearGrads:
    """Gradients of linear from dy (float32, bfloat16 or float16; the residual's gradient
    is dy itself).  z: linear's with need_backward, where act is one.  dx has x's type, dw
    dw_dtype (default x's; float32 also), db (with bias=True) db_dtype (default x's)."""
    return LinearGrads(*_native.linear_backward(dy, x, w, z, _act(act), bias, need_dx, need_dw, dw_dtype, db_dtype))


# ------------------------------------------------------------------ gated feed-forward
# Up to this many input features glu's gradients compute the projections again rather than
# read them: two more products of that depth against 8 bytes a value written and read.
# Layer and gradients, saved and again: 1,000,000 x 64 x 128 566 and 219 us (one pass),
# 100,000 x 256 x 1024 487 and 408, 32768 x 512 x 2048 426 and 403, 32768 x 640 x 2560 610 and
# 604, 32768 x 1024 x 4096 1161 and 1224.  (Of few rows they are close: 4096 x 512 x 2048 80
# and 84.)
_AGAIN_FEATURES = 512


def glu(x, w_gate, w_up, *, x_scale=None, gate_scale=None, up_scale=None, act="silu", out_dtype=None,
        need_backward=False, save=None) -> GluOut:
    """h = act(x Wg^T) * (x Wu^T), both projections in one kernel.

    x [..., in], w_gate, w_up [hidden, in]: bfloat16, float16, or float8_e4m3fn with
    float32 scales per row.  h: x's type, or out_dtype (16 bits, default bfloat16) for
    8-bit x.  need_backward also returns the projections g and u where glu_backward is
    better off reading them (wide inputs; save=True or False decides instead), else None."""
    if need_backward and isinstance(x, torch.Tensor) and x.dim() > 0:   # else it is refused below
        if x.dtype == torch.float8_e4m3fn:
            raise ValueError("need_backward: 8-bit operands have no gradients")
        save = x.shape[-1] > _AGAIN_FEATURES if save is None else save
    return GluOut(*_native.glu(x, w_gate, w_up, x_scale, gate_scale, up_scale, _act(act), out_dtype,
                               need_backward and save))


def glu_backward(dh, x, w_gate, w_up, g=None, u=None, *, act="silu", need_dx=True, need_dw=True,
                 dw_dtype=None) -> GluGrads:
    """Gradients of glu from dh; g, u: glu's with need_backward (None: computed again).  dx has
    x's type, dw_gate and dw_up dw_dtype (default x's; float32 also)."""
    return GluGrads(*_native.glu_backward(dh, x, w_gate, w_up, g, u, _act(act), need_dx, need_dw, dw_dtype))


# ------------------------------------------------------------------ attention
def attention(q, k, v, *, q_starts=None, k_starts=None, k_lengths=None, causal=False, scale=None, out=None,
              need_backward=False) -> AttentionOut:
    """o = softmax(scale q k^T) v, for each head and each of the sequences packed in the rows.

    q [rows, heads, dim], k, v [key rows, key heads, dim]: bfloat16 or float16, dim at most
    128; key heads divide heads (head h uses key head h // (heads // key heads)).  Rows and
    heads may have any strides (slices of one projection's output are fine).  scale: dim^-1/2.
    q_starts, k_starts: int32, sequence s has the rows starts[s] to starts[s + 1] (k_starts:
    default q_starts; without either, one sequence of all rows).  k_lengths: int32, how many
    of a sequence's keys are in use (a cache's slots), without gradients.  causal: the last
    query sees every key, the one before all but one, ...  A query that sees none gives 0.
    out: like q, rows of no sequence are left as they are; else o is allocated, those rows 0
    (lse's are 0 in either case).  It may be q, but shares no memory with k or v."""
    return AttentionOut(*_native.attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale, out, need_backward))


def attention_backward(do, q, k, v, o, lse, *, q_starts=None, k_starts=None, causal=False, scale=None,
                       out=None) -> AttentionGrads:
    """Gradients of attention from do, in q's type; o, lse: attention's with need_backward, the
    other arguments as they were given to it.  (o, already rounded, is checked but not computed
    with, and may be None: the rows' sums of do . o are taken from the terms again.)  out: (dq, dk, dv) to write to (column ranges of
    the projection's gradient, say), rows of no sequence are left as they are; else 0.  They share
    no memory with one another or with the inputs, but that dq may be q or do."""
    dq, dk, dv = (None, None, None) if out is None else out
    return AttentionGrads(*_native.attention_backward(do, q, k, v, o, lse, q_starts, k_starts, causal, scale, dq, dk, dv))


# ------------------------------------------------------------------ block norm
def block_norm(h, x, weight=None, *, post_weight=None, gate=None, scale=1.0, eps=1e-6, out_dtype=None,
               need_backward=False) -> BlockNormOut:
    """What lies between a block's output h, on the residual stream x, and the next block:

        a = h / sqrt(mean(h^2) + eps) * post_weight      (a = h without post_weight)
        s = scale * x + gate * a                          (gate 1 without one)
        y = s / sqrt(mean(s^2) + eps) * weight            (no y without weight)

    over the last dimension.  h, x: float32, bfloat16 or float16 (one type); the weights any
    of them; gate: [columns] of any of them, or like h, a gate a value.  s is rounded to h's
    type; y has out_dtype as in rms_norm (float8_e4m3fn: y * y_scale is the norm)."""
    return BlockNormOut(*_native.block_norm(h, x, weight, post_weight, gate, scale, eps, out_dtype, need_backward))


def block_norm_backward(dy, h, s, weight, rstd, *, post_weight=None, rstd_post=None, gate=None, scale=1.0,
                        ds=None) -> BlockNormGrads:
    """Gradients of block_norm from those of y (dy) and, optionally, of s (ds); rstd, rstd_post:
    block_norm's with need_backward.  Without weight: dy, s, weight and rstd are None, ds is
    required.  dh, dx have h's type, the others that of what they are the gradients of."""
    return BlockNormGrads(*_native.block_norm_backward(dy, h, s, weight, rstd, post_weight, rstd_post, gate, scale, ds))


# ------------------------------------------------------------------ clipping
def clip_norm(tensors, max_norm, *, out=None) -> torch.Tensor:
    """The norm over all values of the tensors (a list; contiguous float32, bfloat16 or float16,
    each of its own memory) as a float32 scalar on their device; the tensors times
    min(1, max_norm / norm) are written to out (a list of as many values each, of any of the
    types), or in place.  Nothing is scaled by a norm that is not finite: the caller sees it in
    the result and can skip the step."""
    return _native.clip_norm(tensors, max_norm, out)
