"""A network that decodes per-Gaussian features into a scene's parameters, trained
through the rasterizer with the layers of ``layers``.

    n  = norm(x)                                  rms_norm
    h  = silu(n Wg^T) * (n Wu^T)                  glu
    s  = x + h Wd^T,  y = norm(s)                 linear, rms_norm with the residual
    params = y W^T + b + base                     linear, into the parameter buffer

With ``heads``, Gaussians also look at the others of their group (consecutive rows) before
that, and both blocks' outputs are normed, gated and added to a scaled residual stream:

    q, k, v = norm(x) Wqkv^T                      rms_norm, linear
    a  = attention(q, k, v) Wo^T                  attention over the groups, linear
    s1 = scale x + gate norm(a),  n = norm(s1)    block_norm
    h  = silu(n Wg^T) * (n Wu^T)                  glu
    s2 = scale s1 + gate norm(h Wd^T), y = norm(s2)   linear, block_norm
    params = y W^T + b + base                     linear

The last product writes ``GaussianTrainer.params`` itself (fp32, one 16- or 64-float
block a Gaussian) and its backward starts from ``GaussianTrainer.grads``.  Features,
activations and weights are bfloat16; the optimizer may keep fp32 masters
(``GaussianDecoder.masters``).  ``decode_e4m3`` serves the same network with the gate
and up projections in 8 bits.

    python -m differentiable_rasterizer_gb300.decoder --steps 60

trains a decoder on the tiny scene's render and prints the loss; --heads 4 one with
attention.  Gradients are clipped to a largest norm over all weights (--clip, clip_norm).
"""
from __future__ import annotations

import argparse

import torch

from . import abi, layers


class GaussianDecoder:
    """features: columns of x; hidden: columns of h; base: [n, stride] parameter blocks that
    the decoded values are added to (a trainer's initial params), or None.

    heads: query heads of an attention block in front (0: none), kv_heads key heads (default
    as many), of head_dim columns (default features / heads); groups: lengths of the runs of
    rows that attend to each other (default: all rows one); residual_scale: of both blocks."""

    WEIGHTS = ("norm1", "w_gate", "w_up", "w_down", "norm2", "w_head", "b_head")
    ATTENTION_WEIGHTS = ("norm0", "w_qkv", "w_out", "post1", "gate1", "post2", "gate2")

    def __init__(self, features: int, hidden: int, sh_degree: int, base: torch.Tensor | None = None, seed: int = 0,
                 device="cuda", heads: int = 0, kv_heads: int | None = None, head_dim: int | None = None, groups=None,
                 residual_scale: float = 1.0):
        self.P = abi.gs_param_rows(sh_degree)
        self.heads, self.scale = heads, residual_scale
        self.base = None if base is None else base[:, :self.P]
        g = torch.Generator().manual_seed(seed)

        def normal(rows, cols, std):
            return torch.randn((rows, cols), generator=g) * std

        self.masters = {
            "norm1": torch.ones(features), "norm2": torch.ones(features),
            "w_gate": normal(hidden, features, features ** -0.5), "w_up": normal(hidden, features, features ** -0.5),
            "w_down": normal(features, hidden, hidden ** -0.5),
            "w_head": normal(self.P, features, 0.02 * features ** -0.5), "b_head": torch.zeros(self.P)}
        if heads:
            self.kv_heads, self.head_dim = kv_heads or heads, head_dim or max(1, features // heads)
            width = self.head_dim * (heads + 2 * self.kv_heads)
            self.masters.update(
                norm0=torch.ones(features), w_qkv=normal(width, features, features ** -0.5),
                w_out=normal(features, heads * self.head_dim, (heads * self.head_dim) ** -0.5),
                post1=torch.ones(features), gate1=torch.full((features,), 0.1),
                post2=torch.ones(features), gate2=torch.full((features,), 0.1))
            self.starts = None
            if groups is not None:
                self.starts = torch.tensor([0, *groups]).cumsum(0).to(device=device, dtype=torch.int32)
        self.masters = {k: v.to(device) for k, v in self.masters.items()}
        self.refresh()

    def refresh(self):
        """bfloat16 weights from the fp32 masters (after an optimizer step)."""
        self.w = {k: v.detach().to(torch.bfloat16) if k != "b_head" else v.detach() for k, v in self.masters.items()}
        self._quantised = None

    # ------------------------------------------------------------------ forward
    def decode(self, x: torch.Tensor, params: torch.Tensor):
        """Writes params[:, :P] ([n, stride] fp32 blocks) from x [n, features] bfloat16; returns
        what backward takes."""
        w = self.w
        if self.heads:
            n0, qkv, a, p, b1 = self._attend(x, need_backward=True)
            u = layers.glu(b1.y, w["w_gate"], w["w_up"], need_backward=True)
            d = layers.linear(u.h, w["w_down"]).y
            b2 = layers.block_norm(d, b1.s, w["norm2"], post_weight=w["post2"], gate=w["gate2"], scale=self.scale,
                                   need_backward=True)
            layers.linear(b2.y, w["w_head"], w["b_head"], residual=self.base, out=params[:, :self.P])
            return x, n0, qkv, a, p, b1, u, d, b2
        n = layers.rms_norm(x, w["norm1"], need_backward=True)
        u = layers.glu(n.y, w["w_gate"], w["w_up"], need_backward=True)
        d = layers.linear(u.h, w["w_down"]).y
        y = layers.rms_norm(d, w["norm2"], residual=x, need_backward=True)
        layers.linear(y.y, w["w_head"], w["b_head"], residual=self.base, out=params[:, :self.P])
        return x, n, u, y

    def _heads(self, qkv):
        """q, k and v of the joint projection [n, columns], as [n, heads, head_dim] views."""
        h, k, d = self.heads, self.kv_heads, self.head_dim
        return qkv[:, :h * d].unflatten(1, (h, d)), *(qkv[:, (h + i * k) * d:(h + i * k + k) * d].unflatten(1, (k, d))
                                                     for i in (0, 1))

    def _attend(self, x, need_backward=False, out_dtype=None):
        w = self.w
        n0 = layers.rms_norm(x, w["norm0"], need_backward=need_backward)
        qkv = layers.linear(n0.y, w["w_qkv"]).y
        a = layers.attention(*self._heads(qkv), q_starts=self.starts, need_backward=need_backward)
        p = layers.linear(a.o.flatten(1), w["w_out"]).y
        return n0, qkv, a, p, layers.block_norm(p, x, w["norm1"], post_weight=w["post1"], gate=w["gate1"], scale=self.scale,
                                                out_dtype=out_dtype, need_backward=need_backward)

    def decode_e4m3(self, x: torch.Tensor, params: torch.Tensor):
        """decode without gradients, gate and up projections in 8 bits."""
        w = self.w
        if self._quantised is None:
            self._quantised = layers.quantize_rows(w["w_gate"]), layers.quantize_rows(w["w_up"])
        (wg, gs), (wu, us) = self._quantised
        if self.heads:
            b1 = self._attend(x, out_dtype=torch.float8_e4m3fn)[-1]
            h = layers.glu(b1.y, wg, wu, x_scale=b1.y_scale, gate_scale=gs, up_scale=us).h
            y = layers.block_norm(layers.linear(h, w["w_down"]).y, b1.s, w["norm2"], post_weight=w["post2"], gate=w["gate2"],
                                  scale=self.scale)
            layers.linear(y.y, w["w_head"], w["b_head"], residual=self.base, out=params[:, :self.P])
            return
        n = layers.rms_norm(x, w["norm1"], out_dtype=torch.float8_e4m3fn)
        h = layers.glu(n.y, wg, wu, x_scale=n.scale, gate_scale=gs, up_scale=us).h
        d = layers.linear(h, w["w_down"]).y
        y = layers.rms_norm(d, w["norm2"], residual=x)
        layers.linear(y.y, w["w_head"], w["b_head"], residual=self.base, out=params[:, :self.P])

    # ------------------------------------------------------------------ backward
    def backward(self, dparams: torch.Tensor, saved) -> dict:
        """Gradients of the weights, and of x under "x", from dparams [n, stride] fp32 (rows of
        Gaussians without gradient zero)."""
        if self.heads:
            return self._backward_attention(dparams, saved)
        x, n, u, y = saved
        w = self.w
        head = layers.linear_backward(dparams[:, :self.P], y.y, w["w_head"], bias=True, dw_dtype=torch.float32,
                                      db_dtype=torch.float32)
        ds, dnorm2 = layers.rms_norm_backward(head.dx, y.s, w["norm2"], y.rstd)
        down = layers.linear_backward(ds, u.h, w["w_down"], dw_dtype=torch.float32)
        gated = layers.glu_backward(down.dx, n.y, w["w_gate"], w["w_up"], u.g, u.u, dw_dtype=torch.float32)
        dx, dnorm1 = layers.rms_norm_backward(gated.dx, n.s, w["norm1"], n.rstd, ds=ds)
        return dict(x=dx, norm1=dnorm1, w_gate=gated.dw_gate, w_up=gated.dw_up, w_down=down.dw, norm2=dnorm2,
                    w_head=head.dw, b_head=head.db)

    def _backward_attention(self, dparams, saved) -> dict:
        x, n0, qkv, a, p, b1, u, d, b2 = saved
        w, f32 = self.w, dict(dw_dtype=torch.float32)
        head = layers.linear_backward(dparams[:, :self.P], b2.y, w["w_head"], bias=True, db_dtype=torch.float32, **f32)
        g2 = layers.block_norm_backward(head.dx, d, b2.s, w["norm2"], b2.rstd, post_weight=w["post2"],
                                        rstd_post=b2.rstd_post, gate=w["gate2"], scale=self.scale)
        down = layers.linear_backward(g2.dh, u.h, w["w_down"], **f32)
        gated = layers.glu_backward(down.dx, b1.y, w["w_gate"], w["w_up"], u.g, u.u, **f32)
        g1 = layers.block_norm_backward(gated.dx, p, b1.s, w["norm1"], b1.rstd, post_weight=w["post1"],
                                        rstd_post=b1.rstd_post, gate=w["gate1"], scale=self.scale, ds=g2.dx)
        out = layers.linear_backward(g1.dh, a.o.flatten(1), w["w_out"], **f32)
        dqkv = torch.zeros_like(qkv) if self.starts is not None else torch.empty_like(qkv)   # rows of no group
        layers.attention_backward(out.dx.unflatten(1, (self.heads, self.head_dim)), *self._heads(qkv), a.o, a.lse,
                                  q_starts=self.starts, out=self._heads(dqkv))
        proj = layers.linear_backward(dqkv, n0.y, w["w_qkv"], **f32)
        dx, dnorm0 = layers.rms_norm_backward(proj.dx, n0.s, w["norm0"], n0.rstd, ds=g1.dx)
        return dict(x=dx, norm0=dnorm0, w_qkv=proj.dw, w_out=out.dw, post1=g1.dpost_weight, gate1=g1.dgate, norm1=g1.dweight,
                    w_gate=gated.dw_gate, w_up=gated.dw_up, w_down=down.dw, post2=g2.dpost_weight, gate2=g2.dgate,
                    norm2=g2.dweight, w_head=head.dw, b_head=head.db)

    def grads(self, trainer, x: torch.Tensor, target: torch.Tensor) -> dict:
        """Decode into the trainer's parameters, render, loss and backward to the weights and x;
        the loss is in trainer.loss."""
        saved = self.decode(x, trainer.params)
        trainer.project()
        trainer.bin_sort()
        trainer.raster(target, count_evals=False)
        trainer.grads.zero_()   # the compaction writes the touched Gaussians' rows only
        trainer.compact()
        return self.backward(trainer.grads, saved)


def main(argv=None):
    from . import pipeline, scenes
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--scene", default="tiny", choices=["tiny", "small", "medium"])
    ap.add_argument("--features", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=128)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--lr", type=float, default=2e-3)
    ap.add_argument("--heads", type=int, default=0, help="of an attention block (0: none)")
    ap.add_argument("--kv-heads", type=int, default=None)
    ap.add_argument("--group", type=int, default=256, help="Gaussians that attend to each other")
    ap.add_argument("--clip", type=float, default=None, help="largest norm over all weights' gradients")
    a = ap.parse_args(argv)
    sc = scenes.make_scene(a.scene)
    trainer = pipeline.GaussianTrainer(sc.params, sc.sh_degree, sc.cameras, sc.opts, sc.lr)
    target = trainer.render().clone()
    base = trainer.params.clone()
    base[:, 11:trainer.P] = 0   # the colours are what the network has to find
    groups = [min(a.group, trainer.n - i) for i in range(0, trainer.n, a.group)]
    dec = GaussianDecoder(a.features, a.hidden, sc.sh_degree, base, heads=a.heads, kv_heads=a.kv_heads, groups=groups)
    x = torch.randn((trainer.n, a.features), generator=torch.Generator().manual_seed(1)).cuda().requires_grad_(False)
    masters = {k: v.requires_grad_(True) for k, v in dict(dec.masters, x=x).items()}
    opt = torch.optim.Adam(masters.values(), lr=a.lr)
    losses = []
    for step in range(a.steps):
        g = dec.grads(trainer, masters["x"].detach().to(torch.bfloat16), target)
        if a.clip is None:
            for k, v in masters.items():
                v.grad = g[k].float()
        else:   # clipped and converted to fp32 in one
            for v in masters.values():
                v.grad = torch.empty_like(v) if v.grad is None else v.grad
            layers.clip_norm([g[k].contiguous() for k in masters], a.clip, out=[v.grad for v in masters.values()])
        opt.step()
        dec.refresh()
        losses.append(trainer.loss.sum().clone())
    losses = torch.stack(losses).cpu().tolist()
    for step in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {step:4d}  L1 {losses[step]:.5f}")
    print(f"step {a.steps - 1:4d}  L1 {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    main()
