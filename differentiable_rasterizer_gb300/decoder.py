"""A network that decodes per-Gaussian features into a scene's parameters, trained
through the rasterizer with the layers of ``layers``.

    n  = norm(x)                                  rms_norm
    h  = silu(n Wg^T) * (n Wu^T)                  glu
    s  = x + h Wd^T,  y = norm(s)                 linear, rms_norm with the residual
    params = y W^T + b + base                     linear, into the parameter buffer

The last product writes ``GaussianTrainer.params`` itself (fp32, one 16- or 64-float
block a Gaussian) and its backward starts from ``GaussianTrainer.grads``.  Features,
activations and weights are bfloat16; the optimizer may keep fp32 masters
(``GaussianDecoder.masters``).  ``decode_e4m3`` serves the same network with the gate
and up projections in 8 bits.

    python -m differentiable_rasterizer_gb300.decoder --steps 60

trains a decoder on the tiny scene's render and prints the loss.
"""
from __future__ import annotations

import argparse

import torch

from . import abi, layers


class GaussianDecoder:
    """features: columns of x; hidden: columns of h; base: [n, stride] parameter blocks that
    the decoded values are added to (a trainer's initial params), or None."""

    WEIGHTS = ("norm1", "w_gate", "w_up", "w_down", "norm2", "w_head", "b_head")

    def __init__(self, features: int, hidden: int, sh_degree: int, base: torch.Tensor | None = None, seed: int = 0,
                 device="cuda"):
        self.P = abi.gs_param_rows(sh_degree)
        self.base = None if base is None else base[:, :self.P]
        g = torch.Generator().manual_seed(seed)

        def normal(rows, cols, std):
            return torch.randn((rows, cols), generator=g) * std

        self.masters = {
            "norm1": torch.ones(features), "norm2": torch.ones(features),
            "w_gate": normal(hidden, features, features ** -0.5), "w_up": normal(hidden, features, features ** -0.5),
            "w_down": normal(features, hidden, hidden ** -0.5),
            "w_head": normal(self.P, features, 0.02 * features ** -0.5), "b_head": torch.zeros(self.P)}
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
        n = layers.rms_norm(x, w["norm1"], need_backward=True)
        u = layers.glu(n.y, w["w_gate"], w["w_up"], need_backward=True)
        d = layers.linear(u.h, w["w_down"]).y
        y = layers.rms_norm(d, w["norm2"], residual=x, need_backward=True)
        layers.linear(y.y, w["w_head"], w["b_head"], residual=self.base, out=params[:, :self.P])
        return x, n, u, y

    def decode_e4m3(self, x: torch.Tensor, params: torch.Tensor):
        """decode without gradients, gate and up projections in 8 bits."""
        w = self.w
        if self._quantised is None:
            self._quantised = layers.quantize_rows(w["w_gate"]), layers.quantize_rows(w["w_up"])
        (wg, gs), (wu, us) = self._quantised
        n = layers.rms_norm(x, w["norm1"], out_dtype=torch.float8_e4m3fn)
        h = layers.glu(n.y, wg, wu, x_scale=n.scale, gate_scale=gs, up_scale=us).h
        d = layers.linear(h, w["w_down"]).y
        y = layers.rms_norm(d, w["norm2"], residual=x)
        layers.linear(y.y, w["w_head"], w["b_head"], residual=self.base, out=params[:, :self.P])

    # ------------------------------------------------------------------ backward
    def backward(self, dparams: torch.Tensor, saved) -> dict:
        """Gradients of the weights, and of x under "x", from dparams [n, stride] fp32 (rows of
        Gaussians without gradient zero)."""
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
    a = ap.parse_args(argv)
    sc = scenes.make_scene(a.scene)
    trainer = pipeline.GaussianTrainer(sc.params, sc.sh_degree, sc.cameras, sc.opts, sc.lr)
    target = trainer.render().clone()
    base = trainer.params.clone()
    base[:, 11:trainer.P] = 0   # the colours are what the network has to find
    dec = GaussianDecoder(a.features, a.hidden, sc.sh_degree, base)
    x = torch.randn((trainer.n, a.features), generator=torch.Generator().manual_seed(1)).cuda().requires_grad_(False)
    masters = {k: v.requires_grad_(True) for k, v in dict(dec.masters, x=x).items()}
    opt = torch.optim.Adam(masters.values(), lr=a.lr)
    losses = []
    for step in range(a.steps):
        g = dec.grads(trainer, masters["x"].detach().to(torch.bfloat16), target)
        for k, v in masters.items():
            v.grad = g[k].float()
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
