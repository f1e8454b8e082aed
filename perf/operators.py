"""Cases of the decoder-network operators: the network in front of the rasterizer that
turns per-Gaussian (or per-token) features into Gaussian parameters.

Three operators, each in its serving and its training form:

  norm    s = x + residual, y = s / rms(s) * weight; y in 16 bits, or in e4m3 with a scale a row
  linear  y = act(x w^T + b) + residual; 16-bit operands, or e4m3 with row and column scales
  ffn     h = act(x Wg^T) * (x Wu^T), y = h Wd^T + residual (gate, up and down projection)
  block   norm (8 bits) -> ffn (gate and up in 8 bits) with the residual stream, as served

Rows are Gaussians or tokens.  ``own`` false computes the plain form (elementary torch
operations in 32 bits, rounded once at the end); true calls the package's layers.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100      # floor of a row's largest magnitude: a row of zeros quantises to zeros
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token through the norm in front of an 8-bit product: a launch's latency
        dict(name="norm-serve-1x1024", op="norm", train=False, rows=1, dim=1024, type="bf16", out="e4m3"),
        # training step of the norm over the 100,000 Gaussians of the small scene, 256 features
        dict(name="norm-train-100000x256", op="norm", train=True, rows=100000, dim=256, type="bf16", out="bf16"),
        # 1,000,000 Gaussians (the medium scene), 256 features, decoded in 8 bits
        dict(name="norm-serve-1000000x256", op="norm", train=False, rows=1000000, dim=256, type="bf16", out="e4m3"),
        # one token through a projection: the weights' bytes
        dict(name="linear-serve-1x1024x4096", op="linear", train=False, rows=1, k=1024, n=4096, type="bf16", out="bf16",
             act="silu", bias=True, residual=False, pitch=0),
        # the decoder's last layer: 59 parameters (SH degree 3) for 1,000,000 Gaussians, fp32, written
        # into the parameter buffer's 64-float blocks
        dict(name="linear-head-1000000x128x59", op="linear", train=False, rows=1000000, k=128, n=59, type="bf16",
             out="f32", act="none", bias=True, residual=False, pitch=64),
        # hidden layer of the decoder on the small scene's Gaussians, training step
        dict(name="linear-train-100000x256x256", op="linear", train=True, rows=100000, k=256, n=256, type="bf16",
             out="bf16", act="gelu", bias=True, residual=True, pitch=0),
        # ragged 8-bit product with a residual: a batch of tokens of odd length and width
        dict(name="linear-serve-e4m3-4099x1040x1111", op="linear", train=False, rows=4099, k=1040, n=1111, type="e4m3",
             out="bf16", act="relu", bias=True, residual=True, pitch=0),
        # one token through the gated block
        dict(name="ffn-serve-1x1024x4096", op="ffn", train=False, rows=1, dim=1024, hidden=4096, type="bf16", act="silu"),
        # narrow decoder block for 1,000,000 Gaussians, training step: bytes, not products
        dict(name="ffn-train-1000000x64x128", op="ffn", train=True, rows=1000000, dim=64, hidden=128, type="bf16",
             act="silu"),
        # wide block of a feed-forward reconstruction model, training step: the tensor cores
        dict(name="ffn-train-32768x1024x4096", op="ffn", train=True, rows=32768, dim=1024, hidden=4096, type="bf16",
             act="silu"),
        # odd sizes in f16, a training step
        dict(name="ffn-train-f16-5003x331x873", op="ffn", train=True, rows=5003, dim=331, hidden=873, type="f16",
             act="gelu"),
        # a served block: residual stream, norm to 8 bits, gate and up in 8 bits, down with the residual
        dict(name="block-serve-2048x1024x4096", op="block", train=False, rows=2048, dim=1024, hidden=4096, type="bf16",
             act="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width in [lo, hi]: a multiple of 8 in half of the draws, any number (odd ones too) in the others."""
    w = _log(rng, lo, hi)
    return max(8, w // 8 * 8) if rng.random() < 0.5 else w


_MOST = dict(flops=18 * 32768 * 1024 * 4096, bytes=1.79e9, values=2.56e8, hidden=1.34e8)   # the largest listed cases


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "ffn", "ffn", "block"])
    case = dict(op=op, train=op != "block" and rng.random() < 0.5, rows=_log(rng, 1, 1000000))
    kind = rng.choice(["bf16", "bf16", "f16"])
    act = rng.choice(["none", "relu", "silu", "gelu"])
    if op == "norm":
        case.update(dim=_width(rng, 16, 8192), type=kind, out=kind if case["train"] else rng.choice([kind, "e4m3"]))
    elif op == "linear":
        if not case["train"] and rng.random() < 0.4:
            kind = "e4m3"
        out = rng.choice(["bf16", "f32"]) if kind == "e4m3" else kind if case["train"] else rng.choice([kind, "f32"])
        n = rng.choice([14, 59]) if rng.random() < 0.2 else _width(rng, 8, 4096)
        case.update(k=_width(rng, 16, 4096), n=n, type=kind, out=out, act=act, bias=rng.random() < 0.6,
                    residual=rng.random() < 0.5, pitch=0)
    else:
        case.update(dim=_width(rng, 16, 2048), hidden=_width(rng, 16, 4096), type="bf16" if op == "block" else kind,
                    act=rng.choice(["silu", "gelu"]))
    while True:
        w = work(case)
        over = max(w["flops"] / _MOST["flops"], w["bytes"] / _MOST["bytes"],
                   case["rows"] * max(case.get(d, 0) for d in ("dim", "k", "n")) / _MOST["values"],
                   case["rows"] * case.get("hidden", 0) / _MOST["hidden"])
        if over <= 1.0 or case["rows"] == 1:
            return case
        case["rows"] = max(1, int(case["rows"] / over * 0.98))


def work(case):
    rows, e = case["rows"], 1 if case["type"] == "e4m3" else 2
    if case["op"] == "norm":
        n = rows * case["dim"]
        if case["train"]:
            # x, r, dy, ds in; s, y, dx out; weight in, its gradient out
            return {"bytes": 14 * n + 4 * case["dim"], "flops": 12 * n}
        return {"bytes": 6 * n + (1 if case["out"] == "e4m3" else 2) * n + 4 * rows, "flops": 6 * n}
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        o = 4 if case["out"] == "f32" else 2
        side = o * rows * n * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0)
        fwd = e * (rows * k + n * k) + side + (4 * (rows + n) if e == 1 else 0)
        if not case["train"]:
            return {"bytes": fwd, "flops": 2 * rows * k * n}
        # dy in; gradients of x, w (and b) out
        return {"bytes": fwd + 2 * (rows * n + rows * k + n * k + n), "flops": 6 * rows * k * n}
    d, f = case["dim"], case["hidden"]
    if case["op"] == "ffn":
        # x, residual, three weights in, y out
        fwd = 2 * (3 * rows * d + 3 * d * f)
        if not case["train"]:
            return {"bytes": fwd, "flops": 6 * rows * d * f}
        # dy in; gradients of x and of three weights out
        return {"bytes": fwd + 2 * (2 * rows * d + 3 * d * f), "flops": 18 * rows * d * f}
    # block: x, residual in, stream and y out; gate and up in 8 bits, down in 16
    return {"bytes": 2 * 4 * rows * d + 4 * d * f, "flops": 6 * rows * d * f}


# ------------------------------------------------------------------------------ inputs
def _quantised(t):
    a = t.abs().amax(dim=1, keepdim=True).clamp_min(TINY)
    return (t * (E4M3_MAX / a)).to(torch.float8_e4m3fn), (a / E4M3_MAX).squeeze(1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["type"] if case["type"] != "e4m3" else "bf16"]
    rows = case["rows"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std

    def like(*shape, std=1.0, dtype=dt):
        return normal(*shape, std=std).to(dtype)

    st = dict(case)
    if case["op"] in ("norm", "block"):
        d = case["dim"]
        # a residual stream whose rows differ in size, a few large channels
        st["x"] = like(rows, d)
        st["r"] = (normal(rows, d) * torch.exp(normal(rows, 1)) * (1 + 9 * (normal(1, d) > 2))).to(dt)
        st["w"] = (1 + 0.2 * normal(d)).to(dt)
        if case["train"]:
            st["dy"], st["ds"] = like(rows, d), like(rows, d)
    if case["op"] == "linear":
        k, n = case["k"], case["n"]
        if case["type"] == "e4m3":
            st["x"], st["xs"] = _quantised(normal(rows, k) * torch.exp(normal(rows, 1)))
            st["w"], st["ws"] = _quantised(normal(n, k, std=k ** -0.5))
        else:
            st["x"], st["w"], st["xs"], st["ws"] = like(rows, k), like(n, k, std=k ** -0.5), None, None
        out = DTYPES[case["out"]]
        st["b"] = like(n, std=0.5, dtype=dt) if case["bias"] else None
        st["r"] = like(rows, n, dtype=out) if case["residual"] else None
        st["y"] = torch.zeros((rows, case["pitch"]), dtype=out, device="cuda")[:, :n] if case["pitch"] else None
        if case["train"]:
            st["dy"] = like(rows, n)
    if case["op"] in ("ffn", "block"):
        d, f = case["dim"], case["hidden"]
        wg, wu = normal(f, d, std=d ** -0.5), normal(f, d, std=d ** -0.5)
        st["wd"] = like(d, f, std=f ** -0.5)
        if case["op"] == "block":
            st["wg"], st["gs"] = _quantised(wg)
            st["wu"], st["us"] = _quantised(wu)
        else:
            st["wg"], st["wu"] = wg.to(dt), wu.to(dt)
            st["x"], st["r"] = like(rows, d), like(rows, d)
            if case["train"]:
                st["dy"] = like(rows, d)
    return st


# ------------------------------------------------------------------------------ plain form
def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain_norm(st):
    s = st["x"].float() + st["r"].float()
    w = st["w"].float()
    rstd = 1 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + EPS)
    return s, w, rstd


def _plain_norm_e4m3(s, w, rstd):
    t = s * w
    a = t.abs().amax(dim=1, keepdim=True).clamp_min(TINY)
    # a division of tensors rounds once; number / tensor would round a reciprocal first
    return (t * (torch.full_like(a, E4M3_MAX) / a)).to(torch.float8_e4m3fn).float(), ((a / E4M3_MAX) * rstd).squeeze(1)


def _run_plain(st):
    op, dt = st["op"], st["x"].dtype
    if op == "norm":
        s, w, rstd = _plain_norm(st)
        if st["out"] == "e4m3":
            q, scale = _plain_norm_e4m3(s, w, rstd)
            return {"q": q, "scale": scale, "s": s.to(dt)}
        out = {"y": (s * rstd * w).to(dt), "s": s.to(dt)}
        if st["train"]:
            dy = st["dy"].float()
            c = (dy * w * s).mean(dim=1, keepdim=True) * rstd * rstd
            out["dx"] = (rstd * (dy * w - s * c) + st["ds"].float()).to(dt)
            out["dw"] = (dy * s * rstd).sum(dim=0).to(dt)
        return out
    if op == "linear":
        x, w = st["x"].float(), st["w"].float()
        if st["xs"] is not None:
            x, w = x * st["xs"][:, None], w * st["ws"][:, None]
        z = x @ w.t()
        if st["b"] is not None:
            z = z + st["b"].float()
        y = _act(z, st["act"])
        if st["r"] is not None:
            y = y + st["r"].float()
        y = y.to(DTYPES[st["out"]])
        if st["y"] is not None:
            st["y"].copy_(y)
            y = st["y"]
        if not st["train"]:
            return {"y": y}
        dz = st["dy"].float() * _act_slope(z, st["act"])
        out = {"y": y, "dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}
        if st["b"] is not None:
            out["db"] = dz.sum(dim=0).to(dt)
        return out
    out = {}
    if op == "block":
        s, w, rstd = _plain_norm(st)
        q, scale = _plain_norm_e4m3(s, w, rstd)
        x, res = q * scale[:, None], s.to(dt).float()
        wg, wu = st["wg"].float() * st["gs"][:, None], st["wu"].float() * st["us"][:, None]
        out["s"] = s.to(dt)
    else:
        x, res, wg, wu = st["x"].float(), st["r"].float(), st["wg"].float(), st["wu"].float()
    wd = st["wd"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a = _act(g, st["act"])
    h = a * u
    out["y"] = (h @ wd.t() + res).to(dt)
    if st["train"]:
        dy = st["dy"].float()
        dh = dy @ wd
        dg, du = dh * u * _act_slope(g, st["act"]), dh * a
        out.update(dx=(dg @ wg + du @ wu).to(dt), dwg=(dg.t() @ x).to(dt), dwu=(du.t() @ x).to(dt),
                   dwd=(dy.t() @ h).to(dt))
    return out


# ------------------------------------------------------------------------------ the package's layers
def _run_own(st):
    from differentiable_rasterizer_gb300 import layers
    op = st["op"]
    if op == "norm":
        o = layers.rms_norm(st["x"], st["w"], residual=st["r"], eps=EPS, out_dtype=DTYPES[st["out"]],
                            need_backward=st["train"])
        if st["out"] == "e4m3":
            return {"q": o.y.float(), "scale": o.scale, "s": o.s}
        out = {"y": o.y, "s": o.s}
        if st["train"]:
            out["dx"], out["dw"] = layers.rms_norm_backward(st["dy"], o.s, st["w"], o.rstd, ds=st["ds"])
        return out
    if op == "linear":
        o = layers.linear(st["x"], st["w"], st["b"], x_scale=st["xs"], w_scale=st["ws"], act=st["act"],
                          residual=st["r"], out=st["y"], out_dtype=DTYPES[st["out"]], need_backward=st["train"])
        if not st["train"]:
            return {"y": o.y}
        gr = layers.linear_backward(st["dy"], st["x"], st["w"], z=o.z, act=st["act"], bias=st["b"] is not None)
        out = {"y": o.y, "dx": gr.dx, "dw": gr.dw}
        if st["b"] is not None:
            out["db"] = gr.db
        return out
    if op == "block":
        o = layers.rms_norm(st["x"], st["w"], residual=st["r"], eps=EPS, out_dtype=torch.float8_e4m3fn)
        h = layers.glu(o.y, st["wg"], st["wu"], x_scale=o.scale, gate_scale=st["gs"], up_scale=st["us"],
                       act=st["act"], out_dtype=st["x"].dtype).h
        return {"s": o.s, "y": layers.linear(h, st["wd"], residual=o.s).y}
    o = layers.glu(st["x"], st["wg"], st["wu"], act=st["act"], need_backward=st["train"])
    out = {"y": layers.linear(o.h, st["wd"], residual=st["r"]).y}
    if st["train"]:
        down = layers.linear_backward(st["dy"], o.h, st["wd"])
        gr = layers.glu_backward(down.dx, st["x"], st["wg"], st["wu"], o.g, o.u, act=st["act"])
        out.update(dx=gr.dx, dwg=gr.dw_gate, dwu=gr.dw_up, dwd=down.dw)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------------------ 64 bits
_EXACT_FLOPS = 6e12     # double-precision work that the card does in some seconds


def exact(case, seed):
    if work(case)["flops"] > _EXACT_FLOPS:
        return None
    st = prepare(case, seed)
    f64 = {k: v.double() for k, v in st.items() if torch.is_tensor(v) and k != "y"}

    def sigma(v):
        return torch.reciprocal(1 + torch.exp(v.neg()))

    def normal_cdf(v):
        return torch.erfc(v * -math.sqrt(0.5)) / 2

    value = {"none": lambda v: v, "relu": lambda v: v.clamp_min(0), "silu": lambda v: v * sigma(v),
             "gelu": lambda v: v * normal_cdf(v)}
    slope = {"none": lambda v: torch.ones_like(v), "relu": lambda v: v.gt(0).double(),
             "silu": lambda v: sigma(v) + v * sigma(v) * sigma(-v),
             "gelu": lambda v: normal_cdf(v) + v * torch.exp(v.square() / -2) / math.sqrt(2 * math.pi)}
    op, res = case["op"], {}
    if op in ("norm", "block"):
        s = torch.add(f64["x"], f64["r"])
        inv = torch.rsqrt(s.square().sum(1) / case["dim"] + EPS)
        weighted = s * f64["w"]
        top = weighted.abs().max(dim=1).values.clamp(min=TINY)
        if op == "block" or case["out"] == "e4m3":
            q = (weighted * (E4M3_MAX / top).unsqueeze(1)).float().to(torch.float8_e4m3fn).double()
            scale = top * inv / E4M3_MAX
    if op == "norm":
        if case["out"] == "e4m3":
            return {"q": q, "scale": scale, "s": s}
        unit = s * inv.unsqueeze(1)
        res = {"y": unit * f64["w"], "s": s}
        if case["train"]:
            up = f64["dy"] * f64["w"]
            along = (up * unit).sum(1, keepdim=True) / case["dim"]
            res["dx"] = f64["ds"] + (up - unit * along) * inv.unsqueeze(1)
            res["dw"] = torch.einsum("rd,rd->d", f64["dy"], unit)
        return res
    if op == "linear":
        x, w = f64["x"], f64["w"]
        if "xs" in f64:
            x, w = x * f64["xs"].unsqueeze(1), w * f64["ws"].unsqueeze(1)
        z = torch.nn.functional.linear(x, w, f64.get("b"))
        res["y"] = value[case["act"]](z) + f64.get("r", 0.0)
        if case["train"]:
            dz = f64["dy"] * slope[case["act"]](z)
            res["dx"] = torch.einsum("mn,nk->mk", dz, w)
            res["dw"] = torch.einsum("mn,mk->nk", dz, x)
            if case["bias"]:
                res["db"] = dz.sum(0)
        return res
    if op == "block":
        x, stream = q * scale.unsqueeze(1), s
        wg, wu = f64["wg"] * f64["gs"].unsqueeze(1), f64["wu"] * f64["us"].unsqueeze(1)
        res["s"] = s
    else:
        x, stream, wg, wu = f64["x"], f64["r"], f64["wg"], f64["wu"]
    gate, lift = torch.einsum("md,fd->mf", x, wg), torch.einsum("md,fd->mf", x, wu)
    h = value[case["act"]](gate).mul(lift)
    res["y"] = stream + torch.einsum("mf,df->md", h, f64["wd"])
    if case["train"]:
        dh = torch.einsum("md,df->mf", f64["dy"], f64["wd"])
        dl, dgate = dh * value[case["act"]](gate), dh * slope[case["act"]](gate) * lift
        res["dx"] = torch.einsum("mf,fd->md", dgate, wg) + torch.einsum("mf,fd->md", dl, wu)
        res["dwg"] = torch.einsum("mf,md->fd", dgate, x)
        res["dwu"] = torch.einsum("mf,md->fd", dl, x)
        res["dwd"] = torch.einsum("md,mf->df", f64["dy"], h)
    return res
