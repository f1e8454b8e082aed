"""Cases of the operators that make the decoder network one of tokens: what surrounds its
norm, linear and gated layers in a block with attention, and in that block's training.

  attention   o = softmax(scale q k^T) v over packed sequences, grouped heads, causal or not;
              one token against a long context, a whole prompt, a training step
  block_norm  s = scale x + gate rms(h) post, y = rms(s) weight: the norm after a block, its
              gate and residual scale and the norm before the next block; y also in e4m3
  clip        the norm over all of a network's gradients, and the gradients scaled to a
              largest norm, written in the optimizer's type

``own`` false computes the plain form (elementary torch operations in 32 bits, rounded once
at the end; sequences padded to the longest); true calls the package's layers.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -100      # floor of a row's largest magnitude: a row of zeros quantises to zeros
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------ cases
# A case's lengths follow from few numbers, so that it stays a dict of plain values: `batch`
# sequences, `q` and `k` tokens the longest ones, `spread` how far below that the others go.
def listed():
    return [
        # one new token of one sequence against its context: latency
        dict(name="attention-serve-1x4097", op="attention", train=False, batch=1, q=1, k=4097, spread=0.0, heads=16,
             kv_heads=4, dim=64, type="bf16", causal=True, behind=0),
        # one new token each of 32 sequences whose contexts differ in length: the context's bytes
        dict(name="attention-serve-32x1x16384", op="attention", train=False, batch=32, q=1, k=16384, spread=0.7,
             heads=32, kv_heads=8, dim=128, type="bf16", causal=True, behind=0),
        # a prompt of odd length in f16
        dict(name="attention-prompt-f16-4099", op="attention", train=False, batch=1, q=4099, k=4099, spread=0.0, heads=16,
             kv_heads=2, dim=128, type="f16", causal=True, behind=0),
        # packed groups of tokens in a training step of the decoder's width (1024: 16 heads of 64), with
        # rows behind the last sequence
        dict(name="attention-train-24x1024", op="attention", train=True, batch=24, q=1024, k=1024, spread=0.9, heads=16,
             kv_heads=4, dim=64, type="bf16", causal=True, behind=37),
        # Gaussians' queries against the tokens of their views, no mask, an odd width of heads
        dict(name="attention-train-cross-f16-5x1111x2049", op="attention", train=True, batch=5, q=1111, k=2049,
             spread=0.5, heads=6, kv_heads=6, dim=72, type="f16", causal=False, behind=0),
        # one long sequence, a training step: the tensor cores
        dict(name="attention-train-16384", op="attention", train=True, batch=1, q=16384, k=16384, spread=0.0, heads=8,
             kv_heads=2, dim=128, type="bf16", causal=True, behind=0),
        # one token between two blocks, y in 8 bits for the next product
        dict(name="block_norm-serve-1x1024", op="block_norm", train=False, rows=1, dim=1024, type="bf16", out="e4m3",
             gate="vector", post=True),
        # training step over the small scene's Gaussians, 256 features, a gate a feature
        dict(name="block_norm-train-100000x256", op="block_norm", train=True, rows=100000, dim=256, type="bf16",
             out="bf16", gate="vector", post=True),
        # odd sizes, f16, a gate a value that the network computes
        dict(name="block_norm-train-f16-20011x331", op="block_norm", train=True, rows=20011, dim=331, type="f16",
             out="f16", gate="rows", post=True),
        # 1,000,000 Gaussians served
        dict(name="block_norm-serve-1000000x256", op="block_norm", train=False, rows=1000000, dim=256, type="bf16",
             out="bf16", gate="vector", post=True),
        # the decoder's own weights (64 features, 128 hidden, fp32): latency
        dict(name="clip-decoder-7", op="clip", tensors=7, values=128 * 64, spread=3.0, type="f32", out="f32", over=True),
        # a network of 16 blocks of 1024 features, 4096 hidden, bf16 gradients to fp32 for the optimizer
        dict(name="clip-blocks-144", op="clip", tensors=144, values=1024 * 4096, spread=1.5, type="bf16", out="f32",
             over=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width in [lo, hi]: a multiple of 8 in half of the draws, any number (odd ones too) in the others."""
    w = _log(rng, lo, hi)
    return max(8, w // 8 * 8) if rng.random() < 0.5 else w


_PAIRS = 16384 * 16384 * 8          # heads x padded pairs of the largest listed training step
_CONTEXT = 32 * 16384 * 8 * 128     # values of keys of the largest listed context
_MOST_FLOPS = 1.93e12               # of the largest listed training step


def _draw_attention(rng):
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128, rng.randrange(8, 129)])
    kv_heads = rng.choice([1, 2, 4, 8, rng.randrange(1, 12)])
    heads = kv_heads * rng.choice([1, 1, 2, 4, 8, rng.randrange(1, 10)])
    case = dict(op="attention", train=False, batch=_log(rng, 1, 64), spread=rng.choice([0.0, rng.random()]), heads=heads,
                kv_heads=kv_heads, dim=dim, type=rng.choice(["bf16", "bf16", "f16"]), causal=rng.random() < 0.6, behind=0)
    if rng.random() < 0.35:         # single tokens, or a few, against a context
        case.update(q=rng.choice([1, 1, rng.randrange(1, 9)]), k=_log(rng, 1, 65536))
    else:
        case.update(q=_log(rng, 1, 16384), train=rng.random() < 0.6, behind=rng.choice([0, rng.randrange(0, 200)]))
        case["k"] = case["q"] if case["causal"] else _log(rng, 1, 16384)
        if case["causal"] and rng.random() < 0.3:
            case["k"] = case["q"] + rng.randrange(0, 1000)     # a chunk behind an earlier context
    while True:
        pairs = case["batch"] * case["heads"] * case["q"] * case["k"] * (1 if case["train"] else 0.3) / _PAIRS
        context = case["batch"] * case["k"] * case["kv_heads"] * case["dim"] / _CONTEXT
        queries = case["batch"] * case["q"] * case["heads"] * case["dim"] / _CONTEXT
        if max(pairs, context, queries, work(case)["flops"] / _MOST_FLOPS) <= 1:
            # one key alone has no gradient: only rounding would be compared
            case["train"] = case["train"] and min(case["q"], case["k"]) >= 32
            return case
        if case["batch"] > 1:
            case["batch"] = max(1, case["batch"] // 2)
        else:
            case["k"] = max(1, int(case["k"] * 0.7))
            case["q"] = min(case["q"], case["k"]) if case["causal"] else max(1, int(case["q"] * 0.7))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "block_norm", "block_norm", "clip"])
    if op == "attention":
        return _draw_attention(rng)
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "clip":
        case = dict(op="clip", tensors=_log(rng, 1, 300), values=_log(rng, 1, 1024 * 4096), spread=rng.uniform(0, 4),
                    type=kind, out=rng.choice([kind, "f32"]), over=rng.random() < 0.7)
        most = sum(_sizes(listed()[-1])) * 2 / (4 if kind == "f32" else 2)
        while sum(_sizes(case)) > most:
            case["tensors"] = max(1, case["tensors"] // 2)
            case["values"] = max(1, case["values"] // 2)
        return case
    dim, train = _width(rng, 16, 8192), rng.random() < 0.5
    rows = min(_log(rng, 1, 1000000), max(1, 256000000 // dim // (2 if kind == "f32" else 1) // (2 if train else 1)))
    return dict(op=op, train=train, rows=rows, dim=dim, type=kind, out=kind if train or kind == "f32" else rng.choice([kind, "e4m3"]),
                gate=rng.choice(["vector", "rows", "none"]), post=rng.random() < 0.8)


def _lengths(case):
    """Tokens of queries and keys of each sequence: the first the longest, the others below by a fixed pattern."""
    q, k = [], []
    for b in range(case["batch"]):
        f = 1 - case["spread"] * ((b * 0.6180339887498949) % 1.0)
        k.append(max(1, int(round(case["k"] * f))))
        # causal: as many tokens short of the keys as the longest is
        q.append(max(1, k[-1] - (case["k"] - case["q"])) if case["causal"] else max(1, int(round(case["q"] * f))))
        if case["q"] <= 8:
            q[-1] = case["q"]
    return q, k


def _sizes(case):
    """Values of each tensor, from `values` down by up to e^spread."""
    return [max(1, int(case["values"] * math.exp(-case["spread"] * ((i * 0.6180339887498949) % 1.0))))
            for i in range(case["tensors"])]


def _places(sizes):
    """Where tensors of these sizes start in one buffer, and its end."""
    at = [0]
    for n in sizes:
        at.append(at[-1] + (n + 63) // 64 * 64)
    return at


def work(case):
    if case["op"] == "clip":
        n = sum(_sizes(case))
        b = {"bf16": 2, "f16": 2, "f32": 4}
        return {"bytes": n * (b[case["type"]] + b[case["out"]]), "flops": 3 * n}
    e = 4 if case["type"] == "f32" else 2
    if case["op"] == "block_norm":
        n = case["rows"] * case["dim"]
        rows = 3 if case["gate"] == "rows" else 2
        if case["train"]:       # h, x, gate, dy, ds in; s, y, dh, dx and the gate's gradient out
            return {"bytes": e * n * (rows + 2 + 4 + (case["gate"] == "rows")) + 16 * case["dim"], "flops": 30 * n}
        return {"bytes": e * n * (rows + 1) + n * (1 if case["out"] == "e4m3" else e) + 4 * case["rows"], "flops": 12 * n}
    ql, kl = _lengths(case)
    pairs = 0
    for a, b in zip(ql, kl):
        if not case["causal"]:
            pairs += a * b
        else:                   # query i sees i + 1 + b - a keys
            first = max(0, a - b)
            pairs += sum((first + 1 + b - a, b)) * (a - first) // 2
    q, k = sum(ql) * case["heads"] * case["dim"], sum(kl) * case["kv_heads"] * case["dim"]
    fwd = 2 * (2 * q + 2 * k)
    if not case["train"]:
        return {"bytes": fwd, "flops": 4 * pairs * case["heads"] * case["dim"]}
    return {"bytes": fwd + 2 * (2 * q + 2 * k), "flops": 14 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["type"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    st = dict(case)
    if case["op"] == "attention":
        ql, kl = _lengths(case)
        d, rows, keys = case["dim"], sum(ql) + case["behind"], sum(kl) + case["behind"]
        # queries and keys whose products spread as a trained layer's do; a few keys that draw much weight
        st["q"] = (normal(rows, case["heads"], d) * 1.5).to(dt)
        st["k"] = (normal(keys, case["kv_heads"], d) * (1 + 2 * (normal(keys, 1, 1) > 2.5))).to(dt)
        st["v"] = normal(keys, case["kv_heads"], d).to(dt)
        if case["train"]:
            st["do"] = (normal(rows, case["heads"], d) * 0.1).to(dt)

        def starts(lengths):
            return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)

        st["q_starts"], st["k_starts"] = starts(ql), starts(kl)
        st["q_most"], st["k_most"] = max(ql), max(kl)
        return st
    if case["op"] == "clip":
        sizes = _sizes(case)
        total = math.sqrt(sum(sizes))
        # gradients whose size differs from tensor to tensor; most cases are above the largest norm
        st["grads"] = [(normal(n) * (0.01 * (1 + i % 5))).to(dt) for i, n in enumerate(sizes)]
        st["most"] = total * (0.01 if case["over"] else 1.0)
        # the optimizer's gradients lie in one buffer, each on 64 elements
        at = _places(sizes)
        st["flat"] = torch.zeros(at[-1], device="cuda", dtype=DTYPES[case["out"]])
        st["clipped"] = [st["flat"][a:a + n] for a, n in zip(at, sizes)]
        return st
    rows, d = case["rows"], case["dim"]
    # a block's output and a residual stream whose rows differ in size, a few large channels
    st["h"] = (normal(rows, d) * torch.exp(0.5 * normal(rows, 1))).to(dt)
    st["x"] = (normal(rows, d) * torch.exp(normal(rows, 1)) * (1 + 9 * (normal(1, d) > 2))).to(dt)
    st["w"] = (1 + 0.2 * normal(d)).to(dt)
    st["p"] = (1 + 0.2 * normal(d)).to(dt) if case["post"] else None
    st["g"] = {"none": lambda: None, "vector": lambda: (0.3 * normal(d)).to(dt),
               "rows": lambda: torch.sigmoid(normal(rows, d)).to(dt)}[case["gate"]]()
    st["scale"] = 0.875
    if case["train"]:
        st["dy"], st["ds"] = normal(rows, d).to(dt), normal(rows, d).to(dt)
    return st


# ------------------------------------------------------------------------------ plain form
def _plain_attention(st):
    dt, heads, group = st["q"].dtype, st["kv_heads"], st["heads"] // st["kv_heads"]
    qs, ks = st["q_starts"].long(), st["k_starts"].long()
    qi = qs[:-1, None] + torch.arange(st["q_most"], device="cuda")          # [sequence, query]: its row
    ki = ks[:-1, None] + torch.arange(st["k_most"], device="cuda")
    q_in, k_in = qi < qs[1:, None], ki < ks[1:, None]
    qi, ki = torch.where(q_in, qi, 0), torch.where(k_in, ki, 0)

    def rows_of(name, at, live):     # [sequence, row, key head, head of its group, column]; nothing in padding
        t = st[name].float()[at] * live[:, :, None, None]
        return t.view(*at.shape, heads, -1, st["dim"])

    scale = st["dim"] ** -0.5
    q, k, v = rows_of("q", qi, q_in), rows_of("k", ki, k_in)[:, :, :, 0], rows_of("v", ki, k_in)[:, :, :, 0]
    t = torch.einsum("bqhgd,bkhd->bhgqk", q, k) * scale
    hidden = ~(q_in[:, :, None] & k_in[:, None, :])
    if st["causal"]:
        short = (ks[1:] - ks[:-1] - qs[1:] + qs[:-1])[:, None, None]
        last = torch.arange(st["q_most"], device="cuda")[None, :, None] + short
        hidden = hidden | (torch.arange(st["k_most"], device="cuda")[None, None, :] > last)
    t = t.masked_fill(hidden[:, None, None], float("-inf"))
    top = t.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(t.sub_(top))
    del t
    total = p.sum(dim=-1, keepdim=True)
    p.div_(torch.where(total > 0, total, 1.0))

    def to_rows(t, at, live, like, dtype):      # back to packed rows; rows of no sequence are zero
        out = torch.zeros(like, device="cuda", dtype=dtype)
        out[at[live]] = t[live].reshape(-1, *like[1:]).to(dtype)
        return out

    o = torch.einsum("bhgqk,bkhd->bqhgd", p, v)
    out = {"o": to_rows(o, qi, q_in, st["q"].shape, dt)}
    if st["train"]:
        lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2)
        out["lse"] = to_rows(lse, qi, q_in, st["q"].shape[:2], torch.float32)
        do = rows_of("do", qi, q_in)
        out["dv"] = to_rows(torch.einsum("bhgqk,bqhgd->bkhd", p, do), ki, k_in, st["v"].shape, dt)
        delta = (do * o).sum(dim=-1).permute(0, 2, 3, 1)
        ds = torch.einsum("bqhgd,bkhd->bhgqk", do, v).sub_(delta[..., None]).mul_(p).mul_(scale)
        del p
        out["dq"] = to_rows(torch.einsum("bhgqk,bkhd->bqhgd", ds, k), qi, q_in, st["q"].shape, dt)
        out["dk"] = to_rows(torch.einsum("bhgqk,bqhgd->bkhd", ds, q), ki, k_in, st["k"].shape, dt)
    return out


def _plain_block_norm(st):
    dt = st["h"].dtype
    h, x, w = st["h"].float(), st["x"].float(), st["w"].float()
    g = 1.0 if st["g"] is None else st["g"].float()
    unit = h
    if st["p"] is not None:
        inv_h = 1 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        unit = h * inv_h
    a = unit if st["p"] is None else unit * st["p"].float()
    s = st["scale"] * x + g * a
    inv = 1 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + EPS)
    out = {"s": s.to(dt)}
    if st["out"] == "e4m3":
        t = s * w
        top = t.abs().amax(dim=1, keepdim=True).clamp_min(TINY)
        out["y"] = (t * (torch.full_like(top, E4M3_MAX) / top)).to(torch.float8_e4m3fn).to(torch.bfloat16)
        out["y_scale"] = ((top / E4M3_MAX) * inv).squeeze(1)
        return out
    out["y"] = (s * inv * w).to(dt)
    if not st["train"]:
        return out
    dy = st["dy"].float()
    along = (dy * w * s).mean(dim=1, keepdim=True) * inv * inv
    ds = inv * (dy * w - s * along) + st["ds"].float()
    out["dw"] = (dy * s * inv).sum(dim=0).to(dt)
    out["dx"] = (st["scale"] * ds).to(dt)
    if st["gate"] == "vector":
        out["dg"] = (ds * a).sum(dim=0).to(dt)
    elif st["gate"] == "rows":
        out["dg"] = (ds * a).to(dt)
    da = ds * g
    if st["p"] is None:
        out["dh"] = da.to(dt)
        return out
    out["dp"] = (da * unit).sum(dim=0).to(dt)
    du = da * st["p"].float()
    out["dh"] = (inv_h * (du - unit * (du * unit).mean(dim=1, keepdim=True))).to(dt)
    return out


def _plain_clip(st):
    squares = torch.stack([(t.float() * t.float()).sum(dtype=torch.float64) for t in st["grads"]])
    norm = torch.sqrt(squares.sum()).float()
    factor = torch.clamp(st["most"] / norm, max=1.0)
    for t, c in zip(st["grads"], st["clipped"]):
        c.copy_(t.float() * factor)
    return {"norm": norm, "clipped": st["flat"]}


# ------------------------------------------------------------------------------ the package's layers
def _run_own(st):
    from differentiable_rasterizer_gb300 import layers
    if st["op"] == "attention":
        seq = dict(q_starts=st["q_starts"], k_starts=st["k_starts"], causal=st["causal"])
        a = layers.attention(st["q"], st["k"], st["v"], need_backward=st["train"], **seq)
        if not st["train"]:
            return {"o": a.o}
        g = layers.attention_backward(st["do"], st["q"], st["k"], st["v"], a.o, a.lse, **seq)
        return {"o": a.o, "lse": a.lse, "dv": g.dv, "dq": g.dq, "dk": g.dk}
    if st["op"] == "clip":
        return {"norm": layers.clip_norm(st["grads"], st["most"], out=st["clipped"]), "clipped": st["flat"]}
    b = layers.block_norm(st["h"], st["x"], st["w"], post_weight=st["p"], gate=st["g"], scale=st["scale"], eps=EPS,
                          out_dtype=DTYPES[st["out"]], need_backward=st["train"])
    if st["out"] == "e4m3":
        return {"s": b.s, "y": b.y.to(torch.bfloat16), "y_scale": b.y_scale}
    out = {"s": b.s, "y": b.y}
    if st["train"]:
        g = layers.block_norm_backward(st["dy"], st["h"], b.s, st["w"], b.rstd, post_weight=st["p"],
                                       rstd_post=b.rstd_post, gate=st["g"], scale=st["scale"], ds=st["ds"])
        out.update(dw=g.dweight, dx=g.dx)
        if st["g"] is not None:
            out["dg"] = g.dgate
        if st["p"] is not None:
            out["dp"] = g.dpost_weight
        out["dh"] = g.dh
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "block_norm": _plain_block_norm, "clip": _plain_clip}[state["op"]](state)


# ------------------------------------------------------------------------------ 64 bits
_EXACT_FLOPS = 6e12     # double-precision work that the card does in some seconds


def _exact_attention(case, st):
    ql, kl = _lengths(case)
    group, c = case["heads"] // case["kv_heads"], math.sqrt(1.0 / case["dim"])
    out = {"o": torch.zeros_like(st["q"], dtype=torch.float64)}
    if case["train"]:
        out["lse"] = torch.zeros(st["q"].shape[:2], device="cuda", dtype=torch.float64)
        out.update({n: torch.zeros_like(st[n[1]], dtype=torch.float64) for n in ("dv", "dq", "dk")})
    q0 = k0 = 0
    for a, b in zip(ql, kl):
        for h in range(case["kv_heads"]):
            hs = slice(h * group, (h + 1) * group)
            q = st["q"][q0:q0 + a, hs].double().transpose(0, 1)         # [group, a, dim]
            k, v = st["k"][k0:k0 + b, h].double(), st["v"][k0:k0 + b, h].double()
            t = torch.matmul(q, k.t()).mul_(c)
            if case["causal"]:
                seen = torch.ones(a, b, device="cuda", dtype=torch.bool).tril_(b - a)
                t = t.where(seen, torch.tensor(float("-inf"), device="cuda", dtype=torch.float64))
            lse = torch.logsumexp(t, dim=-1, keepdim=True)
            w = torch.exp_(t - lse.clamp_min(-1e300))
            del t
            o = w @ v
            out["o"][q0:q0 + a, hs] = o.transpose(0, 1)
            if case["train"]:
                out["lse"][q0:q0 + a, hs] = lse.squeeze(-1).t()
                do = st["do"][q0:q0 + a, hs].double().transpose(0, 1)
                out["dv"][k0:k0 + b, h] = torch.matmul(w.transpose(1, 2), do).sum(0)
                back = w.mul_(torch.matmul(do, v.t()) - (o * do).sum(-1, keepdim=True)).mul_(c)
                out["dq"][q0:q0 + a, hs] = torch.matmul(back, k).transpose(0, 1)
                out["dk"][k0:k0 + b, h] = torch.matmul(back.transpose(1, 2), q).sum(0)
        q0, k0 = q0 + a, k0 + b
    return out


def _exact_block_norm(case, st):
    f64 = {k: v.double() for k, v in st.items() if torch.is_tensor(v)}

    def unit_of(t):
        inv = torch.rsqrt(t.square().sum(1, keepdim=True) / case["dim"] + EPS)
        return t * inv, inv

    def through(d, unit, inv):      # gradient of t from d, the gradient of unit_of(t)
        return inv * (d - unit * torch.einsum("rd,rd->r", d, unit).div(case["dim"]).unsqueeze(1))

    unit_h, inv_h = unit_of(f64["h"]) if case["post"] else (f64["h"], None)
    a = unit_h * f64.get("p", 1.0)
    gate = f64.get("g", torch.ones((), device="cuda", dtype=torch.float64))
    s = torch.addcmul(f64["x"] * st["scale"], gate, a)
    unit, inv = unit_of(s)
    out = {"s": s}
    if case["out"] == "e4m3":
        weighted = s * f64["w"]
        top = weighted.abs().max(dim=1).values.clamp(min=TINY)
        out["y"] = (weighted * (E4M3_MAX / top).unsqueeze(1)).float().to(torch.float8_e4m3fn).double()
        out["y_scale"] = top * inv.squeeze(1) / E4M3_MAX
        return out
    out["y"] = unit * f64["w"]
    if case["train"]:
        ds = f64["ds"] + through(f64["dy"] * f64["w"], unit, inv)
        out["dw"] = torch.einsum("rd,rd->d", f64["dy"], unit)
        out["dx"] = ds * st["scale"]
        if case["gate"] != "none":
            out["dg"] = torch.einsum("rd,rd->d", ds, a) if case["gate"] == "vector" else ds * a
        da = ds * gate
        if case["post"]:
            out["dp"] = torch.einsum("rd,rd->d", da, unit_h)
            da = through(da * f64["p"], unit_h, inv_h)
        out["dh"] = da
    return out


def exact(case, seed):
    if case["op"] == "attention" and work(case)["flops"] * (2 if case["causal"] else 1) > _EXACT_FLOPS:
        return None
    st = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(case, st)
    if case["op"] == "block_norm":
        return _exact_block_norm(case, st)
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in st["grads"]))
    shrink = min(1.0, st["most"] / norm) if norm else 1.0
    flat = torch.zeros(st["flat"].shape, dtype=torch.float64, device="cuda")
    for t, a in zip(st["grads"], _places(_sizes(case))):
        torch.mul(t.double(), shrink, out=flat[a:a + t.numel()])
    return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"), "clipped": flat}
