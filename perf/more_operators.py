"""Cases of the training-step operators between the products and around the
reduced gradients: the token embedding at the bottom of the model with its
gradient, the norms, gate and residual sum between the blocks with their
gradients, and the global gradient norm with clipping before the update.

Operators and their definitions (all sums in 32 bits or more):

* ``embedding``       y[t] = scale W[id[t]].
* ``embedding_grad``  dW[v] = scale sum of dy[t] over the t with id[t] = v;
                      stored for every row of the table (zeros where no token
                      is), or added to what the rows hold.  Tokens of one id,
                      the padding, give no gradient.
* ``block_norm``      between two blocks of a residual stream x, y the output of
                      the block below:
                          N(a, w) = w a / sqrt(mean(a^2) + eps)   (row by row)
                          u = N(y, post)        (u = y without post)
                          r = s x + gate u      (gate per channel, per sequence
                                                 and channel, or per token and
                                                 channel; 1 without)
                          h = N(r, pre)         (what the next block reads)
                      without y: r is x, and only h is formed.
* ``block_norm_grad`` its gradient: from dr (the residual stream's) and dh (the
                      block's) to dx and dy, and to pre, post and gate; the last
                      three stored, or added to what the outputs hold.
* ``clip``            n = sqrt(sum of g^2 over all gradients of the model),
                      c = min(1, max_norm / (n + 1e-6)), g = c g in place; or the
                      norm alone.

Sizes are those of the 402.8M-parameter tree (width 1024, 98304 tokens of
vocabulary) and of the qwen3-0.6b tree (151936 tokens), with odd and ragged ones
between them.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
LAYERS_402M = "98304x1024," + ",".join(["1x1024,1x1024,4*1024x1024,1x1024,1x1024,1024x4096,4096x1024"] * 24) + ",1x1024,1x1024"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a few small odd parameters at the end of a step: latency
        dict(name="clip small", op="clip", shapes="2*100x333,257x64,1x333", dtype="f32", clip=True),
        # one rank's share of the 402.8M tree at 8 ranks, the bf16 gradients that the flush leaves on their owner
        dict(name="clip owner share", op="clip", shapes="12*1024x1024,3*4096x1024,3*1024x4096,12*1x1024", dtype="bf16",
             clip=True),
        # the norm of every bf16 gradient of the 402.8M tree, as a step logs it
        dict(name="norm 402.8M", op="clip", shapes=LAYERS_402M, dtype="bf16", clip=False),
        # one token of generation
        dict(name="embedding 1 token", op="embedding", t=1, v=98304, d=1024, ids="i64", wdtype="bf16", dtype="bf16", scale=1.0,
             pad=0),
        # a training micro-batch, scaled by the square root of the width
        dict(name="embedding batch", op="embedding", t=16384, v=98304, d=1024, ids="i64", wdtype="bf16", dtype="bf16",
             scale=32.0, pad=0),
        # its gradient, stored as the bf16 gradient row that the bucket flush reads
        dict(name="embedding_grad batch", op="embedding_grad", t=16384, v=98304, d=1024, ids="i64", gdtype="bf16",
             dtype="bf16", scale=32.0, accumulate=False, padding=False, pad=0),
        # a padded micro-batch added to the replica's fp32 accumulator of the larger vocabulary
        dict(name="embedding_grad accumulate", op="embedding_grad", t=8192, v=151936, d=1024, ids="i32", gdtype="bf16",
             dtype="f32", scale=1.0, accumulate=True, padding=True, pad=0),
        # a short ragged prompt over a small table whose rows fit no 16-byte vector
        dict(name="embedding_grad ragged", op="embedding_grad", t=333, v=1000, d=777, ids="i32", gdtype="f32",
             dtype="f32", scale=0.5, accumulate=False, padding=True, pad=3),
        # one token of generation between two blocks
        dict(name="block_norm 1 token", op="block_norm", m=1, d=1024, stream="bf16", y=True, post=True, gate="channel", groups=1,
             pre=True, scale=1.0, wdtype="f32", pad=0),
        # a training micro-batch between two blocks
        dict(name="block_norm batch", op="block_norm", m=16384, d=1024, stream="bf16", y=True, post=True, gate="channel",
             groups=1, pre=True, scale=0.5, wdtype="f32", pad=0),
        # its gradient
        dict(name="block_norm_grad batch", op="block_norm_grad", m=16384, d=1024, stream="bf16", y=True, post=True,
             gate="channel", groups=1, pre=True, scale=0.5, wdtype="f32", accumulate=True, pad=0),
        # odd rows of an fp32 stream with a gate for each of three sequences
        dict(name="block_norm_grad ragged", op="block_norm_grad", m=1539, d=777, stream="f32", y=True, post=True,
             gate="sequence", groups=3, pre=True, scale=1.0, wdtype="bf16", accumulate=False, pad=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("clip", "embedding", "embedding_grad", "embedding_grad", "block_norm", "block_norm_grad"))
    pad = rng.choice((0, 0, 0, 8, 3))
    types = ("bf16", "f32")
    if op == "clip":
        parts, left = [], 2e8
        for _ in range(_log(rng, 1, 40)):
            r, c, n = _log(rng, 1, 4096), _log(rng, 1, 4096), rng.randint(1, 8)
            if n * r * c <= left:
                left -= n * r * c
                parts.append("%d*%dx%d" % (n, r, c))
        return dict(op=op, shapes=",".join(parts), dtype=rng.choice(types), clip=rng.random() < 0.7)
    if op in ("embedding", "embedding_grad"):
        t, v, d = _log(rng, 1, 16384), _log(rng, 100, 98304), _log(rng, 16, 1024)
        if rng.random() < 0.6:  # most widths are multiples of 64
            d = max(64, d // 64 * 64)
        c = dict(op=op, t=t, v=v, d=d, ids=rng.choice(("i32", "i64")), dtype=rng.choice(types),
                 scale=rng.choice((1.0, round(math.sqrt(d), 3))), pad=pad)
        if op == "embedding":
            return dict(c, wdtype=rng.choice(types))
        return dict(c, gdtype=rng.choice(types), accumulate=rng.random() < 0.5, padding=rng.random() < 0.5)
    m, d = _log(rng, 1, 16384), _log(rng, 16, 4096)
    if rng.random() < 0.6:
        d = max(64, d // 64 * 64)
    m = max(1, min(m, 16384 * 1024 // d))
    y = rng.random() < 0.8
    gate = rng.choice(("none", "channel", "sequence", "token")) if y else "none"
    groups = 1 if gate in ("none", "channel") else m
    if gate == "sequence":
        groups = rng.randint(1, min(m, 64))
        m = m // groups * groups
    c = dict(op=op, m=m, d=d, stream=rng.choice(types), y=y, post=y and rng.random() < 0.7, gate=gate, groups=groups,
             pre=not y or rng.random() < 0.8, scale=rng.choice((1.0, 0.5)) if y else 1.0, wdtype=rng.choice(types), pad=pad)
    return dict(c, accumulate=rng.random() < 0.5) if op == "block_norm_grad" else c


def _shapes(case):
    """Shapes of a list such as "2*100x333,257x64"."""
    parts = [p.split("*") if "*" in p else ("1", p) for p in case["shapes"].split(",")]
    return [tuple(int(x) for x in s.split("x")) for n, s in parts for _ in range(int(n))]


def _dt(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}[name]


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, shift=0.0, dtype="bf16", pad=0):
        t = torch.randn(*shape[:-1], shape[-1] + pad, device="cuda", generator=gen).mul_(scale).add_(shift)
        return t.to(_dt(dtype))[..., :shape[-1]]  # with pad, rows of a wider tensor

    op = case["op"]
    s = dict(case)
    if op == "clip":
        # the gradients lie back to back, as the tasks of a bucket do
        shapes = _shapes(case)
        sizes = [math.prod(x) for x in shapes]
        s["flat"] = randn(sum(sizes), scale=1e-3, dtype=case["dtype"])
        s["grads"] = [g.view(x) for g, x in zip(s["flat"].split(sizes), shapes)]
        # a threshold at half the usual norm that falls a little from step to step, so that every step clips
        s["max_norm"] = 0.5e-3 * math.sqrt(sum(sizes))
        if own:
            import zero_collectives_gb300 as zc
            s["handle"] = zc.GradClip(s["grads"], eps=EPS)  # kept over the steps, as the optimizer is
        return s
    if op in ("embedding", "embedding_grad"):
        t, v, d, pad = case["t"], case["v"], case["d"], case["pad"]
        # frequent tokens have low ids: the share of the first k tokens grows with log k
        u = torch.rand(t, device="cuda", generator=gen, dtype=torch.float64)
        ids = ((u * math.log(v + 1)).exp().long() - 1).clamp_(0, v - 1)
        s["ids"] = ids.to(_dt(case["ids"]))
        if op == "embedding":
            s["w"] = randn(v, d, scale=0.02, dtype=case["wdtype"], pad=pad)
        else:
            s["pad_id"] = None
            if case["padding"]:  # the last tenth of the batch is padding
                s["pad_id"] = v - 1
                s["ids"][t - t // 10:] = v - 1
            s["dy"] = randn(t, d, scale=1e-3, dtype=case["gdtype"], pad=pad)
            s["dw"] = randn(v, d, scale=1e-2, dtype=case["dtype"], pad=pad)
        return s
    m, d, pad, st, wt = case["m"], case["d"], case["pad"], case["stream"], case["wdtype"]
    s["x" if op == "block_norm" else "r"] = randn(m, d, scale=2.0, dtype=st, pad=pad)
    s["yb"] = randn(m, d, pad=pad) if case["y"] else None
    s["post_w"] = randn(d, scale=0.1, shift=1.0, dtype=wt) if case["post"] else None
    s["gate_w"] = randn(case["groups"], d, scale=0.1, shift=0.3, dtype=wt) if case["gate"] != "none" else None
    s["pre_w"] = randn(d, scale=0.1, shift=1.0, dtype=wt) if case["pre"] else None
    if op == "block_norm_grad":
        s["dr"] = randn(m, d, scale=1e-3, dtype=st, pad=pad)
        s["dh"] = randn(m, d, scale=1e-3, pad=pad) if case["pre"] else None
        for k in ("post", "gate", "pre"):
            w = s[k + "_w"]
            s[k + "_grad"] = None if w is None else randn(*w.shape, scale=1e-2, dtype="f32")
    return s


# -------------------------------------------------------------------- runs --

def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _threshold(s):
    s["max_norm"] *= 0.999
    return s["max_norm"]


def _plain_clip(s):
    norm = s["flat"].float().square().sum().double().sqrt()
    if not s["clip"]:
        return norm.float().reshape(1)
    c = (_threshold(s) / (norm + EPS)).clamp(max=1.0)
    s["flat"].copy_(s["flat"].float() * c.float())
    return {"flat": s["flat"], "result": torch.stack((norm, c)).float()}


def _plain_embedding(s):
    return (s["w"][s["ids"].long()].float() * s["scale"]).to(_dt(s["dtype"]))


def _plain_embedding_grad(s):
    ids, dy = s["ids"].long(), s["dy"].float() * s["scale"]
    if s["pad_id"] is not None:
        dy = torch.where((ids == s["pad_id"])[:, None], torch.zeros_like(dy), dy)
    dw = s["dw"].float() if s["accumulate"] else torch.zeros(s["v"], s["d"], device="cuda")
    s["dw"].copy_(dw.index_add(0, ids, dy))
    return s["dw"]


def _rms(a):
    return 1 / (a.square().mean(-1, keepdim=True) + EPS).sqrt()


def _gate_rows(s):
    """The gate of every token, [m, d] or broadcast to it."""
    g = s["gate_w"]
    return 1.0 if g is None else g.float().repeat_interleave(s["m"] // g.shape[0], 0) if g.shape[0] > 1 else g.float()


def _plain_block_norm(s):
    x = s["x"].float()
    out = {}
    if s["y"]:
        u = s["yb"].float()
        if s["post"]:
            u = u * _rms(u) * s["post_w"].float()
        x = s["scale"] * x + _gate_rows(s) * u
        out["r"] = x.to(_dt(s["stream"]))
    if s["pre"]:
        out["h"] = (x * _rms(x) * s["pre_w"].float()).bfloat16()
    return out


def _norm_grad(a, w, g):
    """Gradients of w a / sqrt(mean(a^2) + eps) to a and w."""
    i = _rms(a)
    n = a * i
    gw = g * w
    return i * (gw - n * (gw * n).mean(-1, keepdim=True)), (g * n).sum(0)


def _plain_block_norm_grad(s):
    g = s["dr"].float()
    out = {}

    def leave(name, value):
        if s["accumulate"]:
            value = s[name] + value
        s[name].copy_(value)
        out[name] = s[name]

    if s["pre"]:
        da, dw = _norm_grad(s["r"].float(), s["pre_w"].float(), s["dh"].float())
        g = g + da
        leave("pre_grad", dw)
    out["dx"] = (s["scale"] * g).to(_dt(s["stream"]))
    if s["y"]:
        y = s["yb"].float()
        if s["gate_w"] is not None:
            u = y * _rms(y) * s["post_w"].float() if s["post"] else y
            leave("gate_grad", (g * u).view(s["groups"], -1, s["d"]).sum(1))
        g = g * _gate_rows(s)
        if s["post"]:
            g, dw = _norm_grad(y, s["post_w"].float(), g)
            leave("post_grad", dw)
        out["dy"] = g.bfloat16()
    return out


_PLAIN = {"clip": _plain_clip, "embedding": _plain_embedding, "embedding_grad": _plain_embedding_grad,
          "block_norm": _plain_block_norm, "block_norm_grad": _plain_block_norm_grad}


def _own_clip(s):
    if not s["clip"]:
        return s["handle"].norm()
    return {"flat": s["flat"], "result": s["handle"].clip(_threshold(s))}


def _own_embedding(s):
    import zero_collectives_gb300 as zc
    return zc.embedding(s["ids"], s["w"], scale=s["scale"], out_dtype=_dt(s["dtype"]))


def _own_embedding_grad(s):
    import zero_collectives_gb300 as zc
    return zc.embedding_grad(s["ids"], s["dy"], s["dw"], scale=s["scale"], padding=s["pad_id"], accumulate=s["accumulate"])


def _own_block_norm(s):
    import zero_collectives_gb300 as zc
    r, h = zc.block_norm(s["x"], y=s["yb"], post=s["post_w"], gate=s["gate_w"], residual_scale=s["scale"], pre=s["pre_w"], eps=EPS)
    return {k: v for k, v in (("r", r if s["y"] else None), ("h", h)) if v is not None}


def _own_block_norm_grad(s):
    import zero_collectives_gb300 as zc
    dx, dy = zc.block_norm_grad(s["r"], dr=s["dr"], dh=s["dh"], y=s["yb"], post=s["post_w"], gate=s["gate_w"],
                                residual_scale=s["scale"], pre=s["pre_w"], eps=EPS, post_grad=s["post_grad"],
                                gate_grad=s["gate_grad"], pre_grad=s["pre_grad"], accumulate=s["accumulate"])
    out = {"dx": dx, "dy": dy, "post_grad": s["post_grad"], "gate_grad": s["gate_grad"], "pre_grad": s["pre_grad"]}
    return {k: v for k, v in out.items() if v is not None}


_OWN = {"clip": _own_clip, "embedding": _own_embedding, "embedding_grad": _own_embedding_grad,
        "block_norm": _own_block_norm, "block_norm_grad": _own_block_norm_grad}


# -------------------------------------------------------------------- work --

def _size(name):
    return {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}[name]


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(math.prod(x) for x in _shapes(case))
        return {"bytes": _size(case["dtype"]) * n * (2 if case["clip"] else 1) + 4, "flops": (3 if case["clip"] else 2) * n}
    if op in ("embedding", "embedding_grad"):
        t, v, d = case["t"], case["v"], case["d"]
        # ids below j have the share log(j + 1) / log(v + 1) of the tokens: how many rows are met at least once
        seen, lo = 0.0, 0
        while lo < v:  # by runs of ids that grow with the id
            hi = min(v, lo + 1 + lo // 8)
            p = math.log((hi + 1) / (lo + 1)) / math.log(v + 1) / (hi - lo)
            seen += (hi - lo) * -math.expm1(t * math.log1p(-p) if p < 1 else -t)
            lo = hi
        rows = min(t, max(1, int(seen)))
        if op == "embedding":
            return {"bytes": _size(case["ids"]) * t + _size(case["wdtype"]) * rows * d + _size(case["dtype"]) * t * d, "flops": t * d}
        written = 2 * rows if case["accumulate"] else v
        return {"bytes": _size(case["ids"]) * t + _size(case["gdtype"]) * t * d + _size(case["dtype"]) * written * d, "flops": 2 * t * d}
    m, d, e, w = case["m"], case["d"], _size(case["stream"]), _size(case["wdtype"])
    weights = case["post"] + case["pre"] + (case["groups"] if case["gate"] != "none" else 0)
    if op == "block_norm":
        return {"bytes": m * d * ((2 * e + 2 if case["y"] else e) + (2 if case["pre"] else 0)) + w * weights * d, "flops": 10 * m * d}
    moved = 2 * e + (e + 2 if case["pre"] else 0) + (4 if case["y"] and (case["post"] or case["gate"] != "none") else 2 if case["y"] else 0)
    return {"bytes": m * d * moved + (w + (8 if case["accumulate"] else 4)) * weights * d, "flops": 25 * m * d}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def d(t):
        return t.to(torch.float64)

    if op == "clip":
        norm = torch.linalg.vector_norm(s["flat"], dtype=torch.float64)
        if not case["clip"]:
            return norm.reshape(1)
        limit = s["max_norm"] * 0.999
        c = limit / (norm + 1e-6) if float(norm) + 1e-6 > limit else torch.ones_like(norm)
        return {"flat": d(s["flat"]) * c, "result": torch.stack([norm, c])}
    if op == "embedding":
        return torch.index_select(d(s["w"]), 0, s["ids"].reshape(-1).to(torch.int64)) * case["scale"]
    if op == "embedding_grad":
        ids = s["ids"].to(torch.int64)
        keep = torch.ones_like(ids, dtype=torch.bool) if s["pad_id"] is None else ids.ne(s["pad_id"])
        out = d(s["dw"]) if case["accumulate"] else torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
        sums = torch.zeros(out.shape, dtype=torch.float64, device="cuda")
        return out + sums.index_add_(0, ids[keep], d(s["dy"])[keep]) * case["scale"]

    def root(a):  # of the mean square
        return torch.sqrt(torch.einsum("md,md->m", a, a) / a.shape[1] + 1e-6)[:, None]

    m, width = case["m"], case["d"]
    gate = None if s["gate_w"] is None else d(s["gate_w"])[:, None, :].expand(-1, m // case["groups"], -1).reshape(m, width)
    if op == "block_norm":
        r, out = d(s["x"]), {}
        if case["y"]:
            u = d(s["yb"])
            if case["post"]:
                u = torch.einsum("md,d->md", u / root(u), d(s["post_w"]))
            r = r * case["scale"] + (u if gate is None else u * gate)
            out["r"] = r
        if case["pre"]:
            out["h"] = torch.einsum("md,d->md", r / root(r), d(s["pre_w"]))
        return out

    def through(a, w, g):
        """Gradient of the norm to a: what is left of g w beside a, over the root."""
        v, q = g * w, root(a)
        along = torch.einsum("md,md->m", v, a)[:, None] / (q * q * a.shape[1])
        return (v - a * along) / q

    out, base = {}, (lambda t: d(t) if case["accumulate"] else 0.0)
    g = d(s["dr"])
    if case["pre"]:
        r = d(s["r"])
        out["pre_grad"] = base(s["pre_grad"]) + torch.einsum("md,md->d", d(s["dh"]), r / root(r))
        g = g + through(r, d(s["pre_w"]), d(s["dh"]))
    out["dx"] = case["scale"] * g
    if case["y"]:
        y = d(s["yb"])
        unit = y / root(y)
        if gate is not None:
            u = unit * d(s["post_w"]) if case["post"] else y
            out["gate_grad"] = base(s["gate_grad"]) + torch.einsum("gld,gld->gd", g.view(case["groups"], -1, width), u.view(case["groups"], -1, width))
            g = g * gate
        if case["post"]:
            out["post_grad"] = base(s["post_grad"]) + torch.einsum("md,md->d", g, unit)
            g = through(y, d(s["post_w"]), g)
        out["dy"] = g
    return out
