"""Cases of the training-step operators around the gradient reduction: the
products that make the gradients (linear layers with their epilogue, forward
and backward) and the optimizer step that consumes the reduced ones
(orthogonalised updates).

Operators and their definitions (all sums in 32 bits or more):

* ``linear``          y = act(x W^T + bias) + residual, optionally storing
                      z = x W^T + bias (the pre-activation).
* ``linear_dgrad``    dx = (dy W + residual) * act'(z).
* ``linear_wgrad``    dW = dy^T x, db = column sums of dy; stored, or added to
                      what the gradient buffers hold.
* ``newton_schulz``   O = p(p(...p(G / (|G|_F + eps)))), five steps of
                      p(X) = a X + (b A + c A^2) X with A = X X^T (or the same
                      on the other side; the polynomial is odd, both agree),
                      in bf16 whatever the gradient's type.
* ``muon_step``       m = mu m + g; u = g + mu m; W = (1 - lr wd) W - lr s O(u)
                      with s = 0.2 sqrt(max(rows, cols)) (an update whose root
                      mean square is near 0.2, for learning rates as AdamW's)
                      or s = sqrt(max(1, rows / cols)) (a spectral norm).

Sizes are those of the 402.8M-parameter tree (width 1024, inner width 4096,
98304 tokens of vocabulary) and of the qwen3-0.6b tree (query width 2048), with
odd and ragged ones between them.
"""
from __future__ import annotations

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu")
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315
NS_STEPS, NS_EPS = 5, 1e-7


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one token of generation through the first MLP product of the 402.8M model
        dict(name="linear 1 token", op="linear", m=1, n=4096, k=1024, act="gelu", bias=True, residual=False,
             preact=False, pad=0),
        # a short ragged prompt through a layer whose sizes fit no tile or 16-byte vector
        dict(name="linear ragged", op="linear", m=333, n=1000, k=777, act="silu", bias=True, residual=True,
             preact=False, pad=0),
        # the first MLP product of a training micro-batch: the pre-activation is kept for backward
        dict(name="linear mlp", op="linear", m=8192, n=4096, k=1024, act="gelu", bias=True, residual=False,
             preact=True, pad=0),
        # the tied output projection over the whole vocabulary
        dict(name="linear vocab", op="linear", m=4096, n=98304, k=1024, act="none", bias=False, residual=False,
             preact=False, pad=0),
        # backward of the second MLP product, with the activation's gradient in its epilogue
        dict(name="dgrad mlp", op="dgrad", m=8192, n=1024, k=4096, act="gelu", residual=False, pad=0),
        # backward of a query projection joining the residual branch's gradient, ragged tokens, strided rows
        dict(name="dgrad residual", op="dgrad", m=1537, n=2048, k=1024, act="none", residual=True, pad=8),
        # weight and bias gradient of a whole micro-batch added to the replica's fp32 accumulator
        dict(name="wgrad accumulate", op="wgrad", m=16384, n=4096, k=1024, dtype="f32", accumulate=True, bias=True,
             pad=0),
        # weight gradient of the ragged layer stored as the bf16 gradient that the bucket flush reads
        dict(name="wgrad ragged", op="wgrad", m=333, n=1000, k=777, dtype="bf16", accumulate=False, bias=True,
             pad=0),
        # one small projection orthogonalised alone: latency
        dict(name="newton_schulz small", op="ns", batch=1, m=128, n=333, dtype="f32"),
        # the square projections of two layers
        dict(name="newton_schulz square", op="ns", batch=8, m=1024, n=1024, dtype="bf16"),
        # one rank's share of the 402.8M tree at 8 ranks: the matrices that it owns, weights in bf16
        dict(name="muon owner share", op="muon", mats="12x1024x1024,3x4096x1024,3x1024x4096", dtype="bf16",
             gdtype="bf16", scale="spectral", lr=0.02, wd=0.01),
        # a few small odd matrices with fp32 weights and gradients, late in a learning-rate schedule
        dict(name="muon small", op="muon", mats="2x100x333,1x257x64", dtype="f32", gdtype="f32", scale="rms",
             lr=1e-4, wd=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "dgrad", "wgrad", "ns", "muon"))
    pad = rng.choice((0, 0, 0, 8, 3))
    if op in ("linear", "dgrad", "wgrad"):
        m, n, k = _log(rng, 1, 16384), _log(rng, 64, 8192), _log(rng, 64, 4096)
        if rng.random() < 0.6:  # most layers' widths are multiples of 64
            n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
        if op == "linear":
            return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS), bias=rng.random() < 0.5,
                        residual=rng.random() < 0.5, preact=rng.random() < 0.5, pad=pad)
        if op == "dgrad":
            return dict(op=op, m=m, n=n, k=k, act=rng.choice(ACTS), residual=rng.random() < 0.5, pad=pad)
        return dict(op=op, m=m, n=n, k=k, dtype=rng.choice(("bf16", "f32")), accumulate=rng.random() < 0.5,
                    bias=rng.random() < 0.5, pad=pad)
    if op == "ns":
        m, n = _log(rng, 16, 2048), _log(rng, 16, 4096)
        most = max(1, min(12, int(3e7 // (m * n))))
        return dict(op=op, batch=rng.randint(1, most), m=m, n=n, dtype=rng.choice(("bf16", "f32")))
    parts = []
    for _ in range(rng.randint(1, 3)):
        m, n = _log(rng, 32, 1536), _log(rng, 32, 1536)
        if rng.random() < 0.5:
            m, n = max(64, m // 64 * 64), max(64, n // 64 * 64)
        parts.append("%dx%dx%d" % (rng.randint(1, 6), m, n))
    scale = rng.choice(("rms", "spectral"))
    return dict(op=op, mats=",".join(parts), dtype=rng.choice(("bf16", "f32")), gdtype=rng.choice(("bf16", "f32")),
                scale=scale, lr=1e-4 if scale == "rms" else 1e-3, wd=rng.choice((0.0, 0.1)))


def _mats(case):
    return [(int(m), int(n)) for c, m, n in (p.split("x") for p in case["mats"].split(",")) for _ in range(int(c))]


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16, pad=0):
        t = torch.randn(*shape[:-1], shape[-1] + pad, device="cuda", generator=gen) * scale
        return t.to(dtype)[..., :shape[-1]]  # with pad, rows of a wider tensor

    def gradient(*shape):
        """A weight gradient: noise with a few strong directions, at the size that backward leaves it."""
        g = torch.randn(*shape, device="cuda", generator=gen)
        r = 4
        u = torch.randn(*shape[:-1], r, device="cuda", generator=gen)
        v = torch.randn(*shape[:-2], r, shape[-1], device="cuda", generator=gen)
        return (g + 1.5 * (u @ v)) * 1e-3

    op = case["op"]
    s = dict(case)
    if op == "linear":
        m, n, k, pad = case["m"], case["n"], case["k"], case["pad"]
        s["x"] = randn(m, k, pad=pad)
        s["w"] = randn(n, k, scale=1.0 / math.sqrt(k))
        s["b"] = randn(n, scale=0.1) if case["bias"] else None
        s["r"] = randn(m, n, pad=pad) if case["residual"] else None
    elif op == "dgrad":
        m, n, k, pad = case["m"], case["n"], case["k"], case["pad"]
        s["dy"] = randn(m, n, scale=1e-3, pad=pad)
        s["w"] = randn(n, k, scale=1.0 / math.sqrt(n))
        s["z"] = randn(m, k, pad=pad) if case["act"] != "none" else None
        s["r"] = randn(m, k, scale=1e-3, pad=pad) if case["residual"] else None
    elif op == "wgrad":
        m, n, k, pad = case["m"], case["n"], case["k"], case["pad"]
        s["dy"] = randn(m, n, scale=1e-3, pad=pad)
        s["x"] = randn(m, k, pad=pad)
        s["dw"] = randn(n, k, scale=1e-2, dtype=_dt(case["dtype"]))
        s["db"] = randn(n, scale=1e-2, dtype=torch.float32) if case["bias"] else None
    elif op == "ns":
        s["g"] = gradient(case["batch"], case["m"], case["n"]).to(_dt(case["dtype"]))
    else:
        mats = _mats(case)
        s["w"] = [randn(m, n, scale=0.02, dtype=_dt(case["dtype"])) for m, n in mats]
        s["mom"] = [gradient(m, n) * 5 for m, n in mats]
        s["grad"] = [gradient(m, n).to(_dt(case["gdtype"])) for m, n in mats]
    return s


# -------------------------------------------------------------------- runs --

def run(s):
    return _OWN[s["op"]](s) if own else _PLAIN[s["op"]](s)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_linear(s):
    z = s["x"].float() @ s["w"].float().T
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.bfloat16()
    return (y, z.bfloat16()) if s["preact"] else y


def _plain_dgrad(s):
    dx = s["dy"].float() @ s["w"].float()
    if s["r"] is not None:
        dx = dx + s["r"].float()
    if s["z"] is not None:
        dx = dx * _act_grad(s["z"].float(), s["act"])
    return dx.bfloat16()


def _plain_wgrad(s):
    dy = s["dy"].float()
    dw, db = dy.T @ s["x"].float(), dy.sum(0) if s["db"] is not None else None
    if s["accumulate"]:
        dw = s["dw"].float() + dw
        db = s["db"] + db if db is not None else None
    s["dw"].copy_(dw)
    if db is None:
        return s["dw"]
    s["db"].copy_(db)
    return s["dw"], s["db"]


def _plain_ns(g):
    """[..., m, n] in 32 bits; the smaller side's product."""
    x = g.float()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        a = x @ x.mT
        x = NS_A * x + (NS_B * a + NS_C * (a @ a)) @ x
    return x.mT if tall else x


def _scale(m, n, rule):
    return 0.2 * math.sqrt(max(m, n)) if rule == "rms" else math.sqrt(max(1.0, m / n))


def _plain_muon(s):
    for w, mom, g in zip(s["w"], s["mom"], s["grad"]):
        g = g.float()
        mom.mul_(0.95).add_(g)
        o = _plain_ns(g + 0.95 * mom)
        w.copy_((1 - s["lr"] * s["wd"]) * w.float() - s["lr"] * _scale(*w.shape, s["scale"]) * o)
    return {"w": s["w"], "mom": s["mom"]}


_PLAIN = {"linear": _plain_linear, "dgrad": _plain_dgrad, "wgrad": _plain_wgrad,
          "ns": lambda s: _plain_ns(s["g"]).bfloat16(), "muon": _plain_muon}


def _own_linear(s):
    import zero_collectives_gb300 as zc
    x, w = s["x"], s["w"]
    z = torch.empty((x.shape[0], w.shape[0]), dtype=torch.bfloat16, device="cuda") if s["preact"] else None
    y = zc.linear(x, w, bias=s["b"], act=s["act"], residual=s["r"], preact=z)
    return (y, z) if z is not None else y


def _own_dgrad(s):
    import zero_collectives_gb300 as zc
    return zc.linear_dgrad(s["dy"], s["w"], preact=s["z"], act=s["act"], residual=s["r"])


def _own_wgrad(s):
    import zero_collectives_gb300 as zc
    zc.linear_wgrad(s["dy"], s["x"], s["dw"], bias_grad=s["db"], accumulate=s["accumulate"])
    return s["dw"] if s["db"] is None else (s["dw"], s["db"])


def _own_ns(s):
    import zero_collectives_gb300 as zc
    return zc.newton_schulz(s["g"])


def _own_muon(s):
    import zero_collectives_gb300 as zc
    zc.muon_step(s["w"], s["mom"], s["grad"], lr=s["lr"], momentum=0.95, weight_decay=s["wd"],
                 scale=s["scale"])
    return {"w": s["w"], "mom": s["mom"]}


_OWN = {"linear": _own_linear, "dgrad": _own_dgrad, "wgrad": _own_wgrad, "ns": _own_ns, "muon": _own_muon}


# -------------------------------------------------------------------- work --

def _ns_flops(m, n):
    """Five steps; X X^T and A^2 are symmetric, so half of each is enough."""
    r, c = min(m, n), max(m, n)
    return NS_STEPS * (r * r * c + r * r * r + 2 * r * r * c)


def work(case):
    op = case["op"]
    if op in ("linear", "dgrad", "wgrad"):
        m, n, k = case["m"], case["n"], case["k"]
        flops = 2 * m * n * k
        if op == "linear":
            outs = 1 + case["residual"] + case["preact"]
            return {"bytes": 2 * (m * k + n * k + outs * m * n) + (2 * n if case["bias"] else 0), "flops": flops}
        if op == "dgrad":
            extra = 1 + case["residual"] + (case["act"] != "none")
            return {"bytes": 2 * (m * n + n * k + extra * m * k), "flops": flops}
        e = 2 if case["dtype"] == "bf16" else 4
        moves = 2 if case["accumulate"] else 1
        return {"bytes": 2 * (m * n + m * k) + moves * (e * n * k + (4 * n if case["bias"] else 0)), "flops": flops}
    if op == "ns":
        b, m, n = case["batch"], case["m"], case["n"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": (e + 2) * b * m * n, "flops": b * _ns_flops(m, n)}
    e = 2 if case["dtype"] == "bf16" else 4
    ge = 2 if case["gdtype"] == "bf16" else 4
    mats = _mats(case)
    return {"bytes": sum((2 * e + 8 + ge) * m * n for m, n in mats), "flops": sum(_ns_flops(m, n) for m, n in mats)}


# ------------------------------------------------------------------- exact --

def _exact_ns(g):
    """The definition in 64 bits, by powers of the Gram matrix on the smaller side."""
    g = g / (torch.linalg.matrix_norm(g, keepdim=True) + NS_EPS)
    left = g.shape[-2] <= g.shape[-1]
    eye = torch.eye(min(g.shape[-2:]), dtype=torch.float64, device=g.device)
    for _ in range(NS_STEPS):
        gram = torch.matmul(g, g.transpose(-2, -1)) if left else torch.matmul(g.transpose(-2, -1), g)
        poly = NS_A * eye + NS_B * gram + NS_C * torch.matmul(gram, gram)
        g = torch.matmul(poly, g) if left else torch.matmul(g, poly)
    return g


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def d(t):
        return t.to(torch.float64)

    def sig(z):
        return torch.special.expit(z)

    if op == "linear":
        z = torch.einsum("mk,nk->mn", d(s["x"]), d(s["w"]))
        if s["b"] is not None:
            z += d(s["b"])[None, :]
        if case["act"] == "relu":
            y = z.clamp(min=0)
        elif case["act"] == "gelu":  # z times the logistic function of twice the tanh form's argument
            y = z * sig(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
        elif case["act"] == "silu":
            y = z * sig(z)
        else:
            y = z
        if s["r"] is not None:
            y = y + d(s["r"])
        return (y, z) if case["preact"] else y
    if op == "dgrad":
        dx = torch.einsum("mn,nk->mk", d(s["dy"]), d(s["w"]))
        if s["r"] is not None:
            dx += d(s["r"])
        if s["z"] is not None:
            z = d(s["z"])
            if case["act"] == "relu":
                dx *= (z > 0)
            elif case["act"] == "gelu":
                q = math.sqrt(8 / math.pi)
                p = sig(q * (z + 0.044715 * z ** 3))
                dx *= p + z * p * (1 - p) * q * (1 + 0.134145 * z ** 2)
            else:
                p = sig(z)
                dx *= p + z * p * (1 - p)
        return dx
    if op == "wgrad":
        dw = torch.einsum("mn,mk->nk", d(s["dy"]), d(s["x"]))
        db = d(s["dy"]).sum(0)
        if case["accumulate"]:
            dw += d(s["dw"])
            db = db + d(s["db"]) if s["db"] is not None else db
        return dw if s["db"] is None else (dw, db)
    if op == "ns":
        return _exact_ns(d(s["g"]))
    w, mom = [], []
    for wi, mi, gi in zip(s["w"], s["mom"], s["grad"]):
        m1 = 0.95 * d(mi) + d(gi)
        o = _exact_ns(d(gi) + 0.95 * m1)
        rows, cols = wi.shape
        size = 0.2 * max(rows, cols) ** 0.5 if case["scale"] == "rms" else max(1.0, rows / cols) ** 0.5
        w.append((1 - case["lr"] * case["wd"]) * d(wi) - case["lr"] * size * o)
        mom.append(m1)
    return {"w": w, "mom": mom}
