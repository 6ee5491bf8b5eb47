"""Measured cases of the normalisation and embedding operators.

Four operators: the layer norm of rows (``norm``), its backward pass with the
reduction of the weight's and the bias's gradient (``norm_grad``), the scaled
embedding lookup (``lookup``) and the gradient of the table from sorted
tokens (``lookup_grad``).  ``run`` computes them either in their plain form
(elementary torch operations in float32) or, with ``own`` set, through the
package's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases

def _norm(op, rows, n, dtype, param, stats=True, gap=0):
    """Rows of n values of `dtype`, weights of type `param`; `gap` values lie
    between two rows (a column range of a wider matrix)."""
    return {"op": op, "rows": rows, "n": n, "dtype": dtype, "param": param, "stats": stats, "gap": gap}


def _lookup(op, tokens, vocab, dim, dtype, ids="i64", spread="zipf", scale=1.0):
    return {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "dtype": dtype, "ids": ids, "spread": spread,
            "scale": scale}


def listed():
    return [
        # one token while text is generated: launch latency
        dict(_norm("norm", 1, 4096, "bf16", "bf16", stats=False), name="norm one token"),
        # a training batch's hidden states, float32 parameters
        dict(_norm("norm", 16384, 4096, "bf16", "f32"), name="norm training"),
        # the matrix of this repository's variance workload
        dict(_norm("norm", 4096, 4096, "f32", "f32"), name="norm square f32"),
        # short rows: one norm per attention head
        dict(_norm("norm", 200000, 128, "bf16", "bf16", stats=False), name="norm per head"),
        # the training batch's backward pass
        dict(_norm("norm_grad", 16384, 4096, "bf16", "f32"), name="norm grad training"),
        # odd row length, rows at odd addresses
        dict(_norm("norm_grad", 5003, 1531, "f16", "f16"), name="norm grad ragged"),
        # few wide rows: a short fine-tuning batch in float32
        dict(_norm("norm_grad", 60, 8192, "f32", "f32"), name="norm grad few rows"),
        # a step of generation for a batch of sequences, scaled by sqrt(dim)
        dict(_lookup("lookup", 48, 64000, 4096, "bf16", spread="uniform", scale=64.0), name="lookup generation"),
        # a training batch's tokens
        dict(_lookup("lookup", 32768, 64000, 4096, "bf16"), name="lookup training"),
        # the table's gradient for a training batch: most rows get no token
        dict(_lookup("lookup_grad", 16384, 64000, 4096, "bf16"), name="lookup grad training"),
        # a byte vocabulary: every row gets hundreds of tokens
        dict(_lookup("lookup_grad", 65536, 256, 512, "f32", ids="i32"), name="lookup grad bytes"),
        # odd sizes, a small batch
        dict(_lookup("lookup_grad", 1001, 5003, 257, "f16", scale=0.5), name="lookup grad ragged"),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _shape(rng, v, step):
    """v, as it is (often odd) or rounded to a multiple of `step`."""
    return v if rng.random() < 0.4 else max(step, v // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "lookup", "lookup_grad"])
    top = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    dtype = rng.choice(["f32", "bf16", "f16"])
    while True:
        if op in ("norm", "norm_grad"):
            case = _norm(op, _log(rng, 1, 200000), _shape(rng, _log(rng, 32, 20000), 64), dtype,
                         rng.choice([dtype, "f32"]), stats=op == "norm_grad" or rng.random() < 0.6,
                         gap=rng.choice([0, 0, 0, 1, 64]))
        else:
            case = _lookup(op, _log(rng, 1, 65536), _log(rng, 100, 130000), _shape(rng, _log(rng, 32, 8192), 64),
                           dtype, ids=rng.choice(["i32", "i64"]), spread=rng.choice(["zipf", "zipf", "uniform"]),
                           scale=rng.choice([1.0, 1.0, 0.125, 22.5]))
        if work(case)["bytes"] <= top:
            return case


def _distinct(case):
    """Expected number of different rows that the tokens name."""
    t, v = case["tokens"], case["vocab"]
    if case["spread"] == "uniform":
        return v * -math.expm1(-t / v)
    ranks = torch.arange(v, dtype=torch.float64)
    p = 1.0 / (ranks + 2.7)
    return float((-torch.expm1(-t * p / p.sum())).sum())


def work(case):
    e = _BYTES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        size, pe = case["rows"] * case["n"], _BYTES[case["param"]]
        if case["op"] == "norm":
            stats = 8 * case["rows"] if case["stats"] else 0
            return {"bytes": 2 * e * size + 2 * pe * case["n"] + stats, "flops": 9 * size}
        return {"bytes": 3 * e * size + 3 * pe * case["n"] + 8 * case["rows"], "flops": 15 * size}
    t, d = case["tokens"], case["dim"]
    idb = t * (4 if case["ids"] == "i32" else 8)
    if case["op"] == "lookup":
        return {"bytes": int(idb + e * d * (t + _distinct(case))), "flops": t * d}
    return {"bytes": idb + e * d * (t + case["vocab"]), "flops": 2 * t * d}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _rows(g, rows, n, gap, dtype, hidden):
    """[rows, n], the row stride n + gap.  `hidden`: hidden states, with an
    offset per row and a few channels far larger than the rest."""
    x = torch.randn(rows, n + gap, generator=g, device="cuda", dtype=torch.float32)
    if hidden:
        channel = torch.rand(n + gap, generator=g, device="cuda").mul_(1.5).add_(0.25)
        channel[torch.rand(n + gap, generator=g, device="cuda") < 0.004] *= 20.0
        x.mul_(channel).add_(torch.randn(rows, 1, generator=g, device="cuda").mul_(0.3))
    return x.to(dtype)[:, :n]


def prepare(case, seed):
    g = _generator(seed)
    dt = _TYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_grad"):
        rows, n, pt = case["rows"], case["n"], _TYPES[case["param"]]
        st = {"case": case, "eps": 1e-5, "x": _rows(g, rows, n, case["gap"], dt, True)}
        st["w"] = (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(pt)
        st["b"] = (0.1 * torch.randn(n, generator=g, device="cuda")).to(pt)
        if case["op"] == "norm_grad":
            st["dy"] = _rows(g, rows, n, 0, dt, False)
            # what the forward pass has left
            x = st["x"].double()
            mean = x.mean(1, keepdim=True)
            st["mean"] = mean[:, 0].float()
            st["rstd"] = ((x - mean).square_().mean(1) + st["eps"]).rsqrt().float()
        return st
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    if case["spread"] == "uniform":
        ids = torch.randint(0, v, (t,), generator=g, device="cuda")
    else:
        # word frequencies fall with the rank; frequent words have low numbers
        p = 1.0 / (torch.arange(v, dtype=torch.float64, device="cuda") + 2.7)
        c = torch.cumsum(p, 0)
        u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64) * c[-1]
        ids = torch.searchsorted(c, u).clamp_(max=v - 1)
    st = {"case": case, "scale": case["scale"], "ids": ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)}
    if case["op"] == "lookup":
        st["table"] = (0.02 * torch.randn(v, d, generator=g, device="cuda")).to(dt)
    else:
        st["dy"] = (0.01 * torch.randn(t, d, generator=g, device="cuda")).to(dt)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import stable_variance_amd as sv

    op = s["case"]["op"]
    if op == "norm":
        return sv.layer_norm(s["x"], s["w"], s["b"], eps=s["eps"], return_stats=s["case"]["stats"])
    if op == "norm_grad":
        return sv.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
    if op == "lookup":
        return sv.embedding(s["ids"], s["table"], scale=s["scale"])
    return sv.embedding_backward(s["dy"], s["ids"], s["case"]["vocab"], scale=s["scale"])


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = ((d * d).mean(1, keepdim=True) + s["eps"]).rsqrt()
        y = (d * rstd * s["w"].float() + s["b"].float()).to(s["x"].dtype)
        return (y, mean[:, 0], rstd[:, 0]) if s["case"]["stats"] else y
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        g = dy * s["w"].float()
        dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
        return (dx.to(s["x"].dtype), (dy * xhat).sum(0).to(s["w"].dtype), dy.sum(0).to(s["w"].dtype))
    ids = s["ids"].long()
    if op == "lookup":
        return (s["table"][ids].float() * s["scale"]).to(s["table"].dtype)
    grad = torch.zeros(s["case"]["vocab"], s["dy"].shape[1], dtype=torch.float32, device="cuda")
    grad.index_add_(0, ids, s["dy"].float())
    return (grad * s["scale"]).to(s["dy"].dtype)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        x, w = s["x"].double(), s["w"].double()
        n = case["n"]
        mean = x.sum(1) / n
        z = x - mean.unsqueeze(1)
        sigma = torch.sqrt((z ** 2).sum(1) / n + s["eps"])
        z /= sigma.unsqueeze(1)
        if op == "norm":
            y = torch.addcmul(s["b"].double(), z, w)
            return (y, mean, 1.0 / sigma) if case["stats"] else y
        dy = s["dy"].double()
        db = dy.sum(0)
        dw = (dy * z).sum(0)
        h = dy * w
        # the derivative of z: the part of h along the ones and along z falls out
        a = h.sum(1, keepdim=True) / n
        c = (h * z).sum(1, keepdim=True) / n
        return (h - a - z * c) / sigma.unsqueeze(1), dw, db
    if op == "lookup":
        return torch.index_select(s["table"].double(), 0, s["ids"].long()) * case["scale"]
    out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    out.index_put_((s["ids"].long(),), s["dy"].double(), accumulate=True)
    return out * case["scale"]
