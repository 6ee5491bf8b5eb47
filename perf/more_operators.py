"""Measured cases of the root-mean-square norm and of the gradients' norm.

Five operators: the root-mean-square norm of rows with the residual's addition
(``rms``), the same with an output in 8 bits and its scales (``rms_fp8``), its
backward pass (``rms_grad``), the norm of a model's gradients as one vector
(``grad_norm``) and their clipping to a largest norm (``clip``).  ``run``
computes them either in their plain form (elementary torch operations in
float32, long sums in float64) or, with ``own`` set, through the package's
entry points.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
_EPS = 1e-6


# ---------------------------------------------------------------- the cases

def _rms(op, rows, n, dtype, param, residual="none", rstd=False, gap=0):
    """Rows of n values of `dtype`, weights of type `param`; `residual`: none,
    or the type of the residual stream (for the backward pass: of the rows
    that were normed, with the gradient of the stream behind them); `gap`
    values lie between two rows of x or dy."""
    return {"op": op, "rows": rows, "n": n, "dtype": dtype, "param": param, "residual": residual, "rstd": rstd,
            "gap": gap}


def _fp8(rows, n, dtype, param, residual="none", to="e4m3", block=128, rstd=False, gap=0):
    """`block`: values that share a scale, 0 for the whole row."""
    return dict(_rms("rms_fp8", rows, n, dtype, param, residual, rstd, gap), to=to, block=block)


def _model(op, vocab, dim, layers, ffn, dtype, param, largest=1.0):
    """Gradients of a model: a table [vocab, dim] and for each layer four
    matrices [dim, dim], two [dim, ffn] and one [ffn, dim] of `dtype`, and two
    norm weights [dim] of type `param`."""
    return {"op": op, "vocab": vocab, "dim": dim, "layers": layers, "ffn": ffn, "dtype": dtype, "param": param,
            "largest": largest}


def listed():
    return [
        # one token while text is generated: launch latency
        dict(_rms("rms", 1, 4096, "bf16", "bf16", "bf16"), name="rms one token"),
        # a training batch's hidden states behind a residual addition, float32 parameters
        dict(_rms("rms", 16384, 4096, "bf16", "f32", "bf16", rstd=True), name="rms training"),
        # short rows: one norm per attention head
        dict(_rms("rms", 200000, 128, "bf16", "bf16"), name="rms per head"),
        # a step of generation for a batch of sequences, for a product in 8 bits
        dict(_fp8(48, 4096, "bf16", "bf16", "bf16"), name="rms fp8 generation"),
        # a batch of prompts
        dict(_fp8(16384, 8192, "bf16", "bf16", "bf16"), name="rms fp8 prompts"),
        # odd row length, one scale per token
        dict(_fp8(5003, 1531, "f16", "f16", block=0), name="rms fp8 ragged"),
        # the training batch's backward pass, with the residual stream's gradient
        dict(_rms("rms_grad", 16384, 4096, "bf16", "f32", "bf16"), name="rms grad training"),
        # odd row length, rows at odd addresses, no residual
        dict(_rms("rms_grad", 5003, 1531, "f16", "f16"), name="rms grad ragged"),
        # a model of the size of a test: launch latency
        dict(_model("grad_norm", 256, 64, 4, 256, "f32", "f32"), name="grad norm small"),
        # three layers and the table of a model in bfloat16
        dict(_model("grad_norm", 64000, 4096, 3, 11000, "bf16", "f32"), name="grad norm model"),
        # the same in float32, clipped
        dict(_model("clip", 64000, 2048, 4, 5504, "f32", "f32"), name="clip model"),
        # odd sizes: tensors at odd addresses
        dict(_model("clip", 5003, 257, 5, 1001, "f16", "f16"), name="clip ragged"),
    ]


def _log(rng, lo, hi):
    """A whole number whose logarithm is uniform."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _shape(rng, v, step):
    """v, as it is (often odd) or rounded to a multiple of `step`."""
    return v if rng.random() < 0.4 else max(step, v // step * step)


def draw(rng):
    op = rng.choice(["rms", "rms_fp8", "rms_grad", "grad_norm", "clip"])
    top = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    dtype = rng.choice(["f32", "bf16", "f16"])
    param = rng.choice([dtype, "f32"])
    while True:
        if op in ("grad_norm", "clip"):
            dim = _shape(rng, _log(rng, 32, 8192), 64)
            case = _model(op, _log(rng, 100, 130000), dim, _log(rng, 1, 40), int(dim * rng.uniform(2.0, 4.0)), dtype,
                          param, largest=rng.choice([1.0, 1.0, 0.25, 100.0]))
        else:
            rows, n = _log(rng, 1, 200000), _shape(rng, _log(rng, 32, 20000), 64)
            residual, gap = rng.choice(["none", dtype, "f32"]), rng.choice([0, 0, 0, 1, 64])
            rstd = rng.random() < 0.5
            if op == "rms_fp8":
                case = _fp8(rows, n, dtype, param, residual, rng.choice(["e4m3", "e4m3", "e5m2"]),
                            rng.choice([128, 128, 0]), rstd, gap)
            else:
                case = _rms(op, rows, n, dtype, param, residual, op == "rms" and rstd, gap)
        if work(case)["bytes"] <= top:
            return case


def _sizes(case):
    """Values of the matrices and of the vectors, tensor by tensor."""
    d, f = case["dim"], case["ffn"]
    matrices = [case["vocab"] * d] + [d * d, d * d, d * d, d * d, d * f, d * f, f * d] * case["layers"]
    return matrices, [d, d] * case["layers"]


def work(case):
    op, e, pe = case["op"], _BYTES[case["dtype"]], _BYTES[case["param"]]
    if op in ("grad_norm", "clip"):
        matrices, vectors = (sum(v) for v in _sizes(case))
        size, passes = matrices * e + vectors * pe, 1 if op == "grad_norm" else 2
        return {"bytes": size * passes, "flops": (2 if op == "grad_norm" else 3) * (matrices + vectors)}
    rows, n = case["rows"], case["n"]
    size = rows * n
    stream = 0 if case["residual"] == "none" else _BYTES[case["residual"]]
    if op == "rms_grad":
        # dy, the rows, dh, and the stream's gradient where there is one
        h = stream or e
        return {"bytes": size * (e + 2 * h + stream) + 2 * pe * n + 4 * rows, "flops": 10 * size}
    stats = 4 * rows if case["rstd"] else 0
    if op == "rms":
        return {"bytes": size * (2 * e + 2 * stream) + pe * n + stats, "flops": 5 * size}
    scales = 4 * rows * (-(-n // case["block"]) if case["block"] else 1)
    return {"bytes": size * (e + 1 + 2 * stream) + pe * n + stats + scales, "flops": 8 * size}


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 6151 + 29)
    return g


def _hidden(g, rows, n, gap, dtype):
    """[rows, n], the row stride n + gap: hidden states, rows of different
    sizes and a few channels far larger than the rest."""
    x = torch.randn(rows, n + gap, generator=g, device="cuda", dtype=torch.float32)
    channel = torch.rand(n + gap, generator=g, device="cuda").mul_(1.5).add_(0.25)
    channel[torch.rand(n + gap, generator=g, device="cuda") < 0.004] *= 20.0
    x.mul_(channel).mul_(torch.randn(rows, 1, generator=g, device="cuda").mul_(0.5).exp_())
    return x.to(dtype)[:, :n]


def _noise(g, rows, n, gap, dtype, scale):
    return torch.randn(rows, n + gap, generator=g, device="cuda").mul_(scale).to(dtype)[:, :n]


def _gradients(g, case):
    """One buffer of all matrices and one of all vectors, as an optimizer
    keeps them, and the tensors: views of them."""
    matrices, vectors = _sizes(case)
    scale = 8.0 / math.sqrt(sum(matrices) + sum(vectors))
    flat = [torch.empty(sum(matrices), dtype=_TYPES[case["dtype"]], device="cuda"),
            torch.empty(sum(vectors), dtype=_TYPES[case["param"]], device="cuda")]
    views = [v for f, sizes in zip(flat, (matrices, vectors)) for v in f.split(sizes)]
    level = torch.randn(len(views), generator=g, device="cuda").mul_(0.4).exp_().mul_(scale)
    for v, s in zip(views, level):
        at = 0
        while at < v.numel():  # in parts, so that float32 values of the whole table are never held
            part = v[at:at + (1 << 26)]
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(s))
            at += 1 << 26
    return flat, views


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op in ("grad_norm", "clip"):
        flat, views = _gradients(g, case)
        st = {"case": case, "flat": flat, "grads": views}
        if op == "clip":
            st["out_flat"] = [torch.empty_like(f) for f in flat]
            st["out"] = [v for f, sizes in zip(st["out_flat"], _sizes(case)) for v in f.split(sizes)]
        return st
    rows, n, dt = case["rows"], case["n"], _TYPES[case["dtype"]]
    stream = None if case["residual"] == "none" else _TYPES[case["residual"]]
    st = {"case": case, "w": (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(_TYPES[case["param"]])}
    if op == "rms_grad":
        st["h"] = _hidden(g, rows, n, 0, stream or dt)
        st["dy"] = _noise(g, rows, n, case["gap"], dt, 0.01)
        st["dsum"] = _noise(g, rows, n, 0, stream, 0.01) if stream else None
        # what the forward pass has left
        st["rstd"] = (st["h"].double().square_().mean(1) + _EPS).rsqrt_().float()
        return st
    st["x"] = _noise(g, rows, n, case["gap"], dt, 0.5) if stream else _hidden(g, rows, n, case["gap"], dt)
    st["residual"] = _hidden(g, rows, n, 0, stream) if stream else None
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import stable_variance_amd as sv

    case = s["case"]
    op = case["op"]
    if op == "rms":
        return sv.rms_norm(s["x"], s["w"], eps=_EPS, residual=s["residual"], return_rstd=case["rstd"])
    if op == "rms_fp8":
        return sv.rms_norm_fp8(s["x"], s["w"], eps=_EPS, residual=s["residual"], dtype=_FP8[case["to"]],
                               block=case["block"] or None, return_rstd=case["rstd"])
    if op == "rms_grad":
        return sv.rms_norm_backward(s["dy"], s["h"], s["rstd"], s["w"], s["dsum"])
    if op == "grad_norm":
        return sv.grad_norm(s["grads"])
    norm = sv.clip_grad_norm(s["grads"], case["largest"], out=s["out"])[1]
    return s["out_flat"][0], s["out_flat"][1], norm


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("grad_norm", "clip"):
        # all tensors of a type are one buffer: one operation instead of one per tensor
        a, b = s["flat"]
        total = a.float().square().sum(dtype=torch.float64) + b.float().square().sum(dtype=torch.float64)
        norm = total.sqrt()
        if op == "grad_norm":
            return norm.float()
        k = (case["largest"] / (norm + 1e-6)).clamp(max=1.0).float()
        p, q = s["out_flat"]
        p.copy_(a.float() * k)
        q.copy_(b.float() * k)
        return p, q, norm.float()
    w = s["w"].float()
    if op == "rms_grad":
        h, r = s["h"].float(), s["rstd"][:, None]
        dy = s["dy"].float()
        xhat = h * r
        g = dy * w
        dh = (g - xhat * (g * xhat).mean(1, keepdim=True)) * r
        if s["dsum"] is not None:
            dh = dh + s["dsum"].float()
        return dh.to(s["h"].dtype), (dy * xhat).sum(0).to(s["w"].dtype)
    out = []
    h = s["x"]
    if s["residual"] is not None:
        h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
        out = [h]
    f = h.float()
    rstd = ((f * f).mean(1, keepdim=True) + _EPS).rsqrt()
    if case["rstd"]:
        out = out + [rstd[:, 0]]
    y = f * rstd * w
    if op == "rms":
        y = y.to(s["x"].dtype)
        return (y, *out) if out else y
    rows, n, block = case["rows"], case["n"], case["block"] or case["n"]
    largest = _LARGEST[case["to"]]
    blocks = -(-n // block)
    padded = torch.nn.functional.pad(y, (0, blocks * block - n)).view(rows, blocks, block)
    scale = (padded.abs().amax(2) / largest).clamp(min=2.0 ** -126)
    q = (padded / scale[:, :, None]).clamp(-largest, largest).view(rows, blocks * block)[:, :n].contiguous()
    return (q.to(_FP8[case["to"]]), scale, *out)


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("grad_norm", "clip"):
        squares = []
        for v in s["grads"]:
            squares += [torch.dot(p.double(), p.double()) for p in v.split(1 << 26)]
        norm = torch.stack(squares).sum().sqrt()
        if op == "grad_norm":
            return norm
        k = min(1.0, case["largest"] / (float(norm) + 1e-6))
        return [f.double() * k for f in s["flat"]] + [norm]
    w, n = s["w"].double(), case["n"]
    if op == "rms_grad":
        h, dy = s["h"].double(), s["dy"].double()
        z = h * s["rstd"].double().unsqueeze(1)
        dw = (dy * z).sum(0)
        dy *= w
        # the derivative of z: the part of dy * w along z falls out
        c = (dy * z).sum(1) / n
        dh = torch.addcmul(dy, z, c.unsqueeze(1), value=-1.0) * s["rstd"].double().unsqueeze(1)
        return dh if s["dsum"] is None else dh + s["dsum"].double(), dw
    out = []
    h = s["x"].double()
    if s["residual"] is not None:
        h += s["residual"].double()
        out.append(h)
        h = h.to(s["residual"].dtype).double()  # what is normed is the sum as it is kept
    sigma = torch.sqrt(torch.linalg.vecdot(h, h) / n + _EPS)
    if case["rstd"]:
        out.append(1.0 / sigma)
    y = h * w / sigma.unsqueeze(1)
    if op == "rms":
        return (y, *out) if out else y
    # the values that the 8 bits stand for, before they are rounded to them
    block, largest = case["block"] or n, _LARGEST[case["to"]]
    scales = torch.stack([p.abs().amax(1) for p in y.split(block, 1)], 1) / largest
    each = torch.repeat_interleave(scales, block, 1)[:, :n]
    return (y / each, scales, *out)
