"""Root-mean-square norm on the GPU against its formulas in float64.

Tolerances are bounds on rounding, with u = 2^-24 and u_T half a step of the
result's type.  The squares are summed in double, so rstd is off by its own
rounding alone (u, and 2^-150 where it is subnormal); y takes two products
more.  A sum of n terms in float32 added pairwise is off by at most
(log2 n + 2) u of the sum of their magnitudes.
"""
import math

import pytest
import torch

import stable_variance_amd as sv

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
TYPES = [F32, BF16, F16]
IDS = {F32: "f32", BF16: "bf16", F16: "f16", None: "none", E4M3: "e4m3", E5M2: "e5m2"}
# half of the smallest step near zero
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}
LARGEST = {E4M3: 448.0, E5M2: 57344.0}
# x's type and the residual's (None: no residual)
STREAMS = [(t, s) for t in TYPES for s in dict.fromkeys((None, t, F32))]
STREAM_IDS = [f"{IDS[t]}-{IDS[s]}" for t, s in STREAMS]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from stable_variance_amd import build as libbuild

    if libbuild.is_stale():
        libbuild.build()
    return torch.device("cuda:0")


def half(t):
    return torch.finfo(t).eps / 2


def close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float(((got - want).abs() / tol)[bad].nan_to_num(float('inf')).max()):.3g} of the tolerance"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def hidden(rows, n, dtype, seed, ld=None, scale=1.0):
    g = gen(seed)
    x = torch.randn(rows, ld or n, generator=g, device="cuda") * (0.5 + torch.rand(ld or n, generator=g, device="cuda"))
    return (x * scale).to(dtype)[:, :n]


def weights(n, dtype, seed):
    return (1 + 0.3 * torch.randn(n, generator=gen(1000 + seed), device="cuda")).to(dtype)


# ---------------------------------------------------------------- forward

def reference(x, w, eps, residual):
    """h (in its type), H, R, Y in float64."""
    h = x if residual is None else (x.double() + residual.double()).to(residual.dtype)
    H = h.double()
    R = ((H * H).sum(-1, keepdim=True) / x.shape[-1] + eps) ** -0.5
    return h, H, R, H * R * (1.0 if w is None else w.double())


def check_forward(x, w, eps=1e-6, residual=None):
    out = sv.rms_norm(x, w, eps=eps, residual=residual, return_rstd=True)
    y, rstd = out[0], out[-1]
    h, H, R, Y = reference(x, w, eps, residual)
    assert y.dtype == x.dtype and y.shape == x.shape and y.is_contiguous()
    assert rstd.dtype == F32 and rstd.shape == x.shape[:-1]
    if residual is None:
        assert len(out) == 2
    else:
        assert out[1].dtype == residual.dtype and torch.equal(out[1], h) and out[1].is_contiguous()
    W = 1.0 if w is None else w.double().abs()
    close(rstd, R[..., 0], 1.001 * U * R[..., 0] + 2.0 ** -150, "rstd")
    close(y, Y, (half(x.dtype) + 4 * U) * Y.abs() + TINY[x.dtype] + 2.0 ** -149 * (W * H.abs() + W + 1), "y")
    return out


LENGTHS = [1, 2, 3, 5, 7, 8, 9, 31, 63, 64, 65, 100, 127, 128, 129, 192, 255, 256, 257, 300, 384, 511, 512, 513, 768,
           1000, 1023, 1024, 1025, 1531, 2047, 2048, 2050, 4095, 4096, 4104, 5000, 5003, 6144, 8191, 8192, 8200, 12288,
           12290, 14000, 16384, 16385, 20001, 32768, 32776, 33000, 70001]


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
def test_lengths(dev, dtype, stream):
    for i, n in enumerate(LENGTHS):
        print("rms", IDS[dtype], IDS[stream], n, flush=True)
        rows = 3 + i % 5
        residual = None if stream is None else hidden(rows, n, stream, 300 + i, scale=2.0)
        check_forward(hidden(rows, n, dtype, i), weights(n, dtype if i % 2 else F32, i), residual=residual)


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
@pytest.mark.parametrize("rows", [1, 2, 255, 1025, 40000])
def test_rows(dev, dtype, stream, rows):
    for n in (24, 200, 1100):
        residual = None if stream is None else hidden(rows, n, stream, 7)
        check_forward(hidden(rows, n, dtype, rows), weights(n, dtype, n), residual=residual)


def test_shapes_and_weights(dev):
    x, r = hidden(30, 40, BF16, 1), hidden(30, 40, BF16, 2)
    w = weights(40, F32, 3)
    check_forward(x, None)
    check_forward(x, None, residual=r)
    check_forward(x.reshape(2, 3, 5, 40), w, residual=r.float().reshape(2, 3, 5, 40))
    one = check_forward(x[0], w)  # one row, no leading dimension
    assert one[1].shape == ()
    y, h, rstd = check_forward(x, w, residual=r)
    assert torch.equal(sv.rms_norm(x, w, residual=r)[0], y)
    assert torch.equal(sv.rms_norm(h, w), y)  # the norm is of the sum as it was written
    check_forward(x, w, eps=0.5, residual=r)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_range(dev, dtype):
    # no square is beyond the range or below it
    big = 1e4 if dtype == F16 else 1e37
    for n in (5, 128, 1531, 4096, 33000):
        w = weights(n, F32, n)
        x = hidden(6, n, F32, n)
        x = x / x.abs().amax()
        scale = torch.tensor([1.0, big, 3 * big, 1e-3, 1e-6, 1.0], device=dev)[:, None]
        check_forward((x * scale).to(dtype), w, eps=0.0)
        check_forward((x * scale).to(dtype), w)
    tiny = (x * 1e-35).to(BF16)
    check_forward(tiny, w, eps=0.0)
    check_forward((x * 3e-37).float(), w, eps=0.0)  # the smaller values are subnormal
    top = torch.full((2, 700), torch.finfo(F32).max, device=dev)
    y, rstd = check_forward(top, None)
    assert rstd.isfinite().all() and ((y - 1).abs() < 1e-5).all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_strides_give_the_same_bits(dev, dtype):
    for n, ld in ((96, 100), (96, 97), (1000, 1003), (1531, 1531), (4096, 4104), (130, 131), (40000, 40001)):
        w = weights(n, dtype, n)
        x, r = hidden(7, n, dtype, n, ld=ld), hidden(7, n, F32, n + 1, ld=ld)
        got = check_forward(x, w, residual=r)
        dense = sv.rms_norm(x.contiguous(), w, residual=r.contiguous(), return_rstd=True)
        assert all(torch.equal(p, q) for p, q in zip(got, dense)), (n, ld)
        # the same rows one value further on: another alignment
        shifted = torch.empty(7 * n + 1, dtype=dtype, device=dev)[1:].view(7, n).copy_(x)
        assert torch.equal(sv.rms_norm(shifted, w, residual=r)[0], got[0])
        xt = x.t().contiguous().t()  # last dimension not contiguous: copied
        assert torch.equal(sv.rms_norm(xt, w, residual=r)[0], got[0])
    row = hidden(1, 64, dtype, 1)
    w = weights(64, dtype, 2)
    assert torch.equal(sv.rms_norm(row.expand(5, 64), w), sv.rms_norm(row.repeat(5, 1), w))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_row_is_independent_of_its_batch(dev, dtype):
    for n in (3, 17, 128, 1531, 4096, 9000, 40000):
        x, r = hidden(70, n, dtype, n), hidden(70, n, dtype, n + 1)
        w = weights(n, dtype, n)
        whole = sv.rms_norm(x, w, residual=r, return_rstd=True)
        again = sv.rms_norm(x, w, residual=r, return_rstd=True)
        assert all(torch.equal(p, q) for p, q in zip(whole, again))
        for i in (0, 1, 33, 69):
            one = sv.rms_norm(x[i:i + 1], w, residual=r[i:i + 1], return_rstd=True)
            assert all(torch.equal(p[i:i + 1], q) for p, q in zip(whole, one)), (n, i)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_zeros_nan_and_inf(dev, dtype):
    for n in (1, 6, 300, 1531, 4096, 40000):
        w = weights(n, F32, n)
        zero = torch.zeros(3, n, dtype=dtype, device=dev)
        for eps in (1e-6, 8.6e-78, 1e-200, 5e-324):
            y, rstd = sv.rms_norm(zero, w, eps=eps, return_rstd=True)
            assert (y == 0).all()
            want = min(float(torch.tensor(float(torch.tensor(eps, dtype=torch.float64) ** -0.5)).float()),
                       torch.finfo(F32).max)
            assert (rstd == want).all(), (eps, rstd, want)
        assert sv.rms_norm(zero, w, eps=0.0).isnan().all()
        x = hidden(8, n, dtype, n).clone()
        clean = sv.rms_norm(x, w)
        x[1, 0] = float("nan")
        x[3, n - 1] = float("inf")
        x[6, n // 2] = float("-inf")
        y = sv.rms_norm(x, w)
        good = [0, 2, 4, 5, 7]
        assert torch.equal(y[good], clean[good])
        assert y[1].isnan().all()
        for r, at in ((3, n - 1), (6, n // 2)):
            rest = torch.ones(n, dtype=torch.bool, device=dev)
            rest[at] = False
            assert y[r, at].isnan() and (y[r][rest] == 0).all()


def test_empty(dev):
    y, rstd = sv.rms_norm(torch.empty(3, 0, device=dev), return_rstd=True)
    assert y.shape == (3, 0) and rstd.isnan().all()
    w = weights(5, F32, 1)
    e = torch.empty(0, 5, device=dev)
    y, h, rstd = sv.rms_norm(e, w, residual=e, return_rstd=True)
    assert y.shape == h.shape == (0, 5) and rstd.shape == (0,)
    dh, dw = sv.rms_norm_backward(y, h, rstd, w)
    assert dh.shape == (0, 5) and torch.equal(dw, torch.zeros_like(w))
    z, s = torch.empty(3, 0, device=dev), torch.zeros(3, device=dev)
    dh, dw = sv.rms_norm_backward(z, z, s)
    assert dh.shape == (3, 0) and dw.shape == (0,)
    for block, blocks in ((128, 0), (None, 1)):
        q, scale, rstd = sv.rms_norm_fp8(z, block=block, return_rstd=True)
        assert q.shape == (3, 0) and scale.shape == (3, blocks) and rstd.isnan().all()
        assert (scale == 2.0 ** -126).all()
        q, scale = sv.rms_norm_fp8(e, block=block)
        assert q.shape == (0, 5) and scale.shape == (0, 1)


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
def test_empty_batches_of_every_type(dev, dtype, stream):
    for shape in ((0, 5), (0, 4096), (2, 0, 8), (3, 0), (0,), (0, 0)):
        x = torch.empty(shape, dtype=dtype, device=dev)
        r = None if stream is None else torch.empty(shape, dtype=stream, device=dev)
        w = weights(shape[-1], F32, 1)
        out = sv.rms_norm(x, w, residual=r, return_rstd=True)
        assert out[0].shape == shape and out[0].dtype == dtype and out[-1].shape == shape[:-1]
        assert r is None or (out[1].shape == shape and out[1].dtype == stream)
        for block, blocks in ((128, -(-shape[-1] // 128)), (None, 1)):
            q = sv.rms_norm_fp8(x, w, residual=r, block=block)
            assert q[0].shape == shape and q[1].shape == shape[:-1] + (blocks,)
        h = x if r is None else out[1]
        dh, dw = sv.rms_norm_backward(out[0], h, out[-1], w, h)
        assert dh.shape == shape and dh.dtype == h.dtype and torch.equal(dw, torch.zeros_like(w))
        leaves = [t.clone().requires_grad_() for t in (x, w) + (() if r is None else (r,))]
        y = sv.rms_norm(leaves[0], leaves[1], residual=None if r is None else leaves[2])
        (y if r is None else y[0] + y[1]).sum().backward()
        assert all(t.grad.shape == t.shape and (t.grad == 0).all() for t in leaves)


def test_rows_far_apart(dev):
    ld = (1 << 30) + 8  # the third row starts beyond 2^31 values
    x = torch.empty(3, ld, dtype=BF16, device=dev)[:, :1000]
    x.copy_(hidden(3, 1000, BF16, 5))
    w = weights(1000, BF16, 5)
    y, h, rstd = check_forward(x, w, residual=x)
    dy = hidden(3, 1000, BF16, 6)
    got = sv.rms_norm_backward(dy, x, rstd, w, x)
    want = sv.rms_norm_backward(dy, x.contiguous(), rstd, w, x.contiguous())
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    a, b = sv.rms_norm_fp8(x, w), sv.rms_norm_fp8(x.contiguous(), w)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- 8 bits

def check_fp8(x, w, dtype, block, eps=1e-6, residual=None):
    out = sv.rms_norm_fp8(x, w, eps=eps, residual=residual, dtype=dtype, block=block, return_rstd=True)
    q, scale, rstd = out[0], out[1], out[-1]
    n = x.shape[-1]
    h, _, R, Y = reference(x, w, eps, residual)
    assert q.dtype == dtype and q.shape == x.shape and q.is_contiguous() and scale.dtype == F32
    if residual is None:
        assert len(out) == 3
    else:
        assert torch.equal(out[2], h)
    close(rstd, R[..., 0], 1.001 * U * R[..., 0] + 2.0 ** -150, "rstd")
    size, blocks = (n, 1) if block is None else (block, -(-n // block))
    assert scale.shape == x.shape[:-1] + (blocks,)
    Y = torch.nn.functional.pad(Y, (0, blocks * size - n)).unflatten(-1, (blocks, size))
    M = LARGEST[dtype]
    S = (Y.abs().amax(-1) / M).clamp(min=2.0 ** -126)
    # y's three roundings and the division's
    close(scale, S, 5 * U * S + 2.0 ** -149, "scale")
    # y / scale is off by 3 + 4 + 2 roundings before its last (and by what a
    # subnormal y has lost): q is the value nearest to one that is no further off
    V, S = Y / S[..., None], S[..., None]
    ends = [(V + d * (12 * U * V.abs() + 2.0 ** -148 / S)).float().clamp(-M, M).to(dtype).float().flatten(-2)[..., :n]
            for d in (-1, 1)]
    lo, hi = torch.minimum(*ends), torch.maximum(*ends)
    f = q.float()
    bad = ~((f >= lo) & (f <= hi))
    assert not bad.any(), f"q: {int(bad.sum())} of {bad.numel()} off"
    return out


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
@pytest.mark.parametrize("block", [128, None])
def test_fp8_lengths(dev, dtype, stream, block):
    for i, n in enumerate(LENGTHS):
        print("fp8", IDS[dtype], IDS[stream], block, n, flush=True)
        rows = 3 + i % 5
        residual = None if stream is None else hidden(rows, n, stream, 300 + i, scale=2.0)
        check_fp8(hidden(rows, n, dtype, i), weights(n, dtype if i % 2 else F32, i), E4M3 if i % 3 else E5M2, block,
                  residual=residual)


@pytest.mark.parametrize("to", [E4M3, E5M2], ids=IDS.get)
def test_fp8_rows_and_range(dev, to):
    for rows in (1, 2, 255, 1025, 40000):
        for n in (24, 200, 1100):
            for block in (128, None):
                check_fp8(hidden(rows, n, BF16, rows), weights(n, BF16, n), to, block, residual=hidden(rows, n, BF16, 3))
    w = weights(600, F32, 1)
    x = hidden(9, 600, F32, 2) * 10.0 ** torch.arange(-4, 5, device=dev)[:, None]
    x[:, 5] = 1e-3 * x[:, 5]
    for block in (128, None):
        check_fp8(x, w, to, block, eps=0.0)
        check_fp8(x * 1e-20, w * 1e-12, to, block)  # scales near the smallest normal number and below
        check_fp8(x, w * 1e-37, to, block)
        check_fp8(x, w * 1e30, to, block)
    # the norm's values are the quantised ones, up to the rounding of 8 bits
    q, scale = sv.rms_norm_fp8(x, w, dtype=to)
    y = sv.rms_norm(x, w)
    back = q.float() * scale.repeat_interleave(128, -1)[:, :600]
    step = half(to)
    assert ((back - y).abs() <= 1.0001 * step * y.abs() + scale.repeat_interleave(128, -1)[:, :600] * 2.0 ** -10).all()


def test_fp8_strides_batches_and_repeats(dev):
    for n, ld in ((96, 97), (1000, 1003), (4096, 4104), (1531, 1531), (40000, 40001)):
        for block in (128, None):
            w = weights(n, F32, n)
            x, r = hidden(40, n, F16, n, ld=ld), hidden(40, n, F16, n + 1)
            a = check_fp8(x, w, E4M3, block, residual=r)
            b = sv.rms_norm_fp8(x.contiguous(), w, residual=r, block=block, return_rstd=True)
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))
            for i in (0, 13, 39):
                c = sv.rms_norm_fp8(x[i:i + 1], w, residual=r[i:i + 1], block=block, return_rstd=True)
                assert all(torch.equal(p[i:i + 1].contiguous().view(torch.uint8), q.view(torch.uint8))
                           for p, q in zip(a, c)), (n, block, i)


def test_fp8_zeros_nan_and_inf(dev):
    for to in (E4M3, E5M2):
        for n in (1, 100, 300, 1531, 4096, 40000):
            x = hidden(6, n, F32, n).clone()
            x[0] = 0.0
            clean = sv.rms_norm_fp8(x, dtype=to)
            assert (clean[0][0].float() == 0).all() and (clean[1][0] == 2.0 ** -126).all()
            x[2, n // 2] = float("nan")
            x[4, n // 3] = float("inf")
            q, scale = sv.rms_norm_fp8(x, dtype=to)
            good = [0, 1, 3, 5]
            assert torch.equal(q[good].view(torch.uint8), clean[0][good].view(torch.uint8))
            assert torch.equal(scale[good], clean[1][good])
            assert q[2].float().isnan().all() and scale[2].isnan().all()
            # the row's other values are 0: blocks without the Inf hold zeros
            at = n // 3
            assert q[4, at].float().isnan() and scale[4, at // 128].isnan()
            rest = torch.arange(n, device=dev) // 128 != at // 128
            assert (q[4][rest].float() == 0).all()
            # a weight that is NaN or Inf: its block alone
            w = torch.ones(n, device=dev)
            w[at] = float("inf")
            x = hidden(2, n, F32, n + 1)
            q, scale = sv.rms_norm_fp8(x, w, dtype=to)
            same = sv.rms_norm_fp8(x, dtype=to)
            assert q[:, at].float().isnan().all() and (scale[:, at // 128] == float("inf")).all()
            assert torch.equal(q[:, rest].view(torch.uint8), same[0][:, rest].view(torch.uint8))
            inside = ~rest
            inside[at] = False
            assert (q[:, inside].float() == 0).all()
            w[at] = float("nan")
            q, scale = sv.rms_norm_fp8(x, w, dtype=to)
            assert q[:, ~rest].float().isnan().all() and scale[:, at // 128].isnan().all()
            assert torch.equal(q[:, rest].view(torch.uint8), same[0][:, rest].view(torch.uint8))


def test_fp8_every_code(dev):
    # a row whose norm runs through every value of the type: each is its own
    # nearest, up to what the scale's rounding moves
    for to in (E4M3, E5M2):
        codes = torch.arange(256, dtype=torch.uint8, device=dev).view(to).float()
        codes = codes[codes.isfinite()]
        x = codes[None, :128].contiguous()
        x[0, 0] = LARGEST[to]
        for block in (128, None):
            check_fp8(x, None, to, block)
            check_fp8(codes[None], None, to, block)


# ---------------------------------------------------------------- backward

def check_backward(h, dy, w, dsum=None, eps=1e-6, param=None, rstd=None, **kw):
    n = h.shape[-1]
    if rstd is None:
        rstd = sv.rms_norm(h, eps=eps, return_rstd=True)[1]
    dh, dw = sv.rms_norm_backward(dy, h, rstd, w, dsum, param_dtype=param, **kw)
    R = rstd.double().reshape(-1, 1)
    G, X = dy.double().reshape(-1, n), h.double().reshape(-1, n) * R
    g = G * w.double() if w is not None else G
    c = (g * X).mean(1, keepdim=True)
    D = 0.0 if dsum is None else dsum.double().reshape(-1, n)
    DH = R * (g - X * c) + D
    # c: three roundings of each product and those of the sum, log2 n deep;
    # then one of g, three of xhat * c, and the difference's, the product's and
    # the last sum's of their own results
    k = (math.ceil(math.log2(max(n, 2))) + 8) * U
    mag = R * (4 * U * g.abs() + X.abs() * (k * (g * X).abs().mean(1, keepdim=True) + 4 * U * c.abs()))
    assert dh.dtype == h.dtype and dh.shape == h.shape and dh.is_contiguous()
    close(dh.reshape(-1, n), DH, (half(h.dtype) + 2 * U) * DH.abs() + TINY[h.dtype] + mag, "dh")
    if dw is not None:
        pt = param or (w.dtype if w is not None else F32)
        DW, S = (G * X).sum(0), (G * X).abs().sum(0)
        assert dw.dtype == pt
        # column sums: two roundings a term, runs of at most 48, joined with
        # compensation
        close(dw, DW, (half(pt) + 2 * U) * DW.abs() + TINY[pt] + 52 * U * S, "dweight")
    return dh, dw


# dy's type, h's type
PAIRS = [(F32, F32), (BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)]
PAIR_IDS = [f"{IDS[a]}-{IDS[b]}" for a, b in PAIRS]


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("with_sum", [False, True])
def test_grad_lengths(dev, dtype, stream, with_sum):
    for i, n in enumerate(LENGTHS):
        print("rms grad", IDS[dtype], IDS[stream], with_sum, n, flush=True)
        rows = 2 + i % 7
        dsum = hidden(rows, n, stream, 900 + i) if with_sum else None
        check_backward(hidden(rows, n, stream, i), hidden(rows, n, dtype, 500 + i), weights(n, dtype if i % 2 else F32, i),
                       dsum)


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 300, 1025, 4097, 70000])
def test_grad_rows(dev, dtype, stream, rows):
    for i, n in enumerate((24, 200, 1100)):
        if rows * n > 20_000_000:
            continue
        dsum = hidden(rows, n, stream, 3) if i % 2 else None
        check_backward(hidden(rows, n, stream, rows), hidden(rows, n, dtype, rows + 1), weights(n, dtype, n), dsum)


def test_grad_options(dev):
    h, dy, dsum = hidden(50, 72, BF16, 1), hidden(50, 72, BF16, 2), hidden(50, 72, BF16, 3)
    w = weights(72, F32, 1)
    full = check_backward(h, dy, w, dsum)
    dh, dw = check_backward(h, dy, w, dsum, weight_grad=False)
    assert dw is None and torch.equal(dh, full[0])
    check_backward(h, dy, None)
    check_backward(h, dy, None, dsum, param=BF16)
    check_backward(h, dy, w.to(BF16))
    check_backward(h.float(), dy, w.to(BF16), dsum.float())
    three = [t.reshape(5, 10, 72) for t in (h, dy, dsum)]
    got = check_backward(three[0], three[1], w, three[2])
    assert torch.equal(got[0].reshape(50, 72), full[0]) and torch.equal(got[1], full[1])
    # rows of very different sizes, and rstd as eps alone makes it
    scale = torch.tensor([1e-6, 1.0, 1e4, 30.0, 0.0], device=dev).repeat(10)[:, None]
    check_backward((h * scale).to(BF16), dy, w, dsum)
    check_backward(h.float() * scale * 1e25, dy.float(), w)


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
def test_grad_strides_and_repeats_give_the_same_bits(dev, dtype, stream):
    for n, ld in ((96, 97), (1000, 1003), (1531, 1531), (4096, 4104), (40000, 40001)):
        w = weights(n, dtype, n)
        h, dy, dsum = (hidden(67, n, t, n + i, ld=ld) for i, t in enumerate((stream, dtype, stream)))
        got = check_backward(h, dy, w, dsum)
        dense = check_backward(h.contiguous(), dy.contiguous(), w, dsum.contiguous())
        assert all(torch.equal(p, q) for p, q in zip(got, dense)), (n, ld)
        one = check_backward(h[5:6], dy[5:6], w, dsum[5:6])  # dh of a row does not depend on the batch
        assert torch.equal(one[0], got[0][5:6])
    g = torch.ones((), dtype=dtype, device=dev).expand(67, 40000)  # every stride 0
    a = check_backward(h, g, w)
    b = check_backward(h, g.contiguous(), w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_grad_nan_stays_in_its_row(dev):
    for n in (40, 1531, 4096, 40000):
        h, dy = hidden(6, n, F32, 1).clone(), hidden(6, n, F32, 2)
        rstd = sv.rms_norm(h, return_rstd=True)[1]
        clean = sv.rms_norm_backward(dy, h, rstd)[0]
        h[2, n // 2] = float("nan")
        rstd = sv.rms_norm(h, return_rstd=True)[1]
        dh, dw = sv.rms_norm_backward(dy, h, rstd)
        keep = [0, 1, 3, 4, 5]
        assert dh[2].isnan().all() and torch.equal(dh[keep], clean[keep])
        assert dw.isnan().all()


def test_gradients_against_differences(dev):
    # the directional derivative of sum(dy * y) + sum(dsum * h) along v, by
    # central differences of the forward call with steps d and 2d.  Truncation:
    # the difference of the two quotients is three times the leading d^2 term of
    # the first, so it bounds it.  Rounding: each y is off by 4 u of itself
    # (|y| <= sqrt(n) |w| < 10 |w|), each h by u of itself (|h| < 16 here).
    n, rows, d = 96, 7, 2.0 ** -5
    x, r, dy, dsum = (hidden(rows, n, F32, 11 + i) for i in range(4))
    w = weights(n, F32, 13)
    y, h, rstd = sv.rms_norm(x, w, residual=r, return_rstd=True)
    dh, dw = sv.rms_norm_backward(dy, h, rstd, w, dsum)

    def loss(x_, w_, r_):
        y_, h_ = sv.rms_norm(x_, w_, residual=r_)
        return float((y_.double() * dy.double()).sum() + (h_.double() * dsum.double()).sum())

    assert float(h.abs().max()) < 15
    noise = U * float((dy.double().abs() * w.double().abs() * 40).sum() + 16 * dsum.double().abs().sum())
    for i, g in enumerate((dh, dw, dh)):
        v = torch.randn(g.shape, generator=gen(20 + i), device=dev)

        def quotient(step):
            up, down = [x, w, r], [x, w, r]
            up[i], down[i] = up[i] + step * v, down[i] - step * v
            real = float(((up[i].double() - down[i].double()) * g.double()).sum())
            return loss(*up) - loss(*down), real

        d1, r1 = quotient(d)
        d2, r2 = quotient(2 * d)
        # the gradient itself: dh and dw within 32 u of their terms
        own = 64 * U * d * float((v.double().abs() * (g.double().abs() + 1) * 10).sum())
        assert abs(d1 - r1) <= abs((d2 / 2 - r2 / 2) - (d1 - r1)) + 2 * noise + own, (i, d1, r1)


# ---------------------------------------------------------------- autograd

def test_autograd(dev):
    for dtype, stream in PAIRS:
        x, r, dy, dsum = (hidden(20, 136, t, i) for i, t in enumerate((dtype, stream, dtype, stream)))
        w = weights(136, F32, 1)
        _, h, rstd = sv.rms_norm(x, w, residual=r, return_rstd=True)
        dh, dw = sv.rms_norm_backward(dy, h, rstd, w, dsum)
        only = sv.rms_norm_backward(dy, h, rstd, w)[0]
        for mask in range(1, 8):
            leaves = [t.clone().requires_grad_(bool(mask >> i & 1)) for i, t in enumerate((x, w, r))]
            y, s = sv.rms_norm(leaves[0], leaves[1], residual=leaves[2])
            torch.autograd.backward((y, s) if s.requires_grad else (y,), (dy, dsum) if s.requires_grad else (dy,))
            for i, (leaf, want) in enumerate(zip(leaves, (dh.to(dtype), dw, dh))):
                assert (leaf.grad is None) == (not mask >> i & 1)
                assert leaf.grad is None or torch.equal(leaf.grad, want), (mask, i)
        # both inputs have a gradient of their own, which may be changed in place
        a, b = (t.clone().requires_grad_() for t in (x, r))
        torch.autograd.backward(sv.rms_norm(a, w, residual=b), (dy, dsum))
        assert a.grad.data_ptr() != b.grad.data_ptr()
        sv.clip_grad_norm([a.grad, b.grad], 1e-3, out=[a.grad, b.grad])
        a, b = (t.clone().requires_grad_() for t in (x, r))
        sv.rms_norm(a, w, residual=b)[1].backward(dsum)
        assert len({a.grad.data_ptr(), b.grad.data_ptr(), dsum.data_ptr()}) == 3
        # one of the two results alone
        a, b = (t.clone().requires_grad_() for t in (x, r))
        sv.rms_norm(a, w, residual=b)[0].backward(dy)
        assert torch.equal(a.grad, only.to(dtype)) and torch.equal(b.grad, only)
        a, b = (t.clone().requires_grad_() for t in (x, r))
        sv.rms_norm(a, w, residual=b)[1].backward(dsum)
        assert torch.equal(a.grad, dsum.to(dtype)) and torch.equal(b.grad, dsum)
        # no residual
        a = x.clone().requires_grad_()
        y, rs = sv.rms_norm(a, w, return_rstd=True)
        assert y.requires_grad and not rs.requires_grad
        y.backward(dy)
        assert torch.equal(a.grad, sv.rms_norm_backward(dy, x, rs, w)[0])
        with torch.no_grad():
            assert not sv.rms_norm(a, w).requires_grad


def test_residual_is_the_row_itself(dev):
    # one tensor as both inputs: the gradients of both reach it
    x = hidden(9, 64, F32, 1).requires_grad_()
    dy = hidden(9, 64, F32, 2)
    y, h = sv.rms_norm(x, residual=x)
    y.backward(dy)
    rstd = sv.rms_norm(h.detach(), return_rstd=True)[1]
    assert torch.equal(x.grad, 2 * sv.rms_norm_backward(dy, h.detach(), rstd)[0])


def test_fp8_refuses_gradients(dev):
    x = hidden(4, 40, BF16, 1).requires_grad_()
    with pytest.raises(NotImplementedError):
        sv.rms_norm_fp8(x)
    with pytest.raises(NotImplementedError):
        sv.rms_norm_fp8(x.detach(), weights(40, F32, 1).requires_grad_())
    with torch.no_grad():
        assert sv.rms_norm_fp8(x)[0].dtype == E4M3


# ---------------------------------------------------------------- refusals

def test_refusals(dev):
    x, w, r = torch.zeros(4, 8, device=dev), torch.ones(8, device=dev), torch.zeros(4, 8, device=dev)
    s = torch.zeros(4, device=dev)
    b = x.to(BF16)
    for call in (lambda: sv.rms_norm(x, w[:7]), lambda: sv.rms_norm(x[0, 0]), lambda: sv.rms_norm(x, w.cpu()),
                 lambda: sv.rms_norm(x, residual=r[:3]), lambda: sv.rms_norm(x, residual=r.cpu()),
                 lambda: sv.rms_norm_fp8(x, w[:7]), lambda: sv.rms_norm_fp8(x, block=64),
                 lambda: sv.rms_norm_fp8(x, block=0), lambda: sv.rms_norm_fp8(x, block=True),
                 lambda: sv.rms_norm_backward(x[:3], x, s), lambda: sv.rms_norm_backward(x, x, s[:3]),
                 lambda: sv.rms_norm_backward(x, x, s, dsum=r[:3]), lambda: sv.rms_norm_backward(x, x, s, w[:3])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sv.rms_norm(x.double()), lambda: sv.rms_norm(x, w.to(BF16)), lambda: sv.rms_norm(x, [1.0] * 8),
                 lambda: sv.rms_norm(b, w.to(F16)), lambda: sv.rms_norm(x, residual=b),
                 lambda: sv.rms_norm(b, residual=b.to(F16)), lambda: sv.rms_norm(b, residual=3.0),
                 lambda: sv.rms_norm_fp8(x, dtype=BF16), lambda: sv.rms_norm_fp8(x, dtype=torch.int8),
                 lambda: sv.rms_norm_fp8(x, block=128.0), lambda: sv.rms_norm_backward(x, b, s),
                 lambda: sv.rms_norm_backward(b, b, s.to(BF16)), lambda: sv.rms_norm_backward(b, b, s, dsum=x),
                 lambda: sv.rms_norm_backward(b, b, s, w, param_dtype=BF16),
                 lambda: sv.rms_norm_backward(x, x, s, param_dtype=BF16)):
        with pytest.raises(TypeError):
            call()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(sv.SvError):
            sv.rms_norm(x, eps=eps)
        with pytest.raises(sv.SvError):
            sv.rms_norm_fp8(x, eps=eps)


# ---------------------------------------------------------------- the two ways into the library

class NoModule:
    """Stands in for the short way: every call takes the general one."""

    @staticmethod
    def rms(*_):
        return None

    rms_backward = grad_norm = clip_grad_norm = rms


def general_way(monkeypatch):
    from stable_variance_amd import gradients, layers

    for module in (layers, gradients):
        monkeypatch.setattr(module, "native", lambda: NoModule)


def test_both_ways_give_the_same(dev, monkeypatch):
    calls = []
    for dtype, stream in STREAMS:
        for shape in ((5, 136), (2, 3, 40), (4096,), (3, 1531)):
            n = shape[-1]
            x = hidden(math.prod(shape[:-1]), n, dtype, 1).reshape(shape)
            r = None if stream is None else hidden(math.prod(shape[:-1]), n, stream, 2).reshape(shape)
            for w in (None, weights(n, dtype, 3), weights(n, F32, 4)):
                for rstd in (False, True):
                    calls.append((lambda x=x, w=w, r=r, rstd=rstd: sv.rms_norm(x, w, 0.01, r, rstd)))
                    for to, block in ((E4M3, 128), (E5M2, None)):
                        calls.append((lambda x=x, w=w, r=r, rstd=rstd, to=to, block=block:
                                      sv.rms_norm_fp8(x, w, 0.01, r, to, block, rstd)))
    from stable_variance_amd import native

    # strided rows: a column range, two dimensions of rows, one row, one column
    for dtype in TYPES:
        wide = hidden(24, 51, dtype, 5)
        for x in (wide[:, 3:43], wide.reshape(4, 6, 51)[..., :40], wide.reshape(2, 3, 4, 51)[:, :, :, 1:42],
                  wide.reshape(4, 1, 6, 51)[..., 5:], wide[:1, 1:], wide[::2, :40], wide[:, 7:8], wide[2, 3:20],
                  wide.reshape(4, 6, 51)[:, :1, 2:9]):
            n = x.shape[-1]
            for r in (None, x.contiguous(), hidden(24 * 51, 2, F32, 6).reshape(-1)[:x.numel()].reshape(x.shape), x):
                w = weights(n, F32, 4)
                calls.append((lambda x=x, w=w, r=r: sv.rms_norm(x, w, 0.01, r, True)))
                calls.append((lambda x=x, w=w, r=r: sv.rms_norm_fp8(x, w, 0.01, r, E4M3, 128, True)))
    real, taken = native(), []

    class Counted:
        @staticmethod
        def rms(*args):
            out = real.rms(*args)
            taken.append(out is not None)
            return out

    from stable_variance_amd import layers

    with monkeypatch.context() as m:
        m.setattr(layers, "native", lambda: Counted)
        short = [c() for c in calls]
    assert taken == [True] * len(calls)
    general_way(monkeypatch)
    for a, c in zip(short, calls):
        b = c()
        assert type(a) is type(b)
        a, b = (a, b) if isinstance(a, tuple) else ((a,), (b,))
        assert len(a) == len(b)
        for p, q in zip(a, b):
            assert p.dtype == q.dtype and p.shape == q.shape and p.device == q.device and not p.requires_grad
            assert torch.equal(p.reshape(-1).view(torch.uint8), q.reshape(-1).view(torch.uint8))


def test_both_ways_back_give_the_same(dev, monkeypatch):
    from stable_variance_amd import layers

    calls, short = [], []
    for dtype, stream in PAIRS:
        for shape in ((5, 136), (2, 3, 40), (4096,), (3, 1531)):
            n, rows = shape[-1], math.prod(shape[:-1])
            h, dy, dsum = (hidden(rows, n, t, i).reshape(shape) for i, t in enumerate((stream, dtype, stream)))
            rstd = sv.rms_norm(h, return_rstd=True)[1]
            for w in (weights(n, dtype, 3), weights(n, F32, 4)):
                for d in (None, dsum):
                    for dw in (True, False):
                        calls.append((dy, h, rstd, w, d, dw))
    for dtype, stream in PAIRS:
        wide, rows = hidden(24, 51, stream, 5), hidden(24, 60, dtype, 6)
        for a, b in ((wide[:, 3:43], rows[:, :40]), (wide.reshape(4, 6, 51)[..., :40], rows.reshape(4, 6, 60)[..., 20:]),
                     (wide[:1, 1:], rows[:1, :50]), (wide[::2, :40], rows[1::2, 3:43]), (wide[2, 3:20], rows[3, 3:20]),
                     (wide[:, 7:8], rows[:, 9:10])):
            rstd = sv.rms_norm(a, return_rstd=True)[1]
            for d in (None, a, a.contiguous()):
                calls.append((b, a, rstd, weights(a.shape[-1], dtype, 3), d, True))
    for dy, h, rstd, w, d, dw in calls:
        out = layers._short_backward(dy, h, rstd, w, d, True, True, dw)
        assert out is not None
        assert torch.equal(out[1], out[0].to(dy.dtype))
        short.append(sv.rms_norm_backward(dy, h, rstd, w, d, weight_grad=dw))
        assert torch.equal(short[-1][0], out[0])
    general_way(monkeypatch)
    for (dy, h, rstd, w, d, dw), want in zip(calls, short):
        got = sv.rms_norm_backward(dy, h, rstd, w, d, weight_grad=dw)
        for p, q in zip(got, want):
            assert p is q is None or (p.dtype == q.dtype and torch.equal(p, q) and not q.requires_grad)
    test_autograd(dev)
    test_refusals(dev)


def test_the_short_way_back_leaves_the_others(dev):
    from stable_variance_amd import native

    m = native()
    dy, h, rstd, w, d = hidden(4, 8, BF16, 1), hidden(4, 8, F32, 2), torch.ones(4, device=dev), weights(8, F32, 1), \
        hidden(4, 8, F32, 3)
    ok = (dy, h, rstd, w, d, True, False, True)
    assert m.rms_backward(*ok) is not None
    for i, bad in ((0, dy.cpu()), (0, dy.double()), (0, dy[:3]), (0, dy.t()), (0, None), (0, dy.to(F16)[:, ::2]), (1, h[:3]),
                   (1, h.to(F16)), (1, h.t()), (1, h[0, 0]), (1, h.cpu()), (2, rstd[:3]), (2, rstd[:, None]),
                   (2, rstd.to(BF16)), (2, rstd.cpu()), (3, None), (3, w[:7]), (3, w.to(F16)), (3, w[None]), (4, d[:3]),
                   (4, d.to(BF16)), (4, d.cpu()), (4, torch._neg_view(d)), (4, 1.0)):
        args = list(ok)
        args[i] = bad
        assert m.rms_backward(*args) is None, (i, bad)
    assert m.rms_backward(dy[:0], h[:0], rstd[:0], *ok[3:]) is None
    with pytest.raises(TypeError):
        m.rms_backward(*ok[:7])


def test_the_short_way_leaves_the_others(dev):
    from stable_variance_amd import native

    m = native()
    x, w, r = hidden(4, 8, BF16, 1), weights(8, F32, 1), hidden(4, 8, F32, 2)
    ok = (x, w, r, 1e-6, False, 0, 0)
    assert m.rms(*ok) is not None
    square = hidden(8, 8, BF16, 4)
    half_view = torch.randn(4, 8, dtype=torch.complex64, device=dev).conj().imag
    for i, bad in ((0, x.cpu()), (0, x.double()), (0, x[:, ::2]), (0, square.t()), (0, square.as_strided((4, 8), (5, 1))),
                   (0, square.reshape(2, 4, 8).transpose(0, 1)), (0, square[:1].expand(4, 8)), (0, x[:0]), (0, x[:, :0]), (0, x[0, 0]),
                   (0, 1.0), (0, None), (0, x.to_sparse()), (0, half_view), (0, torch._neg_view(x)),
                   (0, x.clone().requires_grad_()), (1, w.clone().requires_grad_()), (2, r.clone().requires_grad_()),
                   (1, w[:7]), (1, w[None]), (1, w.to(F16)), (1, w.cpu()), (1, w.double()), (1, [1.0] * 8),
                   (2, r[:3]), (2, r.to(F16)), (2, r.cpu()), (2, r.t()), (2, r.reshape(2, 2, 8)), (2, 0.5),
                   (3, -1.0), (3, float("nan"))):
        args = list(ok)
        args[i] = bad
        assert m.rms(*args) is None, (i, bad)
    with torch.no_grad():
        assert m.rms(x.clone().requires_grad_(), *ok[1:]) is not None
    p = torch.nn.Parameter(w)
    with torch.no_grad():
        assert m.rms(x, p, *ok[2:]) is not None
    for args in ((), (x,), ok + (1,), (x, w, r, "a", False, 0, 0)):
        with pytest.raises(TypeError):
            m.rms(*args)
