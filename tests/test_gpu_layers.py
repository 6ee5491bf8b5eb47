"""Layer norm and embedding on the GPU against their formulas in float64.

Tolerances are bounds on rounding, with u = 2^-24 and u_T half a step of the
result's type.  A sum of n terms in float32 is off by at most (log2 n + 2) u
of the sum of their magnitudes when added pairwise, less when compensated.
"""
import math

import pytest
import torch

import stable_variance_amd as sv

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF16, F16]
IDS = {F32: "f32", BF16: "bf16", F16: "f16"}
# half of the smallest step near zero
TINY = {F32: 2.0 ** -150, BF16: 2.0 ** -134, F16: 2.0 ** -25}


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


def steps(n):
    """Roundings between the data and a row's result, in u: the shift, the
    centring, the sums of log2(n) levels for the mean and the variance, the
    division, the root and the products."""
    return 3 * math.ceil(math.log2(max(n, 2))) + 16


def close(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float(((got - want).abs() / tol)[bad].nan_to_num(float('inf')).max()):.3g} of the tolerance"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def hidden(rows, n, dtype, seed, offset=0.0, ld=None):
    g = gen(seed)
    x = torch.randn(rows, ld or n, generator=g, device="cuda") * (0.5 + torch.rand(ld or n, generator=g, device="cuda"))
    return (x + offset).to(dtype)[:, :n]


def params(n, dtype, seed):
    g = gen(1000 + seed)
    return ((1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(dtype),
            (0.2 * torch.randn(n, generator=g, device="cuda")).to(dtype))


# ---------------------------------------------------------------- forward

def check_forward(x, w, b, eps=1e-5):
    y, mean, rstd = sv.layer_norm(x, w, b, eps=eps, return_stats=True)
    n = x.shape[-1]
    X = x.double()
    M = X.mean(-1, keepdim=True)
    V = ((X - M) ** 2).mean(-1, keepdim=True)
    R = (V + eps) ** -0.5
    H = (X - M) * R
    W = w.double() if w is not None else torch.ones(n, dtype=torch.float64, device=x.device)
    B = b.double() if b is not None else torch.zeros(n, dtype=torch.float64, device=x.device)
    Y = H * W + B
    k = steps(n) * U
    assert y.dtype == x.dtype and y.shape == x.shape and y.is_contiguous()
    assert mean.dtype == rstd.dtype == F32 and mean.shape == rstd.shape == x.shape[:-1]
    close(y, Y, (half(x.dtype) + k) * Y.abs() + TINY[x.dtype] + k * ((H.abs() + 1) * W.abs() + B.abs()), "y")
    close(mean, M[..., 0], (U * M.abs() + k * V.sqrt())[..., 0] + TINY[F32], "mean")
    close(rstd, R[..., 0], k * R[..., 0], "rstd")
    return y, mean, rstd


LENGTHS = [1, 2, 3, 5, 7, 8, 9, 31, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300, 511, 512, 513, 768, 1000, 1023,
           1024, 1025, 1531, 2047, 2048, 2050, 4095, 4096, 4104, 5000, 8191, 8192, 8200, 12288, 12290, 14000, 16384, 16385,
           20001, 32768, 32776, 33000, 70001]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_lengths(dev, dtype):
    for i, n in enumerate(LENGTHS):
        print("norm", IDS[dtype], n, flush=True)
        w, b = params(n, dtype if i % 2 else F32, i)
        check_forward(hidden(3 + i % 5, n, dtype, i), w, b)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("rows", [1, 2, 255, 1025, 40000])
def test_norm_rows(dev, dtype, rows):
    for n in (24, 200, 1100):
        w, b = params(n, dtype, n)
        check_forward(hidden(rows, n, dtype, rows), w, b)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_offsets_and_outliers(dev, dtype):
    w, b = params(1000, F32, 1)
    check_forward(hidden(9, 1000, dtype, 2, offset=1e4), w, b)  # a mean far above the spread
    check_forward(hidden(9, 1000, dtype, 3, offset=-300.0), w, b)
    x = hidden(9, 1000, dtype, 4).clone()
    x[:, 0] = 2.0e4  # the value the row is shifted by
    x[4, 17] = -3.0e4
    check_forward(x, w, b)
    check_forward(hidden(9, 1000, dtype, 5) * 1e-3, w, b, eps=1e-12)


def test_norm_parameters_and_shapes(dev):
    w, b = params(40, F32, 3)
    x = hidden(30, 40, F32, 6)
    for ww, bb in ((None, None), (w, None), (None, b)):
        check_forward(x, ww, bb)
    check_forward(x.reshape(2, 3, 5, 40), w, b)
    y1, m1, r1 = check_forward(x[0], w, b)  # one row, no leading dimension
    assert m1.shape == ()
    assert torch.equal(sv.layer_norm(x, w, b), sv.layer_norm(x, w, b, return_stats=True)[0])
    check_forward(x.to(BF16), w, b)
    check_forward(x.to(F16), w.to(F16), b.to(F16))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_strides_give_the_same_bits(dev, dtype):
    for n, ld in ((96, 100), (96, 97), (1000, 1003), (1531, 1531), (4096, 4104), (130, 131)):
        w, b = params(n, dtype, n)
        x = hidden(7, n, dtype, n, ld=ld)
        if ld > n:
            assert not x.is_contiguous()
        got = check_forward(x, w, b)
        dense = sv.layer_norm(x.contiguous(), w, b, return_stats=True)
        assert all(torch.equal(p, q) for p, q in zip(got, dense)), (n, ld)
        # the same rows one value further on: another alignment
        shifted = torch.empty(7 * n + 1, dtype=dtype, device=dev)[1:].view(7, n).copy_(x)
        assert torch.equal(sv.layer_norm(shifted, w, b), got[0])
        xt = x.t().contiguous().t()  # last dimension not contiguous: copied
        assert torch.equal(sv.layer_norm(xt, w, b), got[0])
    row = hidden(1, 64, dtype, 1)
    w, b = params(64, dtype, 2)
    assert torch.equal(sv.layer_norm(row.expand(5, 64), w, b), sv.layer_norm(row.repeat(5, 1), w, b))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_row_is_independent_of_its_batch(dev, dtype):
    for n in (17, 128, 1531, 4096, 9000, 40000):
        x = hidden(70, n, dtype, n)
        w, b = params(n, dtype, n)
        whole = sv.layer_norm(x, w, b, return_stats=True)
        again = sv.layer_norm(x, w, b, return_stats=True)
        assert all(torch.equal(p, q) for p, q in zip(whole, again))
        for r in (0, 1, 33, 69):
            one = sv.layer_norm(x[r:r + 1], w, b, return_stats=True)
            assert all(torch.equal(p[r:r + 1], q) for p, q in zip(whole, one)), (n, r)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_equal_values_give_the_bias(dev, dtype):
    for n in (1, 5, 64, 1000, 4096, 20000, 50000):
        x = torch.tensor([0.0, 1.0, -3.25, 6.0e4 if dtype == F16 else 1e30], device=dev).to(dtype)[:, None].repeat(1, n)
        w, b = params(n, dtype, n)
        y, mean, rstd = sv.layer_norm(x, w, b, return_stats=True)
        assert torch.equal(y, b.expand_as(y))
        assert torch.equal(mean, x[:, 0].float())
        want = torch.full_like(rstd, float(torch.tensor(1e-5, dtype=torch.float64) ** -0.5))
        assert torch.equal(rstd, want)
        assert sv.layer_norm(x, w, b, eps=0.0).isnan().all()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_nan_and_inf_stay_in_their_row(dev, dtype):
    for n in (6, 300, 1531, 4096, 40000):
        x = hidden(8, n, dtype, n).clone()
        clean = sv.layer_norm(x)
        x[1, 0] = float("nan")
        x[3, n - 1] = float("inf")
        x[6, n // 2] = float("-inf")
        y = sv.layer_norm(x)
        bad = [1, 3, 6]
        good = [0, 2, 4, 5, 7]
        assert y[bad].isnan().all() and torch.equal(y[good], clean[good])


def test_norm_empty(dev):
    y, mean, rstd = sv.layer_norm(torch.empty(3, 0, device=dev), return_stats=True)
    assert y.shape == (3, 0) and mean.isnan().all() and rstd.isnan().all()
    w, b = params(5, F32, 1)
    y, mean, rstd = sv.layer_norm(torch.empty(0, 5, device=dev), w, b, return_stats=True)
    assert y.shape == (0, 5) and mean.shape == (0,)
    dx, dw, db = sv.layer_norm_backward(y, y, mean, rstd, w)
    assert dx.shape == (0, 5) and torch.equal(dw, torch.zeros_like(w)) and torch.equal(db, torch.zeros_like(w))
    z = torch.empty(3, 0, device=dev)
    s = torch.zeros(3, device=dev)
    dx, dw, db = sv.layer_norm_backward(z, z, s, s)
    assert dx.shape == (3, 0) and dw.shape == (0,) and db.shape == (0,)


def test_norm_rows_far_apart(dev):
    ld = (1 << 30) + 8  # the third row starts beyond 2^31 values
    x = torch.empty(3, ld, dtype=BF16, device=dev)[:, :1000]
    x.copy_(hidden(3, 1000, BF16, 5))
    w, b = params(1000, BF16, 5)
    y, mean, rstd = check_forward(x, w, b)
    dy = hidden(3, 1000, BF16, 6)
    got = sv.layer_norm_backward(dy, x, mean, rstd, w)
    want = sv.layer_norm_backward(dy, x.contiguous(), mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


# ---------------------------------------------------------------- backward

def check_backward(x, dy, w, eps=1e-5, param=None, **kw):
    _, mean, rstd = sv.layer_norm(x, w, None, eps=eps, return_stats=True)
    dx, dw, db = sv.layer_norm_backward(dy, x, mean, rstd, w, param_dtype=param, **kw)
    n = x.shape[-1]
    X, G = x.double().reshape(-1, n), dy.double().reshape(-1, n)
    rows = X.shape[0]
    M = X.mean(1, keepdim=True)
    R = (((X - M) ** 2).mean(1, keepdim=True) + eps) ** -0.5
    H = (X - M) * R
    g = G * w.double() if w is not None else G
    DX = R * (g - g.mean(1, keepdim=True) - H * (g * H).mean(1, keepdim=True))
    k = steps(n) * U
    # every term of dx carries `steps` roundings of its own magnitude
    mag = g.abs() + g.abs().mean(1, keepdim=True) + (H.abs() + 1) * (g.abs() * (H.abs() + 1)).mean(1, keepdim=True)
    assert dx.dtype == x.dtype and dx.shape == x.shape
    close(dx.reshape(-1, n), DX, (half(x.dtype) + k) * DX.abs() + TINY[x.dtype] + k * R * mag, "dx")
    # column sums: runs of at most 48 roundings, joined with compensation
    pt = param or (w.dtype if w is not None else F32)
    if dw is not None:
        DW, S = (G * H).sum(0), (G.abs() * (H.abs() + 1)).sum(0)
        assert dw.dtype == pt
        close(dw, DW, (half(pt) + 2 * U) * DW.abs() + TINY[pt] + (k + 48 * U) * S, "dweight")
    if db is not None:
        DB = G.sum(0)
        assert db.dtype == pt
        close(db, DB, (half(pt) + 2 * U) * DB.abs() + TINY[pt] + 48 * U * G.abs().sum(0), "dbias")
    assert rows == 0 or not dx.isnan().any()
    return dx, dw, db


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_grad_lengths(dev, dtype):
    for i, n in enumerate(LENGTHS):
        print("norm grad", IDS[dtype], n, flush=True)
        w, _ = params(n, dtype if i % 2 else F32, i)
        rows = 2 + i % 7
        check_backward(hidden(rows, n, dtype, i), hidden(rows, n, dtype, 500 + i), w)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("rows", [1, 2, 63, 64, 65, 300, 1025, 4097, 70000])
def test_norm_grad_rows(dev, dtype, rows):
    for n in (24, 200, 1100):
        if rows * n > 20_000_000:
            continue
        w, _ = params(n, dtype, n)
        check_backward(hidden(rows, n, dtype, rows), hidden(rows, n, dtype, rows + 1), w)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_grad_offsets(dev, dtype):
    w, _ = params(1000, F32, 1)
    check_backward(hidden(9, 1000, dtype, 2, offset=1e4), hidden(9, 1000, dtype, 7, offset=0.5), w)
    x = hidden(9, 1000, dtype, 4).clone()
    x[:, 0] = 2.0e4
    check_backward(x, hidden(9, 1000, dtype, 8), w)


def test_norm_grad_options(dev):
    x, dy = hidden(50, 72, BF16, 1), hidden(50, 72, BF16, 2)
    w, b = params(72, F32, 1)
    full = check_backward(x, dy, w)
    for wg in (False, True):
        for bg in (False, True):
            dx, dw, db = check_backward(x, dy, w, weight_grad=wg, bias_grad=bg)
            assert (dw is None) == (not wg) and (db is None) == (not bg)
            assert torch.equal(dx, full[0])
            assert (dw is None or torch.equal(dw, full[1])) and (db is None or torch.equal(db, full[2]))
    check_backward(x, dy, None)
    check_backward(x, dy, None, param=BF16)
    check_backward(x, dy, w.to(BF16))
    x3, dy3 = x.reshape(5, 10, 72), dy.reshape(5, 10, 72)
    got = check_backward(x3, dy3, w)
    assert torch.equal(got[0].reshape(50, 72), full[0]) and torch.equal(got[1], full[1])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_norm_grad_strides_and_repeats_give_the_same_bits(dev, dtype):
    for n, ld in ((96, 97), (1000, 1003), (1531, 1531), (4096, 4104), (40000, 40001)):
        w, _ = params(n, dtype, n)
        x, dy = hidden(67, n, dtype, n, ld=ld), hidden(67, n, dtype, n + 1, ld=ld)
        got = check_backward(x, dy, w)
        dense = check_backward(x.contiguous(), dy.contiguous(), w)
        assert all(torch.equal(p, q) for p, q in zip(got, dense)), (n, ld)
        # dx of a row does not depend on the batch
        one = check_backward(x[5:6], dy[5:6], w)
        assert torch.equal(one[0], got[0][5:6])
    g = torch.ones((), dtype=dtype, device=dev).expand(67, 40000)  # every stride 0
    a = check_backward(x, g, w)
    b = check_backward(x, g.contiguous(), w)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_norm_grad_nan_stays_in_its_row(dev):
    for n in (40, 1531, 4096, 40000):
        x, dy = hidden(6, n, F32, 1).clone(), hidden(6, n, F32, 2)
        _, mean, rstd = sv.layer_norm(x, return_stats=True)
        clean = sv.layer_norm_backward(dy, x, mean, rstd)[0]
        x[2, n // 2] = float("nan")
        _, mean, rstd = sv.layer_norm(x, return_stats=True)
        dx, dw, db = sv.layer_norm_backward(dy, x, mean, rstd)
        keep = [0, 1, 3, 4, 5]
        assert dx[2].isnan().all() and torch.equal(dx[keep], clean[keep])
        assert dw.isnan().all() and not db.isnan().any()


def test_norm_gradients_against_differences(dev):
    # the directional derivative of sum(dy * y) along v, by central
    # differences of the forward call with steps h and 2h.  Truncation: the
    # difference of the two quotients is three times the leading h^2 term of
    # the first, so it bounds it.  Rounding: each y is off by `steps` u.
    n, rows, h = 96, 7, 2.0 ** -5
    x, dy = hidden(rows, n, F32, 11), hidden(rows, n, F32, 12)
    w, b = params(n, F32, 13)
    _, mean, rstd = sv.layer_norm(x, w, b, return_stats=True)
    grads = sv.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(x_, w_, b_):
        return float((sv.layer_norm(x_, w_, b_).double() * dy.double()).sum())

    noise = steps(n) * U * float((dy.double().abs() * (w.double().abs() * 5 + 1)).sum())
    for i, g in enumerate(grads):
        v = torch.randn(g.shape, generator=gen(20 + i), device=dev)

        def quotient(step):
            up, down = [x, w, b], [x, w, b]
            up[i], down[i] = up[i] + step * v, down[i] - step * v
            real = float(((up[i].double() - down[i].double()) * g.double()).sum())
            return (loss(*up) - loss(*down)), real

        d1, r1 = quotient(h)
        d2, r2 = quotient(2 * h)
        tol = abs((d2 / 2 - r2 / 2) - (d1 - r1)) + 2 * noise
        assert abs(d1 - r1) <= tol, (i, d1, r1, tol)


# ---------------------------------------------------------------- embedding

def ids_for(kind, tokens, vocab, dtype, seed):
    g = gen(seed)
    if kind == "uniform":
        t = torch.randint(0, max(vocab, 1), (tokens,), generator=g, device="cuda")
    elif kind == "same":
        t = torch.full((tokens,), vocab // 2, device="cuda")
    elif kind == "skewed":
        r = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
        t = (vocab ** r - 1).long().clamp_(0, vocab - 1)
    else:  # one token per row, descending
        t = torch.arange(tokens - 1, -1, -1, device="cuda") % max(vocab, 1)
    return t.to(dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_lookup(dev, dtype, idt):
    for tokens, vocab, dim in ((1, 1, 1), (1, 50, 4096), (7, 33, 5), (300, 1000, 64), (65, 17, 257), (1025, 900, 1000),
                               (70000, 300, 24), (5, 3, 20001)):
        table = torch.randn(vocab, dim, generator=gen(dim), device=dev).to(dtype)
        ids = ids_for("uniform", tokens, vocab, idt, tokens)
        for scale in (1.0, 0.37):
            got = sv.embedding(ids, table, scale=scale)
            want = (table[ids.long()].float() * torch.tensor(scale, dtype=F32, device=dev)).to(dtype)
            assert got.dtype == dtype and torch.equal(got, want), (tokens, vocab, dim, scale)
    ids2 = ids.reshape(1, 5, 1)
    assert sv.embedding(ids2, table).shape == (1, 5, 1, dim)
    assert torch.equal(sv.embedding(ids2, table).reshape(5, dim), table[ids.long()])


def test_lookup_strides_and_bad_ids(dev):
    wide = torch.randn(40, 103, generator=gen(1), device=dev)
    table = wide[:, 3:100]
    ids = torch.tensor([[3, -1, 39], [40, 0, 1 << 30]], device=dev)
    out = sv.embedding(ids, table)
    ok = torch.tensor([[True, False, True], [False, True, False]], device=dev)
    assert torch.equal(out[ok], table[ids[ok]]) and out[~ok].isnan().all()
    assert torch.equal(sv.embedding(ids[:, ::2], table)[ok[:, ::2]], out[:, ::2][ok[:, ::2]])
    big = torch.tensor([-(1 << 62), 1 << 40, (1 << 32) + 5, 5], device=dev)
    out = sv.embedding(big, table)
    assert out[:3].isnan().all() and torch.equal(out[3], table[5])
    tt = table.t().contiguous().t()
    assert torch.equal(sv.embedding(ids, tt)[ok], out.new_tensor(table[ids[ok]].tolist()))
    assert sv.embedding(ids, torch.empty(0, 6, device=dev)).isnan().all()
    assert sv.embedding(torch.empty(0, 4, dtype=torch.int32, device=dev), table).shape == (0, 4, 97)
    assert sv.embedding(ids, torch.empty(9, 0, device=dev)).shape == (2, 3, 0)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_lookup_and_gradient_of_special_values(dev, dtype):
    # signed zeros, subnormals, the largest values, Inf and NaN: rounded as
    # the host rounds them
    tiny, big = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    v = torch.tensor([0.0, -0.0, tiny, -tiny, tiny / 4, -tiny / 8, tiny * 0.75, big, -big, float("inf"), float("-inf"),
                      float("nan"), 1.0, 1.0 + torch.finfo(dtype).eps, 3.0e-41, -1.2e-39], dtype=torch.float64)
    table = v.to(dtype).repeat(3, 5)  # 80 values a row: whole chunks
    ids = torch.arange(3)
    for cols in (80, 77, 3):
        t = table[:, :cols].contiguous()
        for scale in (1.0, 0.5, 3.0, -1.0):
            want = (t.float() * scale).to(dtype)
            got = sv.embedding(ids.to(dev), t.to(dev), scale=scale).cpu()
            assert torch.equal(got.isnan(), want.isnan())
            keep = ~want.isnan()
            assert torch.equal(got[keep], want[keep]) and torch.equal(got[keep].signbit(), want[keep].signbit())
            grad = sv.embedding_backward(t.to(dev), ids.to(dev), 3, scale=scale).cpu()
            assert torch.equal(grad.isnan(), want.isnan()) and torch.equal(grad[keep], want[keep])
    # sums that overflow the type, or meet Inf of both signs
    dy = torch.tensor([[big, big, float("inf"), -big]] * 2 + [[0.0, -big, float("-inf"), 1.0]], dtype=torch.float64)
    got = sv.embedding_backward(dy.to(dtype).to(dev), torch.zeros(3, dtype=torch.int32, device=dev), 1).cpu()[0]
    assert got[0] == float("inf") and got[2].isnan() and got[3] == float("-inf")
    # big + big - big: float32 holds the sum in float16's range only
    assert got[1] == (big if dtype == F16 else float("inf"))


def test_lookup_beyond_2_31_values(dev):
    vocab, dim = (1 << 20) + 40, 2056
    table = torch.zeros(vocab, dim, dtype=F16, device=dev)
    table[-3] = 1.5
    table[1 << 20] = -2.0
    out = sv.embedding(torch.tensor([vocab - 3, 1 << 20, 7], device=dev), table, scale=2.0)
    assert (out[0] == 3).all() and (out[1] == -4).all() and (out[2] == 0).all()


def check_lookup_grad(dy, ids, vocab, scale=1.0, padding=None):
    got = sv.embedding_backward(dy, ids, vocab, scale=scale, padding_idx=padding)
    dim = dy.shape[-1]
    flat = ids.reshape(-1).long()
    D = dy.reshape(-1, dim).double()
    use = (flat >= 0) & (flat < vocab)
    if padding is not None:
        use &= flat != padding
    s = float(torch.tensor(scale, dtype=F32))
    want = torch.zeros(vocab, dim, dtype=torch.float64, device=dy.device).index_add_(0, flat[use], D[use])
    mag = torch.zeros_like(want).index_add_(0, flat[use], D[use].abs())
    count = torch.bincount(flat[use], minlength=vocab).double()[:vocab, None]
    # a compensated sum of c terms: u of the result and (c u)^2 of the
    # magnitudes; then the product and the rounding to the type
    tol = ((half(dy.dtype) + 3 * U) * want.abs() + 2 * (count * U) ** 2 * mag) * abs(s) + TINY[dy.dtype]
    assert got.dtype == dy.dtype and got.shape == (vocab, dim)
    close(got, want * s, tol, "grad")
    assert (got[count[:, 0] == 0] == 0).all()
    return got


GRADS = [  # tokens, vocab, dim, kind
    (1, 1, 1, "same"), (1, 300, 4096, "same"), (2, 2, 3, "uniform"), (50, 1000, 64, "uniform"),
    (64, 5, 257, "uniform"), (65, 7, 96, "same"), (255, 600, 33, "skewed"), (1000, 511, 128, "descending"),
    (1024, 512, 40, "uniform"), (1025, 513, 40, "skewed"), (3000, 3, 72, "uniform"), (5000, 70000, 24, "skewed"),
    (5000, 9, 520, "same"), (20000, 300000, 8, "skewed"), (70000, 2000, 16, "skewed"), (70000, 1, 40, "same"),
    (131, 131, 20001, "skewed"), (200001, 256, 9, "uniform"), (4097, 1 << 20, 2, "uniform"),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_lookup_grad(dev, dtype):
    for i, (tokens, vocab, dim, kind) in enumerate(GRADS):
        print("lookup grad", IDS[dtype], tokens, vocab, dim, kind, flush=True)
        ids = ids_for(kind, tokens, vocab, torch.int32 if i % 2 else torch.int64, i)
        dy = hidden(tokens, dim, dtype, i)
        first = check_lookup_grad(dy, ids, vocab, scale=(1.0, 0.37)[i % 2])
        again = sv.embedding_backward(dy, ids, vocab, scale=(1.0, 0.37)[i % 2])
        assert torch.equal(first, again)


def test_lookup_grad_padding_bad_ids_and_strides(dev):
    tokens, vocab, dim = 4000, 50, 70
    ids = ids_for("skewed", tokens, vocab, torch.int64, 3).clone()
    ids[5::97] = -1
    ids[6::97] = vocab
    ids[7::97] = 1 << 40
    ids[8::97] = -(1 << 40)
    wide = torch.randn(tokens, dim + 5, generator=gen(4), device=dev)
    dy = wide[:, 2:2 + dim]
    a = check_lookup_grad(dy, ids, vocab, padding=0)
    assert torch.equal(a, check_lookup_grad(dy.contiguous(), ids, vocab, padding=0))
    check_lookup_grad(dy, ids, vocab, padding=vocab - 1)
    check_lookup_grad(dy, ids, vocab)
    # NaN in the gradient of a token that takes no part reaches nothing
    dy = dy.clone()
    dy[ids == -1] = float("nan")
    dy[ids == 0] = float("inf")
    assert torch.equal(a, check_lookup_grad(dy, ids, vocab, padding=0))
    all_bad = torch.full((300,), -1, device=dev)
    assert (sv.embedding_backward(dy[:300], all_bad, vocab) == 0).all()
    assert (sv.embedding_backward(dy[:0], ids[:0], vocab) == 0).all()
    assert sv.embedding_backward(dy, ids, 0).shape == (0, dim)
    assert sv.embedding_backward(dy[:, :0], ids, 9).shape == (9, 0)
    g = torch.ones((), device=dev).expand(tokens, dim)
    assert torch.equal(sv.embedding_backward(g, ids, vocab), sv.embedding_backward(g.contiguous(), ids, vocab))
    ids3 = ids.reshape(40, 100).t()  # a transposed view of ids
    dy3 = wide[:, :8].reshape(100, 40, 8)
    check_lookup_grad(dy3, ids3, vocab)


def test_lookup_grad_row_is_independent_of_other_tokens(dev):
    vocab, dim = 40, 48
    ids = ids_for("skewed", 9000, vocab, torch.int64, 8)
    dy = hidden(9000, dim, F32, 9)
    whole = sv.embedding_backward(dy, ids, vocab)
    for v in (0, 1, 20):
        keep = ids == v
        assert torch.equal(sv.embedding_backward(dy[keep], ids[keep], vocab)[v], whole[v])


def test_lookup_grad_keeps_what_cancels(dev):
    # large values that cancel leave the small ones: a plain float32 sum
    # would lose them
    tokens = 30000
    dy = torch.ones(tokens, 4, device=dev)
    dy[::2] = 3.0e7
    dy[1::2] = -3.0e7
    dy[12345:12445] = 0.25
    ids = torch.zeros(tokens, dtype=torch.int64, device=dev)
    got = sv.embedding_backward(dy, ids, 2)
    want = dy.double().sum(0)
    assert torch.equal(got[0].double(), want) and (got[1] == 0).all()


def test_lookup_grad_beyond_2_31_values(dev):
    vocab, dim = (1 << 20) + 40, 2056
    ids = torch.tensor([vocab - 1, 3, vocab - 1, 1 << 20], device=dev)
    dy = torch.ones(4, dim, dtype=F16, device=dev)
    g = sv.embedding_backward(dy, ids, vocab)
    assert (g[vocab - 1] == 2).all() and (g[3] == 1).all() and (g[1 << 20] == 1).all()
    assert int(torch.count_nonzero(g[:, 0])) == 3 and int(torch.count_nonzero(g[:, dim - 1])) == 3


# ---------------------------------------------------------------- together

def reference_block(ids, table, w, b, dy, scale, eps=1e-5):
    """Embedding and layer norm in float64 on the host, with autograd."""
    t, ww, bb = (v.detach().double().cpu().requires_grad_() for v in (table, w, b))
    x = t[ids.cpu().long()] * scale
    m = x.mean(-1, keepdim=True)
    d = x - m
    y = d * ((d * d).mean(-1, keepdim=True) + eps) ** -0.5 * ww + bb
    (y * dy.double().cpu()).sum().backward()
    return y.detach(), t.grad, ww.grad, bb.grad


def test_block_with_autograd(dev):
    vocab, dim, scale = 60, 136, 8.0
    ids = ids_for("skewed", 500, vocab, torch.int64, 1).reshape(5, 100)
    table = (0.1 * torch.randn(vocab, dim, generator=gen(2), device=dev)).requires_grad_()
    w, b = (p.requires_grad_() for p in params(dim, F32, 2))
    dy = torch.randn(5, 100, dim, generator=gen(3), device=dev)
    y = sv.layer_norm(sv.embedding(ids, table, scale=scale), w, b)
    assert y.requires_grad
    (y * dy).sum().backward()
    Y, T, W, B = (v.to(dev) for v in reference_block(ids, table, w.detach(), b.detach(), dy, scale))
    # relative to the largest gradient: `steps` roundings per token's dx and
    # 48 per column run
    k = (steps(dim) + 64) * U
    close(y.detach(), Y, k * (Y.abs() + 4), "y")
    per_row = torch.bincount(ids.reshape(-1), minlength=vocab).double()[:, None]
    rs = float((T.abs().sum(1) / per_row[:, 0].clamp(min=1)).max())
    assert rs > 0
    # |dx| <= scale * rstd * |dy| (1 + 1 + xhat^2 ..): bound each token's terms
    x = table.detach().double()[ids] * scale
    r = (x.var(-1, unbiased=False) + 1e-5) ** -0.5
    bound = (r * scale * dy.double().abs().amax(-1) * 12 * 4).reshape(-1)
    tol = torch.zeros(vocab, dtype=torch.float64, device=dev).index_add_(0, ids.reshape(-1), bound) * k
    close(table.grad, T, tol[:, None] + 1e-300, "table.grad")
    S = dy.double().abs().sum((0, 1))
    close(w.grad, W, k * 5 * S, "w.grad")
    close(b.grad, B, k * S, "b.grad")
    # explicit calls give the same bits
    x = sv.embedding(ids, table.detach(), scale=scale)
    _, mean, rstd = sv.layer_norm(x, w.detach(), b.detach(), return_stats=True)
    dx, dw, db = sv.layer_norm_backward(dy, x, mean, rstd, w.detach())
    assert torch.equal(dw, w.grad) and torch.equal(db, b.grad)
    assert torch.equal(sv.embedding_backward(dx, ids, vocab, scale=scale), table.grad)


def test_autograd_takes_what_is_asked_for(dev):
    x, dy = hidden(20, 30, F32, 1), hidden(20, 30, F32, 2)
    w, b = params(30, F32, 3)
    full = check_backward(x, dy, w)
    for mask in range(1, 8):
        leaves = [t.clone().requires_grad_(bool(mask >> i & 1)) for i, t in enumerate((x, w, b))]
        sv.layer_norm(*leaves).backward(dy)
        for i, (leaf, want) in enumerate(zip(leaves, full)):
            assert (leaf.grad is None) == (not mask >> i & 1)
            assert leaf.grad is None or torch.equal(leaf.grad, want), (mask, i)
    leaf = x.clone().requires_grad_()
    y, mean, rstd = sv.layer_norm(leaf, return_stats=True)
    assert y.requires_grad and not mean.requires_grad and not rstd.requires_grad
    bias = b.to(F32).requires_grad_()
    sv.layer_norm(x.to(BF16), None, bias).backward(dy.to(BF16))
    assert bias.grad.dtype == F32
    with torch.no_grad():
        assert not sv.layer_norm(leaf).requires_grad
    t = torch.randn(9, 30, device=dev)
    assert not sv.embedding(torch.tensor([1], device=dev), t).requires_grad
    tt = t.clone().requires_grad_()
    sv.embedding(torch.tensor([1, 1, 3], device=dev), tt, padding_idx=3).sum().backward()
    assert (tt.grad[1] == 2).all() and (tt.grad[3] == 0).all()


def test_block_captured_and_replayed(dev):
    vocab, dim, tokens = 300, 520, 700
    table = torch.randn(vocab, dim, generator=gen(1), device=dev).to(BF16)
    w, b = params(dim, F32, 1)
    ids = ids_for("skewed", tokens, vocab, torch.int64, 1).clone()
    dy = hidden(tokens, dim, BF16, 2).clone()

    def block():
        x = sv.embedding(ids, table, scale=3.0)
        y, mean, rstd = sv.layer_norm(x, w, b, return_stats=True)
        dx, dw, db = sv.layer_norm_backward(dy, x, mean, rstd, w)
        return y, dw, db, sv.embedding_backward(dx, ids, vocab, scale=3.0)

    data = [(ids_for(k, tokens, vocab, torch.int64, 10 + i), hidden(tokens, dim, BF16, 20 + i))
            for i, k in enumerate(("skewed", "same", "uniform"))]
    want = []
    for i, d in data:
        ids.copy_(i)
        dy.copy_(d)
        want.append([t.clone() for t in block()])
    s = torch.cuda.Stream()
    graphs = []
    for _ in range(2):  # two graphs, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = block()
        graphs.append((g, out))
    for rep in range(6):
        i = rep % 3
        ids.copy_(data[i][0])
        dy.copy_(data[i][1])
        eager = block()
        torch.cuda.synchronize()
        for g, out in graphs:
            for t in out:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want[i])), rep
        assert all(torch.equal(p, q) for p, q in zip(eager, want[i])), rep


def test_block_on_two_streams(dev):
    vocab, dim, tokens = 500, 640, 3000
    sets = []
    for i in range(2):
        sets.append((ids_for("skewed", tokens, vocab, torch.int64, i), hidden(tokens, dim, F32, i),
                     torch.randn(vocab, dim, generator=gen(i), device=dev), *params(dim, F32, i)))

    def block(ids, dy, table, w, b):
        x = sv.embedding(ids, table)
        y, mean, rstd = sv.layer_norm(x, w, b, return_stats=True)
        dx, dw, db = sv.layer_norm_backward(dy, x, mean, rstd, w)
        return y, dw, db, sv.embedding_backward(dx, ids, vocab)

    want = [block(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(block(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[i]))


def test_c_abi_row_strides_leave_the_gaps_alone(dev):
    L = sv.capi()
    st = torch.cuda.current_stream().cuda_stream
    rows, vocab = 37, 50
    for dtype, code in ((F32, 0), (BF16, 1), (F16, 2)):
        for n, gap in ((5, 1), (64, 3), (100, 8), (1531, 5), (4096, 1), (20000, 7), (40001, 2)):
            x, dy = hidden(rows, n, dtype, n), hidden(rows, n, dtype, n + 1)
            w, b = params(n, F32, 1)
            y, mean, rstd = sv.layer_norm(x, w, b, return_stats=True)
            wide = torch.full((rows, n + gap), 7.0, dtype=dtype, device=dev)
            assert L.sv_layer_norm(x.data_ptr(), code, rows, n, n, w.data_ptr(), b.data_ptr(), 0, 1e-5,
                                   wide.data_ptr(), n + gap, None, None, st) == 0
            assert torch.equal(wide[:, :n], y) and (wide[:, n:] == 7).all(), (n, gap)
            want = sv.layer_norm_backward(dy, x, mean, rstd, w)[0]
            wide.fill_(7.0)
            assert L.sv_layer_norm_backward(dy.data_ptr(), n, x.data_ptr(), n, code, rows, n, w.data_ptr(), 0,
                                            mean.data_ptr(), rstd.data_ptr(), wide.data_ptr(), n + gap, None, None,
                                            None, 0, st) == 0
            assert torch.equal(wide[:, :n], want) and (wide[:, n:] == 7).all(), (n, gap)
            ids = ids_for("skewed", rows, vocab, torch.int64, n)
            want = sv.embedding_backward(dy, ids, vocab)
            grad = torch.full((vocab, n + gap), 7.0, dtype=dtype, device=dev)
            need = L.sv_embedding_backward_workspace_size(rows, vocab, n, code)
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
            assert L.sv_embedding_backward(dy.data_ptr(), n, ids.data_ptr(), 8, rows, code, vocab, n, 1.0, -1,
                                           grad.data_ptr(), n + gap, ws.data_ptr(), need, st) == 0
            assert torch.equal(grad[:, :n], want) and (grad[:, n:] == 7).all(), (n, gap)
            assert L.sv_embedding(ids.data_ptr(), 8, rows, grad.data_ptr(), code, vocab, n, n + gap, 1.0,
                                  wide.data_ptr(), n + gap, st) == 0
            assert torch.equal(wide[:, :n], want[ids]) and (wide[:, n:] == 7).all(), (n, gap)


def test_short_rows_are_independent_of_their_batch(dev):
    for dtype in TYPES:
        for n in range(1, 12):
            x, dy = hidden(300, n, dtype, n), hidden(300, n, dtype, n + 20)
            w, b = params(n, dtype, n)
            y, mean, rstd = check_forward(x, w, b)
            dx = check_backward(x, dy, w)[0]
            for r in (0, 150, 299):
                one = sv.layer_norm(x[r:r + 1], w, b, return_stats=True)
                assert torch.equal(one[0], y[r:r + 1]) and torch.equal(one[1], mean[r:r + 1])
                assert torch.equal(sv.layer_norm_backward(dy[r:r + 1], x[r:r + 1], one[1], one[2], w)[0], dx[r:r + 1])


def test_many_equal_tokens(dev):
    # runs of more than 64, 4096 and 64 * 64 pieces
    for tokens in (2049, 2080, 4095, 4096, 4097, 131072, 131105, 270001):
        dy = hidden(tokens, 8, F32, tokens)
        check_lookup_grad(dy, ids_for("same", tokens, 9, torch.int32, 1), 9)
        two = ids_for("same", tokens, 9, torch.int32, 1).clone()
        two[::3] = 8
        check_lookup_grad(dy, two, 9)


# ---------------------------------------------------------------- refusals

def test_refusals(dev):
    x, w = torch.zeros(4, 8, device=dev), torch.ones(8, device=dev)
    s = torch.zeros(4, device=dev)
    ids = torch.zeros(3, dtype=torch.int64, device=dev)
    for call in (lambda: sv.layer_norm(x, w[:7]), lambda: sv.layer_norm(x, w[None]),
                 lambda: sv.layer_norm(x[0, 0]), lambda: sv.layer_norm(x, w.cpu()),
                 lambda: sv.layer_norm_backward(x[:3], x, s, s), lambda: sv.layer_norm_backward(x, x, s[:3], s),
                 lambda: sv.layer_norm_backward(x, x, s, s[:, None]),
                 lambda: sv.embedding(ids, x[0]), lambda: sv.embedding(ids.cpu(), x),
                 lambda: sv.embedding(ids, x, padding_idx=4), lambda: sv.embedding(ids, x, padding_idx=-1),
                 lambda: sv.embedding_backward(x, ids, 9), lambda: sv.embedding_backward(x[:3], ids, -1),
                 lambda: sv.embedding_backward(x[:3, 0], ids, 9),
                 lambda: sv.embedding_backward(x[:3], ids, 9, padding_idx=9)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sv.layer_norm(x.double()), lambda: sv.layer_norm(x, w.to(BF16)),
                 lambda: sv.layer_norm(x.to(BF16), w.to(F16)), lambda: sv.layer_norm(x.to(BF16), w, w.to(BF16)),
                 lambda: sv.layer_norm_backward(x.to(BF16), x, s, s), lambda: sv.layer_norm_backward(x, x, s.to(BF16), s),
                 lambda: sv.layer_norm_backward(x, x, s, s, param_dtype=BF16),
                 lambda: sv.layer_norm_backward(x, x, s, s, w, param_dtype=BF16),
                 lambda: sv.embedding(ids.to(torch.int16), x), lambda: sv.embedding(ids, x.double()),
                 lambda: sv.embedding_backward(x[:3].long(), ids, 9)):
        with pytest.raises(TypeError):
            call()
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(sv.SvError):
            sv.layer_norm(x, eps=eps)
