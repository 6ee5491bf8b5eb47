"""The norm of many tensors and their clipping on the GPU against float64.

The sum of squares is held in double, so the norm is off by its own rounding to
float32 alone (u = 2^-24, with 2^-40 of slack for the sum and the root); the
factor is off by u, or below 2^-126, where float32's steps are 2^-149, by
2^-150; the scaled value by the product's u and its own rounding.
"""
import math

import pytest
import torch

import stable_variance_amd as sv
from test_gpu_rms import BF16, F16, F32, IDS, TINY, TYPES, U, close, dev, gen, half  # noqa: F401

pytestmark = pytest.mark.gpu


def tensors(sizes, dtypes, seed, scale=1.0):
    g = gen(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale * (0.2 + i % 5)).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def exact_norm(ts):
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))


def check_norm(ts):
    got = sv.grad_norm(ts)
    assert got.dtype == F32 and got.shape == ()
    want = exact_norm(ts)
    assert abs(float(got.double()) - want) <= (U + 2.0 ** -40) * want + 2.0 ** -150, (float(got), want)
    return got


def check_clip(ts, max_norm, **kw):
    before = [t.clone() for t in ts]
    want = exact_norm(before)
    out, norm = sv.clip_grad_norm(ts, max_norm, **kw)
    assert torch.equal(norm, sv.grad_norm(before))
    k = min(1.0, max_norm / (want + 1e-6))
    assert len(out) == len(ts)
    for i, (o, t) in enumerate(zip(out, before)):
        assert o.dtype == t.dtype and o.shape == t.shape
        if k == 1.0:
            assert torch.equal(o, t), i
        K = t.double() * k
        close(o, K, (half(t.dtype) + 2.01 * U) * K.abs() + TINY[t.dtype] + 2.0 ** -149
              + t.double().abs() * 2.0 ** -150, f"tensor {i}")
    return out, norm


SIZES = [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 1000, 2047, 2048, 4095, 4096, 4097, 8191, 8192, 8193, 16384, 16385, 100003]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_sizes(dev, dtype):
    for i, n in enumerate(SIZES):
        print("gradients", IDS[dtype], n, flush=True)
        check_norm(tensors([n], [dtype], i))
        check_clip(tensors([n], [dtype], i), 0.37)
        check_clip(tensors([n], [dtype], i), 1e6)
    check_norm(tensors(SIZES, [dtype], 5))
    check_clip(tensors(SIZES, [dtype], 5), 1.0)


@pytest.mark.parametrize("count", [1, 2, 127, 128, 129, 300, 1000])
def test_counts(dev, count):
    # more tensors than a launch holds, types mixed, empty ones among them
    sizes = [(i * 7919) % 5000 for i in range(count)]
    sizes[count // 2] = 70001
    ts = tensors(sizes, TYPES, count)
    check_norm(ts)
    check_clip(ts, 0.5)
    check_clip(ts, 0.5, out=ts)


def test_large(dev):
    # many units for every workgroup
    ts = tensors([120_000_001, 3, 50_000_000, 1, 4096 * 4096], [BF16, F32, F32], 1)
    check_norm(ts)
    check_clip(ts, 2.0)
    check_clip(ts, 2.0, out=ts)


def test_beyond_2_31_values(dev):
    t = torch.zeros((1 << 31) + 5001, dtype=F16, device=dev)
    t[-1] = 3.0
    t[1 << 31] = -4.0
    assert float(sv.grad_norm([t, t[:0]])) == 5.0
    out, norm = sv.clip_grad_norm([t], 1.0, out=[t])
    assert float(norm) == 5.0 and abs(float(t[-1]) - 0.6) <= 0.6 * 2.0 ** -11 and int(torch.count_nonzero(t)) == 2


def test_alignment_and_shapes_give_the_same_bits(dev):
    for dtype in TYPES:
        flat = torch.randn(60000, generator=gen(1), device=dev).to(dtype)
        sizes = [5001, 1, 777, 32000, 3, 10007]
        ts = list(flat[1:1 + sum(sizes)].split(sizes))  # at odd addresses
        copies = [t.clone() for t in ts]
        assert torch.equal(check_norm(ts), check_norm(copies))
        a, b = sv.clip_grad_norm(ts, 0.3)[0], sv.clip_grad_norm(copies, 0.3)[0]
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        shaped = [t.reshape(-1, 1, 1) for t in ts]
        assert torch.equal(sv.grad_norm(shaped), sv.grad_norm(ts))
        first = [t.clone() for t in sv.clip_grad_norm(shaped, 0.3, out=shaped)[0]]
        assert all(torch.equal(p.reshape(-1), q) for p, q in zip(first, a))
        assert (flat[0] == flat.clone()[0]) and torch.equal(flat[1:1 + sum(sizes)], torch.cat(a))
    zero_d = torch.tensor(-3.0, device=dev)
    assert float(sv.grad_norm([zero_d])) == 3.0


def test_neighbours_stay(dev):
    # nothing is written outside the tensors
    for dtype in TYPES:
        for n in (1, 3, 8, 100, 8191, 8193, 50001):
            flat = torch.full((n + 64,), 7.0, dtype=dtype, device=dev)
            flat[33:33 + n] = torch.randn(n, generator=gen(n), device=dev).to(dtype)
            out = torch.full((n + 64,), 5.0, dtype=dtype, device=dev)
            sv.clip_grad_norm([flat[33:33 + n]], 0.1, out=[out[31:31 + n]])
            assert (out[:31] == 5).all() and (out[31 + n:] == 5).all()
            sv.clip_grad_norm([flat[33:33 + n]], 0.1, out=[flat[33:33 + n]])
            assert (flat[:33] == 7).all() and (flat[33 + n:] == 7).all()
            assert torch.equal(flat[33:33 + n], out[31:31 + n])


def test_strides(dev):
    base = torch.randn(40, 50, generator=gen(1), device=dev)
    turned, cut, wide = base.clone().t(), base.clone()[:, 3:17], base.clone()[::2]
    channels = torch.randn(4, 3, 5, 6, generator=gen(2), device=dev).to(memory_format=torch.channels_last)
    ts = [turned, cut, wide, channels]
    check_norm(ts)
    want = [t.clone() for t in check_clip(ts, 0.5)[0]]
    got, _ = sv.clip_grad_norm(ts, 0.5, out=ts)
    # another order in memory is another order of the sum: the factor may be one step off
    for g, w, t in zip(got, want, ts):
        assert g is t
        close(g, w.double(), 3 * U * w.double().abs(), "strided")
    line = torch.ones(1, device=dev).expand(9)
    assert float(sv.grad_norm([line])) == 3.0
    check_clip([line], 1.0)
    with pytest.raises(ValueError):
        sv.clip_grad_norm([line], 1.0, out=[line])
    with pytest.raises(ValueError):
        sv.clip_grad_norm([cut, cut], 1.0, out=[cut, cut])
    neg = torch.randn(30, dtype=torch.complex64, generator=gen(3), device=dev).conj().imag
    assert neg.is_neg()
    check_norm([neg])
    check_clip([neg], 0.1)


def test_range(dev):
    # no square is beyond the range or below it
    for scale in (1e30, 1e-30, 1e-41):
        check_norm([torch.randn(5000, generator=gen(1), device=dev) * scale])
    check_norm([torch.full((3,), 3e38, device=dev) / 2, torch.full((70,), 1e-45, device=dev)])
    big = torch.randn(5000, generator=gen(1), device=dev) * 1e30
    check_clip([big, big.clone().to(BF16)], 1e-3)
    check_clip([torch.full((10,), 1e-30, device=dev)], 1e-31)
    many = torch.full((10000,), 3e38, device=dev)
    assert float(sv.grad_norm([many])) == float("inf")  # beyond float32
    out, _ = sv.clip_grad_norm([many], 1.0)  # but a number before it is rounded
    # the factor is 1 / 3e40, below 2^-126: off by up to 2^-150, here 2.2e-5 of it
    assert ((out[0] - 0.01).abs() <= 3 * U * 0.01 + 3e38 * 2.0 ** -150).all()


def test_zero_nan_and_inf(dev):
    z = [torch.zeros(5000, device=dev), torch.zeros(0, device=dev), torch.zeros(3, dtype=F16, device=dev)]
    assert float(sv.grad_norm(z)) == 0.0
    out, norm = sv.clip_grad_norm(z, 1.0)
    assert float(norm) == 0.0 and all((o == 0).all() for o in out)
    assert float(sv.grad_norm([torch.zeros(0, device=dev)])) == 0.0
    assert sv.clip_grad_norm([torch.zeros(0, device=dev)], 1.0)[0][0].shape == (0,)
    for dtype in TYPES:
        ts = tensors([3000, 20000], [dtype], 1)
        ts[0][17] = float("inf")
        out, norm = sv.clip_grad_norm(ts, 1.0)
        assert float(norm) == float("inf")
        assert out[0][17].isnan() and int(out[0].isnan().sum()) == 1
        assert (out[0][:17] == 0).all() and (out[1] == 0).all()
        ts[1][19999] = float("nan")
        out, norm = sv.clip_grad_norm(ts, 1.0)
        assert norm.isnan() and all(o.isnan().all() for o in out)
    ts = tensors([3000], [F32], 2)
    out, _ = sv.clip_grad_norm(ts, 0.0)
    assert (out[0] == 0).all()
    out, _ = sv.clip_grad_norm(ts, float("inf"))
    assert torch.equal(out[0], ts[0])


def test_in_place_counts_as_a_write(dev):
    t = torch.randn(100, generator=gen(1), device=dev)
    v = t._version
    sv.clip_grad_norm([t], 0.1, out=[t])
    assert t._version > v
    o = torch.empty_like(t)
    v, w = t._version, o._version
    got, _ = sv.clip_grad_norm([t], 0.1, out=[o])
    assert t._version == v and o._version > w and got[0] is o
    with torch.inference_mode():
        s = torch.ones(9, device=dev)
        sv.clip_grad_norm([s], 1.0, out=[s])
        assert ((s - 1 / 3).abs() < 1e-6).all()


def test_refusals(dev):
    a, b = torch.ones(100, device=dev), torch.ones(100, device=dev)
    for call in (lambda: sv.grad_norm([]), lambda: sv.grad_norm([a, b.cpu()]),
                 lambda: sv.clip_grad_norm([a], 1.0, out=[]), lambda: sv.clip_grad_norm([a], 1.0, out=[b[:50]]),
                 lambda: sv.clip_grad_norm([a], 1.0, out=[b.to(BF16)]),
                 lambda: sv.clip_grad_norm([a], 1.0, out=[b.clone().requires_grad_()])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sv.grad_norm(a), lambda: sv.grad_norm([a, None]), lambda: sv.grad_norm([a.double()]),
                 lambda: sv.grad_norm([a.long()]), lambda: sv.grad_norm([a.to_sparse()]),
                 lambda: sv.clip_grad_norm([a], 1.0, out=a)):
        with pytest.raises(TypeError):
            call()
    # memory that two tensors share, one of them written
    for ts, out in (([a, a], [a, a]), ([a, a[50:]], [a, a[50:]]), ([a, b], [b, a]), ([a[:60], a[40:]], None),
                    ([a[:60]], [a[40:]]), ([a, b], [b.clone(), b.clone()])):
        if out is None:
            sv.clip_grad_norm(ts, 1.0)  # read twice only: fine
            continue
        if all(o.data_ptr() not in (a.data_ptr(), b.data_ptr()) for o in out) and len(ts) == 2:
            sv.clip_grad_norm(ts, 1.0, out=out)
            continue
        with pytest.raises(sv.SvError):
            sv.clip_grad_norm(ts, 1.0, out=out)
    assert (a == 1).all() and (b == 1).all()
    for m in (-1.0, float("nan")):
        with pytest.raises(sv.SvError):
            sv.clip_grad_norm([a], m)


# ---------------------------------------------------------------- together

def model(seed, vocab=90, dim=136, layers=3, dtype=BF16):
    g = gen(seed)
    table = (0.5 * torch.randn(vocab, dim, generator=g, device="cuda")).to(dtype)
    ws = [(1 + 0.2 * torch.randn(dim, generator=g, device="cuda")) for _ in range(layers + 1)]
    ms = [(torch.randn(dim, dim, generator=g, device="cuda") / math.sqrt(dim)).to(dtype) for _ in range(layers)]
    ids = torch.randint(0, vocab, (4, 25), generator=g, device="cuda")
    dy = (0.1 * torch.randn(4, 25, dim, generator=g, device="cuda")).to(dtype)
    return table, ws, ms, ids, dy


def forward(table, ws, ms, ids):
    """Norm, product, residual, layer by layer, over embedded tokens."""
    h = sv.embedding(ids, table)
    y = sv.rms_norm(h, ws[0])
    for w, m in zip(ws[1:], ms):
        y, h = sv.rms_norm(y @ m, w, residual=h)
    return y


def test_a_training_step(dev):
    # through autograd in float32, against the same in float64 on the host
    table, ws, ms, ids, dy = model(1, dtype=F32)
    leaves = [t.clone().requires_grad_() for t in [table] + ws + ms]
    n = len(ws)
    y = forward(leaves[0], leaves[1:1 + n], leaves[1 + n:], ids)
    y.backward(dy)
    refs = [t.double().cpu().requires_grad_() for t in [table] + ws + ms]
    h = refs[0][ids.cpu()]
    norm = lambda v, w: v * (v.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * w  # noqa: E731
    z = norm(h, refs[1])
    for w, m in zip(refs[2:1 + n], refs[1 + n:]):
        h = z @ m + h
        z = norm(h, w)
    z.backward(dy.double().cpu())
    grads = [p.grad for p in leaves]
    # some hundred roundings a layer, four layers
    for g, r in zip(grads, refs):
        want = r.grad.to(dev)
        worst = float((g.double() - want).abs().max() / want.abs().max())
        assert worst < 2000 * U, worst
    total = math.sqrt(sum(float(r.grad.square().sum()) for r in refs))
    out, got = sv.clip_grad_norm(grads, 0.5 * total, out=grads)
    assert abs(float(got) - total) <= 2000 * U * total
    assert abs(float(sv.grad_norm(out)) - 0.5 * total) <= 2000 * U * total


def test_serving_agrees_with_training(dev):
    # a token alone gives the bits that it has in its batch
    table, ws, ms, ids, _ = model(2)
    h = sv.embedding(ids, table).reshape(-1, 136)
    x = (h.float() @ ms[0].float()).to(BF16)
    y, s = sv.rms_norm(x, ws[1], residual=h)
    q, scale, s8 = sv.rms_norm_fp8(x, ws[1], residual=h)
    assert torch.equal(s, s8)
    for i in (0, 50, 99):
        one = sv.rms_norm(x[i], ws[1], residual=h[i])
        assert torch.equal(one[0], y[i]) and torch.equal(one[1], s[i])
        one = sv.rms_norm_fp8(x[i], ws[1], residual=h[i])
        assert torch.equal(one[0].view(torch.uint8), q[i].view(torch.uint8)) and torch.equal(one[1], scale[i])


def step(x, r, w, dy, dsum):
    """One call of every operator; the gradients clipped in place."""
    y, h, rstd = sv.rms_norm(x, w, residual=r, return_rstd=True)
    q, scale, _ = sv.rms_norm_fp8(x, w, residual=r)
    dh, dw = sv.rms_norm_backward(dy, h, rstd, w, dsum)
    clipped, norm = sv.clip_grad_norm([dh, dw], 0.25)
    return [y, h, rstd, q.view(torch.uint8), scale, dh, dw, norm, sv.grad_norm([dw, dh, dw]), *clipped]


def data(i, rows=300, n=520):
    g = gen(i)
    r = lambda t: torch.randn(rows, n, generator=g, device="cuda").to(t)  # noqa: E731
    return [r(BF16), r(F32), 1 + 0.1 * torch.randn(n, generator=g, device="cuda"), r(BF16), r(F32)]


def test_captured_and_replayed(dev):
    inputs = [t.clone() for t in data(0)]
    sets = [data(i) for i in range(3)]
    want = [[t.clone() for t in step(*s)] for s in sets]
    stream = torch.cuda.Stream()
    graphs = []
    for _ in range(2):  # two graphs, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            out = step(*inputs)
        graphs.append((g, out))
    for rep in range(6):
        i = rep % 3
        for t, s in zip(inputs, sets[i]):
            t.copy_(s)
        eager = step(*inputs)
        torch.cuda.synchronize()
        for g, out in graphs:
            for t in out:
                t.fill_(77)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want[i])), rep
        assert all(torch.equal(p, q) for p, q in zip(eager, want[i])), rep


def test_on_two_streams(dev):
    sets = [data(i, rows=3000, n=640) for i in range(2)]
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(g, want[i]))


def test_autograd_captured(dev):
    # a backward pass in a graph, no eager graph of the same leaves alive
    x, r, w, dy, dsum = data(5)
    _, h, rstd = sv.rms_norm(x, w, residual=r, return_rstd=True)
    dh, dw = sv.rms_norm_backward(dy, h, rstd, w, dsum)
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]

    def backward():
        y, s = sv.rms_norm(leaves[0], leaves[1], residual=leaves[2])
        return torch.autograd.grad((y, s), leaves, (dy, dsum))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        backward()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = backward()
    for _ in range(3):
        for t in out:
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, (dh.to(BF16), dw, dh)))


def test_c_abi_row_strides_leave_the_gaps_alone(dev):
    from test_gpu_rms import hidden, weights

    L = sv.capi()
    st = torch.cuda.current_stream().cuda_stream
    rows = 37
    for dtype, code in ((F32, 0), (BF16, 1), (F16, 2)):
        for stream, scode in {(dtype, code), (F32, 0)}:
            for n, gap in ((5, 1), (64, 3), (100, 8), (1531, 5), (4096, 1), (20000, 7), (40001, 2)):
                x, r = hidden(rows, n, dtype, n), hidden(rows, n, stream, n + 1)
                dy, dsum = hidden(rows, n, dtype, n + 2), hidden(rows, n, stream, n + 3)
                w = weights(n, F32, 1)
                y, h, rstd = sv.rms_norm(x, w, residual=r, return_rstd=True)
                wy = torch.full((rows, n + gap), 7.0, dtype=dtype, device=dev)
                wh = torch.full((rows, n + gap + 1), 7.0, dtype=stream, device=dev)
                assert L.sv_rms_norm(x.data_ptr(), n, r.data_ptr(), n, code, scode, rows, n, w.data_ptr(), 0, 1e-6,
                                     wy.data_ptr(), n + gap, wh.data_ptr(), n + gap + 1, None, st) == 0
                assert torch.equal(wy[:, :n], y) and (wy[:, n:] == 7).all(), (n, gap)
                assert torch.equal(wh[:, :n], h) and (wh[:, n:] == 7).all(), (n, gap)
                q, scale, _ = sv.rms_norm_fp8(x, w, residual=r)
                wq = torch.full((rows, n + gap), 9, dtype=torch.uint8, device=dev)
                sc = torch.empty_like(scale)
                wh.fill_(7.0)
                assert L.sv_rms_norm_fp8(x.data_ptr(), n, r.data_ptr(), n, code, scode, rows, n, w.data_ptr(), 0, 1e-6,
                                         3, 128, wq.data_ptr(), n + gap, sc.data_ptr(), wh.data_ptr(), n + gap + 1, None,
                                         st) == 0
                assert torch.equal(wq[:, :n], q.view(torch.uint8)) and (wq[:, n:] == 9).all() and torch.equal(sc, scale)
                assert torch.equal(wh[:, :n], h) and (wh[:, n:] == 7).all(), (n, gap)
                dh = sv.rms_norm_backward(dy, h, rstd, w, dsum)[0]
                wy.fill_(7.0)
                wh.fill_(7.0)
                assert L.sv_rms_norm_backward(dy.data_ptr(), n, h.data_ptr(), n, dsum.data_ptr(), n, code, scode, rows,
                                              n, w.data_ptr(), 0, rstd.data_ptr(), wh.data_ptr(), n + gap + 1,
                                              wy.data_ptr(), n + gap, None, None, 0, st) == 0
                assert torch.equal(wh[:, :n], dh) and (wh[:, n:] == 7).all(), (n, gap)
                assert torch.equal(wy[:, :n], dh.to(dtype))  # dh is the float32 value, or in the same type
                assert (wy[:, n:] == 7).all(), (n, gap)


# ---------------------------------------------------------------- the two ways into the library

def test_both_ways_give_the_same(dev, monkeypatch):
    from test_gpu_rms import general_way

    sets = [tensors([5, 0, 4097, 100003], TYPES, 1), tensors([300] * 200, [BF16, F32], 2),
            [t.reshape(-1, 1) for t in tensors([64, 33], [F16], 3)]]
    short = []
    for ts in sets:
        mine = [t.clone() for t in ts]
        outs = [torch.empty_like(t) for t in ts]
        short.append([sv.grad_norm(ts), sv.grad_norm(tuple(ts)), *sv.clip_grad_norm(ts, 0.2)[0],
                      *sv.clip_grad_norm(ts, 0.2, out=outs)[0], *sv.clip_grad_norm(mine, 0.2, out=mine)[0],
                      sv.clip_grad_norm(ts, 0.2)[1]])
        got = sv.clip_grad_norm(ts, 0.2, out=outs)[0]
        assert type(got) is list and all(p is q for p, q in zip(got, outs))
    general_way(monkeypatch)
    for ts, want in zip(sets, short):
        mine = [t.clone() for t in ts]
        outs = [torch.empty_like(t) for t in ts]
        got = [sv.grad_norm(ts), sv.grad_norm(iter(ts)), *sv.clip_grad_norm(ts, 0.2)[0],
               *sv.clip_grad_norm(ts, 0.2, out=outs)[0], *sv.clip_grad_norm(mine, 0.2, out=mine)[0],
               sv.clip_grad_norm(ts, 0.2)[1]]
        assert len(got) == len(want)
        assert all(p.shape == q.shape and p.dtype == q.dtype and torch.equal(p, q) for p, q in zip(got, want))


def test_general_way_refuses_and_converts_too(dev, monkeypatch):
    from test_gpu_rms import general_way

    general_way(monkeypatch)
    test_refusals(dev)
    test_in_place_counts_as_a_write(dev)
    test_zero_nan_and_inf(dev)
    test_strides(dev)
    test_neighbours_stay(dev)


def test_the_short_way_leaves_the_others(dev):
    from stable_variance_amd import native

    m = native()
    a, b = torch.ones(100, device=dev), torch.ones(4, 5, device=dev)
    assert m.grad_norm([a, b]) is not None and m.grad_norm((a,)) is not None
    for bad in ([], (), iter([a]), a, None, [a, None], [a, b.t()], [a.cpu()], [a, a.double()], [a.to_sparse()],
                [a[::2]], [torch._neg_view(a)], [1.0]):
        assert m.grad_norm(bad) is None
        assert m.clip_grad_norm(bad, 1.0, None) is None
    c = a.clone()
    for out in ([], [c, c], [b], [c.to(BF16)], [c.cpu()], [c[:50]], c, [c.requires_grad_()]):
        assert m.clip_grad_norm([a], 1.0, out) is None
    for most in (-1.0, float("nan")):
        assert m.clip_grad_norm([a], most, None) is None
    assert m.clip_grad_norm([a, a], 1.0, [a, a]) is None  # written twice
    assert (a == 1).all()
    with pytest.raises(TypeError):
        m.clip_grad_norm([a], "x", None)
    with pytest.raises(TypeError):
        m.clip_grad_norm([a], 1.0)


def test_c_abi_without_tensors(dev):
    import ctypes

    L = sv.capi()
    st = torch.cuda.current_stream().cuda_stream
    ws = torch.full((256,), 7, dtype=torch.uint8, device=dev)
    norm = torch.full((), 9.0, device=dev)
    for sizes in ([], [0], [0, 0, 0]):
        n = len(sizes)
        p, s, t = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)()
        args = (p, s, t) if n else (None, None, None)
        norm.fill_(9.0)
        assert L.sv_grad_norm(*args, n, norm.data_ptr(), ws.data_ptr(), 256, st) == 0
        assert float(norm) == 0.0
        norm.fill_(9.0)
        assert L.sv_clip_grad_norm(args[0], args[0], *args[1:], n, 1.0, norm.data_ptr(), ws.data_ptr(), 256, st) == 0
        assert float(norm) == 0.0


def test_a_workspace_keeps_nothing(dev):
    # one workspace for calls of different lists in turn, as two graphs would
    # share it in stream order: what one call left does not reach the next
    import ctypes

    L = sv.capi()
    st = torch.cuda.current_stream().cuda_stream
    lists = [tensors([70000, 5, 300], TYPES, 1), tensors([3], [F32], 2), tensors([50] * 300, [BF16], 3)]
    arrays, need = [], 0
    for ts in lists:
        n = len(ts)
        a = ((ctypes.c_void_p * n)(*[t.data_ptr() for t in ts]), (ctypes.c_int64 * n)(*[t.numel() for t in ts]),
             (ctypes.c_int * n)(*[{F32: 0, BF16: 1, F16: 2}[t.dtype] for t in ts]), n)
        arrays.append(a)
        need = max(need, L.sv_grad_norm_workspace_size(a[1], a[2], n))
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device=dev)
    want = [sv.grad_norm(ts) for ts in lists]
    for _ in range(2):
        for a, w in zip(arrays, want):
            norm = torch.empty((), device=dev)
            assert L.sv_grad_norm(*a, norm.data_ptr(), ws.data_ptr(), need, st) == 0
            assert torch.equal(norm, w)


def test_many_tensors_of_one_value(dev):
    flat = torch.arange(1, 5001, device=dev, dtype=F32)
    ts = list(flat.split(1))
    got = check_norm(ts)
    assert abs(float(got) - math.sqrt(5000 * 5001 * 10001 / 6)) <= 2 * U * float(got)
    check_clip(ts, 1.0, out=ts)
    assert abs(float(flat.double().square().sum().sqrt()) - 1) < 1e-6
