"""Root-mean-square norm on the GPU with many rows for every tile: several
rounds of rows per workgroup, inputs larger than the last-level cache (which
are loaded another way), the longest rows, more than one round of workgroups in
the backward pass.  Bounds as in test_gpu_rms.py, from whose checks in float64
these are built."""
import pytest
import torch

import stable_variance_amd as sv
from test_gpu_rms import (BF16, E4M3, E5M2, F16, F32, IDS, PAIR_IDS, PAIRS, STREAM_IDS, STREAMS,  # noqa: F401
                          check_backward, check_forward, check_fp8, dev, hidden, weights)

pytestmark = pytest.mark.gpu

# Lengths that fill a tile, end on a chunk and end inside one.
WHOLE = [8, 40, 64, 128, 200, 256, 512, 1024, 1536, 2048, 4096, 6144, 8192, 12288, 16384, 20000, 32768]
RAGGED = [3, 7, 13, 57, 121, 251, 509, 1021, 1531, 2045, 4093, 5003, 8190, 12283, 16381, 20001, 32763]


def width(t):
    return torch.finfo(t).bits // 8


def pick(rows):
    """Rows of the first, a middle and the last round of the launch."""
    return sorted({0, 1, rows // 3, rows // 2, max(0, rows - 300), rows - 2, rows - 1})


def same(p, q):
    return torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
def test_inputs_beyond_the_cache(dev, dtype, stream):
    each = width(dtype) + (width(stream) if stream else 0)
    for i, n in enumerate(WHOLE):
        rows = (264 << 20) // (n * each) + 3
        print("beyond the cache", IDS[dtype], IDS[stream], rows, n, flush=True)
        x, r = hidden(rows, n, dtype, i), hidden(rows, n, stream, 50 + i) if stream else None
        w = weights(n, dtype if i % 2 else F32, i)
        whole = check_forward(x, w, residual=r)
        for k in pick(rows):
            one = sv.rms_norm(x[k:k + 1], w, residual=None if r is None else r[k:k + 1], return_rstd=True)
            assert all(torch.equal(p[k:k + 1], q) for p, q in zip(whole, one)), (n, k)
        del whole


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
@pytest.mark.parametrize("block", [128, None])
def test_fp8_beyond_the_cache(dev, dtype, stream, block):
    each = width(dtype) + (width(stream) if stream else 0)
    for i, n in enumerate(WHOLE):
        rows = (264 << 20) // (n * each) + 3
        print("fp8 beyond the cache", IDS[dtype], IDS[stream], block, rows, n, flush=True)
        x, r = hidden(rows, n, dtype, i), hidden(rows, n, stream, 50 + i) if stream else None
        w, to = weights(n, dtype if i % 2 else F32, i), E5M2 if i % 3 == 1 else E4M3
        whole = check_fp8(x, w, to, block, residual=r)
        for k in pick(rows):
            one = sv.rms_norm_fp8(x[k:k + 1], w, residual=None if r is None else r[k:k + 1], dtype=to, block=block,
                                  return_rstd=True)
            assert all(same(p[k:k + 1], q) for p, q in zip(whole, one)), (n, k)
        del whole


@pytest.mark.parametrize("dtype,stream", STREAMS, ids=STREAM_IDS)
def test_many_ragged_rows(dev, dtype, stream):
    # at least two rows for every group of threads of the launch
    for i, n in enumerate(RAGGED):
        rows = 77 + (1 << 20 if n < 64 else 140000 if n < 512 else 20000 if n < 2048 else 5000 if n < 9000 else 2500)
        print("ragged", IDS[dtype], IDS[stream], rows, n, flush=True)
        x, r = hidden(rows, n, dtype, i), hidden(rows, n, stream, 50 + i) if stream else None
        w = weights(n, dtype if i % 2 else F32, i)
        whole = check_forward(x, w, residual=r)
        part = check_fp8(x[:rows // 2], w, E4M3, None if i % 2 else 128, residual=None if r is None else r[:rows // 2])
        for k in pick(rows):
            rk = None if r is None else r[k:k + 1]
            one = sv.rms_norm(x[k:k + 1], w, residual=rk, return_rstd=True)
            assert all(torch.equal(p[k:k + 1], q) for p, q in zip(whole, one)), (n, k)
            if k < rows // 2:
                one = sv.rms_norm_fp8(x[k:k + 1], w, residual=rk, block=None if i % 2 else 128, return_rstd=True)
                assert all(same(p[k:k + 1], q) for p, q in zip(part, one)), (n, k)
        del whole, part


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("with_sum", [False, True])
def test_gradients_beyond_the_cache(dev, dtype, stream, with_sum):
    each = width(dtype) + width(stream) * (2 if with_sum else 1)
    for i, n in enumerate(WHOLE):
        rows = (200 << 20) // (n * each) + 3
        print("gradient beyond the cache", IDS[dtype], IDS[stream], with_sum, rows, n, flush=True)
        h, dy = hidden(rows, n, stream, i), hidden(rows, n, dtype, 50 + i)
        d = hidden(rows, n, stream, 90 + i) if with_sum else None
        w = weights(n, dtype if i % 2 else F32, i)
        rstd = sv.rms_norm(h, return_rstd=True)[1]
        whole = check_backward(h, dy, w, d, rstd=rstd)
        for k in pick(rows):
            one = sv.rms_norm_backward(dy[k:k + 1], h[k:k + 1], rstd[k:k + 1], w, None if d is None else d[k:k + 1])
            assert torch.equal(one[0], whole[0][k:k + 1]), (n, k)
        del whole


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
def test_gradients_of_many_ragged_rows(dev, dtype, stream):
    # 256 workgroups of 1 to 1024 groups: at least three rows per group
    for i, n in enumerate(RAGGED):
        rows = 77 + (1 << 20 if n < 16 else 200000 if n < 64 else 60000 if n < 512 else 8000 if n < 2048 else 2000)
        print("ragged gradient", IDS[dtype], IDS[stream], rows, n, flush=True)
        h, dy = hidden(rows, n, stream, i), hidden(rows, n, dtype, 50 + i)
        d = hidden(rows, n, stream, 90 + i) if i % 2 else None
        w = weights(n, F32 if i % 2 else dtype, i)
        rstd = sv.rms_norm(h, return_rstd=True)[1]
        whole = check_backward(h, dy, w, d, rstd=rstd)
        for k in pick(rows):
            one = sv.rms_norm_backward(dy[k:k + 1], h[k:k + 1], rstd[k:k + 1], w, None if d is None else d[k:k + 1])
            assert torch.equal(one[0], whole[0][k:k + 1]), (n, k)
        del whole


@pytest.mark.parametrize("dtype", [F32, BF16], ids=IDS.get)
def test_gradients_in_more_than_one_round_of_workgroups(dev, dtype):
    # more than 32 rows per group of 256 workgroups: 512 of them
    for rows, n in ((8300, 8192), (17000, 5003), (50000, 1600), (800000, 128)):
        print("rounds", IDS[dtype], rows, n, flush=True)
        check_backward(hidden(rows, n, dtype, 1), hidden(rows, n, dtype, 2), weights(n, F32, n))


def test_longest_rows(dev):
    # 2^21 tiles of 64 columns in the join
    for n in ((1 << 27) - 63, 1 << 27):
        print("longest", n, flush=True)
        x = hidden(2, n, BF16, 1)
        w = weights(n, BF16, 3)
        check_forward(x, w, residual=x)
        check_fp8(x, w, E4M3, 128)
        check_fp8(x, w, E4M3, None)
        torch.cuda.empty_cache()
        check_backward(x, hidden(2, n, BF16, 2), w, x)
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, F16], ids=IDS.get)
def test_column_join_in_batches_gives_the_same_bits(dev, dtype):
    for rows, n in ((40, 200), (3, 4096), (700, 1531), (5, 40001)):
        w = weights(n, dtype, n)
        h, dy = hidden(rows, n, dtype, n), hidden(rows, n, dtype, n + 1)
        rstd = sv.rms_norm(h, return_rstd=True)[1]
        want = sv.rms_norm_backward(dy, h, rstd, w)
        for items in (1024, 5000):
            sv.set_tuning("launch_items", items)
            try:
                got = sv.rms_norm_backward(dy, h, rstd, w)
            finally:
                sv.set_tuning("reset", 0)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (rows, n, items)


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
def test_column_sums_of_one_workgroup(dev, dtype, stream):
    # a batch that one workgroup holds writes the weight's gradient itself:
    # the same sums as with a row of zeros far behind, which takes a second one
    for n in (5, 64, 300, 1531, 4096, 8192, 16384):
        for rows in (1, 2, 3):
            w = weights(n, dtype, n)
            h, dy = hidden(rows, n, stream, n), hidden(rows, n, dtype, n + 1)
            rstd = sv.rms_norm(h, return_rstd=True)[1]
            one = check_backward(h, dy, w, rstd=rstd)
            more = torch.zeros(3000, n, dtype=dtype, device=dev)
            more[:rows] = dy
            wide = hidden(3000, n, stream, 3).clone()
            wide[:rows] = h
            long = torch.ones(3000, device=dev)
            long[:rows] = rstd
            check_backward(wide, more, w, rstd=long)
            assert torch.equal(one[0], sv.rms_norm_backward(more, wide, long, w)[0][:rows])


def test_more_than_2_31_values(dev):
    rows, n = 525_000, 4096
    assert rows * n > 1 << 31
    x = torch.empty(rows, n, dtype=BF16, device=dev)
    for i in range(0, rows, 75_000):
        x[i:i + 75_000] = hidden(75_000, n, BF16, i)
    w = weights(n, F32, 1)
    y, h, rstd = sv.rms_norm(x, w, residual=x, return_rstd=True)
    q, scale, h8 = sv.rms_norm_fp8(x, w, residual=x)
    dh, dw = sv.rms_norm_backward(x, h, rstd, w, y)
    for k in (0, 1, 262_144, 524_287, 524_288, rows - 2, rows - 1):
        one = check_forward(x[k:k + 1], w, residual=x[k:k + 1])
        assert all(torch.equal(p[k:k + 1], v) for p, v in zip((y, h, rstd), one)), k
        one8 = check_fp8(x[k:k + 1], w, E4M3, 128, residual=x[k:k + 1])
        assert all(same(p[k:k + 1], v) for p, v in zip((q, scale, h8), one8)), k
        back = check_backward(h[k:k + 1], x[k:k + 1], w, y[k:k + 1], rstd=rstd[k:k + 1])
        assert torch.equal(dh[k:k + 1], back[0]), k
    want, size = torch.zeros(n, dtype=torch.float64, device=dev), torch.zeros(n, dtype=torch.float64, device=dev)
    for i in range(0, rows, 75_000):
        t = x[i:i + 75_000].double() * (h[i:i + 75_000].double() * rstd[i:i + 75_000].double()[:, None])
        want += t.sum(0)
        size += t.abs().sum(0)
    # two roundings a term, runs of at most 48, joined with compensation
    assert ((dw.double() - want).abs() <= 3 * 2.0 ** -24 * want.abs() + 52 * 2.0 ** -24 * size).all()
