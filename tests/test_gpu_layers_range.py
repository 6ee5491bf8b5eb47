"""Layer norm and embedding on the GPU over the ranges that the header gives:
launches cut into batches, the longest rows, the smallest eps, many rows for
every tile, wide tables with long runs of tokens, many tokens, autograd in a
graph.  Bounds as in
test_gpu_layers.py, from whose checks in float64 these are built."""
import pytest
import torch

import stable_variance_amd as sv
from test_gpu_layers import (BF16, F16, F32, IDS, TYPES, check_backward, check_forward, check_lookup_grad,  # noqa: F401
                             dev, gen, hidden, ids_for, params)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- launches

@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_column_join_in_batches_gives_the_same_bits(dev, dtype):
    for rows, n in ((40, 200), (3, 4096), (700, 1531), (5, 20001)):
        w, _ = params(n, dtype, n)
        x, dy = hidden(rows, n, dtype, n), hidden(rows, n, dtype, n + 1)
        _, mean, rstd = sv.layer_norm(x, w, return_stats=True)
        want = sv.layer_norm_backward(dy, x, mean, rstd, w)
        for items in (1024, 5000):
            sv.set_tuning("launch_items", items)
            try:
                got = sv.layer_norm_backward(dy, x, mean, rstd, w)
                only = sv.layer_norm_backward(dy, x, mean, rstd, w, weight_grad=False)
            finally:
                sv.set_tuning("reset", 0)
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (rows, n, items)
            assert torch.equal(only[2], want[2])


def test_longest_rows(dev):
    # 2 * 2^21 tiles of 64 columns: more than one launch of the column join
    for n in ((1 << 27) - 63, 1 << 27):
        print("longest", n, flush=True)
        x, dy = hidden(2, n, BF16, 1), hidden(2, n, BF16, 2)
        w, _ = params(n, F32, 3)
        dx, dw, db = check_backward(x, dy, w)
        del x, dy, dx, dw, db
        torch.cuda.empty_cache()


# ---------------------------------------------------------------- eps

@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_equal_values_give_the_bias_for_the_smallest_eps(dev, dtype):
    # 1 / sqrt(eps) is beyond float32: no 0 * Inf, and no NaN in the gradients
    biggest = torch.finfo(F32).max
    for n in (1, 6, 128, 1531, 4096, 14000, 40000):
        x = torch.tensor([0.0, 1.0, -3.25], device=dev).to(dtype)[:, None].repeat(1, n)
        w, b = params(n, dtype, n)
        for eps in (8.6e-78, 1e-80, 1e-200, 5e-324):
            y, mean, rstd = sv.layer_norm(x, w, b, eps=eps, return_stats=True)
            assert torch.equal(y, b.expand_as(y)), (n, eps)
            assert torch.equal(mean, x[:, 0].float()) and (rstd == biggest).all(), (n, eps)
            dx, dw, db = sv.layer_norm_backward(torch.ones_like(x), x, mean, rstd, w)
            assert not dx.isnan().any() and (dw == 0).all() and (db == 3).all(), (n, eps)
        # in range: rounded as ever
        _, _, rstd = sv.layer_norm(x, w, b, eps=8.7e-78, return_stats=True)
        assert torch.equal(rstd, torch.full_like(rstd, float(torch.tensor(8.7e-78, dtype=torch.float64) ** -0.5)))


# ---------------------------------------------------------------- many rows

# Lengths that fill a tile, end on a 16-byte chunk and end inside one, for
# every tile of 128 threads and more.
LONG = [2048, 1600, 1999, 4096, 3000, 2050, 6144, 5000, 5003, 8192, 7000, 7001, 12288, 10000, 10001, 16384, 14000, 13001,
        32768, 20000, 20001]


def pick(rows):
    """Rows of the first, a middle and the last round of the launch."""
    return sorted({0, 1, rows // 3, rows // 2, rows - 300, rows - 2, rows - 1})


@pytest.mark.parametrize("dtype", [F32, BF16], ids=IDS.get)
def test_norm_many_long_rows(dev, dtype):
    # every group of threads takes at least two rows, most three: the launch
    # has 2048 workgroups of 256 threads (two rows of 128 threads each), 1024
    # of 512 and 512 of 1024
    for i, n in enumerate(LONG):
        rows = 77 + (8192 if n <= 2048 else 4096 if n <= 6144 else 2048 if n <= 12288 else 1024)
        print("many rows", IDS[dtype], rows, n, flush=True)
        w, b = params(n, dtype if i % 2 else F32, i)
        x = hidden(rows, n, dtype, i)
        whole = check_forward(x, w, b)
        for r in pick(rows):
            one = sv.layer_norm(x[r:r + 1], w, b, return_stats=True)
            assert all(torch.equal(p[r:r + 1], q) for p, q in zip(whole, one)), (n, r)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=IDS.get)
def test_norm_grad_many_long_rows(dev, dtype):
    # 256 workgroups of 1 to 6 groups: at least three rows per group
    for i, n in enumerate(LONG):
        rows = 3200 if n <= 2048 else 1700 if n <= 4096 else 1150 if n <= 6144 else 800
        print("many rows", IDS[dtype], rows, n, flush=True)
        w, _ = params(n, dtype if i % 2 else F32, i)
        x, dy = hidden(rows, n, dtype, i), hidden(rows, n, dtype, 900 + i)
        whole = check_backward(x, dy, w)
        for r in pick(rows):
            one = check_backward(x[r:r + 1], dy[r:r + 1], w)
            assert torch.equal(one[0], whole[0][r:r + 1]), (n, r)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=IDS.get)
def test_norm_grad_more_than_one_round_of_workgroups(dev, dtype):
    # more than 32 rows per group of 256 workgroups: 512 of them
    for rows, n in ((8300, 8192), (17000, 5003), (50000, 1600), (800000, 128)):
        print("rounds", IDS[dtype], rows, n, flush=True)
        w, _ = params(n, F32, n)
        x, dy = hidden(rows, n, dtype, 1), hidden(rows, n, dtype, 2)
        whole = check_backward(x, dy, w)
        for r in pick(rows):
            one = check_backward(x[r:r + 1], dy[r:r + 1], w)
            assert torch.equal(one[0], whole[0][r:r + 1]), (n, r)


# ---------------------------------------------------------------- wide tables

@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
def test_lookup_grad_wide_tiles_with_long_runs(dev, dtype):
    # tables and token lists from which two chunks per thread are taken, rows
    # that end inside the second chunk, take several tiles, or one; runs of
    # one token to all of them, in lists searched whole and by samples
    for i, (tokens, vocab, dim, kind) in enumerate((
            (9000, 17000, 1100, "skewed"), (4096, 17000, 1025, "skewed"), (5000, 20000, 600, "same"),
            (4097, 16400, 2049, "same"), (3000, 16384, 520, "skewed"), (70000, 16384, 1000, "skewed"),
            (40000, 20000, 4096, "skewed"), (600000, 300, 513, "skewed"))):
        print("wide", IDS[dtype], tokens, vocab, dim, kind, flush=True)
        ids = ids_for(kind, tokens, vocab, torch.int64 if i % 2 else torch.int32, i)
        dy = hidden(tokens, dim, dtype, i)
        scale = (1.0, 0.37)[i % 2]
        whole = check_lookup_grad(dy, ids, vocab, scale=scale)
        assert torch.equal(whole, sv.embedding_backward(dy, ids, vocab, scale=scale))
        # the same tokens alone, into a table that takes the narrow tiles
        rows = [0, 1, 2, 40, 199] if kind == "skewed" else [vocab // 2]
        for v in rows:
            at = (ids == v).nonzero()[:, 0]
            if len(at) == 0 or len(at) > 500000:
                continue
            alone = sv.embedding_backward(dy[at], torch.zeros_like(at), 1, scale=scale)
            assert torch.equal(alone[0], whole[v]), (tokens, vocab, dim, v, len(at))


# ---------------------------------------------------------------- many tokens

def test_lookup_of_more_tokens_than_one_grid(dev):
    # 2^23 workgroups of 32 tokens each, then a second round
    tokens, vocab = (1 << 28) + 77, 1000
    table = torch.arange(vocab, device=dev, dtype=F32).to(F16)[:, None]
    ids = torch.arange(tokens, device=dev, dtype=torch.int32).remainder_(vocab)
    out = sv.embedding(ids, table, scale=2.0)
    assert out.shape == (tokens, 1) and torch.equal(out[:, 0], ids.to(F16) * 2)


def test_lookup_grad_of_many_tokens(dev):
    tokens, vocab = (1 << 27) + 77, 5
    ids = torch.arange(tokens, device=dev, dtype=torch.int32).remainder_(vocab)
    # whole numbers of mean 0: every partial sum (tens of thousands at most) is
    # exact in float32, and so is the result
    dy = torch.randint(-2, 3, (tokens, 2), generator=gen(1), device=dev).float()
    got = sv.embedding_backward(dy, ids, vocab, scale=0.5)
    want = torch.stack([dy[v::vocab].double().sum(0) for v in range(vocab)])
    assert torch.equal(got.double(), want * 0.5)


# ---------------------------------------------------------------- autograd in a graph

def test_block_with_autograd_captured_and_replayed(dev):
    vocab, dim, tokens = 300, 520, 700
    table = torch.randn(vocab, dim, generator=gen(1), device=dev).to(BF16)
    w, b = params(dim, F32, 1)
    ids = ids_for("skewed", tokens, vocab, torch.int64, 1).clone()
    dy = hidden(tokens, dim, BF16, 2).clone()

    def explicit():
        x = sv.embedding(ids, table, scale=3.0)
        y, mean, rstd = sv.layer_norm(x, w, b, return_stats=True)
        dx, dw, db = sv.layer_norm_backward(dy, x, mean, rstd, w)
        return y, sv.embedding_backward(dx, ids, vocab, scale=3.0), dw, db

    data = [(ids_for(k, tokens, vocab, torch.int64, 10 + i), hidden(tokens, dim, BF16, 20 + i))
            for i, k in enumerate(("skewed", "same", "uniform"))]
    explicit()
    torch.cuda.synchronize()
    # leaves of their own that no eager graph holds
    leaves = [t.clone().requires_grad_() for t in (table, w, b)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        y = sv.layer_norm(sv.embedding(ids, leaves[0], scale=3.0), leaves[1], leaves[2])
        out = (y.detach(), *torch.autograd.grad(y, leaves, dy))
    del y
    for rep in range(6):
        ids.copy_(data[rep % 3][0])
        dy.copy_(data[rep % 3][1])
        want = explicit()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), rep
