"""The weight's gradient where compensation decides.

The columns' terms dy * xhat are given exactly (rstd = 1, and values of few bits
in h and dy).  A batch of 250 rows gives no thread of the held rows' kernel more
than one, so nothing is added up in plain float32 there; the joins, within a
workgroup and of the workgroups' sums, are compensated, and so is every sum of
the kernels for longer rows.  What is left are the rounding of the large
workgroup sum to float32 and that of the result: U of the value each.
"""
import pytest
import torch

import stable_variance_amd as sv
from test_gpu_rms import PAIR_IDS, PAIRS, TINY, U, close, dev, gen, half, hidden, weights  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = 250
LARGE, SMALL = 2.0 ** 25, 1.9375  # SMALL is below half a step of LARGE: plain float32 loses each one behind it


def column_sums(h, dy, rstd=None, w=None):
    rstd = torch.ones(h.shape[0], device=h.device) if rstd is None else rstd
    return sv.rms_norm_backward(dy, h, rstd, w)[1]


def test_what_plain_float32_would_lose():
    # the test below can fail: the tolerance is 4, the loss 480
    s = torch.tensor(LARGE)
    for _ in range(ROWS - 1):
        s = s + SMALL
    want = LARGE + SMALL * (ROWS - 1)
    assert want - float(s) == SMALL * (ROWS - 1) > 100 * 2.01 * U * want


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("n", [5, 8, 64, 136, 300, 1531, 4096, 8192, 12288, 12290, 16384, 20001, 40000])
def test_small_terms_beside_a_large_one(dev, dtype, stream, n):
    want = torch.full((n,), LARGE + SMALL * (ROWS - 1), dtype=torch.float64, device=dev)
    for large in (0, 1, ROWS // 2, ROWS - 1):
        h, dy = torch.ones(ROWS, n, dtype=stream, device=dev), torch.full((ROWS, n), SMALL, dtype=dtype, device=dev)
        h[large], dy[large] = 2.0 ** 12, 2.0 ** 13
        close(column_sums(h, dy), want, 2.01 * U * want, f"dweight, large row {large}")


@pytest.mark.parametrize("dtype,stream", PAIRS, ids=PAIR_IDS)
def test_one_workgroup_and_many_give_the_same_sums(dev, dtype, stream):
    # few rows, which one workgroup adds up by itself, and the same with rows
    # whose terms are zeros far behind, which many do
    for n in (5, 64, 300, 1531, 4096, 8192, 16384, 20001):
        for rows in (1, 2, 3):
            for w in (None, weights(n, dtype, n)):
                def both(h, dy, rstd):
                    more = torch.zeros(3000, n, dtype=dtype, device=dev)
                    wide = hidden(3000, n, stream, 3).clone()
                    long = torch.ones(3000, device=dev)
                    more[:rows], wide[:rows], long[:rows] = dy, h, rstd
                    return column_sums(h, dy, rstd, w), column_sums(wide, more, long, w)

                whole = [torch.randint(-8, 9, (rows, n), generator=gen(n + i), device=dev).to(t)
                         for i, t in enumerate((stream, dtype))]
                few, many = both(*whole, torch.ones(rows, device=dev))
                exact = (whole[0].double() * whole[1].double()).sum(0)
                assert torch.equal(few.double(), exact.to(few.dtype).double()) and torch.equal(few, many), (n, rows)
                h, dy = hidden(rows, n, stream, n), hidden(rows, n, dtype, n + 1)
                few, many = both(h, dy, sv.rms_norm(h, return_rstd=True)[1])
                # each within the result's half step and a rounding of the same sum
                close(few, many.double(), 2 * (half(few.dtype) + U) * (1 + 2 ** -6) * many.double().abs()
                      + 2 * TINY[few.dtype], (n, rows))
