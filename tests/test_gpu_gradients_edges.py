"""Clipping where its limit or the norm is no number, and of tensors that share
memory until one of them is written."""
import pytest
import torch

import stable_variance_amd as sv
from test_gpu_gradients import tensors
from test_gpu_rms import IDS, TYPES, dev, general_way  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(params=["short", "general"])
def way(request, monkeypatch):
    if request.param == "general":
        general_way(monkeypatch)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS.get)
@pytest.mark.parametrize("bad", [INF, -INF])
def test_no_limit_scales_nothing(dev, way, dtype, bad):
    # max_norm = Inf asks for the norm alone, whatever it is but NaN
    ts = tensors([5, 20000, 4097], [dtype], 1)
    ts[1][17] = bad
    kept = [t.clone() for t in ts]
    out, norm = sv.clip_grad_norm(ts, INF)
    assert float(norm) == INF and all(torch.equal(o, t) for o, t in zip(out, kept))
    out, norm = sv.clip_grad_norm(ts, INF, out=ts)
    assert float(norm) == INF and all(torch.equal(o, t) for o, t in zip(ts, kept))
    # with a limit the factor is 0
    out, norm = sv.clip_grad_norm(ts, 1e308)
    assert float(norm) == INF and out[1][17].isnan()
    assert all((o == 0).sum() == o.numel() - i % 2 for i, o in enumerate(out))
    # a NaN stays one
    ts[0][3] = NAN
    out, norm = sv.clip_grad_norm(ts, INF)
    assert norm.isnan() and all(o.isnan().all() for o in out)


def test_no_limit_above_float32(dev, way):
    many = torch.full((10000,), 3e38, device=dev)  # the norm is beyond float32, and a number
    out, norm = sv.clip_grad_norm([many], INF)
    assert float(norm) == INF and torch.equal(out[0], many)


def test_shared_until_written(dev, way):
    # copy-on-write: a tensor and its lazy clone, one memory as long as they are read
    for dtype in TYPES:
        first = tensors([3000], [dtype], 1)[0]
        kept = first.clone()
        want = sv.clip_grad_norm([kept], 0.5)[0][0]
        lazy = torch._lazy_clone(first)
        got, _ = sv.clip_grad_norm([lazy], 0.5, out=[lazy])  # in place
        assert got[0] is lazy and torch.equal(lazy, want) and torch.equal(first, kept)
        lazy = torch._lazy_clone(first)
        sv.clip_grad_norm([first], 0.5, out=[lazy])  # from the other
        assert torch.equal(lazy, want) and torch.equal(first, kept)
        lazy = torch._lazy_clone(first)
        sv.clip_grad_norm([lazy], 0.5, out=[first])
        assert torch.equal(first, want) and torch.equal(lazy, kept)
