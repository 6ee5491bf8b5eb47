"""The binding of the layer norm and the embedding on host tensors, with the
library replaced by a stand-in that computes the lookup and otherwise only
takes the calls: which calls reach the library, and with which data."""
import contextlib
import ctypes

import pytest
import torch
from torch.autograd import forward_ad

import stable_variance_amd as sv
from stable_variance_amd import layers


def values(address, rows, cols, stride):
    """A copy of the float32 [rows, cols] matrix at an address."""
    flat = (ctypes.c_float * ((rows - 1) * stride + cols)).from_address(address)
    return torch.tensor(list(flat)).as_strided((rows, cols), (stride, 1)).clone()


class Library:
    """The C ABI's float32 calls on host memory."""

    def __init__(self):
        self.calls = []

    def sv_layer_norm_backward_workspace_size(self, *_):
        return 0

    def sv_embedding_backward_workspace_size(self, *_):
        return 0

    def sv_layer_norm(self, x, dtype, rows, n, ldx, w, b, pt, eps, y, ldy, mean, rstd, stream):
        self.calls.append(("norm", values(x, rows, n, ldx), w and values(w, 1, n, n), b and values(b, 1, n, n)))
        return 0

    def sv_layer_norm_backward(self, dy, lddy, x, ldx, dtype, rows, n, w, pt, mean, rstd, dx, lddx, dw, db, ws, nbytes,
                               stream):
        self.calls.append(("norm_grad", values(dy, rows, n, lddy), values(x, rows, n, ldx), w and values(w, 1, n, n),
                           values(mean, 1, rows, rows), values(rstd, 1, rows, rows)))
        return 0

    def sv_embedding(self, ids, id_bytes, tokens, table, dtype, vocab, dim, ldt, scale, out, ldo, stream):
        self.calls.append(("lookup", values(table, vocab, dim, ldt)))
        return 0

    def sv_embedding_backward(self, dy, lddy, ids, id_bytes, tokens, dtype, vocab, dim, scale, padding, grad, ldg, ws,
                              nbytes, stream):
        self.calls.append(("lookup_grad", values(dy, tokens, dim, lddy)))
        return 0


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    real = layers._tensor

    def check(t, name, dtypes):
        try:
            real(t, name, dtypes)
        except ValueError as e:
            if "must be on a HIP device" not in str(e):
                raise

    monkeypatch.setattr(layers, "_tensor", check)
    monkeypatch.setattr(layers, "capi", lambda: lib)
    monkeypatch.setattr(layers, "_on", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(layers, "_raw_stream", lambda index: 0)
    return lib


def inputs():
    g = torch.Generator().manual_seed(1)
    r = lambda *shape: torch.randn(*shape, generator=g)
    return dict(x=r(4, 6), dy=r(4, 6), w=r(6), b=r(6), mean=r(4), rstd=r(4), table=r(5, 6),
                ids=torch.tensor([0, 4, 4, 2]))


CALLS = {
    "norm": (("x", "w", "b"), lambda v: sv.layer_norm(v["x"], v["w"], v["b"])),
    "norm_grad": (("dy", "x", "mean", "rstd", "w"),
                  lambda v: sv.layer_norm_backward(v["dy"], v["x"], v["mean"], v["rstd"], v["w"])),
    "lookup": (("table",), lambda v: sv.embedding(v["ids"], v["table"])),
    "lookup_grad": (("dy",), lambda v: sv.embedding_backward(v["dy"], v["ids"], 5)),
}


@pytest.mark.parametrize("op", CALLS)
def test_a_tangent_is_refused(lib, op):
    # no forward-mode derivative is provided: a result without its tangent
    # would be taken for a constant
    names, call = CALLS[op]
    for name in names:
        for requires_grad in (False, True):
            for mode in (contextlib.nullcontext, torch.no_grad):
                v = inputs()
                with forward_ad.dual_level(), mode():
                    p = v[name].requires_grad_(requires_grad)
                    v[name] = forward_ad.make_dual(p, torch.ones_like(p))
                    with pytest.raises(NotImplementedError):
                        call(v)
    assert lib.calls == []
    with forward_ad.dual_level():  # no input with a tangent
        call(inputs())
    call(inputs())
    assert [c[0] for c in lib.calls] == [op, op]


@pytest.mark.parametrize("op", ["norm", "lookup"])
def test_a_tangent_of_the_result_gradient_is_refused(lib, op):
    v = inputs()
    leaf = "x" if op == "norm" else "table"
    v[leaf].requires_grad_()
    y = CALLS[op][1](v)
    with forward_ad.dual_level():
        dy = forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError):
            y.backward(dy)
    assert v[leaf].grad is None


def negated(t, dense):
    """A view of -t that torch negates as it is read (the negative bit set)."""
    if dense:
        return torch._neg_view(-t)
    z = torch.complex(torch.zeros_like(t), -t)  # an imaginary part: strides of 2
    return z.conj().imag


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("op", CALLS)
def test_the_negative_bit_reaches_the_library_as_values(lib, op, dense):
    names, call = CALLS[op]
    for cols in (6, 1):  # single columns are taken with any stride
        v = {k: t[..., :cols].contiguous() if t.dim() == 2 or k in ("w", "b") else t for k, t in inputs().items()}
        call(v)
        for name in names:
            w = dict(v)
            w[name] = negated(v[name], dense)
            assert w[name].is_neg() and torch.equal(w[name], v[name])
            call(w)
        for got in lib.calls[1:]:
            assert all(p is q is None or torch.equal(p, q) for p, q in zip(got[1:], lib.calls[0][1:])), cols
        lib.calls.clear()


def test_arguments_that_are_no_tensors(lib):
    v = inputs()
    for requires_grad in (False, True):
        v["x"].requires_grad_(requires_grad)
        for w, b in (([1.0] * 6, None), (v["w"], 0.5), (None, [0.0] * 6), (1.0, v["b"])):
            with pytest.raises(TypeError):
                sv.layer_norm(v["x"], w, b)
    assert lib.calls == []


def test_numbers_of_rows_are_whole(lib):
    # 1.5 was taken for 1
    v = inputs()
    for bad in (1.5, 2.0, "3", torch.tensor(1.0)):
        with pytest.raises(TypeError):
            sv.embedding(v["ids"], v["table"], padding_idx=bad)
        with pytest.raises(TypeError):
            sv.embedding_backward(v["dy"], v["ids"], 5, padding_idx=bad)
        with pytest.raises(TypeError):
            sv.embedding_backward(v["dy"], v["ids"], bad)
    assert lib.calls == []
    for good in (4, torch.tensor(4), True):
        sv.embedding(v["ids"], v["table"], padding_idx=good)
        sv.embedding_backward(v["dy"], v["ids"], 5, padding_idx=good)
