"""Layer norm and embedding on the host: refusals of the C ABI and of the
binding, workspace sizes.  Nothing here reaches a device."""
import ctypes

import pytest
import torch

import stable_variance_amd as sv

INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 5
P = ctypes.c_void_p(0x1000)    # never dereferenced: every call below fails on the host
ODD = ctypes.c_void_p(0x1001)
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def L():
    return sv.capi()


def norm(L, x=P, dtype=0, rows=4, n=8, ldx=8, w=None, b=None, pt=0, eps=1e-5, y=P, ldy=8):
    return L.sv_layer_norm(x, dtype, rows, n, ldx, w, b, pt, eps, y, ldy, None, None, None)


def test_layer_norm_refusals(L):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(n=-1), dict(ldx=7), dict(ldy=7), dict(x=None),
                dict(y=None), dict(x=ODD), dict(w=ODD), dict(b=ODD), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(pt=1), dict(pt=7), dict(dtype=1, pt=2)):
        assert norm(L, **bad) == INVALID, bad
        assert b"sv_layer_norm" in L.sv_last_error_message()
    assert norm(L, n=(1 << 27) + 1, ldx=1 << 28, ldy=1 << 28) == UNSUPPORTED
    assert norm(L, rows=1 << 30, n=1 << 10, ldx=1 << 10, ldy=1 << 10) == UNSUPPORTED
    assert norm(L, rows=1 << 20, ldx=1 << 40) == UNSUPPORTED
    assert norm(L, rows=(1 << 36) + 1, n=0) == UNSUPPORTED
    assert norm(L, rows=0, x=None, y=None) == 0  # no rows: nothing to do


def norm_bwd(L, dy=P, lddy=8, x=P, ldx=8, dtype=0, rows=4, n=8, w=None, pt=0, mean=P, rstd=P, dx=P, lddx=8, dw=P,
             db=P, ws=P, wsb=1 << 30):
    return L.sv_layer_norm_backward(dy, lddy, x, ldx, dtype, rows, n, w, pt, mean, rstd, dx, lddx, dw, db, ws, wsb,
                                    None)


def test_layer_norm_backward_refusals(L):
    for bad in (dict(dtype=3), dict(rows=-1), dict(n=-1), dict(ldx=7), dict(lddy=7), dict(lddx=7), dict(x=None),
                dict(dy=None), dict(mean=None), dict(rstd=None), dict(x=ODD), dict(dy=ODD), dict(dx=ODD), dict(w=ODD),
                dict(dw=ODD), dict(db=ODD), dict(pt=2), dict(dtype=2, pt=1)):
        assert norm_bwd(L, **bad) == INVALID, bad
    need = L.sv_layer_norm_backward_workspace_size(4, 8, 0)
    assert need > 0
    assert norm_bwd(L, ws=None) == WORKSPACE
    assert norm_bwd(L, wsb=need - 1) == WORKSPACE
    assert norm_bwd(L, ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert norm_bwd(L, n=(1 << 27) + 1, ldx=1 << 28, lddy=1 << 28, lddx=1 << 28) == UNSUPPORTED
    assert norm_bwd(L, n=0) == 0
    assert norm_bwd(L, dx=None, dw=None, db=None, ws=None, wsb=0) == 0  # nothing asked for


def test_layer_norm_backward_workspace_sizes(L):
    size = L.sv_layer_norm_backward_workspace_size
    for rows, n in ((0, 8), (1, 1), (3, 5), (1 << 20, 64), (1, 1 << 27), (512, 1 << 27)):
        assert 0 < size(rows, n, 1) < 1 << 36, (rows, n)
    assert size(5, 0, 0) == 0
    for bad in ((-1, 8, 0), (8, -1, 0), (8, 8, 3), (1, (1 << 27) + 1, 0), (1 << 20, 1 << 20, 0)):
        assert size(*bad) == NONE, bad


def lookup(L, ids=P, idb=8, tokens=4, table=P, dtype=0, vocab=16, dim=8, ldt=8, out=P, ldo=8):
    return L.sv_embedding(ids, idb, tokens, table, dtype, vocab, dim, ldt, 1.0, out, ldo, None)


def test_embedding_refusals(L):
    for bad in (dict(dtype=3), dict(idb=2), dict(tokens=-1), dict(vocab=-1), dict(dim=-1), dict(ids=None),
                dict(table=None), dict(out=None), dict(ids=ODD), dict(table=ODD), dict(out=ODD), dict(ldt=7),
                dict(ldo=7)):
        assert lookup(L, **bad) == INVALID, bad
    assert lookup(L, tokens=(1 << 30) + 1) == UNSUPPORTED
    assert lookup(L, vocab=(1 << 31) - 1) == UNSUPPORTED
    assert lookup(L, dim=(1 << 27) + 1, ldt=1 << 28, ldo=1 << 28) == UNSUPPORTED
    assert lookup(L, vocab=1 << 30, dim=1 << 10, ldt=1 << 10, ldo=1 << 10) == UNSUPPORTED
    assert lookup(L, tokens=0, ids=None, out=None) == 0
    assert lookup(L, dim=0, table=None, out=None) == 0


def lookup_bwd(L, dy=P, lddy=8, ids=P, idb=8, tokens=4, dtype=0, vocab=16, dim=8, padding=-1, grad=P, ldg=8, ws=P,
               wsb=1 << 40):
    return L.sv_embedding_backward(dy, lddy, ids, idb, tokens, dtype, vocab, dim, 1.0, padding, grad, ldg, ws, wsb,
                                   None)


def test_embedding_backward_refusals(L):
    for bad in (dict(dtype=-1), dict(idb=3), dict(tokens=-1), dict(vocab=-1), dict(dim=-1), dict(ids=None),
                dict(dy=None), dict(grad=None), dict(ids=ODD), dict(dy=ODD), dict(grad=ODD), dict(lddy=7),
                dict(ldg=7), dict(padding=16), dict(padding=-2)):
        assert lookup_bwd(L, **bad) == INVALID, bad
    need = L.sv_embedding_backward_workspace_size(4, 16, 8, 0)
    assert need > 0
    assert lookup_bwd(L, ws=None) == WORKSPACE
    assert lookup_bwd(L, wsb=need - 1) == WORKSPACE
    assert lookup_bwd(L, ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert lookup_bwd(L, tokens=(1 << 30) + 1) == UNSUPPORTED
    assert lookup_bwd(L, vocab=0, grad=None) == 0
    size = L.sv_embedding_backward_workspace_size
    for bad in ((-1, 1, 1, 0), (1, -1, 1, 0), (1, 1, -1, 0), (1, 1, 1, 9), ((1 << 30) + 1, 1, 1, 0)):
        assert size(*bad) == NONE, bad
    assert size(0, 10, 10, 0) < NONE and size(1 << 30, 1000, 64, 1) < NONE


def test_binding_refusals_without_a_device():
    x = torch.zeros(4, 8)
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        sv.layer_norm(x)
    with pytest.raises(TypeError):
        sv.layer_norm([1.0])
    with pytest.raises(TypeError):
        sv.layer_norm(x.double())
    with pytest.raises(ValueError):
        sv.layer_norm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(TypeError):
        sv.embedding(ids, x.long())
    with pytest.raises(ValueError):
        sv.embedding(ids, x)
    with pytest.raises(ValueError):
        sv.embedding_backward(x[:3], ids, 10)
    with pytest.raises(TypeError):
        sv.embedding_backward(x[:3].double(), ids, 10)
    with pytest.raises(AttributeError):
        sv.no_such_operator
