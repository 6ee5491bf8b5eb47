"""Root-mean-square norm and the gradients' norm on the host: refusals of the C
ABI and of the binding, workspace sizes, launches within HIP's limit, and the
calls that reach the library.  Nothing here reaches a device."""
import contextlib
import ctypes
import json
import os
import shutil
import subprocess
import sys

import pytest
import torch
from torch.autograd import forward_ad

import stable_variance_amd as sv
from stable_variance_amd import gradients, layers

HERE = os.path.dirname(os.path.abspath(__file__))
INVALID, WORKSPACE, UNSUPPORTED = 1, 2, 5
P = ctypes.c_void_p(0x10000)  # never dereferenced: the calls below fail on the host or launch nothing
ODD = ctypes.c_void_p(0x10001)
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def L():
    return sv.capi()


# ---------------------------------------------------------------- refusals of the C ABI

def norm(L, x=P, ldx=8, res=None, ldr=8, dtype=0, sd=0, rows=4, n=8, w=None, pt=0, eps=1e-6, y=P, ldy=8, sum=None,
         lds=8):
    return L.sv_rms_norm(x, ldx, res, ldr, dtype, sd, rows, n, w, pt, eps, y, ldy, sum, lds, None, None)


def fp8(L, x=P, ldx=8, res=None, ldr=8, dtype=0, sd=0, rows=4, n=8, w=None, pt=0, eps=1e-6, to=3, block=128, q=P,
        ldq=8, scale=P, sum=None, lds=8):
    return L.sv_rms_norm_fp8(x, ldx, res, ldr, dtype, sd, rows, n, w, pt, eps, to, block, q, ldq, scale, sum, lds,
                             None, None)


SHARED = (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(n=-1), dict(ldx=7), dict(x=None), dict(x=ODD), dict(w=ODD),
          dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(pt=1), dict(dtype=1, sd=1, pt=2),
          dict(dtype=1, sd=2), dict(sd=1), dict(dtype=1, sd=0), dict(res=P), dict(sum=P), dict(res=P, sum=P, ldr=7),
          dict(res=P, sum=P, lds=7), dict(res=ODD, sum=P), dict(res=P, sum=ODD), dict(dtype=1, sd=0, res=P, sum=ODD))


def test_forward_refusals(L):
    for bad in SHARED + (dict(y=None), dict(y=ODD), dict(ldy=7)):
        assert norm(L, **bad) == INVALID, bad
        assert b"sv_rms_norm:" in L.sv_last_error_message()
    for bad in SHARED + (dict(q=None), dict(ldq=7), dict(scale=None), dict(scale=ODD), dict(to=0), dict(to=5),
                         dict(block=64), dict(block=-1), dict(block=256), dict(n=0, block=0, scale=None)):
        assert fp8(L, **bad) == INVALID, bad
        assert b"sv_rms_norm_fp8:" in L.sv_last_error_message()
    for call in (norm, fp8):
        out = "ldy" if call is norm else "ldq"
        assert call(L, n=(1 << 27) + 1, ldx=1 << 28, **{out: 1 << 28}) == UNSUPPORTED
        assert call(L, rows=1 << 30, n=1 << 10, ldx=1 << 10, **{out: 1 << 10}) == UNSUPPORTED
        assert call(L, rows=1 << 20, ldx=1 << 40) == UNSUPPORTED
        assert call(L, rows=1 << 20, res=P, sum=P, lds=1 << 40) == UNSUPPORTED
        assert call(L, rows=(1 << 36) + 1, n=0) == UNSUPPORTED
        assert call(L, rows=0, x=None) == 0  # no rows: nothing to do
        assert call(L, rows=0, x=None, dtype=1, sd=0) == 0  # an empty residual may be NULL


def backward(L, dy=P, lddy=8, h=P, ldh=8, ds=None, ldds=8, dtype=0, sd=0, rows=4, n=8, w=None, pt=0, rstd=P, dh=P,
             lddh=8, dx=None, lddx=8, dw=P, ws=P, wsb=1 << 30):
    return L.sv_rms_norm_backward(dy, lddy, h, ldh, ds, ldds, dtype, sd, rows, n, w, pt, rstd, dh, lddh, dx, lddx, dw, ws,
                                  wsb, None)


def test_backward_refusals(L):
    for bad in (dict(dtype=3), dict(rows=-1), dict(n=-1), dict(lddy=7), dict(ldh=7), dict(ds=P, ldds=7), dict(lddh=7),
                dict(dx=P, lddx=7), dict(dy=None), dict(h=None), dict(rstd=None), dict(dy=ODD), dict(h=ODD), dict(ds=ODD),
                dict(dh=ODD), dict(dx=ODD), dict(w=ODD), dict(dw=ODD), dict(pt=2), dict(sd=1), dict(dtype=2, sd=1)):
        assert backward(L, **bad) == INVALID, bad
    need = L.sv_rms_norm_backward_workspace_size(4, 8, 0, 0)
    assert need > 0
    assert backward(L, ws=None) == WORKSPACE
    assert backward(L, wsb=need - 1) == WORKSPACE
    assert backward(L, ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert backward(L, n=(1 << 27) + 1, ldh=1 << 28, lddy=1 << 28, lddh=1 << 28) == UNSUPPORTED
    assert backward(L, n=0) == 0
    assert backward(L, dh=None, dw=None, ws=None, wsb=0) == 0  # nothing asked for
    assert backward(L, rows=0, dw=None, ws=None, wsb=0) == 0
    size = L.sv_rms_norm_backward_workspace_size
    for rows, n in ((0, 8), (1, 1), (3, 5), (1 << 20, 64), (1, 1 << 27), (512, 1 << 27)):
        assert 0 < size(rows, n, 1, 0) < 1 << 36, (rows, n)
    assert size(5, 0, 0, 0) == 0
    for bad in ((-1, 8, 0, 0), (8, -1, 0, 0), (8, 8, 3, 3), (8, 8, 0, 1), (1, (1 << 27) + 1, 0, 0),
                (1 << 20, 1 << 20, 0, 0)):
        assert size(*bad) == NONE, bad


def arrays(tensors):
    """tensors: (address, size, dtype) each."""
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*[t[0] for t in tensors]), (ctypes.c_int64 * n)(*[t[1] for t in tensors]),
            (ctypes.c_int * n)(*[t[2] for t in tensors]), n)


def test_gradients_refusals(L):
    good = [(0x10000, 100, 0), (0x20000, 0, 1), (0x30000, 7, 2)]
    ptrs, sizes, codes, n = arrays(good)
    need = L.sv_grad_norm_workspace_size(sizes, codes, n)
    assert 256 < need < 1 << 20

    def grad(ts=good, norm=P, ws=P, wsb=1 << 30, count=None, **kw):
        p, s, c, k = arrays(ts)
        return L.sv_grad_norm(kw.get("p", p), kw.get("s", s), kw.get("c", c), k if count is None else count, norm, ws,
                              wsb, None)

    def clip(ts=good, out=None, m=1.0, norm=P, ws=P, wsb=1 << 30):
        p, s, c, k = arrays(ts)
        o = (ctypes.c_void_p * k)(*(out or [0x100000 * (i + 1) for i in range(k)]))
        return L.sv_clip_grad_norm(p, o, s, c, k, m, norm, ws, wsb, None)

    for call in (grad, clip):
        for bad in ([(0x10000, 5, 3)], [(0x10000, -1, 0)], [(0, 5, 0)], [(0x10002, 5, 0)], [(0x10001, 5, 1)],
                    good + [(0x10000, 5, -1)]):
            assert call(bad) == INVALID, bad
        assert call(norm=None) == INVALID and call(norm=ODD) == INVALID
        assert call([(0x10000, (1 << 40) + 1, 1)]) == UNSUPPORTED
        assert call(ws=None) == WORKSPACE
        assert call(wsb=need - 1) == WORKSPACE
        assert call(ws=ctypes.c_void_p(0x1010)) == WORKSPACE
    assert grad(count=-1) == INVALID
    assert grad(count=(1 << 20) + 1) == UNSUPPORTED
    for k in ("p", "s", "c"):
        assert grad(**{k: None}) == INVALID
    for bad in (-1.0, float("nan")):
        assert clip(m=bad) == INVALID
    for out in ([0, 0x20000, 0x30000], [0x10001, 0x20000, 0x30000], [0x40000, 0x20000, 0x30001]):
        assert clip(out=out) == INVALID
    assert L.sv_clip_grad_norm(ptrs, None, sizes, codes, n, 1.0, P, P, 1 << 30, None) == INVALID
    # what is written overlaps what is read or written for another tensor
    a, b = (0x10000, 100, 0), (0x10200, 100, 0)  # 400 bytes each, 512 apart
    for ts, out in (([a, a], [0x10000, 0x10000]), ([a, b], [0x10200, 0x10000]), ([a], [0x10004]), ([a, b], [0x10000, 0x10200 - 4]),
                    ([b, a], [0x10200, 0x10200 + 4]), ([a, b], [0x90000, 0x90000 + 396]), ([a, a], [0x10000, 0x90000])):
        assert clip(ts, out) == INVALID, (ts, out)
        assert b"overlaps" in L.sv_last_error_message()
    assert L.sv_grad_norm_workspace_size(None, None, 0) == 256
    for s, c in ((-1, 0), (5, 3), ((1 << 40) + 1, 0)):
        assert L.sv_grad_norm_workspace_size((ctypes.c_int64 * 1)(s), (ctypes.c_int * 1)(c), 1) == NONE
    assert L.sv_grad_norm_workspace_size(None, None, 1) == NONE


def test_binding_refusals_without_a_device():
    x, s = torch.zeros(4, 8), torch.zeros(4)
    for call in (lambda: sv.rms_norm(x), lambda: sv.rms_norm_fp8(x), lambda: sv.rms_norm_backward(x, x, s),
                 lambda: sv.grad_norm([x]), lambda: sv.grad_norm([]), lambda: sv.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sv.rms_norm([1.0]), lambda: sv.rms_norm(x.double()), lambda: sv.rms_norm_fp8(x.double()),
                 lambda: sv.rms_norm_backward(x.double(), x, s), lambda: sv.grad_norm(x), lambda: sv.grad_norm([1.0]),
                 lambda: sv.grad_norm([x.double()]), lambda: sv.clip_grad_norm([x.long()], 1.0)):
        with pytest.raises(TypeError):
            call()


# ---------------------------------------------------------------- launches

# run in a process of its own, with the recorder loaded before the HIP runtime
PROGRAM = r"""
import ctypes, json, sys
rec = ctypes.CDLL(sys.argv[1])
rec.recorded_launches.restype = rec.recorded_largest.restype = ctypes.c_uint64
sys.path.insert(0, sys.argv[2])
import stable_variance_amd as sv
L = sv.capi()
P = ctypes.c_void_p(0x10000)  # never dereferenced
out = []

def call(what, fn, *args):
    rec.recorded_clear()
    status = fn(*args)
    out.append([what, status, rec.recorded_launches(), rec.recorded_largest(),
                L.sv_last_error_message().decode() if status else ""])

for dtype, sd in ((0, 0), (1, 1), (1, 0), (2, 2)):
    for n in [1, 3, 64, 1531, 4096, 16384, 20001, 1 << 20, (1 << 27) - 64, (1 << 27) - 63, (1 << 27) - 1, 1 << 27]:
        for rows in sorted({1, 3, 70000, min(1 << 28, (1 << 36) // n), (1 << 36) // n}):
            if rows * n > 1 << 36:
                continue
            for res in (P, None):
                s = sd if res else dtype
                call(f"norm {dtype} {s} {rows} {n}", L.sv_rms_norm, P, n, res, n, dtype, s, rows, n, None, 0, 1e-6, P, n,
                     res, n, P, None)
                for block in (128, 0):
                    call(f"fp8 {dtype} {s} {rows} {n}", L.sv_rms_norm_fp8, P, n, res, n, dtype, s, rows, n, None, 0, 1e-6,
                         3, block, P, n, P, res, n, P, None)
            need = L.sv_rms_norm_backward_workspace_size(rows, n, dtype, sd)
            for ds in (P, None):
                for dw in (P, None):
                    call(f"gradient {dtype} {sd} {rows} {n} {ds} {dw}", L.sv_rms_norm_backward, P, n, P, n, ds, n, dtype,
                         sd, rows, n, None, 0, P, P, n, None, n, dw, P, need, None)

def tensors(sizes, dtype):
    n, at, ptrs = len(sizes), 0x100000, []
    for s in sizes:
        ptrs.append(at)
        at += s * 4 + 256 & -256
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*[dtype] * n), n)

for dtype in (0, 1, 2):
    for sizes in ([1], [0], [1 << 40], [1 << 40] * 9, [5] * 1000, [1 << 20] * 400, [0, 3, 1 << 31, 7]):
        p, s, c, n = tensors(sizes, dtype)
        need = L.sv_grad_norm_workspace_size(s, c, n)
        call(f"grad norm {dtype} {sizes[:4]}", L.sv_grad_norm, p, s, c, n, P, P, need, None)
        call(f"clip {dtype} {sizes[:4]}", L.sv_clip_grad_norm, p, p, s, c, n, 1.0, P, P, need, None)
print(json.dumps(out))
"""


def test_every_launch_is_within_the_limit(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    so = str(tmp_path / "launch_recorder.so")
    res = subprocess.run([gcc, "-O1", "-Wall", "-Werror", "-shared", "-fPIC", os.path.join(HERE, "launch_recorder.c"),
                          "-o", so], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    # before whatever else is preloaded here
    pre = " ".join(p for p in (so, os.environ.get("LD_PRELOAD", "")) if p)
    res = subprocess.run([sys.executable, "-c", PROGRAM, so, os.path.dirname(HERE)], capture_output=True, text=True,
                         timeout=600, env={**os.environ, "LD_PRELOAD": pre})
    assert res.returncode == 0, res.stderr[-4000:]
    calls = json.loads(res.stdout.strip().splitlines()[-1])
    assert len(calls) > 1000
    bad = [c for c in calls if c[1] != 0 or c[3] > 0xffffffff]
    assert not bad, bad[:10]
    assert all(c[2] > 0 for c in calls)  # the recorder saw the launches


# ---------------------------------------------------------------- what reaches the library

def values(address, rows, cols, stride):
    """A copy of the float32 [rows, cols] matrix at an address."""
    flat = (ctypes.c_float * ((rows - 1) * stride + cols)).from_address(address)
    return torch.tensor(list(flat)).as_strided((rows, cols), (stride, 1)).clone()


class Library:
    """The C ABI's float32 calls on host memory: they take the calls, and the
    clipping copies."""

    def __init__(self):
        self.calls = []

    def sv_rms_norm_backward_workspace_size(self, *_):
        return 0

    def sv_grad_norm_workspace_size(self, *_):
        return 256

    def sv_rms_norm(self, x, ldx, res, ldr, dtype, sd, rows, n, w, pt, eps, y, ldy, h, ldh, rstd, stream):
        self.calls.append(("rms", values(x, rows, n, ldx), res and values(res, rows, n, ldr), w and values(w, 1, n, n)))
        return 0

    def sv_rms_norm_fp8(self, x, ldx, res, ldr, dtype, sd, rows, n, w, pt, eps, to, block, q, ldq, scale, h, ldh, rstd,
                        stream):
        self.calls.append(("fp8", values(x, rows, n, ldx), res and values(res, rows, n, ldr), w and values(w, 1, n, n)))
        return 0

    def sv_rms_norm_backward(self, dy, lddy, h, ldh, ds, ldds, dtype, sd, rows, n, w, pt, rstd, dh, lddh, dx, lddx, dw,
                             ws, nbytes, stream):
        self.calls.append(("rms_grad", values(dy, rows, n, lddy), values(h, rows, n, ldh),
                           ds and values(ds, rows, n, ldds), w and values(w, 1, n, n), values(rstd, 1, rows, rows)))
        return 0

    def tensors(self, p, sizes, n):
        return [values(p[i], 1, sizes[i], sizes[i]) if sizes[i] else torch.empty(1, 0) for i in range(n)]

    def sv_grad_norm(self, p, sizes, codes, n, norm, ws, nbytes, stream):
        self.calls.append(("grad", *self.tensors(p, sizes, n)))
        return 0

    def sv_clip_grad_norm(self, p, out, sizes, codes, n, most, norm, ws, nbytes, stream):
        self.calls.append(("clip", *self.tensors(p, sizes, n)))
        for i in range(n):
            ctypes.memmove(out[i], p[i], 4 * sizes[i])
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
    monkeypatch.setattr(gradients, "_device_type", "cpu")
    for module in (layers, gradients):
        monkeypatch.setattr(module, "capi", lambda: lib)
        monkeypatch.setattr(module, "_on", lambda device: contextlib.nullcontext())
        monkeypatch.setattr(module, "_raw_stream", lambda index: 0)
    return lib


def inputs():
    g = torch.Generator().manual_seed(1)
    r = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    return dict(x=r(4, 6), res=r(4, 6), dy=r(4, 6), h=r(4, 6), ds=r(4, 6), w=r(6), rstd=r(4), a=r(3, 5), b=r(7))


CALLS = {
    "rms": (("x", "res", "w"), lambda v: sv.rms_norm(v["x"], v["w"], residual=v["res"])),
    "fp8": (("x", "res", "w"), lambda v: sv.rms_norm_fp8(v["x"], v["w"], residual=v["res"])),
    "rms_grad": (("dy", "h", "ds", "w", "rstd"),
                 lambda v: sv.rms_norm_backward(v["dy"], v["h"], v["rstd"], v["w"], v["ds"])),
    "grad": (("a", "b"), lambda v: sv.grad_norm([v["a"], v["b"]])),
    "clip": (("a", "b"), lambda v: sv.clip_grad_norm([v["a"], v["b"]], 1.0)),
}


@pytest.mark.parametrize("op", CALLS)
def test_a_tangent_is_refused(lib, op):
    names, call = CALLS[op]
    for name in names:
        for mode in (contextlib.nullcontext, torch.no_grad):
            v = inputs()
            with forward_ad.dual_level(), mode():
                v[name] = forward_ad.make_dual(v[name], torch.ones_like(v[name]))
                with pytest.raises(NotImplementedError):
                    call(v)
    assert lib.calls == []
    with forward_ad.dual_level():  # no input with a tangent
        call(inputs())
    call(inputs())
    assert [c[0] for c in lib.calls] == [op, op]


def test_a_tangent_of_the_result_gradient_is_refused(lib):
    v = inputs()
    v["x"].requires_grad_()
    y, _ = CALLS["rms"][1](v)
    with forward_ad.dual_level():
        dy = forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(NotImplementedError):
            y.backward(dy)
    assert v["x"].grad is None


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
        v = {k: t[..., :cols].contiguous() if t.shape[-1] == 6 else t for k, t in inputs().items()}
        call(v)
        for name in names:
            w = dict(v)
            w[name] = negated(v[name], dense)
            assert w[name].is_neg() and torch.equal(w[name], v[name])
            call(w)
        for got in lib.calls[1:]:
            assert all(p is q is None or torch.equal(p, q) for p, q in zip(got[1:], lib.calls[0][1:])), cols
        lib.calls.clear()


def test_clipping_writes_where_it_is_asked_to(lib):
    # the stand-in copies: out gets the values of grads, whatever the strides
    g = torch.Generator().manual_seed(2)
    base = torch.randn(8, 9, generator=g)
    forms = [lambda: base.clone(), lambda: base.clone().t(), lambda: base.clone()[:, 2:5], lambda: base.clone()[::3],
             lambda: torch._neg_view(-base), lambda: base[None, None], lambda: base[0, 0].clone(), lambda: base[:0].clone()]
    for make in forms:
        t = make()
        new, _ = sv.clip_grad_norm([t], 1.0)
        assert new[0].is_contiguous() and torch.equal(new[0], t)
        same, _ = sv.clip_grad_norm([t], 1.0, out=[t])
        assert same[0] is t and torch.equal(t, make())
        for form in forms:
            o = form()
            if o.shape == t.shape:
                o = o.clone(memory_format=torch.preserve_format) if o.is_neg() else o
                version = o._version
                o.zero_()
                got, _ = sv.clip_grad_norm([t], 1.0, out=[o])
                assert got[0] is o and torch.equal(o, t) and o._version > version + 1
    ts = [base.clone().t(), base.clone()]
    out, _ = sv.clip_grad_norm(ts, 1.0, out=ts)
    assert out == ts or all(p is q for p, q in zip(out, ts))
    cut = base[:, 1:4]
    with pytest.raises(ValueError):
        sv.clip_grad_norm([cut, cut], 1.0, out=[cut, cut])
    with pytest.raises(ValueError):
        sv.clip_grad_norm([torch.ones(1).expand(5)], 1.0, out=[torch.ones(1).expand(5)])
    with pytest.raises(ValueError):
        sv.clip_grad_norm([base], 1.0, out=[base.clone().requires_grad_()])
    with torch.no_grad():
        sv.clip_grad_norm([base], 1.0, out=[base.clone().requires_grad_()])


def test_dense_tensors():
    t = torch.zeros(2, 3, 4, 5)
    for good in (t, t.permute(3, 1, 0, 2), t.to(memory_format=torch.channels_last), t[:, :1].permute(1, 0, 3, 2).contiguous(),
                 torch.zeros(3, 0, 4).transpose(0, 2), torch.zeros(()), torch.zeros(1, 7).t(), t[1]):
        assert gradients._dense(good)
    for bad in (t[:, 1], t[..., ::2], t[..., :3], torch.zeros(1).expand(4), torch.zeros(3, 1).expand(3, 4),
                torch.zeros(20).as_strided((4, 4), (1, 1)), torch.zeros(20).as_strided((4, 4), (4, 2))):
        assert not gradients._dense(bad)


def test_the_native_module_leaves_host_tensors():
    m = sv.native()
    x, w, s = torch.zeros(3, 4), torch.ones(4), torch.ones(3)
    assert m.rms(x, w, None, 1e-6, False, 0, 0) is None and m.rms(x, w, x, 1e-6, True, 3, 128) is None
    assert m.rms(None, None, None, 1e-6, False, 0, 0) is None and m.rms([1.0], w, None, 1e-6, False, 0, 0) is None
    assert m.rms_backward(x, x, s, w, None, True, False, True) is None
    for bad in ([x], [], None, x, (x, w), [None]):
        assert m.grad_norm(bad) is None and m.clip_grad_norm(bad, 1.0, None) is None
    for call in (lambda: m.rms(x, w), lambda: m.rms(x, w, None, "eps", False, 0, 0), lambda: m.rms_backward(x),
                 lambda: m.clip_grad_norm([x], "most", None), lambda: m.clip_grad_norm([x])):
        with pytest.raises(TypeError):
            call()
