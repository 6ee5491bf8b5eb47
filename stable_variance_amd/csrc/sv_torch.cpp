// The binding's short way from torch tensors to the C ABI: a CPython module
// for the calls of the root-mean-square norm and of the gradients' norm.
//
// Every function takes the arguments of the Python function of its name and
// does what that does for ordinary ones: tensors on the current device whose
// values, or whose rows, lie in order in memory, nothing to record for
// autograd.  For anything else, and wherever the library refuses the call, it
// returns None and has launched nothing; the Python function then takes the
// general way, which converts or raises.  A failed launch raises here: some of
// the call may have run.  Other threads run while a call allocates and
// launches, both of which may wait for the device.  A call of rms_norm costs
// the host 5 us here and 9 us there (its launch alone 3), a grad_norm over 37
// tensors 9 and 28.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <vector>

#include "../../include/stable_variance.h"

namespace {

int code_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return SV_DTYPE_F32;
    case at::kBFloat16: return SV_DTYPE_BF16;
    case at::kHalf: return SV_DTYPE_F16;
    default: return -1;
  }
}

// An ordinary tensor of one of the three types: no subclass, no wrapper, in
// device memory.
const at::Tensor *strided(PyObject *obj) {
  if (!THPVariable_CheckExact(obj)) return nullptr;
  const at::Tensor &t = THPVariable_Unpack(obj);
  if (t.layout() != at::kStrided || !t.is_cuda() || !t.has_storage() || code_of(t) < 0 || t.is_neg()) return nullptr;
  return &t;
}

// All of its values in order, too.
const at::Tensor *ordinary(PyObject *obj) {
  const at::Tensor *t = strided(obj);
  return t && t->is_contiguous() ? t : nullptr;
}

// The distance between the rows (of the last dimension) of a tensor that has
// values, each row in order and all rows equally far apart; 0 for another.
int64_t row_stride(const at::Tensor &t) {
  const int64_t n = t.size(-1);
  if (t.is_contiguous()) return n;
  if (n > 1 && t.stride(-1) != 1) return 0;
  int64_t ld = -1, next = 0;  // -1: one row so far
  for (int64_t i = t.dim() - 2; i >= 0; --i) {
    if (t.size(i) == 1) continue;
    if (ld < 0) ld = t.stride(i);
    else if (t.stride(i) != next) return 0;
    next = t.stride(i) * t.size(i);
  }
  return ld < 0 ? n : ld >= n ? ld : 0;
}

bool records(const at::Tensor *t) { return t && t->requires_grad(); }

// Lets other threads run Python as long as it lives: no Python object is
// touched meanwhile, and the tensors in use are held by the caller's arguments
// or by a List.
class Released {
 public:
  Released() : state_(PyEval_SaveThread()) {}
  ~Released() { PyEval_RestoreThread(state_); }
  Released(const Released &) = delete;

 private:
  PyThreadState *state_;
};

// What a call returns for a status that is not SV_OK: None where the library
// refused it, the binding's exception where a launch failed.
PyObject *not_done(sv_status st) {
  if (st != SV_ERR_HIP) Py_RETURN_NONE;
  PyObject *package = PyImport_ImportModule("stable_variance_amd");
  if (!package) return nullptr;
  PyObject *none = PyObject_CallMethod(package, "_check", "i", (int)st);  // raises
  Py_DECREF(package);
  return none;
}

// rms(x, weight, residual, eps, rstd, out_dtype, block): rms_norm for out_dtype
// 0, else rms_norm_fp8 with the type code and the block (0: whole rows).
PyObject *rms(PyObject *, PyObject *const *args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 7) return PyErr_Format(PyExc_TypeError, "rms takes 7 arguments");
  const double eps = PyFloat_AsDouble(args[3]);
  const bool want_rstd = PyObject_IsTrue(args[4]) == 1;
  const long to = PyLong_AsLong(args[5]), block = PyLong_AsLong(args[6]);
  if (PyErr_Occurred()) return nullptr;
  const bool has_w = args[1] != Py_None, has_r = args[2] != Py_None;
  const at::Tensor *x = strided(args[0]), *w = has_w ? ordinary(args[1]) : nullptr,
                   *r = has_r ? strided(args[2]) : nullptr;
  if (!x || (has_w && !w) || (has_r && !r) || x->dim() < 1 || x->numel() == 0) Py_RETURN_NONE;
  if (c10::GradMode::is_enabled() && (records(x) || records(w) || records(r))) Py_RETURN_NONE;
  const int64_t n = x->size(-1), rows = x->numel() / n;
  const int code = code_of(*x), wcode = w ? code_of(*w) : code, rcode = r ? code_of(*r) : code;
  const c10::Device device = x->device();
  if (device.index() != c10::hip::current_device()) Py_RETURN_NONE;
  if (w && (w->dim() != 1 || w->size(0) != n || w->device() != device)) Py_RETURN_NONE;
  if (r && (r->sizes() != x->sizes() || r->device() != device)) Py_RETURN_NONE;
  if ((wcode != code && wcode != SV_DTYPE_F32) || (rcode != code && rcode != SV_DTYPE_F32)) Py_RETURN_NONE;
  const int64_t ldx = row_stride(*x), ldr = r ? row_stride(*r) : n;
  if (!ldx || !ldr) Py_RETURN_NONE;

  at::Tensor y, h, scale, rstd;
  sv_status st;
  {
    Released others;
    const auto options = x->options().requires_grad(false);
    y = at::empty(x->sizes(),
                  to == 0 ? options : options.dtype(to == SV_DTYPE_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2));
    if (r) h = at::empty(x->sizes(), r->options().requires_grad(false));
    const auto lead = x->sizes().slice(0, x->dim() - 1);
    if (want_rstd) rstd = at::empty(lead, options.dtype(at::kFloat));
    if (to != 0) {
      std::vector<int64_t> shape(lead.begin(), lead.end());
      shape.push_back(block ? (n + block - 1) / block : 1);
      scale = at::empty(shape, options.dtype(at::kFloat));
    }
    const auto at_of = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
    const void *wp = w ? w->const_data_ptr() : nullptr, *rp = r ? r->const_data_ptr() : nullptr;
    void *stream = c10::hip::getCurrentHIPStream(device.index()).stream();
    st = to == 0 ? sv_rms_norm(x->const_data_ptr(), ldx, rp, ldr, code, rcode, rows, n, wp, wcode, eps, at_of(y), n,
                               at_of(h), n, (float *)at_of(rstd), stream)
                 : sv_rms_norm_fp8(x->const_data_ptr(), ldx, rp, ldr, code, rcode, rows, n, wp, wcode, eps, (int)to,
                                   block, at_of(y), n, (float *)at_of(scale), at_of(h), n, (float *)at_of(rstd), stream);
  }
  if (st != SV_OK) return not_done(st);
  if (to == 0 && !r && !want_rstd) return THPVariable_Wrap(y);
  PyObject *out = PyTuple_New(1 + (to != 0) + has_r + want_rstd);
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(y));
  if (to != 0) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(scale));
  if (r) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(h));
  if (want_rstd) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(rstd));
  return out;
  END_HANDLE_TH_ERRORS
}

// rms_backward(dy, h, rstd, weight, dsum, dh, dx, dweight): the gradients that
// are asked for by the last three, (dh, dx, dweight) with None for the others.
PyObject *rms_backward(PyObject *, PyObject *const *args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 8) return PyErr_Format(PyExc_TypeError, "rms_backward takes 8 arguments");
  const bool has_d = args[4] != Py_None;
  const at::Tensor *dy = strided(args[0]), *h = strided(args[1]), *rstd = ordinary(args[2]), *w = ordinary(args[3]),
                   *d = has_d ? strided(args[4]) : nullptr;
  if (!dy || !h || !rstd || !w || (has_d && !d) || h->dim() < 1 || h->numel() == 0) Py_RETURN_NONE;
  const int64_t n = h->size(-1), rows = h->numel() / n;
  const int code = code_of(*dy), hcode = code_of(*h), wcode = code_of(*w);
  const c10::Device device = h->device();
  if (device.index() != c10::hip::current_device() || dy->device() != device || rstd->device() != device ||
      w->device() != device || (d && d->device() != device))
    Py_RETURN_NONE;
  if (dy->sizes() != h->sizes() || (d && (d->sizes() != h->sizes() || code_of(*d) != hcode)) ||
      rstd->sizes() != h->sizes().slice(0, h->dim() - 1) || code_of(*rstd) != SV_DTYPE_F32 || w->dim() != 1 ||
      w->size(0) != n)
    Py_RETURN_NONE;
  if ((wcode != code && wcode != SV_DTYPE_F32) || (hcode != code && hcode != SV_DTYPE_F32)) Py_RETURN_NONE;
  const int64_t lddy = row_stride(*dy), ldh = row_stride(*h), ldd = d ? row_stride(*d) : n;
  if (!lddy || !ldh || !ldd) Py_RETURN_NONE;

  at::Tensor out[3];
  const at::Tensor *like[3] = {h, dy, w};
  bool wanted[3];
  for (int i = 0; i < 3; ++i) wanted[i] = PyObject_IsTrue(args[5 + i]) == 1;
  sv_status st;
  {
    Released others;
    at::Tensor ws;
    void *p[3] = {nullptr, nullptr, nullptr};
    for (int i = 0; i < 3; ++i)
      if (wanted[i]) {
        out[i] = at::empty(like[i]->sizes(), like[i]->options().requires_grad(false));
        p[i] = out[i].data_ptr();
      }
    const size_t bytes = p[2] ? sv_rms_norm_backward_workspace_size(rows, n, code, hcode) : 0;
    if (bytes == (size_t)-1) {
      st = SV_ERR_UNSUPPORTED;
    } else {
      if (p[2]) ws = at::empty({(int64_t)bytes}, h->options().requires_grad(false).dtype(at::kByte));
      st = sv_rms_norm_backward(
          dy->const_data_ptr(), lddy, h->const_data_ptr(), ldh, d ? d->const_data_ptr() : nullptr, ldd, code, hcode,
          rows, n, w->const_data_ptr(), wcode, (const float *)rstd->const_data_ptr(), p[0], n, p[1], n, p[2],
          ws.defined() ? ws.data_ptr() : nullptr, bytes, c10::hip::getCurrentHIPStream(device.index()).stream());
    }
  }
  if (st != SV_OK) return not_done(st);
  PyObject *result = PyTuple_New(3);
  if (!result) return nullptr;
  for (int i = 0; i < 3; ++i) {
    if (out[i].defined()) {
      PyTuple_SET_ITEM(result, i, THPVariable_Wrap(out[i]));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(result, i, Py_None);
    }
  }
  return result;
  END_HANDLE_TH_ERRORS
}

// The tensors of a list as the C ABI takes them; they live as long as this,
// whatever another thread does to the list (a tuple of its own holds them: 0.3
// us for 37, where counting the tensors' own references takes 0.7).
struct List {
  THPObjectPtr held;
  std::vector<const at::Tensor *> t;
  std::vector<void *> p;
  std::vector<int64_t> n;
  std::vector<int> type;
};

// false: not a list or tuple of ordinary tensors on the current device.
// `written`: they get values.  A tensor that shares its memory until it is
// written (torch's copy-on-write) then gets its own here, so the list that is
// written comes before the one that is read.
bool list_of(PyObject *obj, List &l, bool written = false) {
  if (!PyList_CheckExact(obj) && !PyTuple_CheckExact(obj)) return false;
  l.held = PySequence_Tuple(obj);
  if (!l.held) throw python_error();
  const Py_ssize_t count = PyTuple_GET_SIZE(l.held.get());
  if (!count) return false;
  c10::DeviceIndex device = -1;
  l.t.reserve(count);
  l.p.reserve(count);
  l.n.reserve(count);
  l.type.reserve(count);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor *t = ordinary(PyTuple_GET_ITEM(l.held.get(), i));
    if (!t) return false;
    if (i == 0) device = c10::hip::current_device();  // not before there is a tensor on a device
    if (t->device().index() != device) return false;
    l.t.push_back(t);
    l.p.push_back(written ? t->data_ptr() : const_cast<void *>(t->const_data_ptr()));
    l.n.push_back(t->numel());
    l.type.push_back(code_of(*t));
  }
  return true;
}

// The norm of `l` and, with `out`, the scaled tensors; the library's status.
sv_status norm_of(const List &l, void *const *out, double max_norm, at::Tensor &norm) {
  const int64_t count = (int64_t)l.t.size();
  const size_t bytes = sv_grad_norm_workspace_size(l.n.data(), l.type.data(), count);
  if (bytes == (size_t)-1) return SV_ERR_UNSUPPORTED;
  const auto options = at::TensorOptions().device(l.t[0]->device());
  norm = at::empty({}, options.dtype(at::kFloat));
  const at::Tensor ws = at::empty({(int64_t)bytes}, options.dtype(at::kByte));
  void *stream = c10::hip::getCurrentHIPStream(l.t[0]->device().index()).stream();
  return out ? sv_clip_grad_norm(l.p.data(), out, l.n.data(), l.type.data(), count, max_norm, (float *)norm.data_ptr(),
                                 ws.data_ptr(), bytes, stream)
             : sv_grad_norm(l.p.data(), l.n.data(), l.type.data(), count, (float *)norm.data_ptr(), ws.data_ptr(),
                            bytes, stream);
}

PyObject *grad_norm(PyObject *, PyObject *grads) {
  HANDLE_TH_ERRORS
  List l;
  if (!list_of(grads, l)) Py_RETURN_NONE;
  at::Tensor norm;
  sv_status st;
  {
    Released others;
    st = norm_of(l, nullptr, 0.0, norm);
  }
  if (st != SV_OK) return not_done(st);
  return THPVariable_Wrap(norm);
  END_HANDLE_TH_ERRORS
}

// clip_grad_norm(grads, max_norm, out)
PyObject *clip_grad_norm(PyObject *, PyObject *const *args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 3) return PyErr_Format(PyExc_TypeError, "clip_grad_norm takes 3 arguments");
  const double max_norm = PyFloat_AsDouble(args[1]);
  if (PyErr_Occurred()) return nullptr;
  List l, given;
  const bool has_out = args[2] != Py_None;
  if ((has_out && !list_of(args[2], given, true)) || !list_of(args[0], l)) Py_RETURN_NONE;
  std::vector<at::Tensor> made;
  std::vector<void *> p;
  if (has_out) {
    if (given.t.size() != l.t.size()) Py_RETURN_NONE;
    for (size_t i = 0; i < l.t.size(); ++i) {
      if (given.t[i]->sizes() != l.t[i]->sizes() || given.type[i] != l.type[i] ||
          (c10::GradMode::is_enabled() && given.t[i]->requires_grad()))
        Py_RETURN_NONE;
    }
    p = given.p;
  }
  at::Tensor norm;
  sv_status st;
  {
    Released others;
    if (!has_out)
      for (const at::Tensor *t : l.t) {
        made.push_back(at::empty(t->sizes(), t->options().requires_grad(false)));
        p.push_back(made.back().data_ptr());
      }
    st = norm_of(l, p.data(), max_norm, norm);
  }
  if (st != SV_OK) return not_done(st);
  for (const at::Tensor *t : given.t)
    if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  THPObjectPtr outs(has_out ? PySequence_List(given.held.get()) : PyList_New((Py_ssize_t)made.size()));
  if (!outs) return nullptr;
  for (size_t i = 0; i < made.size(); ++i) PyList_SET_ITEM(outs.get(), (Py_ssize_t)i, THPVariable_Wrap(made[i]));
  return Py_BuildValue("NN", outs.release(), THPVariable_Wrap(norm));
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rms", (PyCFunction)(void (*)(void))rms, METH_FASTCALL, nullptr},
    {"rms_backward", (PyCFunction)(void (*)(void))rms_backward, METH_FASTCALL, nullptr},
    {"grad_norm", grad_norm, METH_O, nullptr},
    {"clip_grad_norm", (PyCFunction)(void (*)(void))clip_grad_norm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

// The torch and the Python whose headers these are, by which the build and the
// package know the file: with others it would reach into other layouts.
const char tag[] = SV_TORCH_TAG;

PyModuleDef module = {PyModuleDef_HEAD_INIT, "sv_torch", tag, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_sv_torch() { return PyModule_Create(&module); }
