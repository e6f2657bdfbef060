// The language-model operators' calls from Python: the same checks and the
// same C entries as _binding.py, without its interpreter time (6.3 us a call
// of rnn_scan_step become 3.1).  A call that fails a check returns None
// before anything is enqueued; _binding.py then finds and raises the error.
#include <Python.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "rnn.h"

namespace {

// the entries of the library that _binding.py has loaded
enum Entry { STEP, SCAN_FWD, SCAN_BWD, FFN_FWD, FFN_BWD, CKPT_SIZE, CKPT_STORE, CKPT_LOAD, ENTRIES };
void* entry[ENTRIES];
template <class F>
F* as(Entry e) { return reinterpret_cast<F*>(entry[e]); }

int choice(PyObject* o, std::initializer_list<const char*> names) {
  if (!PyUnicode_Check(o)) return -1;
  int i = 0;
  for (const char* n : names) {
    if (PyUnicode_CompareWithASCIIString(o, n) == 0) return i;
    ++i;
  }
  return -1;
}
int scan_mode(PyObject* o) { return choice(o, {"gated", "linear"}); }
int act(PyObject* o) { return choice(o, {"sigmoid", "silu", "gelu"}); }
int save(PyObject* o) { return choice(o, {"none", "full", "int8"}); }

using Sizes = std::initializer_list<int64_t>;

// What one call's tensors have in common, and whether every check held.
struct Call {
  bool ok = true;
  int dev = -1;
  at::ScalarType type = at::kFloat;

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  // the tensor that sets the call's type and device
  const at::Tensor* first(PyObject* o, int dims) {
    const at::Tensor* t = tensor(o);
    if (!ok) return nullptr;
    type = t->scalar_type();
    ok = t->is_cuda() && t->layout() == at::kStrided && t->dim() == dims && (type == at::kFloat || type == at::kBFloat16);
    if (!ok) return nullptr;
    for (int64_t n : t->sizes()) ok = ok && n <= 0x7fffffff;
    dev = t->get_device();
    return ok ? t : nullptr;
  }
  void* data(PyObject* o, at::ScalarType want, Sizes shape, bool optional = false) {
    if (!ok || (optional && o == Py_None)) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!ok) return nullptr;
    ok = t->is_cuda() && t->layout() == at::kStrided && t->get_device() == dev && t->scalar_type() == want &&
         t->sizes() == at::IntArrayRef(shape) && t->is_contiguous();
    return ok ? t->data_ptr() : nullptr;
  }
  void* room(PyObject* o, size_t& bytes, bool optional = false) {
    bytes = 0;
    if (!ok || (optional && o == Py_None)) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!ok) return nullptr;
    ok = t->is_cuda() && t->layout() == at::kStrided && t->get_device() == dev && t->is_contiguous();
    if (!ok) return nullptr;
    bytes = t->nbytes();
    return t->data_ptr();
  }
  rnn_wtype_t wtype() const { return type == at::kBFloat16 ? RNN_W_BF16 : RNN_W_F32; }
  void* stream() {
    if (ok && dev != c10::hip::current_device()) ok = false;
    return ok ? c10::hip::getCurrentHIPStream(dev).stream() : nullptr;
  }
};

// None: a check failed
PyObject* result(const Call& c, rnn_status_t s) {
  if (!c.ok) Py_RETURN_NONE;
  return PyLong_FromLong(s);
}
#define GUARD(n, ...)             \
  if (nargs != n) Py_RETURN_NONE; \
  try {                           \
    __VA_ARGS__                   \
  } catch (...) {                 \
    Py_RETURN_NONE;               \
  }

PyObject* scan_step(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(5, {
    const int mode = scan_mode(a[0]);
    Call c;
    c.ok = mode >= 0;
    const at::Tensor* g = c.ok ? c.first(a[1], 2) : nullptr;
    if (!g || g->size(1) % 2) Py_RETURN_NONE;
    const int64_t B = g->size(0), H = g->size(1) / 2;
    void* gp = c.data(a[1], c.type, {B, 2 * H});
    void* h = c.data(a[2], at::kFloat, {B, H}, true);
    void* y = c.data(a[3], c.type, {B, H}, true);
    void* hy = c.data(a[4], at::kFloat, {B, H});
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_scan_step)>(STEP)(s, (rnn_scan_mode_t)mode, c.wtype(), (int)B, (int)H, gp,
                                                       (const float*)h, y, (float*)hy));
  })
}

// dirs, B, H from a state tensor
bool state_sizes(Call& c, PyObject* o, int64_t& D, int64_t& H) {
  const at::Tensor* t = c.ok ? c.tensor(o) : nullptr;
  if (!t || t->dim() != 3 || t->size(0) > 2) return c.ok = false;
  D = t->size(0);
  H = t->size(2);
  return c.ok = H <= 0x7fffffff;
}

PyObject* scan_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(7, {   // mode, g, h0, lengths, y, hy, ws
    const int mode = scan_mode(a[0]);
    Call c;
    c.ok = mode >= 0;
    const at::Tensor* g = c.ok ? c.first(a[1], 3) : nullptr;
    int64_t D = 0, H = 0;
    if (!g || !state_sizes(c, a[5], D, H)) Py_RETURN_NONE;
    const int64_t T = g->size(0), B = g->size(1);
    size_t room = 0;
    void* gp = c.data(a[1], c.type, {T, B, D * 2 * H});
    void* h0 = c.data(a[2], at::kFloat, {D, B, H}, true);
    void* n = c.data(a[3], at::kInt, {B}, true);
    void* y = c.data(a[4], c.type, {T, B, D * H});
    void* hy = c.data(a[5], at::kFloat, {D, B, H});
    void* ws = c.room(a[6], room);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_scan_forward)>(SCAN_FWD)(s, (rnn_scan_mode_t)mode, c.wtype(), (int)T, (int)B, (int)H,
                                                              (int)D, gp, (const float*)h0, (const int*)n, y, (float*)hy,
                                                              ws, room));
  })
}

PyObject* scan_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(9, {   // mode, g, h0, lengths, dy, dhy, dg, dh0, ws
    const int mode = scan_mode(a[0]);
    Call c;
    c.ok = mode >= 0;
    const at::Tensor* g = c.ok ? c.first(a[1], 3) : nullptr;
    int64_t D = 0, H = 0;
    if (!g || !state_sizes(c, a[7], D, H)) Py_RETURN_NONE;
    const int64_t T = g->size(0), B = g->size(1);
    size_t room = 0;
    void* gp = c.data(a[1], c.type, {T, B, D * 2 * H});
    void* h0 = c.data(a[2], at::kFloat, {D, B, H}, true);
    void* n = c.data(a[3], at::kInt, {B}, true);
    void* dy = c.data(a[4], c.type, {T, B, D * H});
    void* dhy = c.data(a[5], at::kFloat, {D, B, H}, true);
    void* dg = c.data(a[6], c.type, {T, B, D * 2 * H});
    void* dh0 = c.data(a[7], at::kFloat, {D, B, H});
    void* ws = c.room(a[8], room);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_scan_backward)>(SCAN_BWD)(s, (rnn_scan_mode_t)mode, c.wtype(), (int)T, (int)B, (int)H,
                                                               (int)D, gp, (const float*)h0, (const int*)n, dy,
                                                               (const float*)dhy, dg, (float*)dh0, ws, room));
  })
}

PyObject* ffn_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(8, {   // act, x, w_in, w_out, y, ws, save, reserve
    const int f = act(a[0]), sv = save(a[6]);
    Call c;
    c.ok = f >= 0 && sv >= 0;
    const at::Tensor* x = c.ok ? c.first(a[1], 2) : nullptr;
    const at::Tensor* wo = x ? c.tensor(a[3]) : nullptr;
    if (!wo || wo->dim() != 2 || wo->size(1) > 0x7fffffff) Py_RETURN_NONE;
    const int64_t M = x->size(0), D = x->size(1), F = wo->size(1);
    size_t room = 0, kept = 0;
    void* xp = c.data(a[1], c.type, {M, D});
    void* wi = c.data(a[2], c.type, {2 * F, D});
    void* wp = c.data(a[3], c.type, {D, F});
    void* y = c.data(a[4], c.type, {M, D});
    void* ws = c.room(a[5], room);
    void* rs = c.room(a[7], kept, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_ffn_forward)>(FFN_FWD)(s, (rnn_act_t)f, c.wtype(), (rnn_save_t)sv, (int)M, (int)D,
                                                            (int)F, xp, wi, wp, y, ws, room, rs, kept));
  })
}

PyObject* ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(11, {   // act, x, w_in, w_out, dy, dx, dw_in, dw_out, ws, save, reserve
    const int f = act(a[0]), sv = save(a[9]);
    Call c;
    c.ok = f >= 0 && sv >= 0;
    const at::Tensor* dy = c.ok ? c.first(a[4], 2) : nullptr;
    const at::Tensor* wo = dy ? c.tensor(a[3]) : nullptr;
    if (!wo || wo->dim() != 2 || wo->size(1) > 0x7fffffff) Py_RETURN_NONE;
    const int64_t M = dy->size(0), D = dy->size(1), F = wo->size(1);
    size_t room = 0, kept = 0;
    void* xp = c.data(a[1], c.type, {M, D}, true);
    void* wi = c.data(a[2], c.type, {2 * F, D});
    void* wp = c.data(a[3], c.type, {D, F});
    void* dyp = c.data(a[4], c.type, {M, D});
    void* dx = c.data(a[5], c.type, {M, D}, true);
    void* dwi = c.data(a[6], c.type, {2 * F, D}, true);
    void* dwo = c.data(a[7], c.type, {D, F}, true);
    void* ws = c.room(a[8], room);
    void* rs = c.room(a[10], kept);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_ffn_backward)>(FFN_BWD)(s, (rnn_act_t)f, c.wtype(), (rnn_save_t)sv, (int)M, (int)D,
                                                             (int)F, xp, wi, wp, dyp, dx, dwi, dwo, ws, room, rs, kept));
  })
}

PyObject* checkpoint_size(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(2, {
    if (!PyLong_Check(a[0]) || !PyLong_Check(a[1])) Py_RETURN_NONE;
    int over = 0, over2 = 0;
    const long r = PyLong_AsLongAndOverflow(a[0], &over), n = PyLong_AsLongAndOverflow(a[1], &over2);
    if (over || over2 || r < 0 || n < 0 || r > 0x7fffffff || n > 0x7fffffff) Py_RETURN_NONE;
    size_t bytes = 0;
    if (as<decltype(rnn_checkpoint_size)>(CKPT_SIZE)((int)r, (int)n, &bytes) != RNN_STATUS_SUCCESS) Py_RETURN_NONE;
    return PyLong_FromSize_t(bytes);
  })
}

PyObject* checkpoint_store(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(2, {   // x, kept
    Call c;
    const at::Tensor* x = c.first(a[0], 2);
    if (!x) Py_RETURN_NONE;
    size_t room = 0;
    void* xp = c.data(a[0], c.type, {x->size(0), x->size(1)});
    void* k = c.room(a[1], room);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_checkpoint_store)>(CKPT_STORE)(s, c.wtype(), (int)x->size(0), (int)x->size(1), xp, k, room));
  })
}

PyObject* checkpoint_load(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(2, {   // kept, x
    Call c;
    const at::Tensor* x = c.first(a[1], 2);
    if (!x) Py_RETURN_NONE;
    size_t room = 0;
    void* xp = c.data(a[1], c.type, {x->size(0), x->size(1)});
    void* k = c.room(a[0], room);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_checkpoint_load)>(CKPT_LOAD)(s, c.wtype(), (int)x->size(0), (int)x->size(1), k, room, xp));
  })
}

// bind(addresses of the entries, in the order of Entry)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != ENTRIES) {
    PyErr_SetString(PyExc_TypeError, "bind takes the address of every entry");
    return nullptr;
  }
  for (int i = 0; i < ENTRIES; ++i) {
    entry[i] = PyLong_AsVoidPtr(a[i]);
    if (!entry[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry is missing");
      return nullptr;
    }
  }
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),         METHOD(scan_step),       METHOD(scan_forward),     METHOD(scan_backward),
                         METHOD(ffn_forward),  METHOD(ffn_backward),    METHOD(checkpoint_size),  METHOD(checkpoint_store),
                         METHOD(checkpoint_load), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&module); }
