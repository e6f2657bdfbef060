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
enum Entry { STEP, SCAN_FWD, SCAN_BWD, FFN_FWD, FFN_BWD, CKPT_SIZE, CKPT_STORE, CKPT_LOAD, NORM_FWD, NORM_BWD, CONV_FWD, CONV_STEP,
             CONV_BWD, SSM_FWD, SSM_STEP, SSM_BWD, ENTRIES };
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

int norm_kind(PyObject* o) { return choice(o, {"layer", "rms"}); }
int conv_act(PyObject* o) {
  const int i = choice(o, {"none", "silu"});
  return i < 0 ? i : i ? RNN_ACT_SILU : RNN_ACT_NONE;
}
int delta_mode(PyObject* o) { return choice(o, {"softplus", "linear"}); }

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
  // a tensor [.., B, width] whose rows may lie apart: `ld` elements
  void* rows(PyObject* o, Sizes shape, long long& ld, bool optional = false) {
    const int64_t width = shape.end()[-1];
    ld = width;
    if (!ok || (optional && o == Py_None)) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!ok) return nullptr;
    ok = t->is_cuda() && t->layout() == at::kStrided && t->get_device() == dev && t->scalar_type() == type &&
         t->sizes() == at::IntArrayRef(shape);
    if (!ok) return nullptr;
    if (t->numel() == 0) return t->data_ptr();
    const int64_t n = t->dim();
    int64_t inner = 0;   // rows of the steps seen so far, 0: none
    for (int64_t i = n - 2; i >= 0 && ok; --i) {
      if (t->size(i) == 1) continue;
      if (!inner) ld = t->stride(i);
      else ok = t->stride(i) == inner * ld;
      inner = t->size(i);
    }
    ok = ok && (width == 1 || t->stride(n - 1) == 1) && ld >= width;
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

PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(9, {   // kind, x, residual, weight, bias, y, total, stats, eps
    const int kind = norm_kind(a[0]);
    Call c;
    c.ok = kind >= 0 && PyFloat_Check(a[8]);
    const at::Tensor* x = c.ok ? c.first(a[1], 2) : nullptr;
    if (!x) Py_RETURN_NONE;
    const int64_t M = x->size(0), D = x->size(1);
    void* xp = c.data(a[1], c.type, {M, D});
    void* r = c.data(a[2], c.type, {M, D}, true);
    void* w = c.data(a[3], at::kFloat, {D}, true);
    void* b = c.data(a[4], at::kFloat, {D}, true);
    void* y = c.data(a[5], c.type, {M, D});
    void* total = c.data(a[6], c.type, {M, D}, true);
    void* st = c.data(a[7], at::kFloat, {M, 2}, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_norm_forward)>(NORM_FWD)(s, (rnn_norm_t)kind, c.wtype(), (int)M, (int)D, xp, r, (const float*)w,
                                                              (const float*)b, (float)PyFloat_AS_DOUBLE(a[8]), y, total, (float*)st));
  })
}

PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(10, {   // kind, s, weight, stats, dy, dtotal, dx, dweight, dbias, ws
    const int kind = norm_kind(a[0]);
    Call c;
    c.ok = kind >= 0;
    const at::Tensor* x = c.ok ? c.first(a[1], 2) : nullptr;
    if (!x) Py_RETURN_NONE;
    const int64_t M = x->size(0), D = x->size(1);
    size_t room = 0;
    void* xp = c.data(a[1], c.type, {M, D});
    void* w = c.data(a[2], at::kFloat, {D}, true);
    void* st = c.data(a[3], at::kFloat, {M, 2});
    void* dy = c.data(a[4], c.type, {M, D});
    void* dt = c.data(a[5], c.type, {M, D}, true);
    void* dx = c.data(a[6], c.type, {M, D}, true);
    void* dw = c.data(a[7], at::kFloat, {D}, true);
    void* db = c.data(a[8], at::kFloat, {D}, true);
    void* ws = c.room(a[9], room, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_norm_backward)>(NORM_BWD)(s, (rnn_norm_t)kind, c.wtype(), (int)M, (int)D, xp, (const float*)w,
                                                               (const float*)st, dy, dt, dx, (float*)dw, (float*)db, ws, room));
  })
}

// C and K of the convolution's weights
bool conv_sizes(Call& c, const at::Tensor* x, PyObject* w, int64_t& C, int64_t& K) {
  const at::Tensor* t = c.ok ? c.tensor(w) : nullptr;
  if (!t || t->dim() != 2 || t->size(1) > 0x7fffffff || t->size(1) < 1) return c.ok = false;
  C = x->size(x->dim() - 1);
  K = t->size(1);
  return true;
}

PyObject* conv_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(8, {   // act, x, w, bias, s0, lengths, y, sy
    const int f = conv_act(a[0]);
    Call c;
    c.ok = f >= 0;
    const at::Tensor* x = c.ok ? c.first(a[1], 3) : nullptr;
    int64_t C = 0, K = 0;
    if (!x || !conv_sizes(c, x, a[2], C, K)) Py_RETURN_NONE;
    const int64_t T = x->size(0), B = x->size(1);
    long long ldx = 0, ldy = 0;
    void* xp = c.rows(a[1], {T, B, C}, ldx);
    void* w = c.data(a[2], at::kFloat, {C, K});
    void* b = c.data(a[3], at::kFloat, {C}, true);
    void* s0 = c.data(a[4], c.type, {K - 1, B, C}, true);
    void* n = c.data(a[5], at::kInt, {B}, true);
    void* y = c.rows(a[6], {T, B, C}, ldy);
    void* sy = c.data(a[7], c.type, {K - 1, B, C}, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_conv_forward)>(CONV_FWD)(s, (rnn_act_t)f, c.wtype(), (int)T, (int)B, (int)C, (int)K, xp, ldx,
                                                              (const float*)w, (const float*)b, s0, (const int*)n, y, ldy, sy));
  })
}

PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(7, {   // act, x, w, bias, s, y, sy
    const int f = conv_act(a[0]);
    Call c;
    c.ok = f >= 0;
    const at::Tensor* x = c.ok ? c.first(a[1], 2) : nullptr;
    int64_t C = 0, K = 0;
    if (!x || !conv_sizes(c, x, a[2], C, K)) Py_RETURN_NONE;
    const int64_t B = x->size(0);
    long long ldx = 0, ldy = 0;
    void* xp = c.rows(a[1], {B, C}, ldx);
    void* w = c.data(a[2], at::kFloat, {C, K});
    void* b = c.data(a[3], at::kFloat, {C}, true);
    void* s0 = c.data(a[4], c.type, {K - 1, B, C}, true);
    void* y = c.rows(a[5], {B, C}, ldy);
    void* sy = c.data(a[6], c.type, {K - 1, B, C}, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_conv_step)>(CONV_STEP)(s, (rnn_act_t)f, c.wtype(), (int)B, (int)C, (int)K, xp, ldx,
                                                            (const float*)w, (const float*)b, s0, y, ldy, sy));
  })
}

PyObject* conv_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(13, {   // act, x, w, bias, s0, lengths, dy, dsy, dx, dw, dbias, ds0, ws
    const int f = conv_act(a[0]);
    Call c;
    c.ok = f >= 0;
    const at::Tensor* x = c.ok ? c.first(a[1], 3) : nullptr;
    int64_t C = 0, K = 0;
    if (!x || !conv_sizes(c, x, a[2], C, K)) Py_RETURN_NONE;
    const int64_t T = x->size(0), B = x->size(1);
    long long ldx = 0, lddy = 0, lddx = 0;
    size_t room = 0;
    void* xp = c.rows(a[1], {T, B, C}, ldx);
    void* w = c.data(a[2], at::kFloat, {C, K});
    void* b = c.data(a[3], at::kFloat, {C}, true);
    void* s0 = c.data(a[4], c.type, {K - 1, B, C}, true);
    void* n = c.data(a[5], at::kInt, {B}, true);
    void* dy = c.rows(a[6], {T, B, C}, lddy);
    void* dsy = c.data(a[7], c.type, {K - 1, B, C}, true);
    void* dx = c.rows(a[8], {T, B, C}, lddx, true);
    void* dw = c.data(a[9], at::kFloat, {C, K}, true);
    void* db = c.data(a[10], at::kFloat, {C}, true);
    void* ds0 = c.data(a[11], c.type, {K - 1, B, C}, true);
    void* ws = c.room(a[12], room, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_conv_backward)>(CONV_BWD)(s, (rnn_act_t)f, c.wtype(), (int)T, (int)B, (int)C, (int)K, xp, ldx,
                                                               (const float*)w, (const float*)b, s0, (const int*)n, dy, lddy, dsy, dx,
                                                               lddx, (float*)dw, (float*)db, ds0, ws, room));
  })
}

// The inputs of the state-space calls: a[0] mode, u, delta, A, Bm, Cm, D, z, delta_bias.
struct Ssm {
  int mode = -1;
  int64_t T = 1, B = 0, E = 0, N = 0, G = 0;
  rnn_ssm_inputs_t in{};
};
bool ssm_inputs(Call& c, PyObject* const* a, int dims, Ssm& q) {
  q.mode = delta_mode(a[0]);
  c.ok = q.mode >= 0;
  const at::Tensor* u = c.ok ? c.first(a[1], dims) : nullptr;
  const at::Tensor* A = u ? c.tensor(a[3]) : nullptr;
  const at::Tensor* Bm = A ? c.tensor(a[4]) : nullptr;
  if (!Bm || A->dim() != 2 || Bm->dim() != dims) return c.ok = false;
  if (dims == 3) q.T = u->size(0);
  q.B = u->size(dims - 2);
  q.E = u->size(dims - 1);
  q.N = A->size(1);
  const int64_t GN = Bm->size(dims - 1);
  if (q.N < 1 || GN < 1 || GN > 0x7fffffff || GN % q.N) return c.ok = false;
  q.G = GN / q.N;
  auto rows = [&](PyObject* o, int64_t width, long long& ld, bool optional = false) {
    return dims == 3 ? c.rows(o, {q.T, q.B, width}, ld, optional) : c.rows(o, {q.B, width}, ld, optional);
  };
  q.in.u = rows(a[1], q.E, q.in.ldu);
  q.in.delta = rows(a[2], q.E, q.in.lddelta);
  q.in.A = (const float*)c.data(a[3], at::kFloat, {q.E, q.N});
  q.in.Bm = rows(a[4], GN, q.in.ldB);
  q.in.Cm = rows(a[5], GN, q.in.ldC);
  q.in.D = (const float*)c.data(a[6], at::kFloat, {q.E}, true);
  q.in.z = rows(a[7], q.E, q.in.ldz, true);
  q.in.delta_bias = (const float*)c.data(a[8], at::kFloat, {q.E}, true);
  return c.ok;
}

PyObject* ssm_forward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(15, {   // ..., h0, lengths, y, hy, ws, save
    const int sv = choice(a[14], {"none", "full"});
    Call c;
    Ssm q;
    if (sv < 0 || !ssm_inputs(c, a, 3, q)) Py_RETURN_NONE;
    long long ldy = 0;
    size_t room = 0;
    void* h0 = c.data(a[9], at::kFloat, {q.B, q.E, q.N}, true);
    void* n = c.data(a[10], at::kInt, {q.B}, true);
    void* y = c.rows(a[11], {q.T, q.B, q.E}, ldy);
    void* hy = c.data(a[12], at::kFloat, {q.B, q.E, q.N}, true);
    void* ws = c.room(a[13], room);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_ssm_forward)>(SSM_FWD)(s, (rnn_delta_t)q.mode, c.wtype(), (rnn_save_t)sv, (int)q.T, (int)q.B,
                                                            (int)q.E, (int)q.N, (int)q.G, &q.in, (const float*)h0, (const int*)n, y,
                                                            ldy, (float*)hy, ws, room));
  })
}

PyObject* ssm_step(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(12, {   // ..., h, y, hy
    Call c;
    Ssm q;
    if (!ssm_inputs(c, a, 2, q)) Py_RETURN_NONE;
    long long ldy = 0;
    void* h = c.data(a[9], at::kFloat, {q.B, q.E, q.N}, true);
    void* y = c.rows(a[10], {q.B, q.E}, ldy);
    void* hy = c.data(a[11], at::kFloat, {q.B, q.E, q.N}, true);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_ssm_step)>(SSM_STEP)(s, (rnn_delta_t)q.mode, c.wtype(), (int)q.B, (int)q.E, (int)q.N, (int)q.G,
                                                          &q.in, (const float*)h, y, ldy, (float*)hy));
  })
}

PyObject* ssm_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  GUARD(23, {   // ..., h0, lengths, dy, dhy, du, ddelta, dA, dBm, dCm, dD, dz, ddelta_bias, dh0, ws
    Call c;
    Ssm q;
    if (!ssm_inputs(c, a, 3, q) || (a[19] != Py_None && a[7] == Py_None)) Py_RETURN_NONE;
    const int64_t T = q.T, B = q.B, E = q.E, GN = q.G * q.N;
    long long lddy = 0;
    size_t room = 0;
    rnn_ssm_grads_t g{};
    c.data(a[9], at::kFloat, {B, E, q.N}, true);
    void* n = c.data(a[10], at::kInt, {B}, true);
    void* dy = c.rows(a[11], {T, B, E}, lddy);
    void* dhy = c.data(a[12], at::kFloat, {B, E, q.N}, true);
    g.du = c.rows(a[13], {T, B, E}, g.lddu, true);
    g.ddelta = c.rows(a[14], {T, B, E}, g.ldddelta, true);
    g.dA = (float*)c.data(a[15], at::kFloat, {E, q.N}, true);
    g.dBm = c.rows(a[16], {T, B, GN}, g.lddB, true);
    g.dCm = c.rows(a[17], {T, B, GN}, g.lddC, true);
    g.dD = (float*)c.data(a[18], at::kFloat, {E}, true);
    g.dz = c.rows(a[19], {T, B, E}, g.lddz, true);
    g.ddelta_bias = (float*)c.data(a[20], at::kFloat, {E}, true);
    g.dh0 = (float*)c.data(a[21], at::kFloat, {B, E, q.N}, true);
    void* ws = c.room(a[22], room);
    void* s = c.stream();
    if (!c.ok) Py_RETURN_NONE;
    return result(c, as<decltype(rnn_ssm_backward)>(SSM_BWD)(s, (rnn_delta_t)q.mode, c.wtype(), (int)T, (int)B, (int)E, (int)q.N,
                                                             (int)q.G, &q.in, (const int*)n, dy, lddy, (const float*)dhy, &g, ws, room));
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
                         METHOD(checkpoint_load), METHOD(norm_forward),   METHOD(norm_backward),    METHOD(conv_forward),
                         METHOD(conv_step),    METHOD(conv_backward),  METHOD(ssm_forward),      METHOD(ssm_step),
                         METHOD(ssm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&module); }
