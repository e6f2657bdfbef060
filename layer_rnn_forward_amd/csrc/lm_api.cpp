// C ABI of the language-model operators: argument checks, workspace and
// reserve layouts, launch sequences.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_common.h"
#include "rnn.h"

using namespace rnnk;

namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned(const void* p) { return ((uintptr_t)p & (kAlign - 1)) == 0; }

template <class T>
T* at(void* base, size_t off) { return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + off); }
template <class T>
const T* at(const void* base, size_t off) { return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + off); }

rnn_status_t dev(hipError_t e) { return e == hipSuccess ? RNN_STATUS_SUCCESS : RNN_STATUS_DEVICE; }
inline hipStream_t hs(void* s) { return reinterpret_cast<hipStream_t>(s); }

#define LM_TRY(expr)                                 \
  do {                                               \
    const rnn_status_t st_ = (expr);                 \
    if (st_ != RNN_STATUS_SUCCESS) return st_;       \
  } while (0)

bool wtype_ok(int w) { return w == RNN_W_F32 || w == RNN_W_BF16; }
bool scan_mode_ok(int m) { return m == RNN_SCAN_GATED || m == RNN_SCAN_LINEAR; }

// ------------------------------------------------------------------- scan
rnn_status_t scan_sizes(int T, int B, int H, int dirs) {
  if (T < 0 || B < 0 || H < 0 || (dirs != 1 && dirs != 2)) return RNN_STATUS_INVALID_ARG;
  // B * H first: it fits 64 bits, times dirs as well
  if ((long long)B * H * dirs >= (1LL << 30)) return RNN_STATUS_UNSUPPORTED;
  return RNN_STATUS_SUCCESS;
}

size_t scan_bytes(int T, int B, int H, int dirs) {
  return kAlign + align_up((size_t)T * B * H * dirs * 4);
}

// -------------------------------------------------------------------- ffn
rnn_status_t ffn_sizes(int M, int D, int F, int wtype, int save) {
  if (M < 0 || D < 0 || F < 0 || !wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  if (save != RNN_SAVE_NONE && save != RNN_SAVE_FULL && save != RNN_SAVE_INT8) return RNN_STATUS_INVALID_ARG;
  if (D >= (1 << 24) || F >= (1 << 24) || M >= (1 << 30)) return RNN_STATUS_UNSUPPORTED;
  return RNN_STATUS_SUCCESS;
}

size_t ckpt_bytes(size_t rows, size_t cols) { return rows * cols + rows * ((cols + kGroup - 1) / kGroup); }

struct FfnPlan {
  // workspace
  size_t gu = 0, h = 0, x = 0, dh = 0, dgu = 0, ws = 0;
  // reserve
  size_t rgu = 0, rh = 0, rx = 0, reserve = 0;
};

FfnPlan ffn_plan(int M, int D, int F, int wtype, int save) {
  const size_t es = wtype == RNN_W_BF16 ? 2 : 4, m = M, d = D, f = F;
  FfnPlan p;
  size_t o = 0;
  auto take = [](size_t& top, size_t bytes) {
    const size_t at = top;
    top += align_up(bytes);
    return at;
  };
  p.gu = take(o, m * 2 * f * 4);
  p.h = take(o, m * f * es);
  if (save != RNN_SAVE_NONE) {
    p.x = take(o, m * d * es);
    p.dh = take(o, m * f * 4);
    p.dgu = take(o, m * 2 * f * es);
  }
  p.ws = std::max(o, kAlign);
  o = 0;
  if (save == RNN_SAVE_FULL) {
    p.rgu = take(o, m * 2 * f * 4);
    p.rh = take(o, m * f * es);
  } else if (save == RNN_SAVE_INT8) {
    p.rgu = take(o, ckpt_bytes(2 * m, f));
    p.rx = take(o, ckpt_bytes(m, d));
  }
  p.reserve = o;
  return p;
}

}  // namespace

extern "C" {

rnn_status_t rnn_scan_workspace_size(int T, int B, int H, int dirs, size_t* bytes) {
  if (!bytes) return RNN_STATUS_INVALID_ARG;
  LM_TRY(scan_sizes(T, B, H, dirs));
  *bytes = scan_bytes(T, B, H, dirs);
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_scan_step(void* stream, rnn_scan_mode_t mode, rnn_wtype_t wtype, int B, int H, const void* g,
                           const float* h, void* y, float* hy) {
  if (!scan_mode_ok(mode) || !wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(scan_sizes(1, B, H, 1));
  if (B == 0 || H == 0) return RNN_STATUS_SUCCESS;
  if (!g || !hy) return RNN_STATUS_INVALID_ARG;
  return dev(rnn_launch_scan_step(mode, wtype == RNN_W_BF16, B, H, g, h, y, hy, hs(stream)));
}

rnn_status_t rnn_scan_forward(void* stream, rnn_scan_mode_t mode, rnn_wtype_t wtype, int T, int B, int H, int dirs,
                              const void* g, const float* h0, const int* lengths, void* y, float* hy, void* ws,
                              size_t ws_bytes) {
  if (!scan_mode_ok(mode) || !wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(scan_sizes(T, B, H, dirs));
  if (!ws || !aligned(ws)) return RNN_STATUS_INVALID_ARG;
  if (ws_bytes < scan_bytes(T, B, H, dirs)) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (B == 0 || H == 0) return RNN_STATUS_SUCCESS;
  if (T > 0 && (!g || !y)) return RNN_STATUS_INVALID_ARG;
  ScanParams p{};
  p.T = T; p.B = B; p.H = H; p.D = dirs;
  p.g = g; p.h0 = h0; p.lengths = lengths; p.y = y; p.hy = hy;
  p.states = at<float>(ws, kAlign);
  return dev(rnn_launch_scan_fwd(p, mode, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_scan_backward(void* stream, rnn_scan_mode_t mode, rnn_wtype_t wtype, int T, int B, int H, int dirs,
                               const void* g, const float* h0, const int* lengths, const void* dy, const float* dhy,
                               void* dg, float* dh0, void* ws, size_t ws_bytes) {
  if (!scan_mode_ok(mode) || !wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(scan_sizes(T, B, H, dirs));
  if (!ws || !aligned(ws)) return RNN_STATUS_INVALID_ARG;
  if (ws_bytes < scan_bytes(T, B, H, dirs)) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (B == 0 || H == 0) return RNN_STATUS_SUCCESS;
  if (T > 0 && (!g || !dy || !dg)) return RNN_STATUS_INVALID_ARG;
  ScanParams p{};
  p.T = T; p.B = B; p.H = H; p.D = dirs;
  p.g = g; p.h0 = h0; p.lengths = lengths; p.dy = dy; p.dhy = dhy; p.dg = dg; p.dh0 = dh0;
  p.states = at<float>(ws, kAlign);
  return dev(rnn_launch_scan_bwd(p, mode, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_ffn_workspace_size(int M, int D, int F, rnn_wtype_t wtype, rnn_save_t save, size_t* bytes) {
  if (!bytes) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ffn_sizes(M, D, F, wtype, save));
  *bytes = ffn_plan(M, D, F, wtype, save).ws;
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_ffn_reserve_size(int M, int D, int F, rnn_wtype_t wtype, rnn_save_t save, size_t* bytes) {
  if (!bytes) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ffn_sizes(M, D, F, wtype, save));
  *bytes = ffn_plan(M, D, F, wtype, save).reserve;
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_ffn_forward(void* stream, rnn_act_t act, rnn_wtype_t wtype, rnn_save_t save, int M, int D, int F,
                             const void* x, const void* w_in, const void* w_out, void* y, void* ws, size_t ws_bytes,
                             void* reserve, size_t reserve_bytes) {
  if (act < RNN_ACT_SIGMOID || act > RNN_ACT_GELU) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ffn_sizes(M, D, F, wtype, save));
  const FfnPlan p = ffn_plan(M, D, F, wtype, save);
  if (!ws || !aligned(ws) || (p.reserve && (!reserve || !aligned(reserve)))) return RNN_STATUS_INVALID_ARG;
  if (ws_bytes < p.ws || reserve_bytes < p.reserve) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (M == 0 || D == 0) return RNN_STATUS_SUCCESS;
  if (!x || !y || (F > 0 && (!w_in || !w_out))) return RNN_STATUS_INVALID_ARG;
  const int bf = wtype == RNN_W_BF16;
  const hipStream_t s = hs(stream);
  float* gu = save == RNN_SAVE_FULL ? at<float>(reserve, p.rgu) : at<float>(ws, p.gu);
  void* h = save == RNN_SAVE_FULL ? at<void>(reserve, p.rh) : at<void>(ws, p.h);
  LM_TRY(dev(rnn_launch_mat({M, 2 * F, D, x, D, 1, w_in, D, 1, gu, 2LL * F}, bf, bf, 0, s)));
  if (save == RNN_SAVE_INT8) {
    LM_TRY(dev(rnn_launch_ckpt_store(bf, M, D, x, at<void>(reserve, p.rx), s)));
    LM_TRY(dev(rnn_launch_ckpt_store(0, 2 * M, F, gu, at<void>(reserve, p.rgu), s)));
  }
  LM_TRY(dev(rnn_launch_act(act, bf, M, F, gu, h, s)));
  return dev(rnn_launch_mat({M, D, F, h, F, 1, w_out, F, 1, y, D}, bf, bf, bf, s));
}

rnn_status_t rnn_ffn_backward(void* stream, rnn_act_t act, rnn_wtype_t wtype, rnn_save_t save, int M, int D, int F,
                              const void* x, const void* w_in, const void* w_out, const void* dy, void* dx,
                              void* dw_in, void* dw_out, void* ws, size_t ws_bytes, const void* reserve,
                              size_t reserve_bytes) {
  if (act < RNN_ACT_SIGMOID || act > RNN_ACT_GELU || save == RNN_SAVE_NONE) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ffn_sizes(M, D, F, wtype, save));
  const FfnPlan p = ffn_plan(M, D, F, wtype, save);
  if (!ws || !aligned(ws) || (p.reserve && (!reserve || !aligned(reserve)))) return RNN_STATUS_INVALID_ARG;
  if (ws_bytes < p.ws || reserve_bytes < p.reserve) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (D == 0) return RNN_STATUS_SUCCESS;
  const bool rows = M > 0;
  if (rows && (!dy || (F > 0 && (!w_in || !w_out)) || (save != RNN_SAVE_INT8 && dw_in && !x)))
    return RNN_STATUS_INVALID_ARG;
  const int bf = wtype == RNN_W_BF16;
  const hipStream_t s = hs(stream);
  const float* gu = save == RNN_SAVE_FULL ? at<const float>(reserve, p.rgu) : at<float>(ws, p.gu);
  const void* h = save == RNN_SAVE_FULL ? at<const void>(reserve, p.rh) : at<void>(ws, p.h);
  float* dh = at<float>(ws, p.dh);
  void* dgu = at<void>(ws, p.dgu);
  if (save == RNN_SAVE_INT8) {
    LM_TRY(dev(rnn_launch_ckpt_load(0, 2 * M, F, at<const void>(reserve, p.rgu), at<float>(ws, p.gu), s)));
    LM_TRY(dev(rnn_launch_ckpt_load(bf, M, D, at<const void>(reserve, p.rx), at<void>(ws, p.x), s)));
    LM_TRY(dev(rnn_launch_act(act, bf, M, F, gu, at<void>(ws, p.h), s)));
    x = at<void>(ws, p.x);
  }
  LM_TRY(dev(rnn_launch_mat({M, F, D, dy, D, 1, w_out, 1, F, dh, F}, bf, bf, 0, s)));
  LM_TRY(dev(rnn_launch_act_bwd(act, bf, M, F, gu, dh, dgu, s)));
  if (dx) LM_TRY(dev(rnn_launch_mat({M, D, 2 * F, dgu, 2LL * F, 1, w_in, 1, D, dx, D}, bf, bf, bf, s)));
  if (dw_in) LM_TRY(dev(rnn_launch_mat({2 * F, D, M, dgu, 1, 2LL * F, x, 1, D, dw_in, D}, bf, bf, bf, s)));
  if (dw_out) LM_TRY(dev(rnn_launch_mat({D, F, M, dy, 1, D, h, 1, F, dw_out, F}, bf, bf, bf, s)));
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_checkpoint_size(int rows, int cols, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 0) return RNN_STATUS_INVALID_ARG;
  if (cols >= (1 << 30)) return RNN_STATUS_UNSUPPORTED;
  *bytes = ckpt_bytes(rows, cols);
  return RNN_STATUS_SUCCESS;
}

static rnn_status_t ckpt_check(int wtype, int rows, int cols, const void* x, const void* kept, size_t kept_bytes) {
  size_t need = 0;
  if (!wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(rnn_checkpoint_size(rows, cols, &need));
  if (kept_bytes < need) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (need && (!x || !kept || !aligned(kept))) return RNN_STATUS_INVALID_ARG;
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_checkpoint_store(void* stream, rnn_wtype_t wtype, int rows, int cols, const void* x, void* kept,
                                  size_t kept_bytes) {
  LM_TRY(ckpt_check(wtype, rows, cols, x, kept, kept_bytes));
  return dev(rnn_launch_ckpt_store(wtype == RNN_W_BF16, rows, cols, x, kept, hs(stream)));
}

rnn_status_t rnn_checkpoint_load(void* stream, rnn_wtype_t wtype, int rows, int cols, const void* kept,
                                 size_t kept_bytes, void* x) {
  LM_TRY(ckpt_check(wtype, rows, cols, x, kept, kept_bytes));
  return dev(rnn_launch_ckpt_load(wtype == RNN_W_BF16, rows, cols, kept, x, hs(stream)));
}

}  // extern "C"
