// C ABI of the language-model operators: argument checks, workspace and
// reserve layouts, launch sequences.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdlib>

#include "ffn_plan.h"
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
  if (T > 0x7fffffff - 1024) return RNN_STATUS_UNSUPPORTED;   // the last chunk's steps are counted past T
  return RNN_STATUS_SUCCESS;
}

// Chunks of as many waves as there are pieces, `most` at most.
void scan_split(int T, int steps, int most, int& waves, int& chunks) {
  const int pieces = (int)(((long long)T + steps - 1) / steps);
  waves = std::max(1, std::min(most, pieces));
  chunks = std::max(1, (pieces + waves - 1) / waves);
}

struct ScanPlan {
  int fwaves, fchunks, bwaves, bchunks;
  size_t maps, starts, bytes;
};
ScanPlan scan_plan(int T, int B, int H, int dirs) {
  ScanPlan p;
  scan_split(T, kScanFwdSteps, kScanFwdWaves, p.fwaves, p.fchunks);
  scan_split(T, kScanBwdSteps, kScanBwdWaves, p.bwaves, p.bchunks);
  const size_t C = (size_t)B * H * dirs;
  auto words = [](int chunks, int super) { return chunks > 1 ? 3 * (size_t)chunks + chunks / super + 1 : 0; };
  const size_t most = std::max(words(p.fchunks, kScanFwdSuper), words(p.bchunks, kScanBwdSuper));
  p.maps = kAlign + (most ? align_up(((size_t)B * H + 63) / 64 * dirs * 64) : 0);
  p.starts = p.maps + align_up(most * C * 4);
  p.bytes = p.starts + align_up(((size_t)T + kScanKeep - 1) / kScanKeep * C * 4);
  return p;
}

// Polls of a wait before it expires: some seconds, or RNN_SPIN_LIMIT (as for
// the recurrent kernels; 0 expires every wait whose words are not there).
int scan_spin_limit() {
  const char* v = std::getenv("RNN_SPIN_LIMIT");
  return v && *v ? std::max(0, std::atoi(v)) : 1 << 22;
}

void scan_room(ScanParams& p, bool back, void* ws) {
  p.spin_limit = scan_spin_limit();
  const ScanPlan q = scan_plan(p.T, p.B, p.H, p.D);
  p.waves = back ? q.bwaves : q.fwaves;
  p.chunks = back ? q.bchunks : q.fchunks;
  p.head = at<unsigned>(ws, 0);
  p.counters = at<unsigned>(ws, kAlign);
  p.starts = at<float>(ws, q.starts);
  p.maps = at<unsigned long long>(ws, q.maps);
  const size_t C = (size_t)p.B * p.H * p.D;
  p.state = reinterpret_cast<float*>(p.maps + p.chunks * C);
  p.ends = p.state + (p.chunks / (back ? kScanBwdSuper : kScanFwdSuper) + 1) * C;
}

// -------------------------------------------------------------------- ffn
rnn_status_t ffn_sizes(int M, int D, int F, int wtype, int save) {
  if (M < 0 || D < 0 || F < 0 || !wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  if (save != RNN_SAVE_NONE && save != RNN_SAVE_FULL && save != RNN_SAVE_INT8) return RNN_STATUS_INVALID_ARG;
  if (D >= (1 << 20) || F >= (1 << 20) || M >= (1 << 30)) return RNN_STATUS_UNSUPPORTED;
  return RNN_STATUS_SUCCESS;
}

size_t ckpt_bytes(size_t rows, size_t cols) { return rows * cols + rows * ((cols + kGroup - 1) / kGroup); }

// Widths as the products see them: rows of x, dy and w_in in whole 16-byte
// pieces (Dp), rows of w_out likewise (Fo), rows of the library's own
// [M, F] buffers in whole K steps (Fp).
struct FfnPlan {
  int es = 0, Dp = 0, Fo = 0, Fp = 0;
  // workspace: padded copies (used where rows or addresses are not 16-byte
  // aligned, which the size does not know), the gated product, its gradients
  size_t x = 0, w_in = 0, w_out = 0, dy = 0, h = 0, dgu = 0, ws = 0;
  // and the partial sums of split products; the choices do not depend on which
  // gradients are wanted
  FfnGemm gated{}, out{}, grads[3] = {};
  FfnChoice gated_choice, out_choice, grads_choice;
  int order[3] = {0, 1, 2};
  size_t part = 0, grads_part[3] = {};   // forward's products use theirs one after the other
  // reserve
  size_t s0 = 0, s1 = 0, e0 = 0, e1 = 0, rh = 0, rx = 0, reserve = 0;
};

FfnPlan ffn_plan(int M, int D, int F, int wtype, int save) {
  FfnPlan p;
  p.es = wtype == RNN_W_BF16 ? 2 : 4;
  const int piece = 16 / p.es;
  p.Dp = (D + piece - 1) / piece * piece;
  p.Fo = (F + piece - 1) / piece * piece;
  p.Fp = (F + 63) / 64 * 64;
  const size_t m = M, es = p.es;
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  // the block for few rows needs the gated product and the rests of its rounding, and nothing else
  auto few = [&](size_t rows) { return align_up(2 * rows * p.Fp * es); };
  if (save == RNN_SAVE_NONE && M <= kFfnRows) {
    p.ws = std::max(few(m), kAlign);
    return p;
  }
  // copies, the gated product, its gradients; returns where they end for `rows` rows
  auto layout = [&](size_t rows) {
    o = 0;
    p.x = take(rows * p.Dp * es);
    p.w_in = take(2 * (size_t)F * p.Dp * es);
    p.w_out = take((size_t)D * p.Fo * es);
    if (save != RNN_SAVE_FULL) p.h = take(rows * p.Fp * es);
    if (save != RNN_SAVE_NONE) {
      p.dy = take(rows * p.Dp * es);
      p.dgu = take(rows * 2 * p.Fp * es);
    }
    return o;
  };
  const int bf = wtype == RNN_W_BF16;
  ffn_forward_product(M, D, F, p.out);
  p.out_choice = ffn_choose_forward(p.out, bf, false);
  p.out.splits = p.out_choice.splits[0];
  ffn_gated_product(M, D, F, p.gated);
  p.gated_choice = ffn_choose_forward(p.gated, bf, true);
  p.gated.splits = p.gated_choice.splits[0];
  if (save != RNN_SAVE_NONE) ffn_backward_products(M, D, F, p.Fp, p.grads);
  // room for every smaller M as well
  if (save == RNN_SAVE_NONE) p.ws = few(kFfnRows);
  for (int tile : {TILE_128, TILE_64}) {
    int rows = 0;
    size_t part = ffn_part_bound(p.out, tile, bf, false, rows);
    p.ws = std::max(p.ws, layout(rows) + part);
    part = ffn_part_bound(p.gated, tile, bf, true, rows);
    p.ws = std::max(p.ws, layout(rows) + part);
    if (save != RNN_SAVE_NONE) {
      part = ffn_part_bound(p.grads, tile, bf, rows);
      p.ws = std::max(p.ws, layout(rows) + part);
    }
  }
  const size_t parts = layout(m);   // the passes' partial sums share their place
  p.part = take(std::max(ffn_part(p.out, p.out_choice, 0, false), ffn_part(p.gated, p.gated_choice, 0, true)));
  p.ws = std::max({p.ws, o, kAlign});
  if (save != RNN_SAVE_NONE) {
    o = parts;
    p.grads_choice = ffn_choose_backward(p.grads, bf, p.order);
    for (int i = 0; i < 3; ++i) {
      p.grads[i].splits = p.grads_choice.splits[i];
      p.grads_part[i] = take(ffn_part(p.grads[i], p.grads_choice, i, false));
    }
    p.ws = std::max(p.ws, o);
  }
  o = 0;
  if (save != RNN_SAVE_NONE) {
    const size_t vs = save == RNN_SAVE_INT8 ? 1 : wtype == RNN_W_BF16 ? 2 : 4;
    const size_t tiles = (m + 31) / 32 * (p.Fp / 32);
    p.s0 = take(tiles * 1024 * vs);
    p.s1 = take(tiles * 1024 * vs);
    if (vs < 4) {
      p.e0 = take(tiles * 32);
      p.e1 = take(tiles * 32);
    }
    if (save == RNN_SAVE_FULL) p.rh = take(m * p.Fp * es);
    else p.rx = take(ckpt_bytes(m, D));
  }
  p.reserve = o;
  return p;
}

// The padded copies that one call needs, made in one launch.
struct Pads {
  PadJob j{};
  const void* add(const void* src, long long rows, int cols, int ld, void* dst) {
    if (cols == 0 || (cols == ld && ((uintptr_t)src & 15) == 0)) return src;
    const int i = j.n++;
    j.src[i] = src;
    j.dst[i] = dst;
    j.rows[i] = rows;
    j.cols[i] = cols;
    j.ld[i] = ld;
    return dst;
  }
};

int store16(const void* c, long long ld, int es) { return ((uintptr_t)c & 15) == 0 && ld * es % 16 == 0; }

void ffn_saved(FfnGemm& g, const FfnPlan& p, void* reserve) {
  g.s0 = at<void>(reserve, p.s0);
  g.s1 = at<void>(reserve, p.s1);
  g.e0 = at<int8_t>(reserve, p.e0);
  g.e1 = at<int8_t>(reserve, p.e1);
  g.lds = p.Fp / 32;
}

}  // namespace

extern "C" {

rnn_status_t rnn_scan_workspace_size(int T, int B, int H, int dirs, size_t* bytes) {
  if (!bytes) return RNN_STATUS_INVALID_ARG;
  LM_TRY(scan_sizes(T, B, H, dirs));
  *bytes = scan_plan(T, B, H, dirs).bytes;
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
  if (ws_bytes < scan_plan(T, B, H, dirs).bytes) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (B == 0 || H == 0) return RNN_STATUS_SUCCESS;
  if (T > 0 && (!g || !y)) return RNN_STATUS_INVALID_ARG;
  ScanParams p{};
  p.T = T; p.B = B; p.H = H; p.D = dirs;
  p.g = g; p.h0 = h0; p.lengths = lengths; p.y = y; p.hy = hy;
  scan_room(p, false, ws);
  return dev(rnn_launch_scan_fwd(p, mode, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_scan_backward(void* stream, rnn_scan_mode_t mode, rnn_wtype_t wtype, int T, int B, int H, int dirs,
                               const void* g, const float* h0, const int* lengths, const void* dy, const float* dhy,
                               void* dg, float* dh0, void* ws, size_t ws_bytes) {
  if (!scan_mode_ok(mode) || !wtype_ok(wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(scan_sizes(T, B, H, dirs));
  if (!ws || !aligned(ws)) return RNN_STATUS_INVALID_ARG;
  if (ws_bytes < scan_plan(T, B, H, dirs).bytes) return RNN_STATUS_WORKSPACE_TOO_SMALL;
  if (B == 0 || H == 0) return RNN_STATUS_SUCCESS;
  if (T > 0 && (!g || !dy || !dg)) return RNN_STATUS_INVALID_ARG;
  ScanParams p{};
  p.T = T; p.B = B; p.H = H; p.D = dirs;
  p.g = g; p.h0 = h0; p.lengths = lengths; p.dy = dy; p.dhy = dhy; p.dg = dg; p.dh0 = dh0;
  scan_room(p, true, ws);
  return dev(rnn_launch_scan_bwd(p, mode, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_scan_status(void* stream, const void* ws, size_t ws_bytes) {
  if (!ws || !aligned(ws) || ws_bytes < kAlign) return RNN_STATUS_INVALID_ARG;
  unsigned expired[2] = {};
  if (hipStreamSynchronize(hs(stream)) != hipSuccess ||
      hipMemcpy(expired, ws, sizeof(expired), hipMemcpyDeviceToHost) != hipSuccess)
    return RNN_STATUS_DEVICE;
  return expired[0] || expired[1] ? RNN_STATUS_DEVICE_TIMEOUT : RNN_STATUS_SUCCESS;
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
  if (save == RNN_SAVE_NONE && M <= kFfnRows) {
    FfnRows r{};
    r.M = M; r.R = F; r.K = D;
    r.x = x; r.ldx = D; r.w = w_in;
    r.out = ws; r.ldo = p.Fp;
    r.act = act;
    LM_TRY(dev(rnn_launch_ffn_rows(r, bf, 1, s)));
    r.R = D; r.K = F;
    r.x = r.out; r.ldx = p.Fp; r.w = w_out;
    r.out = y; r.ldo = D;
    return dev(rnn_launch_ffn_rows(r, bf, 0, s));
  }
  Pads pads;
  const void* xp = pads.add(x, M, D, p.Dp, at<void>(ws, p.x));
  const void* wi = pads.add(w_in, 2LL * F, D, p.Dp, at<void>(ws, p.w_in));
  const void* wo = pads.add(w_out, D, F, p.Fo, at<void>(ws, p.w_out));
  LM_TRY(dev(rnn_launch_pad(pads.j, bf, s)));
  if (save == RNN_SAVE_INT8) LM_TRY(dev(rnn_launch_ckpt_store(bf, M, D, x, at<void>(reserve, p.rx), s)));
  void* h = save == RNN_SAVE_FULL ? at<void>(reserve, p.rh) : at<void>(ws, p.h);
  FfnGemm g = p.gated;
  g.A = xp; g.lda = p.Dp;
  g.B = wi; g.ldb = p.Dp;
  g.C = h; g.ldc = p.Fp;
  g.part = at<void>(ws, p.part);
  g.act = act;
  if (save != RNN_SAVE_NONE) ffn_saved(g, p, reserve);
  LM_TRY(dev(rnn_launch_ffn_glu(g, p.gated_choice.tile, bf, save, s)));
  FfnGemm o = p.out;
  o.A = h; o.lda = p.Fp;
  o.B = wo; o.ldb = p.Fo;
  o.C = y; o.ldc = D; o.cvec = store16(y, D, p.es);
  o.part = at<void>(ws, p.part);
  return dev(rnn_launch_ffn_store(o, p.out_choice.tile, bf, s));
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
  Pads pads;
  const void* wi = rows && dx ? pads.add(w_in, 2LL * F, D, p.Dp, at<void>(ws, p.w_in)) : nullptr;
  const void* wo = rows ? pads.add(w_out, D, F, p.Fo, at<void>(ws, p.w_out)) : nullptr;
  const void* dyp = rows ? pads.add(dy, M, D, p.Dp, at<void>(ws, p.dy)) : nullptr;
  const void* xp = nullptr;
  if (rows && dw_in) xp = save == RNN_SAVE_INT8 ? at<const void>(ws, p.x) : pads.add(x, M, D, p.Dp, at<void>(ws, p.x));
  LM_TRY(dev(rnn_launch_pad(pads.j, bf, s)));
  if (rows && dw_in && save == RNN_SAVE_INT8)
    LM_TRY(dev(rnn_launch_ckpt_load(bf, M, D, at<const void>(reserve, p.rx), at<void>(ws, p.x), p.Dp, s)));
  void* dgu = at<void>(ws, p.dgu);
  void* res = const_cast<void*>(reserve);   // read only
  const void* h = save == RNN_SAVE_FULL ? at<void>(res, p.rh) : at<void>(ws, p.h);
  FfnGemm g{};
  g.M = M; g.N = F; g.K = D;
  g.A = dyp; g.lda = p.Dp;
  g.B = wo; g.ldb = p.Fo;
  g.C = dgu; g.ldc = 2LL * p.Fp;
  g.segs = 1;
  g.act = act;
  ffn_saved(g, p, res);
  g.h = at<void>(ws, p.h); g.ldh = p.Fp;
  LM_TRY(dev(rnn_launch_ffn_dglu(g, bf, save, s)));
  FfnGemm q[3] = {p.grads[0], p.grads[1], p.grads[2]};
  for (int i = 0; i < 3; ++i) q[i].part = at<void>(ws, p.grads_part[i]);
  q[0].A = dgu; q[0].lda = 2LL * p.Fp;
  q[0].B = wi; q[0].ldb = p.Dp;
  q[0].C = dx; q[0].ldc = D; q[0].cvec = store16(dx, D, p.es);
  if (!dx) q[0].M = 0;
  q[1].A = dgu; q[1].lda = 2LL * p.Fp;
  q[1].B = xp; q[1].ldb = p.Dp;
  q[1].C = dw_in; q[1].ldc = D; q[1].cvec = store16(dw_in, D, p.es);
  if (!dw_in) q[1].M = 0;
  q[2].A = dyp; q[2].lda = p.Dp;
  q[2].B = h; q[2].ldb = p.Fp;
  q[2].C = dw_out; q[2].ldc = F; q[2].cvec = store16(dw_out, F, p.es);
  if (!dw_out) q[2].M = 0;
  return dev(rnn_launch_ffn_grads(q, p.order, p.grads_choice.tile, bf, s));
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
  return dev(rnn_launch_ckpt_load(wtype == RNN_W_BF16, rows, cols, kept, x, cols, hs(stream)));
}

}  // extern "C"
