// C ABI of the operators of a state-space block (normalisation, causal
// convolution, selective state-space scan): argument checks, workspace
// layouts, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "rnn.h"
#include "ssm_common.h"

using namespace rnnk;

namespace {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
inline bool aligned(const void* p) { return ((uintptr_t)p & (kAlign - 1)) == 0; }

rnn_status_t dev(hipError_t e) { return e == hipSuccess ? RNN_STATUS_SUCCESS : RNN_STATUS_DEVICE; }
inline hipStream_t hs(void* s) { return reinterpret_cast<hipStream_t>(s); }

#define LM_TRY(expr)                                 \
  do {                                               \
    const rnn_status_t st_ = (expr);                 \
    if (st_ != RNN_STATUS_SUCCESS) return st_;       \
  } while (0)

bool wtype_ok(int w) { return w == RNN_W_F32 || w == RNN_W_BF16; }

rnn_status_t room(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws)) return RNN_STATUS_INVALID_ARG;
  return have < need ? RNN_STATUS_WORKSPACE_TOO_SMALL : RNN_STATUS_SUCCESS;
}

// ------------------------------------------------------------------- norm
rnn_status_t norm_sizes(int M, int D) {
  if (M < 0 || D < 0) return RNN_STATUS_INVALID_ARG;
  return D >= (1 << 20) || M >= (1 << 30) ? RNN_STATUS_UNSUPPORTED : RNN_STATUS_SUCCESS;
}
bool norm_ok(int kind, int wtype) { return (kind == RNN_NORM_LAYER || kind == RNN_NORM_RMS) && wtype_ok(wtype); }
size_t norm_bytes(int M, int D) { return std::max(kAlign, align_up((size_t)norm_parts(M, D) * 2 * D * 4)); }

// ------------------------------------------------------------------- conv
rnn_status_t conv_sizes(int T, int B, int C, int K) {
  if (T < 0 || B < 0 || C < 0 || K < 1) return RNN_STATUS_INVALID_ARG;
  if (K > kConvMost || (long long)B * C >= (1LL << 30) || T >= (1 << 30)) return RNN_STATUS_UNSUPPORTED;
  // threads of a launch, 256 a workgroup
  return std::max(conv_blocks(T, B, C, false), conv_blocks(T, B, C, true)) >= (1 << 24) ? RNN_STATUS_UNSUPPORTED : RNN_STATUS_SUCCESS;
}
bool conv_ok(int act, int wtype) { return (act == RNN_ACT_NONE || act == RNN_ACT_SILU) && wtype_ok(wtype); }

ConvParams conv_params(int act, int T, int B, int C, int K, bool back) {
  ConvParams p{};
  p.T = T; p.B = B; p.C = C; p.K = K;
  p.silu = act == RNN_ACT_SILU;
  p.piece = conv_piece(T, B, C, back);
  p.pieces = std::max(1, (T + p.piece - 1) / p.piece);
  return p;
}
size_t conv_bytes(int T, int B, int C, int K) {
  return std::max(kAlign, align_up((size_t)conv_parts(T, B, C) * (K + 1) * C * 4));
}

// -------------------------------------------------------------------- ssm
rnn_status_t ssm_sizes(int T, int B, int E, int N, int groups) {
  if (T < 0 || B < 0 || E < 0 || N < 1 || groups < 1 || E % groups) return RNN_STATUS_INVALID_ARG;
  if (N > kSsmStates || E >= (1 << 22) || (long long)B * E >= (1LL << 30) || T >= (1 << 30)) return RNN_STATUS_UNSUPPORTED;
  // threads of a launch, 256 a workgroup
  return ssm_blocks(B, E, N, groups) >= (1 << 24) ? RNN_STATUS_UNSUPPORTED : RNN_STATUS_SUCCESS;
}
bool ssm_ok(int mode, int wtype) { return (mode == RNN_DELTA_SOFTPLUS || mode == RNN_DELTA_LINEAR) && wtype_ok(wtype); }

size_t ssm_bytes(const SsmPlan& q) { return std::max(kAlign, q.all * 4); }

// a pass's segments and its parts of the workspace
void ssm_room(SsmParams& p, const SsmPlan& q, bool back, void* ws) {
  float* f = (float*)ws;
  p.segs = q.segs[back];
  p.sub = q.sub;
  p.seg_steps = q.seg_steps[back];
  p.seg_first = f + q.first;
  p.seg_q = f + q.q;
  p.seg_d = f + q.d;
  p.starts = f + q.starts;
  p.part = f + q.part;
}

// rows `ld` elements apart; over several steps, four of them lie within 32 bits of each other
rnn_status_t ssm_rows(int T, int B, const void* x, long long ld, long long width) {
  if (!x) return RNN_STATUS_SUCCESS;
  if (ld < width) return RNN_STATUS_INVALID_ARG;
  return T > 1 && ld > (1 << 28) / std::max(B, 1) ? RNN_STATUS_UNSUPPORTED : RNN_STATUS_SUCCESS;
}

// the inputs' checks; they are needed where there are steps
rnn_status_t ssm_inputs(SsmParams& p, const rnn_ssm_inputs_t* in, int mode, int T, int B, int E, int N, int groups) {
  if (!in || !in->A) return RNN_STATUS_INVALID_ARG;
  if (T > 0 && (!in->u || !in->delta || !in->Bm || !in->Cm)) return RNN_STATUS_INVALID_ARG;
  const long long GN = (long long)groups * N;
  LM_TRY(ssm_rows(T, B, in->u, in->ldu, E));
  LM_TRY(ssm_rows(T, B, in->delta, in->lddelta, E));
  LM_TRY(ssm_rows(T, B, in->z, in->ldz, E));
  LM_TRY(ssm_rows(T, B, in->Bm, in->ldB, GN));
  LM_TRY(ssm_rows(T, B, in->Cm, in->ldC, GN));
  p.T = T; p.B = B; p.E = E; p.N = N; p.G = groups;
  p.softplus = mode == RNN_DELTA_SOFTPLUS;
  p.u = in->u; p.delta = in->delta; p.z = in->z; p.Bm = in->Bm; p.Cm = in->Cm;
  p.ldu = in->ldu; p.lddelta = in->lddelta; p.ldz = in->ldz; p.ldB = in->ldB; p.ldC = in->ldC;
  p.A = in->A; p.D = in->D; p.delta_bias = in->delta_bias;
  return RNN_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

rnn_status_t rnn_norm_workspace_size(int M, int D, size_t* bytes) {
  if (!bytes) return RNN_STATUS_INVALID_ARG;
  LM_TRY(norm_sizes(M, D));
  *bytes = norm_bytes(M, D);
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_norm_forward(void* stream, rnn_norm_t kind, rnn_wtype_t wtype, int M, int D, const void* x,
                              const void* residual, const float* weight, const float* bias, float eps, void* y,
                              void* total, float* stats) {
  if (!norm_ok(kind, wtype) || !(eps >= 0.f) || !std::isfinite(eps)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(norm_sizes(M, D));
  if (M == 0 || D == 0) return RNN_STATUS_SUCCESS;
  if (!x || !y) return RNN_STATUS_INVALID_ARG;
  NormParams p{};
  p.M = M; p.D = D; p.rms = kind == RNN_NORM_RMS; p.eps = eps;
  p.x = x; p.residual = residual; p.weight = weight; p.bias = bias;
  p.y = y; p.total = total; p.stats = stats;
  return dev(rnn_launch_norm_fwd(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_norm_backward(void* stream, rnn_norm_t kind, rnn_wtype_t wtype, int M, int D, const void* s,
                               const float* weight, const float* stats, const void* dy, const void* dtotal, void* dx,
                               float* dweight, float* dbias, void* ws, size_t ws_bytes) {
  if (!norm_ok(kind, wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(norm_sizes(M, D));
  if (dweight || dbias) LM_TRY(room(ws, ws_bytes, norm_bytes(M, D)));
  if (D == 0) return RNN_STATUS_SUCCESS;
  if (M > 0 && (!s || !stats || !dy)) return RNN_STATUS_INVALID_ARG;
  NormParams p{};
  p.M = M; p.D = D; p.rms = kind == RNN_NORM_RMS;
  p.x = s; p.weight = weight; p.stats = const_cast<float*>(stats);   // read only
  p.dy = dy; p.dtotal = dtotal; p.dx = dx; p.dweight = dweight; p.dbias = dbias;
  p.part = (float*)ws;
  return dev(rnn_launch_norm_bwd(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_conv_forward(void* stream, rnn_act_t act, rnn_wtype_t wtype, int T, int B, int C, int K,
                              const void* x, long long ldx, const float* w, const float* bias, const void* s0,
                              const int* lengths, void* y, long long ldy, void* sy) {
  if (!conv_ok(act, wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(conv_sizes(T, B, C, K));
  if (ldx < C || ldy < C) return RNN_STATUS_INVALID_ARG;
  if (B == 0 || C == 0) return RNN_STATUS_SUCCESS;
  if (!w || (T > 0 && (!x || !y))) return RNN_STATUS_INVALID_ARG;
  ConvParams p = conv_params(act, T, B, C, K, false);
  p.x = x; p.ldx = ldx; p.w = w; p.bias = bias; p.s0 = s0; p.lengths = lengths;
  p.y = y; p.ldy = ldy; p.sy = sy;
  return dev(rnn_launch_conv_fwd(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_conv_step(void* stream, rnn_act_t act, rnn_wtype_t wtype, int B, int C, int K, const void* x,
                           long long ldx, const float* w, const float* bias, const void* s, void* y, long long ldy,
                           void* sy) {
  if (!conv_ok(act, wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(conv_sizes(1, B, C, K));
  if (ldx < C || ldy < C) return RNN_STATUS_INVALID_ARG;
  if (B == 0 || C == 0) return RNN_STATUS_SUCCESS;
  if (!w || !x || !y) return RNN_STATUS_INVALID_ARG;
  ConvParams p = conv_params(act, 1, B, C, K, false);
  p.x = x; p.ldx = ldx; p.w = w; p.bias = bias; p.s0 = s;
  p.y = y; p.ldy = ldy; p.sy = sy;
  return dev(rnn_launch_conv_step(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_conv_workspace_size(int T, int B, int C, int K, size_t* bytes) {
  if (!bytes) return RNN_STATUS_INVALID_ARG;
  LM_TRY(conv_sizes(T, B, C, K));
  *bytes = conv_bytes(T, B, C, K);
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_conv_backward(void* stream, rnn_act_t act, rnn_wtype_t wtype, int T, int B, int C, int K,
                               const void* x, long long ldx, const float* w, const float* bias, const void* s0,
                               const int* lengths, const void* dy, long long lddy, const void* dsy, void* dx,
                               long long lddx, float* dw, float* dbias, void* ds0, void* ws, size_t ws_bytes) {
  if (!conv_ok(act, wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(conv_sizes(T, B, C, K));
  if (ldx < C || lddy < C || (dx && lddx < C)) return RNN_STATUS_INVALID_ARG;
  if (dw || dbias) LM_TRY(room(ws, ws_bytes, conv_bytes(T, B, C, K)));
  if (C == 0) return RNN_STATUS_SUCCESS;
  if (B > 0 && (!w || (T > 0 && (!x || !dy)))) return RNN_STATUS_INVALID_ARG;
  ConvParams p = conv_params(act, T, B, C, K, true);
  p.x = x; p.ldx = ldx; p.w = w; p.bias = bias; p.s0 = s0; p.lengths = lengths;
  p.dy = dy; p.lddy = lddy; p.dsy = dsy;
  p.dx = dx; p.lddx = lddx; p.dw = dw; p.dbias = dbias; p.ds0 = ds0;
  p.part = (float*)ws;
  return dev(rnn_launch_conv_bwd(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_ssm_step(void* stream, rnn_delta_t mode, rnn_wtype_t wtype, int B, int E, int N, int groups,
                          const rnn_ssm_inputs_t* in, const float* h, void* y, long long ldy, float* hy) {
  if (!ssm_ok(mode, wtype)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ssm_sizes(1, B, E, N, groups));
  if (B == 0 || E == 0) return RNN_STATUS_SUCCESS;
  SsmParams p{};
  LM_TRY(ssm_inputs(p, in, mode, 1, B, E, N, groups));
  if (!y) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ssm_rows(1, B, y, ldy, E));
  p.h0 = h; p.y = y; p.ldy = ldy; p.hy = hy;
  return dev(rnn_launch_ssm_step(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_ssm_workspace_size(int T, int B, int E, int N, int groups, rnn_save_t save, size_t* bytes) {
  if (!bytes || (save != RNN_SAVE_NONE && save != RNN_SAVE_FULL)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ssm_sizes(T, B, E, N, groups));
  *bytes = ssm_bytes(ssm_plan(T, B, E, N, groups, save == RNN_SAVE_FULL));
  return RNN_STATUS_SUCCESS;
}

rnn_status_t rnn_ssm_forward(void* stream, rnn_delta_t mode, rnn_wtype_t wtype, rnn_save_t save, int T, int B, int E,
                             int N, int groups, const rnn_ssm_inputs_t* in, const float* h0, const int* lengths,
                             void* y, long long ldy, float* hy, void* ws, size_t ws_bytes) {
  if (!ssm_ok(mode, wtype) || (save != RNN_SAVE_NONE && save != RNN_SAVE_FULL)) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ssm_sizes(T, B, E, N, groups));
  const SsmPlan plan = ssm_plan(T, B, E, N, groups, save == RNN_SAVE_FULL);
  LM_TRY(room(ws, ws_bytes, ssm_bytes(plan)));
  if (B == 0 || E == 0) return RNN_STATUS_SUCCESS;
  SsmParams p{};
  LM_TRY(ssm_inputs(p, in, mode, T, B, E, N, groups));
  if (T > 0 && !y) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ssm_rows(T, B, y, ldy, E));
  p.h0 = h0; p.lengths = lengths; p.y = y; p.ldy = ldy; p.hy = hy;
  ssm_room(p, plan, false, ws);
  if (save == RNN_SAVE_NONE) p.starts = nullptr;
  return dev(rnn_launch_ssm_fwd(p, wtype == RNN_W_BF16, hs(stream)));
}

rnn_status_t rnn_ssm_backward(void* stream, rnn_delta_t mode, rnn_wtype_t wtype, int T, int B, int E, int N,
                              int groups, const rnn_ssm_inputs_t* in, const int* lengths, const void* dy,
                              long long lddy, const float* dhy, const rnn_ssm_grads_t* grads, void* ws,
                              size_t ws_bytes) {
  if (!ssm_ok(mode, wtype) || !grads) return RNN_STATUS_INVALID_ARG;
  LM_TRY(ssm_sizes(T, B, E, N, groups));
  const SsmPlan plan = ssm_plan(T, B, E, N, groups, true);
  LM_TRY(room(ws, ws_bytes, ssm_bytes(plan)));
  SsmParams p{};
  const long long GN = (long long)groups * N;
  const rnn_ssm_grads_t& g = *grads;
  if (E > 0) {
    LM_TRY(ssm_inputs(p, in, mode, B > 0 ? T : 0, B, E, N, groups));
    if ((B > 0 && T > 0 && !dy) || (g.dz && !in->z)) return RNN_STATUS_INVALID_ARG;
  } else {                               // dB and dC, sums over no channels, are 0
    p.T = T; p.B = B; p.N = N; p.G = groups;
  }
  LM_TRY(ssm_rows(T, B, dy, lddy, E));
  LM_TRY(ssm_rows(T, B, g.du, g.lddu, E));
  LM_TRY(ssm_rows(T, B, g.ddelta, g.ldddelta, E));
  LM_TRY(ssm_rows(T, B, g.dz, g.lddz, E));
  LM_TRY(ssm_rows(T, B, g.dBm, g.lddB, GN));
  LM_TRY(ssm_rows(T, B, g.dCm, g.lddC, GN));
  p.lengths = lengths; p.dy = dy; p.lddy = lddy; p.dhy = dhy;
  p.du = g.du; p.ddelta = g.ddelta; p.dz = g.dz; p.dBm = g.dBm; p.dCm = g.dCm;
  p.lddu = g.lddu; p.ldddelta = g.ldddelta; p.lddz = g.lddz; p.lddB = g.lddB; p.lddC = g.lddC;
  p.dA = g.dA; p.dD = g.dD; p.ddelta_bias = g.ddelta_bias; p.dh0 = g.dh0;
  ssm_room(p, plan, true, ws);
  return dev(rnn_launch_ssm_bwd(p, wtype == RNN_W_BF16, hs(stream)));
}

}  // extern "C"
