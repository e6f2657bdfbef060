// Selective state-space scan (gfx950), forward and single steps:
//   h_t[n] = exp(d_t A[n]) h_(t-1)[n] + d_t u_t B_t[n],  y_t = (C_t . h_t + D u_t) silu(z_t)
//
// A workgroup holds 64 / S channels of one row and walks their steps in blocks
// of 64.  Its waves hold consecutive pieces of a block: each composes its piece
// from a state of zero (h = P h' + Q with P = exp(A sum d)), the maps go
// through LDS, and each wave walks its piece again from the true state with the
// exponentials still in registers.  P is kept as its square root: applied
// twice, it carries a state through a decay of up to 2^-252 without loss.
#include <algorithm>

#include "ssm_util.h"

using namespace rnnk;

namespace {

constexpr int kSteps = 16, kWaves = kSsmBlock / kSteps;   // of a wave's piece, of a block

template <bool BF, int S>
__global__ __launch_bounds__(256) void step_kernel(const SsmParams p, int waves) {
  constexpr int R = kSsmPer;
  const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (wave >= waves) return;
  const SsmPlace q = ssm_place<S>(p, wave);
  if (!q.live) return;
  const int left = p.N - q.n;
  const long long st = ((long long)q.b * p.E + q.e) * p.N + q.n;
  float A[R], B[R], C[R], h[R] = {};
  load_states(p.A + (long long)q.e * p.N + q.n, left, A);
  if (p.h0) load_states(p.h0 + st, left, h);
  load_piece<BF, R>((const El<BF>*)p.Bm + q.b * p.ldB + q.g * p.N + q.n, left, B);
  load_piece<BF, R>((const El<BF>*)p.Cm + q.b * p.ldC + q.g * p.N + q.n, left, C);
  const float u = el_load<BF>((const El<BF>*)p.u + q.b * p.ldu + q.e);
  float d = el_load<BF>((const El<BF>*)p.delta + q.b * p.lddelta + q.e) + (p.delta_bias ? p.delta_bias[q.e] : 0.f);
  const float z = p.z ? el_load<BF>((const El<BF>*)p.z + q.b * p.ldz + q.e) : 0.f;
  const float D = p.D ? p.D[q.e] : 0.f;
  if (p.softplus) d = softplus(d);
  const float du = d * u;
  float o = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    h[r] = fmaf(__builtin_amdgcn_exp2f(d * (A[r] * kLog2e)), h[r], du * B[r]);
    o = fmaf(C[r], h[r], o);
  }
  if (p.hy) store_states(p.hy + st, left, h);
  o = sum_channel<S>(o);
  if (q.j) return;
  o = fmaf(D, u, o);
  if (p.z) {
    float a, da;
    act_pair<ACT_SILU>(z, a, da);
    o *= a;
  }
  el_store<BF>((El<BF>*)p.y + q.b * p.ldy + q.e, o);
}

template <bool BF, int S>
__global__ __launch_bounds__(64 * kWaves) void fwd_kernel(const SsmParams p) {
  constexpr int R = kSsmPer, G = kSteps, W = kWaves, NP = S * R, I = G / S, PER = kSsmBlock * 2 * NP / (64 * W);
  __shared__ __align__(16) float bc[3][kSsmBlock][2][NP];
  __shared__ __align__(16) float maps[2][W][2][64 * R];
  const SsmPlace q = ssm_place<S>(p, blockIdx.x);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int left = q.live ? p.N - q.n : 0;
  const long long st = ((long long)q.b * p.E + q.e) * p.N + q.n;
  float A2[R], carry[R] = {};
  load_states(p.A + (long long)q.e * p.N + q.n, left, A2);
  if (p.h0) load_states(p.h0 + st, left, carry);
#pragma unroll
  for (int r = 0; r < R; ++r) A2[r] *= kLog2e;
  const float bias = p.delta_bias && q.live ? p.delta_bias[q.e] : 0.f, D = p.D && q.live ? p.D[q.e] : 0.f;
  const int blocks = (q.len + kSsmBlock - 1) / kSsmBlock;

  float ru[I], rd[I], rz[I], rbc[PER];
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int t = k * kSsmBlock + wave * G + i * S + q.j;
      const bool on = t < q.len && q.live;
      const long long row = (long long)t * p.B + q.b;
      ru[i] = on ? el_load<BF>((const El<BF>*)p.u + row * p.ldu + q.e) : 0.f;
      rd[i] = on ? el_load<BF>((const El<BF>*)p.delta + row * p.lddelta + q.e) : 0.f;
      rz[i] = on && p.z ? el_load<BF>((const El<BF>*)p.z + row * p.ldz + q.e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = threadIdx.x + i * 64 * W, n = x % NP, c = x / NP % 2, t = k * kSsmBlock + x / (2 * NP);
      const long long row = (long long)t * p.B + q.b;
      rbc[i] = 0.f;
      if (t < q.len && n < p.N)
        rbc[i] = c ? el_load<BF>((const El<BF>*)p.Cm + row * p.ldC + q.g * p.N + n) : el_load<BF>((const El<BF>*)p.Bm + row * p.ldB + q.g * p.N + n);
    }
  };
  auto stage = [&](int k) {
    float* to = &bc[k % 3][0][0][0];
#pragma unroll
    for (int i = 0; i < PER; ++i) to[threadIdx.x + i * 64 * W] = rbc[i];
  };
  if (blocks) {
    load(0);
    stage(0);
    __syncthreads();
  }
  for (int k = 0; k < blocks; ++k) {
    float u[I], d[I], du[I], z[I], sum = 0.f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const bool on = k * kSsmBlock + wave * G + i * S + q.j < q.len && q.live;
      u[i] = ru[i];
      z[i] = rz[i];
      d[i] = rd[i] + bias;
      if (p.softplus) d[i] = softplus(d[i]);
      if (!on) d[i] = 0.f;
      du[i] = d[i] * u[i];
      sum += d[i];
    }
    sum = sum_channel<S>(sum);
    if (k + 1 < blocks) load(k + 1);
    const float* from = &bc[k % 3][wave * G][0][q.n];
    float a[G][R], h[R] = {};
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const float ds = from_lane<S>(d[s / S], s % S), dus = from_lane<S>(du[s / S], s % S);
      float B[R];
      lds_get(from + s * 2 * NP, B);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a[s][r] = __builtin_amdgcn_exp2f(ds * A2[r]);
        h[r] = fmaf(a[s][r], h[r], dus * B[r]);
      }
    }
    float P[R];
#pragma unroll
    for (int r = 0; r < R; ++r) P[r] = __builtin_amdgcn_exp2f(fminf(0.5f * A2[r] * sum, 127.f));
    lds_put(&maps[k & 1][wave][0][lane * R], P);
    lds_put(&maps[k & 1][wave][1][lane * R], h);
    // a wave may still walk block k - 1: its B and C are a third buffer's, its maps the other one's
    if (k + 1 < blocks) stage(k + 1);
    __syncthreads();
    if (p.starts && wave == 0 && q.live)
      store_states(p.starts + (((long long)k * p.B + q.b) * p.E + q.e) * NP + q.n, R, carry);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      float Q[R];
      lds_get(&maps[k & 1][w][0][lane * R], P);
      lds_get(&maps[k & 1][w][1][lane * R], Q);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (w == wave) h[r] = carry[r];
        carry[r] = fmaf(P[r], P[r] * carry[r], Q[r]);
      }
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float part[S];
#pragma unroll
      for (int l = 0; l < S; ++l) {
        const int s = i * S + l;
        const float dus = from_lane<S>(du[i], l);
        float B[R], C[R];
        lds_get(from + s * 2 * NP, B);
        lds_get(from + s * 2 * NP + NP, C);
        part[l] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          h[r] = fmaf(a[s][r], h[r], dus * B[r]);
          part[l] = fmaf(C[r], h[r], part[l]);
        }
      }
      float o = fmaf(D, u[i], sum_to_lane<S>(part));
      if (p.z) {
        float g, slope;
        act_pair<ACT_SILU>(z[i], g, slope);
        o *= g;
      }
      const int t = k * kSsmBlock + wave * G + i * S + q.j;
      if (q.live && t < p.T) el_store<BF>((El<BF>*)p.y + ((long long)t * p.B + q.b) * p.ldy + q.e, t < q.len ? o : 0.f);
    }
  }
  if (!q.live) return;
  for (int t = blocks * kSsmBlock + wave * S + q.j; t < p.T; t += W * S)
    el_store<BF>((El<BF>*)p.y + ((long long)t * p.B + q.b) * p.ldy + q.e, 0.f);
  if (p.hy && wave == 0) store_states(p.hy + st, left, carry);
}

template <bool BF, int S>
hipError_t start(const SsmParams& p, bool step, hipStream_t s) {
  constexpr int CH = 64 / S;
  const long long tiles = (p.E / p.G + CH - 1) / CH, all = tiles * p.G * p.B;   // at most B * E
  if (step) hipLaunchKernelGGL((step_kernel<BF, S>), dim3((unsigned)((all + 3) / 4)), dim3(256), 0, s, p, (int)all);
  else hipLaunchKernelGGL((fwd_kernel<BF, S>), dim3((unsigned)all), dim3(64 * kWaves), 0, s, p);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch(const SsmParams& p, bool step, hipStream_t s) {
  if (p.B == 0 || p.E == 0) return hipSuccess;
  switch (ssm_lanes(p.N)) {
    case 1: return start<BF, 1>(p, step, s);
    case 2: return start<BF, 2>(p, step, s);
    case 4: return start<BF, 4>(p, step, s);
    case 8: return start<BF, 8>(p, step, s);
    default: return start<BF, 16>(p, step, s);
  }
}

}  // namespace

hipError_t rnn_launch_ssm_step(const SsmParams& p, int bf16, hipStream_t s) {
  return bf16 ? launch<true>(p, true, s) : launch<false>(p, true, s);
}
hipError_t rnn_launch_ssm_fwd(const SsmParams& p, int bf16, hipStream_t s) {
  return bf16 ? launch<true>(p, false, s) : launch<false>(p, false, s);
}
