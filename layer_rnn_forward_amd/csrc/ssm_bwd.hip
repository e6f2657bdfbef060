// Gradients of the selective state-space scan (gfx950).  With do = dy silu(z)
// and g_t the gradient of h_t,
//   g_t = C_t do_t + a_(t+1) g_(t+1),  a = exp(d A)
//   dC_t = sum_e do h_t     dB_t = sum_e g d u     du = d (g . B) + D do
//   dd = sum_n A g a h_(t-1) + u (g . B)           dA = sum_t d g a h_(t-1)
//
// A workgroup walks the blocks of 64 steps backwards.  Forward left the state
// before every block; each wave holds 8 steps (16 with 16 lanes a channel), composes its forward
// map and its map of g (which has the same decay), and after one exchange
// through LDS walks its steps forwards for the states and backwards for the
// gradients, with exponentials and states in registers.  The sums over
// channels of dB and dC are made within a wave, written for each tile of
// channels, and added in a second launch; parameters' gradients stay in
// registers over all steps and are added over rows there, too.  All in a fixed
// order.
#include <algorithm>

#include "ssm_util.h"

using namespace rnnk;

namespace {

// steps of a wave's piece (a lane of a channel owns at least one)
constexpr int steps_of(int S) { return S < 8 ? 8 : S; }

// Partial sums in the workspace: [tiles][T][B][G][2][NP] of dB and dC, then
// [B][E][NP] of dA and [B][E] of dD and ddelta_bias.
struct Parts {
  float *bc, *A, *D, *bias;
};
Parts parts_of(const SsmParams& p, int tiles, int NP) {
  Parts r;
  r.bc = p.part;
  r.A = r.bc + (size_t)tiles * p.T * p.B * p.G * 2 * NP;
  r.D = r.A + (size_t)p.B * p.E * NP;
  r.bias = r.D + (size_t)p.B * p.E;
  return r;
}

// V values a lane, summed over the lanes whose indexes differ in the bits BIT
// (32 first) down to S: while there are several values each fold halves them,
// then every lane gets the sum.  Lane bit 32 holds the upper half of the values, ...
template <int S, int BIT, int V>
__device__ __forceinline__ void sum_channels(float (&v)[V]) {
  if constexpr (BIT >= S) {
    if constexpr (V > 1) {
      float h[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) h[i] = fold<BIT>(v[i], v[i + V / 2]);
      sum_channels<S, BIT / 2, V / 2>(h);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) v[i] = h[i];
    } else {
      if constexpr (BIT >= 16) v[0] = fold<BIT>(v[0], v[0]);
      else v[0] += lane_xor<BIT>(v[0]);
      sum_channels<S, BIT / 2, V>(v);
    }
  }
}

template <bool BF, int S>
__global__ __launch_bounds__(64 * (kSsmBlock / steps_of(S))) void bwd_kernel(const SsmParams p, const Parts out) {
  constexpr int R = kSsmPer, G = steps_of(S), W = kSsmBlock / G, NP = S * R, I = G / S, PER = kSsmBlock * 2 * NP / (64 * W), CH = 64 / S;
  __shared__ __align__(16) float bc[3][kSsmBlock][2][NP];
  __shared__ __align__(16) float maps[2][W][3][64 * R];
  const SsmPlace q = ssm_place<S>(p, blockIdx.x);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int left = q.live ? p.N - q.n : 0;
  const long long st = ((long long)q.b * p.E + q.e) * p.N + q.n;
  float A[R], carry[R] = {}, dA[R] = {}, dD = 0.f, dbias = 0.f;
  load_states(p.A + (long long)q.e * p.N + q.n, left, A);
  if (p.dhy) load_states(p.dhy + st, left, carry);
  const float bias = p.delta_bias && q.live ? p.delta_bias[q.e] : 0.f, D = p.D && q.live ? p.D[q.e] : 0.f;
  const int blocks = (q.len + kSsmBlock - 1) / kSsmBlock;

  float ru[I], rd[I], rz[I], rdy[I], rbc[PER], start[R];
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int t = k * kSsmBlock + wave * G + i * S + q.j;
      const bool on = t < q.len && q.live;
      const long long row = (long long)t * p.B + q.b;
      ru[i] = on ? el_load<BF>((const El<BF>*)p.u + row * p.ldu + q.e) : 0.f;
      rd[i] = on ? el_load<BF>((const El<BF>*)p.delta + row * p.lddelta + q.e) : 0.f;
      rz[i] = on && p.z ? el_load<BF>((const El<BF>*)p.z + row * p.ldz + q.e) : 0.f;
      rdy[i] = on ? el_load<BF>((const El<BF>*)p.dy + row * p.lddy + q.e) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = threadIdx.x + i * 64 * W, n = x % NP, c = x / NP % 2, t = k * kSsmBlock + x / (2 * NP);
      const long long row = (long long)t * p.B + q.b;
      rbc[i] = 0.f;
      if (t < q.len && n < p.N)
        rbc[i] = c ? el_load<BF>((const El<BF>*)p.Cm + row * p.ldC + q.g * p.N + n) : el_load<BF>((const El<BF>*)p.Bm + row * p.ldB + q.g * p.N + n);
    }
    load_states(p.starts + (((long long)k * p.B + q.b) * p.E + q.e) * NP + q.n, q.live ? R : 0, start);
  };
  auto stage = [&](int k) {
    float* to = &bc[k % 3][0][0][0];
#pragma unroll
    for (int i = 0; i < PER; ++i) to[threadIdx.x + i * 64 * W] = rbc[i];
  };
  if (blocks) {
    load(blocks - 1);
    stage(blocks - 1);
    __syncthreads();
  }
  for (int k = blocks - 1; k >= 0; --k) {
    float u[I], d[I], du[I], z[I], dy[I], go[I], slope[I], sum = 0.f, first[R];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const bool on = k * kSsmBlock + wave * G + i * S + q.j < q.len && q.live;
      u[i] = ru[i];
      z[i] = rz[i];
      dy[i] = rdy[i];
      const float pre = rd[i] + bias;
      d[i] = pre;
      slope[i] = 1.f;                    // of d to delta
      if (p.softplus) {
        float neg;
        d[i] = softplus(pre);
        sigmoid_pair(pre, slope[i], neg);
      }
      if (!on) d[i] = slope[i] = 0.f;
      du[i] = d[i] * u[i];
      go[i] = dy[i];
      if (p.z) {
        float g, unused;
        act_pair<ACT_SILU>(z[i], g, unused);
        go[i] *= g;
      }
      sum += d[i];
    }
    sum = sum_channel<S>(sum);
#pragma unroll
    for (int r = 0; r < R; ++r) first[r] = start[r];
    if (k > 0) load(k - 1);
    const float* from = &bc[k % 3][wave * G][0][q.n];
    float a[G][R], h[R] = {}, e[R] = {};
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const float ds = from_lane<S>(d[s / S], s % S), dus = from_lane<S>(du[s / S], s % S);
      float B[R];
      lds_get(from + s * 2 * NP, B);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        a[s][r] = __builtin_amdgcn_exp2f(ds * (A[r] * kLog2e));
        h[r] = fmaf(a[s][r], h[r], dus * B[r]);
      }
    }
#pragma unroll
    for (int s = G - 1; s >= 0; --s) {
      const float gs = from_lane<S>(go[s / S], s % S);
      float C[R];
      lds_get(from + s * 2 * NP + NP, C);
#pragma unroll
      for (int r = 0; r < R; ++r) e[r] = a[s][r] * fmaf(C[r], gs, e[r]);
    }
    float P[R];
#pragma unroll
    for (int r = 0; r < R; ++r) P[r] = __builtin_amdgcn_exp2f(fminf(0.5f * kLog2e * A[r] * sum, 127.f));
    lds_put(&maps[k & 1][wave][0][lane * R], P);
    lds_put(&maps[k & 1][wave][1][lane * R], h);
    lds_put(&maps[k & 1][wave][2][lane * R], e);
    if (k > 0) stage(k - 1);
    __syncthreads();
    // the state before the wave's steps, and what of g its last step gets from the steps that follow
#pragma unroll
    for (int r = 0; r < R; ++r) h[r] = first[r];
    for (int w = 0; w < wave; ++w) {
      float Q[R];
      lds_get(&maps[k & 1][w][0][lane * R], P);
      lds_get(&maps[k & 1][w][1][lane * R], Q);
#pragma unroll
      for (int r = 0; r < R; ++r) h[r] = fmaf(P[r], P[r] * h[r], Q[r]);
    }
#pragma unroll
    for (int w = W - 1; w >= 0; --w) {
      float Q[R];
      lds_get(&maps[k & 1][w][0][lane * R], P);
      lds_get(&maps[k & 1][w][2][lane * R], Q);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (w == wave) e[r] = carry[r];
        carry[r] = fmaf(P[r], P[r] * carry[r], Q[r]);
      }
    }
    // forwards: the state before every step, and what the gate multiplied
    float hb[G][R], o[I];
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
          hb[s][r] = h[r];
          h[r] = fmaf(a[s][r], h[r], dus * B[r]);
          part[l] = fmaf(C[r], h[r], part[l]);
        }
      }
      o[i] = fmaf(D, u[i], sum_to_lane<S>(part));
    }
    // backwards
    float gB[I], gA[I];
#pragma unroll
    for (int i = I - 1; i >= 0; --i) {
      float pB[S], pA[S];
#pragma unroll
      for (int l = S - 1; l >= 0; --l) {
        const int s = i * S + l;
        const float ds = from_lane<S>(d[i], l), dus = from_lane<S>(du[i], l), gs = from_lane<S>(go[i], l);
        float B[R], C[R], v[2 * R];
        lds_get(from + s * 2 * NP, B);
        lds_get(from + s * 2 * NP + NP, C);
        pB[l] = pA[l] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float g = fmaf(C[r], gs, e[r]);
          v[r] = g * dus;
          v[R + r] = gs * (s == G - 1 ? h[r] : hb[s == G - 1 ? s : s + 1][r]);
          pB[l] = fmaf(g, B[r], pB[l]);
          e[r] = g * a[s][r];
          const float x = e[r] * hb[s][r];
          pA[l] = fmaf(x, A[r], pA[l]);
          dA[r] = fmaf(x, ds, dA[r]);
        }
        sum_channels<S, 32, 2 * R>(v);
        // the values a lane has left: folds of the bits 32, 16, ... chose them
        constexpr int LEFT = 2 * R > CH ? 2 * R / CH : 1;
        int first_value = 0;
        bool mine = true;
#pragma unroll
        for (int bit = 32, half = R; bit >= S; bit /= 2, half /= 2) {
          if (half >= 1) first_value += lane & bit ? half : 0;
          else mine = mine && !(lane & bit);
        }
        const int t = k * kSsmBlock + wave * G + s;
        if (mine && t < q.len) {
          float* to = out.bc + (((((long long)q.tile * p.T + t) * p.B + q.b) * p.G + q.g) * 2) * NP;
#pragma unroll
          for (int i2 = 0; i2 < LEFT; ++i2) {
            const int x = first_value + i2;
            to[(x / R) * NP + q.n + x % R] = v[i2];
          }
        }
      }
      gB[i] = sum_to_lane<S>(pB);
      gA[i] = sum_to_lane<S>(pA);
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int t = k * kSsmBlock + wave * G + i * S + q.j;
      const float dd = slope[i] * fmaf(u[i], gB[i], gA[i]);
      dD = fmaf(go[i], u[i], dD);
      dbias += dd;
      if (!q.live || t >= p.T) continue;
      const long long row = (long long)t * p.B + q.b;
      const bool on = t < q.len;
      if (p.du) el_store<BF>((El<BF>*)p.du + row * p.lddu + q.e, on ? fmaf(D, go[i], d[i] * gB[i]) : 0.f);
      if (p.ddelta) el_store<BF>((El<BF>*)p.ddelta + row * p.ldddelta + q.e, on ? dd : 0.f);
      if (p.dz) {
        float g, dg;
        act_pair<ACT_SILU>(z[i], g, dg);
        el_store<BF>((El<BF>*)p.dz + row * p.lddz + q.e, on ? dy[i] * o[i] * dg : 0.f);
      }
    }
  }
  if (q.live)
    for (int t = blocks * kSsmBlock + wave * S + q.j; t < p.T; t += W * S) {
      const long long row = (long long)t * p.B + q.b;
      if (p.du) el_store<BF>((El<BF>*)p.du + row * p.lddu + q.e, 0.f);
      if (p.ddelta) el_store<BF>((El<BF>*)p.ddelta + row * p.ldddelta + q.e, 0.f);
      if (p.dz) el_store<BF>((El<BF>*)p.dz + row * p.lddz + q.e, 0.f);
    }
  if (p.dh0 && wave == 0 && q.live) store_states(p.dh0 + st, left, carry);
  // the waves' sums of the parameters' gradients
  dD = sum_channel<S>(dD);
  dbias = sum_channel<S>(dbias);
  __syncthreads();
  lds_put(&maps[0][wave][0][lane * R], dA);
  maps[0][wave][1][lane] = dD;
  maps[0][wave][2][lane] = dbias;
  __syncthreads();
  if (wave || !q.live) return;
#pragma unroll
  for (int w = 1; w < W; ++w) {
    float v[R];
    lds_get(&maps[0][w][0][lane * R], v);
#pragma unroll
    for (int r = 0; r < R; ++r) dA[r] += v[r];
    dD += maps[0][w][1][lane];
    dbias += maps[0][w][2][lane];
  }
  const long long at = (long long)q.b * p.E + q.e;
  store_states(out.A + at * NP + q.n, R, dA);
  if (q.j == 0) {
    out.D[at] = dD;
    out.bias[at] = dbias;
  }
}

// dB and dC: the tiles' sums
template <bool BF>
__global__ __launch_bounds__(256) void channels_kernel(const SsmParams p, const Parts in, int tiles, int NP) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, all = (long long)p.T * p.B * p.G * 2 * NP;
  if (i >= all) return;
  const int n = (int)(i % NP), c = (int)(i / NP % 2), g = (int)(i / (2 * NP) % p.G);
  const long long row = i / (2LL * NP * p.G);
  if (n >= p.N) return;
  const int b = (int)(row % p.B), len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
  void* to = c ? p.dCm : p.dBm;
  if (!to) return;
  float s = 0.f;
  if (row / p.B < len)
    for (int x = 0; x < tiles; ++x) s += in.bc[x * all + i];
  el_store<BF>((El<BF>*)to + row * (c ? p.lddC : p.lddB) + g * p.N + n, s);
}

// dA, dD, ddelta_bias: the rows' sums
__global__ __launch_bounds__(256) void rows_kernel(const SsmParams p, const Parts in, int NP) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int per = NP + 2, e = (int)(i / per), n = (int)(i % per);
  if (e >= p.E) return;
  float s = 0.f;
  for (int b = 0; b < p.B; ++b) {
    const long long at = (long long)b * p.E + e;
    s += n < NP ? in.A[at * NP + n] : n == NP ? in.D[at] : in.bias[at];
  }
  if (n < p.N) {
    if (p.dA) p.dA[(long long)e * p.N + n] = s;
  } else if (n == NP) {
    if (p.dD) p.dD[e] = s;
  } else if (n == NP + 1) {
    if (p.ddelta_bias) p.ddelta_bias[e] = s;
  }
}

template <bool BF, int S>
hipError_t start(const SsmParams& p, hipStream_t s) {
  constexpr int CH = 64 / S, NP = S * kSsmPer;
  const int tiles = (p.E / p.G + CH - 1) / CH;
  const Parts parts = parts_of(p, tiles, NP);
  if (p.B > 0) hipLaunchKernelGGL((bwd_kernel<BF, S>), dim3((unsigned)(tiles * p.G * p.B)), dim3(64 * (kSsmBlock / steps_of(S))), 0, s, p, parts);
  const long long all = (long long)p.T * p.B * p.G * 2 * NP;
  if ((p.dBm || p.dCm) && all) hipLaunchKernelGGL(channels_kernel<BF>, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, p, parts, tiles, NP);
  if (p.dA || p.dD || p.ddelta_bias)
    hipLaunchKernelGGL(rows_kernel, dim3((unsigned)(((long long)p.E * (NP + 2) + 255) / 256)), dim3(256), 0, s, p, parts, NP);
  return hipGetLastError();
}

template <bool BF>
hipError_t launch(const SsmParams& p, hipStream_t s) {
  switch (ssm_lanes(p.N)) {
    case 1: return start<BF, 1>(p, s);
    case 2: return start<BF, 2>(p, s);
    case 4: return start<BF, 4>(p, s);
    case 8: return start<BF, 8>(p, s);
    default: return start<BF, 16>(p, s);
  }
}

}  // namespace

size_t rnnk::ssm_part_floats(int T, int B, int E, int N, int G) {
  const size_t S = ssm_lanes(N), CH = 64 / S, NP = S * kSsmPer, tiles = (E / G + CH - 1) / CH;
  return tiles * T * B * G * 2 * NP + (size_t)B * E * (NP + 2);
}
size_t rnnk::ssm_start_floats(int T, int B, int E, int N) {
  return ((size_t)T + kSsmBlock - 1) / kSsmBlock * B * E * ssm_lanes(N) * kSsmPer;
}

hipError_t rnn_launch_ssm_bwd(const SsmParams& p, int bf16, hipStream_t s) {
  if (p.E == 0) return hipSuccess;
  return bf16 ? launch<true>(p, s) : launch<false>(p, s);
}
