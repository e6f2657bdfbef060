// Gradients of the selective state-space scan (gfx950).  With do = dy silu(z)
// and g_t the gradient of h_t,
//   g_t = C_t do_t + a_(t+1) g_(t+1),  a = exp(d A)
//   dC_t = sum_e do h_t     dB_t = sum_e g d u     du = d (g . B) + D do
//   dd = sum_n A g a h_(t-1) + u (g . B)           dA = sum_t d g a h_(t-1)
//
// A wave walks the chunks of its 16 channels (16 states each) backwards: from
// the state that forward left before a chunk it walks the chunk forwards, keeps
// the exponentials and the states, and walks it back.  The sums over channels
// of dB and dC are made within a wave, then over the workgroup's waves through
// the LDS, then (where a group has more channels) in a second launch, which
// adds the parameters' gradients of the rows and segments, too.  All in a fixed
// order.
//
// Bound: vector instructions, 107 of them a step and wave (256 states).  2048
// steps of 8 rows of 2048 channels, bf16: 0.51 ms in two segments (their issue
// slots alone 0.40 at 2.4 GHz), the segments' first launch 0.07, the sums of dB
// and dC 0.02.  Two waves a SIMD (204 registers): with three (168 registers and
// 108 bytes spilled) 0.73 ms where two took 0.57, with one segment of one wave a
// SIMD 0.87 where two took 0.61 + 0.11.  Chunks of 16 steps spill: 1.6 ms.
//
// What spills all the same: 79 (16 states) to 149 scalar registers, most of them
// the addresses and strides of the seven tensors that are walked, into lanes of
// vector registers, which every chunk reads back; and with one lane a
// channel (up to 4 states), where a lane owns all 8 steps of a chunk, 76 to 98 of
// 256 vector registers (160 to 204 bytes of scratch): 4 states a channel take as
// long as 16 (0.82 ms for the same pass).
#include <algorithm>

#include "ssm_util.h"

using namespace rnnk;

namespace {

// Partial sums in the workspace: [workgroups of a group][T][B][G][2][NP] of dB and
// dC (where there are several), then [segs * B][E][NP] of dA and [segs * B][E]
// of dD and ddelta_bias.
struct Parts {
  float *bc, *A, *D, *bias;
  int groups;
};
Parts parts_of(const SsmParams& p, int groups, int NP) {
  Parts r;
  r.groups = groups;
  r.bc = p.part;
  r.A = r.bc + (groups > 1 ? (size_t)groups * p.T * p.B * p.G * 2 * NP : 0);
  r.D = r.A + (size_t)p.segs * p.B * p.E * NP;
  r.bias = r.D + (size_t)p.segs * p.B * p.E;
  return r;
}

// V values a lane, summed over the lanes whose indexes differ in the bits BIT
// (32 first) down to S: while there are several values each fold halves them
// (lanes with the bit set go on with the upper half), then every lane gets the
// sum.  sums_left(), first_sum(): how many values a lane has left, and which;
// has_sums(): whether the lane is the one of several with the same to keep them.
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
template <int S, int V>
constexpr int sums_left() { return V * S > 64 ? V * S / 64 : 1; }
template <int S, int V>
__device__ __forceinline__ int first_sum(int lane) {
  int first = 0;
#pragma unroll
  for (int bit = 32, half = V / 2; bit >= S && half >= 1; bit /= 2, half /= 2) first += lane & bit ? half : 0;
  return first;
}
template <int S, int V>
__device__ __forceinline__ bool has_sums(int lane) {
  bool mine = true;
#pragma unroll
  for (int bit = 32, half = V / 2; bit >= S; bit /= 2, half /= 2)
    if (half < 1) mine = mine && !(lane & bit);
  return mine;
}

// LOCAL: the segments' maps of g (but the first one's), no outputs.  PAD: some
// lanes' states are not there; they and their gradients are held at 0, whatever
// d, du and do.
template <bool BF, int S, bool LOCAL, bool PAD>
__global__ __launch_bounds__(64 * kSsmTiles, 2) void bwd_kernel(const SsmParams p, const Parts out) {
  constexpr int R = kSsmPer, G = kSsmKeep, NP = S * R, Q = S < 4 ? S : 4, I = G / Q, CH = 64 / S, W = kSsmTiles;
  __shared__ __align__(16) float bc[W][G][2][NP];
  __shared__ __align__(16) float zeros[LOCAL ? 1 : G][2][NP];
  __shared__ float sums[LOCAL ? 1 : 2][W][G][2][NP];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  SsmPlace q = ssm_place<S>(p, blockIdx.x, wave);
  if (LOCAL) q.seg += p.sub;             // in parts of segments, of which the first segment's are not needed
  if (LOCAL && !__any(q.live)) return;
  const int left = q.live ? p.N - q.n : 0;
  // Lanes of channels that are not there read zeros for B and C: an infinite one
  // must not reach the sums over channels through them.  (Every wave writes them.)
  if constexpr (!LOCAL)
    for (int x = lane; x < G * 2 * NP; x += 64) (&zeros[0][0][0])[x] = 0.f;
  const float* const bcs = (LOCAL || q.live ? &bc[wave][0][0][0] : &zeros[0][0][0]) + q.n;
  const long long at = (long long)q.b * p.E + q.e;
  float A[R], e[R] = {}, dA[R] = {}, dD = 0.f, dbias = 0.f, total = 0.f;
  load_states(p.A + (long long)q.e * p.N + q.n, left, A);
  if (p.segs == 1 || LOCAL) {
    if (p.dhy) load_states(p.dhy + at * p.N + q.n, left, e);
    if (LOCAL) {                       // dhy may be written over by the first segment
      if (q.seg == p.segs * p.sub - 1 && q.live) store_states(p.seg_first + at * NP + q.n, R, e);
#pragma unroll
      for (int r = 0; r < R; ++r) e[r] = 0.f;
    }
  } else if (q.live) {
    load_states(p.seg_first + at * NP + q.n, R, e);
    for (int i = p.segs * p.sub - 1; i >= (q.seg + 1) * p.sub; --i) {
      float Q[R];
      const long long m = (long long)i * p.B * p.E + at;
      load_states(p.seg_q + m * NP + q.n, R, Q);
      const float sum = p.seg_d[m];
#pragma unroll
      for (int r = 0; r < R; ++r) e[r] = through(A[r], sum, Q[r], e[r]);
    }
  }
  const float bias = p.delta_bias ? p.delta_bias[q.e] : 0.f, D = p.D ? p.D[q.e] : 0.f;
  const uint32_t skip = p.D ? ~0u : 0u;  // without D, no product of 0 and what may be infinite
  const int steps = LOCAL ? p.seg_steps / p.sub : p.seg_steps;
  const int begin = min(q.seg * steps, p.T), stop = min(begin + steps, p.T), end = min(stop, q.len);
  int t0 = begin + (end - begin + G - 1) / G * G - G;      // the last chunk with steps, if there is one
  SsmRows xu = ssm_rows<BF, Q>(p, q, p.u, p.ldu, t0), xd = ssm_rows<BF, Q>(p, q, p.delta, p.lddelta, t0),
          xz = ssm_rows<BF, Q>(p, q, p.z, p.ldz, t0), xdy = ssm_rows<BF, Q>(p, q, p.dy, p.lddy, t0);
  SsmRows ydu = ssm_rows<BF, Q>(p, q, p.du, p.lddu, t0), ydd = ssm_rows<BF, Q>(p, q, p.ddelta, p.ldddelta, t0),
          ydz = ssm_rows<BF, Q>(p, q, p.dz, p.lddz, t0);
  El<BF> ru[I] = {}, rd[I], rz[I] = {}, rdy[I];
  RawFour<BF> rbc[bc_pieces<G, NP>()];
  float start[R] = {};
  auto load = [&](int t0) {
    const int left = q.len - t0;
    load_own<BF, Q, true, I>(xd, q, left, rd);
    if (p.z) load_own<BF, Q, true, I>(xz, q, left, rz);
    load_own<BF, Q, true, I>(xdy, q, left, rdy);
    if constexpr (!LOCAL) load_own<BF, Q, true, I>(xu, q, left, ru);
    load_bc<BF, G, NP>(p, q, t0, rbc);
    if constexpr (!LOCAL) {
      load_states(p.starts + ((long long)(t0 / G) * p.B * p.E + at) * NP + q.n, q.live ? R : 0, start);
    }
  };
  if (begin < end) load(t0);
  if constexpr (!LOCAL) {                // the steps past the row's length
    const float none[I] = {};
    const int from = begin < end ? t0 + G : begin;
    SsmRows zdu = ssm_rows<BF, Q>(p, q, p.du, p.lddu, from), zdd = ssm_rows<BF, Q>(p, q, p.ddelta, p.ldddelta, from),
            zdz = ssm_rows<BF, Q>(p, q, p.dz, p.lddz, from);
    for (int t = from; t < stop; t += G) {
      if (p.du) store_own<BF, Q, false, I>(zdu, q, stop - t, none);
      if (p.ddelta) store_own<BF, Q, false, I>(zdd, q, stop - t, none);
      if (p.dz) store_own<BF, Q, false, I>(zdz, q, stop - t, none);
    }
  }
  // A chunk's outputs are stored in the next one, before its loads: a wait for
  // those then has no young stores to wait for.  The waves' sums of dB and dC
  // are added there, too; the other half of `sums` is written meanwhile.
  float rows[3][I] = {};
  // the thread's place in the partial sums: value x of a step, of the chunk's step x / (2 NP)
  const long long step = (long long)p.B * p.G * 2 * NP;
  float* part = out.bc + (((long long)q.group * p.T + t0 + (int)threadIdx.x / (2 * NP)) * p.B + q.b) * p.G * 2 * NP + q.g * 2 * NP + threadIdx.x % (2 * NP);
  auto flush = [&](int t0) {
    if (p.du) store_own<BF, Q, true, I>(ydu, q, stop - t0, rows[0]);
    if (p.ddelta) store_own<BF, Q, true, I>(ydd, q, stop - t0, rows[1]);
    if (p.dz) store_own<BF, Q, true, I>(ydz, q, stop - t0, rows[2]);
    if (!p.dBm && !p.dCm) return;
    __syncthreads();
    if (out.groups > 1) {
#pragma unroll
      for (int i = 0; i < (G * 2 * NP + 64 * W - 1) / (64 * W); ++i) {
        const int x = threadIdx.x + i * 64 * W, s = x / (2 * NP);
        if (G * 2 * NP % (64 * W) && x >= G * 2 * NP) break;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) v += (&sums[LOCAL ? 0 : t0 / G & 1][w][0][0][0])[x];
        if (t0 + s < end) part[i * (64 * W / (2 * NP)) * step] = v;
      }
      part -= G * step;
      return;
    }
    for (int x = threadIdx.x; x < G * 2 * NP; x += 64 * W) {
      const int s = x / (2 * NP), c = x / NP % 2, n = x % NP, t = t0 + s;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += sums[LOCAL ? 0 : t0 / G & 1][w][s][c][n];
      if (t < end && n < p.N && (c ? p.dCm : p.dBm))
        el_store<BF>((El<BF>*)(c ? p.dCm : p.dBm) + ((long long)t * p.B + q.b) * (c ? p.lddC : p.lddB) + q.g * p.N + n, v);
    }
  };
  const int top = t0;
  if (begin < end)
    for (; t0 >= begin; t0 -= G) {
      float u[I], d[I], du[I], go[I], gz[I], slope[I], h[R];
#pragma unroll
      for (int i = 0; i < I; ++i) {
        d[i] = el_load<BF>(&rd[i]) + bias;
        slope[i] = 1.f;                    // of d to delta
      }
      if (p.softplus)
#pragma unroll
        for (int i = 0; i < I; ++i) {
          float neg;
          sigmoid_pair(d[i], slope[i], neg);
          d[i] = softplus(d[i]);
        }
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const bool on = t0 + i * Q + q.j < end && q.live;
        u[i] = on ? el_load<BF>(&ru[i]) : 0.f;
        go[i] = on ? el_load<BF>(&rdy[i]) : 0.f;
        d[i] = on ? d[i] : 0.f;
        slope[i] = on ? slope[i] : 0.f;
        du[i] = d[i] * u[i];
        gz[i] = 0.f;
        total += d[i];
      }
      if (p.z)
#pragma unroll
        for (int i = 0; i < I; ++i) {      // go: of what the gate multiplied, gz: dy times the gate's slope
          const bool on = t0 + i * Q + q.j < end && q.live;
          float g, dg;
          act_pair<ACT_SILU>(on ? el_load<BF>(&rz[i]) : 0.f, g, dg);
          gz[i] = go[i] * dg;
          go[i] *= g;
        }
#pragma unroll
      for (int r = 0; r < R; ++r) h[r] = start[r];
      put_bc<BF, G, NP>(&bc[wave][0][0][0], rbc);
      if (!LOCAL && t0 < top) flush(t0 + G);
      if (t0 > begin) load(t0 - G);
      // GUARD: states that are not there and their gradients are held at 0 (an
      // infinite d, du or do would make them NaN, 0 times it), and steps past the
      // end add nothing to dA (an infinite state would, 0 times it): a way of its
      // own, since selects in every chunk cost more (a training pass of 2048 x 8 x
      // 2048 with 16 states 840 us instead of 832; with one lane a channel, where
      // the second way spills more registers, 808 instead of 937).
      float o[I], gB[I], gA[I];
      constexpr bool ENDS = !LOCAL && S > 1;
      const bool usual = (!ENDS || t0 + G <= end) && (!PAD || (all_finite(d, du) && all_finite(go, go)));
#pragma unroll
      for (int way = 0; way < (PAD || ENDS ? 2 : 1); ++way) {
        const bool GUARD = way == 1;
        if ((PAD || ENDS) && usual == GUARD) continue;
        if (GUARD)
#pragma unroll
          for (int i = 0; i < I; ++i) asm volatile("" : "+v"(d[i]), "+v"(du[i]), "+v"(go[i]));
        if constexpr (LOCAL) {
#pragma unroll
          for (int s = G - 1; s >= 0; --s) {
            const float ds = from_lane<Q>(d[s / Q], s % Q), gs = from_lane<Q>(go[s / Q], s % Q);
            float C[R];
            lds_get(bcs + s * 2 * NP + NP, C);
#pragma unroll
            for (int r = 0; r < R; ++r) {
              e[r] = __builtin_amdgcn_exp2f(ds * (A[r] * kLog2e)) * fmaf(C[r], gs, e[r]);
              if (GUARD && r >= left) e[r] = 0.f;
            }
          }
          continue;
        }
        // forwards: the exponentials, the state before every step, what the gate multiplied
        float a[G][R], hb[G][R];
#pragma unroll
        for (int i = 0; i < I; ++i) {
          float part[Q];
#pragma unroll
          for (int l = 0; l < Q; ++l) {
            const int s = i * Q + l;
            const float ds = from_lane<Q>(d[i], l), dus = from_lane<Q>(du[i], l);
            float B[R], C[R];
            lds_get(bcs + s * 2 * NP, B);
            lds_get(bcs + s * 2 * NP + NP, C);
            part[l] = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              a[s][r] = __builtin_amdgcn_exp2f(ds * (A[r] * kLog2e));
              hb[s][r] = h[r];
              h[r] = fmaf(a[s][r], h[r], dus * B[r]);
              if (GUARD && r >= left) a[s][r] = h[r] = 0.f;
              part[l] = fmaf(C[r], h[r], part[l]);
            }
          }
          o[i] = sum_to_lane<S, Q>(part);
          o[i] = fmaf(D, masked(u[i], skip), o[i]);
        }
        // backwards
        float (*const to)[2][NP] = sums[LOCAL ? 0 : t0 / G & 1][wave];
        float v[2][2][R];
#pragma unroll
        for (int i = I - 1; i >= 0; --i) {
          float pB[Q], pA[Q];
#pragma unroll
          for (int l = Q - 1; l >= 0; --l) {
            const int s = i * Q + l;
            const float ds = from_lane<Q>(d[i], l), dus = from_lane<Q>(du[i], l), gs = from_lane<Q>(go[i], l);
            float B[R], C[R];
            lds_get(bcs + s * 2 * NP, B);
            lds_get(bcs + s * 2 * NP + NP, C);
            pB[l] = pA[l] = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float g = GUARD && r >= left ? 0.f : fmaf(C[r], gs, e[r]);
              v[s & 1][0][r] = g * dus;
              v[s & 1][1][r] = gs * (s == G - 1 ? h[r] : hb[s == G - 1 ? s : s + 1][r]);
              pB[l] = fmaf(g, B[r], pB[l]);
              e[r] = g * a[s][r];
              const float x = e[r] * hb[s][r];
              pA[l] = fmaf(x, A[r], pA[l]);
              dA[r] = (ENDS && !GUARD) || t0 + s < end ? fmaf(x, ds, dA[r]) : dA[r];
            }
            if (s & 1) continue;
            // two steps' dB and dC: [2][2][R] values
            constexpr int V = 4 * R;
            float f[V];
#pragma unroll
            for (int x = 0; x < V; ++x) f[x] = v[x / (2 * R)][x / R % 2][x % R];
            sum_channels<S, 32, V>(f);
            if (has_sums<S, V>(lane))
#pragma unroll
              for (int x = 0; x < sums_left<S, V>(); ++x) {
                const int y = first_sum<S, V>(lane) + x;
                to[s + y / (2 * R)][y / R % 2][q.n + y % R] = f[x];
              }
          }
          gB[i] = sum_to_lane<S, Q>(pB);
          gA[i] = sum_to_lane<S, Q>(pA);
        }
      }
      if constexpr (LOCAL) continue;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const float dd = slope[i] * fmaf(u[i], gB[i], gA[i]);
        const bool on = t0 + i * Q + q.j < end;
        dD = fmaf(go[i], u[i], dD);
        dbias += on ? dd : 0.f;
        rows[0][i] = on ? fmaf(D, masked(go[i], skip), d[i] * gB[i]) : 0.f;
        rows[1][i] = on ? dd : 0.f;
        rows[2][i] = on ? o[i] * gz[i] : 0.f;
      }
    }
  if (!LOCAL && begin < end) flush(begin);
  if constexpr (LOCAL) {
    if (!q.live) return;
    const long long m = (long long)q.seg * p.B * p.E + at;
    store_states(p.seg_q + m * NP + q.n, R, e);
    total = sum_channel<1, Q>(total);
    if (q.owner && q.j == 0) p.seg_d[m] = total;
    return;
  }
  if (out.groups == 1) {               // the steps past the row's length
    for (long long x = threadIdx.x; x < (long long)(stop - max(begin, end)) * 2 * p.N; x += 64 * W) {
      const int n = (int)(x % p.N), c = (int)(x / p.N % 2);
      const long long row = (max(begin, end) + x / (2 * p.N)) * p.B + q.b;
      if (c ? p.dCm : p.dBm) el_store<BF>((El<BF>*)(c ? p.dCm : p.dBm) + row * (c ? p.lddC : p.lddB) + q.g * p.N + n, 0.f);
    }
  }
  dD = sum_channel<1, Q>(dD);
  dbias = sum_channel<1, Q>(dbias);
  if (!q.live) return;
  if (p.dh0 && q.seg == 0) store_states(p.dh0 + at * p.N + q.n, left, e);
  const long long m = (long long)q.seg * p.B * p.E + at;
  store_states(out.A + m * NP + q.n, R, dA);
  if (q.owner && q.j == 0) {
    out.D[m] = dD;
    out.bias[m] = dbias;
  }
}

// dB and dC: the workgroups' sums
template <bool BF>
__global__ __launch_bounds__(256) void channels_kernel(const SsmParams p, const Parts in, int NP) {
  const long long all = (long long)p.T * p.B * p.G * 2 * NP;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const int n = (int)(i % NP), c = (int)(i / NP % 2), g = (int)(i / (2 * NP) % p.G);
    const long long row = i / (2LL * NP * p.G);
    void* to = c ? p.dCm : p.dBm;
    if (n >= p.N || !to) continue;
    const int b = (int)(row % p.B), len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    float s = 0.f;
    if (row / p.B < len)
      for (int x = 0; x < in.groups; ++x) s += in.bc[x * all + i];
    el_store<BF>((El<BF>*)to + row * (c ? p.lddC : p.lddB) + g * p.N + n, s);
  }
}

// dA, dD, ddelta_bias: the sums over rows and segments; 64 values a workgroup, every fourth row a wave
__global__ __launch_bounds__(256) void rows_kernel(const SsmParams p, const Parts in, int NP) {
  __shared__ float lds[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, per = NP + 2;
  const long long i = (long long)blockIdx.x * 64 + lane;
  const int e = (int)(i / per), n = (int)(i % per), rows = p.segs * p.B;
  float s = 0.f;
  if (e < p.E) {
    const float* from = n < NP ? in.A + (long long)e * NP + n : (n == NP ? in.D : in.bias) + e;
    const long long step = (long long)p.E * (n < NP ? NP : 1);
#pragma unroll 4
    for (int b = wave; b < rows; b += 4) s += from[b * step];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave || e >= p.E) return;
  s = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
  if (n < p.N) {
    if (p.dA) p.dA[(long long)e * p.N + n] = s;
  } else if (n == NP) {
    if (p.dD) p.dD[e] = s;
  } else if (n == NP + 1) {
    if (p.ddelta_bias) p.ddelta_bias[e] = s;
  }
}

template <bool BF, int S, bool PAD>
hipError_t start(const SsmParams& p, hipStream_t s) {
  constexpr int NP = S * kSsmPer;
  const int groups = ssm_groups(p, S);   // 0: no channels
  const Parts parts = parts_of(p, groups, NP);
  const unsigned tiles = (unsigned)groups * p.G * p.B;
  const dim3 block(64 * kSsmTiles);
  if (tiles > 0) {
    if (p.segs > 1) hipLaunchKernelGGL((bwd_kernel<BF, S, true, PAD>), dim3(tiles * (p.segs - 1) * p.sub), block, 0, s, p, parts);
    hipLaunchKernelGGL((bwd_kernel<BF, S, false, PAD>), dim3(tiles * p.segs), block, 0, s, p, parts);
  }
  const long long all = (long long)p.T * p.B * p.G * 2 * NP;
  if ((p.dBm || p.dCm) && all && groups != 1)
    hipLaunchKernelGGL(channels_kernel<BF>, dim3((unsigned)std::min<long long>((all + 255) / 256, 1 << 20)), dim3(256), 0, s, p, parts, NP);
  if (p.E > 0 && (p.dA || p.dD || p.ddelta_bias))
    hipLaunchKernelGGL(rows_kernel, dim3((unsigned)(((long long)p.E * (NP + 2) + 63) / 64)), dim3(256), 0, s, p, parts, NP);
  return hipGetLastError();
}

template <bool BF, int S>
hipError_t start(const SsmParams& p, hipStream_t s) {
  return p.N < S * kSsmPer ? start<BF, S, true>(p, s) : start<BF, S, false>(p, s);
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

hipError_t rnn_launch_ssm_bwd(const SsmParams& p, int bf16, hipStream_t s) {
  return bf16 ? launch<true>(p, s) : launch<false>(p, s);
}
