// Selective state-space scan (gfx950), forward and single steps:
//   h_t[n] = exp(d_t A[n]) h_(t-1)[n] + d_t u_t B_t[n],  y_t = (C_t . h_t + D u_t) silu(z_t)
//
// A wave walks the steps of 16 channels (16 states each) one after the other,
// the states in registers.  Bound: vector instructions.  Each step and state
// takes a product, an exponential (half the rate), a product and two fused
// ones, 6 issue slots of the 10 that a pass takes in all.  The memory's time is
// less than half of the pass's (in bf16 8 bytes a step and channel, 16 in
// training with the states kept).  2048 steps of 8 rows of 2048 channels, bf16,
// training: 0.23 ms, 1.7 times the slots' own time (0.137 ms at 2.4 GHz), since
// this is one wave a SIMD, which waits for its own results; cut into 4 segments
// the same walk takes 0.19 ms but the segments' first launch 0.10.  A prompt of
// 8192 steps of 3520 channels (220 waves a segment, 18 segments): 0.11 + 0.15 ms.
//
// Measured against it (the same training pass): the exponentials kept over
// pieces of a block that the waves of a workgroup exchange, so that states are
// walked twice but exponentials computed once, 0.56 ms; 2 states a lane (twice
// the waves) 0.28 where 4 took 0.24.
//
// The last segment composes the maps of all before it, one after the other, each
// with a round trip to memory: 16384 steps of 16 channels (512 segments) take 6 us
// in the first launch and 142 in the second.

#include <algorithm>

#include "ssm_util.h"

using namespace rnnk;

namespace {

template <bool BF, int S>
__global__ __launch_bounds__(64 * kSsmTiles) void step_kernel(const SsmParams p) {
  constexpr int R = kSsmPer;
  const SsmPlace q = ssm_place<S>(p, blockIdx.x, threadIdx.x >> 6);
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
    if (r >= left) h[r] = 0.f;           // not there (an infinite d or du times 0)
    o = fmaf(C[r], h[r], o);
  }
  if (p.hy) store_states(p.hy + st, left, h);
  o = sum_channel<1, S>(o);
  if (q.n) return;
  if (p.D) o = fmaf(D, u, o);            // (an infinite u times 0 would be NaN)
  if (p.z) {
    float a, da;
    act_pair<ACT_SILU>(z, a, da);
    o *= a;
  }
  el_store<BF>((El<BF>*)p.y + q.b * p.ldy + q.e, o);
}

// LOCAL: the segments' maps (but the last one's), no outputs.  PAD: some lanes'
// states are not there.
template <bool BF, int S, bool LOCAL, bool PAD>
__global__ __launch_bounds__(64 * kSsmTiles) void fwd_kernel(const SsmParams p) {
  constexpr int R = kSsmPer, G = ssm_chunk(S), NP = S * R, Q = S < 4 ? S : 4, I = G / Q;
  __shared__ __align__(16) float bc[kSsmTiles][G][2][NP];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const SsmPlace q = ssm_place<S>(p, blockIdx.x, wave);
  if (!__any(q.live)) return;
  const int left = q.live ? p.N - q.n : 0;
  const long long at = (long long)q.b * p.E + q.e;
  float A[R], h[R] = {};
  load_states(p.A + (long long)q.e * p.N + q.n, left, A);
  if (p.segs == 1 || LOCAL) {
    if (p.h0) load_states(p.h0 + at * p.N + q.n, left, h);
    if (LOCAL) {                       // the states may be written over by the last segment
      if (q.seg == 0 && q.live) store_states(p.seg_first + at * NP + q.n, R, h);
#pragma unroll
      for (int r = 0; r < R; ++r) h[r] = 0.f;
    }
  } else {
    load_states(p.seg_first + at * NP + q.n, R, h);
    for (int i = 0; i < q.seg; ++i) {
      float Q[R];
      const long long m = (long long)i * p.B * p.E + at;
      load_states(p.seg_q + m * NP + q.n, R, Q);
      const float sum = p.seg_d[m];
#pragma unroll
      for (int r = 0; r < R; ++r) h[r] = through(A[r], sum, Q[r], h[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) A[r] *= kLog2e;
  const float bias = p.delta_bias ? p.delta_bias[q.e] : 0.f, D = p.D ? p.D[q.e] : 0.f;
  const uint32_t skip = p.D ? ~0u : 0u;  // without D, no product of 0 and what may be infinite
  const int begin = min(q.seg * p.seg_steps, p.T), stop = min(begin + p.seg_steps, p.T), end = min(stop, q.len);
  SsmRows xu = ssm_rows<BF, Q>(p, q, p.u, p.ldu, begin), xd = ssm_rows<BF, Q>(p, q, p.delta, p.lddelta, begin),
          xz = ssm_rows<BF, Q>(p, q, p.z, p.ldz, begin), xy = ssm_rows<BF, Q>(p, q, p.y, p.ldy, begin);
  El<BF> ru[I], rd[I], rz[I] = {};
  RawFour<BF> rbc[bc_pieces<G, NP>()];
  float total = 0.f;
  auto load = [&](int t0) {
    const int left = q.len - t0;
    load_own<BF, Q, false, I>(xu, q, left, ru);
    load_own<BF, Q, false, I>(xd, q, left, rd);
    if (!LOCAL && p.z) load_own<BF, Q, false, I>(xz, q, left, rz);
    load_bc<BF, G, NP>(p, q, t0, rbc);
  };
  if (begin < end) load(begin);
  int t0 = begin;
  float y[I] = {}, mid[R] = {};
  for (; t0 < end; t0 += G) {
    float u[I], d[I], du[I], gate[I];
#pragma unroll
    for (int i = 0; i < I; ++i) d[i] = el_load<BF>(&rd[i]) + bias;
    if (p.softplus)
#pragma unroll
      for (int i = 0; i < I; ++i) d[i] = softplus(d[i]);
#pragma unroll
    for (int i = 0; i < I; ++i) gate[i] = 1.f;
    if (!LOCAL && p.z)
#pragma unroll
      for (int i = 0; i < I; ++i) {
        float slope;
        act_pair<ACT_SILU>(el_load<BF>(&rz[i]), gate[i], slope);
      }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const bool on = t0 + i * Q + q.j < end;
      u[i] = on ? el_load<BF>(&ru[i]) : 0.f;
      d[i] = on ? d[i] : 0.f;
      du[i] = d[i] * u[i];
      total += d[i];
    }
    float* own = &bc[wave][0][0][0];
    put_bc<BF, G, NP>(own, rbc);
    // what this and the last chunk have to store goes before the next loads: a
    // wait for those then has no young stores to wait for
    if constexpr (!LOCAL) {
      if (t0 > begin) store_own<BF, Q, false, I>(xy, q, G, y);
      if (p.starts && q.live) {
        float* to = p.starts + ((long long)(t0 / kSsmKeep) * p.B * p.E + at) * NP + q.n;
        if (G > kSsmKeep && t0 > begin) store_states(to - (long long)p.B * p.E * NP, R, mid);
        store_states(to, R, h);
      }
    }
    if (t0 + G < end) load(t0 + G);
    // B and C of Q steps are read while the Q steps before them are walked (the
    // empty asm statement holds the reads there)
    float B[2][Q][R], C[2][Q][R];
    auto read = [&](int i) {
#pragma unroll
      for (int l = 0; l < Q; ++l) {
        const float* row = own + (i * Q + l) * 2 * NP + q.n;
        lds_get(row, B[i & 1][l]);
        if constexpr (!LOCAL) lds_get(row + NP, C[i & 1][l]);
      }
    };
    read(0);
    // GUARD: states that are not there are held at 0 (an infinite d or du would
    // make them NaN, 0 times it, and through them the sum over the states), in a
    // way of its own: 13 states of the training pass above 0.25 ms instead of 0.27
    // with selects in every chunk.  The empty asm statement keeps the compiler from
    // sharing the ways' values (with what they share computed before the branch
    // 199 registers instead of 144).
    const bool usual = !PAD || all_finite(d, du);
#pragma unroll
    for (int way = 0; way < (PAD ? 2 : 1); ++way) {
      const bool GUARD = way == 1;
      if (PAD && usual == GUARD) continue;
      if (GUARD)
#pragma unroll
        for (int i = 0; i < I; ++i) asm volatile("" : "+v"(d[i]), "+v"(du[i]));
#pragma unroll
      for (int i = 0; i < I; ++i) {
        if (i + 1 < I) read(i + 1);
        if (G > kSsmKeep && i * Q == kSsmKeep)
#pragma unroll
          for (int r = 0; r < R; ++r) mid[r] = h[r];
        asm volatile("" ::: "memory");
        float part[Q];
#pragma unroll
        for (int l = 0; l < Q; ++l) {
          const float ds = from_lane<Q>(d[i], l), dus = from_lane<Q>(du[i], l);
          part[l] = 0.f;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            h[r] = fmaf(__builtin_amdgcn_exp2f(ds * A[r]), h[r], dus * B[i & 1][l][r]);
            if (GUARD && r >= left) h[r] = 0.f;
            if constexpr (!LOCAL) part[l] = fmaf(C[i & 1][l][r], h[r], part[l]);
          }
        }
        if constexpr (!LOCAL) {
          y[i] = fmaf(D, masked(u[i], skip), sum_to_lane<S, Q>(part)) * gate[i];
          if (t0 + i * Q + q.j >= end) y[i] = 0.f;
        }
      }
    }
  }
  if constexpr (LOCAL) {
    if (!q.live) return;
    const long long m = (long long)q.seg * p.B * p.E + at;
    store_states(p.seg_q + m * NP + q.n, R, h);
    total = sum_channel<1, Q>(total);
    if (q.owner && q.j == 0) p.seg_d[m] = total;
  } else {
    const float none[I] = {};
    if (t0 > begin) {
      store_own<BF, Q, false, I>(xy, q, stop - (t0 - G), y);
      if (G > kSsmKeep && p.starts && q.live && t0 - G + kSsmKeep < end)
        store_states(p.starts + ((long long)((t0 - G) / kSsmKeep + 1) * p.B * p.E + at) * NP + q.n, R, mid);
    }
    for (; t0 < stop; t0 += G) store_own<BF, Q, false, I>(xy, q, stop - t0, none);
    if (q.live && p.hy && q.seg == p.segs - 1) store_states(p.hy + at * p.N + q.n, left, h);
  }
}

template <bool BF, int S, bool PAD>
hipError_t start(const SsmParams& p, bool step, hipStream_t s) {
  const unsigned tiles = (unsigned)ssm_blocks(p.B, p.E, p.N, p.G);
  const dim3 block(64 * kSsmTiles);
  if (step) {
    hipLaunchKernelGGL((step_kernel<BF, S>), dim3(tiles), block, 0, s, p);
    return hipGetLastError();
  }
  if (p.segs > 1) hipLaunchKernelGGL((fwd_kernel<BF, S, true, PAD>), dim3(tiles * (p.segs - 1)), block, 0, s, p);
  hipLaunchKernelGGL((fwd_kernel<BF, S, false, PAD>), dim3(tiles * p.segs), block, 0, s, p);
  return hipGetLastError();
}

template <bool BF, int S>
hipError_t start(const SsmParams& p, bool step, hipStream_t s) {
  return p.N < S * kSsmPer ? start<BF, S, true>(p, step, s) : start<BF, S, false>(p, step, s);
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

// Segments of a pass with `tiles` waves a segment: as many as fill the device
// (forward with 4 waves a SIMD: 264 us for the prompt above, 281 with 2; backward
// with 2, what its registers allow: 0.72 ms for 1024 waves, 0.87 in one segment),
// of 32 steps at least.  Forward one from 800 waves on: the first launch then
// costs more than the waiting of few waves (0.25 against 0.29 ms with 1024).
static int segments(long long tiles, int T, bool back) {
  if (tiles == 0 || (!back && tiles >= 800)) return 1;
  return (int)std::max(1LL, std::min<long long>((back ? 2048 : 4096) / tiles, T / 32));
}

long long rnnk::ssm_blocks(int B, int E, int N, int G) { return (long long)ssm_groups(E, G, ssm_lanes(N)) * G * B; }

SsmPlan rnnk::ssm_plan(int T, int B, int E, int N, int G, bool save) {
  SsmPlan r{};
  const int S = ssm_lanes(N), CH = 64 / S, step = ssm_chunk(S), NP = S * kSsmPer;
  const long long row = (long long)(E / G + CH - 1) / CH * G, tiles = row * B;   // waves of a row, of a segment
  for (int back = 0; back < (save ? 2 : 1); ++back) {
    const int n = segments(tiles, T, back);
    // backward's first launch holds less in a wave: it cuts the segments into parts
    // until it has 2048 waves or more (1024 waves 110 -> 84 us)
    int sub = 1;
    while (back && n > 1 && tiles * (n - 1) * sub < 2048 && T / (n * sub) >= 64) sub *= 2;
    const int whole = step * sub;
    if (back) r.sub = sub;
    r.seg_steps[back] = std::max(whole, ((T + n - 1) / n + whole - 1) / whole * whole);
    r.segs[back] = std::max(1, (T + r.seg_steps[back] - 1) / r.seg_steps[back]);
  }
  // The sizes follow from bounds of the above that do not fall with more steps or
  // rows, so that a workspace does for fewer of both: there are several segments
  // with up to 1024 waves a segment and 64 steps or more; n B <= 4096 / row
  // forward, 2048 / row backward, and n sub B <= 8192 / row (the last doubling
  // found less than 2048 waves in n - 1 segments), all at most B T / 32.
  auto most = [&](long long waves) { return row ? std::min(waves / row, (long long)B * (T / 32)) : 0; };
  const size_t C = (size_t)B * E;
  size_t o = 0;
  auto take = [&o](size_t floats) {
    const size_t at = o;
    o += (floats + 63) & ~(size_t)63;
    return at;
  };
  if (save) r.starts = take(((size_t)T + kSsmKeep - 1) / kSsmKeep * C * NP);
  if (row > 0 && row <= 1024 && T >= 64) {
    const size_t maps = most(save ? 8192 : 4096) * (size_t)E;
    r.first = take(std::min<size_t>(B, 1024 / row) * E * NP);
    r.q = take(maps * NP);
    r.d = take(maps);
  }
  if (save) {
    const size_t groups = ssm_groups(E, G, S);
    r.part = take((groups > 1 ? groups * T * B * G * 2 * NP : 0) + std::max((size_t)B, (size_t)most(2048)) * E * (NP + 2));
  }
  r.all = o;
  return r;
}

hipError_t rnn_launch_ssm_step(const SsmParams& p, int bf16, hipStream_t s) {
  return bf16 ? launch<true>(p, true, s) : launch<false>(p, true, s);
}
hipError_t rnn_launch_ssm_fwd(const SsmParams& p, int bf16, hipStream_t s) {
  return bf16 ? launch<true>(p, false, s) : launch<false>(p, false, s);
}
