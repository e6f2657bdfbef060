// What the passes of the selective state-space scan share (gfx950): lanes and
// states, the step d, sums and broadcasts among the lanes of a channel, the
// segments of the time axis.
//
// A channel's N states are held by S neighbouring lanes, R = 4 states each (N
// <= 4 S = NP); a wave holds 64 / S neighbouring channels of one row and group
// (a tile) and walks their steps in chunks of G.  Of a chunk a lane also owns
// every Q-th step, Q = min(S, 4): it loads u, delta, z of those and computes
// what depends on a channel and a step alone, once for Q lanes.  B and C of a
// chunk lie in the wave's own part of the LDS.
//
// Where the tiles are too few to fill the device the time axis is cut into
// segments.  A first launch walks each from a state of zero: the segment's
// steps compose to h -> P h + Q with P = exp(A sum d).  P is kept as sum d and
// applied as its square root, twice: it carries a state through a decay of up
// to 2^-252 without loss.
#pragma once

#include "ssm_common.h"

namespace rnnk {

constexpr float kLog2e = 1.4426950408889634f;

// Steps of a chunk.  Backward's hold the exponentials and states of all their
// steps in registers, and forward keeps the state before each of them.
constexpr int ssm_chunk(int S) { return S == 1 ? 8 : 16; }
constexpr int kSsmKeep = 8;
constexpr int kSsmPer = 4;      // states of a lane
constexpr int kSsmTiles = 4;    // neighbouring tiles of a workgroup, a wave each
// lanes of a channel with N states
inline int ssm_lanes(int N) {
  int S = 1;
  while (S * kSsmPer < N) S *= 2;
  return S;
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|); log1p(e) = 2 atanh(s) with
// s = e / (2 + e) <= 1/3, whose series through s^13 is within 2^-25 of it.
__device__ __forceinline__ float softplus(float x) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e), z = s * s;
  float r = fmaf(z, 1.f / 13.f, 1.f / 11.f);
  r = fmaf(z, r, 1.f / 9.f);
  r = fmaf(z, r, 1.f / 7.f);
  r = fmaf(z, r, 1.f / 5.f);
  r = fmaf(z, r, 1.f / 3.f);
  r = fmaf(z, r, 1.f);
  return fmaxf(x, 0.f) + 2.f * s * r;
}

// v of the k-th of a quad's (or pair's) Q lanes, in all of them
template <int Q>
__device__ __forceinline__ float from_lane(float v, int k) {
  const int i = __float_as_int(v);
  if constexpr (Q == 1) {
    return v;
  } else if constexpr (Q == 2) {
    return __int_as_float(k ? __builtin_amdgcn_update_dpp(i, i, 0xf5, 0xf, 0xf, true) : __builtin_amdgcn_update_dpp(i, i, 0xa0, 0xf, 0xf, true));
  } else {
    return __int_as_float(k == 0   ? __builtin_amdgcn_update_dpp(i, i, 0x00, 0xf, 0xf, true)
                          : k == 1 ? __builtin_amdgcn_update_dpp(i, i, 0x55, 0xf, 0xf, true)
                          : k == 2 ? __builtin_amdgcn_update_dpp(i, i, 0xaa, 0xf, 0xf, true)
                                   : __builtin_amdgcn_update_dpp(i, i, 0xff, 0xf, 0xf, true));
  }
}

// the sum over the lanes FROM, FROM + 1, ... of a channel's S (FROM, S powers of two), in all of them
template <int FROM, int S>
__device__ __forceinline__ float sum_channel(float v) {
  if constexpr (FROM <= 1 && S >= 2) v += lane_xor<1>(v);
  if constexpr (FROM <= 2 && S >= 4) v += lane_xor<2>(v);
  if constexpr (FROM <= 4 && S >= 8) v += lane_xor<4>(v);
  if constexpr (FROM <= 8 && S >= 16) v += lane_xor<8>(v);
  return v;
}

// v[k] summed over a channel's S lanes, in the lanes whose index is k modulo Q
template <int S, int Q>
__device__ __forceinline__ float sum_to_lane(float (&v)[Q]) {
  if constexpr (Q == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = fold<2>(v[i], v[i + 2]);
  }
  if constexpr (Q >= 2) v[0] = fold<1>(v[0], v[1]);
  return sum_channel<4, S>(v[0]);
}

// v or, where the mask is 0, 0
__device__ __forceinline__ float masked(float v, uint32_t mask) { return __uint_as_float(__float_as_uint(v) & mask); }

// whether all lanes' values are finite
template <int I>
__device__ __forceinline__ bool all_finite(const float (&v)[I], const float (&w)[I]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i) s = fmaf(0.f, w[i], fmaf(0.f, v[i], s));
  return !__any(s != 0.f);               // an infinity or NaN times 0 is NaN
}

// a lane's states, `left` of which are there
__device__ __forceinline__ void load_states(const float* p, int left, float (&v)[kSsmPer]) { load_piece<false, kSsmPer>(p, left, v); }
__device__ __forceinline__ void store_states(float* p, int left, const float (&v)[kSsmPer]) { store_piece<false, kSsmPer>(p, left, v); }

// as many values of LDS
__device__ __forceinline__ void lds_get(const float* p, float (&v)[kSsmPer]) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}

// The tile of a wave and a lane's place in it.
struct SsmPlace {
  int b, g, seg, group;  // row, group, segment, workgroup's tiles in the group
  int e, j, n;           // channel, the lane's own step of Q, its first state
  bool live, owner;      // the channel is there; and this lane writes its steps
  int len;               // the row's steps
};
// workgroups of a group's tiles
__host__ __device__ inline int ssm_groups(int E, int G, int S) {
  const int channels = 64 / S * kSsmTiles;
  return (E / G + channels - 1) / channels;
}
__host__ __device__ inline int ssm_groups(const SsmParams& p, int S) { return ssm_groups(p.E, p.G, S); }
template <int S>
__device__ __forceinline__ SsmPlace ssm_place(const SsmParams& p, unsigned at, int wave) {
  constexpr int CH = 64 / S, Q = S < 4 ? S : 4;
  const unsigned per = p.E / p.G, groups = ssm_groups(p, S), lane = threadIdx.x & 63;
  SsmPlace q;
  q.group = at % groups;
  at /= groups;
  q.g = at % p.G;
  at /= p.G;
  q.b = at % p.B;
  q.seg = at / p.B;
  const unsigned c = (q.group * kSsmTiles + wave) * CH + lane / S;
  q.live = c < per;
  q.owner = q.live && lane % S < Q;
  q.e = q.g * per + (q.live ? c : 0);
  q.j = lane % Q;
  q.n = lane % S * kSsmPer;
  q.len = p.lengths ? min(max(p.lengths[q.b], 0), p.T) : p.T;
  return q;
}

// The rows of a time-major tensor as a wave walks them, chunk after chunk: a
// uniform address and the lane's part of it, of up to three steps and a row, in
// 32 bits (B * ld <= 2^28 over several steps; a single step may lie in rows
// farther apart, and what its lanes own past it is not read).
// (Pointers say that they are to global memory: the compiler does not look
// through the asm statements below for it.)
using GlobalBytes = __attribute__((address_space(1))) char*;
template <bool BF>
using GlobalEl = __attribute__((address_space(1))) El<BF>*;
// What a load brings stays as it is until it is used: were it widened or made a
// float at once, the wave would wait for it there (the forward training pass of
// 2048 x 8 x 2048 in bf16 414 us instead of 240).
struct SsmRows {
  GlobalBytes row;        // of the chunk's first step
  long long hop;          // bytes from one of a lane's own steps to the next
  unsigned own;           // the lane's first step and its channel
};
template <bool BF, int Q>
__device__ __forceinline__ SsmRows ssm_rows(const SsmParams& p, const SsmPlace& q, const void* x, long long ld, int t0) {
  constexpr int ES = BF ? 2 : 4;
  const long long step = p.T > 1 ? p.B * ld * ES : 0;
  SsmRows r;
  r.row = (GlobalBytes)(uintptr_t)x + q.b * ld * ES + t0 * step;
  r.hop = Q * step;
  r.own = (unsigned)(q.j * step) + q.e * ES;
  return r;
}

// The lane's own steps of a chunk, and on to the next chunk (BACK: the one
// before).  `left` steps of the chunk are there (one at least): those past it
// repeat the last.  (The empty asm statements keep the compiler from making
// every address anew from products.)
template <bool BF, int Q, bool BACK, int I>
__device__ __forceinline__ void load_own(SsmRows& r, const SsmPlace& q, int left, El<BF> (&v)[I]) {
  if (left >= I * Q) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      v[i] = *(GlobalEl<BF>)(r.row + r.own);
      r.row += r.hop;
      asm("" : "+s"(r.row));
    }
    if constexpr (BACK) r.row -= 2 * I * r.hop;
  } else {
    const long long step = r.hop / Q;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int back = max(0, i * Q + q.j - (left - 1));
      v[i] = *(GlobalEl<BF>)(r.row + i * r.hop + r.own - back * step);
    }
    r.row += (BACK ? -I : I) * r.hop;
  }
}
template <bool BF, int Q, bool BACK, int I>
__device__ __forceinline__ void store_own(SsmRows& r, const SsmPlace& q, int left, const float (&v)[I]) {
  GlobalBytes row = r.row;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    El<BF> w;
    el_store<BF>(&w, v[i]);
    if (q.owner && i * Q + q.j < left) *(GlobalEl<BF>)(row + r.own) = w;
    row += r.hop;
    asm("" : "+s"(row));
  }
  r.row = BACK ? row - 2 * I * r.hop : row;
}

// B and C of a chunk, four states a piece: lane x of the wave holds the pieces x, x + 64, ... of [G][2][NP / 4]
template <int G, int NP>
constexpr int bc_pieces() { return (G * 2 * (NP / 4) + 63) / 64; }
template <bool BF>
using RawFour = RawPiece<BF, 4>;
template <bool BF, int G, int NP>
__device__ __forceinline__ void load_bc(const SsmParams& p, const SsmPlace& q, int t0, RawFour<BF> (&v)[bc_pieces<G, NP>()]) {
  constexpr int PP = NP / 4;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < bc_pieces<G, NP>(); ++i) {
    const int x = lane + 64 * i, n = x % PP * 4, t = t0 + x / (2 * PP);
    const bool c = x / PP % 2, on = t < q.len && x < G * 2 * PP;
    const long long row = (long long)(on ? t : q.len - 1) * p.B + q.b;
    const El<BF>* from = (const El<BF>*)(c ? p.Cm : p.Bm) + row * (c ? p.ldC : p.ldB) + q.g * p.N + n;
    v[i] = load_raw<BF, 4>(from, on ? p.N - n : 0);
  }
}
template <bool BF, int G, int NP>
__device__ __forceinline__ void put_bc(float* to, const RawFour<BF> (&v)[bc_pieces<G, NP>()]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < bc_pieces<G, NP>(); ++i)
    if (64 * (i + 1) <= G * 2 * (NP / 4) || lane + 64 * i < G * 2 * (NP / 4)) {
      uint4 w;
      if constexpr (BF) w = make_uint4(v[i].w[0] << 16, v[i].w[0] & 0xffff0000u, v[i].w[1] << 16, v[i].w[1] & 0xffff0000u);
      else w = make_uint4(v[i].w[0], v[i].w[1], v[i].w[2], v[i].w[3]);
      *reinterpret_cast<uint4*>(to + (lane + 64 * i) * 4) = w;
    }
}

// a state through a map: P from the sum of d, twice its root (which is held above
// 0, so that an infinite state stays so; of finite ones its square leaves nothing)
__device__ __forceinline__ float through(float A, float sum, float Q, float h) {
  const float P = fmaxf(__builtin_amdgcn_exp2f(fminf(0.5f * kLog2e * A * sum, 127.f)), 0x1p-149f);
  return fmaf(P, P * h, Q);
}

}  // namespace rnnk
