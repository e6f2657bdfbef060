// What the passes of the selective state-space scan share (gfx950): lanes and
// states, the step d, sums and broadcasts among the lanes of a channel.
//
// A channel's states are held by S neighbouring lanes, kSsmPer states each; a
// wave holds 64 / S neighbouring channels of one row and group.  A lane also owns
// every S-th step of its wave's piece: it loads u, delta, z of those and
// computes what depends on a channel and a step alone, once for all S lanes.
#pragma once

#include "ssm_common.h"

namespace rnnk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSsmBlock = 64;   // steps between two saved states

constexpr int kSsmPer = 4;      // states of a lane

// lanes of a channel with N states: 1, 2, 4, 8 or 16
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

// v of the k-th of a channel's S lanes, in all of them
template <int S>
__device__ __forceinline__ float from_lane(float v, int k) {
  const int i = __float_as_int(v);
  if constexpr (S == 1) {
    return v;
  } else if constexpr (S == 2) {
    return __int_as_float(k ? __builtin_amdgcn_update_dpp(i, i, 0xf5, 0xf, 0xf, true) : __builtin_amdgcn_update_dpp(i, i, 0xa0, 0xf, 0xf, true));
  } else if constexpr (S == 4) {
    return __int_as_float(k == 0   ? __builtin_amdgcn_update_dpp(i, i, 0x00, 0xf, 0xf, true)
                          : k == 1 ? __builtin_amdgcn_update_dpp(i, i, 0x55, 0xf, 0xf, true)
                          : k == 2 ? __builtin_amdgcn_update_dpp(i, i, 0xaa, 0xf, 0xf, true)
                                   : __builtin_amdgcn_update_dpp(i, i, 0xff, 0xf, 0xf, true));
  } else if constexpr (S == 16) {
    switch (k) {                                  // row_newbcast
#define ROW_LANE(K) case K: return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x150 + K, 0xf, 0xf, true));
      ROW_LANE(0) ROW_LANE(1) ROW_LANE(2) ROW_LANE(3) ROW_LANE(4) ROW_LANE(5) ROW_LANE(6) ROW_LANE(7)
      ROW_LANE(8) ROW_LANE(9) ROW_LANE(10) ROW_LANE(11) ROW_LANE(12) ROW_LANE(13) ROW_LANE(14)
      default: return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x15f, 0xf, 0xf, true));
#undef ROW_LANE
    }
  } else {
    switch (k) {
      case 0: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18));
      case 1: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 1 << 5));
      case 2: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 2 << 5));
      case 3: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 3 << 5));
      case 4: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 4 << 5));
      case 5: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 5 << 5));
      case 6: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 6 << 5));
      default: return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x18 | 7 << 5));
    }
  }
}

// the sum over a channel's S lanes, in all of them
template <int S>
__device__ __forceinline__ float sum_channel(float v) {
  if constexpr (S >= 2) v += lane_xor<1>(v);
  if constexpr (S >= 4) v += lane_xor<2>(v);
  if constexpr (S >= 8) v += lane_xor<4>(v);
  if constexpr (S >= 16) v += lane_xor<8>(v);
  return v;
}

// v[k] summed over a channel's S lanes, in its k-th lane
template <int S>
__device__ __forceinline__ float sum_to_lane(float (&v)[S]) {
  if constexpr (S >= 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fold<8>(v[i], v[i + 8]);
  }
  if constexpr (S >= 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fold<4>(v[i], v[i + 4]);
  }
  if constexpr (S >= 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = fold<2>(v[i], v[i + 2]);
  }
  if constexpr (S >= 2) v[0] = fold<1>(v[0], v[1]);
  return v[0];
}

// a lane's states, `left` of which are there
__device__ __forceinline__ void load_states(const float* p, int left, float (&v)[kSsmPer]) { load_piece<false, 4>(p, left, v); }
__device__ __forceinline__ void store_states(float* p, int left, const float (&v)[kSsmPer]) { store_piece<false, 4>(p, left, v); }

// as many values of LDS
__device__ __forceinline__ void lds_get(const float* p, float (&v)[kSsmPer]) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void lds_put(float* p, const float (&v)[kSsmPer]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// The channels of a workgroup (or wave) and a lane's place among them.
struct SsmPlace {
  int b, g, tile;        // row, group, tile of 64 / S channels in the group
  int e, j, n;           // channel, lane of the channel, its first state
  bool live;             // the channel is there
  int len;               // the row's steps
};
template <int S>
__device__ __forceinline__ SsmPlace ssm_place(const SsmParams& p, int at) {
  constexpr int CH = 64 / S;
  const int per = p.E / p.G, tiles = (per + CH - 1) / CH, lane = threadIdx.x & 63;
  SsmPlace q;
  q.tile = at % tiles;
  at /= tiles;
  q.g = at % p.G;
  q.b = at / p.G;
  const int c = q.tile * CH + lane / S;
  q.live = c < per;
  q.e = q.g * per + (q.live ? c : 0);
  q.j = lane % S;
  q.n = q.j * kSsmPer;
  q.len = p.lengths ? min(max(p.lengths[q.b], 0), p.T) : p.T;
  return q;
}

}  // namespace rnnk
