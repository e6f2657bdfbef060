// Parameters and launchers of the operators of a state-space block:
// normalisation, causal convolution, selective state-space scan
// (include/rnn.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lm_math.h"

namespace rnnk {

struct NormParams {
  int M, D, rms;
  float eps;
  const void* x;         // backward: what was normalised
  const void* residual;  // or null
  const float* weight;   // or null
  const float* bias;     // or null
  void* y;
  void* total;           // or null
  float* stats;          // [M, 2]; forward: or null
  const void* dy;        // backward, as what follows
  const void* dtotal;    // or null
  void* dx;              // or null
  float* dweight;        // or null
  float* dbias;          // or null
  float* part;           // [parts][2][D], without dbias [parts][1][D]
  int parts;
};
int norm_parts(int M, int D);   // rows of partial sums of the parameters' gradients

constexpr int kConvMost = 8;    // widest convolution
struct ConvParams {
  int T, B, C, K, silu;
  int piece, pieces;     // steps of a wave, pieces of the time axis
  const void* x;
  long long ldx;
  const float* w;
  const float* bias;     // or null
  const void* s0;        // or null
  const int* lengths;    // or null
  void* y;
  long long ldy;
  void* sy;              // or null
  const void* dy;        // backward, as what follows
  long long lddy;
  const void* dsy;       // or null
  void* dx;              // or null
  long long lddx;
  float* dw;             // or null
  float* dbias;          // or null
  void* ds0;             // or null
  float* part;           // [B * groups of pieces][K + 1][C]
};
constexpr int kConvWaves = 4;   // consecutive pieces of a workgroup
int conv_piece(int T, int B, int C, bool back);
long long conv_blocks(int T, int B, int C, bool back);   // workgroups of a launch
long long conv_parts(int T, int B, int C);               // rows of partial sums that a workspace has room for

constexpr int kSsmStates = 64;  // most states of a channel
struct SsmParams {
  int T, B, E, N, G, softplus;
  const void *u, *delta, *z, *Bm, *Cm;
  long long ldu, lddelta, ldz, ldB, ldC;
  const float *A, *D, *delta_bias, *h0;
  const int* lengths;
  void* y;
  long long ldy;
  float* hy;
  float* starts;         // the state before every chunk of steps, or null
  // segments of the time axis, the parts of a segment that backward's first
  // launch walks, a segment's steps (whole chunks in each part); with more than
  // one segment: the state that the first one starts from, the segments' or
  // parts' maps
  int segs, sub, seg_steps;
  float* seg_first;      // [B][E][NP]
  float* seg_q;          // [segs (* sub)][B][E][NP]
  float* seg_d;          // [segs (* sub)][B][E]
  const void* dy;        // backward, as what follows
  long long lddy;
  const float* dhy;
  void *du, *ddelta, *dz, *dBm, *dCm;
  long long lddu, ldddelta, lddz, lddB, lddC;
  float *dA, *dD, *ddelta_bias, *dh0;
  float* part;           // workspace of the backward pass
};
// A call's segments (forward's or backward's) and the parts of the workspace, in floats
struct SsmPlan {
  int segs[2], seg_steps[2], sub;
  size_t starts, first, q, d, part, all;   // offsets; all: the size
};
long long ssm_blocks(int B, int E, int N, int G);   // workgroups of a segment
SsmPlan ssm_plan(int T, int B, int E, int N, int G, bool save);

// 16 bytes of a row at any alignment
template <bool BF>
constexpr int piece_width() { return BF ? 8 : 4; }

// VW neighbouring elements (VW * size: 8 or 16 bytes) as they are in memory;
// those from `left` on are not there and read as 0.  (Unpacked where they are
// used: a conversion next to the load would wait for it, and the loads would
// come one after the other.)
template <bool BF, int VW>
using RawPiece = Bytes<VW*(BF ? 2 : 4)>;
template <bool BF, int VW>
__device__ __forceinline__ RawPiece<BF, VW> load_raw(const El<BF>* p, int left) {
  RawPiece<BF, VW> w = {};
  if (left >= VW) {
    w = *reinterpret_cast<const RawPiece<BF, VW>*>(p);
  } else {
#pragma unroll
    for (int j = 0; j < VW - 1; ++j)
      if (j < left) {
        if constexpr (BF) w.w[j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
        else w.w[j] = __float_as_uint(p[j]);
      }
  }
  return w;
}
template <bool BF, int VW>
__device__ __forceinline__ void unpack(const RawPiece<BF, VW>& w, float (&o)[VW]) {
  if constexpr (BF) {
#pragma unroll
    for (int j = 0; j < VW / 2; ++j) {
      o[2 * j] = __uint_as_float(w.w[j] << 16);
      o[2 * j + 1] = __uint_as_float(w.w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < VW; ++j) o[j] = __uint_as_float(w.w[j]);
  }
}
template <bool BF, int VW>
__device__ __forceinline__ void load_piece(const El<BF>* p, int left, float (&o)[VW]) {
  unpack<BF, VW>(load_raw<BF, VW>(p, left), o);
}
template <bool BF, int VW>
__device__ __forceinline__ void store_piece(El<BF>* p, int left, const float (&v)[VW]) {
  if (left >= VW) {
    constexpr int ES = BF ? 2 : 4;
    Bytes<VW * ES> w;
    if constexpr (BF) {
#pragma unroll
      for (int j = 0; j < VW / 2; ++j) w.w[j] = pack2bf(v[2 * j], v[2 * j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < VW; ++j) w.w[j] = __float_as_uint(v[j]);
    }
    *reinterpret_cast<Bytes<VW * ES>*>(p) = w;
  } else {
#pragma unroll
    for (int j = 0; j < VW; ++j)
      if (j < left) el_store<BF>(p + j, v[j]);
  }
}

// v of the lane whose index differs in bit M, for M = 1, 2, 4, 8
template <int M>
__device__ __forceinline__ float lane_xor(float v) {
  const int i = __float_as_int(v);
  if constexpr (M == 1) return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0xb1, 0xf, 0xf, true));        // quad_perm 1,0,3,2
  else if constexpr (M == 2) return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x4e, 0xf, 0xf, true));   // quad_perm 2,3,0,1
  else if constexpr (M == 4) return __int_as_float(__builtin_amdgcn_ds_swizzle(i, 0x1f | 4 << 10));
  else return __int_as_float(__builtin_amdgcn_update_dpp(i, i, 0x128, 0xf, 0xf, true));                        // row_ror:8
}

// Lanes with bit M clear: v0 of both lanes of the pair, added; the others: v1.
template <int M>
__device__ __forceinline__ float fold(float v0, float v1) {
  if constexpr (M >= 16) {
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    const unsigned a = __float_as_uint(v0), b = __float_as_uint(v1);
    u2 r;
    if constexpr (M == 32) r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    else r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
  } else {
    const bool up = threadIdx.x & M;
    return (up ? v1 : v0) + lane_xor<M>(up ? v0 : v1);
  }
}

// the sum over the lanes whose indexes differ in the bits FROM .. 32, in all of them
template <int FROM>
__device__ __forceinline__ float sum_lanes(float v) {
  if constexpr (FROM <= 32) v = fold<32>(v, v);
  if constexpr (FROM <= 16) v = fold<16>(v, v);
  if constexpr (FROM <= 8) v += lane_xor<8>(v);
  if constexpr (FROM <= 4) v += lane_xor<4>(v);
  if constexpr (FROM <= 2) v += lane_xor<2>(v);
  if constexpr (FROM <= 1) v += lane_xor<1>(v);
  return v;
}

// Workgroups (of up to 1024 threads) in two dimensions, the last row of them partly
// past the end: a launch has fewer than 2^32 threads in a dimension.
inline dim3 wide_grid(long long blocks) {
  const long long x = blocks < (1LL << 21) ? blocks : 1LL << 21;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}

// Column i of `rows` rows of n partial sums: a workgroup of 16 waves takes 64
// columns, every 16th row a wave; the sum is the first wave's.
constexpr int kSumWaves = 16;
__device__ __forceinline__ float column_sum(const float* part, long long n, long long i, int rows, float (*lds)[64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float s = 0.f;
  if (i < n)
#pragma unroll 8
    for (int r = wave; r < rows; r += kSumWaves) s += part[r * n + i];
  lds[wave][lane] = s;
  __syncthreads();
  s = 0.f;
  if (wave == 0)
#pragma unroll
    for (int w = 0; w < kSumWaves; ++w) s += lds[w][lane];
  return s;
}

}  // namespace rnnk

hipError_t rnn_launch_norm_fwd(const rnnk::NormParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_norm_bwd(const rnnk::NormParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_conv_fwd(const rnnk::ConvParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_conv_bwd(const rnnk::ConvParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_conv_step(const rnnk::ConvParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_ssm_step(const rnnk::SsmParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_ssm_fwd(const rnnk::SsmParams& p, int bf16, hipStream_t s);
hipError_t rnn_launch_ssm_bwd(const rnnk::SsmParams& p, int bf16, hipStream_t s);
