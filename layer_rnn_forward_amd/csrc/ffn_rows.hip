// Feed-forward block of a few rows (gfx950): tokens that are generated.
//
//   GLU:  h[m, f] = act(sum_k x[m, k] Wg[f, k]) * (sum_k x[m, k] Wu[f, k])
//   else: y[m, n] = sum_k h[m, k] W[n, k]
//
// Bound by reading the weights once.  A workgroup owns 16 weight rows (8 for up
// to 8 rows of x; GLU: of each half); its waves split k and a wave asks for all of several 64 byte
// pieces of its 16 rows at once, straight into the registers that the MFMA
// takes them from, at whatever alignment the rows have (the tile product needs
// padded copies of ragged rows, which would move the weights twice more).  The
// rows of x are the MFMA's other operand, 16 at a time; rows past M repeat the
// last one and are not stored.  The waves' sums meet in LDS and are added in
// the waves' order.
//
// In bf16 the gated product is passed on as two bf16 numbers, its rounding and
// the rest (16 bits together): the second product then adds nothing to the
// output's own rounding, at the cost of matrix instructions that the weights'
// way here hides.
//
// One row, D 2048, F 8192 in bf16: 13.0 us for the gated product (5.2 TB/s of
// weights) and 8.0 us for the second (4.2 TB/s); with 16 weight rows a
// workgroup 13.7 and 13.5 us, half or twice the waves 14.0 and 15.1 us (gated),
// the 128 x 128 tile product 24 and 77 us.
#include <algorithm>

#include "lm_math.h"

using namespace rnnk;

namespace {

constexpr int kWaves = 8;

// MB: blocks of 16 rows of x.  PAIR (8 rows of x at most): 8 weight rows, and
// of each two pieces side by side: in both operands the slots 8 .. 15 hold the
// second piece's k, so the sums are those of slots (r, m) and (r + 8, m + 8),
// and the other half of the MFMA's result is not used.  Twice the workgroups,
// and runs of 128 bytes.
template <bool BF, bool GLU, int MB, bool PAIR>
__global__ __launch_bounds__(64 * kWaves) void rows_kernel(const FfnRows p) {
  constexpr int ES = BF ? 2 : 4, NT = GLU ? 2 : 1, XB = BF && !GLU ? 2 * MB : MB;   // MB blocks, then their rests
  constexpr int NB = 24 / (NT + XB);   // pieces in flight: 96 registers
  __shared__ f32x4 part[kWaves][NT * MB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
  constexpr int ROWS = PAIR ? 8 : 16, PIECE = PAIR ? 128 : 64;
  const int r0 = blockIdx.x * ROWS, i = lane & (ROWS - 1), q = lane >> 4;
  const int off = PAIR ? (lane >> 3 & 1) * 64 + q * 16 : q * 16;   // of the lane's 16 bytes in a piece
  const char* wp[NT];
  const char* xp[XB];
#pragma unroll
  for (int t = 0; t < NT; ++t) wp[t] = (const char*)p.w + ((long long)t * p.R + min(r0 + i, p.R - 1)) * p.K * ES + off;
#pragma unroll
  for (int b = 0; b < XB; ++b)
    xp[b] = (const char*)p.x + (min(b % MB * 16 + i, p.M - 1) + (long long)(b / MB) * p.M) * p.ldx * ES + off;
  const int bytes = p.K * ES, pieces = (bytes + PIECE - 1) / PIECE, whole = bytes / PIECE;
  const int per = (pieces + W - 1) / W, c1 = min(pieces, (wave + 1) * per);
  int c = wave * per;

  f32x4 acc[NT][MB];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto load = [](const char* at) {
    const auto v = *reinterpret_cast<const Bytes<16>*>(at);
    return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  };
  auto several = [&](auto count) {
    constexpr int N = decltype(count)::value;
    uint4 fw[N][NT], fx[N][XB];
#pragma unroll
    for (int s = 0; s < N; ++s) {
#pragma unroll
      for (int t = 0; t < NT; ++t) fw[s][t] = load(wp[t] + (long long)(c + s) * PIECE);
#pragma unroll
      for (int b = 0; b < XB; ++b) fx[s][b] = load(xp[b] + (long long)(c + s) * PIECE);
    }
    __builtin_amdgcn_sched_barrier(0);   // all of them are asked for before the first is used
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < XB; ++b) acc[t][b % MB] = mfma_chunk<BF>(fw[s][t], fx[s][b], acc[t][b % MB]);
    c += N;
  };
  const int c1w = min(c1, whole);
  while (c + NB <= c1w) several(std::integral_constant<int, NB>{});
  while (c + 2 <= c1w) several(std::integral_constant<int, 2>{});
  while (c < c1w) several(std::integral_constant<int, 1>{});
  if (c < c1) {   // the ragged end of the rows: value by value
    const int left = (bytes - c * PIECE - off) / ES;
    auto ragged = [&](const char* at) {
      unsigned v[4] = {};
#pragma unroll
      for (int j = 0; j < 16 / ES; ++j)
        if (j < left) {
          if constexpr (BF) v[j / 2] |= (unsigned)((const uint16_t*)at)[j] << (16 * (j & 1));
          else v[j] = ((const unsigned*)at)[j];
        }
      return make_uint4(v[0], v[1], v[2], v[3]);
    };
    uint4 fx[XB];
#pragma unroll
    for (int b = 0; b < XB; ++b) fx[b] = ragged(xp[b] + (long long)c * PIECE);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const uint4 fw = ragged(wp[t] + (long long)c * PIECE);
#pragma unroll
      for (int b = 0; b < XB; ++b) acc[t][b % MB] = mfma_chunk<BF>(fw, fx[b], acc[t][b % MB]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < MB; ++b) part[wave][t * MB + b][lane] = acc[t][b];
  __syncthreads();

  // a wave per block of x's rows: lane i is row m, its values weight rows 4q .. 4q+3
  for (int b = wave; b < MB; b += W) {
    f32x4 s[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      s[t] = part[0][t * MB + b][lane];
      for (int w = 1; w < W; ++w) s[t] += part[w][t * MB + b][lane];
      if constexpr (PAIR)
        for (int w = 0; w < W; ++w) s[t] += part[w][t * MB + b][(lane + 40) & 63];
    }
    const int m = b * 16 + i;
    if (m >= p.M || (PAIR && (lane & 8 || q > 1))) continue;
    El<BF>* out = (El<BF>*)p.out + m * p.ldo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 4 * q + e;
      float v = s[0][e];
      if constexpr (GLU) v = act_of(p.act, v) * s[NT - 1][e];
      if (r < p.R) {
        el_store<BF>(out + r, v);
        if constexpr (BF && GLU) {
          const float rest = v - bf2f(f2bf(v));   // (none where v is no number or rounds to infinity)
          el_store<BF>(out + p.M * p.ldo + r, fabsf(rest) < 3e38f ? rest : 0.f);
        }
      }
    }
  }
}

template <bool BF, bool GLU>
hipError_t pick(const FfnRows& p, hipStream_t s) {
  if (p.M <= 0 || p.R <= 0) return hipSuccess;
  const bool pair = p.M <= 8;
  const int tiles = pair ? (p.R + 7) / 8 : (p.R + 15) / 16, bytes = p.K * (BF ? 2 : 4);
  const int pieces = pair ? (bytes + 127) / 128 : (bytes + 63) / 64;
  // enough waves to keep the memory busy (16 a CU), while each has work
  int w = 1;
  while (w < kWaves && (long long)tiles * w < 4096 && 2 * w <= pieces) w *= 2;
  const dim3 grid(tiles), block(64 * w);
  if (pair) hipLaunchKernelGGL((rows_kernel<BF, GLU, 1, true>), grid, block, 0, s, p);
  else if (p.M <= 16) hipLaunchKernelGGL((rows_kernel<BF, GLU, 1, false>), grid, block, 0, s, p);
  else if (p.M <= 32) hipLaunchKernelGGL((rows_kernel<BF, GLU, 2, false>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((rows_kernel<BF, GLU, 4, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t rnn_launch_ffn_rows(const FfnRows& p, int bf16, int glu, hipStream_t s) {
  if (bf16) return glu ? pick<true, true>(p, s) : pick<true, false>(p, s);
  return glu ? pick<false, true>(p, s) : pick<false, false>(p, s);
}
