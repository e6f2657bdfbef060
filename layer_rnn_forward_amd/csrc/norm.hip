// Normalisation of rows (gfx950): layer norm and root-mean-square norm with
// the residual addition before them, and their gradients.
//
// A row lies in the registers of L lanes, 16 bytes a piece, so it is read once;
// mean and variance are two sums over registers (the second about the mean:
// no cancellation).  Backward keeps the parameters' gradients of its columns
// in registers over all rows that a group of lanes walks, and adds the groups'
// sums in a second launch, in a fixed order.
//
// Bound: memory.  16384 rows of 2048, bf16, with residual: forward 47 us (5.7
// TB/s: what it writes stays in the last cache level), backward 48 us, the sums 6
// us; 4291 rows of 1357 in fp32: 12, 17 and 6 us.  16 rows: one launch of 3 us.
// Backward with a bias gradient spills on rows of 8193 to 16384 columns (1024
// lanes, 128 registers each): 74 registers in fp32, 6 in bf16.
#include <algorithm>

#include "ssm_common.h"

using namespace rnnk;

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ long long row_block() { return (long long)blockIdx.y * gridDim.x + blockIdx.x; }

// sum over L lanes (64: a wave, else the workgroup); `slot` alternates between calls
template <int L>
__device__ __forceinline__ float row_sum(float v, float* lds, int& slot) {
  v = sum_lanes<1>(v);
  if constexpr (L > 64) {
    constexpr int W = L / 64;
    float* at = lds + slot * W;
    slot ^= 1;
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += at[w];
  }
  return v;
}

template <bool BF, int L, int P>
__global__ __launch_bounds__(L < kThreads ? kThreads : L) void fwd_kernel(const NormParams p) {
  constexpr int VW = piece_width<BF>(), ROWS = L < kThreads ? kThreads / L : 1;
  __shared__ float lds[2 * (L / 64)];
  int slot = 0;
  const int lane = threadIdx.x % L;
  const long long row = row_block() * ROWS + threadIdx.x / L;
  if (row >= p.M) return;                        // (a whole workgroup, or a wave of those without barriers)
  const long long at = row * p.D;
  const El<BF>* x = (const El<BF>*)p.x + at;
  const El<BF>* r = (const El<BF>*)p.residual + at;
  float v[P][VW], sum = 0.f;
  RawPiece<BF, VW> rx[P], rr[P];
#pragma unroll
  for (int i = 0; i < P; ++i) rx[i] = load_raw<BF, VW>(x + (i * L + lane) * VW, p.D - (i * L + lane) * VW);
  if (p.residual)
#pragma unroll
    for (int i = 0; i < P; ++i) rr[i] = load_raw<BF, VW>(r + (i * L + lane) * VW, p.D - (i * L + lane) * VW);
#pragma unroll
  for (int i = 0; i < P; ++i) unpack<BF, VW>(rx[i], v[i]);
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float b[VW];
      unpack<BF, VW>(rr[i], b);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        v[i][j] += b[j];
        if constexpr (BF) v[i][j] = bf2f(f2bf(v[i][j]));   // as the residual stream holds it
      }
    }
  }
  if (p.total) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * L + lane) * VW;
      store_piece<BF, VW>((El<BF>*)p.total + at + c, p.D - c, v[i]);
    }
  }
  const float inv = 1.f / (float)p.D;
  float mean = 0.f;
  if (!p.rms) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < VW; ++j) sum += v[i][j];
    mean = row_sum<L>(sum, lds, slot) * inv;
  }
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int left = p.D - (i * L + lane) * VW;
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      v[i][j] -= mean;
      if (j < left) sq = fmaf(v[i][j], v[i][j], sq);
    }
  }
  const float rstd = 1.f / sqrtf(row_sum<L>(sq, lds, slot) * inv + p.eps);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = (i * L + lane) * VW, left = p.D - c;
    float w[VW], b[VW];
    if (p.weight) load_piece<false, VW>(p.weight + c, left, w);
    if (p.bias) load_piece<false, VW>(p.bias + c, left, b);
#pragma unroll
    for (int j = 0; j < VW; ++j) v[i][j] = fmaf(v[i][j] * rstd, p.weight ? w[j] : 1.f, p.bias ? b[j] : 0.f);
    store_piece<BF, VW>((El<BF>*)p.y + at + c, left, v[i]);
  }
  if (p.stats && lane == 0) {
    p.stats[2 * row] = mean;
    p.stats[2 * row + 1] = rstd;
  }
}

// dx = rstd (g - mean(g) - xh mean(g xh)) + dtotal, g = dy weight (without
// mean(g) for RMS); the rows' sums of dy xh and (BIAS) dy go to `part`, a row of
// them for each workgroup
constexpr int back_threads(int L) { return L == 64 ? 512 : L; }
template <bool BF, int L, int P, bool BIAS>
__global__ __launch_bounds__(back_threads(L)) void bwd_kernel(const NormParams p) {
  constexpr int VW = piece_width<BF>(), ROWS = back_threads(L) / L;
  __shared__ float lds[2 * (L / 64)];
  __shared__ float both[ROWS > 1 ? 2 * P * L * VW : 1];
  int slot = 0;
  const int lane = threadIdx.x % L;
  const int group = blockIdx.x * ROWS + threadIdx.x / L, groups = gridDim.x * ROWS;
  float dw[P][VW] = {}, db[BIAS ? P : 1][VW] = {};
  const float inv = 1.f / (float)p.D;
  for (long long row = group; row < p.M; row += groups) {
    const long long at = row * p.D;
    const float mean = p.stats[2 * row], rstd = p.stats[2 * row + 1];
    RawPiece<BF, VW> rx[P], rg[P], rt[P];
    float x[P][VW], g[P][VW], s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * L + lane) * VW;
      rx[i] = load_raw<BF, VW>((const El<BF>*)p.x + at + c, p.D - c);
      rg[i] = load_raw<BF, VW>((const El<BF>*)p.dy + at + c, p.D - c);
    }
    if (p.dtotal)
#pragma unroll
      for (int i = 0; i < P; ++i) rt[i] = load_raw<BF, VW>((const El<BF>*)p.dtotal + at + (i * L + lane) * VW, p.D - (i * L + lane) * VW);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * L + lane) * VW, left = p.D - c;
      float w[VW];
      if (p.weight) load_piece<false, VW>(p.weight + c, left, w);
      unpack<BF, VW>(rx[i], x[i]);
      unpack<BF, VW>(rg[i], g[i]);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        x[i][j] = j < left ? (x[i][j] - mean) * rstd : 0.f;
        dw[i][j] = fmaf(g[i][j], x[i][j], dw[i][j]);
        if constexpr (BIAS) db[i][j] += g[i][j];
        if (p.weight) g[i][j] *= w[j];
        s0 += g[i][j];
        s1 = fmaf(g[i][j], x[i][j], s1);
      }
    }
    if (!p.dx) continue;
    s0 = p.rms ? 0.f : row_sum<L>(s0, lds, slot) * inv;
    s1 = row_sum<L>(s1, lds, slot) * inv;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * L + lane) * VW, left = p.D - c;
      float t[VW];
      if (p.dtotal) unpack<BF, VW>(rt[i], t);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        const float d = rstd * (g[i][j] - fmaf(x[i][j], s1, s0));
        t[j] = p.dtotal ? d + t[j] : d;
      }
      store_piece<BF, VW>((El<BF>*)p.dx + at + c, left, t);
    }
  }
  if (!p.part) return;
  // the waves' sums, one wave after the other
  if constexpr (ROWS > 1) {
    for (int r = 0; r < ROWS; ++r) {
      if ((int)threadIdx.x / L == r) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            float* to = both + (i * VW + j) * L + lane;
            if (r > 0) dw[i][j] += *to;
            *to = dw[i][j];
            if constexpr (BIAS) {
              to += P * L * VW;
              if (r > 0) db[i][j] += *to;
              *to = db[i][j];
            }
          }
      }
      __syncthreads();
    }
    if ((int)threadIdx.x / L != ROWS - 1) return;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = (i * L + lane) * VW, left = p.D - c;
    float* to = p.part + (long long)blockIdx.x * (BIAS ? 2 : 1) * p.D + c;
    store_piece<false, VW>(to, left, dw[i]);
    if constexpr (BIAS) store_piece<false, VW>(to + p.D, left, db[i]);
  }
}

// Rows too long for a workgroup's registers: read again for every sum.
template <bool BF>
__global__ __launch_bounds__(1024) void fwd_long_kernel(const NormParams p) {
  constexpr int VW = piece_width<BF>();
  __shared__ float lds[32];
  int slot = 0;
  const long long row = row_block(), at = row * p.D;
  if (row >= p.M) return;
  const float inv = 1.f / (float)p.D;
  // the row's values: what an earlier walk has left in `total`, else x (+ residual)
  auto value = [&](int c, bool again, float(&v)[VW]) {
    if (again && p.total) {
      load_piece<BF, VW>((const El<BF>*)p.total + at + c, p.D - c, v);
      return;
    }
    load_piece<BF, VW>((const El<BF>*)p.x + at + c, p.D - c, v);
    if (p.residual) {
      float b[VW];
      load_piece<BF, VW>((const El<BF>*)p.residual + at + c, p.D - c, b);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        v[j] += b[j];
        if constexpr (BF) v[j] = bf2f(f2bf(v[j]));
      }
    }
  };
  float v[VW], mean = 0.f, sum = 0.f;
  if (!p.rms || p.total) {
    for (int c = threadIdx.x * VW; c < p.D; c += 1024 * VW) {
      value(c, false, v);
      if (p.total) store_piece<BF, VW>((El<BF>*)p.total + at + c, p.D - c, v);
#pragma unroll
      for (int j = 0; j < VW; ++j) sum += v[j];
    }
    if (!p.rms) mean = row_sum<1024>(sum, lds, slot) * inv;
  }
  float sq = 0.f;
  for (int c = threadIdx.x * VW; c < p.D; c += 1024 * VW) {
    value(c, true, v);
#pragma unroll
    for (int j = 0; j < VW; ++j)
      if (j < p.D - c) sq = fmaf(v[j] - mean, v[j] - mean, sq);
  }
  const float rstd = 1.f / sqrtf(row_sum<1024>(sq, lds, slot) * inv + p.eps);
  for (int c = threadIdx.x * VW; c < p.D; c += 1024 * VW) {
    value(c, true, v);
    float w[VW], b[VW];
    if (p.weight) load_piece<false, VW>(p.weight + c, p.D - c, w);
    if (p.bias) load_piece<false, VW>(p.bias + c, p.D - c, b);
#pragma unroll
    for (int j = 0; j < VW; ++j) v[j] = fmaf((v[j] - mean) * rstd, p.weight ? w[j] : 1.f, p.bias ? b[j] : 0.f);
    store_piece<BF, VW>((El<BF>*)p.y + at + c, p.D - c, v);
  }
  if (p.stats && threadIdx.x == 0) {
    p.stats[2 * row] = mean;
    p.stats[2 * row + 1] = rstd;
  }
}

template <bool BF>
__global__ __launch_bounds__(1024) void bwd_long_kernel(const NormParams p) {
  constexpr int VW = piece_width<BF>();
  __shared__ float lds[32];
  int slot = 0;
  const long long row = row_block(), at = row * p.D;
  if (row >= p.M) return;
  const float inv = 1.f / (float)p.D, mean = p.stats[2 * row], rstd = p.stats[2 * row + 1];
  float x[VW], g[VW], w[VW], s0 = 0.f, s1 = 0.f;
  auto values = [&](int c) {
    const int left = p.D - c;
    load_piece<BF, VW>((const El<BF>*)p.x + at + c, left, x);
    load_piece<BF, VW>((const El<BF>*)p.dy + at + c, left, g);
    if (p.weight) load_piece<false, VW>(p.weight + c, left, w);
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      x[j] = j < left ? (x[j] - mean) * rstd : 0.f;
      g[j] *= p.weight ? w[j] : 1.f;
    }
  };
  for (int c = threadIdx.x * VW; c < p.D; c += 1024 * VW) {
    values(c);
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      s0 += g[j];
      s1 = fmaf(g[j], x[j], s1);
    }
  }
  s0 = p.rms ? 0.f : row_sum<1024>(s0, lds, slot) * inv;
  s1 = row_sum<1024>(s1, lds, slot) * inv;
  for (int c = threadIdx.x * VW; c < p.D; c += 1024 * VW) {
    values(c);
    float t[VW];
    if (p.dtotal) load_piece<BF, VW>((const El<BF>*)p.dtotal + at + c, p.D - c, t);
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      const float d = rstd * (g[j] - fmaf(x[j], s1, s0));
      t[j] = p.dtotal ? d + t[j] : d;
    }
    store_piece<BF, VW>((El<BF>*)p.dx + at + c, p.D - c, t);
  }
}

// dy xh and dy over every gridDim.y-th row, column by column
template <bool BF>
__global__ __launch_bounds__(kThreads) void columns_kernel(const NormParams p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= p.D) return;
  float dw = 0.f, db = 0.f;
  for (long long row = blockIdx.y; row < p.M; row += gridDim.y) {
    const float g = el_load<BF>((const El<BF>*)p.dy + row * p.D + c);
    const float x = el_load<BF>((const El<BF>*)p.x + row * p.D + c);
    dw = fmaf(g, (x - p.stats[2 * row]) * p.stats[2 * row + 1], dw);
    db += g;
  }
  float* to = p.part + (long long)blockIdx.y * (p.dbias ? 2 : 1) * p.D + c;
  to[0] = dw;
  if (p.dbias) to[p.D] = db;
}

__global__ __launch_bounds__(64 * kSumWaves) void sum_kernel(const NormParams p) {
  __shared__ float lds[kSumWaves][64];
  const long long c = (long long)blockIdx.x * 64 + (threadIdx.x & 63), n = (p.dbias ? 2LL : 1LL) * p.D;
  const float s = column_sum(p.part, n, c, p.parts, lds);
  if (threadIdx.x >= 64 || c >= n) return;
  if (c >= p.D) p.dbias[c - p.D] = s;
  else if (p.dweight) p.dweight[c] = s;
}

// Lanes and pieces of a row.
struct Shape {
  int lanes, pieces;       // lanes 0: too long for registers
};
constexpr int kMost = 32;  // values of a row that a lane holds at most (of 1024 lanes: half of it, a quarter of the registers)
Shape shape(int D, int vw) {
  const int pieces = (D + vw - 1) / vw;
  Shape s;
  // a wave a row where it holds the row in one piece a lane; a workgroup with few
  // pieces a lane hides more latency than a wave with many (16384 x 2048 bf16
  // backward 47 us, with a wave a row 51)
  s.lanes = pieces <= 64 ? 64 : pieces <= 256 * (kMost / vw) ? 256 : 1024;
  s.pieces = 1;
  while (s.pieces * s.lanes < pieces) s.pieces *= 2;
  if (s.pieces * vw > (s.lanes == 1024 ? kMost / 2 : kMost)) s.lanes = 0;
  return s;
}

template <bool BF, int L, int P>
void start(const NormParams& p, bool back, int blocks, hipStream_t s) {
  constexpr int threads = L < kThreads ? kThreads : L, rows = threads / L;
  if (back && p.dbias) hipLaunchKernelGGL((bwd_kernel<BF, L, P, true>), dim3(blocks), dim3(back_threads(L)), 0, s, p);
  else if (back) hipLaunchKernelGGL((bwd_kernel<BF, L, P, false>), dim3(blocks), dim3(back_threads(L)), 0, s, p);
  else hipLaunchKernelGGL((fwd_kernel<BF, L, P>), wide_grid(((long long)p.M + rows - 1) / rows), dim3(threads), 0, s, p);
}

template <bool BF>
void pick(const NormParams& p, bool back, const Shape& sh, int blocks, hipStream_t s) {
  const int n = sh.pieces;
  if (sh.lanes == 64) return start<BF, 64, 1>(p, back, blocks, s);
  if (sh.lanes == 256) {
    if (n == 1) return start<BF, 256, 1>(p, back, blocks, s);
    if (n == 2) return start<BF, 256, 2>(p, back, blocks, s);
    if (BF || n == 4) return start<BF, 256, 4>(p, back, blocks, s);
    return start<BF, 256, BF ? 4 : 8>(p, back, blocks, s);
  }
  start<BF, 1024, BF ? 2 : 4>(p, back, blocks, s);                   // more than 8192 columns
}

// workgroups of the backward launch, and rows of partial sums
int back_blocks(int M, int lanes) {
  if (lanes == 64) return std::max(1, std::min((M + 7) / 8, 512));
  return std::max(1, std::min(M, lanes == 1024 ? 256 : 1024));
}
int back_parts(int M, int lanes) { return lanes ? back_blocks(M, lanes) : std::min(M, 64); }

template <bool BF>
hipError_t launch(const NormParams& p, bool back, hipStream_t s) {
  const Shape sh = shape(p.D, piece_width<BF>());
  if (sh.lanes) {
    const int blocks = back ? back_blocks(p.M, sh.lanes) : 0;
    pick<BF>(p, back, sh, blocks, s);
  } else if (!back) {
    hipLaunchKernelGGL(fwd_long_kernel<BF>, wide_grid(p.M), dim3(1024), 0, s, p);
  } else {
    if (p.dx) hipLaunchKernelGGL(bwd_long_kernel<BF>, wide_grid(p.M), dim3(1024), 0, s, p);
    if (p.part) hipLaunchKernelGGL(columns_kernel<BF>, dim3((p.D + kThreads - 1) / kThreads, (unsigned)p.parts), dim3(kThreads), 0, s, p);
  }
  return hipGetLastError();
}

}  // namespace

// the larger of both types' (the workspace's size does not know the type)
int rnnk::norm_parts(int M, int D) {
  int most = 1;
  for (int vw : {4, 8}) {
    const Shape sh = shape(D, vw);
    most = std::max(most, back_parts(M, sh.lanes));
  }
  return most;
}

hipError_t rnn_launch_norm_fwd(const NormParams& p, int bf16, hipStream_t s) {
  if (p.M == 0 || p.D == 0) return hipSuccess;
  return bf16 ? launch<true>(p, false, s) : launch<false>(p, false, s);
}

hipError_t rnn_launch_norm_bwd(const NormParams& q, int bf16, hipStream_t s) {
  if (q.D == 0) return hipSuccess;
  NormParams p = q;
  const bool sums = p.dweight || p.dbias;
  if (!sums) p.part = nullptr;
  const Shape sh = shape(p.D, bf16 ? 8 : 4);
  p.parts = p.M == 0 ? 0 : back_parts(p.M, sh.lanes);
  if (p.M > 0 && (p.dx || sums)) {
    const hipError_t e = bf16 ? launch<true>(p, true, s) : launch<false>(p, true, s);
    if (e != hipSuccess) return e;
  }
  if (sums) hipLaunchKernelGGL(sum_kernel, dim3((unsigned)(((p.dbias ? 2LL : 1LL) * p.D + 63) / 64)), dim3(64 * kSumWaves), 0, s, p);
  return hipGetLastError();
}
