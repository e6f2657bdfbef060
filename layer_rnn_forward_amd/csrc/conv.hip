// Depthwise causal convolution over time (gfx950): v_t = bias +
// sum_k w[c, k] x_(t - K + 1 + k), y = v or silu(v), its gradients, and its
// form for single steps.
//
// A lane holds 4 neighbouring channels (kWidth) and walks a piece of the time axis with
// the last K inputs in registers, so an input is read once, and again only by
// the piece that follows (K - 1 steps).  Backward walks K - 1 steps further
// than its piece, which makes the v' that its last inputs need, keeps the last
// K of them, and sums the weights' gradients over its own steps; pieces' sums
// are added in a second launch, in a fixed order.
//
// Bound: memory (two values a step and channel forward, three backward).  2048
// steps of 8 rows of 2048 channels, bf16, K = 4: forward 31 us, backward 51 us,
// the sums 5 us (4.3 and 3.9 TB/s).  With a branch for every step and lane,
// which makes each wait for loads one for the stores before them, too, 36 us
// forward (32 without); with pieces of 32 steps backward (1.3 rounds of the waves
// that fit) 67 us instead of 50.  Channels past the last whole 256 take the walk
// with the branches: 1237 x 7 packed x 357, fp32, K = 3: 7 and 12 us, the sums 4.

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ssm_common.h"

using namespace rnnk;

namespace {

// Steps whose loads are asked for at once, forward and backward.  Where all of
// them and the channels of all lanes are there (most of a long piece) they are
// walked without a branch, so that a wait for the next steps' loads counts past
// the stores between.
constexpr int kAhead = 8, kBackAhead = 4;

constexpr int kWidth = 4;     // channels of a lane

// silu and its slope
__device__ __forceinline__ float silu(float v) {
  float a, da;
  act_pair<ACT_SILU>(v, a, da);
  return a;
}

struct Place {
  int c, left;               // first channel, channels from there on
  bool whole;                // every lane has all of its channels
  int b, len;
  int t0, t1;                // steps of the piece
};
template <int VW>
__device__ __forceinline__ Place place(const ConvParams& p) {
  Place r;
  const int tiles = (p.C + 64 * VW - 1) / (64 * VW);
  int i = blockIdx.x;
  const int tile = i % tiles;
  i /= tiles;
  r.b = i % p.B;
  const int piece = i / p.B * kConvWaves + (int)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // uniform, as what follows from it
  r.c = (tile * 64 + (int)(threadIdx.x & 63)) * VW;
  r.left = p.C - r.c;
  r.whole = (tile + 1) * 64 * VW <= p.C;
  r.t0 = r.t1 = -1;
  if (piece < p.pieces) {
    r.t0 = piece * p.piece;
    r.t1 = min(r.t0 + p.piece, p.T);
  }
  r.len = p.lengths ? min(max(p.lengths[r.b], 0), p.T) : p.T;
  return r;
}

// values of a lane's weights from the i-th 16 bytes on, where `left` channels are
// there (all of them may be 2^30: times K they are past 32 bits)
template <int K, int VW>
__host__ __device__ constexpr int weights_left(int left, int i) { return (left < VW ? left : VW) * K - 4 * i; }
static_assert(weights_left<kConvMost, kWidth>((1 << 30) - 1, 1) == kConvMost * kWidth - 4, "no overflow with the most channels");

template <int K, int VW>
__device__ __forceinline__ void load_weights(const ConvParams& p, const Place& at, float (&w)[K][VW], float (&bias)[VW]) {
  // the lane's weights are neighbours: 16 bytes a load
  const float* from = p.w + (long long)at.c * K;
  RawPiece<false, 4> raw[VW * K / 4];
#pragma unroll
  for (int i = 0; i < VW * K / 4; ++i) raw[i] = load_raw<false, 4>(from + 4 * i, weights_left<K, VW>(at.left, i));
  load_piece<false, VW>(p.bias + at.c, p.bias ? at.left : 0, bias);
#pragma unroll
  for (int j = 0; j < VW; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][j] = __uint_as_float(raw[(j * K + k) / 4].w[(j * K + k) % 4]);
}

// input of step t >= -(K - 1); steps past the row's length are not used
template <bool BF, int K, int VW>
__device__ __forceinline__ RawPiece<BF, VW> input(const ConvParams& p, const Place& at, int t) {
  if (t >= at.len || (t < 0 && !p.s0)) return {};
  const El<BF>* from = t >= 0 ? (const El<BF>*)p.x + ((long long)t * p.B + at.b) * p.ldx + at.c
                              : (const El<BF>*)p.s0 + ((long long)(t + K - 1) * p.B + at.b) * p.C + at.c;
  return load_raw<BF, VW>(from, at.left);
}
template <bool BF, int K, int VW>
__device__ __forceinline__ void input(const ConvParams& p, const Place& at, int t, float (&v)[VW]) {
  unpack<BF, VW>(input<BF, K, VW>(p, at, t), v);
}

// the inputs before the step that follows the row's last
template <bool BF, int K, int VW>
__device__ __forceinline__ void last_inputs(const ConvParams& p, const Place& at) {
  if constexpr (K > 1) {
    float v[K - 1][VW];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) input<BF, K, VW>(p, at, at.len - (K - 1) + j, v[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_piece<BF, VW>((El<BF>*)p.sy + ((long long)j * p.B + at.b) * p.C + at.c, at.left, v[j]);
  }
}

template <bool BF, int K, bool SILU>
__global__ __launch_bounds__(64 * kConvWaves) void fwd_kernel(const ConvParams p) {
  constexpr int VW = kWidth;
  const Place at = place<VW>(p);
  if (at.t0 < 0 || at.left <= 0) return;
  float w[K][VW], bias[VW], x[K][VW];
  load_weights<K, VW>(p, at, w, bias);
#pragma unroll
  for (int k = 0; k < K - 1; ++k) input<BF, K, VW>(p, at, at.t0 - (K - 1) + k, x[k + 1]);
  RawPiece<BF, VW> raw[kAhead], next[kAhead];
  auto load = [&](int t, auto fast) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if constexpr (decltype(fast)::value)
        next[i] = *reinterpret_cast<const RawPiece<BF, VW>*>((const El<BF>*)p.x + ((long long)(t + i) * p.B + at.b) * p.ldx + at.c);
      else
        next[i] = input<BF, K, VW>(p, at, min(t + i, at.t1 - 1));
    }
  };
  auto walk = [&](int t, auto fast) {
    constexpr bool FAST = decltype(fast)::value;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!FAST && t + i >= at.t1) break;
      float v[VW], in[VW];
      unpack<BF, VW>(raw[i], in);
#pragma unroll
      for (int j = 0; j < VW; ++j) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) x[k][j] = x[k + 1][j];
        x[K - 1][j] = in[j];
        v[j] = bias[j];
#pragma unroll
        for (int k = 0; k < K; ++k) v[j] = fmaf(w[k][j], x[k][j], v[j]);
        if (SILU) v[j] = silu(v[j]);
        if (!FAST && t + i >= at.len) v[j] = 0.f;
      }
      store_piece<BF, VW>((El<BF>*)p.y + ((long long)(t + i) * p.B + at.b) * p.ldy + at.c, FAST ? VW : at.left, v);
    }
  };
  // whole groups of steps of the piece and the row
  const int fast = at.whole ? max(0, min(at.t1, at.len) - at.t0) / kAhead * kAhead : 0;
  int t = at.t0;
  if (fast) {
    load(t, std::true_type{});
    for (; t < at.t0 + fast; t += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) raw[i] = next[i];
      load(min(t + kAhead, at.t0 + fast - kAhead), std::true_type{});   // the last time: the same once more
      walk(t, std::true_type{});
    }
  }
  for (; t < at.t1; t += kAhead) {
    load(t, std::false_type{});
#pragma unroll
    for (int i = 0; i < kAhead; ++i) raw[i] = next[i];
    walk(t, std::false_type{});
  }
  // s0 is read by the first piece alone, so sy may take its place
  if (p.sy && at.t0 == 0) last_inputs<BF, K, VW>(p, at);
}

template <bool BF, int K, bool SILU>
__global__ __launch_bounds__(64 * kConvWaves) void bwd_kernel(const ConvParams p) {
  constexpr int VW = kWidth;
  const Place at = place<VW>(p);
  __shared__ float sums[kConvWaves][K + 1][64 * VW];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float dw[K][VW], db[VW];
#pragma unroll
  for (int j = 0; j < VW; ++j) {
    db[j] = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k][j] = 0.f;
  }
  if (at.t0 >= 0 && at.left > 0) {
    float w[K][VW], bias[VW], x[K][VW], dv[K][VW];
    load_weights<K, VW>(p, at, w, bias);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < VW; ++j) dv[k][j] = 0.f;
#pragma unroll
    for (int k = 0; k < K - 1; ++k) input<BF, K, VW>(p, at, at.t0 - (K - 1) + k, x[k + 1]);
    // after step t the gradient of input t - K + 1 is whole
    const int end = at.t1 + K - 1;
    RawPiece<BF, VW> rx[kBackAhead], rdy[kBackAhead], nx[kBackAhead], ndy[kBackAhead];
    auto load = [&](int t, auto fast) {
#pragma unroll
      for (int i = 0; i < kBackAhead; ++i) {
        constexpr bool FAST = decltype(fast)::value;
        const int s = FAST ? t + i : min(t + i, end - 1);
        const El<BF>* x = (const El<BF>*)p.x + ((long long)s * p.B + at.b) * p.ldx + at.c;
        const El<BF>* dy = (const El<BF>*)p.dy + ((long long)s * p.B + at.b) * p.lddy + at.c;
        if constexpr (FAST) {
          nx[i] = *reinterpret_cast<const RawPiece<BF, VW>*>(x);
          ndy[i] = *reinterpret_cast<const RawPiece<BF, VW>*>(dy);
        } else {
          nx[i] = ndy[i] = {};
          if (s < at.len) {
            nx[i] = load_raw<BF, VW>(x, at.left);
            ndy[i] = load_raw<BF, VW>(dy, at.left);
          }
        }
      }
    };
    auto turn = [&] {
#pragma unroll
      for (int i = 0; i < kBackAhead; ++i) {
        rx[i] = nx[i];
        rdy[i] = ndy[i];
      }
    };
    auto walk = [&](int t, auto fast) {
      constexpr bool FAST = decltype(fast)::value;
#pragma unroll
      for (int i = 0; i < kBackAhead; ++i) {
        if (!FAST && t + i >= end) break;
        const int s = t + i - (K - 1);      // the input whose gradient is whole
        const bool mine = FAST || t + i < min(at.t1, at.len);   // (past the row's length: 0 times an infinite input)
        float dx[VW], more[VW], in[VW], dy[VW];
        unpack<BF, VW>(rx[i], in);
        unpack<BF, VW>(rdy[i], dy);
        const int j0 = s - at.len + K - 1;
        const bool last = !FAST && p.dsy && j0 >= 0 && j0 < K - 1 && (s >= at.t0 || at.t0 == 0);
        if (last) load_piece<BF, VW>((const El<BF>*)p.dsy + ((long long)j0 * p.B + at.b) * p.C + at.c, at.left, more);
#pragma unroll
        for (int j = 0; j < VW; ++j) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) x[k][j] = x[k + 1][j];
          x[K - 1][j] = in[j];
          float d = dy[j];
          if (SILU) {
            float v = bias[j], a, da;
#pragma unroll
            for (int k = 0; k < K; ++k) v = fmaf(w[k][j], x[k][j], v);
            act_pair<ACT_SILU>(v, a, da);
            d = FAST || t + i < at.len ? d * da : 0.f;
          }
#pragma unroll
          for (int k = K - 1; k > 0; --k) dv[k][j] = dv[k - 1][j];
          dv[0][j] = d;
          if (mine) {
            db[j] += d;
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][j] = fmaf(d, x[k][j], dw[k][j]);
          }
          dx[j] = last ? more[j] : 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) dx[j] = fmaf(w[k][j], dv[k][j], dx[j]);
          if (!FAST && s >= at.len) dx[j] = 0.f;                // whatever the weights
        }
        if (FAST || s >= at.t0) {
          if (FAST || p.dx) store_piece<BF, VW>((El<BF>*)p.dx + ((long long)s * p.B + at.b) * p.lddx + at.c, FAST ? VW : at.left, dx);
        } else if (at.t0 == 0 && p.ds0) {
          store_piece<BF, VW>((El<BF>*)p.ds0 + ((long long)(s + K - 1) * p.B + at.b) * p.C + at.c, at.left, dx);
        }
      }
    };
    // the first steps complete inputs before the piece, the last ones are past it
    // or the row; between them whole groups
    constexpr int HEAD = (K - 1 + kBackAhead - 1) / kBackAhead * kBackAhead;
    int t = at.t0;
    const int fast = at.whole && p.dx ? max(0, min(at.t1, at.len) - t - HEAD) / kBackAhead * kBackAhead : 0;
    const int to = fast ? t + HEAD + fast : 0;
    for (; t < end; t += kBackAhead) {
      if (t + fast == to && fast) {          // HEAD steps are done
        load(t, std::true_type{});
        for (; t < to; t += kBackAhead) {
          turn();
          load(min(t + kBackAhead, to - kBackAhead), std::true_type{});   // the last time: the same once more
          walk(t, std::true_type{});
        }
      }
      load(t, std::false_type{});
      turn();
      walk(t, std::false_type{});
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int j = 0; j < VW; ++j) {
#pragma unroll
    for (int k = 0; k < K; ++k) sums[wave][k][lane * VW + j] = dw[k][j];
    sums[wave][K][lane * VW + j] = db[j];
  }
  __syncthreads();
  const int tiles = (p.C + 64 * VW - 1) / (64 * VW), tile = blockIdx.x % tiles;
  float* to = p.part + (long long)(blockIdx.x / tiles) * (K + 1) * p.C;
  for (int i = threadIdx.x; i < (K + 1) * 64 * VW; i += 64 * kConvWaves) {
    const int k = i / (64 * VW), c = i - k * (64 * VW);
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kConvWaves; ++q) s += sums[q][k][c];
    if (tile * 64 * VW + c < p.C) to[(long long)k * p.C + tile * 64 * VW + c] = s;
  }
}

__global__ __launch_bounds__(64 * kSumWaves) void sum_kernel(const ConvParams p, int rows) {
  __shared__ float lds[kSumWaves][64];
  const long long n = (long long)(p.K + 1) * p.C, i = ((long long)blockIdx.y * gridDim.x + blockIdx.x) * 64 + (threadIdx.x & 63);
  const float s = column_sum(p.part, n, i, rows, lds);
  if (threadIdx.x >= 64 || i >= n) return;
  const int k = (int)(i / p.C), c = (int)(i - (long long)k * p.C);
  if (k == p.K) {
    if (p.dbias) p.dbias[c] = s;
  } else if (p.dw) {
    p.dw[(long long)c * p.K + k] = s;
  }
}

template <bool BF, int K>
__global__ __launch_bounds__(256) void step_kernel(const ConvParams p) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)p.B * p.C) return;
  const int b = (int)(i / p.C), c = (int)(i - (long long)b * p.C);
  const long long n = (long long)p.B * p.C;
  El<BF> x[K];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) x[k] = p.s0 ? ((const El<BF>*)p.s0)[k * n + i] : El<BF>(0);
  x[K - 1] = ((const El<BF>*)p.x)[b * p.ldx + c];
  float v = p.bias ? p.bias[c] : 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) v = fmaf(p.w[(long long)c * K + k], el_load<BF>(&x[k]), v);
  if (p.silu) v = silu(v);
  if (p.sy)
#pragma unroll
    for (int k = 0; k < K - 1; ++k) ((El<BF>*)p.sy)[k * n + i] = x[k + 1];
  el_store<BF>((El<BF>*)p.y + b * p.ldy + c, v);
}

enum Pass { FWD, BWD, STEP };
template <bool BF, int K>
void start(const ConvParams& p, Pass what, hipStream_t s) {
  if (what == STEP) {
    hipLaunchKernelGGL((step_kernel<BF, K>), dim3((unsigned)(((long long)p.B * p.C + 255) / 256)), dim3(256), 0, s, p);
    return;
  }
  const long long width = 64 * kWidth, tiles = (p.C + width - 1) / width;
  const dim3 grid((unsigned)(tiles * p.B * ((p.pieces + kConvWaves - 1) / kConvWaves))), block(64 * kConvWaves);
  if (what == FWD && p.silu) hipLaunchKernelGGL((fwd_kernel<BF, K, true>), grid, block, 0, s, p);
  else if (what == FWD) hipLaunchKernelGGL((fwd_kernel<BF, K, false>), grid, block, 0, s, p);
  else if (p.silu) hipLaunchKernelGGL((bwd_kernel<BF, K, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((bwd_kernel<BF, K, false>), grid, block, 0, s, p);
}

template <bool BF>
void pick(const ConvParams& p, Pass what, hipStream_t s) {
  switch (p.K) {
    case 1: return start<BF, 1>(p, what, s);
    case 2: return start<BF, 2>(p, what, s);
    case 3: return start<BF, 3>(p, what, s);
    case 4: return start<BF, 4>(p, what, s);
    case 5: return start<BF, 5>(p, what, s);
    case 6: return start<BF, 6>(p, what, s);
    case 7: return start<BF, 7>(p, what, s);
    default: return start<BF, 8>(p, what, s);
  }
}

hipError_t launch(const ConvParams& p, Pass what, int bf16, hipStream_t s) {
  if (p.B == 0 || p.C == 0) return hipSuccess;
  if (bf16) pick<true>(p, what, s);
  else pick<false>(p, what, s);
  return hipGetLastError();
}

}  // namespace

// Steps of a wave's piece (at least K - 1 of them): as many as give each SIMD 4
// waves forward and 3 backward, so that all run at once where its registers hold as
// many: with K up to 4, and mostly with 5 and 6 forward, 5 backward.  Of wider filters
// they hold 3 forward (K = 8; in fp32 7, too, and 5 with silu) and 2 backward (K = 7
// and 8; 6 but for bf16 without silu; in fp32 5 with silu), so that a launch is up to
// 1.5 rounds of what fits.
int rnnk::conv_piece(int T, int B, int C, bool back) {
  const double steps = (double)B * ((C + 64 * kWidth - 1) / (64 * kWidth)) * T / (1024 * (back ? 3 : 4));
  return (int)std::min(std::max(1.0, std::ceil(steps / 8)), std::ceil(std::max(T, 1) / 8.0)) * 8;
}

long long rnnk::conv_blocks(int T, int B, int C, bool back) {
  const long long tiles = (C + 64 * kWidth - 1) / (64 * kWidth), steps = (long long)conv_piece(T, B, C, back) * kConvWaves;
  return tiles * B * std::max(1LL, (T + steps - 1) / steps);
}

// At least the B * groups of pieces of a backward pass, and no fewer with more
// steps or rows, so that a workspace does for fewer of both: a piece has at
// least 8 steps and its share of 1024 * 3 waves.
long long rnnk::conv_parts(int T, int B, int C) {
  const long long tiles = std::max(1, (C + 64 * kWidth - 1) / (64 * kWidth)), waves = 1024 * 3 / kConvWaves;
  return std::min((waves + tiles - 1) / tiles + 2LL * B, B * std::max(1LL, (T + 8LL * kConvWaves - 1) / (8 * kConvWaves)));
}

hipError_t rnn_launch_conv_fwd(const ConvParams& p, int bf16, hipStream_t s) { return launch(p, FWD, bf16, s); }
hipError_t rnn_launch_conv_step(const ConvParams& p, int bf16, hipStream_t s) { return launch(p, STEP, bf16, s); }
hipError_t rnn_launch_conv_bwd(const ConvParams& q, int bf16, hipStream_t s) {
  ConvParams p = q;
  const bool sums = p.dw || p.dbias;
  if (!sums) p.part = nullptr;
  if (p.B == 0 || p.C == 0) p.pieces = 0;
  const hipError_t e = launch(p, BWD, bf16, s);
  if (e != hipSuccess || !sums || p.C == 0) return e;
  const int rows = p.B * ((p.pieces + kConvWaves - 1) / kConvWaves);
  hipLaunchKernelGGL(sum_kernel, wide_grid(((long long)(p.K + 1) * p.C + 63) / 64), dim3(64 * kSumWaves), 0, s, p, rows);
  return hipGetLastError();
}
