// Plain products of the gated feed-forward block (ffn_gemm.h), and the copy
// that pads rows which are not whole 16-byte pieces.
#include <algorithm>

#include "ffn_gemm.h"

using namespace rnnk;

namespace {

// Eight (bf16) or four (fp32) values a lane: 16 bytes out, in at any alignment.
template <bool BF>
__global__ __launch_bounds__(256) void pad_kernel(const PadJob j) {
  constexpr int V = BF ? 8 : 4;
  const int z = blockIdx.z;
  const El<BF>* src = (const El<BF>*)j.src[z];
  El<BF>* dst = (El<BF>*)j.dst[z];
  const int cols = j.cols[z], ld = j.ld[z], per = ld / V;
  const long long n = j.rows[z] * per;
  const unsigned step = gridDim.x * 256;
  const int srow = (int)(step / (unsigned)per), spiece = (int)(step - (unsigned)srow * (unsigned)per);
  long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  long long r = i / per;
  int c = (int)(i - r * per);
  for (; i < n; i += step) {
    const El<BF>* from = src + r * cols + c * V;
    uint32_t w[4] = {};
    if (c * V + V <= cols) {
      const auto b = *reinterpret_cast<const Bytes<16>*>(from);
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = b.w[k];
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (c * V + k < cols) {
          if constexpr (BF) w[k / 2] |= (uint32_t)from[k] << (16 * (k & 1));
          else w[k] = __float_as_uint(from[k]);
        }
    }
    *reinterpret_cast<uint4*>(dst + r * ld + c * V) = make_uint4(w[0], w[1], w[2], w[3]);
    r += srow;
    c += spiece;
    if (c >= per) {
      c -= per;
      ++r;
    }
  }
}

// Up to three products in one launch.  Backward's three, once dgate and dup
// are there, fill the CUs together, where each alone leaves part of its last
// round empty.
struct Jobs {
  FfnGemm p[3];
  int begin[3], blocks[3];
};
__device__ __forceinline__ int job_of(const Jobs& j, int b) {
  for (int i = 0; i < 2; ++i)
    if (b >= j.begin[i] && b < j.begin[i] + j.blocks[i]) return i;
  return 2;
}

template <bool BF, int T, int OCC>
__global__ __launch_bounds__(256, OCC) void store_kernel(const Jobs j) {
  __shared__ __attribute__((aligned(1024))) char smem[ffn_lds(64 * T, 64 * T)];
  ffn_product<BF, true, true, T, T, FFN_STORE, SAVE_NONE, 0>(j.p[0], smem, (int)blockIdx.x, j.blocks[0]);
}
template <bool BF, int T, int OCC>
__global__ __launch_bounds__(256, OCC) void grads_kernel(const Jobs j) {
  __shared__ __attribute__((aligned(1024))) char smem[ffn_lds(64 * T, 64 * T)];
  const int b = (int)blockIdx.x, i = job_of(j, b);
  const FfnGemm p = j.p[i];
  if (i == 0) ffn_product<BF, true, false, T, T, FFN_STORE, SAVE_NONE, 0>(p, smem, b - j.begin[0], j.blocks[0]);
  else ffn_product<BF, false, false, T, T, FFN_STORE, SAVE_NONE, 0>(p, smem, b - j.begin[i], j.blocks[i]);
}
template <bool BF, int T>
__global__ __launch_bounds__(256) void sum_kernel(const Jobs j) {
  const int b = (int)blockIdx.x, i = job_of(j, b);
  const FfnGemm p = j.p[i];
  ffn_sum<BF, T, T, FFN_STORE, SAVE_NONE, 0>(p, b - j.begin[i]);
}

template <bool BACK, bool BF, int T, int OCC>
void start(const Jobs& j, long long blocks, hipStream_t s) {
  if (BACK) hipLaunchKernelGGL((grads_kernel<BF, T, OCC>), dim3((unsigned)blocks), dim3(256), 0, s, j);
  else hipLaunchKernelGGL((store_kernel<BF, T, OCC>), dim3((unsigned)blocks), dim3(256), 0, s, j);
}

template <bool BACK>
hipError_t run(Jobs& j, const int (&order)[3], int tile, int bf16, hipStream_t s) {
  Jobs sums = j;
  long long at = 0, sum_at = 0;
  for (int i : order) {
    const long long tiles = ffn_tiles(j.p[i], tile, false), blocks = (tiles * std::max(j.p[i].splits, 1) + 7) / 8 * 8;
    if (at + blocks > 0x7ffffff0LL) return hipErrorInvalidValue;
    j.begin[i] = (int)at;
    j.blocks[i] = (int)blocks;
    at += blocks;
    sums.begin[i] = (int)sum_at;
    sums.blocks[i] = j.p[i].splits > 1 ? (int)tiles : 0;
    sum_at += sums.blocks[i];
  }
  if (at == 0) return hipSuccess;
  if (!bf16) {
    if (tile == TILE_128) start<BACK, false, 2, 2>(j, at, s);
    else start<BACK, false, 1, 3>(j, at, s);
  } else if (tile == TILE_256) {
    start<BACK, true, 4, 1>(j, at, s);
  } else if (tile == TILE_128) {
    start<BACK, true, 2, 2>(j, at, s);
  } else {
    start<BACK, true, 1, 3>(j, at, s);
  }
  if (sum_at > 0) {
    const dim3 grid((unsigned)sum_at), block(256);
    if (!bf16) {
      if (tile == TILE_128) hipLaunchKernelGGL((sum_kernel<false, 2>), grid, block, 0, s, sums);
      else hipLaunchKernelGGL((sum_kernel<false, 1>), grid, block, 0, s, sums);
    } else if (tile == TILE_128) {   // (256 x 256 tiles are not split)
      hipLaunchKernelGGL((sum_kernel<true, 2>), grid, block, 0, s, sums);
    } else {
      hipLaunchKernelGGL((sum_kernel<true, 1>), grid, block, 0, s, sums);
    }
  }
  return hipGetLastError();
}

}  // namespace

hipError_t rnn_launch_ffn_store(const FfnGemm& p, int tile, int bf16, hipStream_t s) {
  Jobs j{};
  j.p[0] = p;
  const int order[3] = {0, 1, 2};
  return run<false>(j, order, tile, bf16, s);
}

hipError_t rnn_launch_ffn_grads(const FfnGemm (&p)[3], const int (&order)[3], int tile, int bf16, hipStream_t s) {
  Jobs j{{p[0], p[1], p[2]}, {}, {}};
  return run<true>(j, order, tile, bf16, s);
}

hipError_t rnn_launch_pad(const PadJob& j, int bf16, hipStream_t s) {
  if (j.n == 0) return hipSuccess;
  long long n = 0;
  for (int i = 0; i < j.n; ++i) n = std::max(n, j.rows[i] * (j.ld[i] / (bf16 ? 8 : 4)));
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<long long>((n + 255) / 256, 256 * 8), 1, j.n);
  if (bf16) hipLaunchKernelGGL(pad_kernel<true>, grid, dim3(256), 0, s, j);
  else hipLaunchKernelGGL(pad_kernel<false>, grid, dim3(256), 0, s, j);
  return hipGetLastError();
}
