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

// The three products of the backward pass that are left once dgate and dup are
// there, in one launch: their tiles fill the CUs together, where each alone
// leaves part of its last round empty.
struct Grads {
  FfnGemm dx, dw_in, dw_out;
  int begin[3], blocks[3];
};
template <bool BF, int T, int OCC>
__global__ __launch_bounds__(256, OCC) void grads_kernel(const Grads g) {
  __shared__ __attribute__((aligned(1024))) char smem[ffn_lds<BF, T, T>()];
  const int b = (int)blockIdx.x;
  if (b >= g.begin[0] && b < g.begin[0] + g.blocks[0]) {
    ffn_product<BF, true, false, T, T, FFN_STORE, SAVE_NONE, 0>(g.dx, smem, b - g.begin[0], g.blocks[0]);
  } else {
    const bool in = b >= g.begin[1] && b < g.begin[1] + g.blocks[1];
    const FfnGemm p = in ? g.dw_in : g.dw_out;
    ffn_product<BF, false, false, T, T, FFN_STORE, SAVE_NONE, 0>(p, smem, b - g.begin[in ? 1 : 2], g.blocks[in ? 1 : 2]);
  }
}

}  // namespace

hipError_t rnn_launch_ffn_store(const FfnGemm& p, int bf16, hipStream_t s) {
  return ffn_pick<true, true, FFN_STORE, SAVE_NONE, 0>(p, bf16, s);
}

hipError_t rnn_launch_ffn_grads(const FfnGemm& dx, const FfnGemm& dw_in, const FfnGemm& dw_out, int bf16, hipStream_t s) {
  const FfnGemm* all[3] = {&dx, &dw_in, &dw_out};
  Grads g{dx, dw_in, dw_out, {}, {}};
  int order[3] = {0, 1, 2};   // the longest tiles first
  if (ffn_steps(dx, bf16) < ffn_steps(dw_in, bf16)) order[0] = 1, order[1] = 2, order[2] = 0;
  const FfnGemm* sorted[3] = {all[order[0]], all[order[1]], all[order[2]]};
  const int tile = ffn_tile(sorted, 3, bf16, false);
  long long at = 0;
  for (int i : order) {
    const long long blocks = (ffn_tiles(*all[i], tile, false) + 7) / 8 * 8;
    if (at + blocks > 0x7ffffff0LL) return hipErrorInvalidValue;
    g.begin[i] = (int)at;
    g.blocks[i] = (int)blocks;
    at += blocks;
  }
  if (at == 0) return hipSuccess;
  const dim3 grid((unsigned)at), block(256);
  if (!bf16) {
    if (tile == TILE_128) hipLaunchKernelGGL((grads_kernel<false, 2, 2>), grid, block, 0, s, g);
    else hipLaunchKernelGGL((grads_kernel<false, 1, 3>), grid, block, 0, s, g);
  } else if (tile == TILE_256) {
    hipLaunchKernelGGL((grads_kernel<true, 4, 1>), grid, block, 0, s, g);
  } else if (tile == TILE_128) {
    hipLaunchKernelGGL((grads_kernel<true, 2, 2>), grid, block, 0, s, g);
  } else {
    hipLaunchKernelGGL((grads_kernel<true, 1, 3>), grid, block, 0, s, g);
  }
  return hipGetLastError();
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
