// Plain products of the gated feed-forward block (ffn_gemm.h), and the copy
// that pads rows which are not whole 16-byte pieces.
#include <algorithm>

#include "ffn_gemm.h"

using namespace rnnk;

namespace {

template <bool BF>
__global__ __launch_bounds__(256) void pad_kernel(const PadJob j) {
  const int z = blockIdx.z;
  const El<BF>* src = (const El<BF>*)j.src[z];
  El<BF>* dst = (El<BF>*)j.dst[z];
  const int cols = j.cols[z], ld = j.ld[z];
  const long long n = j.rows[z] * ld;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / ld;
    const int c = (int)(i - r * ld);
    dst[i] = c < cols ? src[r * cols + c] : (El<BF>)0;
  }
}

}  // namespace

hipError_t rnn_launch_ffn_store(const FfnGemm& p, int bf16, int layout, hipStream_t s) {
  if (layout == 0) return ffn_pick<true, true, FFN_STORE, SAVE_NONE, 0>(p, bf16, s);
  if (layout == 1) return ffn_pick<true, false, FFN_STORE, SAVE_NONE, 0>(p, bf16, s);
  return ffn_pick<false, false, FFN_STORE, SAVE_NONE, 0>(p, bf16, s);
}

hipError_t rnn_launch_pad(const PadJob& j, int bf16, hipStream_t s) {
  if (j.n == 0) return hipSuccess;
  long long n = 0;
  for (int i = 0; i < j.n; ++i) n = std::max(n, j.rows[i] * j.ld[i]);
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)std::min<long long>((n + 255) / 256, 256 * 16), 1, j.n);
  if (bf16) hipLaunchKernelGGL(pad_kernel<true>, grid, dim3(256), 0, s, j);
  else hipLaunchKernelGGL(pad_kernel<false>, grid, dim3(256), 0, s, j);
  return hipGetLastError();
}
