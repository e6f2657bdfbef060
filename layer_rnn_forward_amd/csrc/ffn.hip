// Launches of the gated feed-forward block's products (ffn_gemm.h), and the
// copy that pads rows which are not whole 16-byte pieces.
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

template <bool BF, bool AROWS, bool BROWS, int MT, int NT, int EPI, int SAVE, int OCC>
hipError_t launch(const FfnGemm& p, hipStream_t s) {
  constexpr int FN = EPI == FFN_GLU ? 32 * NT : 64 * NT;
  const long long tiles = ((p.M + 64LL * MT - 1) / (64 * MT)) * ((p.N + FN - 1LL) / FN);
  if (tiles > 0x7ffffff0LL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((ffn_gemm_kernel<BF, AROWS, BROWS, MT, NT, EPI, SAVE, OCC>), dim3((unsigned)((tiles + 7) / 8 * 8)),
                     dim3(256), 0, s, p);
  return hipGetLastError();
}

// 256 x 256 tiles, one workgroup per CU, where their rounds cost less than
// those of 128 x 128 tiles at two per CU
template <bool AROWS, bool BROWS, int EPI, int SAVE>
hipError_t pick(const FfnGemm& p, int bf16, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  if (!bf16) return launch<false, AROWS, BROWS, 2, 2, EPI, SAVE, 2>(p, s);
  const long long cols = EPI == FFN_GLU ? 2LL * p.N : p.N;
  const long long t256 = ((p.M + 255LL) / 256) * ((cols + 255) / 256), t128 = ((p.M + 127LL) / 128) * ((cols + 127) / 128);
  if (8 * ((t256 + 255) / 256) <= 5 * ((t128 + 511) / 512)) return launch<true, AROWS, BROWS, 4, 4, EPI, SAVE, 1>(p, s);
  return launch<true, AROWS, BROWS, 2, 2, EPI, SAVE, 2>(p, s);
}

}  // namespace

hipError_t rnn_launch_ffn_glu(const FfnGemm& p, int bf16, int save, hipStream_t s) {
  if (save == SAVE_NONE) return pick<true, true, FFN_GLU, SAVE_NONE>(p, bf16, s);
  if (save == SAVE_FULL) return pick<true, true, FFN_GLU, SAVE_FULL>(p, bf16, s);
  return pick<true, true, FFN_GLU, SAVE_INT8>(p, bf16, s);
}

hipError_t rnn_launch_ffn_dglu(const FfnGemm& p, int bf16, int save, hipStream_t s) {
  if (save == SAVE_FULL) return pick<true, false, FFN_DGLU, SAVE_FULL>(p, bf16, s);
  return pick<true, false, FFN_DGLU, SAVE_INT8>(p, bf16, s);
}

hipError_t rnn_launch_ffn_store(const FfnGemm& p, int bf16, int layout, hipStream_t s) {
  if (layout == 0) return pick<true, true, FFN_STORE, SAVE_NONE>(p, bf16, s);
  if (layout == 1) return pick<true, false, FFN_STORE, SAVE_NONE>(p, bf16, s);
  return pick<false, false, FFN_STORE, SAVE_NONE>(p, bf16, s);
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
