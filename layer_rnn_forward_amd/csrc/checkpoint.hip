// 8-bit checkpoints of a matrix (gfx950): groups of 32 columns of a row share
// a power of two 2^e, e = exponent of the group's largest magnitude - 6 (so
// that it lands in [64, 128) units), at least -126; values are whole numbers
// of units within -127 .. 127.  Both scalings are by powers of two, so the
// only rounding is the one to whole units (ties to even), and what is read
// back has at most 7 significant bits: exact in fp32 and in bf16.
//
// One lane per value, 32 lanes per group.
#include <type_traits>

#include "lm_math.h"

using namespace rnnk;

namespace {

constexpr int kNanGroup = -128;   // exponent byte of a group that holds an infinity or a NaN

template <bool BF16>
__global__ __launch_bounds__(256) void store_kernel(int rows, int cols, const void* xv, int8_t* q, int8_t* ex) {
  const int gpr = (cols + kGroup - 1) / kGroup;
  const long long groups = (long long)rows * gpr;
  const long long step = (long long)gridDim.x * 8;
  for (long long k = (long long)blockIdx.x * 8 + threadIdx.x / kGroup; k < groups; k += step) {
    const long long r = k / gpr;
    const int c = (int)(k - r * gpr) * kGroup + threadIdx.x % kGroup;
    const float v = c < cols ? el_load<BF16>((const El<BF16>*)xv + r * cols + c) : 0.f;
    // magnitudes order like their bit patterns, infinities and NaNs on top
    unsigned top = __float_as_uint(v) & 0x7fffffffu;
    for (int o = 16; o; o >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, o, 32));
    const int e = max((int)(top >> 23) - 133, -126);
    const float x = rintf(v * __uint_as_float((unsigned)(127 - e) << 23));
    const bool bad = top >= 0x7f800000u;
    if (c < cols) q[r * cols + c] = bad ? 0 : (int8_t)fminf(fmaxf(x, -127.f), 127.f);
    if (threadIdx.x % kGroup == 0) ex[k] = bad ? kNanGroup : (int8_t)e;
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void load_kernel(int rows, int cols, const int8_t* q, const int8_t* ex, void* xv,
                                                   long long ld) {
  const int gpr = (cols + kGroup - 1) / kGroup;
  const long long groups = (long long)rows * gpr;
  const long long step = (long long)gridDim.x * 8;
  for (long long k = (long long)blockIdx.x * 8 + threadIdx.x / kGroup; k < groups; k += step) {
    const long long r = k / gpr;
    const int c = (int)(k - r * gpr) * kGroup + threadIdx.x % kGroup;
    const int e = ex[k];
    if (c < cols) {
      const float v = e == kNanGroup ? __uint_as_float(0x7fc00000u)
                                     : (float)q[r * cols + c] * __uint_as_float((unsigned)(127 + e) << 23);
      el_store<BF16>((El<BF16>*)xv + r * ld + c, v);
    } else if (c < ld) {
      el_store<BF16>((El<BF16>*)xv + r * ld + c, 0.f);
    }
  }
}

int grid_for(int rows, int cols) {
  const long long groups = (long long)rows * ((cols + kGroup - 1) / kGroup);
  return (int)std::min<long long>((groups + 7) / 8, 256LL * 32);
}

}  // namespace

hipError_t rnn_launch_ckpt_store(int bf16, int rows, int cols, const void* x, void* kept, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  int8_t* q = (int8_t*)kept;
  int8_t* ex = q + (long long)rows * cols;
  const dim3 grid(grid_for(rows, cols));
  if (bf16) hipLaunchKernelGGL(store_kernel<true>, grid, dim3(256), 0, s, rows, cols, x, q, ex);
  else hipLaunchKernelGGL(store_kernel<false>, grid, dim3(256), 0, s, rows, cols, x, q, ex);
  return hipGetLastError();
}

hipError_t rnn_launch_ckpt_load(int bf16, int rows, int cols, const void* kept, void* x, long long ld, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const int8_t* q = (const int8_t*)kept;
  const int8_t* ex = q + (long long)rows * cols;
  const dim3 grid(grid_for(rows, cols));
  if (bf16) hipLaunchKernelGGL(load_kernel<true>, grid, dim3(256), 0, s, rows, cols, q, ex, x, ld);
  else hipLaunchKernelGGL(load_kernel<false>, grid, dim3(256), 0, s, rows, cols, q, ex, x, ld);
  return hipGetLastError();
}
