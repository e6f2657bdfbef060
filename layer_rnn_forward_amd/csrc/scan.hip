// Gated linear recurrence h_t = a_t h_(t-1) + b_t (gfx950).
//
// One thread per (direction, row, unit) walks the steps in order; the forward
// pass keeps every state in the workspace for the backward pass.
#include <type_traits>

#include "lm_math.h"

using namespace rnnk;

namespace {

template <int MODE>
__device__ __forceinline__ void coeffs(float p, float q, float& a, float& na, float& n) {
  if constexpr (MODE == SCAN_GATED) {
    sigmoid_pair(p, a, na);
    n = tanhf_(q);
  } else {
    a = p;
    na = 1.f;
    n = q;
  }
}

template <bool BF16, int MODE>
__global__ __launch_bounds__(256) void step_kernel(int B, int H, const void* gv, const float* h, void* yv, float* hy) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)B * H) return;
  const int b = (int)(i / H), u = (int)(i - (long long)b * H);
  const El<BF16>* g = (const El<BF16>*)gv + (long long)b * 2 * H + u;
  float a, na, n;
  coeffs<MODE>(el_load<BF16>(g), el_load<BF16>(g + H), a, na, n);
  const float v = fmaf(a, h ? h[i] : 0.f, na * n);
  if (yv) el_store<BF16>((El<BF16>*)yv + i, v);
  hy[i] = v;
}

template <bool BF16, int MODE>
__global__ __launch_bounds__(64) void fwd_kernel(const ScanParams p) {
  const long long C = (long long)p.D * p.B * p.H;
  const long long c = (long long)blockIdx.x * 64 + threadIdx.x;
  if (c >= C) return;
  const int u = (int)(c % p.H), b = (int)(c / p.H % p.B), d = (int)(c / ((long long)p.H * p.B));
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
  const El<BF16>* g = (const El<BF16>*)p.g;
  El<BF16>* y = (El<BF16>*)p.y;
  float h = p.h0 ? p.h0[c] : 0.f;
  for (int i = 0; i < p.T; ++i) {
    const int t = d ? p.T - 1 - i : i;
    const long long row = ((long long)t * p.B + b) * p.D + d;
    float out = 0.f;
    if (t < len) {
      float a, na, n;
      coeffs<MODE>(el_load<BF16>(g + row * 2 * p.H + u), el_load<BF16>(g + row * 2 * p.H + p.H + u), a, na, n);
      if (p.states) p.states[i * C + c] = h;
      out = h = fmaf(a, h, na * n);
    }
    el_store<BF16>(y + row * p.H + u, out);
  }
  if (p.hy) p.hy[c] = h;
}

template <bool BF16, int MODE>
__global__ __launch_bounds__(64) void bwd_kernel(const ScanParams p) {
  const long long C = (long long)p.D * p.B * p.H;
  const long long c = (long long)blockIdx.x * 64 + threadIdx.x;
  if (c >= C) return;
  const int u = (int)(c % p.H), b = (int)(c / p.H % p.B), d = (int)(c / ((long long)p.H * p.B));
  const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
  const El<BF16>* g = (const El<BF16>*)p.g;
  const El<BF16>* dy = (const El<BF16>*)p.dy;
  El<BF16>* dg = (El<BF16>*)p.dg;
  float dh = p.dhy ? p.dhy[c] : 0.f;
  for (int i = p.T - 1; i >= 0; --i) {
    const int t = d ? p.T - 1 - i : i;
    const long long row = ((long long)t * p.B + b) * p.D + d;
    float dp = 0.f, dq = 0.f;
    if (t < len) {
      float a, na, n;
      coeffs<MODE>(el_load<BF16>(g + row * 2 * p.H + u), el_load<BF16>(g + row * 2 * p.H + p.H + u), a, na, n);
      dh += el_load<BF16>(dy + row * p.H + u);
      const float before = p.states[i * C + c];
      if constexpr (MODE == SCAN_GATED) {
        dp = dh * (before - n) * a * na;
        dq = dh * na * (1.f - n * n);
      } else {
        dp = dh * before;
        dq = dh;
      }
      dh *= a;
    }
    el_store<BF16>(dg + row * 2 * p.H + u, dp);
    el_store<BF16>(dg + row * 2 * p.H + p.H + u, dq);
  }
  if (p.dh0) p.dh0[c] = dh;
}

}  // namespace

#define SCAN_PICK(KERNEL, GRID, BLOCK, ...)                                                              \
  do {                                                                                                   \
    if (bf16 && mode == SCAN_GATED) hipLaunchKernelGGL((KERNEL<true, SCAN_GATED>), GRID, BLOCK, 0, s, __VA_ARGS__); \
    else if (bf16) hipLaunchKernelGGL((KERNEL<true, SCAN_LINEAR>), GRID, BLOCK, 0, s, __VA_ARGS__);      \
    else if (mode == SCAN_GATED) hipLaunchKernelGGL((KERNEL<false, SCAN_GATED>), GRID, BLOCK, 0, s, __VA_ARGS__); \
    else hipLaunchKernelGGL((KERNEL<false, SCAN_LINEAR>), GRID, BLOCK, 0, s, __VA_ARGS__);               \
  } while (0)

hipError_t rnn_launch_scan_step(int mode, int bf16, int B, int H, const void* g, const float* h, void* y, float* hy,
                                hipStream_t s) {
  const long long n = (long long)B * H;
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)((n + 255) / 256));
  SCAN_PICK(step_kernel, grid, dim3(256), B, H, g, h, y, hy);
  return hipGetLastError();
}

hipError_t rnn_launch_scan_fwd(const ScanParams& p, int mode, int bf16, hipStream_t s) {
  const long long C = (long long)p.D * p.B * p.H;
  if (C == 0) return hipSuccess;
  SCAN_PICK(fwd_kernel, dim3((unsigned)((C + 63) / 64)), dim3(64), p);
  return hipGetLastError();
}

hipError_t rnn_launch_scan_bwd(const ScanParams& p, int mode, int bf16, hipStream_t s) {
  const long long C = (long long)p.D * p.B * p.H;
  if (C == 0) return hipSuccess;
  SCAN_PICK(bwd_kernel, dim3((unsigned)((C + 63) / 64)), dim3(64), p);
  return hipGetLastError();
}
