// Products and activations of the gated feed-forward block (gfx950).
//
// mat_kernel: one 64 x 64 tile per workgroup, staged through LDS as fp32;
// any strides.
#include <algorithm>
#include <type_traits>

#include "lm_math.h"

using namespace rnnk;

namespace {

template <bool AB, bool BB, bool CB>
__global__ __launch_bounds__(256) void mat_kernel(const MatParams p) {
  __shared__ float as[16][65], bs[16][65];
  const El<AB>* A = (const El<AB>*)p.A;
  const El<BB>* B = (const El<BB>*)p.B;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tid = threadIdx.x, tm = tid / 16 * 4, tn = tid % 16 * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += 16) {
    for (int i = tid; i < 64 * 16; i += 256) {
      // the operand's contiguous axis along the lanes
      const int ra = p.sak == 1 ? i / 16 : i % 64, ka = p.sak == 1 ? i % 16 : i / 64;
      const int rb = p.sbk == 1 ? i / 16 : i % 64, kb = p.sbk == 1 ? i % 16 : i / 64;
      as[ka][ra] = m0 + ra < p.M && k0 + ka < p.K ? el_load<AB>(A + (m0 + ra) * p.sam + (k0 + ka) * p.sak) : 0.f;
      bs[kb][rb] = n0 + rb < p.N && k0 + kb < p.K ? el_load<BB>(B + (n0 + rb) * p.sbn + (k0 + kb) * p.sbk) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][tm + i], bs[k][tn + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j)
      if (m0 + tm + i < p.M && n0 + tn + j < p.N)
        el_store<CB>((El<CB>*)p.C + (m0 + tm + i) * p.ldc + n0 + tn + j, acc[i][j]);
}

template <bool BF16, int ACT>
__global__ __launch_bounds__(256) void act_kernel(int M, int F, const float* gu, void* h) {
  const long long n = (long long)M * F;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long m = i / F, f = i - m * F;
    float a, da;
    act_pair<ACT>(gu[m * 2 * F + f], a, da);
    el_store<BF16>((El<BF16>*)h + i, a * gu[m * 2 * F + F + f]);
  }
}

template <bool BF16, int ACT>
__global__ __launch_bounds__(256) void act_bwd_kernel(int M, int F, const float* gu, const float* dh, void* dgu) {
  const long long n = (long long)M * F;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long m = i / F, f = i - m * F;
    float a, da;
    act_pair<ACT>(gu[m * 2 * F + f], a, da);
    el_store<BF16>((El<BF16>*)dgu + m * 2 * F + f, dh[i] * gu[m * 2 * F + F + f] * da);
    el_store<BF16>((El<BF16>*)dgu + m * 2 * F + F + f, dh[i] * a);
  }
}

unsigned flat_grid(long long n) { return (unsigned)std::min<long long>((n + 255) / 256, 256LL * 32); }

}  // namespace

hipError_t rnn_launch_mat(const MatParams& p, int a_bf16, int b_bf16, int c_bf16, hipStream_t s) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  const dim3 grid((p.N + 63) / 64, (p.M + 63) / 64);
  if (a_bf16 && b_bf16 && c_bf16) hipLaunchKernelGGL((mat_kernel<true, true, true>), grid, dim3(256), 0, s, p);
  else if (a_bf16 && b_bf16) hipLaunchKernelGGL((mat_kernel<true, true, false>), grid, dim3(256), 0, s, p);
  else if (!a_bf16 && !b_bf16 && !c_bf16) hipLaunchKernelGGL((mat_kernel<false, false, false>), grid, dim3(256), 0, s, p);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

#define ACT_PICK(KERNEL, ...)                                                                                  \
  do {                                                                                                         \
    const dim3 grid(flat_grid((long long)M * F));                                                              \
    if (M == 0 || F == 0) return hipSuccess;                                                                   \
    if (bf16 && act == ACT_SIGMOID) hipLaunchKernelGGL((KERNEL<true, ACT_SIGMOID>), grid, dim3(256), 0, s, __VA_ARGS__);  \
    else if (bf16 && act == ACT_SILU) hipLaunchKernelGGL((KERNEL<true, ACT_SILU>), grid, dim3(256), 0, s, __VA_ARGS__);   \
    else if (bf16) hipLaunchKernelGGL((KERNEL<true, ACT_GELU>), grid, dim3(256), 0, s, __VA_ARGS__);            \
    else if (act == ACT_SIGMOID) hipLaunchKernelGGL((KERNEL<false, ACT_SIGMOID>), grid, dim3(256), 0, s, __VA_ARGS__);    \
    else if (act == ACT_SILU) hipLaunchKernelGGL((KERNEL<false, ACT_SILU>), grid, dim3(256), 0, s, __VA_ARGS__);          \
    else hipLaunchKernelGGL((KERNEL<false, ACT_GELU>), grid, dim3(256), 0, s, __VA_ARGS__);                     \
  } while (0)

hipError_t rnn_launch_act(int act, int bf16, int M, int F, const float* gu, void* h, hipStream_t s) {
  ACT_PICK(act_kernel, M, F, gu, h);
  return hipGetLastError();
}

hipError_t rnn_launch_act_bwd(int act, int bf16, int M, int F, const float* gu, const float* dh, void* dgu,
                              hipStream_t s) {
  ACT_PICK(act_bwd_kernel, M, F, gu, dh, dgu);
  return hipGetLastError();
}
