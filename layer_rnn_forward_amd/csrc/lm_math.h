// Activations and elements of the language-model operators (gfx950).
#pragma once

#include <type_traits>

#include "device_util.h"
#include "lm_common.h"

namespace rnnk {

template <bool BF16>
using El = typename std::conditional<BF16, uint16_t, float>::type;

template <bool BF16>
__device__ __forceinline__ float el_load(const El<BF16>* p) {
  if constexpr (BF16) return bf2f(*p); else return *p;
}
template <bool BF16>
__device__ __forceinline__ void el_store(El<BF16>* p, float v) {
  if constexpr (BF16) *p = f2bf(v); else *p = v;
}

// N bytes at any address (global loads and stores take 16 bytes at any alignment)
template <int N>
struct __attribute__((packed, aligned(1))) Bytes {
  uint32_t w[N / 4];
};

// sigmoid(p) and sigmoid(-p) from e = exp(-|p|) <= 1: 1/(1+e) is the larger
// of the two and e/(1+e) the smaller, so neither cancels nor overflows.
__device__ __forceinline__ void sigmoid_pair(float p, float& pos, float& neg) {
  const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(p));
  const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
  pos = p >= 0.f ? big : small;
  neg = p >= 0.f ? small : big;
}

// act(g) and its derivative.
template <int ACT>
__device__ __forceinline__ void act_pair(float g, float& a, float& da) {
  if constexpr (ACT == ACT_GELU) {
    constexpr float c = 0.7978845608028654f;   // sqrt(2 / pi)
    const float g2 = g * g;
    const float t = tanhf_(c * (g + 0.044715f * g2 * g));
    a = 0.5f * g * (1.f + t);
    da = 0.5f * (1.f + t) + 0.5f * g * (1.f - t * t) * c * (1.f + 0.134145f * g2);
  } else {
    float s, n;
    sigmoid_pair(g, s, n);
    if constexpr (ACT == ACT_SIGMOID) {
      a = s;
      da = s * n;
    } else {
      a = g * s;
      da = s + g * s * n;
    }
  }
}

__device__ __forceinline__ float act_of(int act, float g) {
  float a, da;
  if (act == ACT_SILU) act_pair<ACT_SILU>(g, a, da);
  else if (act == ACT_GELU) act_pair<ACT_GELU>(g, a, da);
  else act_pair<ACT_SIGMOID>(g, a, da);
  return a;
}

}  // namespace rnnk
