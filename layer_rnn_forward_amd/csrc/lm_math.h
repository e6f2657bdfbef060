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

// act(g) and its derivative.  silu(g) = g s(g) and, with 2z = 2 sqrt(2/pi)
// (g + 0.044715 g^3), gelu(g) = g (1 + tanh z) / 2 = g s(2z): one exponential
// and one reciprocal each.  (g s(w))' = s + g s (1 - s) w'.
template <int ACT>
__device__ __forceinline__ void act_pair(float g, float& a, float& da) {
  if constexpr (ACT == ACT_SIGMOID) {
    float n;
    sigmoid_pair(g, a, n);
    da = a * n;
  } else {
    constexpr float c = 1.5957691216057308f, c3 = c * 0.044715f, l = -1.4426950408889634f;   // c = 2 sqrt(2 / pi)
    float x = l * g, slope = 1.f;
    if constexpr (ACT == ACT_GELU) {
      const float g2 = fminf(g * g, 1e10f);   // beyond, s is 0 or 1 and the slope must not overflow
      x = fmaf(l * c3, g2, l * c) * g;
      slope = fmaf(3.f * c3, g2, c);
    }
    // x > 128: the exponential is infinite and s is 0, as it should be
    const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x));
    a = g * s;
    const float n = 1.f - s;
    da = fmaf(ACT == ACT_GELU ? slope * n : n, a, s);
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
