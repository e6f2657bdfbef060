// Gated linear recurrence h_t = a_t h_(t-1) + b_t (gfx950): one pass over the
// gates, with the time axis split among workgroups.
//
// The steps s .. e of one channel compose to h_e = A h_(s-1) + B, and two such
// maps compose to (A2 A1, A2 B1 + B2).  A lane holds VW neighbouring channels
// over 16 steps (forward) or 8 (backward) in registers, as coefficients in 32
// bits, so the gates are read once; the waves of a workgroup hold consecutive
// pieces of one chunk.  Each wave composes its piece, the first wave the
// chunk; it publishes the chunk's (A, B), waits for what precedes it, and the
// waves then walk their pieces from the true state.  Only the first chunk reads
// the caller's state, and publishes it: the last may write over it.
//
// What precedes a chunk is the state before its group of SUPER chunks,
// followed by the maps of the group's chunks before it.  Every chunk composes
// those in order, and the last chunk of a group publishes the state that its
// successors start from: the sequence of roundings never depends on which
// chunk came first, and a sequence of N chunks waits N / SUPER times in a row
// instead of N.  A workgroup takes its chunk from its channels' counter, in
// walking order, so everything a chunk waits for is done or running (one
// counter for all workgroups cost 20 % of a pass over 2048 steps).
//
// A map can leave fp32's range although no state does: linear steps with
// |a| > 1, or a small product that a large state makes count.  Maps mark the
// first (A is NaN); strays() finds the second from the state that the map is
// applied to.  Such a chunk is walked piece after piece from its state, for the
// channels that need it; a chunk whose map is not clean (no number, or small)
// also publishes the state after it, for those that cannot use the map.  (The
// checks cost 2 - 3 % of a pass that needs none of it; 2048 steps of 8 rows of
// 1024 that grow and are reset: forward 0.076, backward 0.126 ms.)
//
// Published words are their own flags: a kernel sets them beforehand to a
// pattern that no published value has (kUnset, a NaN pattern replaced by
// another NaN when a result has it), so a wait costs one round trip.  Waits
// are bounded; one that expires sets its pass's word at the workspace's start
// and carries on with NaN.
//
// The backward pass is the same recurrence walked the other way
// (D_(t-1) = a_t (dy_t + D_t)).  It composes the states again from the gates
// and the state before every 8th step, which the forward pass leaves in the
// workspace: 0.5 bytes a value instead of 4 for the states themselves.
//
// Bound: 6 (forward) and 10.5 (backward) bytes a value in bf16 against about
// 39 and 59 issue slots of vector work (exponentials and reciprocals count
// four), which is 0.5 to 0.8 of the memory's time; waves that wait for each
// other leave the two overlapped in part.  65536 steps of 1760 channels in
// bf16: forward 0.21 ms, backward 0.34 ms (3.4 and 3.6 TB/s); 2048 steps of 8
// rows of 1024: 0.031 and 0.042 ms.  One thread per channel that walks every
// step took 96 ms and 2.7 ms for both passes.  Measured against the split
// used (forward 16 steps x 8 waves in groups of 8, backward 8 x 8 in groups
// of 4; forward / backward ms of the long case): 4 waves 0.24 / 0.37, 8 steps
// forward 0.25, 16 steps backward 0.36, groups of 16 0.23 / 0.39, of 32
// backward 0.48.
// Workgroups that stay and load the next chunk while one waits and is walked:
// forward 0.33 ms at best (the next chunk's registers halve what a CU holds).
#include <algorithm>
#include <type_traits>

#include "lm_math.h"
#include "recurrent_util.h"

using namespace rnnk;

// sums and products are fused where fmaf says so and nowhere else, so that the
// variants of one kernel round alike
#pragma clang fp contract(off)

namespace {

constexpr unsigned kUnset = 0xffffffffu;

template <bool BF, int VW>
struct Vec {
  static_assert(VW == 1 || BF, "");
  using T = typename std::conditional<BF, typename std::conditional<VW == 2, uint32_t, uint16_t>::type, float>::type;
  static __device__ __forceinline__ void get(const T& v, float (&o)[VW]) {
    if constexpr (BF && VW == 2) {
      o[0] = __uint_as_float(v << 16);
      o[1] = __uint_as_float(v & 0xffff0000u);
    } else if constexpr (BF) {
      o[0] = bf2f(v);
    } else {
      o[0] = v;
    }
  }
  static __device__ __forceinline__ T make(const float (&o)[VW]) {
    if constexpr (BF && VW == 2) return pack2bf(o[0], o[1]);
    else if constexpr (BF) return f2bf(o[0]);
    else return o[0];
  }
};

// a, 1 - a, the candidate n of a gated step and its slope 1 - n^2.  1 - a from
// the same exponential (no cancellation); tanh from one exponential
// t = e^(-2|q|), and from its series q - q^3/3 + 2q^5/15 below 1/16, where 1 - t
// would cancel (both are within 12 units in the last place); the slope as
// 4 t / (1 + t)^2 (1 - n^2 has lost all its digits at |q| = 9).
__device__ __forceinline__ void gate(float p, float q, float& a, float& na, float& n, float& slope) {
  const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(p));
  const float x = fabsf(q), t = __builtin_amdgcn_exp2f(-2.8853900817779268f * x);
  const float e1 = 1.f + e, t1 = 1.f + t, r = __builtin_amdgcn_rcpf(e1 * t1);
  const float big = r * t1, small = e * big, rt = r * e1;
  a = p >= 0.f ? big : small;
  na = p >= 0.f ? small : big;
  const float far = (1.f - t) * rt;
  const float z = q * q, near = fmaf(x * z, fmaf(z, 2.f / 15.f, -1.f / 3.f), x);
  n = copysignf(x < 0.0625f ? near : far, q);
  slope = 4.f * t * (rt * rt);
}

template <int MODE>
__device__ __forceinline__ void coeffs(float p, float q, float& a, float& na, float& n, float& slope) {
  if constexpr (MODE == SCAN_GATED) {
    gate(p, q, a, na, n, slope);
  } else {
    a = p;
    na = 1.f;
    n = q;
    slope = 1.f;
  }
}

// A map (A, B) stands for the steps it was composed from unless A or B left
// fp32's range (steps with |a| > 1; A is then NaN), or what an A near the
// bottom of the range has lost, up to 2^-142, times h would count in
// r = A h + B.
__device__ __forceinline__ bool clean(float A) { return fabsf(A) >= 0x1p-102f; }
__device__ __forceinline__ bool strays(float h, float r) { return !(fabsf(r) >= fabsf(h) * 0x1p-118f); }
// `low`: the smallest product on the way, `grew`: whether a coefficient was
// above 1; growth after such a loss carries it further
__device__ __forceinline__ float mark(float A, float B, bool grew, float low) {
  return __builtin_isfinite(A) && __builtin_isfinite(B) && !(grew && low < 0x1p-102f) ? A : __uint_as_float(0x7fc00000u);
}

__device__ __forceinline__ unsigned word(float v) {
  const unsigned u = __float_as_uint(v);
  return u == kUnset ? 0x7fffffffu : u;
}
__device__ __forceinline__ void publish(float* p, float v) { flag_store(reinterpret_cast<unsigned*>(p), word(v)); }
__device__ __forceinline__ unsigned peek(const float* p) { return flag_load(reinterpret_cast<const unsigned*>(p)); }
// a map (A, B) is one 8-byte word, A in its lower half
__device__ __forceinline__ void publish2(unsigned long long* p, float A, float B) {
  __hip_atomic_store(p, word(A) | (unsigned long long)word(B) << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long peek2(const unsigned long long* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool BF16, int MODE>
__global__ __launch_bounds__(256) void step_kernel(int B, int H, const void* gv, const float* h, void* yv, float* hy) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= (long long)B * H) return;
  const int b = (int)(i / H), u = (int)(i - (long long)b * H);
  const El<BF16>* g = (const El<BF16>*)gv + (long long)b * 2 * H + u;
  float a, na, n, slope;
  coeffs<MODE>(el_load<BF16>(g), el_load<BF16>(g + H), a, na, n, slope);
  const float v = fmaf(a, h ? h[i] : 0.f, na * n);
  if (yv) el_store<BF16>((El<BF16>*)yv + i, v);
  hy[i] = v;
}

// Words for waits that expired: forward's, then backward's.  A forward pass
// clears both, a backward pass its own: what forward noted stays to be read
// after the step.
template <bool BACK>
__device__ __forceinline__ void clear_expired(unsigned* head) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (!BACK) head[0] = 0;
    head[1] = 0;
  }
}

// counters to zero, published words to kUnset, 16 bytes a lane
template <bool BACK>
__global__ __launch_bounds__(256) void clear_kernel(unsigned* head, long long counters, long long all) {
  clear_expired<BACK>(head);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
    const unsigned v = i < counters ? 0u : kUnset;
    reinterpret_cast<uint4*>(head + 64)[i] = make_uint4(v, v, v, v);
  }
}

// Read `count` words at once, and those again that were unset.
template <bool BACK, int N, int VW, class Load, class Word>
__device__ __forceinline__ void wait_words(const ScanParams& p, int count, Word (&v)[N][VW], Load load) {
  unsigned need = (1u << count) - 1u;
  for (int spin = 0; need; ++spin) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (need >> j & 1)
#pragma unroll
        for (int e = 0; e < VW; ++e) v[j][e] = load(j, e);
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (need >> j & 1) {
        bool ok = true;
#pragma unroll
        for (int e = 0; e < VW; ++e) ok &= (unsigned)v[j][e] != kUnset;
        if (__all(ok)) need &= ~(1u << j);
      }
    if (!need) break;
    if (spin >= p.spin_limit) {
      flag_store(p.head + BACK, 1u);
      break;                             // the unset words are NaNs
    }
    __builtin_amdgcn_s_sleep(1);
  }
}

// The state that chunk `pos` (in walking order) starts from: the wave's VW
// channels at `c` of `C`.  The maps since the last published state are composed
// (A, B) first, then that state (s) is waited for.
template <bool BACK, int MODE, int VW, int SUPER>
__device__ __forceinline__ void wait_state(const ScanParams& p, int pos, long long C, long long c, bool live, float (&A)[VW],
                                           float (&B)[VW], float (&s)[VW]) {
  const int sup = pos / SUPER, n = pos - sup * SUPER;
  constexpr int N = 4;
  float low[VW];
  bool grew[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    low[e] = 1.f;
    grew[e] = false;
  }
  for (int j0 = 0; j0 < n; j0 += N) {
    unsigned long long m[N][VW];
    const unsigned long long* from = p.maps + (long long)(sup * SUPER + j0) * C + c;
    const int count = min(N, n - j0);
    wait_words<BACK, N, VW>(p, count, m, [&](int j, int e) { return live ? peek2(from + j * C + e) : 0ull; });
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < count)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const float a = __uint_as_float((unsigned)m[j][e]);
          A[e] *= a;
          B[e] = fmaf(a, B[e], __uint_as_float((unsigned)(m[j][e] >> 32)));
          if constexpr (MODE == SCAN_LINEAR) {
            grew[e] |= fabsf(a) > 1.f;
            low[e] = fminf(low[e], fabsf(A[e]));
          }
        }
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) A[e] = mark(A[e], B[e], grew[e], low[e]);
  unsigned u[1][VW];
  wait_words<BACK, 1, VW>(p, 1, u, [&](int, int e) { return live ? peek(p.state + (long long)sup * C + c + e) : 0u; });
#pragma unroll
  for (int e = 0; e < VW; ++e) s[e] = __uint_as_float(u[0][e]);
}

// For the channels `again`, whose composed maps stray: the chunks' maps once
// more, one after the other from the group's first state; a chunk whose map is
// not clean publishes the state after it, too.
template <bool BACK, int VW, int SUPER>
__device__ __forceinline__ void step_by_step(const ScanParams& p, int pos, long long C, long long c, const bool (&again)[VW],
                                             float (&h)[VW]) {
  const int sup = pos / SUPER, n = pos - sup * SUPER;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const long long at = (long long)(sup * SUPER + j) * C + c;
    bool wait[VW], any = false;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const unsigned long long m = again[e] ? peek2(p.maps + at + e) : 0ull;
      const float A = __uint_as_float((unsigned)m);
      wait[e] = again[e] && !clean(A);
      if (again[e]) h[e] = fmaf(A, h[e], __uint_as_float((unsigned)(m >> 32)));
      any |= wait[e];
    }
    if (!__any(any)) continue;
    unsigned u[1][VW];
    wait_words<BACK, 1, VW>(p, 1, u, [&](int, int e) { return wait[e] ? peek(p.ends + at + e) : 0u; });
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (wait[e]) h[e] = __uint_as_float(u[0][e]);
  }
}

// The chunk and channels of a workgroup.
struct Place {
  int pos;           // chunk, in walking order
  int d, c0;         // direction, first channel (of B * H)
};
template <bool BACK>
__device__ __forceinline__ Place place(const ScanParams& p, int VW, unsigned& shared) {
  const int per = (p.B * p.H + 64 * VW - 1) / (64 * VW), tile = (int)(blockIdx.x % (unsigned)(per * p.D));
  Place r;
  r.pos = 0;
  if (p.chunks > 1) {
    perturb_pause(wave_tag(), 0u, 3u);
    if (threadIdx.x == 0) shared = atomicAdd(p.counters + tile * 16LL, 1u);
    __syncthreads();
    r.pos = __builtin_amdgcn_readfirstlane(shared);
  } else {
    clear_expired<BACK>(p.head);
  }
  r.d = tile / per;
  r.c0 = (tile - r.d * per) * 64 * VW;
  return r;
}

// LDS of a workgroup's exchange: the waves' maps and whether one could stray,
// the state before the chunk (and, where the pieces are walked one after the
// other, before and after each), the lanes that need that
template <int VW, int MW>
struct Exchange {
  float A[MW][64 * VW], B[MW][64 * VW], h[MW + 1][64 * VW];
  unsigned risk[MW], any;
  unsigned long long slow[VW], out[VW];
};

// compose the waves' maps to the chunk's, find the state before the chunk,
// pass it on; returns the state before this wave's piece.  end(x): the state x
// before this wave's piece becomes the one after it.
template <bool BACK, int MODE, int VW, int SUPER, int MW, class End>
__device__ __forceinline__ void join(const ScanParams& p, int pos, long long C, long long c, bool live, const float* first,
                                     int wave, int lane, int W, Exchange<VW, MW>& x, const float (&A)[VW], const float (&B)[VW],
                                     float (&h)[VW], End end) {
  bool small = false;
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    x.A[wave][lane * VW + e] = A[e];
    x.B[wave][lane * VW + e] = B[e];
    small |= live && !clean(A[e]);
  }
  const bool risk = __any(small);
  if (lane == 0) x.risk[wave] = risk;
  __syncthreads();
  const bool ends = pos % SUPER == SUPER - 1, more = pos + 1 < p.chunks;
  if (wave == 0) {
    float tA[VW], tB[VW], low[VW];
    bool grew[VW];
    const bool look = __any(lane < W && x.risk[lane & (MW - 1)]);
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      tA[e] = A[e];
      tB[e] = B[e];
      low[e] = fabsf(A[e]);
      grew[e] = low[e] > 1.f;
    }
    for (int w = 1; w < W; ++w)
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float a = x.A[w][lane * VW + e];
        tA[e] *= a;
        tB[e] = fmaf(a, tB[e], x.B[w][lane * VW + e]);
        if constexpr (MODE == SCAN_LINEAR) {
          grew[e] |= fabsf(a) > 1.f;
          low[e] = fminf(low[e], fabsf(tA[e]));
        }
      }
#pragma unroll
    for (int e = 0; e < VW; ++e) tA[e] = mark(tA[e], tB[e], MODE == SCAN_LINEAR && grew[e], low[e]);
    perturb_pause(wave_tag(), pos, 4u);
    if (more && !ends && live)
#pragma unroll
      for (int e = 0; e < VW; ++e) publish2(p.maps + (long long)pos * C + c + e, tA[e], tB[e]);
    float gA[VW], gB[VW], s[VW], r[VW];
    bool unclean[VW], dirty = false;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      unclean[e] = live && more && !clean(tA[e]);
      dirty |= unclean[e];
      gA[e] = 1.f;
      gB[e] = 0.f;
      s[e] = 0.f;
    }
    if (pos == 0) {
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        if (first && live) s[e] = first[c + e];
        if (more && live) publish(p.state + c + e, s[e]);
      }
    }
    dirty = __any(dirty);
    if (pos > 0) wait_state<BACK, MODE, VW, SUPER>(p, pos, C, c, live, gA, gB, s);
    perturb_pause(wave_tag(), pos, 5u);
    float* const next = (ends ? p.state + (long long)(pos / SUPER + 1) * C : p.ends + (long long)pos * C) + c;
    bool again[VW], out[VW] = {}, any = false;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      h[e] = fmaf(gA[e], s[e], gB[e]);
      r[e] = fmaf(tA[e], h[e], tB[e]);
      again[e] = live && strays(s[e], h[e]);
      any |= again[e];
    }
    if (dirty) {
#pragma unroll
      for (int e = 0; e < VW; ++e) out[e] = unclean[e] && strays(h[e], r[e]);
    }
    // both channels' before the stores: a wait for the second's word among them would be one for the first's store
    if constexpr (VW == 2) asm volatile("" : "+v"(r[0]), "+v"(r[VW - 1]));
#pragma unroll
    for (int e = 0; e < VW; ++e)
      if (more && live && (ends || unclean[e]) && !again[e] && !out[e]) publish(next + e, r[e]);
    if (__builtin_expect(__any(any), 0)) {
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (again[e]) h[e] = s[e];
      step_by_step<BACK, VW, SUPER>(p, pos, C, c, again, h);
#pragma unroll
      for (int e = 0; e < VW; ++e)
        if (again[e]) {
          r[e] = fmaf(tA[e], h[e], tB[e]);
          out[e] = unclean[e] && strays(h[e], r[e]);
          if (more && (ends || unclean[e]) && !out[e]) publish(next + e, r[e]);
        }
    }
    any = false;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      x.h[0][lane * VW + e] = h[e];
      any |= out[e];
    }
    const bool slow = look || __any(any);
    if (lane == 0) x.any = slow;
    if (__builtin_expect(slow, 0)) {
      any = false;
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float v = h[e];
        bool walk = out[e];
#pragma unroll 1
        for (int w = 0; w < W - 1; ++w) {
          const float to = fmaf(x.A[w][lane * VW + e], v, x.B[w][lane * VW + e]);
          walk |= live && strays(v, to);
          v = to;
        }
        const unsigned long long mw = __ballot(walk), mo = __ballot(out[e]);
        any |= mw != 0;
        if (lane == 0) {
          x.slow[e] = mw;
          x.out[e] = mo;
        }
      }
      if (lane == 0) x.any = any;
    }
  }
  __syncthreads();
  const bool slow = x.any != 0;   // the same for every wave
#pragma unroll
  for (int e = 0; e < VW; ++e) h[e] = x.h[0][lane * VW + e];
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int e = 0; e < VW; ++e) h[e] = fmaf(x.A[w][lane * VW + e], h[e], x.B[w][lane * VW + e]);
  if (__builtin_expect(!slow, 1)) return;
#pragma unroll 1
  for (int w = 0; w < W; ++w) {
    if (w == wave) {
      float s[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        s[e] = x.h[w][lane * VW + e];
        if (x.slow[e] >> lane & 1) h[e] = s[e];
      }
      end(s);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        x.h[w + 1][lane * VW + e] = s[e];
        if (w == W - 1 && x.out[e] >> lane & 1)
          publish((ends ? p.state + (long long)(pos / SUPER + 1) * C : p.ends + (long long)pos * C) + c + e, s[e]);
      }
    }
    __syncthreads();
  }
}

// Where a lane's values lie in a step's row: the elements up to the
// workgroup's first channel are uniform (gbase, ybase), the bytes from there
// to the lane's p and y fit 32 bits.
struct Lanes {
  unsigned g, y;
  int b;             // batch row
  bool live;
};
template <bool BF, int VW>
__device__ __forceinline__ void lanes(const ScanParams& p, const Place& at, int lane, long long& gbase, long long& ybase,
                                      Lanes& l) {
  constexpr int ES = BF ? 2 : 4;
  const int BH = p.B * p.H;
  int c = at.c0 + lane * VW;
  l.live = c < BH;
  if (!l.live) c = at.c0;                     // reads what the first lane reads, writes nothing
  l.b = c / p.H;
  const int b0 = at.c0 / p.H, u0 = at.c0 - b0 * p.H;
  ybase = ((long long)b0 * p.D + at.d) * p.H + u0;
  gbase = ((long long)b0 * p.D + at.d) * 2 * p.H + u0;
  const long long y = ((long long)l.b * p.D + at.d) * p.H + (c - l.b * p.H);
  const long long g = ((long long)l.b * p.D + at.d) * 2 * p.H + (c - l.b * p.H);
  l.y = (unsigned)((y - ybase) * ES);
  l.g = (unsigned)((g - gbase) * ES);
}

template <class T>
__device__ __forceinline__ T ld(const char* row, unsigned off) { return *reinterpret_cast<const T*>(row + off); }
template <class T>
__device__ __forceinline__ void st(char* row, unsigned off, T v) { *reinterpret_cast<T*>(row + off) = v; }

// mark() of a wave's map; whether a coefficient was above 1 is looked up only
// where a product came out small
template <int MODE, int G, int VW>
__device__ __forceinline__ void mark_piece(const float (&a)[G][VW], const float (&B)[VW], const float (&low)[VW], float (&A)[VW]) {
  bool grew[VW] = {}, small = false;
  if constexpr (MODE == SCAN_LINEAR) {
#pragma unroll
    for (int e = 0; e < VW; ++e) small |= low[e] < 0x1p-102f;
    if (__builtin_expect(__any(small), 0))
#pragma unroll
      for (int s = 0; s < G; ++s)
#pragma unroll
        for (int e = 0; e < VW; ++e) grew[e] |= fabsf(a[s][e]) > 1.f;
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) A[e] = mark(A[e], B[e], grew[e], low[e]);
}

template <bool BF, int MODE, int VW>
__global__ __launch_bounds__(64 * kScanFwdWaves, kScanFwdEu) void fwd_kernel(const ScanParams p) {
  using V = Vec<BF, VW>;
  using T = typename V::T;
  constexpr int ES = BF ? 2 : 4, G = kScanFwdSteps;
  __shared__ Exchange<VW, kScanFwdWaves> x;
  __shared__ unsigned shared;
  const Place at = place<false>(p, VW, shared);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
  const long long C = (long long)p.D * p.B * p.H;
  long long gbase, ybase;
  Lanes l;
  lanes<BF, VW>(p, at, lane, gbase, ybase, l);
  const long long c = (long long)at.d * p.B * p.H + at.c0 + lane * VW;
  const long long grow = (long long)p.B * p.D * 2 * p.H * ES, yrow = grow / 2;
  const char* g = (const char*)p.g + gbase * ES;
  char* y = (char*)p.y + ybase * ES;
  const int i0 = (at.pos * W + wave) * G;
  const long long half = (long long)p.H * ES;
  const int len = p.lengths ? min(max(p.lengths[l.b], 0), p.T) : p.T;
  const bool whole = !p.lengths && i0 + G <= p.T;

  T rp[G], rq[G];
#pragma unroll
  for (int s = 0; s < G; ++s) {
    const int i = min(i0 + s, p.T - 1), t = at.d ? p.T - 1 - i : i;
    const char* row = g + t * grow;
    rp[s] = ld<T>(row, l.g);
    rq[s] = ld<T>(row + half, l.g);
  }
  float a[G][VW], b[G][VW], A[VW], B[VW], h[VW], low[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    A[e] = low[e] = 1.f;
    B[e] = 0.f;
  }
  // WHOLE: every step of the piece belongs to every row; otherwise steps past
  // the sequence or the row are a = 1, b = 0 (they read a step that is there)
  auto compose = [&](auto w) {
    constexpr bool WHOLE = decltype(w)::value;
#pragma unroll
    for (int s = 0; s < G; ++s) {
      float vp[VW], vq[VW];
      V::get(rp[s], vp);
      V::get(rq[s], vq);
      const int i = i0 + s, t = at.d ? p.T - 1 - i : i;
      const bool valid = WHOLE || (i < p.T && t < len);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float na, n, slope;
        coeffs<MODE>(vp[e], vq[e], a[s][e], na, n, slope);
        b[s][e] = valid ? na * n : 0.f;
        if (!valid) a[s][e] = 1.f;
        A[e] *= a[s][e];
        B[e] = fmaf(a[s][e], B[e], b[s][e]);
        if constexpr (MODE == SCAN_LINEAR) low[e] = fminf(low[e], fabsf(A[e]));
      }
    }
  };
  if (whole) compose(std::true_type{});
  else compose(std::false_type{});
  mark_piece<MODE>(a, B, low, A);
  join<false, MODE, VW, kScanFwdSuper, kScanFwdWaves>(p, at.pos, C, c, l.live, p.h0, wave, lane, W, x, A, B, h, [&](float (&s)[VW]) {
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int e = 0; e < VW; ++e) s[e] = fmaf(a[i][e], s[e], b[i][e]);
  });
  if (!l.live) return;
  auto walk = [&](auto w) {
    constexpr bool WHOLE = decltype(w)::value;
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const int i = i0 + s, t = at.d ? p.T - 1 - i : i;
      if (s % kScanKeep == 0 && (WHOLE || i < p.T)) {
        float* kept = p.starts + (long long)(i / kScanKeep) * C + c;
#pragma unroll
        for (int e = 0; e < VW; ++e) kept[e] = h[e];
      }
      float o[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        h[e] = fmaf(a[s][e], h[e], b[s][e]);
        o[e] = WHOLE || t < len ? h[e] : 0.f;
      }
      if (WHOLE || i < p.T) st<T>(y + t * yrow, l.y, V::make(o));
    }
  };
  if (whole) walk(std::true_type{});
  else walk(std::false_type{});
  if (p.hy && at.pos == p.chunks - 1 && wave == W - 1)
#pragma unroll
    for (int e = 0; e < VW; ++e) p.hy[c + e] = h[e];
}

template <bool BF, int MODE, int VW>
__global__ __launch_bounds__(64 * kScanBwdWaves, kScanBwdEu) void bwd_kernel(const ScanParams p) {
  using V = Vec<BF, VW>;
  using T = typename V::T;
  constexpr int ES = BF ? 2 : 4, G = kScanBwdSteps;
  __shared__ Exchange<VW, kScanBwdWaves> x;
  __shared__ unsigned shared;
  const Place at = place<true>(p, VW, shared);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
  const long long C = (long long)p.D * p.B * p.H;
  long long gbase, ybase;
  Lanes l;
  lanes<BF, VW>(p, at, lane, gbase, ybase, l);
  const long long c = (long long)at.d * p.B * p.H + at.c0 + lane * VW;
  const long long grow = (long long)p.B * p.D * 2 * p.H * ES, yrow = grow / 2;
  const char* g = (const char*)p.g + gbase * ES;
  const char* dy = (const char*)p.dy + ybase * ES;
  char* dg = (char*)p.dg + gbase * ES;
  const long long half = (long long)p.H * ES;
  const int len = p.lengths ? min(max(p.lengths[l.b], 0), p.T) : p.T;
  // the first wave of the first chunk has the last steps
  const int piece = (p.chunks - 1 - at.pos) * W + (W - 1 - wave), i0 = piece * G;
  const bool whole = !p.lengths && i0 + G <= p.T;

  T rp[G], rq[G], rd[G];
  float h[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) h[e] = i0 < p.T && l.live ? p.starts[(long long)(i0 / kScanKeep) * C + c + e] : 0.f;
#pragma unroll
  for (int s = 0; s < G; ++s) {
    const int i = min(i0 + s, p.T - 1), t = at.d ? p.T - 1 - i : i;
    const char* row = g + t * grow;
    rp[s] = ld<T>(row, l.g);
    rq[s] = ld<T>(row + half, l.g);
    rd[s] = ld<T>(dy + t * yrow, l.y);
  }
  // a, dp = f (dy + D), dq = f2 (dy + D)
  float a[G][VW], f[G][VW], f2[G][VW], A[VW], B[VW], D[VW], low[VW];
  auto compose = [&](auto w) {
    constexpr bool WHOLE = decltype(w)::value;
#pragma unroll
    for (int s = 0; s < G; ++s) {
      float vp[VW], vq[VW];
      V::get(rp[s], vp);
      V::get(rq[s], vq);
      const int i = i0 + s, t = at.d ? p.T - 1 - i : i;
      const bool valid = WHOLE || (i < p.T && t < len);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        float na, n, slope;
        coeffs<MODE>(vp[e], vq[e], a[s][e], na, n, slope);
        if constexpr (MODE == SCAN_GATED) {
          f[s][e] = (h[e] - n) * (a[s][e] * na);
          f2[s][e] = na * slope;
        } else {
          f[s][e] = h[e];
          f2[s][e] = 1.f;
        }
        if (!valid) {
          a[s][e] = 1.f;
          f[s][e] = f2[s][e] = 0.f;
        }
        h[e] = fmaf(a[s][e], h[e], valid ? na * n : 0.f);
      }
      if (!valid) {
        float zero[VW] = {};
        rd[s] = V::make(zero);
      }
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      A[e] = a[G - 1][e];
      B[e] = 0.f;
      low[e] = fabsf(A[e]);
    }
    // B: dy + D of the step, D of nothing being 0
    V::get(rd[G - 1], B);
#pragma unroll
    for (int s = G - 2; s >= 0; --s) {
      float v[VW];
      V::get(rd[s], v);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        A[e] *= a[s][e];
        B[e] = fmaf(a[s + 1][e], B[e], v[e]);
        if constexpr (MODE == SCAN_LINEAR) low[e] = fminf(low[e], fabsf(A[e]));
      }
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) B[e] *= a[0][e];
  };
  if (whole) compose(std::true_type{});
  else compose(std::false_type{});
  mark_piece<MODE>(a, B, low, A);
  join<true, MODE, VW, kScanBwdSuper, kScanBwdWaves>(p, at.pos, C, c, l.live, p.dhy, wave, lane, W, x, A, B, D, [&](float (&s)[VW]) {
#pragma unroll
    for (int i = G - 1; i >= 0; --i) {
      float v[VW];
      V::get(rd[i], v);
#pragma unroll
      for (int e = 0; e < VW; ++e) s[e] = i == G - 1 ? s[e] + v[e] : fmaf(a[i == G - 1 ? i : i + 1][e], s[e], v[e]);
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) s[e] *= a[0][e];
  });
  if (!l.live) return;
  auto walk = [&](auto w) {
    constexpr bool WHOLE = decltype(w)::value;
#pragma unroll
    for (int s = G - 1; s >= 0; --s) {
      const int i = i0 + s, t = at.d ? p.T - 1 - i : i;
      float v[VW], op[VW], oq[VW];
      V::get(rd[s], v);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        D[e] = s == G - 1 ? D[e] + v[e] : fmaf(a[s == G - 1 ? s : s + 1][e], D[e], v[e]);
        const bool valid = WHOLE || t < len;
        op[e] = valid ? D[e] * f[s][e] : 0.f;    // D itself may be infinite or NaN
        oq[e] = valid ? D[e] * f2[s][e] : 0.f;
      }
      if (WHOLE || i < p.T) {
        char* row = dg + t * grow;
        st<T>(row, l.g, V::make(op));
        st<T>(row + half, l.g, V::make(oq));
      }
    }
  };
  if (whole) walk(std::true_type{});
  else walk(std::false_type{});
  if (p.dh0 && at.pos == p.chunks - 1 && wave == W - 1)
#pragma unroll
    for (int e = 0; e < VW; ++e) p.dh0[c + e] = a[0][e] * D[e];
}

// T == 0: the states pass through
template <bool BACK>
__global__ __launch_bounds__(256) void pass_kernel(unsigned* head, long long n, const float* from, float* to) {
  clear_expired<BACK>(head);
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (to && i < n) to[i] = from ? from[i] : 0.f;
}

template <bool BACK, bool BF, int MODE>
void start(const ScanParams& p, bool two, dim3 grid, dim3 block, hipStream_t s) {
  if constexpr (BACK) {
    if (BF && two) hipLaunchKernelGGL((bwd_kernel<BF, MODE, BF ? 2 : 1>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((bwd_kernel<BF, MODE, 1>), grid, block, 0, s, p);
  } else {
    if (BF && two) hipLaunchKernelGGL((fwd_kernel<BF, MODE, BF ? 2 : 1>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((fwd_kernel<BF, MODE, 1>), grid, block, 0, s, p);
  }
}

template <bool BACK>
hipError_t launch(const ScanParams& p, int mode, int bf16, hipStream_t s) {
  const long long C = (long long)p.D * p.B * p.H;
  if (C == 0) return hipSuccess;
  if (p.T == 0) {
    float* to = BACK ? p.dh0 : p.hy;
    hipLaunchKernelGGL(pass_kernel<BACK>, dim3((unsigned)((C + 255) / 256)), dim3(256), 0, s, p.head, C, BACK ? p.dhy : p.h0, to);
    return hipGetLastError();
  }
  // bf16: two channels (4 bytes) a lane where they never straddle two rows of
  // the batch and are aligned; fp32 has 4 bytes a lane with one
  const uintptr_t bases = (uintptr_t)p.g | (BACK ? (uintptr_t)p.dy | (uintptr_t)p.dg : (uintptr_t)p.y);
  const bool two = bf16 && p.H % 2 == 0 && (bases & 3) == 0;
  const long long BH = (long long)p.B * p.H, tiles = (BH + (two ? 127 : 63)) / (two ? 128 : 64) * p.D;
  if (tiles * p.chunks > 0x7fffffffLL) return hipErrorInvalidValue;
  if (p.chunks > 1) {
    const long long words = (3LL * p.chunks + p.chunks / (BACK ? kScanBwdSuper : kScanFwdSuper) + 1) * C;
    const long long counters = ((char*)p.maps - (char*)p.counters) / 16, all = counters + (words + 3) / 4;
    const dim3 grid((unsigned)std::min<long long>((all + 255) / 256, 2048));
    hipLaunchKernelGGL(clear_kernel<BACK>, grid, dim3(256), 0, s, p.head, counters, all);
  }
  const dim3 grid((unsigned)(tiles * p.chunks)), block(64 * p.waves);
  if (bf16 && mode == SCAN_GATED) start<BACK, true, SCAN_GATED>(p, two, grid, block, s);
  else if (bf16) start<BACK, true, SCAN_LINEAR>(p, two, grid, block, s);
  else if (mode == SCAN_GATED) start<BACK, false, SCAN_GATED>(p, two, grid, block, s);
  else start<BACK, false, SCAN_LINEAR>(p, two, grid, block, s);
  return hipGetLastError();
}

}  // namespace

hipError_t rnn_launch_scan_step(int mode, int bf16, int B, int H, const void* g, const float* h, void* y, float* hy,
                                hipStream_t s) {
  const long long n = (long long)B * H;
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)((n + 255) / 256)), block(256);
  if (bf16 && mode == SCAN_GATED) hipLaunchKernelGGL((step_kernel<true, SCAN_GATED>), grid, block, 0, s, B, H, g, h, y, hy);
  else if (bf16) hipLaunchKernelGGL((step_kernel<true, SCAN_LINEAR>), grid, block, 0, s, B, H, g, h, y, hy);
  else if (mode == SCAN_GATED) hipLaunchKernelGGL((step_kernel<false, SCAN_GATED>), grid, block, 0, s, B, H, g, h, y, hy);
  else hipLaunchKernelGGL((step_kernel<false, SCAN_LINEAR>), grid, block, 0, s, B, H, g, h, y, hy);
  return hipGetLastError();
}

hipError_t rnn_launch_scan_fwd(const ScanParams& p, int mode, int bf16, hipStream_t s) { return launch<false>(p, mode, bf16, s); }
hipError_t rnn_launch_scan_bwd(const ScanParams& p, int mode, int bf16, hipStream_t s) { return launch<true>(p, mode, bf16, s); }
