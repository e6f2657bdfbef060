// The MFMA product of the gated feed-forward block (gfx950).
//
//   C[m, n] = sum_k A(m, k) B(n, k)
//
// Each operand either has its k contiguous in memory ("rows": element (r, k)
// at r * ld + k) or its r ("columns": element (r, k) at k * ld + r), so that
// the same kernel makes x W^T (rows, rows), dy W (rows, columns) and dy^T x
// (columns, columns) without a transposed copy of anything.
//
// Tile: 64*MT x 64*NT per workgroup of 2 x 2 waves, each wave MT x NT
// accumulators of 32 x 32; 128 bytes of k per step (64 bf16 or 32 fp32
// values), two LDS stages filled by 16-byte buffer loads straight into LDS.
// Every lane's byte offset in a tile is fixed and the tile's base advances in
// scalar registers; a lane whose row or k lies outside the operand asks for
// an offset past the buffer's range, which the hardware answers with zeros,
// so edges cost one select and no branch.  The fragments of the next 16 (or
// 8) k are read while those of this one are multiplied, and the step's
// barrier stands before its last quarter of products, when every fragment of
// the stage is in registers: the stage is refilled at once and the products
// hide the wait.
//
// LDS layouts (16-byte pieces, so that the lanes of a read hit distinct
// banks):  rows: tile row r is 128 bytes, piece c at c ^ (r & 7).  columns:
// LDS row k holds the tile's r, piece c at c ^ swz(k); bf16 fragments are
// read with the transposing 8-byte LDS read (four k of one r per lane).
//
// The weight operand B is the MFMA's first operand, so a lane's accumulators
// are runs of four neighbouring n of one row m: rows of C are stored in
// 16-byte pieces, and the 32 columns of a group that shares an exponent lie
// in two lanes.
#pragma once

#include <type_traits>

#include "lm_math.h"

namespace rnnk {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr unsigned kOutside = 0x80000000u;   // byte offset past any operand tile: reads zeros

// s_waitcnt immediate (gfx9 encoding), export count not waited on.
constexpr int wait_imm(int vm, int lgkm) { return (((vm >> 4) & 3) << 14) | ((lgkm & 15) << 8) | (7 << 4) | (vm & 15); }

template <bool BF, bool ROWS, int R>   // R: tile rows (m or n) of the operand
struct Operand {
  static constexpr int ES = BF ? 2 : 4;
  static constexpr int BK = 128 / ES;
  static constexpr int BYTES = R * 128;              // one stage
  static constexpr int LOADS = BYTES / 4096;         // 1 KB loads per wave and stage
  static constexpr int PITCH = ROWS ? 128 : R * ES;  // bytes of an LDS row

  unsigned voff[LOADS];   // byte offset of each load's piece in the tile (kOutside: no such row)
  int klane[ROWS ? 1 : LOADS];   // k (in elements) of each load's piece within a step

  static __device__ __forceinline__ int swz(int k) {   // XOR on the 16-byte piece of LDS row k ("columns")
    if constexpr (!BF) return 0;
    else return PITCH % 256 == 0 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
  }

  // row(r): index of tile row r in the operand, or -1
  template <class F>
  __device__ __forceinline__ void init(long long ld, int wave, int lane, F row) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int pos = (4 * j + wave) * 1024 + lane * 16;
      if constexpr (ROWS) {
        const int r = pos / 128, c = (lane & 7) ^ (r & 7);
        const int gr = row(r);
        klane[0] = c * (16 / ES);      // r & 7 = lane / 8 for every load
        voff[j] = gr < 0 ? kOutside : (unsigned)(gr * ld * ES) + (unsigned)(c * 16);
      } else {
        const int k = pos / PITCH, c = (pos % PITCH) / 16 ^ swz(k);
        const int gr = row(c * (16 / ES));
        klane[j] = k;
        voff[j] = gr < 0 ? kOutside : (unsigned)(k * ld * ES) + (unsigned)(gr * ES);
      }
    }
  }

  // fill one stage: k values base + [0, BK), those at or past kleft are zero.
  // HALF > 0: of every 2 * HALF tile rows the second HALF are read from base2
  template <int HALF = 0>
  __device__ __forceinline__ void load(const char* base, int kleft, lds_char* stage, int wave,
                                       const char* base2 = nullptr) const {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const unsigned v = klane[ROWS ? 0 : j] < kleft ? voff[j] : kOutside;
      const char* b = base;
      if constexpr (HALF > 0) b = (8 * (4 * j + wave)) % (2 * HALF) >= HALF ? base2 : base;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)b, 0, 0x7fffffff, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(stage + (4 * j + wave) * 1024),
                                               16, v, 0, 0, 0);
    }
  }
};

// Fragment reader of a wave's T tiles of 32 rows.
template <bool BF, bool ROWS, int R, int T>
struct Reader {
  using Op = Operand<BF, ROWS, R>;
  int off[ROWS ? 4 : T];

  __device__ __forceinline__ void init(int first, int lane) {   // first: the wave's first tile row
    const int q = lane >> 5, i = lane & 31;
    if constexpr (ROWS) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) off[kk] = (first + i) * 128 + (((kk * 2 + q) ^ (i & 7)) * 16);
    } else if constexpr (BF) {
      // 16 lanes read 4 k x 16 r: lane j of them k = j / 4, r = 4 (j % 4)..+3, and receive r = j, 4 k
      const int j = lane & 15, k = q * 8 + (j >> 2);
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int c = (first + t * 32 + ((lane >> 4) & 1) * 16 + (j & 3) * 4) / 8;
        off[t] = k * Op::PITCH + ((c ^ Op::swz(k)) * 16) + (j & 1) * 8;
      }
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) off[t] = q * 4 * Op::PITCH + (first + t * 32 + i) * 4;
    }
  }
  __device__ __forceinline__ void read(const lds_char* stage, int kk, u32x4 (&f)[T]) const {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if constexpr (ROWS) {
        f[t] = *(const __attribute__((address_space(3))) u32x4*)(stage + off[kk] + t * 32 * 128);
      } else if constexpr (BF) {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const lds_char* p = stage + off[t] + kk * 16 * Op::PITCH;
        const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
        const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * Op::PITCH)));
        f[t] = u32x4{a.x, a.y, b.x, b.y};
      } else {
        const lds_char* p = stage + off[t] + kk * 8 * Op::PITCH;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[t][e] = *(const __attribute__((address_space(3))) unsigned*)(p + e * Op::PITCH);
      }
    }
  }
};

// 16 (bf16) or 8 (fp32) k of a 32 x 32 tile.  fp32: the lanes of half q hold
// k = 4q .. 4q+3, both operands alike, so any order of the four is right.
template <bool BF>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, f32x16 c) {
  if constexpr (BF) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
}

// ------------------------------------------------------------- epilogues
// A lane's 16 accumulators v of a 32 x 32 tile are columns 8j + 4h + e of its
// row (v[4j + e], h = lane / 32): exchange between the two lanes of a row so
// that lane half h holds columns 16i + 8h .. +7 in o[i] as bf16.
__device__ __forceinline__ void pack_row(const float (&v)[16], u32x4 (&o)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned x0 = pack2bf(v[8 * i], v[8 * i + 1]), x1 = pack2bf(v[8 * i + 2], v[8 * i + 3]);
    const unsigned y0 = pack2bf(v[8 * i + 4], v[8 * i + 5]), y1 = pack2bf(v[8 * i + 6], v[8 * i + 7]);
    const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
    o[i] = u32x4{s0[0], s1[0], s0[1], s1[1]};
  }
}

// Store a lane's 16 values to columns n .. n+31 of a row: `row` points at
// column n; columns at or past `left` are not stored.
template <bool BF>
__device__ __forceinline__ void store_row(El<BF>* row, const float (&v)[16], int h, int left, bool vec) {
  if (vec && left >= 32) {
    if constexpr (BF) {
      u32x4 o[2];
      pack_row(v, o);
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(row + 16 * i + 8 * h) = o[i];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(row + 8 * j + 4 * h) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (8 * j + 4 * h + e < left) el_store<BF>(row + 8 * j + 4 * h + e, v[4 * j + e]);
}

// The two lanes of a row agree on the bit pattern of the group's largest
// magnitude.
__device__ __forceinline__ unsigned group_top(const float (&v)[16]) {
  unsigned t = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) t = max(t, __float_as_uint(v[i]) & 0x7fffffffu);
  const auto s = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  return max(s[0], s[1]);
}

constexpr int kBadGroup = -128;   // exponent byte of a group that holds an infinity or a NaN

// 32 columns of a row as 8-bit checkpoint units; q points at the group's first byte.
__device__ __forceinline__ void store_group8(int8_t* q, int8_t* ex, const float (&v)[16], int h) {
  const unsigned top = group_top(v);
  const bool bad = top >= 0x7f800000u;
  const int e = max((int)(top >> 23) - 133, -126);
  const float inv = bad ? 0.f : __uint_as_float((unsigned)(127 - e) << 23);
  unsigned w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = (int)fminf(fmaxf(rintf(v[4 * j + k] * inv), -127.f), 127.f);
      w[j] |= (unsigned)(x & 255) << (8 * k);
    }
  }
  // four columns a word: after the exchange half h holds columns 16i + 8h .. +7
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(w[2 * i], w[2 * i + 1], false, false);
    *reinterpret_cast<u32x2*>(q + 16 * i + 8 * h) = u32x2{s[0], s[1]};
  }
  if (h == 0) *ex = bad ? kBadGroup : (int8_t)e;
}
__device__ __forceinline__ void load_group8(const int8_t* q, int ex, float (&v)[16], int h) {
  const float s = ex == kBadGroup ? __uint_as_float(0x7fc00000u) : __uint_as_float((unsigned)(127 + ex) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const unsigned w = *reinterpret_cast<const unsigned*>(q + 8 * j + 4 * h);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * j + k] = (float)(int8_t)(w >> (8 * k)) * s;
  }
}

// 32 columns of a row in 16 bits: whole numbers of 2^e, |q| <= 2^14, e the
// exponent of the group's largest magnitude - 14, so the error is at most
// 2^-14 of that magnitude (bf16 would be off by up to 2^-8 of each value, and
// a product of two such values by twice that).  Adding 1.5 * 2^23 rounds to
// the nearest whole number, ties to even, and leaves it in the low bits.
__device__ __forceinline__ void store_group16(int16_t* q, int8_t* ex, const float (&v)[16], int h) {
  const unsigned top = group_top(v);
  const bool bad = top >= 0x7f800000u;
  const int e = max((int)(top >> 23) - 140, -126);
  const float inv = bad ? 0.f : __uint_as_float((unsigned)(127 - e) << 23);
  unsigned w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned lo = __float_as_uint(fmaf(v[2 * i], inv, 12582912.f)), hi = __float_as_uint(fmaf(v[2 * i + 1], inv, 12582912.f));
    w[i] = (lo & 0xffffu) | (hi << 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s0 = __builtin_amdgcn_permlane32_swap(w[4 * i], w[4 * i + 2], false, false);
    const auto s1 = __builtin_amdgcn_permlane32_swap(w[4 * i + 1], w[4 * i + 3], false, false);
    *reinterpret_cast<u32x4*>(q + 16 * i + 8 * h) = u32x4{s0[0], s1[0], s0[1], s1[1]};
  }
  if (h == 0) *ex = bad ? kBadGroup : (int8_t)e;
}
__device__ __forceinline__ void load_group16(const int16_t* q, int ex, float (&v)[16], int h) {
  const float s = ex == kBadGroup ? __uint_as_float(0x7fc00000u) : __uint_as_float((unsigned)(127 + ex) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(q + 8 * j + 4 * h);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * j + k] = (float)(int16_t)(w[k / 2] >> (16 * (k & 1))) * s;
  }
}

template <int ACT, bool BF, int SAVE>
__device__ __forceinline__ void glu_tile(const f32x16& gv, const f32x16& uv, const FfnGemm& p, long long m, int f, int h) {
  float a[16], da[16], o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    act_pair<ACT>(gv[i], a[i], da[i]);
    o[i] = a[i] * uv[i];
  }
  store_row<BF>((El<BF>*)p.C + m * p.ldc + f, o, h, 32, true);
  if constexpr (SAVE == SAVE_FULL) {
#pragma unroll
    for (int i = 0; i < 16; ++i) da[i] *= uv[i];
    const long long at = m * p.lds + f, ate = m * p.lde + f / kGroup;
    if constexpr (BF) {
      store_group16((int16_t*)p.s0 + at, p.e0 + ate, a, h);
      store_group16((int16_t*)p.s1 + at, p.e1 + ate, da, h);
    } else {
      store_row<false>((float*)p.s0 + at, a, h, 32, true);
      store_row<false>((float*)p.s1 + at, da, h, 32, true);
    }
  } else if constexpr (SAVE == SAVE_INT8) {
    const long long at = m * p.lds + f, ate = m * p.lde + f / kGroup;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      a[i] = gv[i];
      da[i] = uv[i];
    }
    store_group8((int8_t*)p.s0 + at, p.e0 + ate, a, h);
    store_group8((int8_t*)p.s1 + at, p.e1 + ate, da, h);
  }
}

// dh of 32 columns -> dgate, dup (and the gated product again, from 8 bits)
template <int ACT, bool BF, int SAVE>
__device__ __forceinline__ void dglu_tile(const f32x16& dh, const FfnGemm& p, long long m, int f, int h) {
  const long long at = m * p.lds + f, ate = m * p.lde + f / kGroup;
  float a[16], b[16];
  if constexpr (SAVE == SAVE_FULL) {
    if constexpr (BF) {
      load_group16((const int16_t*)p.s0 + at, p.e0[ate], a, h);
      load_group16((const int16_t*)p.s1 + at, p.e1[ate], b, h);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = *reinterpret_cast<const float4*>((const float*)p.s0 + at + 8 * j + 4 * h);
        const float4 y = *reinterpret_cast<const float4*>((const float*)p.s1 + at + 8 * j + 4 * h);
        a[4 * j] = x.x, a[4 * j + 1] = x.y, a[4 * j + 2] = x.z, a[4 * j + 3] = x.w;
        b[4 * j] = y.x, b[4 * j + 1] = y.y, b[4 * j + 2] = y.z, b[4 * j + 3] = y.w;
      }
    }
  } else {
    float hh[16];
    load_group8((const int8_t*)p.s0 + at, p.e0[ate], a, h);
    load_group8((const int8_t*)p.s1 + at, p.e1[ate], b, h);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x, dx;
      act_pair<ACT>(a[i], x, dx);
      hh[i] = x * b[i];
      a[i] = x;
      b[i] *= dx;
    }
    store_row<BF>((El<BF>*)p.h + m * p.ldh + f, hh, h, 32, true);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] *= dh[i];
    b[i] *= dh[i];
  }
  El<BF>* row = (El<BF>*)p.C + m * p.ldc + f;
  store_row<BF>(row, b, h, 32, true);
  store_row<BF>(row + p.ldc / 2, a, h, 32, true);
}

}  // namespace

enum FfnEpi { FFN_STORE = 0, FFN_GLU = 1, FFN_DGLU = 2 };

template <bool BF, bool AROWS, bool BROWS, int MT, int NT, int EPI, int SAVE, int OCC>
__global__ __launch_bounds__(256, OCC) void ffn_gemm_kernel(const FfnGemm p) {
  constexpr int TM = 64 * MT, TN = 64 * NT, ES = BF ? 2 : 4, BK = 128 / ES;
  constexpr int FN = EPI == FFN_GLU ? TN / 2 : TN;   // columns of C per tile
  using OpA = Operand<BF, AROWS, TM>;
  using OpB = Operand<BF, BROWS, TN>;
  constexpr int STAGE = OpA::BYTES + OpB::BYTES;
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
  lds_char* const lds = (lds_char*)smem;

  // tiles: contiguous runs per XCD; inside, groups of 8 tile rows, column by
  // column, so that the tiles in flight on one XCD share few row blocks
  const int tm = (p.M + TM - 1) / TM, tn = (p.N + FN - 1) / FN;
  const int per = (int)gridDim.x / 8;
  const int lin = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (lin >= tm * tn) return;
  constexpr int GM = 8;
  const int grp = lin / (GM * tn), in = lin - grp * GM * tn, gm = min(GM, tm - grp * GM);
  const int m0 = (grp * GM + in % gm) * TM, n0 = (in / gm) * FN;

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * 32 * MT, wn = (wave & 1) * 32 * NT;

  OpA la;
  OpB lb;
  la.init(p.lda, wave, lane, [&](int r) { return m0 + r < p.M ? r : -1; });
  if constexpr (EPI == FFN_GLU) {
    // each wave's rows: 16*NT gate columns, then the up columns of the same
    lb.init(p.ldb, wave, lane, [&](int r) {
      const int f = r / (32 * NT) * 16 * NT + r % (16 * NT);
      return n0 + f < p.N ? f : -1;
    });
  } else {
    lb.init(p.ldb, wave, lane, [&](int r) { return n0 + r < p.N ? r : -1; });
  }
  const char* abase = (const char*)p.A + (AROWS ? m0 * p.lda : (long long)m0) * ES;
  const char* bbase = (const char*)p.B + (BROWS ? n0 * p.ldb : (long long)n0) * ES;
  const long long astep = (AROWS ? (long long)BK : BK * p.lda) * ES, bstep = (BROWS ? (long long)BK : BK * p.ldb) * ES;

  // K in up to two segments of p.kseg (a multiple of BK) columns of A, of
  // which p.K are real; the second starts p.kseg later in A and p.K later in B
  const int nseg = (p.K + BK - 1) / BK, nk = nseg * p.segs;
  auto fill = [&](int kt, int st) {
    const int seg = kt >= nseg ? 1 : 0, k0 = kt - seg * nseg;
    const char* a = abase + k0 * astep + seg * (AROWS ? (long long)p.kseg : p.kseg * p.lda) * ES;
    const char* b = bbase + k0 * bstep + seg * (BROWS ? (long long)p.K : p.K * p.ldb) * ES;
    const int left = p.K - k0 * BK;
    la.load(a, left, lds + st * STAGE, wave);
    if constexpr (EPI == FFN_GLU)
      lb.template load<16 * NT>(b, left, lds + st * STAGE + OpA::BYTES, wave, b + p.N * p.ldb * ES);
    else
      lb.load(b, left, lds + st * STAGE + OpA::BYTES, wave);
  };

  Reader<BF, AROWS, TM, MT> ra;
  Reader<BF, BROWS, TN, NT> rb;
  ra.init(wm, lane);
  rb.init(wn, lane);

  f32x16 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  u32x4 fa[2][MT], fb[2][NT];
  if (nk > 0) {
    fill(0, 0);
    __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (nk > 1) fill(1, 1);
    ra.read(lds, 0, fa[0]);
    rb.read(lds + OpA::BYTES, 0, fb[0]);
  }
  for (int kt = 0; kt < nk; ++kt) {
    const lds_char* sa = lds + (kt & 1) * STAGE;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk < 3) {
        ra.read(sa, kk + 1, fa[(kk + 1) & 1]);
        rb.read(sa + OpA::BYTES, kk + 1, fb[(kk + 1) & 1]);
      } else {
        // this stage's fragments are in registers; the next stage is whole
        // once this wave's loads and everyone's have landed
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (kt + 1 < nk) {
          const lds_char* sn = lds + ((kt + 1) & 1) * STAGE;
          ra.read(sn, 0, fa[0]);
          rb.read(sn + OpA::BYTES, 0, fb[0]);
          if (kt + 2 < nk) fill(kt + 2, kt & 1);
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma32<BF>(fb[kk & 1][j], fa[kk & 1][i], acc[i][j]);
    }
  }

  const int h = lane >> 5;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long long m = m0 + wm + i * 32 + (lane & 31);
    if (m >= p.M) continue;
    if constexpr (EPI == FFN_STORE) {
      // rows of the second half (p.mseg and on) close the gap of the first's padding
      long long row = m;
      if (p.mseg) {
        const int half = m >= p.mseg ? 1 : 0;
        const long long in2 = m - (half ? p.mseg : 0);
        if (in2 >= p.mreal) continue;
        row = half * (long long)p.mreal + in2;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int n = n0 + wn + j * 32;
        if (n >= p.N) continue;
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e];
        store_row<BF>((El<BF>*)p.C + row * p.ldc + n, v, h, p.N - n, p.cvec);
      }
    } else if constexpr (EPI == FFN_GLU) {
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        const int f = n0 + (wave & 1) * 16 * NT + j * 32;
        if (f >= p.N) continue;
        if (p.act == ACT_SILU) glu_tile<ACT_SILU, BF, SAVE>(acc[i][j], acc[i][j + NT / 2], p, m, f, h);
        else if (p.act == ACT_GELU) glu_tile<ACT_GELU, BF, SAVE>(acc[i][j], acc[i][j + NT / 2], p, m, f, h);
        else glu_tile<ACT_SIGMOID, BF, SAVE>(acc[i][j], acc[i][j + NT / 2], p, m, f, h);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int f = n0 + wn + j * 32;
        if (f >= p.N) continue;
        if (SAVE == SAVE_FULL || p.act == ACT_SILU) dglu_tile<ACT_SILU, BF, SAVE>(acc[i][j], p, m, f, h);
        else if (p.act == ACT_GELU) dglu_tile<ACT_GELU, BF, SAVE>(acc[i][j], p, m, f, h);
        else dglu_tile<ACT_SIGMOID, BF, SAVE>(acc[i][j], p, m, f, h);
      }
    }
  }
}

}  // namespace rnnk
