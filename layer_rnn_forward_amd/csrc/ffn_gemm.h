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
// values), filled by 16-byte buffer loads straight into LDS: three stages of A
// and two of B, which is all of the 160 KB for 256 x 256 tiles.  Every lane's
// byte offset in a tile is fixed and the tile's base advances in scalar
// registers; a lane whose row or k lies outside the operand asks for an offset
// past the buffer's range, which the hardware answers with zeros, so edges
// cost one select and no branch.  The fragments of the next 16 (or 8) k are
// read while those of this one are multiplied, and the step's barrier stands
// before its last quarter of products, when every fragment of the stage is in
// registers.
//
// LDS layouts (16-byte pieces, so that the lanes of a read hit distinct
// banks):  rows: tile row r is 128 bytes, piece c at c ^ (r >> 1 & 7).
// columns: LDS row k holds the tile's r, piece c at c ^ swz(k); bf16 fragments
// are read with the transposing 8-byte LDS read (four k of one r per lane).
//
// The weight operand B is the MFMA's first operand, so a lane's accumulators
// are runs of four neighbouring n of one row m: rows of C are stored in
// 16-byte pieces, and the 32 columns of a group that shares an exponent lie
// in two lanes.
//
// Bound by the matrix cores at the clock that power leaves them (1.6 - 1.7 GHz):
// 275 GFLOP (8192 x 2048, k 8192, rows x rows) take 0.235 ms after a rest and 0.214 in a steady run, 1170
// and 1285 TFLOP/s, the MFMA busy for 70 % of the cycles; with every refill left out it is 0.160 ms at
// 2.2 GHz.  Measured on that product, or on the 8192 x 2048 x 8192 training step
// (now 2.07 - 2.12 ms):  all loads right after the barrier 2.26 ms (a CU takes 16
// cycles for each, and the wave that waits for its turn issues no products);
// 64-byte steps in four stages 0.268 ms (rows then ask the L2 for twice as many
// lines, one a cycle and channel: all it has); pieces at c ^ (r & 7) conflict
// two ways; groups of 8 tile rows 2.09 ms; the fragments' reads ahead of the
// loads or spread evenly: the same.  16 x 16 accumulators (0.226 ms) need 64
// more fragment registers, and the epilogues then spill.
#pragma once

#include <algorithm>
#include <type_traits>

#include "ffn_plan.h"
#include "lm_math.h"

namespace rnnk {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) char lds_char;

constexpr unsigned kOutside = 0x80000000u;   // byte offset past any operand tile: reads zeros

// s_waitcnt immediate (gfx9 encoding), export count not waited on.
constexpr int wait_imm(int vm, int lgkm) { return (((vm >> 4) & 3) << 14) | ((lgkm & 15) << 8) | (7 << 4) | (vm & 15); }

template <bool BF, bool ROWS, int R>   // R: tile rows (m or n) of the operand
struct Operand {
  static constexpr int ES = BF ? 2 : 4;
  static constexpr int BK = kStep / ES;
  static constexpr int BYTES = R * kStep;              // one stage
  static constexpr int LOADS = BYTES / 4096;           // 1 KB loads per wave and stage
  static constexpr int PITCH = ROWS ? kStep : R * ES;  // bytes of an LDS row

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
        const int r = pos / kStep, c = (lane & 7) ^ (r >> 1 & 7);
        const int gr = row(r);
        klane[0] = c * (16 / ES);      // r >> 1 & 7 is the same for every load
        voff[j] = gr < 0 ? kOutside : (unsigned)(gr * ld * ES) + (unsigned)(c * 16);
      } else {
        const int k = pos / PITCH, c = (pos % PITCH) / 16 ^ swz(k);
        const int gr = row(c * (16 / ES));
        klane[j] = k;
        voff[j] = gr < 0 ? kOutside : (unsigned)(k * ld * ES) + (unsigned)(gr * ES);
      }
    }
  }

  // load j of the fill of one stage: k values base + [0, BK), those at or past
  // kleft are zero.  HALF > 0: of every 2 * HALF tile rows the second HALF are
  // read from base2
  template <int HALF = 0>
  __device__ __forceinline__ void load(int j, const char* base, int kleft, lds_char* stage, int wave,
                                       const char* base2 = nullptr) const {
    const unsigned v = klane[ROWS ? 0 : j] < kleft ? voff[j] : kOutside;
    const char* b = base;
    if constexpr (HALF > 0) b = (8 * (4 * j + wave)) % (2 * HALF) >= HALF ? base2 : base;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)b, 0, 0x7fffffff, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(stage + (4 * j + wave) * 1024), 16,
                                             v, 0, 0, 0);
  }
};

// The transposing LDS read.  (A restrict pointer: without it the compiler waits
// for every load into LDS before each of these; the product's own waits and
// barriers order them.)
__device__ __forceinline__ u32x2 read_tr(const lds_char* __restrict p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// Fragment reader of a wave's T tiles of 32 rows.
template <bool BF, bool ROWS, int R, int T>
struct Reader {
  using Op = Operand<BF, ROWS, R>;
  int off[ROWS ? 4 : T];

  __device__ __forceinline__ void init(int first, int lane) {   // first: the wave's first tile row
    const int q = lane >> 5, i = lane & 31;
    if constexpr (ROWS) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) off[kk] = (first + i) * kStep + (((kk * 2 + q) ^ (i >> 1 & 7)) * 16);
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
  __device__ __forceinline__ void read(const lds_char* stage, int kk, int t, u32x4& f) const {
    if constexpr (ROWS) {
      f = *(const __attribute__((address_space(3))) u32x4*)(stage + off[kk] + t * 32 * kStep);
    } else if constexpr (BF) {
      const lds_char* p = stage + off[t] + kk * 16 * Op::PITCH;
      const u32x2 a = read_tr(p), b = read_tr(p + 4 * Op::PITCH);
      f = u32x4{a.x, a.y, b.x, b.y};
    } else {
      const lds_char* p = stage + off[t] + kk * 8 * Op::PITCH;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = *(const __attribute__((address_space(3))) unsigned*)(p + e * Op::PITCH);
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

// Zeros after the last column of a row that is an operand of the next product
// with its columns as k: that product reads whole 16-byte pieces against zeros,
// and an infinity or a NaN of the row's own (times this product's zeros) must
// not be there.  `row` points at the row's last 32 columns; the lane that
// stored a piece clears its end.
template <bool BF>
__device__ __forceinline__ void clear_end(El<BF>* row, int left, int h) {
  constexpr int P = BF ? 8 : 4;
  if (left >= 32 || (left / P & 1) != h) return;
#pragma unroll 1
  for (int c = left; c % P; ++c) row[c] = 0;
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

// A wave's MT x NT tiles to C: rows from m0, columns from n0.
template <bool BF, int MT, int NT>
__device__ __forceinline__ void store_tiles(const f32x16 (&acc)[MT][NT], const FfnGemm& p, long long m0, int n0, int lane) {
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long long m = m0 + i * 32 + (lane & 31);
    // rows of the second half (p.mseg and on) close the gap of the first's padding
    long long row = m;
    bool real = m < p.M;
    if (p.mseg) {
      const int half = m >= p.mseg ? 1 : 0;
      const long long in = m - (half ? p.mseg : 0);
      real = real && in < p.mreal;
      row = half * (long long)p.mreal + in;
    }
    if (real) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int n = n0 + j * 32;
        if (n < p.N) {
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e];
          store_row<BF>((El<BF>*)p.C + row * p.ldc + n, v, lane >> 5, p.N - n, p.cvec);
        }
      }
    }
  }
}

// What is saved for backward lies tile by tile: 32 rows x 32 columns, each
// lane's 16 values where its lane number says, so that a wave writes and reads
// them in runs of 1 KB (rows of C would be 64 byte pieces).  A group of 32
// columns is a row of a tile, and its exponent byte is at the row's number.
//
// 8 bits: checkpoint units (include/rnn.h), 16 bytes a lane.
__device__ __forceinline__ u32x4 pack8(const float (&v)[16], int& ex) {
  const unsigned top = group_top(v);
  const bool bad = top >= 0x7f800000u;
  const int e = max((int)(top >> 23) - 133, -126);
  const float inv = bad ? 0.f : __uint_as_float((unsigned)(127 - e) << 23);
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // + 1.5 * 2^23 rounds to the nearest whole number, ties to even, and leaves it in the low bits
      const float u = __builtin_amdgcn_fmed3f(fmaf(v[4 * j + k], inv, 12582912.f), 12582912.f - 127.f, 12582912.f + 127.f);
      w[j] |= (__float_as_uint(u) & 255u) << (8 * k);
    }
  }
  ex = bad ? kBadGroup : e;
  return w;
}
__device__ __forceinline__ void unpack8(const u32x4& w, int ex, float (&v)[16]) {
  const float s = ex == kBadGroup ? __uint_as_float(0x7fc00000u) : __uint_as_float((unsigned)(127 + ex) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * j + k] = (float)(int8_t)(w[j] >> (8 * k)) * s;
}

// 16 bits: fp16 numbers times 2^e, e the exponent of the group's largest finite
// magnitude - 14, which brings it into [2^14, 2^15).  Half a step is 2^-11 of
// each value (2^-39 of the group's largest below 2^-28 of it); bf16 would be
// off by up to 2^-8, and a product of two such values by twice that.  A value
// far out takes nothing from its neighbours, and an infinity or a NaN is its
// own (whole numbers of a common 2^e, 2^-14 of the largest for every value,
// lost both, and took as long).
__device__ __forceinline__ void pack16(const float (&v)[16], u32x4 (&w)[2], int& ex) {
  // without the sign, and one up in the exponent: infinities and NaNs wrap to the bottom
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, (__float_as_uint(v[i]) << 1) + 0x01000000u);
  const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
  const int e = max((int)(max(both[0], both[1]) >> 24) - 142, -126);
  const float inv = __uint_as_float((unsigned)(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const h16x2 h = {(_Float16)(v[2 * i] * inv), (_Float16)(v[2 * i + 1] * inv)};
    w[i / 4][i % 4] = __builtin_bit_cast(unsigned, h);
  }
  ex = e;
}
__device__ __forceinline__ void unpack16(const u32x4 (&w)[2], int ex, float (&v)[16]) {
  const float s = __uint_as_float((unsigned)(127 + ex) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned both = w[i / 4][i % 4];   // (a copy: a cast of the vector's element itself takes its first one)
    const h16x2 h = __builtin_bit_cast(h16x2, both);
    v[2 * i] = (float)h.x * s;
    v[2 * i + 1] = (float)h.y * s;
  }
}

// One of the two saved tensors' tile: 1 (8 bits), 2 (16 bits) or 4 (fp32)
// pieces of 16 bytes a lane.
template <bool BF, int SAVE>
struct Saved {
  static constexpr int N = SAVE == SAVE_INT8 ? 1 : BF ? 2 : 4;
  u32x4 w[N];
  int ex;

  __device__ __forceinline__ void pack(const float (&v)[16]) {
    if constexpr (SAVE == SAVE_INT8) w[0] = pack8(v, ex);
    else if constexpr (BF) pack16(v, w, ex);
    else
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = __float_as_uint(v[i]);
  }
  __device__ __forceinline__ void unpack(float (&v)[16]) const {
    if constexpr (SAVE == SAVE_INT8) unpack8(w[0], ex, v);
    else if constexpr (BF) unpack16(w, ex, v);
    else
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i / 4][i % 4]);
  }
  // values at `to` + tile * 1 KB * N, exponents at `e` + tile * 32
  __device__ __forceinline__ void store(void* to, int8_t* e, long long tile, int lane) const {
    u32x4* p = (u32x4*)to + tile * (64 * N) + lane;
#pragma unroll
    for (int i = 0; i < N; ++i) p[64 * i] = w[i];
    if ((BF || SAVE == SAVE_INT8) && lane < 32) e[tile * 32 + lane] = (int8_t)ex;
  }
  __device__ __forceinline__ void load(const void* from, const int8_t* e, long long tile, int lane) {
    const u32x4* p = (const u32x4*)from + tile * (64 * N) + lane;
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = p[64 * i];
    ex = BF || SAVE == SAVE_INT8 ? e[tile * 32 + (lane & 31)] : 0;
  }
};

// projections of 32 columns -> the gated product, and what is saved.  In bf16
// the product is rounded to bf16 here, as the next product's operand: an output's
// error is sqrt(2) of its own rounding's (0.0023 relative for 0.0017).  Passed on
// as two numbers it would double that product (8192 x 2048, k 8192: 0.21 ms).
template <int ACT, bool BF, int SAVE>
__device__ __forceinline__ void glu_tile(const f32x16& gv, const f32x16& uv, const FfnGemm& p, long long m, int f, int lane) {
  float a[16], da[16], o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    act_pair<ACT>(gv[i], a[i], da[i]);
    o[i] = a[i] * uv[i];
    da[i] *= uv[i];
  }
  El<BF>* row = (El<BF>*)p.C + m * p.ldc + f;
  store_row<BF>(row, o, lane >> 5, 32, true);
  clear_end<BF>(row, p.N - f, lane >> 5);
  if constexpr (SAVE != SAVE_NONE) {
    const long long tile = (m >> 5) * p.lds + (f >> 5);
    Saved<BF, SAVE> s0, s1;
    if constexpr (SAVE == SAVE_INT8) {
      float g[16], u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        g[i] = gv[i];
        u[i] = uv[i];
      }
      s0.pack(g);
      s1.pack(u);
    } else {
      s0.pack(a);
      s1.pack(da);
    }
    s0.store(p.s0, p.e0, tile, lane);
    s1.store(p.s1, p.e1, tile, lane);
  }
}

// A wave's tiles, 16 * NT gate columns and then the up columns of the same:
// rows from m0, columns from f0.
template <int ACT, bool BF, int SAVE, int MT, int NT>
__device__ __forceinline__ void glu_tiles(const f32x16 (&acc)[MT][NT], const FfnGemm& p, long long m0, int f0, int lane) {
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const long long m = m0 + i * 32 + (lane & 31);
    if (m < p.M) {
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        const int f = f0 + j * 32;
        if (f < p.N) glu_tile<ACT, BF, SAVE>(acc[i][j], acc[i][j + NT / 2], p, m, f, lane);
      }
    }
  }
}

// dh of 32 columns -> dgate, dup, rounded to bf16 as the next products' operands
// likewise (and the gated product again, from 8 bits)
template <int ACT, bool BF, int SAVE>
__device__ __forceinline__ void dglu_tile(const f32x16& dh, const Saved<BF, SAVE>& s0, const Saved<BF, SAVE>& s1,
                                          const FfnGemm& p, long long m, int f, int lane) {
  const int h = lane >> 5;
  float a[16], b[16];
  s0.unpack(a);
  s1.unpack(b);
  if constexpr (SAVE == SAVE_INT8) {
    float hh[16];
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
  clear_end<BF>(row, p.N - f, h);
  clear_end<BF>(row + p.ldc / 2, p.N - f, h);
}

}  // namespace

enum FfnEpi { FFN_STORE = 0, FFN_GLU = 1, FFN_DGLU = 2 };

// Tile `lin` of tm x tn: groups of 4 tile rows, column by column.
__device__ __forceinline__ void tile_at(int lin, int tm, int tn, int& m, int& n) {
  constexpr int GM = 4;
  const int grp = lin / (GM * tn), in = lin - grp * GM * tn, gm = min(GM, tm - grp * GM);
  m = grp * GM + in % gm;
  n = in / gm;
}

// Piece `block` of a product that has `blocks` (a multiple of 8) workgroups: a
// tile, or a split of a tile's k, whose sums go to p.part.
template <bool BF, bool AROWS, bool BROWS, int MT, int NT, int EPI, int SAVE, int ACT>
__device__ __forceinline__ void ffn_product(const FfnGemm& p, char* smem, int block, int blocks) {
  constexpr int TM = 64 * MT, TN = 64 * NT, ES = BF ? 2 : 4, BK = kStep / ES;
  constexpr int FN = EPI == FFN_GLU ? TN / 2 : TN;   // columns of C per tile
  constexpr bool SPLIT = EPI != FFN_DGLU && MT < 4;
  using OpA = Operand<BF, AROWS, TM>;
  using OpB = Operand<BF, BROWS, TN>;
  lds_char* const lds_a = (lds_char*)smem;
  lds_char* const lds_b = lds_a + kStagesA * OpA::BYTES;

  // tiles: contiguous runs per XCD; inside, groups of 4 tile rows, column by
  // column, so that the tiles in flight on one XCD share few row blocks
  const int tm = (p.M + TM - 1) / TM, tn = (p.N + FN - 1) / FN;
  int lin = block % 8 * (blocks / 8) + block / 8, split = 0;
  if (SPLIT && p.splits > 1) {
    split = lin % p.splits;
    lin /= p.splits;
  }
  if (lin >= tm * tn) return;
  int m0, n0;
  tile_at(lin, tm, tn, m0, n0);
  m0 *= TM;
  n0 *= FN;

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
  // which p.K are real; the second starts p.kseg later in A and p.K later in
  // B.  Steps past the last fill their stage with zeros that nobody reads.
  const int nseg = (p.K + BK - 1) / BK;
  int k0 = 0, nk = nseg * p.segs;
  if (SPLIT && p.splits > 1) {
    const int per = (nk + p.splits - 1) / p.splits;
    k0 = min(split * per, nk);
    nk = min(per, nk - k0);
  }
  struct Fill {
    const char* at;
    int left, kt;
  };
  auto advance = [&](Fill& q, const char* second, long long step) {
    q.at += step;
    q.left -= BK;
    if (++q.kt == nseg && p.segs == 2) {
      q.at = second;
      q.left = p.K;
    }
  };
  const char* const a2nd = abase + (AROWS ? (long long)p.kseg : p.kseg * p.lda) * ES;
  const char* const b2nd = bbase + (BROWS ? (long long)p.K : p.K * p.ldb) * ES;
  const int seg = k0 >= nseg ? 1 : 0, kin = k0 - seg * nseg;
  Fill qa{(seg ? a2nd : abase) + kin * astep, p.K - kin * BK, k0}, qb{(seg ? b2nd : bbase) + kin * bstep, p.K - kin * BK, k0};
  auto next_a = [&] { advance(qa, a2nd, astep); };
  auto next_b = [&] { advance(qb, b2nd, bstep); };
  constexpr int LA = OpA::LOADS, LB = OpB::LOADS;
  auto fill_a = [&](int from, int to, lds_char* stage) {
#pragma unroll
    for (int j = 0; j < LA; ++j)
      if (j >= from && j < to) la.load(j, qa.at, qa.left, stage, wave);
  };
  auto fill_b = [&](int from, int to, lds_char* stage) {
#pragma unroll
    for (int j = 0; j < LB; ++j)
      if (j >= from && j < to) {
        if constexpr (EPI == FFN_GLU) lb.template load<16 * NT>(j, qb.at, qb.left, stage, wave, qb.at + p.N * p.ldb * ES);
        else lb.load(j, qb.at, qb.left, stage, wave);
      }
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

  // FFN_DGLU: the saved tiles, asked for AHEAD tiles before they are used (the
  // first before the products).  Tiles past the edges repeat the last one, and
  // their values are not used.
  constexpr int AHEAD = 2;
  Saved<BF, SAVE> saved[EPI == FFN_DGLU ? AHEAD + 1 : 1][2];
  auto prefetch = [&](int t) {
    const int i = t / NT, j = t % NT;
    const long long tile = min((m0 + wm) / 32 + i, (p.M - 1) / 32) * p.lds + min((n0 + wn) / 32 + j, (int)p.lds - 1);
    saved[t % (AHEAD + 1)][0].load(p.s0, p.e0, tile, lane);
    saved[t % (AHEAD + 1)][1].load(p.s1, p.e1, tile, lane);
  };
  if constexpr (EPI == FFN_DGLU) {
#pragma unroll
    for (int t = 0; t < AHEAD && t < MT * NT; ++t) prefetch(t);
  }

  u32x4 fa[2][MT], fb[2][NT];
  lds_char *a0 = lds_a, *a1 = a0 + OpA::BYTES, *a2 = a1 + OpA::BYTES;   // of steps kt, kt + 1, kt + 2
  lds_char *b0 = lds_b, *b1 = b0 + OpB::BYTES;
  if (nk > 0) {
    fill_b(0, LB, b0);
    next_b();
    fill_a(0, LA, a0);
    next_a();
    fill_a(0, LA, a1);
    next_a();
    fill_b(0, LB * 3 / 4, b1);
    __builtin_amdgcn_s_waitcnt(wait_imm(LA + LB * 3 / 4, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NT; ++j) rb.read(b0, 0, j, fb[0][j]);
#pragma unroll
    for (int i = 0; i < MT; ++i) ra.read(a0, 0, i, fa[0][i]);
  }
  for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk == 3) {
        // this step's fragments are in registers; the next step's stages are
        // whole once this wave's loads and everyone's have landed, all but
        // those of the step after it
        __builtin_amdgcn_s_waitcnt(wait_imm(LA, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      // Among the products: the next fragments, then a few loads.  The order is
      // kept as written: one wave a SIMD has nothing else to cover them with.
      // The loads are spread over the step because a CU takes 16 cycles for
      // each, and a wave that has to wait for its turn issues no products.
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[i][j] = mfma32<BF>(fb[kk & 1][j], fa[kk & 1][i], acc[i][j]);
          constexpr int S = MT * NT;
          const int at = i * NT + j;
          auto share = [&](int from, int n, int k) { return from + n * k / S; };   // of n loads from `from` on
          // fragments in the order in which they will be used
#pragma unroll
          for (int r = 0; r < MT + NT; ++r) {
            if (r < share(0, MT + NT, at) || r >= share(0, MT + NT, at + 1)) continue;
            if (r == 0) rb.read(kk < 3 ? b0 : b1, (kk + 1) & 3, 0, fb[(kk + 1) & 1][0]);
            else if (r == 1) ra.read(kk < 3 ? a0 : a1, (kk + 1) & 3, 0, fa[(kk + 1) & 1][0]);
            else if (r <= NT) rb.read(kk < 3 ? b0 : b1, (kk + 1) & 3, r - 1, fb[(kk + 1) & 1][r - 1]);
            else ra.read(kk < 3 ? a0 : a1, (kk + 1) & 3, r - NT, fa[(kk + 1) & 1][r - NT]);
          }
          if (kk == 3) {
            fill_b(share(0, LB * 3 / 4, at), share(0, LB * 3 / 4, at + 1), b0);
          } else if (kk == 0) {
            constexpr int X = LB - LB * 3 / 4;
            const int lo = share(0, X + LA / 4, at), hi = share(0, X + LA / 4, at + 1);
            fill_b(LB - X + min(lo, X), LB - X + min(hi, X), b1);
            if (lo < X && hi >= X) next_b();
            fill_a(max(lo - X, 0), max(hi - X, 0), a2);
          } else {
            constexpr int Y = LA * 5 / 8;
            if (kk == 1) fill_a(share(LA / 4, Y - LA / 4, at), share(LA / 4, Y - LA / 4, at + 1), a2);
            else fill_a(share(Y, LA - Y, at), share(Y, LA - Y, at + 1), a2);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (kk == 2) next_a();
    }
    lds_char* const t = a0;
    a0 = a1;
    a1 = a2;
    a2 = t;
    lds_char* const u = b0;
    b0 = b1;
    b1 = u;
  }
  // no load into LDS outlives the workgroup
  __builtin_amdgcn_s_waitcnt(wait_imm(0, 0));

  if constexpr (SPLIT) {
    if (p.splits > 1) {
      float4* to = (float4*)p.part + ((long long)split * tm * tn + lin) * (MT * NT * 4 * 256) + tid;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            to[((i * NT + j) * 4 + e) * 256] =
                make_float4(acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]);
      return;
    }
  }
  if constexpr (EPI == FFN_STORE) {
    store_tiles<BF, MT, NT>(acc, p, m0 + wm, n0 + wn, lane);
  } else if constexpr (EPI == FFN_GLU) {
    glu_tiles<ACT, BF, SAVE, MT, NT>(acc, p, m0 + wm, n0 + (wave & 1) * 16 * NT, lane);
  } else {
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const long long m = m0 + wm + i * 32 + (lane & 31);
      if (m < p.M) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int f = n0 + wn + j * 32;
          const int t = i * NT + j;
          if (t + AHEAD < MT * NT) prefetch(t + AHEAD);
          const Saved<BF, SAVE>(&s)[2] = saved[t % (AHEAD + 1)];
          if (f < p.N) dglu_tile<ACT, BF, SAVE>(acc[i][j], s[0], s[1], p, m, f, lane);
        }
      }
    }
  }
}

template <bool BF, bool AROWS, bool BROWS, int MT, int NT, int EPI, int SAVE, int ACT, int OCC>
__global__ __launch_bounds__(256, OCC) void ffn_gemm_kernel(const FfnGemm p) {
  __shared__ __attribute__((aligned(1024))) char smem[ffn_lds(64 * MT, 64 * NT)];
  ffn_product<BF, AROWS, BROWS, MT, NT, EPI, SAVE, ACT>(p, smem, (int)blockIdx.x, (int)gridDim.x);
}

// Add the splits of a tile in their order; the epilogue.
template <bool BF, int MT, int NT, int EPI, int SAVE, int ACT>
__device__ __forceinline__ void ffn_sum(const FfnGemm& p, int lin) {
  constexpr int FN = EPI == FFN_GLU ? 32 * NT : 64 * NT;
  const int tm = (p.M + 64 * MT - 1) / (64 * MT), tn = (p.N + FN - 1) / FN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float4* from = (const float4*)p.part + (long long)lin * (MT * NT * 4 * 256) + tid;
  const long long next = (long long)tm * tn * (MT * NT * 4 * 256);
  f32x16 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
      for (int s = 0; s < p.splits; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 v = from[s * next + ((i * NT + j) * 4 + e) * 256];
          acc[i][j][4 * e] += v.x;
          acc[i][j][4 * e + 1] += v.y;
          acc[i][j][4 * e + 2] += v.z;
          acc[i][j][4 * e + 3] += v.w;
        }
    }
  int m, n;
  tile_at(lin, tm, tn, m, n);
  const long long m0 = m * 64 * MT + (wave >> 1) * 32 * MT;
  const int n0 = n * FN + (wave & 1) * (FN / 2);
  if constexpr (EPI == FFN_GLU) glu_tiles<ACT, BF, SAVE, MT, NT>(acc, p, m0, n0, lane);
  else store_tiles<BF, MT, NT>(acc, p, m0, n0, lane);
}
template <bool BF, int MT, int NT, int EPI, int SAVE, int ACT>
__global__ __launch_bounds__(256) void ffn_sum_kernel(const FfnGemm p) {
  ffn_sum<BF, MT, NT, EPI, SAVE, ACT>(p, (int)blockIdx.x);
}

// ---------------------------------------------------------------- launches
template <bool BF, bool AROWS, bool BROWS, int MT, int NT, int EPI, int SAVE, int ACT, int OCC>
hipError_t ffn_launch(const FfnGemm& p, long long tiles, hipStream_t s) {
  const int splits = std::max(p.splits, 1);
  if (tiles * splits > 0x7ffffff0LL) return hipErrorInvalidValue;
  hipLaunchKernelGGL((ffn_gemm_kernel<BF, AROWS, BROWS, MT, NT, EPI, SAVE, ACT, OCC>),
                     dim3((unsigned)((tiles * splits + 7) / 8 * 8)), dim3(256), 0, s, p);
  if constexpr (EPI == FFN_GLU && MT < 4) {
    if (splits > 1) hipLaunchKernelGGL((ffn_sum_kernel<BF, MT, NT, EPI, SAVE, ACT>), dim3((unsigned)tiles), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

template <bool AROWS, bool BROWS, int EPI, int SAVE, int ACT>
hipError_t ffn_pick(const FfnGemm& p, int tile, int bf16, hipStream_t s) {
  if (p.M <= 0 || p.N <= 0) return hipSuccess;
  const long long tiles = ffn_tiles(p, tile, EPI == FFN_GLU);
  constexpr int N64 = EPI == FFN_GLU ? 2 : 1, OCC64 = ffn_places(TILE_64, EPI == FFN_GLU);
  if (!bf16) {
    if (tile == TILE_128) return ffn_launch<false, AROWS, BROWS, 2, 2, EPI, SAVE, ACT, 2>(p, tiles, s);
    return ffn_launch<false, AROWS, BROWS, 1, N64, EPI, SAVE, ACT, OCC64>(p, tiles, s);
  }
  if (tile == TILE_256) return ffn_launch<true, AROWS, BROWS, 4, 4, EPI, SAVE, ACT, 1>(p, tiles, s);
  if (tile == TILE_128) return ffn_launch<true, AROWS, BROWS, 2, 2, EPI, SAVE, ACT, 2>(p, tiles, s);
  return ffn_launch<true, AROWS, BROWS, 1, N64, EPI, SAVE, ACT, OCC64>(p, tiles, s);
}

}  // namespace rnnk
