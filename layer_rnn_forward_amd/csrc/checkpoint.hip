// 8-bit checkpoints of a matrix (gfx950): groups of 32 columns of a row share
// a power of two 2^e, e = exponent of the group's largest magnitude - 6 (so
// that it lands in [64, 128) units), at least -126; values are whole numbers
// of units within -127 .. 127.  Both scalings are by powers of two, so the
// only rounding is the one to whole units (ties to even), and what is read
// back has at most 7 significant bits: exact in fp32 and in bf16.
//
// Bound by memory: 3.03 (bf16) or 5.03 (fp32) bytes a value each way.  Four
// lanes hold a group, eight values each, so that values move in 16 byte
// pieces and codes in 8 byte ones, at whatever alignment the rows have; two
// groups a lane are in flight.  A lane's row and group advance by constants
// (no division in the loop).  65536 x 2048 in bf16: store 92 us, load 74 us (4.4
// and 5.5 TB/s).  One value a lane took 279 and 304 us.
#include <algorithm>
#include <type_traits>

#include "lm_math.h"

using namespace rnnk;

namespace {

constexpr int kNanGroup = -128;   // exponent byte of a group that holds an infinity or a NaN
constexpr int kFlight = 2;        // groups a lane works on at once

// groups of a launch: quad q takes groups q, q + quads, ...: `rows` rows and
// `groups` groups further each time
struct Steps {
  int rows, cols, per;             // per: groups of a row
  int srow, sgroup;
};

template <bool BF16>
__global__ __launch_bounds__(256) void store_kernel(const Steps s, const void* xv, int8_t* q, int8_t* ex) {
  const El<BF16>* x = (const El<BF16>*)xv;
  const long long k0 = ((long long)blockIdx.x * 256 + threadIdx.x) / 4;
  const int part = threadIdx.x & 3;
  long long r = k0 / s.per;
  int g = (int)(k0 - r * s.per);
  while (r < s.rows) {
    float v[kFlight][8];
    long long row[kFlight];
    int grp[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      row[i] = r;
      grp[i] = g;
      r += s.srow;
      g += s.sgroup;
      if (g >= s.per) {
        g -= s.per;
        ++r;
      }
      const int c = grp[i] * kGroup + part * 8, left = row[i] < s.rows ? s.cols - c : 0;
      const El<BF16>* p = x + row[i] * s.cols + c;
      if (left >= 8) {
        if constexpr (BF16) {
          const auto w = *reinterpret_cast<const Bytes<16>*>(p);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][2 * j] = __uint_as_float(w.w[j] << 16);
            v[i][2 * j + 1] = __uint_as_float(w.w[j] & 0xffff0000u);
          }
        } else {
          const auto a = *reinterpret_cast<const Bytes<16>*>(p), b = *reinterpret_cast<const Bytes<16>*>(p + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][j] = __uint_as_float(a.w[j]);
            v[i][4 + j] = __uint_as_float(b.w[j]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = j < left ? el_load<BF16>(p + j) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      // magnitudes order like their bit patterns, infinities and NaNs on top
      unsigned top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
      // the other lane of the pair, then the other pair of the four
      top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0xb1, 0xf, 0xf, true));
      top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0x4e, 0xf, 0xf, true));
      const int e = max((int)(top >> 23) - 133, -126);
      const float inv = __uint_as_float((unsigned)(127 - e) << 23);
      const bool bad = top >= 0x7f800000u;
      uint32_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        w[j] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // + 1.5 * 2^23 rounds to the nearest whole number, ties to even, and leaves it in the low bits
          const float u = __builtin_amdgcn_fmed3f(v[i][4 * j + k] * inv, -127.f, 127.f) + 12582912.f;
          w[j] |= (__float_as_uint(u) & 255u) << (8 * k);
        }
        if (bad) w[j] = 0;
      }
      const int c = grp[i] * kGroup + part * 8, left = row[i] < s.rows ? s.cols - c : 0;
      int8_t* p = q + row[i] * s.cols + c;
      if (left >= 8) {
        *reinterpret_cast<Bytes<8>*>(p) = Bytes<8>{{w[0], w[1]}};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) p[j] = (int8_t)(w[j / 4] >> (8 * (j & 3)));
      }
      if (part == 0 && row[i] < s.rows) ex[row[i] * s.per + grp[i]] = bad ? kNanGroup : (int8_t)e;
    }
  }
}

// ld: values between the rows of x; columns cols .. ld - 1 (all in the last group) become zeros
template <bool BF16>
__global__ __launch_bounds__(256) void load_kernel(const Steps s, const int8_t* q, const int8_t* ex, void* xv, long long ld) {
  El<BF16>* x = (El<BF16>*)xv;
  const long long k0 = ((long long)blockIdx.x * 256 + threadIdx.x) / 4;
  const int part = threadIdx.x & 3;
  long long r = k0 / s.per;
  int g = (int)(k0 - r * s.per);
  while (r < s.rows) {
    uint32_t w[kFlight][2];
    int e[kFlight], grp[kFlight];
    long long row[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      row[i] = r;
      grp[i] = g;
      r += s.srow;
      g += s.sgroup;
      if (g >= s.per) {
        g -= s.per;
        ++r;
      }
      const int c = grp[i] * kGroup + part * 8, left = row[i] < s.rows ? s.cols - c : 0;
      const int8_t* p = q + row[i] * s.cols + c;
      w[i][0] = w[i][1] = 0;
      if (left >= 8) {
        const auto b = *reinterpret_cast<const Bytes<8>*>(p);
        w[i][0] = b.w[0];
        w[i][1] = b.w[1];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) w[i][j / 4] |= (uint32_t)(uint8_t)p[j] << (8 * (j & 3));
      }
      e[i] = row[i] < s.rows ? ex[row[i] * s.per + grp[i]] : 0;
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (row[i] >= s.rows) break;
      const int c = grp[i] * kGroup + part * 8;
      const float unit = e[i] == kNanGroup ? __uint_as_float(0x7fc00000u) : __uint_as_float((unsigned)(127 + e[i]) << 23);
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = (float)(int8_t)(w[i][j / 4] >> (8 * (j & 3))) * unit;
        if (c + j >= s.cols) v[j] = 0.f;
      }
      El<BF16>* p = x + row[i] * ld + c;
      if (c + 8 <= ld) {
        if constexpr (BF16) {
          *reinterpret_cast<Bytes<16>*>(p) =
              Bytes<16>{{pack2bf(v[0], v[1]), pack2bf(v[2], v[3]), pack2bf(v[4], v[5]), pack2bf(v[6], v[7])}};
        } else {
          Bytes<16> a, b;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a.w[j] = __float_as_uint(v[j]);
            b.w[j] = __float_as_uint(v[4 + j]);
          }
          *reinterpret_cast<Bytes<16>*>(p) = a;
          *reinterpret_cast<Bytes<16>*>(p + 4) = b;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < ld) el_store<BF16>(p + j, v[j]);
      }
    }
  }
}

int split(int rows, int cols, Steps& s) {
  s.rows = rows;
  s.cols = cols;
  s.per = (cols + kGroup - 1) / kGroup;
  const long long groups = (long long)rows * s.per;
  const int grid = (int)std::min<long long>((groups + 63) / 64, 256LL * 8);
  const long long quads = grid * 64LL;
  s.srow = (int)(quads / s.per);
  s.sgroup = (int)(quads - (long long)s.srow * s.per);
  return grid;
}

}  // namespace

hipError_t rnn_launch_ckpt_store(int bf16, int rows, int cols, const void* x, void* kept, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  int8_t* q = (int8_t*)kept;
  int8_t* ex = q + (long long)rows * cols;
  Steps t;
  const dim3 grid(split(rows, cols, t));
  if (bf16) hipLaunchKernelGGL(store_kernel<true>, grid, dim3(256), 0, s, t, x, q, ex);
  else hipLaunchKernelGGL(store_kernel<false>, grid, dim3(256), 0, s, t, x, q, ex);
  return hipGetLastError();
}

hipError_t rnn_launch_ckpt_load(int bf16, int rows, int cols, const void* kept, void* x, long long ld, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const int8_t* q = (const int8_t*)kept;
  const int8_t* ex = q + (long long)rows * cols;
  Steps t;
  const dim3 grid(split(rows, cols, t));
  if (bf16) hipLaunchKernelGGL(load_kernel<true>, grid, dim3(256), 0, s, t, q, ex, x, ld);
  else hipLaunchKernelGGL(load_kernel<false>, grid, dim3(256), 0, s, t, q, ex, x, ld);
  return hipGetLastError();
}
