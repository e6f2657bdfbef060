// Parameters and launchers of the language-model operators: gated scan,
// gated feed-forward block, 8-bit checkpoints (include/rnn.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rnnk {

enum ScanMode { SCAN_GATED = 0, SCAN_LINEAR = 1 };
enum Act { ACT_SIGMOID = 0, ACT_SILU = 1, ACT_GELU = 2 };
enum Save { SAVE_NONE = 0, SAVE_FULL = 1, SAVE_INT8 = 2 };

constexpr int kGroup = 32;   // columns that share one exponent in a checkpoint

// Scan: the forward pass keeps the state before every kScanKeep-th step; for
// each pass the steps of a wave's piece (multiples of kScanKeep), the waves of
// a workgroup, the chunks between two published states
constexpr int kScanKeep = 8;
constexpr int kScanFwdSteps = 16, kScanFwdWaves = 8, kScanFwdSuper = 8, kScanFwdEu = 4;
constexpr int kScanBwdSteps = 8, kScanBwdWaves = 8, kScanBwdSuper = 4, kScanBwdEu = 4;

struct ScanParams {
  int T, B, H, D;
  const void* g;
  const float* h0;       // or null
  const int* lengths;    // or null
  void* y;               // forward
  float* hy;             // forward, or null
  const void* dy;        // backward
  const float* dhy;      // backward, or null
  void* dg;              // backward
  float* dh0;            // backward, or null
  int waves, chunks;     // chunks of `waves` pieces
  int spin_limit;        // polls of a wait before it expires
  // workspace, in this order: [0], [1] a wait of the forward, of the backward
  // pass expired (256 bytes); started chunks
  // of each workgroup's channels, 64 bytes apart; the chunks' maps (A, B), the
  // states before every group of chunks and the states after chunks that had
  // to be walked, contiguous; the state before every kScanKeep-th step
  unsigned* head;
  unsigned* counters;        // [ceil(B * H / 64)][D][16]
  unsigned long long* maps;  // [chunks][D][B][H]
  float* state;              // [chunks / group + 1][D][B][H], from the caller's first on
  float* ends;               // [chunks][D][B][H]
  float* starts;             // [ceil(T / kScanKeep)][D][B][H]
};

// One product of the feed-forward block (ffn_gemm.h).  Leading dimensions in
// elements, multiples of 16 bytes; bases 16-byte aligned.
struct FfnGemm {
  int M, N, K;           // N: columns of C (the gated product's: F)
  const void* A;
  long long lda;
  const void* B;         // FFN_GLU: F gate rows, then F up rows
  long long ldb;
  void* C;
  long long ldc;
  int cvec;              // 16-byte stores of C are aligned
  // K in `segs` (1 or 2) segments: K real values each; the second starts kseg
  // later in A and K later in B
  int segs, kseg;
  // mseg > 0: rows [0, mreal) and [mseg, mseg + mreal) of the product are
  // rows [0, 2 * mreal) of C
  int mseg, mreal;
  // splits > 1: k in that many pieces, whose sums are added in a second launch
  int splits;
  void* part;
  int act;
  // saved for backward in tiles of 32 x 32 with their exponents, lds tiles a
  // row of tiles: act(g) and u act'(g) (RNN_SAVE_FULL; 16 bits, or fp32
  // without exponents), or g and u (RNN_SAVE_INT8)
  void* s0;
  void* s1;
  int8_t* e0;
  int8_t* e1;
  long long lds;
  void* h;               // FFN_DGLU with RNN_SAVE_INT8: the gated product, again
  long long ldh;
};

// One product of the block for few rows (ffn_rows.hip): w [R or 2R, K]
// contiguous, any alignment.
constexpr int kFfnRows = 64;   // rows at most
// bf16: the gated product's rows are followed by the rests of their rounding
struct FfnRows {
  int M, R, K;
  const void* x;
  long long ldx;
  const void* w;
  void* out;
  long long ldo;
  int act;               // of the gated product
};

// Copies of up to four matrices with rows padded by zeros to a multiple of
// 16 bytes.
struct PadJob {
  int n;
  const void* src[4];
  void* dst[4];
  long long rows[4];
  int cols[4], ld[4];    // ld: columns of dst
};

}  // namespace rnnk

hipError_t rnn_launch_scan_step(int mode, int bf16, int B, int H, const void* g, const float* h, void* y, float* hy,
                                hipStream_t s);
hipError_t rnn_launch_scan_fwd(const rnnk::ScanParams& p, int mode, int bf16, hipStream_t s);
hipError_t rnn_launch_scan_bwd(const rnnk::ScanParams& p, int mode, int bf16, hipStream_t s);

hipError_t rnn_launch_ffn_glu(const rnnk::FfnGemm& p, int tile, int bf16, int save, hipStream_t s);
hipError_t rnn_launch_ffn_dglu(const rnnk::FfnGemm& p, int bf16, int save, hipStream_t s);
// y, and dx, dw_in, dw_out (those that are not wanted have M = 0); `order`:
// longest first
hipError_t rnn_launch_ffn_store(const rnnk::FfnGemm& p, int tile, int bf16, hipStream_t s);
hipError_t rnn_launch_ffn_grads(const rnnk::FfnGemm (&p)[3], const int (&order)[3], int tile, int bf16, hipStream_t s);
hipError_t rnn_launch_ffn_rows(const rnnk::FfnRows& p, int bf16, int glu, hipStream_t s);
hipError_t rnn_launch_pad(const rnnk::PadJob& j, int bf16, hipStream_t s);

hipError_t rnn_launch_ckpt_store(int bf16, int rows, int cols, const void* x, void* kept, hipStream_t s);
// ld: elements between the rows of x; columns from cols on are set to zero
hipError_t rnn_launch_ckpt_load(int bf16, int rows, int cols, const void* kept, void* x, long long ld, hipStream_t s);
