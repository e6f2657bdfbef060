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
  float* states;         // [D][B][H][T] (workspace): every state, written by the forward pass
};

// C[m, n] = sum_k A[m*sam + k*sak] * B[n*sbn + k*sbk], fp32 accumulation
struct MatParams {
  int M, N, K;
  const void* A;
  long long sam, sak;
  const void* B;
  long long sbn, sbk;
  void* C;
  long long ldc;
};

}  // namespace rnnk

hipError_t rnn_launch_scan_step(int mode, int bf16, int B, int H, const void* g, const float* h, void* y, float* hy,
                                hipStream_t s);
hipError_t rnn_launch_scan_fwd(const rnnk::ScanParams& p, int mode, int bf16, hipStream_t s);
hipError_t rnn_launch_scan_bwd(const rnnk::ScanParams& p, int mode, int bf16, hipStream_t s);

hipError_t rnn_launch_mat(const rnnk::MatParams& p, int a_bf16, int b_bf16, int c_bf16, hipStream_t s);
// h = act(g) * u from gu [M][2F] fp32
hipError_t rnn_launch_act(int act, int bf16, int M, int F, const float* gu, void* h, hipStream_t s);
// dgu [M][2F] (element type) from dh [M][F] and gu [M][2F] fp32
hipError_t rnn_launch_act_bwd(int act, int bf16, int M, int F, const float* gu, const float* dh, void* dgu,
                              hipStream_t s);

hipError_t rnn_launch_ckpt_store(int bf16, int rows, int cols, const void* x, void* kept, hipStream_t s);
hipError_t rnn_launch_ckpt_load(int bf16, int rows, int cols, const void* kept, void* x, hipStream_t s);
