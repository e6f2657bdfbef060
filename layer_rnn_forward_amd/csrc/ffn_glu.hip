// The feed-forward block's projections with the gated product in the epilogue
// (ffn_gemm.h).
#include "ffn_gemm.h"

using namespace rnnk;

template <int ACT>
static hipError_t glu(const FfnGemm& p, int tile, int bf16, int save, hipStream_t s) {
  if (save == SAVE_NONE) return ffn_pick<true, true, FFN_GLU, SAVE_NONE, ACT>(p, tile, bf16, s);
  if (save == SAVE_FULL) return ffn_pick<true, true, FFN_GLU, SAVE_FULL, ACT>(p, tile, bf16, s);
  return ffn_pick<true, true, FFN_GLU, SAVE_INT8, ACT>(p, tile, bf16, s);
}

hipError_t rnn_launch_ffn_glu(const FfnGemm& p, int tile, int bf16, int save, hipStream_t s) {
  if (p.act == ACT_SILU) return glu<ACT_SILU>(p, tile, bf16, save, s);
  if (p.act == ACT_GELU) return glu<ACT_GELU>(p, tile, bf16, save, s);
  return glu<ACT_SIGMOID>(p, tile, bf16, save, s);
}
