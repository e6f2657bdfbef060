// The gradient of the feed-forward block's gated product, in the epilogue of
// dy W (ffn_gemm.h).
#include "ffn_gemm.h"

using namespace rnnk;

// with RNN_SAVE_FULL the activation is in what was saved
hipError_t rnn_launch_ffn_dglu(const FfnGemm& p, int bf16, int save, hipStream_t s) {
  const FfnGemm* one[1] = {&p};
  const int tile = ffn_choose(one, 1, bf16, false, false).tile;
  if (save == SAVE_FULL) return ffn_pick<true, false, FFN_DGLU, SAVE_FULL, ACT_SILU>(p, tile, bf16, s);
  if (p.act == ACT_SILU) return ffn_pick<true, false, FFN_DGLU, SAVE_INT8, ACT_SILU>(p, tile, bf16, s);
  if (p.act == ACT_GELU) return ffn_pick<true, false, FFN_DGLU, SAVE_INT8, ACT_GELU>(p, tile, bf16, s);
  return ffn_pick<true, false, FFN_DGLU, SAVE_INT8, ACT_SIGMOID>(p, tile, bf16, s);
}
