// Host program over ffn_plan.h: "places" prints, for each tile and kind of product, the workgroups a CU is taken to hold,
// a workgroup's LDS and a CU's; otherwise the arguments are M D F bf16 ..., and each line has the tiles and splits chosen
// for the gated product, its gradient, y, and the three gradients.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "ffn_plan.h"

using namespace rnnk;

int main(int argc, char** argv) {
  if (argc > 1 && !std::strcmp(argv[1], "places")) {
    for (int glu = 0; glu < 2; ++glu)
      for (int t = TILE_256; t <= TILE_64; ++t)
        std::printf("%d %d %d %d %d\n", glu, kTile[t], ffn_places(t, glu), ffn_lds(kTile[t], glu && t == TILE_64 ? 128 : kTile[t]),
                    kLds);
    return 0;
  }
  for (int i = 1; i + 3 < argc; i += 4) {
    const int M = std::atoi(argv[i]), D = std::atoi(argv[i + 1]), F = std::atoi(argv[i + 2]), bf = std::atoi(argv[i + 3]);
    FfnGemm g{}, y{}, q[3] = {};
    ffn_gated_product(M, D, F, g);
    ffn_forward_product(M, D, F, y);
    ffn_backward_products(M, D, F, (F + 63) / 64 * 64, q);
    int order[3];
    const FfnGemm* one[1] = {&g};
    const FfnChoice cg = ffn_choose_forward(g, bf, true), cd = ffn_choose(one, 1, bf, false, false),
                    cy = ffn_choose_forward(y, bf, false), cq = ffn_choose_backward(q, bf, order);
    std::printf("%d %d %d %d %d %d %d %d %d\n", kTile[cg.tile], cg.splits[0], kTile[cd.tile], kTile[cy.tile], cy.splits[0],
                kTile[cq.tile], cq.splits[0], cq.splits[1], cq.splits[2]);
  }
}
