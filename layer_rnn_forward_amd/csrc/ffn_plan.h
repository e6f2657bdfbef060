// Host side of the feed-forward block's products: tile sizes and splits.
#pragma once

#include <algorithm>

#include "lm_common.h"

namespace rnnk {

constexpr int kStep = 128;     // bytes of k in a step
constexpr int kStagesA = 3, kStagesB = 2;   // steps of each operand in LDS
constexpr int kLds = 160 * 1024;            // of a CU

// Tiles: 256 x 256, 128 x 128, 64 x 64 (of the gated product 64 x 128).
enum FfnTile { TILE_256 = 0, TILE_128 = 1, TILE_64 = 2 };
constexpr int kTile[3] = {256, 128, 64};

// LDS of a workgroup, and workgroups that a CU holds: as many as fit its LDS
// (one of 256 x 256, two of 128 x 128 and of 64 x 128), three of 64 x 64 (its
// registers).
constexpr int ffn_lds(int rows, int cols) { return (kStagesA * rows + kStagesB * cols) * kStep; }
constexpr int ffn_places(int tile, bool glu) {
  const int fit = kLds / ffn_lds(kTile[tile], glu && tile == TILE_64 ? 128 : kTile[tile]);
  return fit < 3 ? fit : 3;
}

inline long long ffn_tiles(const FfnGemm& p, int tile, bool glu) {
  if (p.M <= 0 || p.N <= 0) return 0;
  const int fn = !glu ? kTile[tile] : tile == TILE_64 ? 64 : kTile[tile] / 2;   // columns of C
  return ((long long)p.M + kTile[tile] - 1) / kTile[tile] * (((long long)p.N + fn - 1) / fn);
}
// Accumulators of a tile.
inline int ffn_area(int tile, bool glu) { return kTile[tile] * kTile[tile] * (glu && tile == TILE_64 ? 2 : 1); }
inline long long ffn_steps(const FfnGemm& p, int bf16) {
  const int bk = kStep / (bf16 ? 2 : 4);
  return ((long long)p.K + bk - 1) / bk * p.segs;
}

struct FfnChoice {
  int tile = 0;
  int splits[3] = {1, 1, 1};
};

// Time of products that run together, longest first: their pieces are dealt
// to the places of 256 CUs.  A step's time, measured (units of 10 ns), with the
// CU to itself and with all of its places taken (in between: linear):
//   bf16   256: 1.45 us   128: 0.50 us, two a CU 0.86 us   64: 0.31 us, three a CU 0.54 us
//   fp32                  128: 1.9 us,  two a CU 3.8 us    64: 0.5 us,  three a CU 1.44 us
// of the gated product, fp32 128: 2.08 us, two a CU 3.7 us; 64 x 128: 1.22 and 2.18 us (bf16: 0.46 and 0.63 us).
inline double ffn_time(const FfnGemm* const* p, int n, int bf16, bool glu, const FfnChoice& c) {
  static constexpr double alone[2][5] = {{0, 190, 50, 208, 122}, {145, 50, 31, 50, 46}},
                          full[2][5] = {{0, 380, 144, 370, 218}, {145, 86, 54, 86, 63}};
  const int t = glu && c.tile != TILE_256 ? 2 + c.tile : c.tile, most = ffn_places(c.tile, glu);
  long long all = 0;
  double after = 0;
  for (int i = 0; i < n; ++i) {
    const long long pieces = ffn_tiles(*p[i], c.tile, glu) * c.splits[i];
    all += pieces;
    // a second launch, and the partial sums' way out and back at about 3 TB/s
    if (c.splits[i] > 1) after = std::max(after, 500.0) + (double)pieces * ffn_area(c.tile, glu) * 8 / 3e4;
  }
  const int occ = (int)std::max(1LL, std::min<long long>(most, (all + 255) / 256)), places = 256 * occ;
  auto step_of = [&](int held) {
    const double share = held > 1 ? (held - 1.0) / (most - 1) : 0;
    return alone[bf16][t] + share * (full[bf16][t] - alone[bf16][t]);
  };
  const double step = step_of(occ);
  // The gated product: full rounds, and the rest of the pieces on fewer places a
  // CU.  (Not for bf16's larger tiles, where a last round of one a CU takes as
  // long as one of two: 4187 x 2392 x 1224 on 128 x 128 107 us, on 256 x 256 88.)
  if (glu && (!bf16 || c.tile == TILE_64)) {
    const double steps = (double)((ffn_steps(*p[0], bf16) + c.splits[0] - 1) / c.splits[0]) + 4;
    const long long whole = all / (256 * most), rest = all - whole * 256 * most;
    return after + steps * ((double)whole * step_of(most) + (rest ? step_of((int)((rest + 255) / 256)) : 0));
  }
  struct Group {
    double time;
    long long count;
  } g[8] = {{0, places}};
  int groups = 1;
  double last = 0;
  for (int i = 0; i < n; ++i) {
    long long pieces = ffn_tiles(*p[i], c.tile, glu) * c.splits[i];
    const long long steps = (ffn_steps(*p[i], bf16) + c.splits[i] - 1) / c.splits[i];
    const double len = ((double)steps + 4) * step;   // 4: its start and end
    while (pieces > 0) {
      const long long whole = pieces / places;
      if (groups == 1 && whole > 1) {   // full rounds
        g[0].time += (double)whole * len;
        last = std::max(last, g[0].time);
        pieces -= whole * places;
        continue;
      }
      int e = 0;   // the places that are free first
      for (int k = 1; k < groups; ++k)
        if (g[k].time < g[e].time) e = k;
      const long long m = std::min(pieces, g[e].count);
      const Group put{g[e].time + len, m};
      last = std::max(last, put.time);
      pieces -= m;
      if (m == g[e].count) {
        g[e] = put;
        continue;
      }
      g[e].count -= m;
      int k = 0;
      while (k < groups && (k == e || g[k].time != put.time)) ++k;
      if (k < groups) g[k].count += m;
      else if (groups < 8) g[groups++] = put;
      else g[e].count += m;
    }
  }
  return last + after;
}

// The tile that takes least, each with whole k and (the smaller two) with k in
// pieces of an equal share of the work for one to four places a CU, 8 steps at
// least.  A product alone has no more pieces than those places (one more would
// start a second round); with shorter products beside it, its last piece may be
// the shorter one.
// Forward's projections split or whole, cold caches: 270 x 3272 x 848 fp32 92 or
// 158 us a forward pass, 189 x 2776 x 392 bf16 28 or 48, 129 x 4096 x 4096 fp32
// 206 or 222; 70 x 2501 x 130 fp32 with gradients 108 or 175.
inline FfnChoice ffn_choose(const FfnGemm* const* p, int n, int bf16, bool glu, bool may_split) {
  FfnChoice best;
  double least = -1;
  for (int t = bf16 ? TILE_256 : TILE_128; t <= TILE_64; ++t) {
    long long work = 0;
    for (int i = 0; i < n; ++i) work += ffn_tiles(*p[i], t, glu) * ffn_steps(*p[i], bf16);
    for (int share = 0; share <= (may_split && t != TILE_256 ? 4 : 0); ++share) {
      FfnChoice c;
      c.tile = t;
      if (share) {
        const long long piece = std::max(8LL, (work + 256 * share - 1) / (256 * share));
        bool any = false;
        for (int i = 0; i < n; ++i) {
          const long long steps = ffn_steps(*p[i], bf16);
          if (2 * steps >= 3 * piece) c.splits[i] = (int)std::min(64LL, n > 1 ? (steps + piece - 1) / piece : steps / piece);
          any = any || c.splits[i] > 1;
        }
        if (!any) continue;
      }
      const double time = ffn_time(p, n, bf16, glu, c);
      if (least < 0 || time < least) {
        least = time;
        best = c;
      }
    }
  }
  return best;
}

// Bytes of the partial sums of product i.
inline size_t ffn_part(const FfnGemm& p, const FfnChoice& c, int i, bool glu) {
  if (c.splits[i] <= 1) return 0;
  return (size_t)ffn_tiles(p, c.tile, glu) * c.splits[i] * ffn_area(c.tile, glu) * 4;
}

// Bounds of the partial sums over all numbers of rows up to some M, so that a
// workspace of M rows does for fewer.  With pieces of at least work / 1024 and 8
// steps, a product alone is split while it has at most 512 tiles, into 1024
// pieces at most; of several, one that is split has at least 3 work / 2048
// steps, and the pieces are at most 1024 and one a tile of theirs.
inline long long ffn_pieces(const FfnGemm& p, int tile, int bf16, bool glu) {
  const long long steps = ffn_steps(p, bf16);
  return steps < 12 ? 0 : ffn_tiles(p, tile, glu) * std::min(64LL, (steps + 7) / 8);
}
// Forward's product p: its bound, and the rows m <= p.M at which it is reached.
inline size_t ffn_part_bound(const FfnGemm& p, int tile, int bf16, bool glu, int& m) {
  FfnGemm q = p;
  q.M = 1;
  const long long across = ffn_tiles(q, tile, glu);
  m = across ? (int)std::min<long long>(p.M, 512 / across * kTile[tile]) : 0;
  q.M = m;
  return (size_t)std::min(1024LL, ffn_pieces(q, tile, bf16, glu)) * ffn_area(tile, glu) * 4;
}
// Backward's: dx has more tiles with more rows, and the others more steps.
inline size_t ffn_part_bound(const FfnGemm (&p)[3], int tile, int bf16, int& m) {
  FfnGemm q = p[0], one = p[1];
  const long long fixed = ffn_tiles(p[1], tile, false) + ffn_tiles(p[2], tile, false), deep = ffn_steps(p[0], bf16);
  auto splits = [&](int rows) {   // whether dx may be
    q.M = one.K = rows;
    return 3 * (ffn_tiles(q, tile, false) * deep + fixed * ffn_steps(one, bf16)) <= 2048 * deep;
  };
  int lo = 0, hi = p[0].M;
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (splits(mid)) lo = mid;
    else hi = mid - 1;
  }
  q.M = m = lo;
  long long pieces = ffn_pieces(q, tile, bf16, false), tiles = ffn_tiles(q, tile, false);
  if (fixed <= 682 && ffn_pieces(p[1], tile, bf16, false) + ffn_pieces(p[2], tile, bf16, false) > 0) {
    pieces += ffn_pieces(p[1], tile, bf16, false) + ffn_pieces(p[2], tile, bf16, false);
    tiles += fixed;
    m = p[0].M;
  }
  return (size_t)std::min(1024 + tiles, pieces) * ffn_area(tile, false) * 4;
}

// The products that may be split, by their sizes alone: forward's two, and
// backward's last three, longest first (the order that ffn_choose_backward
// gives).
inline void ffn_gated_product(int M, int D, int F, FfnGemm& g) {
  g.M = M;
  g.N = F;
  g.K = D;
  g.segs = 1;
}
inline void ffn_forward_product(int M, int D, int F, FfnGemm& o) {
  o.M = M;
  o.N = D;
  o.K = F;
  o.segs = 1;
}
inline void ffn_backward_products(int M, int D, int F, int Fp, FfnGemm (&o)[3]) {
  o[0].M = M;             // dx: k runs over dgate's columns, then dup's
  o[0].N = D;
  o[0].K = F;
  o[0].segs = 2;
  o[0].kseg = Fp;
  o[1].M = F > 0 ? 2 * Fp : 0;   // dw_in: rows of dgate and dup with their padding
  o[1].N = D;
  o[1].K = M;
  o[1].segs = 1;
  o[1].mseg = Fp;
  o[1].mreal = F;
  o[2].M = D;             // dw_out
  o[2].N = F;
  o[2].K = M;
  o[2].segs = 1;
}
inline FfnChoice ffn_choose_forward(const FfnGemm& o, int bf16, bool glu) {
  const FfnGemm* one[1] = {&o};
  return ffn_choose(one, 1, bf16, glu, true);
}
// splits in the products' own order; order: longest first
inline FfnChoice ffn_choose_backward(const FfnGemm (&o)[3], int bf16, int (&order)[3]) {
  order[0] = 0, order[1] = 1, order[2] = 2;
  if (ffn_steps(o[0], bf16) < ffn_steps(o[1], bf16)) order[0] = 1, order[1] = 2, order[2] = 0;
  const FfnGemm* sorted[3] = {&o[order[0]], &o[order[1]], &o[order[2]]};
  const FfnChoice c = ffn_choose(sorted, 3, bf16, false, true);
  FfnChoice r;
  r.tile = c.tile;
  for (int i = 0; i < 3; ++i) r.splits[order[i]] = c.splits[i];
  return r;
}

}  // namespace rnnk
