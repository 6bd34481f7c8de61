// How vocab_head.cu cuts its products into tiles, deals them to the CTA pairs
// and cuts the vocabulary into pieces.  Index arithmetic only, for the host as
// well.
#pragma once

#include <algorithm>

#include "moe_device.cuh"

namespace moe {

namespace {

constexpr int kTile = 256;      // rows and columns of a pair's tile
constexpr int kBK = 128;        // k of a stage
// Row tiles that are worked on side by side, all of them before the next run of
// the vocabulary.  Without stores many share a read of W (64: 1242 us at 32768 x
// 768 x 50001, 24: 1260; 2133 and 2167 at 8192 x 2048 x 131072); dz of few rows at a
// time is written with less contention (24: 1486 us, 64: 1492, 128: 1528, 8: 1518; of
// the wider case's 32 row tiles 24 2328, 64 2310, 8 2391).
constexpr int kGroupStats = 64, kGroupDz = 24;

enum Mode { kStats, kDz, kGrad };

// What one launch has to do.
struct VocabWork {
  int nmt, nnt;    // kStats, kDz: row tiles, vocabulary tiles
  int run, items;  // vocabulary tiles of one item; items in all
  // k blocks of a tile; kGrad: of dx (0) and of dW (1), with the splits along
  // them, the tiles and the units that this makes
  int nkb[2];
  int splits[2], n_units[2], tiles_m[2], tiles_n;
  int longer;  // which of the two has the longer units
};

// What a unit takes, in k blocks: its own and one to begin with, or the epilogue
// that runs beside the next unit's, about three (backward of 8 x 704 x 194036: 189
// us; with its own blocks, but at least two of them 200, at least four 202; of 300 x
// 1024 x 100000: 207, with at least three and none to begin with 222).
__host__ MOE_DEV int unit_cost(int nkb, int splits) {
  const int blocks = (nkb + splits - 1) / splits;
  return blocks > 2 ? blocks + 1 : 3;
}

__host__ MOE_DEV int least(int a, int b) { return a < b ? a : b; }

struct Unit {
  int m, n;         // tile
  int kb0, kb1;     // k blocks
  int which;        // kGrad: 0 dx, 1 dW
  int split;
  int first, last;  // kStats, kDz: of its run
  int slot;         // the run
};

// The units of pair `pair` in order; every role of both CTAs walks the same list.
template <int kMode>
struct Walk {
  int it = -1;

  __host__ MOE_DEV bool next(const VocabWork& p, int pair, int npairs, Unit& u) {
    constexpr int kGroup = kMode == kStats ? kGroupStats : kGroupDz;
    for (;;) {
      ++it;
      const int item = pair + it / p.run * npairs;
      if (item >= p.items) return false;
      const int sub = it % p.run;
      // row tiles in groups; within a group all its rows before the next run of the vocabulary
      const int runs = (p.nnt + p.run - 1) / p.run;
      const int g = item / (kGroup * runs);
      const int in_group = least(kGroup, p.nmt - g * kGroup);
      const int r = item - g * kGroup * runs;
      u.slot = r / in_group;
      u.m = g * kGroup + r % in_group;
      u.n = u.slot * p.run + sub;
      if (u.n >= p.nnt) continue;
      u.first = sub == 0;
      u.last = sub == p.run - 1 || u.n == p.nnt - 1;
      u.kb0 = 0;
      u.kb1 = p.nkb[0];
      u.which = 0;
      u.split = 0;
      return true;
    }
  }
};

// kGrad: the class of longer units first, dealt round robin; then the other's: as
// many as fit go to the pairs that got one long unit less, the rest to all.  Where
// a pair's share of each begins is worked out once, not for every unit (1290 x 576
// x 72446: 290 us, with those divisions 305).
template <>
struct Walk<kGrad> {
  int stage = -1, idx = 0, step = 0, left = 0;

  __host__ MOE_DEV void begin(const VocabWork& p, int pair, int npairs) {
    const int a = p.longer, b = a ^ 1, na = p.n_units[a], nb = p.n_units[b];
    const int r = na % npairs;  // the first r pairs have one more
    const int cost_a = unit_cost(p.nkb[a], p.splits[a]), cost_b = unit_cost(p.nkb[b], p.splits[b]);
    const int fill = r == 0 ? 0 : least(nb, (npairs - r) * (cost_a / cost_b));
    int end;
    if (stage == 0) {
      idx = pair, step = npairs, end = na;
    } else if (stage == 1) {
      idx = pair >= r ? pair - r : fill, step = npairs - r, end = fill;
    } else {
      idx = fill + (pair - r + npairs) % npairs, step = npairs, end = nb;
    }
    left = idx < end ? (end - idx - 1) / step + 1 : 0;
  }

  __host__ MOE_DEV bool next(const VocabWork& p, int pair, int npairs, Unit& u) {
    idx += step;
    while (left == 0) {
      if (++stage == 3) return false;
      begin(p, pair, npairs);
    }
    --left;
    const int which = stage == 0 ? p.longer : p.longer ^ 1;
    const unsigned tile = static_cast<unsigned>(idx) / static_cast<unsigned>(p.tiles_n);
    u.which = which;
    u.n = idx - static_cast<int>(tile) * p.tiles_n;
    u.split = 0;
    u.m = static_cast<int>(tile);
    u.kb0 = 0;
    u.kb1 = p.nkb[which];
    if (p.splits[which] > 1) {
      // splits differ by at most one block, and none is empty
      u.split = u.m / p.tiles_m[which];
      u.m -= u.split * p.tiles_m[which];
      u.kb0 = p.nkb[which] * u.split / p.splits[which];
      u.kb1 = p.nkb[which] * (u.split + 1) / p.splits[which];
    }
    return true;
  }
};

constexpr int kPlanPairs = 76;  // pairs that work is planned for (the plans decide the workspaces)

inline int ceil_div(long a, long b) { return static_cast<int>((a + b - 1) / b); }

// Vocabulary tiles of one item.  A longer run writes fewer pairs; the items are
// dealt round robin, so it must leave each pair many, or just one where that
// takes no more rounds of tiles (219 x 576 x 143711: 43 us, with runs of one tile 50;
// 30 x 4096 x 50346: 80 and 83).
inline int run_of(int nmt, int nnt) {
  const long tiles = static_cast<long>(nmt) * nnt;
  if (nmt <= kPlanPairs) {
    const int run = ceil_div(nnt, kPlanPairs / nmt);
    if (run <= ceil_div(tiles, kPlanPairs)) return run;
  }
  return tiles >= 64 * kPlanPairs ? 4 : tiles >= 24 * kPlanPairs ? 2 : 1;
}

struct ForwardPlan {
  int nmt, nnt, run, runs, rows_padded;
};
inline ForwardPlan forward_plan(int T, int V) {
  ForwardPlan f;
  f.nmt = ceil_div(T, kTile);
  f.nnt = ceil_div(V, kTile);
  f.run = run_of(f.nmt, f.nnt);
  f.runs = ceil_div(f.nnt, f.run);
  f.rows_padded = ceil_div(T, 32) * 32;
  return f;
}

// Most bytes of dz that one piece holds, except that it may have kLeastPiece columns at
// any number of tokens: past 2^20 those are more, 64 GiB at 2^24.
constexpr size_t kPieceBytes = static_cast<size_t>(1) << 32;
constexpr int kLeastPiece = 8 * kTile;
constexpr int kMinSplitBlocks = 12;                           // k blocks that a split has at least
constexpr int kMaxSplits = kPlanPairs;                        // (32 x 64 x 150000: 59 us, with up to 16 splits 76)

struct BackwardPlan {
  int piece, pieces;       // vocabulary rows of a piece
  int nmt, ndt;
  int splits_x, splits_w;
};
inline BackwardPlan backward_plan(int T, int D, int V) {
  BackwardPlan b;
  const long most = static_cast<long>(kPieceBytes / 2 / static_cast<size_t>(std::max(T, 1))) / kTile * kTile;
  b.pieces = ceil_div(V, std::max<long>(most, kLeastPiece));
  b.piece = b.pieces == 1 ? ceil_div(V, 64) * 64 : ceil_div(ceil_div(V, b.pieces), kTile) * kTile;
  b.pieces = ceil_div(V, b.piece);
  b.nmt = ceil_div(T, kTile);
  b.ndt = ceil_div(D, kTile);
  // A tile whose reduction is longer than a pair's share of all work is split
  // along it.
  const long kx = ceil_div(b.piece, kBK), kw = ceil_div(T, kBK);
  const long ux = static_cast<long>(b.nmt) * b.ndt, uw = static_cast<long>(ceil_div(b.piece, kTile)) * b.ndt;
  const long work = ux * unit_cost(kx, 1) + uw * unit_cost(kw, 1);
  const long share = std::max<long>(kMinSplitBlocks, (work + kPlanPairs - 1) / kPlanPairs);
  b.splits_x = static_cast<int>(std::min<long>(kMaxSplits, (kx + share - 1) / share));
  b.splits_w = b.pieces > 1 ? 1 : static_cast<int>(std::min<long>(kMaxSplits, (kw + share - 1) / share));
  return b;
}

inline VocabWork forward_work(const ForwardPlan& f, int D) {
  VocabWork w = {};
  w.nmt = f.nmt;
  w.nnt = f.nnt;
  w.run = f.run;
  w.items = f.nmt * f.runs;
  w.nkb[0] = ceil_div(D, kBK);
  return w;
}

// Both launches of a piece of Vc rows: the tiles of dz and the units of its products.
inline VocabWork dz_work(const BackwardPlan& b, int D, int Vc) {
  VocabWork w = {};
  w.nmt = b.nmt;
  w.nnt = ceil_div(Vc, kTile);
  w.run = run_of(w.nmt, w.nnt);
  w.items = w.nmt * ceil_div(w.nnt, w.run);
  w.nkb[0] = ceil_div(D, kBK);
  return w;
}
inline VocabWork grad_work(const BackwardPlan& b, int T, int Vc) {
  VocabWork w = {};
  w.nkb[0] = ceil_div(Vc, kBK);
  w.nkb[1] = ceil_div(T, kBK);
  w.splits[0] = std::min(b.splits_x, w.nkb[0]);  // the last piece may be a short one
  w.splits[1] = b.splits_w;
  w.tiles_n = b.ndt;
  w.tiles_m[0] = b.nmt;
  w.tiles_m[1] = ceil_div(Vc, kTile);
  for (int i = 0; i < 2; ++i) w.n_units[i] = w.tiles_m[i] * w.tiles_n * w.splits[i];
  w.longer = w.nkb[0] / w.splits[0] >= w.nkb[1] / w.splits[1] ? 0 : 1;
  return w;
}

}  // namespace

}  // namespace moe
