// How the tiles of a product with a fused epilogue are dealt out to its workers
// (CTAs, or pairs of them): the host's choice, the kernel's walk over its items
// and the joining launch's list of a tile's parts, in one place, since what the
// join reads has to be what the walk wrote.  Plain C++ that the host compiles too.
//
// Whole tiles go round by round to all workers.  The tiles of a last, unfilled
// round may be split: their blocks of k are numbered through, and `dealers` workers
// take a run of them each, about as long as one another's.  A run that holds
// only a part of a tile's k leaves its sums in a slot of its worker, the first of
// its two or, for a part that does not begin the run, the second.  There are no more
// dealers than blocks, so every run has one at least, and the parts of a tile are
// those of consecutive workers.
#pragma once

#include <algorithm>

#include "fused.h"

namespace mpg {

// The first of the split tiles' blocks of k that dealer w takes.
__host__ __device__ __forceinline__ int64_t first_unit(int64_t units, int64_t w, int64_t dealers) { return units * w / dealers; }

struct FusedTile {
  int mb, nb;
};
__host__ __device__ __forceinline__ FusedTile fused_tile(const FusedProduct& p, int t) {
  // groups of tile rows, walked column by column, every other group backwards
  const int per = p.group_m * p.num_n_blk;
  const int g = t / per;
  const int first = g * p.group_m;
  const int gm = p.group_m < p.num_m_blk - first ? p.group_m : p.num_m_blk - first;
  const int within = t - g * per;
  FusedTile c;
  c.mb = first + within % gm;
  c.nb = within / gm;
  if (g & 1) c.nb = p.num_n_blk - 1 - c.nb;
  return c;
}

// A worker's tiles: the first product's whole ones round by round, then its run of
// the split tiles' blocks of k (that product's, then the second's where all of
// its tiles are dealt out: p.units_first of the blocks are the first's), then the
// second product's whole ones.  Workers p.late .. have one tile of the first product less than those before them; they
// take p.late_rounds rounds of the second's alone, about as long as that tile,
// and then go first in the rounds of all.
struct FusedItem {
  int which;                         // product
  int mb, nb, kb0, kb1;
  int slot;                          // of a part of a tile's k; -1: all of it
};
struct FusedItems {
  int t, round, worker, workers;
  int64_t u, u0, u1;
  __host__ __device__ __forceinline__ FusedItems(const FusedGemmParams& p, int w, int n) : t(w), round(0), worker(w), workers(n) {
    u = u0 = u1 = 0;
    if (w < p.dealers) {
      u = u0 = first_unit(p.units, w, p.dealers);
      u1 = first_unit(p.units, w + 1, p.dealers);
    }
  }
  template <bool kMore>                              // whether there may be a second product
  __host__ __device__ __forceinline__ bool next(const FusedGemmParams& p, FusedItem& x) {
    int tile;
    x.which = 0;
    x.kb0 = 0;
    x.kb1 = p.prod[0].num_k_blk;
    x.slot = -1;
    if (t < p.whole_tiles) {
      tile = t;
      t += workers;
    } else if (u < u1) {
      x.which = kMore && u >= p.units_first ? 1 : 0;
      const int kb = p.prod[x.which].num_k_blk;
      const int64_t v = x.which ? u - p.units_first : u;
      const int64_t j = v / kb;
      tile = (x.which ? 0 : p.whole_tiles) + (int)j;
      x.kb0 = (int)(v - j * kb);
      x.kb1 = kb - x.kb0 < u1 - u ? kb : (int)(x.kb0 + (u1 - u));
      x.slot = x.kb1 - x.kb0 == kb ? -1 : 2 * worker + (u == u0 ? 0 : 1);
      u += x.kb1 - x.kb0;
    } else if (kMore && p.prod[1].num_tiles && p.units <= p.units_first) {
      int rank = worker - p.late;
      if (rank >= 0 && round < p.late_rounds) {
        tile = round * p.late_workers + rank;
      } else {
        if (rank < 0) rank += workers;
        const int more = worker >= p.late ? round - p.late_rounds : round;
        tile = p.late_rounds * p.late_workers + more * workers + rank;
      }
      ++round;
      if (tile >= p.prod[1].num_tiles) return false;
      x.which = 1;
      x.kb1 = p.prod[1].num_k_blk;
    } else {
      return false;
    }
    const FusedTile c = fused_tile(p.prod[kMore ? x.which : 0], tile);
    x.mb = c.mb;
    x.nb = c.nb;
    return true;
  }
};

// The parts of a tile whose blocks of k are u0 .. u1 of those dealt out: `count`
// slots, `first` and then the first slots of the workers after `worker`.  One part
// is a whole tile, done without a slot.
struct FusedParts {
  int worker, count, first;
  __host__ __device__ __forceinline__ FusedParts(const FusedGemmParams& p, int64_t u0, int64_t u1) {
    worker = (int)(((u0 + 1) * p.dealers - 1) / p.units);                        // the last that begins at u0 or before
    count = (int)((u1 * p.dealers + p.units - 1) / p.units) - worker;            // up to the last that begins before u1
    first = 2 * worker + (first_unit(p.units, worker, p.dealers) < u0 ? 1 : 0);
  }
  __host__ __device__ __forceinline__ int slot(int j) const { return j ? 2 * (worker + j) : first; }
};

// ---------------------------------------------------------------------------
// the host's choice
// ---------------------------------------------------------------------------
constexpr int64_t kMinUnits = 4;       // blocks of k of a worker with a part of a tile, about
constexpr int64_t kMaxPairs = kMaxCtas / 2;

struct FusedShape {
  int64_t mb, nb, kb, tiles, units;    // blocks of one matrix and one part of k; all tiles, all blocks of k
};
inline FusedShape shape_of(const FusedLaunch& l, int64_t tile) {
  const bool two = l.epi == FusedEpi::kGated || l.epi == FusedEpi::kGatedGrad;
  FusedShape s;
  s.mb = (l.m + tile - 1) / tile;
  s.nb = (l.n + (two ? tile / 2 : tile) - 1) / (two ? tile / 2 : tile);
  s.kb = (l.k + 63) / 64;
  s.tiles = s.mb * (l.second_m ? 2 : 1) * s.nb;
  s.units = s.tiles * s.kb * (l.second_k ? 2 : 1);
  return s;
}

// What the forms take on a GB300 (us): a way in and out, and a time for each
// block of 64 k of a round of tiles.  Workers with parts of split tiles are at
// different places of k: where the operands do not fit into L2 each fetches its
// own blocks, at about 8300 bytes a ns together (a last round of 52 pairs' tiles
// over k = 32768, dealt to 76: 210 us where the round takes 173), so that
// splitting pays where it gives many idle workers something to do.  The parts
// go through memory twice, and the second launch takes 3 us.
// Split behind whole rounds, against one more round (us, gated tokens x hidden x inner
// and losses tokens x hidden over classes):
//   gated  64 x 4096 x  9856     2 tiles behind 152    36.9 |  45.8
//   gated  64 x 4096 x 10300     9 behind 152          40.4 |  49.2
//   gated 256 x 4096 x  9856     1 behind 76           43.1 |  49.0
//   gated 2183 x 4096 x 2131     1 behind 152          55.8 |  63.5
//   gated 256 x 4096 x 10500     7 behind 76           52.8 |  51.7
//   gated 4096 x 4096 x 4920    16 behind 608           182 |   181
//   loss   64 x 4096, 19500      1 behind 152          39.0 |  50.5
//   loss  120 x 2304, 58752      3 behind 456          57.8 |  61.6
//   loss 1092 x 2752, 93248      1 behind 1824          369 |   378
//   loss 1024 x 2048,  9800      4 behind 152          47.2 |  46.2
constexpr double kOneEpi = 1.9, kPairEpi = 3.8;    // a tile's way out, beside the next one's products
constexpr double kOneEdge = 4.3, kPairEdge = 7.5, kOneBlock = 0.29, kPairBlock = 0.31;
constexpr double kJoin = 3.0, kApartBytes = 8.3e6, kPartBytes = 5.0e6;     // bytes a us
constexpr double kL2Bytes = 100e6;

// Dealers of tiles split into `units` blocks of k: never more than blocks, since a tile has one at least.
inline int64_t dealers_of(int64_t tiles, int64_t units, int64_t most) {
  return std::min(most, std::max(tiles, units / kMinUnits));
}

struct FusedDeal {
  int64_t workers, whole, dealers;     // whole: tiles taken round by round; dealers: workers with a run of the others' blocks
  double time;
};
inline FusedDeal deal(const FusedLaunch& l, int64_t tile, int64_t most, bool may_split) {
  const FusedShape s = shape_of(l, tile);
  const double edge = tile == 256 ? kPairEdge : kOneEdge, block = tile == 256 ? kPairBlock : kOneBlock;
  const int64_t kb = s.units / s.tiles;
  const int64_t rounds = (s.tiles + most - 1) / most;
  const double round = std::max((double)kb * block, tile == 256 ? kPairEpi : kOneEpi);
  FusedDeal d{std::min(s.tiles, most), s.tiles, 0, edge + (double)rounds * round};
  const int64_t rest = s.tiles % most;
  if (!may_split || !rest || kb < 2) return d;
  const int64_t whole = s.tiles - rest;
  const int64_t dealers = dealers_of(rest, rest * kb, most);
  const double operands = 128.0 * (double)kb * (double)((l.second_m ? 2 : 1) * l.m + l.n);
  const double apart = operands < kL2Bytes ? block : std::max(block, 256.0 * (double)tile * (double)dealers / kApartBytes);
  const double parts = (double)(rest + dealers) * (double)(tile * tile) * 4.0;
  const double time = edge + kJoin + 2.0 * parts / kPartBytes + (double)(whole / most) * round +
                      (double)((rest * kb + dealers - 1) / dealers) * apart;
  if (time < d.time) d = FusedDeal{whole ? most : dealers, whole, dealers, time};
  return d;
}

}  // namespace mpg
