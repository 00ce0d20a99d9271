// Host side of the products with fused epilogues: which form a product takes,
// how its tiles are dealt out, and the launch.
#include <cstring>

#include "fused.h"

namespace mpg {

namespace {

constexpr int64_t kMinUnits = 4;       // blocks of k of a worker with a part of a tile, at least
constexpr int64_t kMaxPairs = kMaxCtas / 2;

struct Shape {
  int64_t mb, nb, kb, tiles, units;    // blocks of one matrix and one part of k; all tiles, all blocks of k
};
Shape shape_of(const FusedLaunch& l, int64_t tile) {
  const bool two = l.epi == FusedEpi::kGated || l.epi == FusedEpi::kGatedGrad;
  Shape s;
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
constexpr double kOneEdge = 4.3, kPairEdge = 7.5, kOneBlock = 0.29, kPairBlock = 0.31;
constexpr double kJoin = 3.0, kApartBytes = 8.3e6, kPartBytes = 5.0e6;     // bytes a us
constexpr double kL2Bytes = 100e6;

struct Deal {
  int64_t workers, whole;              // whole: tiles taken round by round
  double time;
};
Deal deal(const FusedLaunch& l, const Shape& s, int64_t tile, int64_t most, double edge, double block, bool may_split) {
  const int64_t kb = s.units / s.tiles;
  const int64_t rounds = (s.tiles + most - 1) / most;
  Deal d{std::min(s.tiles, most), s.tiles, edge + (double)(rounds * kb) * block};
  const int64_t rest = s.tiles % most;
  if (!may_split || !rest) return d;
  const int64_t whole = s.tiles - rest;
  const int64_t workers = whole ? most : std::min(most, std::max(rest, rest * kb / kMinUnits));
  const double operands = 128.0 * (double)kb * (double)((l.second_m ? 2 : 1) * l.m + l.n);
  const double apart = operands < kL2Bytes ? block : std::max(block, 256.0 * (double)tile * (double)workers / kApartBytes);
  const double parts = (double)(rest + workers) * (double)(tile * tile) * 4.0;
  const double time = edge + kJoin + 2.0 * parts / kPartBytes + (double)(whole / most * kb) * block +
                      (double)((rest * kb + workers - 1) / workers) * apart;
  if (time < d.time) d = Deal{workers, whole, time};
  return d;
}

}  // namespace

size_t fused_slot_bytes(const FusedLaunch& l) {
  size_t most = 0;
  for (int64_t tile : {(int64_t)128, (int64_t)256}) {
    const Shape s = shape_of(l, tile);
    const int64_t workers = std::min(tile == 256 ? kMaxPairs : (int64_t)kMaxCtas, std::max(s.tiles, s.units / kMinUnits));
    most = std::max(most, (size_t)(2 * workers * tile * tile) * sizeof(float));
  }
  return most;
}

mpg_status fused_map(CUtensorMap* map, const void* ptr, int64_t ld, mpg_dtype dt, bool mn_major, int64_t rows, int64_t k) {
  const Operand x{ptr, ld, 0, dt, MPG_ROW_MAJOR};
  return mn_major ? encode_map(map, x, rows, k, 1, 64, 64) : encode_map(map, x, k, rows, 1, 64, 64);
}

mpg_status launch_fused(DeviceInfo* dev, const FusedLaunch& l, FusedGemmParams& p, float* slots, cudaStream_t stream) {
  FusedKernel one, two;
  fused_lookup(l.epi, false, &one);
  fused_lookup(l.epi, true, &two);
  int pairs = 0;
  mpg_status st = resident_clusters(dev, two.fn, two.block, two.smem_bytes, 2, &pairs);
  if (st != MPG_OK) return st;
  if ((st = allow_smem(dev, one.fn, one.smem_bytes)) != MPG_OK) return st;
  const Shape s1 = shape_of(l, one.tile), s2 = shape_of(l, two.tile);
  const bool split = l.split && slots;
  const Deal d1 = deal(l, s1, one.tile, std::min(dev->sm_count, kMaxCtas), kOneEdge, kOneBlock, split);
  const Deal d2 = deal(l, s2, two.tile, std::min<int64_t>(pairs, kMaxPairs), kPairEdge, kPairBlock, split);
  const bool pair = d2.time < d1.time;
  const Shape& s = pair ? s2 : s1;
  const Deal& d = pair ? d2 : d1;
  const FusedKernel& k = pair ? two : one;
  if (s.tiles > kFusedMaxExtent || s.units / s.tiles > kFusedMaxExtent) return fail(MPG_ERR_INVALID_ARG, "too many tiles");
  p.m = (int32_t)l.m;
  p.n = (int32_t)l.n;
  p.num_m_blk = (int32_t)(s.mb * (l.second_m ? 2 : 1));
  p.num_n_blk = (int32_t)s.nb;
  p.num_k_blk = (int32_t)(s.units / s.tiles);
  p.kb_second = l.second_k ? (int32_t)s.kb : INT32_MAX;
  p.mb_second = l.second_m ? (int32_t)s.mb : INT32_MAX;
  p.num_tiles = (int32_t)s.tiles;
  p.group_m = pair ? 8 : 16;
  p.whole_tiles = (int32_t)d.whole;
  p.units = (s.tiles - d.whole) * p.num_k_blk;
  p.slots = slots;
  p.status = dev->status;
  p.wait_limit_ns = kDefaultWaitNs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(d.workers * k.ctas));
  cfg.blockDim = dim3((unsigned)k.block);
  cfg.dynamicSmemBytes = (size_t)k.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, k.ctas);
  cfg.attrs = attr;
  void* args[] = {&p};
  cudaError_t e = cudaLaunchKernelExC(&cfg, k.fn, args);
  if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "product launch: %s", cudaGetErrorString(e));
  if (p.units) {
    e = launch_fused_join(p, k.tile, (int)d.workers, stream);
    if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "join launch: %s", cudaGetErrorString(e));
  }
  return MPG_OK;
}

}  // namespace mpg
