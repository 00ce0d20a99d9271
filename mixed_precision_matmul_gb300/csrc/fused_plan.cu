// Host side of the products with fused epilogues: which form a product takes,
// how its tiles are dealt out, and the launch.
#include <cstring>
#include <utility>

#include "fused_deal.h"

namespace mpg {

size_t fused_slot_bytes(const FusedLaunch& l, const FusedLaunch* second) {
  size_t most = 0;
  for (int64_t tile : {(int64_t)128, (int64_t)256}) {
    FusedShape s = shape_of(l, tile);
    if (second) {
      const FusedShape t = shape_of(*second, tile);
      s.tiles += t.tiles;
      s.units += t.units;
    }
    if (s.units == s.tiles) return 0;                 // (one block of k is not split)
    const int64_t workers = std::min(tile == 256 ? kMaxPairs : (int64_t)kMaxCtas, std::max(s.tiles, s.units / kMinUnits));
    most = std::max(most, (size_t)(2 * workers * tile * tile) * sizeof(float));
  }
  return most;
}

mpg_status fused_map(CUtensorMap* map, const void* ptr, int64_t ld, mpg_dtype dt, bool mn_major, int64_t rows, int64_t k) {
  const Operand x{ptr, ld, 0, dt, MPG_ROW_MAJOR};
  return mn_major ? encode_map(map, x, rows, k, 1, 64, 64) : encode_map(map, x, k, rows, 1, 64, 64);
}

namespace {

struct Forms {
  FusedKernel kernel[2];               // on single CTAs, on pairs
  int64_t workers[2];
};
mpg_status forms_of(DeviceInfo* dev, FusedEpi epi, int act, Forms* f) {
  for (int pair = 0; pair < 2; ++pair) {
    FusedKernel* k = &f->kernel[pair];
    switch (epi) {
      case FusedEpi::kPlain: fused_lookup_plain(pair, k); break;
      case FusedEpi::kGated: fused_lookup_gated(pair, act, k); break;
      case FusedEpi::kGatedGrad: fused_lookup_gated_grad(pair, act, k); break;
      default: fused_lookup_loss(epi, pair, k);
    }
  }
  int pairs = 0;
  const FusedKernel& two = f->kernel[1];
  mpg_status st = resident_clusters(dev, two.fn, two.block, two.smem_bytes, 2, &pairs);
  if (st != MPG_OK) return st;
  f->workers[0] = std::min(dev->sm_count, kMaxCtas);
  f->workers[1] = std::min<int64_t>(pairs, kMaxPairs);
  return allow_smem(dev, f->kernel[0].fn, f->kernel[0].smem_bytes);
}
FusedDeal deal_form(const FusedLaunch& l, const Forms& f, int pair, bool split) {
  return deal(l, f.kernel[pair].tile, f.workers[pair], split);
}

mpg_status fill_product(FusedProduct& p, const FusedLaunch& l, int64_t tile, bool pair) {
  const FusedShape s = shape_of(l, tile);
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
  return MPG_OK;
}

// dealers: of the workers, those with a run of the split tiles' blocks of k;
// dealt: both products' tiles are split.
mpg_status launch(DeviceInfo* dev, const FusedKernel& k, FusedGemmParams& p, int64_t workers, int64_t dealers, bool dealt,
                  float* slots, cudaStream_t stream) {
  p.units_first = (int64_t)(p.prod[0].num_tiles - p.whole_tiles) * p.prod[0].num_k_blk;
  p.units = p.units_first + (dealt ? (int64_t)p.prod[1].num_tiles * p.prod[1].num_k_blk : 0);
  p.dealers = (int32_t)dealers;
  // (a dealer without a block would leave its slots as they are, and the join adds them)
  if (dealers > workers || p.units < dealers || (p.units > 0) != (dealers > 0))
    return fail(MPG_ERR_INVALID_ARG, "%lld blocks for %lld of %lld workers", (long long)p.units, (long long)dealers, (long long)workers);
  p.slots = slots;
  p.status = dev->status;
  p.wait_limit_ns = kDefaultWaitNs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(workers * k.ctas));
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
    e = k.join(p, stream);
    if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "join launch: %s", cudaGetErrorString(e));
  }
  return MPG_OK;
}

}  // namespace

mpg_status launch_fused(DeviceInfo* dev, const FusedLaunch& l, FusedGemmParams& p, float* slots, cudaStream_t stream) {
  Forms f;
  mpg_status s = forms_of(dev, l.epi, p.act, &f);
  if (s != MPG_OK) return s;
  const bool split = slots != nullptr;
  const FusedDeal d1 = deal_form(l, f, 0, split), d2 = deal_form(l, f, 1, split);
  const int pair = d2.time < d1.time;
  const FusedDeal& d = pair ? d2 : d1;
  if ((s = fill_product(p.prod[0], l, f.kernel[pair].tile, pair)) != MPG_OK) return s;
  p.prod[1].num_tiles = 0;
  p.whole_tiles = (int32_t)d.whole;
  return launch(dev, f.kernel[pair], p, d.workers, d.dealers, false, slots, stream);
}

// In one launch the second product's tiles fill what the first's last round
// leaves, and one way in and out is saved: 4096 tokens' gradients over 32768
// classes and 2048 channels take 1728 blocks of k a worker instead of 1920.
// Where both have few tiles of many blocks, all blocks are dealt out: 5377
// tokens' gradients of 64 channels and 1408 inner values 25 blocks a worker
// instead of 85.
mpg_status launch_fused_two(DeviceInfo* dev, const FusedLaunch& l0, const FusedLaunch& l1, FusedGemmParams& p, float* slots,
                            cudaStream_t stream) {
  Forms f;
  mpg_status s = forms_of(dev, FusedEpi::kPlain, 0, &f);
  if (s != MPG_OK) return s;
  const FusedLaunch* l[2] = {&l0, &l1};
  const FusedShape first = shape_of(l0, 256), second = shape_of(l1, 256);
  const bool swap = second.units / second.tiles > first.units / first.tiles;     // the longer k goes first
  if (swap) {
    std::swap(l[0], l[1]);
    std::swap(p.prod[0], p.prod[1]);
  }
  double apart = 0.0;
  for (const FusedLaunch* x : l) apart += std::min(deal_form(*x, f, 0, slots != nullptr).time, deal_form(*x, f, 1, slots != nullptr).time);
  double best = apart;
  int form = -1;
  int64_t late = 0, late_workers = 0, late_rounds = 0, workers = 0;
  bool dealt = false;
  for (int pair = 0; pair < 2; ++pair) {
    const int64_t tile = f.kernel[pair].tile, w = f.workers[pair];
    const FusedShape a = shape_of(*l[0], tile), b = shape_of(*l[1], tile);
    const int64_t ka = a.units / a.tiles, kb = b.units / b.tiles;
    const int64_t busy = a.tiles % w;                                             // workers with one tile more than the others
    const int64_t idle = busy ? w - busy : 0;
    const int64_t rounds = std::min(idle ? ka / kb : 0, idle ? (b.tiles + idle - 1) / idle : 0);
    const int64_t rest = std::max<int64_t>(0, b.tiles - rounds * idle);
    const double block = pair ? kPairBlock : kOneBlock, way_out = pair ? kPairEpi : kOneEpi;
    const double time = (pair ? kPairEdge : kOneEdge) + (double)((a.tiles + w - 1) / w) * std::max((double)ka * block, way_out) +
                        (double)((rest + w - 1) / w) * std::max((double)kb * block, way_out);
    if (time < best) {
      best = time;
      form = pair;
      dealt = false;
      late = busy;
      late_workers = idle;
      late_rounds = rounds;
    }
    const int64_t units = a.units + b.units, all = std::min(w, std::max(units / kMinUnits, (int64_t)1));
    const double operands = 128.0 * ((double)ka * (double)((l[0]->second_m ? 2 : 1) * l[0]->m + l[0]->n) +
                                     (double)kb * (double)((l[1]->second_m ? 2 : 1) * l[1]->m + l[1]->n));
    const double apart_block = operands < kL2Bytes ? block : std::max(block, 256.0 * (double)tile * (double)all / kApartBytes);
    const double parts = (double)std::min(2 * all, a.tiles + b.tiles + all) * (double)(tile * tile) * 4.0;
    const double even = (pair ? kPairEdge : kOneEdge) + kJoin + 2.0 * parts / kPartBytes +
                        std::max((double)((units + all - 1) / all) * apart_block, (double)((a.tiles + b.tiles) / all) * way_out);
    if (slots && kb >= kMinUnits && a.tiles + b.tiles <= 2 * w && even < best) {
      best = even;
      form = pair;
      dealt = true;
      workers = all;
    }
  }
  if (form < 0) {
    // apart: one after the other
    FusedProduct other = p.prod[1];
    if ((s = launch_fused(dev, *l[0], p, slots, stream)) != MPG_OK) return s;
    p.prod[0] = other;
    return launch_fused(dev, *l[1], p, slots, stream);
  }
  const FusedKernel& k = f.kernel[form];
  for (int i = 0; i < 2; ++i)
    if ((s = fill_product(p.prod[i], *l[i], k.tile, form)) != MPG_OK) return s;
  if (dealt) {
    p.whole_tiles = 0;
    return launch(dev, k, p, workers, workers, true, slots, stream);
  }
  p.whole_tiles = p.prod[0].num_tiles;
  p.late = (int32_t)late;
  p.late_workers = (int32_t)late_workers;
  p.late_rounds = (int32_t)late_rounds;
  const int64_t tiles = (int64_t)p.prod[0].num_tiles + p.prod[1].num_tiles;
  return launch(dev, k, p, std::min(f.workers[form], tiles), 0, false, slots, stream);
}

}  // namespace mpg
