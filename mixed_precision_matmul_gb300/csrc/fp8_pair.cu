// The block-scaled 8-bit product on pairs of CTAs (sm_103a, cta_group::2): a
// persistent cluster of two CTAs computes 256 x 256 tiles of D.
//
// Each CTA holds 128 rows of the tile's R panel and 128 lines of its C panel
// for a block of 128 k.  Four M = 256, N = 256, K = 32 instructions leave the
// block's product in one of two TMEM buffers (256 columns each), and eight
// epilogue warps in each CTA (32 rows x 128 columns a warp, 128 running sums a
// thread, in registers for the whole k range) add it under its scales while
// the tensor cores fill the other buffer.  Where each column has a scale of its
// own, two warps fetch those, up to eight blocks ahead; rows' scales (and those
// of 128 columns) go straight to registers, three blocks ahead.
//
// A block's products take the tensor cores 512 cycles (about 620 here: the
// operands' way in and out of shared memory).  The epilogue has to keep up:
// 64 packed multiply-adds a warp (128 and 32 loads with a scale for each
// column), four reads of TMEM and the hand-overs, two warps to a scheduler.
// It is bound by latencies, so everything that is not one of these is on other
// warps, and reads overlap additions.
//
// On a GB300, from a graph: 8192^3 with a scale for each 128 columns takes 437
// us (2516 TFLOP/s; the MMAs alone, never read, 299 us), about 870 cycles a
// block: the way round MMA, commit, read and release through two buffers, all
// that 512 columns of TMEM hold.  With a scale for each column and fp32 C 4096^3
// takes 125 us (single CTAs: 117), 8192^3 770 (829).  Measured and not kept, at
// 8192^3: half-width accumulators in four buffers (642 us: the tensor cores read
// R twice), 256 x 128 tiles (644 us); at 4096^3, the 16-lane read of TMEM that
// lets a thread keep its columns' scales in registers (4 us slower: that read
// takes three times as long).
#include <type_traits>

#include "fp8_tc.cuh"

namespace mpg {
namespace {

template <bool kColVec_>
struct Fp8PairTraits {
  static constexpr bool kColVec = kColVec_;
  static constexpr int BM = 128;                    // rows of R and lines of C held by one CTA
  static constexpr int kTile = 256;
  static constexpr int kRTile = BM * kFp8RowBytes;
  static constexpr int kStage = 2 * kRTile;
  static constexpr int kStages = 6;
  static constexpr int kAccBufs = 2;
  static constexpr int kTmemCols = kAccBufs * kTile;
  static constexpr int kEpiWarps = 8;
  static constexpr int kScaleWarps = kColVec ? 2 : 0;      // each fetches the scales of half the columns
  static constexpr int kCols = kTile / (kEpiWarps / 4);
  static constexpr int kThreads = (4 + kEpiWarps) * 32;
  // Registers: the block is launched with 168 a thread; the first warpgroup
  // (producer, MMA, two for column scales) gives up all but 40, the two of the
  // epilogue take 232: 128 running sums, 64 columns on their way.
  static constexpr int kLaunchRegs = 168, kIdleRegs = 40, kEpiRegs = 232;
  static_assert(128 * kIdleRegs + kEpiWarps * 32 * kEpiRegs <= kThreads * kLaunchRegs, "register split");
  // Scales of the tile's columns, by blocks of k (two warps of their own fetch them).
  static constexpr int kScaleSlots = kColVec ? 8 : 0;
  static constexpr int kScaleSlot = kTile;
  static constexpr int kScaleBytes = (kScaleSlots * kScaleSlot * 4 + 15) / 16 * 16;
  static constexpr int kEpiBytes = kEpiWarps * 2048;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 2 * kScaleSlots + 1;
  static constexpr int kSmemBytes = 1024 + kStages * kStage + kEpiBytes + kScaleBytes + kNumBars * 8 + 16 + kScaleWarps * Notes::kBytes;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct PairTile {
  int rb, cb;
};
__device__ __forceinline__ PairTile pair_tile(const Fp8GemmParams& p, int t) {
  // groups of tile rows, walked column by column, every other group backwards
  const int per = p.group * p.num_c_blk;
  const int g = t / per;
  const int first = g * p.group;
  const int gm = min(p.group, p.num_r_blk - first);
  const int within = t - g * per;
  PairTile c;
  c.rb = first + within % gm;
  c.cb = within / gm;
  if (g & 1) c.cb = p.num_c_blk - 1 - c.cb;
  return c;
}

template <class T>
__global__ void __launch_bounds__(T::kThreads, 1) fp8_pair_kernel(const __grid_constant__ Fp8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi_base = smem + T::kStages * T::kStage;
  uint8_t* scale_base = epi_base + T::kEpiBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(scale_base + T::kScaleBytes);
  uint64_t* op_full = bars;                         // rank 0: both CTAs' halves of a stage landed
  uint64_t* op_empty = bars + T::kStages;           // each CTA: the pair's MMAs consumed the stage
  uint64_t* acc_full = bars + 2 * T::kStages;       // each CTA: a block's product is complete
  uint64_t* acc_empty = acc_full + T::kAccBufs;     // rank 0: both CTAs' epilogues read it
  uint64_t* scale_full = acc_empty + T::kAccBufs;   // a block's scales are in their slot
  uint64_t* scale_empty = scale_full + T::kScaleSlots;
  uint64_t* done_bar = scale_empty + T::kScaleSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // each half's notes on the tiles' column scales
  auto notes_of = [&](int h) {
    Notes x;
    x.full = reinterpret_cast<uint64_t*>(tmem_slot + 2) + h * 2 * kNotes;
    x.empty = x.full + kNotes;
    x.word = reinterpret_cast<uint32_t*>(reinterpret_cast<uint64_t*>(tmem_slot + 2) + T::kScaleWarps * 2 * kNotes) + h * kNotes;
    return x;
  };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int worker = (int)cluster_id_x(), workers = (int)num_clusters_x();
  const int nkb = p.num_k_blk;

  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(&op_full[i], 1);
      mbar_init(&op_empty[i], 1);
    }
    for (int i = 0; i < T::kAccBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * T::kEpiWarps);
    }
    for (int i = 0; i < T::kScaleSlots; ++i) {
      mbar_init(&scale_full[i], 64);                // the copies of each lane of the two scale warps
      mbar_init(&scale_empty[i], T::kEpiWarps);
    }
    mbar_init(done_bar, 1);
    for (int i = 0; i < T::kScaleWarps * (int)kNotes; ++i) {
      mbar_init(&notes_of(i / kNotes).full[i % kNotes], 1);
      mbar_init(&notes_of(i / kNotes).empty[i % kNotes], T::kEpiWarps / 2);
    }
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.map_r);
    tma_prefetch_map(&p.map_c);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, T::kTmemCols);
    tmem_relinquish_pair();
    tc_fence_before_sync();
  }
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  WaitCtl ctl;
  ctl.abort = abort_flag;
  ctl.peer_abort = cluster_generic_ptr(const_cast<int*>(abort_flag), rank ^ 1u);
  ctl.status = p.status;
  ctl.limit_ns = p.wait_limit_ns;
  ctl.late_clock = true;
  const uint32_t op_smem = smem_addr(smem);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(T::kIdleRegs));
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full0 = cluster_smem_addr(smem_addr(op_full), 0);
      uint32_t it = 0;
      bool ok = true;
      for (int t = worker; t < p.num_tiles && ok; t += workers) {
        const PairTile tc = pair_tile(p, t);
        const int rrow = tc.rb * T::kTile + (int)rank * T::BM;
        const int crow = tc.cb * T::kTile + (int)rank * T::BM;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t st = it % T::kStages;
          if (!mbar_wait(&op_empty[st], ((it / T::kStages) & 1u) ^ 1u, ctl)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&op_full[st], 2 * T::kStage);
          uint8_t* dst = smem + st * T::kStage;
          tma_load_3d_pair(dst, &p.map_r, full0 + st * 8u, kb * kFp8Block, rrow, 0);
          tma_load_3d_pair(dst + T::kRTile, &p.map_c, full0 + st * 8u, kb * kFp8Block, crow, 0);
        }
      }
      // a stage is released after its copies landed and were read
      const uint32_t n_drain = it < (uint32_t)T::kStages ? it : (uint32_t)T::kStages;
      for (uint32_t i = it - n_drain; i < it; ++i)
        drain_wait(&op_empty[i % T::kStages], (i / T::kStages) & 1u, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (rank 0)
    if (rank == 0) {
      const bool leader = elect_one();
      const uint32_t idesc = make_idesc(0u, false, false, T::kTile, T::kTile) | p.fmt_bits;
      // the start address sits in the descriptor's low bits, in units of 16 bytes
      const uint64_t r_desc = fp8_desc(op_smem, 0), c_desc = fp8_desc(op_smem + T::kRTile, 0);
      const uint32_t d_base = __shfl_sync(0xffffffffu, tmem_base, 0);
      uint32_t it = 0, st = 0, st_ph = 0;
      bool ok = true;
      for (int t = worker; t < p.num_tiles && ok; t += workers) {
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t ab = it % T::kAccBufs;
          if (!warp_wait(&op_full[st], st_ph, ctl)) { ok = false; break; }
          if (!warp_wait_relaxed(&acc_empty[ab], ((it / T::kAccBufs) & 1u) ^ 1u, ctl)) { ok = false; break; }
          tc_fence_after_sync();
          const uint64_t at = (uint64_t)(st * (T::kStage / 16));
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f8_pair(d_base + ab * T::kTile, r_desc + at + 2 * ks, c_desc + at + 2 * ks, idesc, ks > 0 ? 1u : 0u);
            mma_commit_multicast(&acc_full[ab], 0x3);
            mma_commit_multicast(&op_empty[st], 0x3);
          }
          __syncwarp();
          if (++st == T::kStages) {
            st = 0;
            st_ph ^= 1u;
          }
        }
      }
      if (leader) {
        mma_commit_multicast(done_bar, 0x1);
        drain_wait(done_bar, 0, p.wait_limit_ns);
      }
      __syncwarp();
    }
  } else if (T::kColVec) {
    // ------------------------------------------------------------ column scales
    uint32_t slot = 0, ph = 0, n = 0;
    bool ok = true;
    const Notes notes = notes_of(warp - 2);
    ColumnScan scan;                                   // of the next tile
    for (int t = worker; t < p.num_tiles && ok; t += workers, ++n) {
      ColumnLines lines;
      lines.start(p, pair_tile(p, t).cb * T::kTile + (warp - 2) * T::kCols, lane);
      const bool more = t + workers < p.num_tiles;
      if (more) scan.start(p, pair_tile(p, t + workers).cb * T::kTile + (warp - 2) * T::kCols, lane);
      for (int kb = 0; kb < nkb; ++kb) {
        if (!warp_wait(&scale_empty[slot], ph ^ 1u, ctl)) { ok = false; break; }
        const uint32_t dst = smem_addr(scale_base) + (slot * T::kScaleSlot + (warp - 2) * T::kCols + lane) * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < lines.count) cp_async4(dst + i * 128, lines.column(p, i));
        lines.next(p);
        cp_async_arrive(&scale_full[slot]);
        if (more) scan.block(p);
        if (++slot == T::kScaleSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
      if (ok && more) ok = notes.leave(n, scan.result(), lane, ctl);
    }
    cp_async_wait_all();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(T::kEpiRegs));
    // ------------------------------------------------------------ running sums
    const int q = warp & 3;
    const int ew = warp - 4;
    const uint32_t half = (uint32_t)(ew / 4);
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + half * T::kCols;
    const uint32_t stg = smem_addr(epi_base) + ew * 2048;
    const uint32_t acc_empty0 = cluster_smem_addr(smem_addr(acc_empty), 0);
    // One block of k's hand-over: the buffer goes back to rank 0, and the next
    // block's product is waited for (`ready`: its barrier, asked early, said
    // that it is complete).
    auto hand_over = [&](uint32_t it, bool more, bool ready) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + (it % T::kAccBufs) * 8u);
      if (more && !__all_sync(0xffffffffu, ready) &&
          !warp_wait(&acc_full[(it + 1) % T::kAccBufs], ((it + 1) / T::kAccBufs) & 1u, ctl))
        return false;
      tc_fence_after_sync();
      return true;
    };
    uint32_t it = 0, slot = 0, slot_ph = 0, n = 0;
    bool ok = true;
    bool plain_tile = true;                           // the columns' scales, where each has its own
    if constexpr (T::kColVec)
      plain_tile = scan_together<T::kEpiWarps * 32, T::kTile>(p, ew * 32 + lane, pair_tile(p, worker).cb * T::kTile, 0, nkb);
    for (int t = worker; t < p.num_tiles && ok; t += workers, ++n) {
      if (T::kColVec && n > 0 && !notes_of((int)half).read(n - 1, lane, ctl, &plain_tile)) break;
      f32x2 acc[T::kCols / 2];
#pragma unroll
      for (int j = 0; j < T::kCols / 2; ++j) acc[j] = 0;
      if (!warp_wait(&acc_full[it % T::kAccBufs], (it / T::kAccBufs) & 1u, ctl)) { ok = false; break; }
      tc_fence_after_sync();
      // A row a lane.  The row's scale (and that of this half's columns, where
      // they share one) goes from global memory straight into registers, three
      // blocks ahead: shared memory is busy with operands, and a load from it
      // takes longer than a block's additions.
      const PairTile tc0 = pair_tile(p, t);
      const int row = tc0.rb * T::kTile + (int)rank * T::BM + 32 * q + lane;
      const int col = tc0.cb * T::kTile + (int)half * T::kCols;
      const float* row_src = p.sr + (int64_t)(min(row, p.rows - 1) >> p.sr_shift) * p.sr_row;
      const float* col_src = p.sc + (int64_t)(min(col, p.cols - 1) >> p.sc_shift) * p.sc_row;
      float rsc[4], csc[4];
      auto fetch_scales = [&](int i, int kb) {
        if (kb < nkb) {
          rsc[i] = ld_global(row_src);
          row_src += p.sr_k;
          if (!T::kColVec) {
            csc[i] = ld_global(col_src);
            col_src += p.sc_k;
          }
        }
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rsc[i] = 0.0f;
        csc[i] = 1.0f;
        if (i < 3) fetch_scales(i, i);
      }
      // Columns are read 32 at a time, two reads on their way, across the
      // blocks of k too.
      constexpr int kN = T::kCols / 32;
      static_assert(kN == 4, "two pairs of reads a block");
      const uint32_t scales = smem_addr(scale_base) + half * (T::kCols * 4);
      float v[2][32];
      tmem_ld_32cols(tacc + (it & 1u) * T::kTile, v[0]);
      tmem_ld_32cols(tacc + (it & 1u) * T::kTile + 32, v[1]);
      bool known = false;
      bool plain_next = true;                         // one scale for all columns: the next block's form
      auto begin_block = [&](int kb) {
        fetch_scales(3, kb + 3);
        return !T::kColVec || __all_sync(0xffffffffu, known) || warp_wait(&scale_full[slot], slot_ph, ctl);
      };
      auto add = [&](bool more, auto plain) {
        constexpr bool kPlain = decltype(plain)::value;
        const uint32_t here = tacc + (it & 1u) * T::kTile, next = tacc + ((it + 1) & 1u) * T::kTile;
        const uint32_t sl = scales + slot * (T::kScaleSlot * 4) - 128;
        tmem_ld_wait();
        scale_add<32, T::kColVec, kPlain>(acc, v[0], sl, 0, rsc[0], csc[0]);
        tmem_ld_32cols(here + 64, v[0]);
        scale_add<32, T::kColVec, kPlain>(acc + 16, v[1], sl, 32, rsc[0], csc[0]);
        tmem_ld_32cols(here + 96, v[1]);
        // barriers take a while to answer: asked early
        const bool ready = more && mbar_test(&acc_full[(it + 1) & 1u], ((it + 1) >> 1) & 1u);
        if constexpr (!T::kColVec) plain_next = __all_sync(0xffffffffu, plain_scale(rsc[1], csc[1])) != 0;
        tmem_ld_wait();
        if (!hand_over(it, more, ready)) return false;
        scale_add<32, T::kColVec, kPlain>(acc + 32, v[0], sl, 64, rsc[0], csc[0]);
        if (more) tmem_ld_32cols(next, v[0]);
        if constexpr (T::kColVec) {
          const uint32_t ns = slot + 1 == T::kScaleSlots ? 0 : slot + 1;
          known = more && mbar_test(&scale_full[ns], ns == 0 ? slot_ph ^ 1u : slot_ph);
        }
        scale_add<32, T::kColVec, kPlain>(acc + 48, v[1], sl, 96, rsc[0], csc[0]);
        if (more) tmem_ld_32cols(next + 32, v[1]);
        return true;
      };
      auto end_block = [&]() {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          rsc[i] = rsc[i + 1];
          csc[i] = csc[i + 1];
        }
        if constexpr (T::kColVec) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&scale_empty[slot]);
          if (++slot == T::kScaleSlots) {
            slot = 0;
            slot_ph ^= 1u;
          }
        }
      };
      if constexpr (T::kColVec) {
        auto blocks = [&](auto plain) {
#pragma unroll 1
          for (int kb = 0; kb < nkb; ++kb) {
            const bool more = kb + 1 < nkb;
            if (!begin_block(kb)) return false;
            if (!add(more, plain)) return false;
            end_block();
            ++it;
          }
          return true;
        };
        ok = plain_tile ? blocks(std::true_type()) : blocks(std::false_type());
      } else {
        bool plain_block = __all_sync(0xffffffffu, plain_scale(rsc[0], csc[0])) != 0;
#pragma unroll 1
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          begin_block(kb);
          ok = plain_block ? add(kb + 1 < nkb, std::true_type()) : add(kb + 1 < nkb, std::false_type());
          if (!ok) break;
          plain_block = plain_next;
          end_block();
        }
      }
      if (!ok) break;
      // ---------------------------------------------------------- C
      const PairTile tc = pair_tile(p, t);
      const int row_base = tc.rb * T::kTile + (int)rank * T::BM + 32 * q;
      const int col_first = tc.cb * T::kTile + (int)half * T::kCols;
      if (row_base >= p.rows) continue;
#pragma unroll
      for (int cc = 0; cc < T::kCols / 32; ++cc)
        if (col_first + cc * 32 < p.cols)
          store_rows32(p, stg, lane, acc + cc * 16, row_base, col_first + cc * 32);
    }
  }

  // neither CTA leaves while the other may address its shared memory
  __syncwarp();
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, T::kTmemCols);
  }
}

template <class T>
bool fill(Fp8Kernel* out) {
  out->fn = reinterpret_cast<const void*>(&fp8_pair_kernel<T>);
  out->block = T::kThreads;
  out->smem_bytes = T::kSmemBytes;
  out->tile_rows = T::kTile;
  out->tile_cols = T::kTile;
  return true;
}

}  // namespace

bool fp8_lookup_pair(bool col_vec, Fp8Kernel* out) {
  return col_vec ? fill<Fp8PairTraits<true>>(out) : fill<Fp8PairTraits<false>>(out);
}

}  // namespace mpg
