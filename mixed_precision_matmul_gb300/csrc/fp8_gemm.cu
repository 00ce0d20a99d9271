// The block-scaled 8-bit product on single CTAs (sm_103a, cta_group::1): one
// 128 x BN tile of D per CTA, or per cluster of up to 8 CTAs that divide the
// tile's k-blocks among them; or, direct, 128 x 128 tiles one after another.
//
// Roles:
//   warp 0      TMA producer (one line of 128 k per row and stage)
//   warp 1      TMEM allocation; one elected lane issues the MMAs, one
//               accumulator buffer per k-block (four buffers in turn)
//   the last    (direct, a scale for each column) looks at the column scales of
//               the tiles to come (fp8_tc.cuh)
//   warps 2..   epilogue: read each k-block's accumulator, add it to the
//               running sums under its scales (fp8_tc.cuh), and at the end
//               put the sums into shared memory, where the tile is read back
//               in the order that C is stored in.  Direct: each warp stores
//               its own rows, while the tensor cores are on the next tile (up
//               to four blocks ahead).  With a cluster, each CTA
//               reads its share of the rows from all CTAs' shared memory and
//               adds the partial sums in rank order, so the result does not
//               depend on timing and needs no workspace.
//
// Few tokens (m <= 64): R, the 128-row operand, is the weights and the tokens
// are the columns (BN = 16, 32 or 64), so that the tensor core's rows are full
// and each weight byte is read once; the kernel is then bound by the weights'
// bytes, and the k range is divided so that most SMs have some in flight.
//
// On a GB300, from a graph: 1 x 8192 by 8192 x 8192 takes 15.0 us with weights
// from DRAM (4.5 TB/s), 12.4 with what the L2 cache keeps of them; 33 x 4160 by
// 4096 x 4160 takes 9.0 and 8.9 us, bound by the latency of a chain of blocks (a
// block's load, MMAs and addition) and by the way in and out of the kernel.
// Direct tiles take 335 ns a block of k, which is the operands' way from the L2
// cache (32 KB an SM, 15 TB/s in all; the tensor cores need 140 ns), 460 with a
// scale for each column: 1000 x 4112 by 1531 x 4112 takes 17.3 us, 4096^3 with a
// scale for each column 117 us in fp32.  Measured and not kept for the latter,
// beside 118: eight epilogue warps instead of sixteen (123), one tile a CTA
// (121), the next block's columns read during the additions (139).
#include <type_traits>

#include "fp8_tc.cuh"

namespace mpg {
namespace {

// kDirect: tile after tile on one CTA, sums from registers to C; else one tile,
// of which the CTAs of a cluster may have shares.
template <int BN_, bool kSwapped_, bool kColVec_, bool kDirect_>
struct Fp8Traits {
  static constexpr int BM = 128;
  static constexpr int BN = BN_;
  static constexpr bool kSwapped = kSwapped_;
  static constexpr bool kColVec = kColVec_;
  static constexpr bool kDirect = kDirect_;
  static_assert(!kDirect || !kSwapped, "rows of C");
  static constexpr int kStage = (BM + BN) * kFp8RowBytes;
  // few columns: two CTAs to an SM, so that one's start and end overlap the
  // other's loads, and as many stages as fit: the weights come from DRAM, and
  // with one CTA on most SMs the copies in flight bound the rate.  1 x 8192 by
  // 8192 x 8192, weights not in the L2 cache: 14.7 us; three CTAs of three
  // stages 17.0; one of ten stages 14.7, but 64 x 2048 x 8192 12.0 and 15.7,
  // where clusters of eight SMs of their own do not all find room at once.
  static constexpr int kCtasPerSm = BN >= 128 ? 1 : 2;
  static constexpr int kStages = BN >= 128 ? (kDirect ? 5 : 6) : BN >= 64 ? 4 : BN >= 32 ? 5 : 6;
  static constexpr int kAccBufs = 4;
  static constexpr int kAccStride = BN < 32 ? 32 : BN;
  static constexpr int kTmemCols = kAccBufs * kAccStride;
  static constexpr int kEpiWarps = kDirect ? 16 : BN >= 64 ? 8 : 4;
  static constexpr int kCols = BN / (kEpiWarps / 4);      // columns of one epilogue warp
  static constexpr bool kScans = kDirect && kColVec;     // a warp looks at later tiles' column scales
  static constexpr int kThreads = (2 + kEpiWarps + kScans) * 32;
  using Ring = ScaleRing<kCols, kSwapped || kDirect ? 4 : 8>;
  static constexpr int kRingBytes = kColVec ? kEpiWarps * Ring::kBytes : 0;
  // The staged tile's lines run along C's: columns of a row, or, swapped, the
  // rows of a column.  (132: rows written by 16 bytes a lane reach all banks.)
  static constexpr int kLines = kSwapped ? BN : BM;
  static constexpr int kPitch = kSwapped ? BM : BN + 4;   // floats
  static constexpr int kEpiBytes = kDirect ? kEpiWarps * 2048 : 0;   // rows on their way to C, tile after tile
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 1;
  static constexpr int kSmemBytes = 1024 + kStages * kStage + kRingBytes + kEpiBytes + kNumBars * 8 + 16 + (kScans ? Notes::kBytes : 0);
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 233472, "shared memory budget");
  static_assert(kLines * kPitch * 4 <= kStages * kStage, "the staged tile reuses the operand stages");
  static_assert(kCtasPerSm * kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM budget");
};

template <class T>
__global__ void __launch_bounds__(T::kThreads, T::kCtasPerSm) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same offset in every CTA of a cluster (the partial sums are read by address)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring_base = smem + T::kStages * T::kStage;
  uint8_t* epi_base = ring_base + T::kRingBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi_base + T::kEpiBytes);
  uint64_t* op_full = bars;
  uint64_t* op_empty = bars + T::kStages;
  uint64_t* acc_full = bars + 2 * T::kStages;
  uint64_t* acc_empty = acc_full + T::kAccBufs;
  uint64_t* done_bar = acc_empty + T::kAccBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Notes notes;
  notes.full = reinterpret_cast<uint64_t*>(tmem_slot + 2);
  notes.empty = notes.full + kNotes;
  notes.word = reinterpret_cast<uint32_t*>(notes.empty + kNotes);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();          // this CTA's share of the k range
  const int tile = (int)(blockIdx.x / (uint32_t)p.splits);
  const int step = T::kDirect ? (int)gridDim.x : p.num_tiles;
  auto row_of = [&](int t) { return t % p.num_r_blk * T::BM; };
  auto col_of = [&](int t) { return t / p.num_r_blk * T::BN; };
  const int row0 = row_of(tile), col0 = col_of(tile);
  const int kb0 = (int)rank * p.kb_per_split;
  const int nkb = max(0, min(p.num_k_blk, kb0 + p.kb_per_split) - kb0);

  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(&op_full[i], 1);
      mbar_init(&op_empty[i], 1);
    }
    for (int i = 0; i < T::kAccBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], T::kEpiWarps);
    }
    mbar_init(done_bar, 1);
    for (int i = 0; i < (T::kScans ? (int)kNotes : 0); ++i) {
      mbar_init(&notes.full[i], 1);
      mbar_init(&notes.empty[i], T::kEpiWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.map_r);
    tma_prefetch_map(&p.map_c);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  WaitCtl ctl;
  ctl.abort = abort_flag;
  ctl.status = p.status;
  ctl.limit_ns = p.wait_limit_ns;
  ctl.late_clock = true;
  const uint32_t op_smem = smem_addr(smem);
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t i = 0;
      for (int t = tile; t < p.num_tiles && ok; t += step) {
        const int r = row_of(t), c = col_of(t);
        for (int kb = 0; kb < nkb; ++kb, ++i) {
          const uint32_t st = i % T::kStages;
          if (!mbar_wait(&op_empty[st], ((i / T::kStages) & 1u) ^ 1u, ctl)) { ok = false; break; }
          mbar_arrive_expect_tx(&op_full[st], T::kStage);
          uint8_t* dst = smem + st * T::kStage;
          const int k0 = (kb0 + kb) * kFp8Block;
          tma_load_3d(dst, &p.map_r, &op_full[st], k0, r, 0);
          tma_load_3d(dst + T::BM * kFp8RowBytes, &p.map_c, &op_full[st], k0, c, 0);
        }
      }
      // the stages' last releases cover the copies still in flight
      for (uint32_t j = i < (uint32_t)T::kStages ? 0u : i - T::kStages; j < i; ++j)
        drain_wait(&op_empty[j % T::kStages], (j / T::kStages) & 1u, p.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc = make_idesc(0u, false, false, T::BM, T::BN) | p.fmt_bits;
    const uint64_t r_desc = fp8_desc(op_smem, 0), c_desc = fp8_desc(op_smem + T::BM * kFp8RowBytes, 0);
    const uint32_t d_base = __shfl_sync(0xffffffffu, tmem_base, 0);
    uint32_t i = 0, st = 0, st_ph = 0;
    for (int t = tile; t < p.num_tiles && ok; t += step) {
      for (int kb = 0; kb < nkb; ++kb, ++i) {
        const uint32_t ab = i % T::kAccBufs;
        if (!warp_wait(&op_full[st], st_ph, ctl)) { ok = false; break; }
        if (!warp_wait(&acc_empty[ab], ((i / T::kAccBufs) & 1u) ^ 1u, ctl)) { ok = false; break; }
        tc_fence_after_sync();
        const uint64_t at = (uint64_t)(st * (T::kStage / 16));
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_f8(d_base + ab * T::kAccStride, r_desc + at + 2 * ks, c_desc + at + 2 * ks, idesc, ks > 0 ? 1u : 0u);
          mma_commit(&acc_full[ab]);
          mma_commit(&op_empty[st]);
        }
        __syncwarp();
        if (++st == T::kStages) {
          st = 0;
          st_ph ^= 1u;
        }
      }
    }
    if (leader) {
      mma_commit(done_bar);
      drain_wait(done_bar, 0, p.wait_limit_ns);
    }
    __syncwarp();
  } else if (T::kScans && warp == 2 + T::kEpiWarps) {
    // ------------------------------------------------------------ column scales of the tiles to come
    uint32_t n = 0;
    for (int t = tile + step; t < p.num_tiles && ok; t += step, ++n)
      ok = notes.leave(n, scan_alone<T::BN>(p, lane, col_of(t), kb0, nkb), lane, ctl);
  } else {
    // ------------------------------------------------------------ running sums
    const int q = warp & 3;
    const int ew = warp - 2;
    const int wc0 = (ew / 4) * T::kCols;                  // this warp's first column in the tile
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + wc0;
    f32x2 acc[T::kCols / 2];
    auto release = [&](uint32_t ab) {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
    };
    // a whole tile's sums to C, while the tensor cores are on the next tile
    auto store = [&](int t) {
      if constexpr (T::kDirect) {
        const int row = row_of(t) + 32 * q, col = col_of(t) + wc0;
        if (row >= p.rows) return;
#pragma unroll
        for (int cc = 0; cc < T::kCols / 32; ++cc)
          if (col + cc * 32 < p.cols)
            store_rows32(p, smem_addr(epi_base) + ew * 2048, lane, acc + cc * 16, row, col + cc * 32);
      }
    };
    uint32_t i = 0;
    if constexpr (T::kColVec) {
      // scales by way of shared memory, a ring of blocks that only this warp uses
      typename T::Ring ring;
      auto begin = [&](int t) {
        ring.start(p, smem_addr(ring_base) + ew * T::Ring::kBytes, lane, row_of(t) + 32 * q, col_of(t) + wc0, kb0, nkb);
      };
      auto block = [&](int kb, auto form) {
        const uint32_t ab = i % T::kAccBufs;
        __syncwarp();                                    // every lane is done with the last block's slot
        ring.fetch(kb + T::Ring::kDepth - 1);
        cp_async_wait<T::Ring::kDepth - 1>();
        if (!warp_wait(&acc_full[ab], (i / T::kAccBufs) & 1u, ctl)) return false;
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t slot = ring.slot(kb);
        const float s = ld_shared_f32(slot + lane * 4);
        add_block<T::kCols, decltype(form)::value>(acc, tacc + ab * T::kAccStride, slot, s, [&]() { release(ab); });
        return true;
      };
      begin(tile);
      if constexpr (T::kDirect) {
        // Tiles of one form from tile t on; the first of the other form (or the
        // end) is left in t.  (Each form has a loop of its own: chosen inside
        // one loop over the tiles, 4096^3 takes 120 us instead of 117.)
        int t = tile;
        uint32_t n = 0;
        auto tiles = [&](auto form) {
          for (;;) {
#pragma unroll
            for (int j = 0; j < T::kCols / 2; ++j) acc[j] = 0;
#pragma unroll 1
            for (int kb = 0; kb < nkb; ++kb, ++i)
              if (!block(kb, form)) { ok = false; return false; }
            __syncwarp();
            const bool more = t + step < p.num_tiles;
            if (more) begin(t + step);                   // (its scales are on their way during the stores)
            store(t);
            t += step;
            bool plain = true;
            if (!more || !(ok = notes.read(n++, lane, ctl, &plain))) return false;
            if (plain != decltype(form)::value) return true;
          }
        };
        bool plain = scan_together<T::kEpiWarps * 32, T::BN>(p, ew * 32 + lane, col0, kb0, nkb);
        while (plain ? tiles(std::true_type()) : tiles(std::false_type())) plain = !plain;
      } else {
        auto blocks = [&](auto form) {
#pragma unroll 1
          for (int kb = 0; kb < nkb; ++kb, ++i)
            if (!block(kb, form)) return false;
          return true;
        };
        bool plain;
        if constexpr (T::kSwapped) plain = scan_alone<T::kCols>(p, lane, col0 + wc0, kb0, nkb);
        else plain = scan_together<T::kEpiWarps * 32, T::BN>(p, ew * 32 + lane, col0, kb0, nkb);
#pragma unroll
        for (int j = 0; j < T::kCols / 2; ++j) acc[j] = 0;
        ok = plain ? blocks(std::true_type()) : blocks(std::false_type());
      }
    } else {
      // A row a lane: its scale and that of all columns go from global memory
      // into registers, three blocks ahead.  Columns are read 32 at a time, the
      // next block's as soon as this one's are added.
      static_assert(T::kCols % 32 == 0, "whole reads");
      constexpr int kReads = T::kCols / 32;
      const float* row_src;
      const float* col_src;
      float rsc[4], csc[4];
      auto fetch_scales = [&](int j, int kb) {
        if (kb < nkb) {
          rsc[j] = ld_global(row_src);
          csc[j] = ld_global(col_src);
          row_src += p.sr_k;
          col_src += p.sc_k;
        }
      };
      auto begin = [&](int t) {
        row_src = p.sr + (int64_t)(min(row_of(t) + 32 * q + lane, p.rows - 1) >> p.sr_shift) * p.sr_row + kb0 * p.sr_k;
        col_src = p.sc + (int64_t)(min(col_of(t) + wc0, p.cols - 1) >> p.sc_shift) * p.sc_row + kb0 * p.sc_k;
#pragma unroll
        for (int j = 0; j < 4; ++j) rsc[j] = csc[j] = 0.0f;
#pragma unroll
        for (int j = 0; j < 3; ++j) fetch_scales(j, j);
      };
      float v[kReads][32];
      auto load = [&](uint32_t it) {
        if (!warp_wait(&acc_full[it % T::kAccBufs], (it / T::kAccBufs) & 1u, ctl)) return false;
        tc_fence_after_sync();
        return true;
      };
      begin(tile);
      for (int t = tile; t < p.num_tiles && ok; t += step) {
#pragma unroll
        for (int j = 0; j < T::kCols / 2; ++j) acc[j] = 0;
        ok = nkb > 0 && load(i);
        if (ok) {
#pragma unroll
          for (int c = 0; c < kReads; ++c) tmem_ld_32cols(tacc + (i % T::kAccBufs) * T::kAccStride + c * 32, v[c]);
        }
#pragma unroll 1
        for (int kb = 0; kb < nkb && ok; ++kb, ++i) {
          const bool more = kb + 1 < nkb;
          const uint32_t next = tacc + ((i + 1) % T::kAccBufs) * T::kAccStride;
          fetch_scales(3, kb + 3);
          const bool plain_here = __all_sync(0xffffffffu, plain_scale(rsc[0], csc[0])) != 0;
          tmem_ld_wait();
          release(i % T::kAccBufs);
          if (more && !load(i + 1)) { ok = false; break; }
          auto add = [&](auto plain) {
#pragma unroll
            for (int c = 0; c < kReads; ++c) {
              scale_add<32, false, decltype(plain)::value>(acc + c * 16, v[c], 0, 0, rsc[0], csc[0]);
              if (more) tmem_ld_32cols(next + c * 32, v[c]);
            }
          };
          if (plain_here) add(std::true_type());
          else add(std::false_type());
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            rsc[j] = rsc[j + 1];
            csc[j] = csc[j + 1];
          }
        }
        if (!T::kDirect || !ok) break;
        if (t + step < p.num_tiles) begin(t + step);
        store(t);
      }
    }
    cp_async_wait<0>();
    if (!T::kDirect && ok) {
      // every MMA of this CTA is complete: the operand stages are free
      const int r = 32 * q + lane;
#pragma unroll
      for (int j = 0; j < T::kCols; j += 4) {
        float x[4];
        unpack2(acc[j / 2], x[0], x[1]);
        unpack2(acc[j / 2 + 1], x[2], x[3]);
        if constexpr (T::kSwapped) {
#pragma unroll
          for (int i = 0; i < 4; ++i) st_shared_f32(op_smem + (uint32_t)((wc0 + j + i) * T::kPitch + r) * 4u, x[i]);
        } else {
          st_shared_v4(op_smem + (uint32_t)(r * T::kPitch + wc0 + j) * 4u, __float_as_uint(x[0]), __float_as_uint(x[1]),
                       __float_as_uint(x[2]), __float_as_uint(x[3]));
        }
      }
    }
  }

  // ---------------------------------------------------------------- C
  tc_fence_before_sync();
  if (p.splits > 1) cluster_sync_all();
  else __syncthreads();
  if (!T::kDirect && *abort_flag == 0) {
    // This CTA's share of the tile's rows, in vectors of four elements that
    // are neighbours in C and in the staged lines; of each, the ranges' partial
    // sums are loaded before the first is added (a load from another SM takes
    // about a microsecond).
    const int splits = p.splits;
    const int rows_per = ((T::BM + splits - 1) / splits + 3) & ~3;
    const int ra = (int)rank * rows_per;
    const int rows_here = min(min(T::BM, ra + rows_per), p.rows - row0) - ra;
    const int cols_here = min(T::BN, p.cols - col0);
    const int lines = T::kSwapped ? cols_here : rows_here;               // of C, in this share
    const int length = T::kSwapped ? rows_here : cols_here;
    const int first = T::kSwapped ? ra : 0;                              // offset in a staged line
    const int line0 = T::kSwapped ? 0 : ra;
    const int vecs = (length + 3) / 4;
    uint32_t peer[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) peer[s] = s < splits ? cluster_smem_addr(op_smem, (uint32_t)s) : 0u;
    const int64_t c0 = T::kSwapped ? (int64_t)col0 * p.ld_out + row0 + ra : (int64_t)(row0 + ra) * p.ld_out + col0;
    if (p.out_vec) {
      for (int u = threadIdx.x; length > 0 && u < lines * vecs; u += T::kThreads) {
        const int line = u / vecs, c = (u - line * vecs) * 4;
        const uint32_t off = (uint32_t)((line0 + line) * T::kPitch + first + c) * 4u;
        float4 x;
        if (splits == 1) {
          x = ld_shared_f4(op_smem + off);
        } else {
          float4 part[8];
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (s < splits) part[s] = ld_cluster_f4(peer[s] + off);
          x = part[0];
#pragma unroll
          for (int s = 1; s < 8; ++s)
            if (s < splits) {
              x.x += part[s].x;
              x.y += part[s].y;
              x.z += part[s].z;
              x.w += part[s].w;
            }
        }
        const int64_t idx = c0 + (int64_t)line * p.ld_out + c;
        x.x *= p.alpha;
        x.y *= p.alpha;
        x.z *= p.alpha;
        x.w *= p.alpha;
        if (c + 4 <= length) {
          if (p.beta != 0.0f) {
            const float4 z = out_load4(p.out, idx, p.out_dtype);
            x.x = fmaf(p.beta, z.x, x.x);
            x.y = fmaf(p.beta, z.y, x.y);
            x.z = fmaf(p.beta, z.z, x.z);
            x.w = fmaf(p.beta, z.w, x.w);
          }
          out_store4(p.out, idx, x, p.out_dtype);
        } else {
          const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < length)
              out_store(p.out, idx + j, p.beta != 0.0f ? fmaf(p.beta, out_load(p.out, idx + j, p.out_dtype), e[j]) : e[j],
                        p.out_dtype);
        }
      }
    } else {
      // lines of C off the vectors' alignment: neighbouring threads take
      // neighbouring elements, four of a line each
      for (int u = threadIdx.x; length > 0 && u < lines * vecs; u += T::kThreads) {
        const int line = u / vecs, v = u - line * vecs;
        const uint32_t row = (uint32_t)((line0 + line) * T::kPitch + first) * 4u;
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t off = row + (uint32_t)min(v + j * vecs, length - 1) * 4u;
          if (splits == 1) {
            x[j] = ld_shared_f32(op_smem + off);
          } else {
            float part[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
              if (s < splits) part[s] = ld_cluster_f32(peer[s] + off);
            x[j] = part[0];
#pragma unroll
            for (int s = 1; s < 8; ++s)
              if (s < splits) x[j] += part[s];
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = v + j * vecs;
          if (c >= length) break;
          const int64_t idx = c0 + (int64_t)line * p.ld_out + c;
          const float y = p.alpha * x[j];
          out_store(p.out, idx, p.beta != 0.0f ? fmaf(p.beta, out_load(p.out, idx, p.out_dtype), y) : y, p.out_dtype);
        }
      }
    }
  }
  // no CTA exits while another may still read its shared memory
  __syncwarp();
  if (p.splits > 1) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, T::kTmemCols);
  }
}

template <class T>
bool fill(Fp8Kernel* out) {
  out->fn = reinterpret_cast<const void*>(&fp8_gemm_kernel<T>);
  out->block = T::kThreads;
  out->smem_bytes = T::kSmemBytes;
  out->tile_rows = T::BM;
  out->tile_cols = T::BN;
  return true;
}

}  // namespace

bool fp8_lookup(int bn, bool swapped, bool col_vec, bool direct, Fp8Kernel* out) {
  if (swapped) {
    switch (bn) {
      case 16: return fill<Fp8Traits<16, true, true, false>>(out);
      case 32: return fill<Fp8Traits<32, true, true, false>>(out);
      case 64: return fill<Fp8Traits<64, true, true, false>>(out);
      default: return false;
    }
  }
  if (bn != 128) return false;
  if (direct) return col_vec ? fill<Fp8Traits<128, false, true, true>>(out) : fill<Fp8Traits<128, false, false, true>>(out);
  return col_vec ? fill<Fp8Traits<128, false, true, false>>(out) : fill<Fp8Traits<128, false, false, false>>(out);
}

}  // namespace mpg
