// 16-bit products whose epilogues do the work around them (sm_103a).
//
// One persistent kernel, on pairs of CTAs (256 x 256 accumulators, M = 256
// instructions of cta_group::2) or on single CTAs (128 x 128), for five
// epilogues:
//
//   kGated      Y = act(gate) * up, gate = X Wg^T, up = X Wu^T; for the backward
//               pass act(gate) and up act'(gate) too.  The B operand of a tile is half of
//               lines of Wg and half of the same lines of Wu, so gate and up
//               are two halves of one accumulator, and a thread of the
//               epilogue holds both of an element.  On a pair the instruction
//               splits B between the CTAs: rank 0 holds Wg's lines, rank 1 Wu's.
//   kGatedGrad  the same accumulators; dgate = dY up act'(gate), dup = dY act(gate).
//   kStats      logits X W^T; a thread holds a row's part of the tile and keeps
//               the maximum and the sum of exponentials in one pass, and the
//               target's logit.  Logits are in units of ln 2, so that the exponential is
//               one instruction.
//   kProb       the same logits; (e^(l - lse) - [target]) dloss, rounded to 16 bits,
//               for a piece of the vocabulary.
//   kPlain      the gradients' products.  Both operands may be MN-major, k may
//               consist of two parts with maps of their own (dgate Wg + dup Wu:
//               one sum in fp32), and so may the rows (dgate^T X and dup^T X:
//               one launch).
//
// Roles (320 threads): warp 0 loads by TMA, warp 1 (of rank 0) issues the MMAs,
// warps 2-9 are the epilogue: 32 rows and half of the tile's columns each.
// Accumulators are double-buffered in TMEM, so the epilogue runs beside the
// next tile's products.
//
// Tiles go round by round to the workers.  What does not fill a round may be split:
// its blocks of k are dealt out evenly, in runs of a few at least, and a worker
// whose run holds only a part of a tile's k leaves its sums in a slot (fused_deal.h).  A
// second launch adds the slots of a tile in the order of k and does the epilogue's
// work: the result does not depend on timing.  Or (kPlain) a second product's
// tiles, shorter ones, fill the first's last round: the gradients of an input and
// of a weight are two products from the same D, and in one launch no worker waits
// for the other's end.
//
// What bounds it: the tensor cores, and how tiles fill 76 pairs.  A pair takes
// about 0.33 us for a block of 64 k (512 cycles of MMAs); on a GB300 the gated
// product of 8192 x 4096 x 11008 takes 0.82 ms (1.80 PFLOP/s; a library's plain
// product reaches 1.96), logits of 4096 tokens, 32768 classes and 2048 channels
// 0.31 ms with their statistics (1.78) and 0.31 with their gradient, and both
// products of that gradient 0.59 (1.86).  Back to back the card's power limit
// lowers all of them by about a tenth.  Epilogues are hidden behind products of 512
// k and more; with one block of k a tile's way out (1.9 us for 128 x 128 on one CTA)
// is all.
//
// Waits are bounded, and a timeout raises the abort flag of both CTAs: every
// role drains what it has in flight before TMEM is released.
#pragma once

#include <algorithm>
#include <climits>

#include "cluster.cuh"
#include "fused.cuh"
#include "fused_deal.h"
#include "outio.cuh"
#include "staging.cuh"
#include "tc_gemm.cuh"

namespace mpg {
namespace {

template <FusedEpi E, bool kPair_, int kAct_ = 0>
struct FusedTraits {
  static constexpr FusedEpi kEpi = E;
  static constexpr bool kPair = kPair_;
  static constexpr int kAct = kAct_;
  static constexpr bool kTwo = E == FusedEpi::kGated || E == FusedEpi::kGatedGrad;   // gate and up
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int kTile = 128 * kCtas;         // rows, and columns of the accumulators
  static constexpr int kTileN = kTwo ? kTile / 2 : kTile;
  static constexpr int BM = 128;                    // rows of A held by one CTA
  static constexpr int BK = 64;
  static constexpr int kRowBytes = 128;
  static constexpr uint32_t kSwizzle = kSwizzle128B;
  static constexpr int kInstrK = 16;
  static constexpr int kKSteps = BK / kInstrK;
  static constexpr int kHalf = 64 * kRowBytes;      // one 64 x 64 box
  static constexpr int kATile = 2 * kHalf;
  static constexpr int kStage = 2 * kATile;
  static constexpr int kStages = 6;
  // Blocks of k that are summed by the tensor cores at a time: their sums cut off
  // what fp32 does not hold, always towards zero, and the loss is an fp32 number
  // (2e-6 off at k = 4096 in one sum, 5e-7 in sums of 1024 added by the epilogue).
  static constexpr int kChunk = E == FusedEpi::kStats ? 16 : INT_MAX;
  static constexpr int kAccBufs = 2;
  static constexpr int kTmemCols = kAccBufs * kTile;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;
  static constexpr int kEpiBytes = kEpiWarps * 4096;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 1;
  static constexpr int kSmemBytes = 1024 + kStages * kStage + kEpiBytes + kNumBars * 8 + 16;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_shared_h(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_h(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
// 32 rows of 64 bytes: chunk c (16 bytes) of row r at slot c ^ ((r / 2) & 3),
// which spreads writes (a row a lane) and reads (four lanes a row) over all banks.
__device__ __forceinline__ uint32_t half_chunk(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

// 32 x 32 block of 16-bit values, a row a lane, to rows row0.. and columns col0..
// (The way from shared memory to the matrix is a function of its own: inlined at
// every store the code outgrows the instruction caches, and a kernel of few tiles
// waits for it: 1531 x 1001 x 2741 in two rounds of tiles 22 us, 9 of them MMAs.)
struct Block16 {
  void* base;
  int64_t ld;
  int row0, rows, col0, cols;
  bool vec;
};
__device__ __noinline__ void flush_block16(uint32_t stg, const Block16 b) {
  const int lane = threadIdx.x & 31;
  uint16_t* out = static_cast<uint16_t*>(b.base);
  if (b.vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2), c = lane & 3;
      const int left = b.row0 + r < b.rows ? b.cols - b.col0 - c * 8 : 0;
      uint16_t* to = out + (int64_t)(b.row0 + r) * b.ld + b.col0 + c * 8;
      const uint4 x = ld_shared_v4(stg + half_chunk(r, c));
      if (left >= 8) {
        *reinterpret_cast<uint4*>(to) = x;
      } else if (left > 0) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < left) to[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  } else {
    // by elements, sixteen rows at a time
    uint16_t* to = out + (int64_t)b.row0 * b.ld + b.col0 + lane;
    const int rows = b.col0 + lane < b.cols ? b.rows - b.row0 : 0;
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 16) {
      uint16_t x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = ld_shared_h(stg + half_chunk(r0 + r, lane >> 3) + (lane & 7) * 2);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (r0 + r < rows) *to = x[r];
        to += b.ld;
      }
    }
  }
  __syncwarp();
}
__device__ __forceinline__ void store_block16(uint32_t stg, int lane, const uint32_t (&w)[16], const Block16& b) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    st_shared_v4(stg + half_chunk(lane, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
  flush_block16(stg, b);
}
// The same block read: row row0 + lane, 32 columns (0 beyond the matrix).
__device__ __noinline__ void fill_block16(uint32_t stg, const Block16 b) {
  const int lane = threadIdx.x & 31;
  const uint16_t* src = static_cast<const uint16_t*>(b.base) + (int64_t)b.row0 * b.ld + b.col0 + lane;
  const int rows = b.col0 + lane < b.cols ? b.rows - b.row0 : 0;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 16) {
    uint16_t x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      x[r] = r0 + r < rows ? *src : (uint16_t)0;
      src += b.ld;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) st_shared_h(stg + half_chunk(r0 + r, lane >> 3) + (lane & 7) * 2, x[r]);
  }
  __syncwarp();
}
__device__ __forceinline__ void load_block16(uint32_t stg, int lane, uint32_t (&w)[16], const Block16& b) {
  if (!b.vec || (b.col0 + 32 > b.cols && b.cols % 8 != 0)) {
    fill_block16(stg, b);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 x = ld_shared_v4(stg + half_chunk(lane, c));
      w[4 * c] = x.x;
      w[4 * c + 1] = x.y;
      w[4 * c + 2] = x.z;
      w[4 * c + 3] = x.w;
    }
    __syncwarp();
    return;
  }
  const bool in = b.row0 + lane < b.rows;
  const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(b.base) + (int64_t)(in ? b.row0 + lane : b.row0) * b.ld + b.col0);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 x = in && b.col0 + 8 * c < b.cols ? ld_global(at + c) : make_uint4(0, 0, 0, 0);
    w[4 * c] = x.x;
    w[4 * c + 1] = x.y;
    w[4 * c + 2] = x.z;
    w[4 * c + 3] = x.w;
  }
}

// The class of a token (-1: ignored, -2: none), and the weight of its gradient: an
// ignored token has none, whatever its dloss; one of no class gives NaN.
__device__ __forceinline__ int64_t row_target(const FusedGemmParams& p, int row) {
  return target_of(p.target, p.target_bytes, p.target_stride, p.ignore_index, p.vocab, row);
}
__device__ __forceinline__ float row_weight(const FusedGemmParams& p, int row, int64_t target, const Scale& sc) {
  if (target < 0) return target == -1 ? 0.0f : NAN;
  return sc.mul * (ld_global(p.dloss + (int64_t)row * p.dloss_stride) / sc.div);
}

template <class T>
__global__ void __launch_bounds__(T::kThreads, 1) fused_gemm_kernel(const __grid_constant__ FusedGemmParams p) {
  if constexpr (T::kEpi == FusedEpi::kGatedGrad) {
    if (p.again) {
      // (every thread of both CTAs finds the same)
      griddep_launch_dependents();
      griddep_wait();
      if (!GradTop::needed(p, blockIdx.x == 0 && threadIdx.x < 32)) return;
    }
  }
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi_base = smem + T::kStages * T::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi_base + T::kEpiBytes);
  uint64_t* op_full = bars;                         // rank 0: a stage's copies landed in every CTA
  uint64_t* op_empty = bars + T::kStages;           // each CTA: the MMAs consumed the stage
  uint64_t* acc_full = bars + 2 * T::kStages;       // each CTA: an accumulator is complete
  uint64_t* acc_empty = acc_full + T::kAccBufs;     // rank 0: every epilogue warp has read it
  uint64_t* done_bar = acc_empty + T::kAccBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = T::kPair ? cluster_ctarank() : 0u;
  const int worker = T::kPair ? (int)cluster_id_x() : (int)blockIdx.x;
  const int workers = T::kPair ? (int)num_clusters_x() : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(&op_full[i], 1);
      mbar_init(&op_empty[i], 1);
    }
    for (int i = 0; i < T::kAccBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], T::kCtas * T::kEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.prod[0].map_a[0]);
    tma_prefetch_map(&p.prod[0].map_b[0]);
  }
  if (warp == 1) {
    if constexpr (T::kPair) {
      tmem_alloc_pair(tmem_slot, T::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, T::kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before_sync();
  }
  if constexpr (T::kPair) cluster_sync_all();
  else __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  WaitCtl ctl;
  ctl.abort = abort_flag;
  if constexpr (T::kPair) ctl.peer_abort = cluster_generic_ptr(const_cast<int*>(abort_flag), rank ^ 1u);
  ctl.status = p.status;
  ctl.limit_ns = p.wait_limit_ns;
  const uint32_t op_smem = smem_addr(smem);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full0 = T::kPair ? cluster_smem_addr(smem_addr(op_full), 0) : smem_addr(op_full);
      uint32_t it = 0;
      bool ok = true;
      FusedItems items(p, worker, workers);
      FusedItem x;
      while (ok && items.template next<T::kEpi == FusedEpi::kPlain>(p, x)) {
        const FusedProduct& pr = p.prod[x.which];
        const bool second = x.mb >= pr.mb_second;
        const int arow = (second ? x.mb - pr.mb_second : x.mb) * T::kTile + (int)rank * T::BM;
        for (int kb = x.kb0; kb < x.kb1; ++kb, ++it) {
          const uint32_t st = it % T::kStages;
          if (!mbar_wait(&op_empty[st], ((it / T::kStages) & 1u) ^ 1u, ctl)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&op_full[st], T::kCtas * T::kStage);
          uint8_t* dst = smem + st * T::kStage;
          const bool late = kb >= pr.kb_second;
          const int k0 = (late ? kb - pr.kb_second : kb) * T::BK;
          auto box = [&](const CUtensorMap* map, uint8_t* to, bool mn, int row) {
            const int c0 = mn ? row : k0, c1 = mn ? k0 : row;
            if constexpr (T::kPair) tma_load_3d_pair(to, map, full0 + st * 8u, c0, c1, 0);
            else tma_load_3d(to, map, &op_full[st], c0, c1, 0);
          };
          const CUtensorMap* ma = &pr.map_a[second || late ? 1 : 0];
#pragma unroll
          for (int h = 0; h < 2; ++h) box(ma, dst + h * T::kHalf, pr.a_mn_major != 0, arow + h * 64);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint8_t* to = dst + T::kATile + h * T::kHalf;
            if constexpr (T::kTwo) {
              // a pair: this CTA's 128 lines of one weight; one CTA: 64 of each
              const int which = T::kPair ? (int)rank : h;
              box(&pr.map_b[which], to, false, x.nb * T::kTileN + (T::kPair ? h * 64 : 0));
            } else {
              box(&pr.map_b[late ? 1 : 0], to, pr.b_mn_major != 0, x.nb * T::kTile + (int)rank * 128 + h * 64);
            }
          }
        }
      }
      // a stage is released after its copies landed and were read
      const uint32_t n_drain = it < (uint32_t)T::kStages ? it : (uint32_t)T::kStages;
      for (uint32_t i = it - n_drain; i < it; ++i)
        drain_wait(&op_empty[i % T::kStages], (i / T::kStages) & 1u, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const bool leader = elect_one();
      const uint32_t d_base = __shfl_sync(0xffffffffu, tmem_base, 0);
      auto commit = [&](uint64_t* bar, uint16_t mask) {
        if constexpr (T::kPair) mma_commit_multicast(bar, mask);
        else mma_commit(bar);
      };
      uint32_t g = 0, st = 0, st_ph = 0;
      bool ok = true;
      FusedItems items(p, worker, workers);
      FusedItem x;
      while (ok && items.template next<T::kEpi == FusedEpi::kPlain>(p, x)) {
        const bool a_mn = p.prod[x.which].a_mn_major != 0, b_mn = p.prod[x.which].b_mn_major != 0;
        const uint32_t idesc = make_idesc(p.bf16 ? 1u : 0u, a_mn, b_mn, T::kTile, T::kTile);
        // the start address sits in the descriptor's low bits, in units of 16 bytes
        const uint64_t a_desc = operand_desc<T>(op_smem, a_mn, 0), b_desc = operand_desc<T>(op_smem + T::kATile, b_mn, 0);
        const uint32_t a_step = (a_mn ? T::kInstrK * T::kRowBytes : 32) / 16, b_step = (b_mn ? T::kInstrK * T::kRowBytes : 32) / 16;
        for (int c0 = x.kb0; ok && c0 < x.kb1; ++g) {
          const int c1 = x.kb1 - c0 > T::kChunk ? c0 + T::kChunk : x.kb1;
          const uint32_t ab = g % T::kAccBufs;
          const uint32_t ph = ((g / T::kAccBufs) & 1u) ^ 1u;
          if (!(T::kPair ? warp_wait_relaxed(&acc_empty[ab], ph, ctl) : warp_wait(&acc_empty[ab], ph, ctl))) { ok = false; break; }
          tc_fence_after_sync();
          const uint32_t d0 = d_base + ab * T::kTile;
          for (int kb = c0; kb < c1; ++kb) {
            if (!warp_wait(&op_full[st], st_ph, ctl)) { ok = false; break; }
            tc_fence_after_sync();
            const uint64_t at = (uint64_t)(st * (T::kStage / 16));
            if (leader) {
#pragma unroll
              for (int ks = 0; ks < T::kKSteps; ++ks) {
                const uint64_t da = a_desc + at + ks * a_step, db = b_desc + at + ks * b_step;
                const uint32_t acc = (kb > c0 || ks > 0) ? 1u : 0u;
                if constexpr (T::kPair) mma_f16_pair(d0, da, db, idesc, acc);
                else mma_f16(d0, da, db, idesc, acc);
              }
              commit(&op_empty[st], 0x3);
              if (kb + 1 == c1) commit(&acc_full[ab], 0x3);
            }
            __syncwarp();
            if (++st == T::kStages) {
              st = 0;
              st_ph ^= 1u;
            }
          }
          c0 = c1;
        }
      }
      // every MMA completes before TMEM is released
      if (leader) {
        commit(done_bar, 0x1);
        drain_wait(done_bar, 0, p.wait_limit_ns);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - 2) / 4;
    const uint32_t stg = smem_addr(epi_base) + (warp - 2) * 4096;
    const uint32_t acc_empty0 = T::kPair ? cluster_smem_addr(smem_addr(acc_empty), 0) : 0u;
    constexpr int kCc = T::kTileN / 32 / 2;         // 32-column chunks of one warp
    const int cc0 = half * kCc;
    const bool bf16 = p.bf16 != 0;
    const Scale sc = T::kEpi == FusedEpi::kGatedGrad ? GradTop::scale(p) : warp_scale(p.scale, p.scale_count, p.scale_exp, p.scale_largest != 0);
    uint32_t g = 0;
    float top = 0.0f;                                // kGatedGrad: the largest gradient of a thread
    FusedItems items(p, worker, workers);
    constexpr bool kAhead = T::kEpi == FusedEpi::kGatedGrad;
    FusedItem x, ahead;
    bool more = kAhead && items.template next<false>(p, ahead);
    // dY's elements of a chunk, a row a lane, on their way while the accumulator is waited for
    uint32_t dyw[16];
    auto first_row = [&](const FusedItem& i) { return i.mb * T::kTile + (int)rank * T::BM + 32 * q; };
    auto fetch_dy = [&](int row, int col) {
      if (row < p.prod[0].m && col < p.prod[0].n)
        load_block16(stg, lane, dyw, Block16{const_cast<void*>(p.dy), p.lddy, row, p.prod[0].m, col, p.prod[0].n, p.dy_vec != 0});
    };
    if (more) fetch_dy(first_row(ahead), ahead.nb * T::kTileN + cc0 * 32);
    while (true) {
      if constexpr (kAhead) {
        if (!more) break;
        x = ahead;
        more = items.template next<false>(p, ahead);
      } else {
        if (!items.template next<T::kEpi == FusedEpi::kPlain>(p, x)) break;
      }
      const FusedProduct& pr = p.prod[x.which];
      const bool second = x.mb >= pr.mb_second;
      const uint32_t ab = g % T::kAccBufs;
      const uint32_t tacc = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + ab * T::kTile;
      const int row0 = (second ? x.mb - pr.mb_second : x.mb) * T::kTile + (int)rank * T::BM + 32 * q;
      const int row = row0 + lane;
      const int col_tile = x.nb * T::kTileN;
      auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          // (TMEM alone is handed over: a release would wait for the stores)
          if constexpr (T::kPair) mbar_arrive_cluster_relaxed(acc_empty0 + ab * 8u);
          else mbar_arrive(&acc_empty[ab]);
        }
      };
      // what a row needs is fetched before the accumulator is waited for
      int64_t target = -1;
      float lse2 = 0.0f, weight = 0.0f;
      if constexpr (T::kEpi == FusedEpi::kStats || T::kEpi == FusedEpi::kProb) {
        if (row < pr.m) {
          target = row_target(p, row);
          if constexpr (T::kEpi == FusedEpi::kProb) {
            lse2 = kLog2e * ld_global(p.lse + row);
            weight = row_weight(p, row, target, sc);
          }
        }
      }
      if constexpr (T::kEpi == FusedEpi::kStats) {
        // the chunks' sums, in registers: a row's half of the tile
        constexpr int kCols = T::kTile / 2;
        float acc[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
        bool live = true;
        for (int c0 = x.kb0; c0 < x.kb1; c0 = x.kb1 - c0 > T::kChunk ? c0 + T::kChunk : x.kb1, ++g) {
          const uint32_t buf = g % T::kAccBufs;
          if (!warp_wait(&acc_full[buf], (g / T::kAccBufs) & 1u, ctl)) { live = false; break; }
          tc_fence_after_sync();
          const uint32_t from = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + buf * T::kTile + half * kCols;
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            float v[16];
            tmem_ld_16cols(from + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += v[j];
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if constexpr (T::kPair) mbar_arrive_cluster_relaxed(acc_empty0 + buf * 8u);
            else mbar_arrive(&acc_empty[buf]);
          }
        }
        if (!live) break;
        if (x.slot >= 0) {
          if (row0 >= pr.m) continue;
          float* slot = p.slots + (int64_t)x.slot * (T::kTile * T::kTile) + (int64_t)((int)rank * T::BM + 32 * q) * T::kTile + half * kCols;
#pragma unroll
          for (int c = 0; c < kCols; c += 32) {
            stage_write_row(stg, lane, acc + c);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(slot + (i * 4 + (lane >> 3)) * T::kTile + c + (lane & 7) * 4) = stage_read_chunk(stg, lane, i);
            __syncwarp();
          }
          continue;
        }
        const int left = pr.n - col_tile - half * kCols;        // columns of the matrix from here on
        const int64_t at = target - (p.col0 + col_tile + half * kCols);   // (without a class: below 0)
        float top = -INFINITY, sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        bool nan = false;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          // (a bit for the target's column: compared with its index, the values went to local memory)
          const uint32_t mine = at >= c && at < c + 32 ? 1u << (at - c) : 0u;
          if (mine) {
            float l = 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) l = mine & (1u << j) ? acc[c + j] : l;
            p.target_logit[row] = l;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            acc[c + j] = c + j < left ? kLog2e * acc[c + j] : -INFINITY;
            nan = nan || acc[c + j] != acc[c + j];
            top = fmaxf(top, acc[c + j]);
          }
        }
        const float base = fabsf(top) == INFINITY ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum[j % 4] += ex2(acc[j] - base);
        if (row < pr.m)
          p.stats[(int64_t)(x.nb * 2 + half) * pr.m + row] = make_float2(top, nan ? NAN : (sum[0] + sum[1]) + (sum[2] + sum[3]));
        continue;
      } else {
        if (!warp_wait(&acc_full[ab], (g / T::kAccBufs) & 1u, ctl)) break;
        tc_fence_after_sync();
        ++g;
        if (x.slot >= 0) {
          // sums of a part of k, as they are: rows of the tile, whole lines a store
          float* slot = p.slots + (int64_t)x.slot * (T::kTile * T::kTile) + (int64_t)((int)rank * T::BM + 32 * q) * T::kTile;
          constexpr int kAll = T::kTile / 64;
#pragma unroll 1
          for (int cc = half * kAll; cc < (half + 1) * kAll; ++cc) {
            float v[32];
            tmem_ld_32cols(tacc + cc * 32, v);
            tmem_ld_wait();
            if (cc == (half + 1) * kAll - 1) release();
            if (row0 >= pr.m) continue;
            stage_write_row(stg, lane, v);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(slot + (i * 4 + (lane >> 3)) * T::kTile + cc * 32 + (lane & 7) * 4) =
                  stage_read_chunk(stg, lane, i);
            __syncwarp();
          }
          if (kAhead && more) fetch_dy(first_row(ahead), ahead.nb * T::kTileN + cc0 * 32);
          continue;
        }

        if constexpr (T::kTwo) {
#pragma unroll 1
          for (int cc = cc0; cc < cc0 + kCc; ++cc) {
            const int col0 = col_tile + cc * 32;
            float gt[32], up[32];
            tmem_ld_32cols(tacc + cc * 32, gt);
            tmem_ld_32cols(tacc + T::kTile / 2 + cc * 32, up);
            tmem_ld_wait();
            if (cc == cc0 + kCc - 1) release();
            uint32_t here[16];
            if constexpr (T::kEpi == FusedEpi::kGatedGrad) {
#pragma unroll
              for (int j = 0; j < 16; ++j) here[j] = dyw[j];
              // dY's elements of the next chunk, the next tile's first after the last
              if (cc + 1 < cc0 + kCc) fetch_dy(row0, col0 + 32);
              else if (more) fetch_dy(first_row(ahead), ahead.nb * T::kTileN + cc0 * 32);
            }
            if (row0 >= pr.m || col0 >= pr.n) continue;
            auto store = [&](int i, const uint32_t (&w)[16]) {
              store_block16(stg, lane, w, Block16{pr.out[i], pr.ldo[i], row0, pr.m, col0, pr.n, pr.out_vec[i] != 0});
            };
            uint32_t w[16];
            if constexpr (T::kEpi == FusedEpi::kGated) {
              if (pr.out[1]) {
                // act(gate) and up act'(gate), which the gradients are dY's multiples of
                uint32_t ka[16], kb[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                  float a0, d0, a1, d1;
                  act_both(gt[j], T::kAct, a0, d0);
                  act_both(gt[j + 1], T::kAct, a1, d1);
                  ka[j >> 1] = pack_kept(a0, a1, bf16);
                  kb[j >> 1] = pack_kept(up[j] * d0, up[j + 1] * d1, bf16);
                  w[j >> 1] = pack16(a0 * up[j], a1 * up[j + 1], bf16);
                }
                store(1, ka);
                store(2, kb);
              } else {
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                  w[j >> 1] = pack16(act_value(gt[j], T::kAct) * up[j], act_value(gt[j + 1], T::kAct) * up[j + 1], bf16);
              }
              store(0, w);
            } else {
              uint32_t wu[16];
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float2 dy = unpack16(here[j >> 1], bf16);
                const float y0 = sc.mul * dy.x, y1 = sc.mul * dy.y;
                float a0, d0, a1, d1;
                act_both(gt[j], T::kAct, a0, d0);
                act_both(gt[j + 1], T::kAct, a1, d1);
                const float g0 = y0 * (up[j] * d0), g1 = y1 * (up[j + 1] * d1), u0 = y0 * a0, u1 = y1 * a1;
                top = largest_finite(largest_finite(largest_finite(largest_finite(top, g0), g1), u0), u1);
                w[j >> 1] = pack16(g0, g1, bf16);
                wu[j >> 1] = pack16(u0, u1, bf16);
              }
              store(0, w);
              store(1, wu);
            }
          }
        } else if constexpr (T::kEpi == FusedEpi::kProb) {
          float v[32];
          tmem_ld_32cols(tacc + cc0 * 32, v);
#pragma unroll 1
          for (int cc = cc0; cc < cc0 + kCc; ++cc) {
            tmem_ld_wait();
            const int col0 = col_tile + cc * 32;
            uint32_t w[16];
            const bool in = row0 < pr.m && col0 < pr.n;
            if (in) {
              const int64_t at = target - (p.col0 + col0);
              const uint32_t mine = at >= 0 && at < 32 ? 1u << at : 0u;
              const bool any = __any_sync(0xffffffffu, mine != 0u);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = ex2(fmaf(kLog2e, v[j], -lse2));
              if (any) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = mine & (1u << j) ? v[j] - 1.0f : v[j];
              }
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[j] = weight == 0.0f ? 0u : pack16(weight * v[2 * j], weight * v[2 * j + 1], bf16);
            }
            if (cc + 1 < cc0 + kCc) tmem_ld_32cols(tacc + (cc + 1) * 32, v);
            else release();
            if (in) store_block16(stg, lane, w, Block16{pr.out[0], pr.ldo[0], row0, pr.m, col0, pr.n, pr.out_vec[0] != 0});
          }
        } else {
          const int dt = pr.out_dtype;
          void* out = pr.out[second ? 1 : 0];
          const int64_t ldo = pr.ldo[second ? 1 : 0];
          const bool vec = pr.out_vec[second ? 1 : 0] != 0;
          // (the next chunk's accumulators are on their way while this one is stored)
          float v[32];
          tmem_ld_32cols(tacc + cc0 * 32, v);
#pragma unroll 1
          for (int cc = cc0; cc < cc0 + kCc; ++cc) {
            tmem_ld_wait();
            const int col0 = col_tile + cc * 32;
            const bool in = row0 < pr.m && col0 < pr.n;
            auto next_chunk = [&]() {
              if (cc + 1 < cc0 + kCc) tmem_ld_32cols(tacc + (cc + 1) * 32, v);
              else release();
            };
            if (!in) {
              next_chunk();
              continue;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= sc.inv;
            if (dt != kOutF32 && !pr.add) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = pack16(v[2 * j], v[2 * j + 1], dt == kOutBF16);
              next_chunk();
              store_block16(stg, lane, w, Block16{out, ldo, row0, pr.m, col0, pr.n, vec});
              continue;
            }
            stage_write_row(stg, lane, v);
            __syncwarp();
            next_chunk();
            // (add has lines of whole 16-byte chunks)
            if (vec && col0 + 32 <= pr.n) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = row0 + i * 4 + (lane >> 3), c = col0 + (lane & 7) * 4;
                float4 o = stage_read_chunk(stg, lane, i);
                if (r < pr.m) {
                  if (pr.add) {
                    const float4 y = out_load4(pr.add, (int64_t)r * pr.ldadd + c, kOutF32);
                    o.x += y.x;
                    o.y += y.y;
                    o.z += y.z;
                    o.w += y.w;
                  }
                  out_store4(out, (int64_t)r * ldo + c, o, dt);
                }
              }
            } else if (col0 + lane < pr.n) {
#pragma unroll 4
              for (int r = 0; r < 32; ++r) {
                float o = stage_read_elem(stg, lane, r);
                if (row0 + r < pr.m) {
                  if (pr.add) o += out_load(pr.add, (int64_t)(row0 + r) * pr.ldadd + col0 + lane, kOutF32);
                  out_store(out, (int64_t)(row0 + r) * ldo + col0 + lane, o, dt);
                }
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if constexpr (T::kEpi == FusedEpi::kGatedGrad) {
      __syncwarp();
      if (p.record) GradTop::record(p.record, (int)blockIdx.x * T::kEpiWarps + warp - 2, top);
    }
  }

  // neither CTA of a pair leaves while the other may address its shared memory
  __syncwarp();
  tc_fence_before_sync();
  if constexpr (T::kPair) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (T::kPair) tmem_dealloc_pair(tmem_base, T::kTmemCols);
    else tmem_dealloc(tmem_base, T::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// split tiles
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store_four(void* out, int64_t at, const float (&v)[4], int left, bool vec, int dt) {
  if (vec && left >= 4) {
    out_store4(out, at, make_float4(v[0], v[1], v[2], v[3]), dt);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) out_store(out, at + j, v[j], dt);
  }
}
__device__ __forceinline__ void store_kept(void* out, int64_t at, const float (&v)[4], int left, bool vec, bool bf16) {
  const uint32_t w[2] = {pack_kept(v[0], v[1], bf16), pack_kept(v[2], v[3], bf16)};
  uint16_t* to = static_cast<uint16_t*>(out) + at;
  if (vec && left >= 4) {
    *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) to[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void load_four(float (&v)[4], const void* src, int64_t at, int left, bool vec, int dt) {
  if (vec && left >= 4) {
    const float4 y = out_load4(src, at, dt);
    v[0] = y.x;
    v[1] = y.y;
    v[2] = y.z;
    v[3] = y.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < left ? out_load(src, at + j, dt) : 0.0f;
  }
}

// Adds a tile's parts in the order of k, four columns a thread, and does what the
// epilogue does with the sums.  Tiles that one worker had whole are done already.
// A tile of many parts (few tiles, long k) has kSlices warps that
// add a run of them each: 150 parts of one tile 27 us with one.
constexpr int kJoinThreads = 256;
template <class T, int kSlices>
__global__ void __launch_bounds__(kJoinThreads) fused_join_kernel(const __grid_constant__ FusedGemmParams p) {
  constexpr int kPerRow = T::kTileN / 4;
  constexpr int kAt = kJoinThreads / kSlices;        // places of a block
  __shared__ float4 slices[kSlices > 1 ? kSlices : 1][T::kTwo ? 2 : 1][kSlices > 1 ? kAt : 1];
  griddep_wait();
  griddep_launch_dependents();
  if (T::kEpi == FusedEpi::kGatedGrad && !GradTop::needed(p, false)) return;
  const int tiles0 = p.prod[0].num_tiles - p.whole_tiles;                       // the second product's come after them
  const int which = T::kEpi == FusedEpi::kPlain && (int)blockIdx.x >= tiles0 ? 1 : 0;
  const FusedProduct& pr = p.prod[which];
  const int tile = which ? (int)blockIdx.x - tiles0 : p.whole_tiles + (int)blockIdx.x;
  const int64_t u0 = which ? p.units_first + (int64_t)tile * pr.num_k_blk : (int64_t)blockIdx.x * pr.num_k_blk;
  const int64_t u1 = u0 + pr.num_k_blk;
  const FusedParts parts(p, u0, u1);
  const int n = parts.count;
  if (n == 1) return;
  const FusedTile tc = fused_tile(pr, tile);
  const bool second = tc.mb >= pr.mb_second;
  const int place = threadIdx.x % kAt, slice = threadIdx.x / kAt;
  const int i = blockIdx.y * kAt + place;
  const int r = i / kPerRow, c = i % kPerRow * 4;
  const int row = (second ? tc.mb - pr.mb_second : tc.mb) * T::kTile + r, col = tc.nb * T::kTileN + c;
  const Scale sc = T::kEpi == FusedEpi::kGatedGrad ? GradTop::scale(p) : warp_scale(p.scale, p.scale_count, p.scale_exp, p.scale_largest != 0);
  const bool in = row < pr.m;
  const int left = pr.n - col;                       // columns of the matrix from here on
  constexpr int64_t kSlot = T::kTile * T::kTile;
  auto sum = [&](int which, int column, float (&v)[4]) {
    const float* at = p.slots + (int64_t)r * T::kTile + column;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4& y) {
      o.x += y.x;
      o.y += y.y;
      o.z += y.z;
      o.w += y.w;
    };
    if (in && left > 0) {
      const int j0 = kSlices > 1 ? n * slice / kSlices : 0, j1 = kSlices > 1 ? n * (slice + 1) / kSlices : n;
      if (j0 == 0) add(out_load4(at, parts.slot(0) * kSlot, kOutF32));
#pragma unroll 4
      for (int j = max(j0, 1); j < j1; ++j) add(out_load4(at, parts.slot(j) * kSlot, kOutF32));
    }
    if constexpr (kSlices > 1) {
      slices[slice][which][place] = o;
      __syncthreads();
      o = slices[0][which][place];
#pragma unroll
      for (int j = 1; j < kSlices; ++j) add(slices[j][which][place]);
    }
    v[0] = o.x;
    v[1] = o.y;
    v[2] = o.z;
    v[3] = o.w;
  };
  const int type = p.bf16 ? kOutBF16 : kOutF16;
  if constexpr (T::kTwo) {
    float gt[4], up[4];
    sum(0, c, gt);
    sum(1, T::kTile / 2 + c, up);
    const bool none = slice > 0 || !in || left <= 0;
    if (T::kEpi != FusedEpi::kGatedGrad && none) return;
    float top = 0.0f;
    if (!none) {
      auto at = [&](int k) { return (int64_t)row * pr.ldo[k] + col; };
      if constexpr (T::kEpi == FusedEpi::kGated) {
        if (pr.out[1]) {
          float ka[4], kb[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float d;
            act_both(gt[j], T::kAct, ka[j], d);
            kb[j] = up[j] * d;
          }
          store_kept(pr.out[1], at(1), ka, left, pr.out_vec[1], p.bf16 != 0);
          store_kept(pr.out[2], at(2), kb, left, pr.out_vec[2], p.bf16 != 0);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) gt[j] = act_value(gt[j], T::kAct) * up[j];
      } else {
        float dy[4];
        load_four(dy, p.dy, (int64_t)row * p.lddy + col, left, p.dy_vec, type);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float a, d;
          act_both(gt[j], T::kAct, a, d);
          const float y = sc.mul * dy[j];
          gt[j] = y * (up[j] * d);
          up[j] = y * a;
          if (j < left) top = largest_finite(largest_finite(top, gt[j]), up[j]);
        }
        store_four(pr.out[1], at(1), up, left, pr.out_vec[1], type);
      }
      store_four(pr.out[0], at(0), gt, left, pr.out_vec[0], type);
    }
    if constexpr (T::kEpi == FusedEpi::kGatedGrad) {
      __syncwarp();
      if (p.record) GradTop::record(p.record, (int)(blockIdx.x * gridDim.y + blockIdx.y) * (kJoinThreads / 32) + (int)(threadIdx.x >> 5), top);
    }
  } else {
    float v[4];
    sum(0, c, v);
    if (slice > 0) return;
    if constexpr (T::kEpi == FusedEpi::kPlain) {
      if (!in || left <= 0) return;
      const int k = second ? 1 : 0;
      float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (pr.add) load_four(y, pr.add, (int64_t)row * pr.ldadd + col, left, pr.out_vec[k], kOutF32);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fmaf(v[j], sc.inv, y[j]);
      store_four(pr.out[k], (int64_t)row * pr.ldo[k] + col, v, left, pr.out_vec[k], pr.out_dtype);
    } else {
      const int64_t target = in ? row_target(p, row) : -1;
      const int64_t at = target >= 0 ? target - (p.col0 + col) : -1;       // of these four columns: 0 .. 3
      if constexpr (T::kEpi == FusedEpi::kStats) {
        // half of the tile's columns of a row: kTile / 8 neighbouring lanes
        constexpr int kWidth = T::kTile / 8;
        float top = -INFINITY, s = 0.0f;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (at == j && j < left) p.target_logit[row] = v[j];
          v[j] = j < left ? kLog2e * v[j] : -INFINITY;
          nan = nan || v[j] != v[j];
          top = fmaxf(top, v[j]);
        }
#pragma unroll
        for (int o = kWidth / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float b = fabsf(top) == INFINITY ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < 4; ++j) s += ex2(v[j] - b);
        if (nan) s = NAN;
#pragma unroll
        for (int o = kWidth / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (in && i % kWidth == 0)
          p.stats[(int64_t)(tc.nb * 2 + c / (T::kTile / 2)) * pr.m + row] = make_float2(top, s);
      } else {
        if (!in || left <= 0) return;
        const float lse2 = kLog2e * ld_global(p.lse + row), weight = row_weight(p, row, target, sc);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = ex2(fmaf(kLog2e, v[j], -lse2));
          v[j] = weight == 0.0f ? 0.0f : weight * (at == j ? e - 1.0f : e);
        }
        store_four(pr.out[0], (int64_t)row * pr.ldo[0] + col, v, left, pr.out_vec[0], type);
      }
    }
  }
}

template <class T>
cudaError_t launch_fused_join(const FusedGemmParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const bool both = p.units > p.units_first;
  const int tiles = p.prod[0].num_tiles - p.whole_tiles + (both ? p.prod[1].num_tiles : 0);
  const bool many = p.dealers >= 8 * tiles;
  const int rows = both ? std::max(p.prod[0].m, p.prod[1].m) : p.prod[0].m;
  const int places = std::min(T::kTile, rows) * (T::kTileN / 4), at = many ? kJoinThreads / 8 : kJoinThreads;
  cfg.gridDim = dim3((unsigned)tiles, (unsigned)((places + at - 1) / at));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  return many ? cudaLaunchKernelEx(&cfg, fused_join_kernel<T, 8>, p)
              : cudaLaunchKernelEx(&cfg, fused_join_kernel<T, 1>, p);
}

template <class T>
FusedKernel fused_describe() {
  return FusedKernel{reinterpret_cast<const void*>(&fused_gemm_kernel<T>), T::kThreads, T::kSmemBytes, T::kTile, T::kCtas,
                     &launch_fused_join<T>};
}

}  // namespace
}  // namespace mpg
