// Device pieces shared by the two kernels of the block-scaled 8-bit product
// (fp8_gemm.cu on single CTAs, fp8_pair.cu on CTA pairs).
//
// The product's sum is over k in blocks of 128, and every block has its own
// scales: sum_kb sr[r, kb] sc[c, kb] P_kb[r, c].  The tensor cores compute each
// P_kb (four K = 32 instructions of kind::f8f6f4 into a fresh fp32
// accumulator in TMEM); the epilogue warps read it back and add sr * sc * P_kb
// to running sums in fp32 registers while the tensor cores work on the next
// block in another TMEM buffer.
#pragma once

#include "cluster.cuh"
#include "fp8.h"
#include "outio.cuh"
#include "staging.cuh"
#include "tc_gemm.cuh"

namespace mpg {

constexpr int kFp8RowBytes = 128;   // one line of a stage: 128 k of one row, 128B-swizzled

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// K-major 128B-swizzled operand, k-step ks of 32 bytes.
__device__ __forceinline__ uint64_t fp8_desc(uint32_t tile_addr, int ks) {
  return make_smem_desc(tile_addr + ks * 32u, 16u, 8u * kFp8RowBytes, kSwizzle128B);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// One arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_b64(uint32_t addr, unsigned long long v) {
  asm volatile("st.shared.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Pairs of fp32 values in one 64-bit register, and their packed arithmetic
// (each element rounded to nearest, as the scalar forms do).  Running sums are
// kept in this form: built from single registers at each use they cost a move
// an element.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ void fma2(f32x2& a, f32x2 x, f32x2 y) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(x), "l"(y));
}
__device__ __forceinline__ f32x2 mul2(f32x2 x, f32x2 y) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ void ld_shared_pairs(uint32_t addr, f32x2& a, f32x2& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

// How a block's two scales meet its sum P, |P| in [2^-32, 2^39) or 0: scales may
// be any fp32 values, and no step but the last may leave fp32's normal range.
//   one scale for all columns   P * (row * column), where that product of the
//                               scales is in the normal range or one of them
//                               is 0;
//   a scale for each column     (P * column) * row, where the columns' scales
//                               are 0 or in [2^-94, 2^89), so that P * column is
//                               in range.  (In the other order the multiply-add
//                               has three operands that change: 126 us instead
//                               of 118 at 4096^3.)
// With one scale for all columns each block's form is chosen by itself (8192^3:
// 437 us; 432 without the choice, 487 with one for every 32 columns).  With a
// scale for each column that takes too long beside the additions (4096^3: 126
// us; 118 without the choice): a tile's form is chosen by its columns' scales in
// all blocks (117 us), which the epilogue's threads look at before the first
// tile, while its first operands are on their way, and a warp beside them for
// each tile after.
// Elsewhere the row's scale is taken in two parts, first * last, last a power
// of two: ((P * first) * column) * last.  For tiny rows first is in
// [2^-94, 2^-39): P * first * column cannot overflow, and where it is below the
// normal range the result is below 2^-181.  For huge rows first is in
// [2^69, 2^89): the reverse.  (All blocks in that form: 8192^3 856 us, 4096^3
// with a scale for each column 133.)
__device__ __forceinline__ uint32_t scale_field(float s) { return (__float_as_uint(s) >> 23) & 255u; }
__device__ __forceinline__ bool plain_scale(float row, float col) {
  return scale_field(row * col) - 1u < 254u || fminf(fabsf(row), fabsf(col)) == 0.0f;
}
__device__ __forceinline__ bool plain_column(float col) {
  return scale_field(col) - (127u - 94u) < 94u + 89u || col == 0.0f;
}
__device__ __forceinline__ void split_scale(float row, float& first, float& last) {
  const int e = (int)scale_field(row) - 127;
  int shift = 0;                                 // (also of infinities and NaN, e = 128)
  if (e < -94) shift = -55;
  else if (e >= 108 && e < 128) shift = 39;
  else if (e >= 89 && e < 128) shift = 20;
  first = row * __uint_as_float((uint32_t)(127 - shift) << 23);
  last = __uint_as_float((uint32_t)(127 + shift) << 23);
}

// Whether the scales of kTileCols columns from col0 on are plain in n blocks;
// `thread` of kThreads looks at its share of them, sixteen loads at a time.
template <int kThreads, int kTileCols>
__device__ __forceinline__ bool scan_share(const Fp8GemmParams& p, int thread, int col0, int kb0, int n) {
  static_assert(kThreads % kTileCols == 0 || kTileCols % kThreads == 0, "whole blocks at a time");
  constexpr int kStep = kThreads > kTileCols ? kThreads / kTileCols : 1;     // blocks side by side
  constexpr int kPer = kTileCols > kThreads ? kTileCols / kThreads : 1;      // columns of a thread
  constexpr int kAtOnce = 16 / kPer;
  const int col = col0 + thread % kTileCols;
  bool ok = true;
#pragma unroll 1
  for (int kb = thread / kTileCols; kb < n; kb += kAtOnce * kStep) {
    float x[kPer][kAtOnce];
#pragma unroll
    for (int c = 0; c < kPer; ++c) {
      const float* src = p.sc + (int64_t)((col + c * kThreads) >> p.sc_shift) * p.sc_row + (int64_t)kb0 * p.sc_k;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
        x[c][u] = col + c * kThreads < p.cols && kb + u * kStep < n ? ld_global(src + (kb + u * kStep) * p.sc_k) : 1.0f;
    }
#pragma unroll
    for (int c = 0; c < kPer; ++c)
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) ok = ok && plain_column(x[c][u]);
  }
  return ok;
}
// By the kThreads threads of the epilogue together, before anything that they
// may give up waiting for.
constexpr int kScanBarrier = 1;
template <int kThreads, int kTileCols>
__device__ __forceinline__ bool scan_together(const Fp8GemmParams& p, int thread, int col0, int kb0, int n) {
  const bool ok = scan_share<kThreads, kTileCols>(p, thread, col0, kb0, n);
  __syncwarp();
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "barrier.cta.red.and.pred b, %2, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "n"(kScanBarrier), "n"(kThreads)
      : "memory");
  return all != 0;
}
// By a warp, for itself.
template <int kTileCols>
__device__ __forceinline__ bool scan_alone(const Fp8GemmParams& p, int lane, int col0, int kb0, int n) {
  const bool ok = scan_share<32, kTileCols>(p, lane, col0, kb0, n);
  return __all_sync(0xffffffffu, ok) != 0;
}

// A lane's columns of 128 (lane, lane + 32, ..) where each has its own scale, in
// the block `at` points to: few registers, for warps that have few.
struct ColumnLines {
  const float* at;
  int count;                 // of the lane's columns inside the matrix
  __device__ __forceinline__ void start(const Fp8GemmParams& p, int col0, int lane) {
    count = (p.cols - 1 - col0 - lane + 32) / 32;        // (<= 0: none)
    at = p.sc + (int64_t)(col0 + lane) * p.sc_row;
  }
  __device__ __forceinline__ const float* column(const Fp8GemmParams& p, int i) const { return at + (int64_t)(32 * i) * p.sc_row; }
  __device__ __forceinline__ void next(const Fp8GemmParams& p) { at += p.sc_k; }
};
// Looks at such columns a block at each call (at its loads in the next one).
struct ColumnScan {
  ColumnLines lines;
  float x[4];
  bool ok;
  __device__ __forceinline__ void start(const Fp8GemmParams& p, int col0, int lane) {
    ok = true;
    lines.start(p, col0, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 1.0f;
  }
  __device__ __forceinline__ void look() {
#pragma unroll
    for (int i = 0; i < 4; ++i) ok = ok && plain_column(x[i]);
  }
  __device__ __forceinline__ void block(const Fp8GemmParams& p) {
    look();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < lines.count) x[i] = ld_global(lines.column(p, i));
    lines.next(p);
  }
  __device__ __forceinline__ bool result() {
    look();
    return __all_sync(0xffffffffu, ok) != 0;
  }
};

// What a warp beside the epilogue finds for the tiles after a CTA's first is
// left in notes, a ring of kNotes.
constexpr uint32_t kNotes = 4;
struct Notes {
  uint32_t* word;
  uint64_t* full;        // one arrival: the note is there
  uint64_t* empty;       // kReaders arrivals: it has been read
  static constexpr int kBytes = kNotes * (4 + 2 * 8);
  // note number i (from 0), written by one warp; false when a wait gave up
  __device__ __forceinline__ bool leave(uint32_t i, bool plain, int lane, const WaitCtl& ctl) const {
    if (!warp_wait(&empty[i % kNotes], ((i / kNotes) & 1u) ^ 1u, ctl)) return false;
    if (lane == 0) {
      word[i % kNotes] = plain;
      mbar_arrive(&full[i % kNotes]);
    }
    __syncwarp();
    return true;
  }
  __device__ __forceinline__ bool read(uint32_t i, int lane, const WaitCtl& ctl, bool* plain) const {
    if (!warp_wait(&full[i % kNotes], (i / kNotes) & 1u, ctl)) return false;
    *plain = ld_shared_u32(smem_addr(word + i % kNotes)) != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[i % kNotes]);
    return true;
  }
};

// The scales of one epilogue warp, its 32 rows and `kCols` columns, fetched
// kDepth - 1 blocks of k ahead into a ring in shared memory that only this
// warp uses.
template <int kCols, int kDepth_>
struct ScaleRing {
  static constexpr int kDepth = kDepth_;
  static constexpr int kSlot = 32 + kCols;                          // floats
  static constexpr int kBytes = kDepth * kSlot * 4;
  static constexpr int kColLoads = (kCols + 31) / 32;
  uint32_t base;
  const float* row_src;                  // the next block's to fetch
  const float* col_src[kColLoads];
  int64_t row_k, col_k;
  int lane, left;                        // blocks still to fetch

  // rows row0 .. row0 + 31, columns col0 .. col0 + kCols - 1, clamped to the
  // operands' last line, of `n` blocks from k-block kb0 on; fetches the first
  __device__ __forceinline__ void start(const Fp8GemmParams& p, uint32_t smem, int lane_, int row0, int col0, int kb0,
                                        int n) {
    base = smem;
    lane = lane_;
    left = n;
    row_k = p.sr_k;
    col_k = p.sc_k;
    row_src = p.sr + (int64_t)(min(row0 + lane, p.rows - 1) >> p.sr_shift) * p.sr_row + (int64_t)kb0 * p.sr_k;
#pragma unroll
    for (int i = 0; i < kColLoads; ++i)
      col_src[i] = p.sc + (int64_t)(min(col0 + i * 32 + lane, p.cols - 1) >> p.sc_shift) * p.sc_row + (int64_t)kb0 * p.sc_k;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i);
  }
  __device__ __forceinline__ uint32_t slot(uint32_t i) const { return base + (i % kDepth) * (kSlot * 4); }
  // the next block's scales into slot i, if there is one
  __device__ __forceinline__ void fetch(uint32_t i) {
    if (left > 0) {
      --left;
      const uint32_t s = slot(i) + lane * 4;
      cp_async4(s, row_src);
      row_src += row_k;
#pragma unroll
      for (int j = 0; j < kColLoads; ++j) {
        if (kCols % 32 == 0 || j * 32 + lane < kCols) cp_async4(s + 128 + j * 128, col_src[j]);
        col_src[j] += col_k;
      }
    }
    cp_async_commit();
  }
};

// acc += row scale * column scale * v on kN columns from column c0 of the
// warp's slot (col: the scale of all columns).  kPlain: the caller branches
// once a block or a tile, and this code stays in one piece with the reads of
// TMEM around it.
template <int kN, bool kColVec, bool kPlain>
__device__ __forceinline__ void scale_add(f32x2* acc, const float* v, uint32_t slot, int c0, float row, float col) {
  float f, l;
  if constexpr (kPlain) f = l = kColVec ? row : row * col;
  else split_scale(row, f, l);
  const f32x2 first = pack2(f, f), last = pack2(l, l), cols = pack2(col, col);
#pragma unroll
  for (int j = 0; j < kN; j += 4) {
    const f32x2 v0 = pack2(v[j], v[j + 1]), v1 = pack2(v[j + 2], v[j + 3]);
    f32x2 s0 = cols, s1 = cols;
    if constexpr (kColVec) ld_shared_pairs(slot + 128 + (c0 + j) * 4, s0, s1);
    if constexpr (!kPlain) {
      fma2(acc[j / 2], mul2(mul2(v0, first), s0), last);
      fma2(acc[j / 2 + 1], mul2(mul2(v1, first), s1), last);
    } else if constexpr (kColVec) {
      fma2(acc[j / 2], mul2(v0, s0), last);
      fma2(acc[j / 2 + 1], mul2(v1, s1), last);
    } else {
      fma2(acc[j / 2], v0, last);
      fma2(acc[j / 2 + 1], v1, last);
    }
  }
}

// One block of k with a scale for each column: the accumulator at `ta` (kCols
// columns of this warp's 32 lanes) added to the running sums under the row's
// scale and the column scales in `slot`, two reads of 32 columns on their
// way.  `release` runs when all columns are in registers.
template <int kCols, bool kPlain, class Release>
__device__ __forceinline__ void add_block(f32x2 (&acc)[kCols / 2], uint32_t ta, uint32_t slot, float row,
                                          Release release) {
  constexpr int kChunk = kCols >= 32 ? 32 : 16;
  constexpr int kN = kCols / kChunk;
  static_assert(kN <= 2, "all reads at once");
  float v[kN][kChunk];
#pragma unroll
  for (int c = 0; c < kN; ++c) {
    if constexpr (kChunk == 32) tmem_ld_32cols(ta + c * kChunk, v[c]);
    else tmem_ld_16cols(ta + c * kChunk, v[c]);
  }
  tmem_ld_wait();
  release();
#pragma unroll
  for (int c = 0; c < kN; ++c) scale_add<kChunk, true, kPlain>(acc + c * kChunk / 2, v[c], slot, c * kChunk, row, 1.0f);
}

// alpha x + beta C for 32 rows (one a lane) and 32 columns (x[j]: columns 2j
// and 2j + 1).  Rows pass through 64-byte lines of shared memory (32 16-bit values, or 16
// fp32 values twice), chunk c of row r at slot c ^ ((r / 2) & 3): writes and
// reads (four lanes a row) reach all banks.  Each store then covers 8 rows x
// 64 bytes.
__device__ __forceinline__ void store_rows32(const Fp8GemmParams& p, uint32_t stg, int lane, const f32x2* x,
                                             int row_base, int col_base) {
  auto at = [&](int r, int c) { return stg + r * 64 + ((c ^ ((r >> 1) & 3)) << 4); };   // 16-byte chunk c of row r
  const int dt = p.out_dtype;
  if (dt != kOutF32 && p.beta == 0.0f) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float lo, hi;
      unpack2(x[j], lo, hi);
      w[j] = dt == kOutF16 ? pack_f16x2(p.alpha * lo, p.alpha * hi) : pack_bf16x2(p.alpha * lo, p.alpha * hi);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) st_shared_v4(at(lane, c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    __syncwarp();
    uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)row_base * p.ld_out + col_base;
    if (p.out_vec16 && col_base + 32 <= p.cols) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), c = lane & 3;
        const float4 y = stage_ld16(at(r, c));
        if (row_base + r < p.rows) *reinterpret_cast<float4*>(out + (int64_t)r * p.ld_out + c * 8) = y;
      }
    } else if (col_base + lane < p.cols) {
      // lines off 16 bytes: a row at a time, a column a lane
#pragma unroll 8
      for (int r = 0; r < 32; ++r) {
        const uint16_t y = ld_shared_u16(at(r, lane >> 3) + (lane & 7) * 2);
        if (row_base + r < p.rows) out[(int64_t)r * p.ld_out + lane] = y;
      }
    }
    __syncwarp();
    return;
  }
#pragma unroll
  for (int hc = 0; hc < 2; ++hc) {                        // 16 columns
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        st_shared_b64(at(lane, c), x[hc * 8 + 2 * c]);
        st_shared_b64(at(lane, c) + 8, x[hc * 8 + 2 * c + 1]);
      }
    __syncwarp();
    if (p.out_vec && col_base + 16 * hc + 16 <= p.cols) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), c = lane & 3;
        const float4 y = stage_ld16(at(r, c));
        if (row_base + r >= p.rows) continue;
        const int64_t idx = (int64_t)(row_base + r) * p.ld_out + col_base + 16 * hc + 4 * c;
        float4 o = make_float4(p.alpha * y.x, p.alpha * y.y, p.alpha * y.z, p.alpha * y.w);
        if (p.beta != 0.0f) {
          const float4 z = out_load4(p.out, idx, dt);
          o.x = fmaf(p.beta, z.x, o.x);
          o.y = fmaf(p.beta, z.y, o.y);
          o.z = fmaf(p.beta, z.z, o.z);
          o.w = fmaf(p.beta, z.w, o.w);
        }
        out_store4(p.out, idx, o, dt);
      }
    } else {
      // two rows at a time, a column a lane
      const int col = col_base + 16 * hc + (lane & 15);
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int r = 2 * i + (lane >> 4);
        const float y = p.alpha * stage_ld4(at(r, (lane & 15) >> 2) + (lane & 3) * 4);
        if (row_base + r < p.rows && col < p.cols) {
          const int64_t idx = (int64_t)(row_base + r) * p.ld_out + col;
          out_store(p.out, idx, p.beta != 0.0f ? fmaf(p.beta, out_load(p.out, idx, dt), y) : y, dt);
        }
      }
    }
    __syncwarp();
  }
}

}  // namespace mpg
