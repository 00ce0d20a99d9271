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
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// acc += x * y on two packed fp32 values (each a round-to-nearest fma).
__device__ __forceinline__ void fma2(float& a0, float& a1, float x0, float x1, float y0, float y1) {
  asm("{\n\t.reg .b64 a, x, y;\n\t"
      "mov.b64 a, {%0, %1};\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "fma.rn.f32x2 a, x, y, a;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}
__device__ __forceinline__ void mul2(float& r0, float& r1, float x0, float x1, float y0, float y1) {
  asm("{\n\t.reg .b64 r, x, y;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 r, x, y;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(x0), "f"(x1), "f"(y0), "f"(y1));
}

// The scales of one epilogue warp: its 32 rows and `kCols` columns (or the one
// scale of all its columns), fetched kDepth - 1 blocks of k ahead into a ring
// in shared memory that only this warp uses.
template <int kCols, bool kColVec>
struct ScaleRing {
  static constexpr int kDepth = 8;
  static constexpr int kSlot = 32 + (kColVec ? kCols : 32);        // floats
  static constexpr int kBytes = kDepth * kSlot * 4;
  uint32_t base;
  const float* row_src;
  const float* col_src[kColVec ? (kCols + 31) / 32 : 1];
  int64_t row_k, col_k;
  int lane;

  // rows row0 .. row0 + 31, columns col0 .. col0 + kCols - 1, clamped to the
  // operands' last line; k-block kb0 is block 0 of this ring
  __device__ __forceinline__ void start(const Fp8GemmParams& p, uint32_t smem, int lane_, int row0, int col0, int kb0) {
    base = smem;
    lane = lane_;
    row_k = p.sr_k;
    col_k = p.sc_k;
    const int r = min(row0 + lane, p.rows - 1) >> p.sr_shift;
    row_src = p.sr + (int64_t)r * p.sr_row + (int64_t)kb0 * p.sr_k;
#pragma unroll
    for (int i = 0; i < (kColVec ? (kCols + 31) / 32 : 1); ++i) {
      const int c = min(kColVec ? col0 + i * 32 + lane : col0, p.cols - 1) >> p.sc_shift;
      col_src[i] = p.sc + (int64_t)c * p.sc_row + (int64_t)kb0 * p.sc_k;
    }
  }
  __device__ __forceinline__ uint32_t slot(int i) const { return base + (uint32_t)(i % kDepth) * (kSlot * 4); }
  __device__ __forceinline__ void fetch(int i, int n) const {
    if (i < n) {
      const uint32_t s = slot(i);
      cp_async4(s + lane * 4, row_src + i * row_k);
      if constexpr (kColVec) {
#pragma unroll
        for (int j = 0; j < (kCols + 31) / 32; ++j)
          if (kCols % 32 == 0 || j * 32 + lane < kCols) cp_async4(s + 128 + (j * 32 + lane) * 4, col_src[j] + i * col_k);
      } else {
        cp_async4(s + 128 + lane * 4, col_src[0] + i * col_k);
      }
    }
    cp_async_commit();
  }
};

// acc[j] += row scale * column scale * v[j] for `kN` columns from column
// offset c0 of the warp's slot.
template <int kN, bool kColVec>
__device__ __forceinline__ void scale_add(float* acc, const float* v, uint32_t slot, int c0, float rs, float rcs) {
  if constexpr (kColVec) {
#pragma unroll
    for (int j = 0; j < kN; j += 4) {
      const float4 s = ld_shared_f4(slot + 128 + (c0 + j) * 4);
      float x0, x1, x2, x3;
      mul2(x0, x1, v[j], v[j + 1], s.x, s.y);
      mul2(x2, x3, v[j + 2], v[j + 3], s.z, s.w);
      fma2(acc[j], acc[j + 1], x0, x1, rs, rs);
      fma2(acc[j + 2], acc[j + 3], x2, x3, rs, rs);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kN; j += 2) fma2(acc[j], acc[j + 1], v[j], v[j + 1], rcs, rcs);
  }
}

}  // namespace mpg
