// Internal structures of the 8-bit operators: the quantiser (fp8_quant.cu) and
// the block-scaled product (fp8_gemm.cu, fp8_pair.cu), launched from
// fp8_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mpg {

constexpr int kFp8Block = 128;   // elements of k that share a scale

struct Fp8QuantParams {
  const void* x;
  int64_t ldx;
  int32_t rows, cols;
  int32_t x_align;            // alignment of every line of x in bytes: 16, 8, 4 or 2
  uint8_t* q;                 // rows x cols, or null
  int64_t ldq;
  int32_t q_vec;              // 8-byte chunks of q are aligned
  float* s;
  int64_t s_row, s_k;
  uint8_t* qt;                // cols x rows, or null
  int64_t ldqt;
  int32_t qt_vec;             // 16-byte chunks of qt are aligned
  float* st;
  int64_t st_row, st_k;
};
cudaError_t launch_fp8_quantize(const Fp8QuantParams& p, int x_dtype, int format, int scale_rows,
                                cudaStream_t stream);

// Lines of `cols` bytes copied, from any alignment, to lines of ld_out bytes
// (ld_out = 16 chunks, out 16-byte aligned, padding zeroed).  rows 0: no copy.
struct Fp8AlignJob {
  const uint8_t* in;
  int64_t ld_in, rows, cols, chunks;
  uint8_t* out;
  int64_t ld_out;
};
cudaError_t launch_fp8_align(const Fp8AlignJob& a, const Fp8AlignJob& b, int sm_count, cudaStream_t stream);

// The product D[r, c] = sum_kb sr[r, kb] sc[c, kb] (R_kb C_kb^T)[r, c], where
// R (rows x k) feeds the 128 rows of a tensor-core tile and C (cols x k) its
// columns.  `swapped`: R is the caller's B and C the caller's A (few tokens),
// and D is stored transposed.
struct Fp8GemmParams {
  CUtensorMap map_r, map_c;
  const float* sr;
  const float* sc;
  int64_t sr_row, sr_k, sc_row, sc_k;   // element strides of the scales
  int32_t sr_shift, sc_shift;           // 7: one scale for 128 rows, 0: one a row
  void* out;
  int64_t ld_out;
  int32_t out_dtype;
  int32_t out_vec;                      // 4-element vectors of C are aligned
  int32_t out_vec16;                    // 16-byte chunks of C are aligned
  int32_t rows, cols;                   // extents of D
  int32_t num_r_blk, num_c_blk, num_k_blk;
  int32_t splits, kb_per_split;
  int32_t num_tiles, group;             // persistent kernel
  uint32_t fmt_bits;                    // operand formats in the instruction descriptor
  float alpha, beta;
  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct Fp8Kernel {
  const void* fn;
  int block, smem_bytes;
  int tile_rows, tile_cols;
};
// One-CTA tiles of 128 x bn: bn = 128 (D as the caller's C; col_vec: a scale
// for each column, else one for all 128), bn = 16, 32, 64 (swapped).
// `direct`: tile after tile on one CTA; else a tile, or a share of its k, to each.
bool fp8_lookup(int bn, bool swapped, bool col_vec, bool direct, Fp8Kernel* out);
// 256 x 256 tiles on CTA pairs.
bool fp8_lookup_pair(bool col_vec, Fp8Kernel* out);

}  // namespace mpg
