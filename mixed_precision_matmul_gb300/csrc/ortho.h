// Internal structures of the orthogonalised update: the norm and scaling
// kernels and the fp16 product with a fused linear epilogue (ortho.cu),
// launched from ortho_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mpg {

// Blocks that sum the squares of one matrix, at most.
constexpr int kOrthoNormBlocks = 384;
constexpr int kOrthoMaxSteps = 100;

struct OrthoScaleParams {
  const void* g;
  int64_t ldg, stride_g;
  int32_t rows, cols, batch;
  int32_t g_vec;              // 8-element chunks of a line of g are 16-byte aligned
  int32_t flat;               // neither g nor x has gaps between its lines
  double* partial;            // [batch][kOrthoNormBlocks]
  int32_t blocks;             // partial sums of one matrix
  uint16_t* x;                // fp16 [batch][rows][ldx], ldx % 8 == 0
  int64_t ldx;
  float* factor;              // [step][batch]: the iterate is factor * what is stored of it; powers of two but for the first
  int32_t steps;
  float coeff_size[3];        // |a|, |b|, |c|
  int32_t target_exp;         // x is scaled by a power of two to a norm in [2^t, 2^(t+1))
  int32_t store_exp;          // iterates with singular values near 1 are stored times 2^s
  float eps;
};
cudaError_t launch_ortho_scale(const OrthoScaleParams& p, int g_dtype, cudaStream_t stream);

// D = ca * A B + cz * Z + co * D, for each matrix of the batch.
struct OrthoGemmParams {
  CUtensorMap map_a, map_b;   // fp16; box 64 x 128 (K-major) or 64 x 64 (MN-major)
  int32_t a_mn_major, b_mn_major;
  int32_t m, n, k, batch;
  int32_t symmetric;          // D and Z are symmetric: tiles above the diagonal are stored twice
  int32_t num_m_blk, num_n_blk, num_k_blk, tiles_per_matrix, num_tiles, group_m;
  const uint16_t* z;          // fp16, or null
  int64_t ldz, stride_z;
  void* d;
  int64_t ldd, stride_d;
  int32_t d_dtype;            // 0 fp32, 1 fp16, 2 bf16
  int32_t vec;                // 4-element vectors of D are aligned
  int32_t vec16;              // 16-byte chunks of a 16-bit D are aligned
  float ca, cz, co;
  const float* factor;        // of each matrix, or null
  const float* next;          // of each matrix's next iterate, or null
  int32_t square;             // ca is multiplied by factor^2; else ca and cz by factor / next
  int32_t splits, kb_per_split;   // divided form: ranges of k, each on a CTA of one cluster
  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct OrthoKernel {
  const void* fn;
  int block, smem_bytes;
  int tile;                   // tiles are tile x tile
  int ctas;                   // CTAs that share a tile
};
enum class OrthoForm { kOne, kPair, kDivided };
void ortho_lookup(OrthoForm form, OrthoKernel* out);

}  // namespace mpg
