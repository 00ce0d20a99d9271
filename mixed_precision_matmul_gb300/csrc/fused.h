// Internal structures of the 16-bit products with fused epilogues: the gated
// feed-forward product, the projection onto a vocabulary with its cross
// entropy, and the products of their gradients (fused_gemm.cuh, few_rows.cu,
// fused_aux.cu), launched from gated_api.cu and loss_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "host.h"

namespace mpg {

// What a product's accumulators become.
enum class FusedEpi {
  kPlain,      // C = inverse * sum (+ what earlier products left), fp32 or 16 bits
  kGated,      // Y = act(gate) * up; act(gate) and up act'(gate) too, where they are kept
  kGatedGrad,  // gradients of gate and up from that of Y
  kStats,      // maximum and sum of exponentials of a row's part; the target's logit
  kProb,       // gradient of the logits
};

constexpr int kMaxCtas = 160;          // workers of a launch, at most: the slots of split tiles are laid out for them
constexpr int kScaleBlocks = 304;      // partial maxima behind a scale
constexpr int kTopParts = 128;         // of the largest gradients made with it

// Rows that a product of few rows takes (few_rows.cu).
constexpr int kFewRows = 16;

// One product: operands, extents and where the result goes.
struct FusedProduct {
  CUtensorMap map_a[2], map_b[2];   // boxes of 64 x 64
  int32_t a_mn_major, b_mn_major;
  int32_t m, n;                     // of the result (kGated, kGatedGrad: n of each half)
  int32_t num_m_blk, num_n_blk, num_k_blk;
  int32_t kb_second;                // first block of k that comes from map_a[1] and map_b[1]
  int32_t mb_second;                // first row block of the second matrix: map_a[1], out[1]
  int32_t num_tiles, group_m;
  void* out[3];                     // kPlain: C, second C; kGated: Y, and act(gate), up act'(gate) (or null); kGatedGrad: dgate, dup; kProb: D
  int64_t ldo[3];
  int32_t out_vec[3];               // 8 elements of 16 bits (4 of fp32) are aligned
  int32_t out_dtype;
  const float* add;                 // kPlain: fp32, added to the result, or null
  int64_t ldadd;
};

struct FusedGemmParams {
  FusedProduct prod[2];             // kPlain: two products may share a launch, the longer k first
  int32_t bf16;
  int32_t whole_tiles;              // of the first: taken round by round; the others' blocks of k are dealt out evenly
  int64_t units, units_first;       // blocks of k of those others (and of all of the second's tiles); of the first's
  int32_t dealers;                  // workers that they are dealt to (0: none), no more than there are blocks
  float* slots;                     // partial tiles, two for each of those
  int32_t late, late_workers, late_rounds;   // the second's tiles: see FusedItems

  int32_t act;
  const void* dy;                   // kGatedGrad
  int64_t lddy;
  int32_t dy_vec;
  const float* scale;               // values whose largest sets the scale that 16-bit gradients carry, or null
  int32_t scale_count, scale_exp, scale_largest;   // see Scale
  float *record, *again;            // kGatedGrad: see GradTop (one of them, or neither)

  // cross entropy
  const void* target;
  int32_t target_bytes;
  int64_t target_stride, ignore_index;
  int32_t col0;                     // class of the first column
  int32_t vocab;
  float2* stats;                    // [part][m]: maximum (of logits times log2 e) and sum of 2^(. - maximum)
  float* target_logit;              // [m]
  const float* lse;
  const float* dloss;
  int64_t dloss_stride;

  uint32_t* status;
  uint64_t wait_limit_ns;
};

struct FusedKernel {
  const void* fn;
  int block, smem_bytes;
  int tile;                         // rows of a tile, and columns of its accumulators
  int ctas;
  // sums the parts of split tiles and does the epilogue's work
  cudaError_t (*join)(const FusedGemmParams& p, cudaStream_t stream);
};
void fused_lookup_plain(bool pair, FusedKernel* out);
void fused_lookup_gated(bool pair, int act, FusedKernel* out);
void fused_lookup_gated_grad(bool pair, int act, FusedKernel* out);
void fused_lookup_loss(FusedEpi epi, bool pair, FusedKernel* out);
// The product of few rows, with the epilogues of the tiles (but kPlain).
struct FewRowsParams {
  const void *x, *w, *wu;           // X: rows x k; weights: n x k; lines of whole 16 bytes, k a multiple of 8
  int64_t ldx, ldw, ldwu;
  int32_t bf16, rows, n, k;
  int32_t strips;
  int32_t act;
  void *y, *ka, *kb;                // Y, act(gate) and up act'(gate) (or null); dgate and dup; D
  int64_t ldy, lda, ldb;
  const void* dy;
  int64_t lddy;
  const float* scale;
  int32_t scale_count, scale_exp, scale_largest;
  float *record, *again;            // kGatedGrad: see GradTop
  const void* target;
  int32_t target_bytes;
  int64_t target_stride, ignore_index;
  int32_t col0, vocab;              // class of the first line; of all
  float2* stats;
  float* target_logit;
  const float *lse, *dloss;
  int64_t dloss_stride;
  uint32_t* status;
  uint64_t wait_limit_ns;
};
mpg_status launch_few_rows(DeviceInfo* dev, FewRowsParams& p, FusedEpi epi, cudaStream_t stream);
int few_rows_parts(int64_t n);      // of the statistics of n logits

// Weight gradients of few tokens: out[i] = inverse * d[i]^T x (few_grad.cu).  Blocks
// of rows are counted in a grid's second dimension.
constexpr int kFewGradTokens = 64;
constexpr int64_t kFewGradRows = 65535ll * 128;
struct FewGradParams {
  const uint16_t *d[2], *x;         // tokens x rows, tokens x cols; lines start on 16 bytes
  int64_t ldd, ldx;
  int32_t tokens, rows, cols, count, bf16;
  void* out[2];                     // lines start on 16 bytes
  int64_t ldo[2];
  const float* scale;
  int32_t scale_count, scale_exp, scale_largest;
};
cudaError_t launch_few_grad(const FewGradParams& p, cudaStream_t stream);

// Copies of matrices whose lines TMA cannot describe.
struct PadParams {
  struct Matrix {
    const uint16_t* src;
    uint16_t* dst;
    int64_t ld_src, ld_dst, rows, cols;
  } mat[4];
  int32_t count;
};
cudaError_t launch_pad(const PadParams& p, int sm_count, cudaStream_t stream);

// Partial maxima of |x| over a matrix (16 bits) or of |dloss| over the tokens that count.
struct MaxParams {
  const void* x;
  int64_t ld, rows, cols;
  int32_t vec, flat;                // flat: aligned lines of whole 16 bytes without gaps
  const float* dloss;
  int64_t dloss_stride;
  const void* target;
  int32_t target_bytes;
  int64_t target_stride, ignore_index;
  float* partial;                   // [kScaleBlocks]
  float* top;                       // [kTopParts], set to 0; or null
};
cudaError_t launch_max(const MaxParams& p, cudaStream_t stream);

// dgate = dY b and dup = dY a from the kept a = act(gate) and b = up act'(gate).
struct GatedGradParams {
  const void *dy, *a, *b;
  int64_t lddy, lda, ldb;
  uint16_t *dg, *du;
  int64_t ldd;
  int64_t rows, cols;
  int32_t vec, bf16;
  const float* scale;
  int32_t scale_count, scale_exp;
  float *record, *again;            // see GradTop
};
cudaError_t launch_gated_grad(const GatedGradParams& p, int sm_count, cudaStream_t stream);

// loss and lse from the parts' maxima and sums.
struct LossJoinParams {
  const float2* stats;
  int32_t parts;
  int64_t rows;
  const float* target_logit;
  const void* target;
  int32_t target_bytes;
  int64_t target_stride, ignore_index, vocab;
  float *loss, *lse;
};
cudaError_t launch_loss_join(const LossJoinParams& p, cudaStream_t stream);

// ---- host services shared by the two APIs (fused_plan.cu)
struct FusedLaunch {
  FusedEpi epi;
  int64_t m, n, k;                  // k: of the first part where there are two
  bool second_k = false;            // the second part of k has the same length
  bool second_m = false;            // a second matrix of m rows
};
mpg_status launch_fused(DeviceInfo* dev, const FusedLaunch& l, FusedGemmParams& p, float* slots, cudaStream_t stream);
// Both of p's products, in one launch where that takes less.
mpg_status launch_fused_two(DeviceInfo* dev, const FusedLaunch& l0, const FusedLaunch& l1, FusedGemmParams& p, float* slots,
                            cudaStream_t stream);
// Bytes of the slots that a launch (of two products) may need.
size_t fused_slot_bytes(const FusedLaunch& l, const FusedLaunch* second = nullptr);
// rows x k operand of a product: K-major if k is the matrix's contiguous side.
mpg_status fused_map(CUtensorMap* map, const void* ptr, int64_t ld, mpg_dtype dt, bool mn_major, int64_t rows, int64_t k);

constexpr int64_t kFusedMaxExtent = 0x7FFFFFFF - 255;   // the last tile's end, and a block beyond it, still fit 32 bits
inline int64_t fused_line(int64_t n) { return (n + 7) / 8 * 8; }
// Lines of the library's own matrices start on 128 bytes: a TMA box of lines that
// cross those takes half as long again (900 cycles a block of k instead of 600).
inline int64_t fused_wide_line(int64_t n) { return (n + 63) / 64 * 64; }
inline bool fused_aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// TMA can describe rows x cols lines of 16-bit elements
inline bool fused_lines_ok(const void* p, int64_t ld) { return fused_aligned(p, 16) && ld % 8 == 0; }

}  // namespace mpg
