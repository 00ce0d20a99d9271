// Weight gradients of few tokens, out = inverse * D^T X with up to 64 tokens
// (sm_103a): every element of the result is a sum of at most 64 products, and what
// counts is how fast results are written.
//
// A CTA has 128 rows by 128 columns; its tokens' D and X lie in shared memory, and
// a warp has 16 rows.  Operands of mma.sync m16n8k16 come by transposing ldmatrix
// loads, since both have tokens as their lines.  X's columns are permuted within
// each 32 as they are stored: column 8a + 2j + e goes to place 8j + 2a + e, so that
// a thread's results of four instructions are eight neighbouring columns, which it
// stores at once.  Sums of 32 columns at a time need few registers, and four or
// more CTAs on an SM cover each other's loads.
//
// Results' lines start on 16 bytes (others go the tiles' way).  The tiles of tcgen05
// are bound by their epilogue's instructions here: 23488 x 2432 from 2 tokens (114
// MB) take them 42 us, and this kernel 25 (4.5 TB/s).
#include "fused.cuh"

namespace mpg {
namespace {

constexpr int kGradTile = 128;
constexpr int kGradThreads = 256;
constexpr int kGradPitch = kGradTile * 2 + 16;        // bytes of a token's line: ldmatrix rows in different banks

__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void grad_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool bf16) {
  if (bf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Elements c .. c+7 of a token's line, zeros beyond `end` columns.
__device__ __forceinline__ uint4 line_chunk(const uint16_t* line, int c, int end) {
  if (!line || c >= end) return make_uint4(0, 0, 0, 0);
  if (c + 8 <= end) return ld_global(reinterpret_cast<const uint4*>(line + c));
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = c + 2 * j < end ? line[c + 2 * j] : 0, hi = c + 2 * j + 1 < end ? line[c + 2 * j + 1] : 0;
    w[j] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kSteps>                                  // of 16 tokens
__global__ void __launch_bounds__(kGradThreads) few_grad_kernel(const __grid_constant__ FewGradParams p) {
  constexpr int kTokens = 16 * kSteps;
  __shared__ __align__(16) uint8_t ds[kTokens * kGradPitch];
  __shared__ __align__(16) uint8_t xs[kTokens * kGradPitch];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int which = (int)blockIdx.z;
  const int row0 = (int)blockIdx.y * kGradTile, col0 = (int)blockIdx.x * kGradTile;
  const uint16_t* d = p.d[which];
  const Scale sc = warp_scale(p.scale, p.scale_count, p.scale_exp, p.scale_largest != 0);
  const bool bf16 = p.bf16 != 0;
  for (int i = threadIdx.x; i < kTokens * (kGradTile / 8); i += kGradThreads) {
    const int t = i / (kGradTile / 8), c = i % (kGradTile / 8) * 8;
    const bool in = t < p.tokens;
    const uint4 a = line_chunk(in ? d + (int64_t)t * p.ldd : nullptr, row0 + c, p.rows);
    const uint4 b = line_chunk(in ? p.x + (int64_t)t * p.ldx : nullptr, col0 + c, p.cols);
    const uint32_t da = smem_addr(ds) + t * kGradPitch + c * 2;
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(da), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w) : "memory");
    // (chunk a of a group of 32 columns: pair j to place 8 j + 2 a)
    const uint32_t xa = smem_addr(xs) + t * kGradPitch + ((c & ~31) + (c & 31) / 8 * 2) * 2;
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("st.shared.u32 [%0], %1;" ::"r"(xa + j * 16), "r"(w[j]) : "memory");
  }
  __syncthreads();
  // D's fragments: rows 16 warp .., all tokens.  Lanes 0-7 address tokens 0-7 of rows
  // 0-7, 8-15 of rows 8-15, 16-23 tokens 8-15 of rows 0-7, 24-31 of rows 8-15.
  uint32_t a[kSteps][4];
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    ldmatrix_trans(a[s], smem_addr(ds) + (16 * s + (lane & 7) + (lane >> 4) * 8) * kGradPitch + (16 * warp + (lane >> 3 & 1) * 8) * 2);
  const int g = lane >> 2, tig = lane & 3;
  uint16_t* out = static_cast<uint16_t*>(p.out[which]);
#pragma unroll 1
  for (int n = 0; n < kGradTile; n += 32) {
    if (col0 + n >= p.cols) break;
    float c[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[j][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        // X's fragments of two instructions: tokens 0-7 and 8-15 of places 8 j .., then of 8 (j + 1) ..
        uint32_t b[4];
        ldmatrix_trans(b, smem_addr(xs) + (16 * s + (lane & 15)) * kGradPitch + (n + 8 * (j + (lane >> 4))) * 2);
        grad_mma(c[j], a[s], b[0], b[1], bf16);
        grad_mma(c[j + 1], a[s], b[2], b[3], bf16);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = row0 + 16 * warp + g + 8 * h, col = col0 + n + 8 * tig;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack16(sc.inv * c[j][2 * h], sc.inv * c[j][2 * h + 1], bf16);
      const int left = row < p.rows ? p.cols - col : 0;
      uint16_t* to = out + (int64_t)row * p.ldo[which] + col;
      if (left >= 8) {
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < left) to[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

}  // namespace

cudaError_t launch_few_grad(const FewGradParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.cols + kGradTile - 1) / kGradTile), (unsigned)((p.rows + kGradTile - 1) / kGradTile), (unsigned)p.count);
  cfg.blockDim = dim3(kGradThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  if (p.tokens <= 16) return cudaLaunchKernelEx(&cfg, few_grad_kernel<1>, p);
  if (p.tokens <= 32) return cudaLaunchKernelEx(&cfg, few_grad_kernel<2>, p);
  return cudaLaunchKernelEx(&cfg, few_grad_kernel<4>, p);
}

}  // namespace mpg
