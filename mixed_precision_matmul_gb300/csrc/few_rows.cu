// Products of few rows (a token or a few dozen being decoded or scored): the
// weights are read once, and their bytes are all that counts (sm_103a).
//
// Weight lines are the M side of mma.sync m16n8k16 and the rows of X its N
// side, eight at a time, so that nothing but X is padded.  A strip is 16 lines:
// 8 of Wg and the same 8 of Wu (gated; c0, c1 of a thread are gates and c2, c3
// the same elements' ups), or 16 classes of a vocabulary.  The order of k inside
// a sum is free, so a thread takes 16 contiguous bytes of a line as its values
// of two instructions, and the same bytes of X's rows: fragments come straight
// from global memory, without shared memory between.
//
// Eight warps take the 64-wide chunks of k in turn and their sums meet in
// shared memory.  A CTA has one strip (two with more than 16 rows, where X's
// bytes from L2 would count), and CTAs of other strips on the SM cover its way
// in and out.
#include "fused.cuh"

namespace mpg {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void mma_sync(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, bool bf16) {
  if (bf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Elements k .. k+7 of a line (0 beyond the line's end; null: none).
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* line, int k, int end) {
  if (!line || k >= end) return make_uint4(0, 0, 0, 0);
  if (kVec && k + 8 <= end) return ld_global(reinterpret_cast<const uint4*>(line + k));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = k + 2 * i < end ? line[k + 2 * i] : 0, hi = k + 2 * i + 1 < end ? line[k + 2 * i + 1] : 0;
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kGated, int kNt, bool kVec>
__global__ void __launch_bounds__(kWarps * 32) few_rows_kernel(const __grid_constant__ FewRowsParams p) {
  constexpr int kStrips = kNt > 2 ? 2 : 1;
  constexpr int kTokens = 8 * kNt;
  constexpr int kLines = (kGated ? 8 : 16) * kStrips;          // elements of a row of the result
  __shared__ float red[kWarps][kStrips * 16][kTokens + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
  const int first = (int)blockIdx.x * kLines;
  const bool bf16 = p.bf16 != 0;

  const uint16_t* lo[kStrips];
  const uint16_t* hi[kStrips];
#pragma unroll
  for (int s = 0; s < kStrips; ++s) {
    const int a = first + s * (kGated ? 8 : 16) + g, b = kGated ? a : a + 8;
    lo[s] = a < p.n ? static_cast<const uint16_t*>(p.w) + (int64_t)a * p.ldw : nullptr;
    hi[s] = b >= p.n ? nullptr
            : kGated ? static_cast<const uint16_t*>(p.wu) + (int64_t)b * p.ldwu
                     : static_cast<const uint16_t*>(p.w) + (int64_t)b * p.ldw;
  }
  const uint16_t* xr[kNt];
#pragma unroll
  for (int i = 0; i < kNt; ++i)
    xr[i] = 8 * i + g < p.rows ? static_cast<const uint16_t*>(p.x) + (int64_t)(8 * i + g) * p.ldx : nullptr;

  float c[kStrips][kNt][4];
#pragma unroll
  for (int s = 0; s < kStrips; ++s)
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[s][i][j] = 0.0f;

  // chunks of 64 of k; two at a time, so that each thread has eight loads of weights on their way
  constexpr int kAtOnce = 2;
  for (int k0 = warp * 64; k0 < p.k; k0 += kWarps * 64 * kAtOnce) {
    uint4 a[kAtOnce][2][kStrips], b[kAtOnce][2][kStrips];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s = 0; s < kStrips; ++s) {
          const int k = k0 + u * kWarps * 64 + h * 32 + tig * 8;
          a[u][h][s] = load8<kVec>(lo[s], k, p.k);
          b[u][h][s] = load8<kVec>(hi[s], k, p.k);
        }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + u * kWarps * 64 + h * 32 + tig * 8;
#pragma unroll
        for (int i = 0; i < kNt; ++i) {
          const uint4 x = load8<kVec>(xr[i], k, p.k);
#pragma unroll
          for (int s = 0; s < kStrips; ++s) {
            mma_sync(c[s][i], a[u][h][s].x, b[u][h][s].x, a[u][h][s].y, b[u][h][s].y, x.x, x.y, bf16);
            mma_sync(c[s][i], a[u][h][s].z, b[u][h][s].z, a[u][h][s].w, b[u][h][s].w, x.z, x.w, bf16);
          }
        }
      }
  }
#pragma unroll
  for (int s = 0; s < kStrips; ++s)
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[warp][s * 16 + g + 8 * (j >> 1)][8 * i + 2 * tig + (j & 1)] = c[s][i][j];
  __syncthreads();

  if constexpr (kGated) {
    for (int e = threadIdx.x; e < kLines * kTokens; e += kWarps * 32) {
      const int j = e % kLines, t = e / kLines;
      const int line = (j >> 3) * 16 + (j & 7);
      float gt = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gt += red[w][line][t];
        up += red[w][line + 8][t];
      }
      if (t < p.rows && first + j < p.n) {
        auto store = [&](void* base, int64_t ld, float v) {
          static_cast<uint16_t*>(base)[(int64_t)t * ld + first + j] = (uint16_t)pack16(v, 0.0f, bf16);
        };
        store(p.y, p.ldy, act_value(gt, p.act) * up);
        if (p.g) {
          store(p.g, p.ldg, gt);
          store(p.u, p.ldu, up);
        }
      }
    }
  } else {
    for (int e = threadIdx.x; e < kLines * kTokens; e += kWarps * 32) {
      const int j = e % kLines, t = e / kLines;
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l += red[w][j][t];
      red[0][j][t] = l;
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < p.rows) {
      const int64_t target = target_of(p.target, p.target_bytes, p.target_stride, p.ignore_index, p.n, t);
      if (target >= first && target < first + kLines) p.target_logit[t] = red[0][(int)(target - first)][t];
      float top = -INFINITY, sum = 0.0f;
      bool nan = false;
      for (int j = 0; j < kLines && first + j < p.n; ++j) {
        const float l = kLog2e * red[0][j][t];
        nan = nan || l != l;
        top = fmaxf(top, l);
      }
      const float b = fabsf(top) == INFINITY ? 0.0f : top;
      for (int j = 0; j < kLines && first + j < p.n; ++j) sum += ex2(kLog2e * red[0][j][t] - b);
      p.stats[(int64_t)blockIdx.x * p.rows + t] = make_float2(top, nan ? NAN : top == -INFINITY ? 0.0f : sum);
    }
  }
}

template <bool kGated, int kNt>
cudaError_t launch(const FewRowsParams& p, cudaLaunchConfig_t& cfg) {
  constexpr int kLines = (kGated ? 8 : 16) * (kNt > 2 ? 2 : 1);
  cfg.gridDim = dim3((unsigned)((p.n + kLines - 1) / kLines));
  return p.vec ? cudaLaunchKernelEx(&cfg, few_rows_kernel<kGated, kNt, true>, p)
               : cudaLaunchKernelEx(&cfg, few_rows_kernel<kGated, kNt, false>, p);
}

}  // namespace

int few_rows_parts(int rows, int64_t n) {
  const int lines = rows > 16 ? 32 : 16;
  return (int)((n + lines - 1) / lines);
}

cudaError_t launch_few_rows(const FewRowsParams& p, bool gated, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  if (p.rows <= 8) return gated ? launch<true, 1>(p, cfg) : launch<false, 1>(p, cfg);
  if (p.rows <= 16) return gated ? launch<true, 2>(p, cfg) : launch<false, 2>(p, cfg);
  return gated ? launch<true, 4>(p, cfg) : launch<false, 4>(p, cfg);
}

}  // namespace mpg
