// Quantiser to 8 bits with a power-of-two scale for each block of 128, and the
// alignment copy of 8-bit operands (sm_103a).
//
// For a block (1 x 128 along a line, or 128 x 128) with a = max |x| over its
// finite values and M the largest value of the type (448 = 1.75 * 2^8 for
// e4m3, 57344 = 1.75 * 2^15 for e5m2), the scale is the smallest 2^t >= a / M
// with t >= -126, and 1 for a block of zeros.  In a's bits (exponent field E,
// fraction f) that is the exponent field E - 8 (e5m2: E - 15), plus one when
// f > 0x600000, i.e. when a's significand is above 1.75.  A power of two makes
// x / s exact, so each value is rounded once, to nearest even, to the 8-bit
// grid (half a step: 2^-4 relative in e4m3, 2^-3 in e5m2), and the result does
// not depend on how the division is done.  Rounding the scale itself up to a
// power of two costs at most one bit of range, none of precision.
//
// The kernel is bound by memory: x is read once, in 128 x 128 tiles held in
// registers (an 8 x 8 patch per thread), and both the row-wise and the
// transposed form come from that one read.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.h"
#include "internal.h"
#include "ptx.cuh"

namespace mpg {
namespace {

template <int kFmt>   // 0 e4m3, 1 e5m2
__device__ __forceinline__ uint32_t scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0) return 127u;
  const int e = (int)(b >> 23) - (kFmt == 0 ? 8 : 15) + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 1);
}
__device__ __forceinline__ float exponent_to_scale(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float exponent_to_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Two values to two 8-bit codes (x in the low byte).  The conversion
// saturates, and blocks are scaled so that no finite value needs it; x * 0 is
// NaN for inf and NaN, which makes both come out as NaN.
template <int kFmt>
__device__ __forceinline__ uint32_t cvt2(float x, float y, float ix, float iy) {
  const float a = fmaf(x, ix, x * 0.0f), b = fmaf(y, iy, y * 0.0f);
  uint16_t r;
  if constexpr (kFmt == 0) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  } else {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  }
  return r;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < __uint_as_float(0x7F800000u) ? a : 0.0f;   // inf and NaN do not set the scale
}

template <class XT>
__device__ __forceinline__ float to_f32(XT v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Eight consecutive elements from `src` (16-byte aligned).
template <class XT>
__device__ __forceinline__ void load8(const XT* src, float (&v)[8]) {
  if constexpr (sizeof(XT) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(src));
    const float4 b = __ldg(reinterpret_cast<const float4*>(src) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      XT lo, hi;
      const uint16_t l = (uint16_t)(w[i] & 0xFFFFu), h = (uint16_t)(w[i] >> 16);
      memcpy(&lo, &l, 2);
      memcpy(&hi, &h, 2);
      v[2 * i] = to_f32<XT>(lo);
      v[2 * i + 1] = to_f32<XT>(hi);
    }
  }
}

constexpr int kThreads = 256;

template <class XT, int kFmt, bool kTile, bool kTrans>
__global__ void __launch_bounds__(kThreads) fp8_quant_kernel(const __grid_constant__ Fp8QuantParams p) {
  __shared__ float red[8][128];                                  // column maxima of each warp / tile maxima
  __shared__ __align__(16) uint8_t tr[kTrans ? 128 * 128 : 16];  // the tile's codes, transposed
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid & 15, rg = tid >> 4;                        // columns 8cg.., rows 8rg..
  const int ncb = (p.cols + 127) / 128;
  const int rb = (int)blockIdx.x / ncb, cb = (int)blockIdx.x - rb * ncb;
  const int r0 = rb * 128, c0 = cb * 128;
  const int col = c0 + cg * 8;
  const bool full_cols = col + 8 <= p.cols;
  griddep_wait();
  griddep_launch_dependents();

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = r0 + rg * 8 + i;
    const XT* src = reinterpret_cast<const XT*>(p.x) + (int64_t)row * p.ldx + col;
    if (row < p.rows && full_cols && p.x_vec) {
      load8<XT>(src, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = (row < p.rows && col + j < p.cols) ? to_f32<XT>(src[j]) : 0.0f;
    }
  }

  uint32_t tile_exp = 127u;
  if constexpr (kTile) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(v[i][j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[0][w]);
    tile_exp = scale_exponent<kFmt>(m);
    if (tid == 0) {
      const float s = exponent_to_scale(tile_exp);
      if (p.q) p.s[(int64_t)rb * p.s_row + (int64_t)cb * p.s_k] = s;
      if (kTrans) p.st[(int64_t)cb * p.st_row + (int64_t)rb * p.st_k] = s;
    }
  }

  if (p.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = r0 + rg * 8 + i;
      float inv;
      if constexpr (kTile) {
        inv = exponent_to_inverse(tile_exp);
      } else {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, finite_abs(v[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t e = scale_exponent<kFmt>(m);
        inv = exponent_to_inverse(e);
        if (cg == 0 && row < p.rows) p.s[(int64_t)row * p.s_row + (int64_t)cb * p.s_k] = exponent_to_scale(e);
      }
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = cvt2<kFmt>(v[i][2 * j], v[i][2 * j + 1], inv, inv);
      if (row < p.rows) {
        uint8_t* dst = p.q + (int64_t)row * p.ldq + col;
        if (full_cols && p.q_vec) {
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < p.cols) dst[j] = (uint8_t)(w[j >> 1] >> (8 * (j & 1)));
        }
      }
    }
  }

  if constexpr (kTrans) {
    float inv[8];
    if constexpr (kTile) {
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = exponent_to_inverse(tile_exp);
    } else {
      // maxima of the columns: over this thread's 8 rows, the warp's 16, then the block's 128
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, finite_abs(v[i][j]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane < 16) red[warp][cg * 8 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w][cg * 8 + j]);
        const uint32_t e = scale_exponent<kFmt>(m);
        inv[j] = exponent_to_inverse(e);
        if (rg == 0 && col + j < p.cols)
          p.st[(int64_t)(col + j) * p.st_row + (int64_t)rb * p.st_k] = exponent_to_scale(e);
      }
    }
    // Line c of the transposed tile is 16 chunks of 8 bytes (one per row group);
    // chunk g is kept at slot g ^ (c / 8), so that the 16 lanes of a store
    // phase (one column of each of the 16 column groups) reach 16 slots.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = cvt2<kFmt>(v[2 * i][j], v[2 * i + 1][j], inv[j], inv[j]);
      *reinterpret_cast<uint2*>(tr + (cg * 8 + j) * 128 + ((rg ^ cg) << 3)) =
          make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = i * 32 + (tid >> 3), ch = tid & 7;            // 16 bytes: rows 16ch .. 16ch+15 of column c
      const uint2 a = *reinterpret_cast<const uint2*>(tr + c * 128 + (((2 * ch) ^ (c >> 3)) << 3));
      const uint2 b = *reinterpret_cast<const uint2*>(tr + c * 128 + (((2 * ch + 1) ^ (c >> 3)) << 3));
      const int row = r0 + ch * 16;
      if (c0 + c < p.cols && row < p.rows) {
        uint8_t* dst = p.qt + (int64_t)(c0 + c) * p.ldqt + row;
        if (p.qt_vec && row + 16 <= p.rows) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
          const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (row + j < p.rows) dst[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
}

// Each thread builds 16 bytes of an output line from the aligned 4-byte words
// that hold them (only words with at least one byte of the line are read).
__global__ void __launch_bounds__(256) fp8_align_kernel(const uint8_t* __restrict__ in, int64_t ld_in, int64_t rows,
                                                        int64_t cols, uint8_t* __restrict__ out, int64_t ld_out) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t per = ld_out / 16;
  const int64_t total = rows * per;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / per, c = (i - r * per) * 16;
    const int64_t left = cols - c;                                 // bytes of the line from here on
    uint32_t o[4] = {0, 0, 0, 0};
    if (left > 0) {
      const uint8_t* src = in + r * ld_in + c;
      const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(src) & 3u);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(src - sh);
      uint32_t x[5];
#pragma unroll
      for (int j = 0; j < 5; ++j) x[j] = (4 * j - (int64_t)sh < left && (j < 4 || sh > 0)) ? __ldg(w + j) : 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __funnelshift_r(x[j], x[j + 1], 8 * sh);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t valid = left - 4 * j;                        // bytes of this word inside the line
        if (valid <= 0) o[j] = 0;
        else if (valid < 4) o[j] &= (1u << (8 * valid)) - 1u;
      }
    }
    *reinterpret_cast<uint4*>(out + r * ld_out + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <class XT, int kFmt, bool kTile>
cudaError_t launch_form(const Fp8QuantParams& p, cudaLaunchConfig_t& cfg) {
  return p.qt ? cudaLaunchKernelEx(&cfg, fp8_quant_kernel<XT, kFmt, kTile, true>, p)
              : cudaLaunchKernelEx(&cfg, fp8_quant_kernel<XT, kFmt, kTile, false>, p);
}
template <class XT>
cudaError_t launch_type(const Fp8QuantParams& p, int format, bool tile, cudaLaunchConfig_t& cfg) {
  if (format == 0) return tile ? launch_form<XT, 0, true>(p, cfg) : launch_form<XT, 0, false>(p, cfg);
  return tile ? launch_form<XT, 1, true>(p, cfg) : launch_form<XT, 1, false>(p, cfg);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantParams& p, int x_dtype, int format, int scale_rows,
                                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((p.cols + 127) / 128) * ((p.rows + 127) / 128)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool tile = scale_rows != 1;
  switch (x_dtype) {
    case 0: return launch_type<float>(p, format, tile, cfg);
    case 1: return launch_type<__half>(p, format, tile, cfg);
    default: return launch_type<__nv_bfloat16>(p, format, tile, cfg);
  }
}

cudaError_t launch_fp8_align(const uint8_t* in, int64_t ld_in, int64_t rows, int64_t cols, uint8_t* out,
                             int64_t ld_out, int sm_count, cudaStream_t stream) {
  const int64_t total = rows * (ld_out / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)min((total + 255) / 256, (int64_t)sm_count * 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_align_kernel, in, ld_in, rows, cols, out, ld_out);
}

}  // namespace mpg
