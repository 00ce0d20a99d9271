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
// transposed form come from that one read.  On a GB300: 8190 x 8192 bf16 in
// both directions takes 50 us, 5.4 TB/s (a plain copy: 6.8); 4096 x 11008 fp32
// in tiles 43 us, 6.3 TB/s; one row of 8192 3 us, a launch's latency.  1531 x
// 4100 fp16 takes 8.3 us where 1536 x 4096 takes 5.4: the tiles at the edges,
// whose cut patches are loaded element by element and whose lines end in single
// bytes, take 2 us longer than the others, either edge as much as both (1531 x
// 4096 7.7, 1536 x 4100 7.6 us); that lines of x start off 16 bytes costs nothing.
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

// Two values to two 8-bit codes (x in the low byte).  The conversion saturates;
// blocks are scaled so that no finite value needs it.
template <int kFmt>
__device__ __forceinline__ uint32_t cvt2(float x, float y) {
  uint16_t r;
  if constexpr (kFmt == 0) {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  } else {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  }
  return r;
}

// Both halves times a power of two each.
__device__ __forceinline__ float2 scale2(float2 v, float sx, float sy) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(v.x), "f"(v.y), "f"(sx), "f"(sy));
  return r;
}

// A thread's patch of 8 rows x 8 columns as pairs of neighbouring columns, in
// the source's own type: 16-bit pairs are compared packed, which halves the
// work of the maxima.  Maxima ignore NaN, as the hardware's do.
template <class XT>
struct Pair;
template <>
struct Pair<float> {
  using T = float2;
  static __device__ __forceinline__ T zero() { return make_float2(0.0f, 0.0f); }
  static __device__ __forceinline__ T make(const float* p, bool x, bool y) { return make_float2(x ? p[0] : 0.0f, y ? p[1] : 0.0f); }
  static __device__ __forceinline__ T abs(T a) { return make_float2(fabsf(a.x), fabsf(a.y)); }
  static __device__ __forceinline__ T max(T a, T b) { return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y)); }
  static __device__ __forceinline__ float2 wide(T a) { return a; }
  static __device__ __forceinline__ T no_inf(T a) {
    const float nan = __uint_as_float(0x7FC00000u), inf = __uint_as_float(0x7F800000u);
    return make_float2(fabsf(a.x) == inf ? nan : a.x, fabsf(a.y) == inf ? nan : a.y);
  }
};
template <>
struct Pair<__half> {
  using T = __half2;
  static __device__ __forceinline__ T zero() { return __half2half2(__ushort_as_half(0)); }
  static __device__ __forceinline__ T make(const __half* p, bool x, bool y) {
    const __half z = __ushort_as_half(0);
    return __halves2half2(x ? p[0] : z, y ? p[1] : z);
  }
  static __device__ __forceinline__ T abs(T a) { return __habs2(a); }
  static __device__ __forceinline__ T max(T a, T b) { return __hmax2(a, b); }
  static __device__ __forceinline__ float2 wide(T a) { return __half22float2(a); }
  static __device__ __forceinline__ T no_inf(T a) {
    const __half nan = __ushort_as_half(0x7FFF);
    return __halves2half2(__hisinf(__low2half(a)) ? nan : __low2half(a), __hisinf(__high2half(a)) ? nan : __high2half(a));
  }
};
template <>
struct Pair<__nv_bfloat16> {
  using T = __nv_bfloat162;
  static __device__ __forceinline__ T zero() { return __bfloat162bfloat162(__ushort_as_bfloat16(0)); }
  static __device__ __forceinline__ T make(const __nv_bfloat16* p, bool x, bool y) {
    const __nv_bfloat16 z = __ushort_as_bfloat16(0);
    return __halves2bfloat162(x ? p[0] : z, y ? p[1] : z);
  }
  static __device__ __forceinline__ T abs(T a) { return __habs2(a); }
  static __device__ __forceinline__ T max(T a, T b) { return __hmax2(a, b); }
  static __device__ __forceinline__ float2 wide(T a) { return __bfloat1622float2(a); }
  static __device__ __forceinline__ T no_inf(T a) {
    const __nv_bfloat16 nan = __ushort_as_bfloat16(0x7FFF);
    return __halves2bfloat162(__hisinf(__low2bfloat16(a)) ? nan : __low2bfloat16(a),
                              __hisinf(__high2bfloat16(a)) ? nan : __high2bfloat16(a));
  }
};

constexpr int kThreads = 256;

template <class XT, int kFmt, bool kTile, bool kTrans>
__global__ void __launch_bounds__(kThreads, sizeof(XT) == 2 ? 4 : 2) fp8_quant_kernel(const __grid_constant__ Fp8QuantParams p) {
  using P = Pair<XT>;
  using PT = typename P::T;
  __shared__ __align__(16) float red[8][128];                    // column maxima of each warp / tile maxima
  __shared__ __align__(16) float col_inv[128];
  __shared__ __align__(16) uint8_t tr[kTrans ? 128 * 128 : 16];  // the tile's codes, transposed
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid & 15, rg = tid >> 4;                        // columns 8cg.., rows 8rg..
  const int ncb = (p.cols + 127) / 128;
  const int rb = (int)blockIdx.x / ncb, cb = (int)blockIdx.x - rb * ncb;
  const int r0 = rb * 128, c0 = cb * 128;
  const int col = c0 + cg * 8, row0 = r0 + rg * 8;
  const bool full_cols = col + 8 <= p.cols;
  griddep_wait();
  griddep_launch_dependents();

  PT v[8][4];
  const XT* src = reinterpret_cast<const XT*>(p.x) + (int64_t)row0 * p.ldx + col;
  if (full_cols && p.x_align > (int)sizeof(XT) && row0 + 8 <= p.rows) {
    // the widest loads that the lines' alignment allows (non-coherent: an
    // ordinary launch, which starts after the kernel that wrote x)
    auto load_patch = [&](auto unit) {
      using U = decltype(unit);
      constexpr int kUnits = 8 * sizeof(XT) / sizeof(U);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        U a[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) a[u] = __ldg(reinterpret_cast<const U*>(src + i * p.ldx) + u);
        memcpy(&v[i][0], a, sizeof(a));
      }
    };
    if (p.x_align == 16) load_patch(uint4{});
    else if (p.x_align == 8) load_patch(uint2{});
    else load_patch(uint32_t{});
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[i][j] = row0 + i < p.rows
                      ? P::make(src + i * p.ldx + 2 * j, col + 2 * j < p.cols, col + 2 * j + 1 < p.cols)
                      : P::zero();
  }

  // maxima of the patch's rows and columns; infinities (found in the columns'
  // maxima) become NaN, which sets no scale and comes out as NaN
  float row_max[8];
  PT col_max[4];
  auto maxima = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) col_max[j] = P::zero();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      PT a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[j] = P::abs(v[i][j]);
        col_max[j] = P::max(col_max[j], a[j]);
      }
      const float2 m = P::wide(P::max(P::max(a[0], a[1]), P::max(a[2], a[3])));
      row_max[i] = fmaxf(fmaxf(m.x, m.y), 0.0f);                 // (0: a row of NaN)
    }
    const float2 m = P::wide(P::max(P::max(col_max[0], col_max[1]), P::max(col_max[2], col_max[3])));
    return fmaxf(fmaxf(m.x, m.y), 0.0f);
  };
  float patch_max = maxima();
  if (patch_max > 3.4028235e38f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = P::no_inf(v[i][j]);
    patch_max = maxima();
  }

  float tile_inv = 0.0f;
  if constexpr (kTile) {
    float m = patch_max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[0][w]);
    const uint32_t e = scale_exponent<kFmt>(m);
    tile_inv = exponent_to_inverse(e);
    if (tid == 0) {
      const float s = exponent_to_scale(e);
      if (p.q) p.s[(int64_t)rb * p.s_row + (int64_t)cb * p.s_k] = s;
      if (kTrans) p.st[(int64_t)cb * p.st_row + (int64_t)rb * p.st_k] = s;
    }
  } else if constexpr (kTrans) {
    // over the warp's 16 rows: each half of the lanes keeps 4 of the 8 columns
    float2 lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 mine = P::wide(lane < 16 ? col_max[j] : col_max[j + 2]);
      const float2 send = P::wide(lane < 16 ? col_max[j + 2] : col_max[j]);
      lo[j].x = fmaxf(mine.x, __shfl_xor_sync(0xffffffffu, send.x, 16));
      lo[j].y = fmaxf(mine.y, __shfl_xor_sync(0xffffffffu, send.y, 16));
    }
    *reinterpret_cast<float4*>(&red[warp][cg * 8 + (lane >> 4) * 4]) = make_float4(lo[0].x, lo[0].y, lo[1].x, lo[1].y);
    __syncthreads();
    if (tid < 128) {
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w][tid]);
      const uint32_t e = scale_exponent<kFmt>(m);
      col_inv[tid] = exponent_to_inverse(e);
      if (c0 + tid < p.cols) p.st[(int64_t)(c0 + tid) * p.st_row + (int64_t)rb * p.st_k] = exponent_to_scale(e);
    }
  }

  if (p.q) {
    float row_inv = tile_inv;
    if constexpr (!kTile) {
      // maxima over the 16 lanes of a row, each pair of lanes keeping one of
      // the 8 rows: 4 + 2 + 1 values exchanged, then the pair's
      float a[4], b[2], m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool up = lane & 8;
        a[i] = fmaxf(up ? row_max[i + 4] : row_max[i], __shfl_xor_sync(0xffffffffu, up ? row_max[i] : row_max[i + 4], 8));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool up = lane & 4;
        b[i] = fmaxf(up ? a[i + 2] : a[i], __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 4));
      }
      {
        const bool up = lane & 2;
        m = fmaxf(up ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 2));
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const int i = ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1);
      const uint32_t e = scale_exponent<kFmt>(m);
      row_inv = exponent_to_inverse(e);
      if (!(lane & 1) && row0 + i < p.rows) p.s[(int64_t)(row0 + i) * p.s_row + (int64_t)cb * p.s_k] = exponent_to_scale(e);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float inv =
          kTile ? tile_inv
                : __shfl_sync(0xffffffffu, row_inv, (lane & 16) | ((i >> 2) << 3) | (((i >> 1) & 1) << 2) | ((i & 1) << 1));
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = scale2(P::wide(v[i][j]), inv, inv);
        w[j] = cvt2<kFmt>(x.x, x.y);
      }
      if (row0 + i < p.rows) {
        uint8_t* dst = p.q + (int64_t)(row0 + i) * p.ldq + col;
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
    if constexpr (!kTile) {
      __syncthreads();
      const float4 a = *reinterpret_cast<const float4*>(&col_inv[cg * 8]);
      const float4 b = *reinterpret_cast<const float4*>(&col_inv[cg * 8 + 4]);
      inv[0] = a.x; inv[1] = a.y; inv[2] = a.z; inv[3] = a.w;
      inv[4] = b.x; inv[5] = b.y; inv[6] = b.z; inv[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) inv[j] = tile_inv;
    }
    // Line c of the transposed tile is 16 chunks of 8 bytes (one per row group);
    // chunk g is kept at slot g ^ (c / 8), so that the 16 lanes of a store
    // phase (one column of each of the 16 column groups) reach 16 slots.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w0[4], w1[4];                                     // columns 2j and 2j + 1
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = scale2(P::wide(v[2 * i][j]), inv[2 * j], inv[2 * j + 1]);
        const float2 b = scale2(P::wide(v[2 * i + 1][j]), inv[2 * j], inv[2 * j + 1]);
        w0[i] = cvt2<kFmt>(a.x, b.x);
        w1[i] = cvt2<kFmt>(a.y, b.y);
      }
      uint8_t* line = tr + (cg * 8 + 2 * j) * 128 + ((rg ^ cg) << 3);
      *reinterpret_cast<uint2*>(line) = make_uint2(w0[0] | (w0[1] << 16), w0[2] | (w0[3] << 16));
      *reinterpret_cast<uint2*>(line + 128) = make_uint2(w1[0] | (w1[1] << 16), w1[2] | (w1[3] << 16));
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
// One launch copies one or two operands.
__global__ void __launch_bounds__(256) fp8_align_kernel(const __grid_constant__ Fp8AlignJob ja,
                                                        const __grid_constant__ Fp8AlignJob jb) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t ta = ja.rows * ja.chunks, total = ta + jb.rows * jb.chunks;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const Fp8AlignJob& j = i < ta ? ja : jb;
    const int64_t k = i < ta ? i : i - ta;
    int64_t r, ch;
    if (total < (int64_t(1) << 31)) {                              // (64-bit division is a long routine)
      r = (uint32_t)k / (uint32_t)j.chunks;
      ch = (uint32_t)k - (uint32_t)r * (uint32_t)j.chunks;
    } else {
      r = k / j.chunks;
      ch = k - r * j.chunks;
    }
    const int64_t c = ch * 16;
    const int64_t left = j.cols - c;                               // bytes of the line from here on (>= 1)
    const uint8_t* src = j.in + r * j.ld_in + c;
    const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(src) & 3u);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(src - sh);
    uint32_t x[5], o[4];
#pragma unroll
    for (int n = 0; n < 5; ++n) x[n] = (4 * n - (int64_t)sh < left && (n < 4 || sh > 0)) ? ld_global(w + n) : 0u;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      o[n] = __funnelshift_r(x[n], x[n + 1], 8 * sh);
      const int64_t valid = left - 4 * n;                          // bytes of this word inside the line
      if (valid <= 0) o[n] = 0;
      else if (valid < 4) o[n] &= (1u << (8 * valid)) - 1u;
    }
    *reinterpret_cast<uint4*>(j.out + r * j.ld_out + c) = make_uint4(o[0], o[1], o[2], o[3]);
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
  // (an ordinary launch: as a programmatic dependent it costs the host 2.4 us
  // more, of 14 a call)
  cfg.stream = stream;
  const bool tile = scale_rows != 1;
  switch (x_dtype) {
    case 0: return launch_type<float>(p, format, tile, cfg);
    case 1: return launch_type<__half>(p, format, tile, cfg);
    default: return launch_type<__nv_bfloat16>(p, format, tile, cfg);
  }
}

cudaError_t launch_fp8_align(const Fp8AlignJob& a, const Fp8AlignJob& b, int sm_count, cudaStream_t stream) {
  const int64_t total = a.rows * a.chunks + b.rows * b.chunks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)min((total + 255) / 256, (int64_t)sm_count * 16));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_align_kernel, a, b);
}

}  // namespace mpg
