// Device pieces shared by the products with fused epilogues and the kernels
// around them: activations, 16-bit packing, the power-of-two scale of fp16
// gradients, targets.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fused.h"
#include "ptx.cuh"

namespace mpg {

enum : int { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2 };

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-x): 0 far below 0, where e^-x is infinite.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-kLog2e * x)); }

// Standard normal distribution function, (1 + erf(x / sqrt 2)) / 2, by erfc, which
// keeps its relative precision far below 0.
__device__ __forceinline__ float normal_cdf(float x) { return 0.5f * erfcf(x * -0.70710678118654752f); }

// act(x), and with it act'(x).
//   silu       x s(x), s(x) = 1 / (1 + e^-x);        s (1 + x (1 - s))
//   gelu       x P(x), P the normal distribution;    P + x e^(-x^2/2) / sqrt(2 pi)
//   gelu_tanh  x s(2 z), z = sqrt(2/pi) (x + 0.044715 x^3), as (1 + tanh z) / 2 = s(2 z);
//              s + 2 x s (1 - s) z'
__device__ __forceinline__ float act_value(float x, int act) {
  if (act == kActSilu) return x * sigmoid(x);
  if (act == kActGelu) return x * normal_cdf(x);
  const float c = fminf(fmaxf(x, -64.0f), 64.0f);         // (s is 0 or 1 beyond)
  return x * sigmoid(2.0f * 0.79788456080286536f * c * fmaf(0.044715f * c, c, 1.0f));
}
__device__ __forceinline__ void act_both(float x, int act, float& a, float& d) {
  if (act == kActSilu) {
    const float s = sigmoid(x);
    a = x * s;
    d = fmaf(a, 1.0f - s, s);
  } else if (act == kActGelu) {
    const float c = normal_cdf(x);
    a = x * c;
    d = fmaf(x * 0.39894228040143268f, ex2(-0.5f * kLog2e * x * x), c);
  } else {
    // (s is 0 or 1 beyond +-64, where x^2 may not fit)
    const float c = fminf(fmaxf(x, -64.0f), 64.0f), x2 = 0.044715f * c * c;
    const float s = sigmoid(2.0f * 0.79788456080286536f * c * (1.0f + x2));
    a = x * s;
    d = fmaf(2.0f * 0.79788456080286536f * a * (1.0f - s), fmaf(3.0f, x2, 1.0f), s);
  }
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  uint32_t r;
  if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack16(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
__device__ __forceinline__ float load16(const void* base, int64_t idx, bool bf16) {
  const uint16_t w = reinterpret_cast<const uint16_t*>(base)[idx];
  return bf16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
}

// Eight 16-bit elements from element `shift` (0 .. 7) of two neighbouring words on.
__device__ __forceinline__ uint4 shift_words(const uint4& a, const uint4& b, int shift) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t t[5], r[4];
  // by whole registers (shift / 2, in two steps), then by half of one
#pragma unroll
  for (int j = 0; j < 5; ++j) {
    const uint32_t lo = shift & 4 ? w[j + 2 < 8 ? j + 2 : 7] : w[j];
    const uint32_t hi = shift & 4 ? w[j + 3 < 8 ? j + 3 : 7] : w[j + 1];
    t[j] = shift & 2 ? hi : lo;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = shift & 1 ? __funnelshift_r(t[j], t[j + 1], 16) : t[j];
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The class of a token: -1 where it is ignored, -2 where it is no class.
__device__ __forceinline__ int64_t target_of(const void* target, int bytes, int64_t stride, int64_t ignore, int64_t vocab,
                                             int64_t row) {
  const int64_t t = bytes == 8 ? static_cast<const int64_t*>(target)[row * stride]
                               : (int64_t) static_cast<const int32_t*>(target)[row * stride];
  return t == ignore ? -1 : t < 0 || t >= vocab ? -2 : t;
}

// The power of two that brings the largest of a tensor's absolute values to
// [2^exp, 2^(exp+1)), and its inverse; 1 where the largest is 0 or not finite.
// Gradients in fp16 are multiplied by it before they are rounded for the
// tensor cores, and the products by the inverse: fp16 has 5 bits of exponent,
// and a gradient of a mean over thousands of tokens leaves them.
struct Pow2 {
  float mul, inv;
};
__device__ __forceinline__ Pow2 scale_pow2(float largest, int exp) {
  if (!(largest > 0.0f) || largest > 3.0e38f) return Pow2{1.0f, 1.0f};
  int e = exp - (ilogbf(largest));
  e = e > 126 ? 126 : e < -126 ? -126 : e;
  return Pow2{__uint_as_float((uint32_t)(127 + e) << 23), __uint_as_float((uint32_t)(127 - e) << 23)};
}
// By a whole warp, after griddep_wait.
__device__ __forceinline__ Pow2 warp_scale(const float* partial, int exp) {
  if (!partial) return Pow2{1.0f, 1.0f};
  float x = 0.0f;
  for (int i = threadIdx.x & 31; i < kScaleBlocks; i += 32) x = fmaxf(x, ld_global(partial + i));
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return scale_pow2(x, exp);
}

}  // namespace mpg
