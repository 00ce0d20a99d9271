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

// Codes of what a bf16 layer keeps for its gradients, act(gate) and up act'(gate):
// sign, 6 bits of exponent (bias 31), 9 of fraction, subnormals down to 2^-39,
// infinity and NaN above 2^32.  Their rounding is a quarter of bf16's, so that the
// gradients are off by the two roundings that any 16-bit product has, of its operand
// and its result (with gate and up kept in bf16 0.0031 of the norm instead of 0.0024
// at 8192 x 4096 x 11008), and their range is far beyond fp16's, which an activation
// may leave.
__device__ __forceinline__ uint32_t encode_kept(float x) {
  const uint32_t b = __float_as_uint(fabsf(x) * 0x1p-96f);        // the exponent's bias, subnormals too
  const uint32_t c = min((b + 0x1fffu + ((b >> 14) & 1u)) >> 14, 0x7e00u);
  return (x != x ? 0x7fffu : c) | (__float_as_uint(x) >> 16 & 0x8000u);
}
__device__ __forceinline__ float decode_kept(uint32_t w) {
  const uint32_t c = w & 0x7fffu;
  const float x = __uint_as_float(c << 14) * 0x1p96f;
  return __uint_as_float((c >= 0x7e00u ? 0x7f800000u | (c & 0x1ffu) << 14 : __float_as_uint(x)) | (w & 0x8000u) << 16);
}
__device__ __forceinline__ uint32_t pack_kept(float lo, float hi, bool bf16) {
  return bf16 ? encode_kept(lo) | encode_kept(hi) << 16 : pack16(lo, hi, false);
}
__device__ __forceinline__ float2 unpack_kept(uint32_t w, bool bf16) {
  return bf16 ? make_float2(decode_kept(w & 0xffffu), decode_kept(w >> 16)) : unpack16(w, false);
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

// The scale of gradients that are rounded to 16 bits for the tensor cores: they
// are divided by `div` and multiplied by `mul` before, and the products by `inv`.
// fp16 has 5 bits of exponent, and a gradient of a mean over thousands of tokens
// leaves them.
//   by a power of two  the largest of the tensor's absolute values comes to
//                      [2^exp, 2^(exp+1));
//   by the largest     it comes to 2^exp: where all tokens weigh the same, their
//                      weight is then exact, and not off by one rounding in all of
//                      them at once (half a step of bf16 in the whole gradient).
// 1 where the largest is 0 or not finite.
//
// The gradients of gate and up are dY times what may be far above 1 (channels in
// which gate and up are large together) or below.  They are made with the scale of dY
// alone first, and the largest of them is kept in `record` (kTopParts parts, of
// finite values): where it does not fit into fp16, or all of them are small, the
// scale brings it to [2^14, 2^15) instead, and the launch that made them is done `again`.
// As a rule that launch finds that they fit, and ends.  It leaves what the products
// are multiplied by behind the parts, for those that come after it.
struct Scale {
  float div, mul, inv;
};
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ int scale_exponent(int e) { return e > 126 ? 126 : e < -126 ? -126 : e; }
__device__ __forceinline__ Scale make_scale(float largest, int exp, bool by_largest, int more) {
  const bool none = !(largest > 0.0f) || largest > 3.0e38f;
  if (by_largest) return none ? Scale{1.0f, 1.0f, 1.0f} : Scale{largest, pow2(exp), largest * pow2(-exp)};
  const int e = scale_exponent((none ? 0 : scale_exponent(exp - ilogbf(largest))) + more);
  return Scale{1.0f, pow2(e), pow2(-e)};
}
__device__ __forceinline__ float warp_largest(const float* partial, int count) {
  float x = 0.0f;
  for (int i = threadIdx.x & 31; i < count; i += 32) x = fmaxf(x, fabsf(ld_global(partial + i)));
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// By a whole warp, after griddep_wait, as what follows.
__device__ __forceinline__ Scale warp_scale(const float* partial, int count, int exp, bool by_largest, int more = 0) {
  if (!partial) return Scale{1.0f, 1.0f, 1.0f};
  return make_scale(warp_largest(partial, count), exp, by_largest, more);
}
// The gradients' largest.  `more`: what it adds to the exponent of the scale that they were
// made with: nothing from 2^-4 (the smallest normal number is 2^-10 of that) to fp16's largest.
struct GradTop {
  static __device__ __forceinline__ int more(const float* top) {
    const float x = warp_largest(top, kTopParts);
    return x == 0.0f || (x >= 0.0625f && x <= 65504.0f) ? 0 : 14 - ilogbf(x);
  }
  // A launch that may be the second: whether its work is to be done (the same in all of its threads).
  // `first`: one of its warps, which leaves the products' factor.
  template <class P>
  static __device__ __forceinline__ bool needed(const P& p, bool first) {
    if (!p.again) return true;
    const int m = more(p.again);
    if (first) {
      const float inv = warp_scale(p.scale, p.scale_count, p.scale_exp, false, m).inv;
      if ((threadIdx.x & 31) == 0) p.again[kTopParts] = inv;
    }
    return m != 0;
  }
  template <class P>
  static __device__ __forceinline__ Scale scale(const P& p) {
    return warp_scale(p.scale, p.scale_count, p.scale_exp, false, p.again ? more(p.again) : 0);
  }
  // The largest of a warp's gradients (none below 0, so that their bits are in the same
  // order), into one of the parts.
  static __device__ __forceinline__ void record(float* top, int part, float x) {
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(x));
    uint32_t* to = reinterpret_cast<uint32_t*>(top) + part % kTopParts;
    if ((threadIdx.x & 31) == 0 && bits > ld_global(to)) atomicMax(to, bits);
  }
};
__device__ __forceinline__ float largest_finite(float top, float x) {
  x = fabsf(x);
  return x < INFINITY ? fmaxf(top, x) : top;
}

}  // namespace mpg
