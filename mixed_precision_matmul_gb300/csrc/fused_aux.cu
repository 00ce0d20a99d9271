// Memory-bound kernels around the products with fused epilogues (sm_103a):
// copies of operands whose lines TMA cannot describe, the largest absolute
// value behind the scale of fp16 gradients, the gradients of gate and up from
// what the forward pass kept, and the joining of a row's parts into its loss.
#include <climits>

#include "fused.cuh"

namespace mpg {
namespace {

// Chunk i of a matrix whose lines have per_line chunks of 8: its row and first column.
struct Chunk {
  int64_t row, col;
};
__device__ __forceinline__ Chunk chunk_at(int64_t i, int64_t per_line, bool small) {
  Chunk c;
  if (small) {
    const uint32_t r = (uint32_t)i / (uint32_t)per_line;
    c.row = r;
    c.col = 8 * (int64_t)((uint32_t)i - r * (uint32_t)per_line);
  } else {
    c.row = i / per_line;
    c.col = 8 * (i - c.row * per_line);
  }
  return c;
}
__device__ __forceinline__ uint4 load_chunk(const void* base, int64_t idx, int64_t left, bool vec) {
  const uint16_t* at = static_cast<const uint16_t*>(base) + idx;
  if (vec && left >= 8) return ld_global(reinterpret_cast<const uint4*>(at));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < left ? at[2 * i] : 0, hi = 2 * i + 1 < left ? at[2 * i + 1] : 0;
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Copies to lines of whole 16-byte chunks; one matrix to each row of blocks.  A
// chunk's eight elements lie in two aligned 16-byte words, which are loaded whole
// and shifted (eight loads of 2 bytes took 7.4 us for 12 MB); next to the matrix's
// ends they are read by elements, so that nothing outside it is touched.
__global__ void __launch_bounds__(256) pad_kernel(const __grid_constant__ PadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const PadParams::Matrix& m = p.mat[blockIdx.y];
  const int64_t per_line = (m.cols + 7) / 8, n = m.rows * per_line;
  const bool small = n < INT_MAX;
#pragma unroll 2
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const Chunk c = chunk_at(i, per_line, small);
    const int64_t off = c.row * m.ld_src + c.col;
    const uint16_t* at = m.src + off;
    uint4 v;
    if (off < 8 || off + 16 > (m.rows - 1) * m.ld_src + m.cols) {
      v = load_chunk(at, 0, m.cols - c.col, false);
    } else {
      const uintptr_t addr = reinterpret_cast<uintptr_t>(at);
      const uint4* word = reinterpret_cast<const uint4*>(addr & ~(uintptr_t)15);
      const int shift = (int)(addr & 15) / 2;          // elements
      v = shift_words(ld_global(word), shift ? ld_global(word + 1) : make_uint4(0, 0, 0, 0), shift);
    }
    const int64_t left = m.cols - c.col;
    if (left < 8) {
      // zeros behind the line's end
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = 2 * j >= left ? 0u : 2 * j + 1 == left ? w[j] & 0xffffu : w[j];
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(m.dst + c.row * m.ld_dst + c.col) = v;
  }
}

__device__ __forceinline__ float abs_max8(const uint4& v, bool bf16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = unpack16(w[i], bf16);
    x = fmaxf(x, fmaxf(fabsf(y.x), fabsf(y.y)));
  }
  return x;
}

__global__ void __launch_bounds__(512) max_kernel(const __grid_constant__ MaxParams p) {
  griddep_wait();
  griddep_launch_dependents();
  float x = 0.0f;
  if (p.x) {
    // (fp16: only its gradients are scaled); four loads on their way
    const int64_t per_line = (p.cols + 7) / 8, n = p.rows * per_line;
    const bool small = n < INT_MAX;
    constexpr int kAtOnce = 4;
    constexpr int64_t kStep = (int64_t)kScaleBlocks * 512;
    int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x;
    if (p.flat) {
      const uint4* at = static_cast<const uint4*>(p.x);
      for (; i + (kAtOnce - 1) * kStep < n; i += kAtOnce * kStep) {
        uint4 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) v[j] = ld_global(at + i + j * kStep);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) x = fmaxf(x, abs_max8(v[j], false));
      }
    }
    for (; i < n; i += kStep) {
      const Chunk c = chunk_at(i, per_line, small);
      x = fmaxf(x, abs_max8(load_chunk(p.x, c.row * p.ld + c.col, p.cols - c.col, p.vec != 0), false));
    }
  } else {
    for (int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x; i < p.rows; i += (int64_t)kScaleBlocks * 512)
      if (target_of(p.target, p.target_bytes, p.target_stride, p.ignore_index, INT64_MAX, i) >= 0)
        x = fmaxf(x, fabsf(ld_global(p.dloss + i * p.dloss_stride)));
  }
  __shared__ float warps[16];
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x < 32) {
    x = threadIdx.x < 16 ? warps[threadIdx.x] : 0.0f;
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (threadIdx.x == 0) p.partial[blockIdx.x] = x;
    if (threadIdx.x == 0 && p.top && blockIdx.x < kTopParts) p.top[blockIdx.x] = 0.0f;
  }
}

// Three reads and two writes of 16 bits an element: 8192 x 11008 128 us, 7.0 TB/s.
__global__ void __launch_bounds__(256) gated_grad_kernel(const __grid_constant__ GatedGradParams p) {
  griddep_wait();
  griddep_launch_dependents();
  if (!GradTop::needed(p, blockIdx.x == 0 && threadIdx.x < 32)) return;
  const bool bf16 = p.bf16 != 0, vec = p.vec != 0;
  const float s = GradTop::scale(p).mul;
  float top = 0.0f;
  const int64_t per_line = (p.cols + 7) / 8, n = p.rows * per_line;
  const bool small = n < INT_MAX;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const Chunk c = chunk_at(i, per_line, small);
    const int64_t left = p.cols - c.col;
    const uint4 y4 = load_chunk(p.dy, c.row * p.lddy + c.col, left, vec);
    const uint4 a4 = load_chunk(p.a, c.row * p.lda + c.col, left, vec);
    const uint4 b4 = load_chunk(p.b, c.row * p.ldb + c.col, left, vec);
    const uint32_t y[4] = {y4.x, y4.y, y4.z, y4.w}, a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
    uint32_t dg[4], du[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 yy = unpack16(y[j], bf16), aa = unpack_kept(a[j], bf16), bb = unpack_kept(b[j], bf16);
      const float y0 = s * yy.x, y1 = s * yy.y;
      const float g0 = y0 * bb.x, g1 = y1 * bb.y, u0 = y0 * aa.x, u1 = y1 * aa.y;
      if (p.record) top = largest_finite(largest_finite(largest_finite(largest_finite(top, g0), g1), u0), u1);
      dg[j] = pack16(g0, g1, bf16);
      du[j] = pack16(u0, u1, bf16);
    }
    // (the lines of dg and du are padded to whole chunks; what lies beyond the columns is not read)
    *reinterpret_cast<uint4*>(p.dg + c.row * p.ldd + c.col) = make_uint4(dg[0], dg[1], dg[2], dg[3]);
    *reinterpret_cast<uint4*>(p.du + c.row * p.ldd + c.col) = make_uint4(du[0], du[1], du[2], du[3]);
  }
  if (p.record) {
    // (a warp of each block: from all of them at once the atomics took longer than the reads)
    __shared__ float warps[8];
    __syncwarp();
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) GradTop::record(p.record, (int)blockIdx.x, threadIdx.x < 8 ? warps[threadIdx.x] : 0.0f);
  }
}

// Two parts of a row: maxima (in units of ln 2) and sums of 2^(l - maximum).
// A part without values is (-inf, 0); a NaN stays in the sum.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float top = fmaxf(a.x, b.x);
  if (top == -INFINITY) return make_float2(top, a.y + b.y);
  const float base = top == INFINITY ? 0.0f : top;
  return make_float2(top, a.y * ex2(a.x - base) + b.y * ex2(b.x - base));
}

constexpr int kJoinThreads = 1024;
// kRows rows a block (8: neighbouring lanes read 64 bytes of neighbouring rows).
template <int kRows>
__global__ void __launch_bounds__(kJoinThreads) loss_join_kernel(const __grid_constant__ LossJoinParams p) {
  constexpr int kPer = kJoinThreads / kRows;            // threads of a row
  __shared__ float2 part[kRows > 1 ? kPer : 32][kRows];
  griddep_wait();
  griddep_launch_dependents();
  const int r = threadIdx.x % kRows, s = threadIdx.x / kRows;
  const int64_t row = (int64_t)blockIdx.x * kRows + r;
  float2 x = make_float2(-INFINITY, 0.0f);
  if (row < p.rows) {
#pragma unroll 4
    for (int i = s; i < p.parts; i += kPer) {
      const float* at = reinterpret_cast<const float*>(p.stats + (int64_t)i * p.rows + row);
      x = join(x, make_float2(ld_global(at), ld_global(at + 1)));
    }
  }
  if constexpr (kRows == 1) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
      x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][0] = x;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    x = part[threadIdx.x][0];
#pragma unroll
    for (int o = 16; o; o >>= 1)
      x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
    if (threadIdx.x) return;
  } else {
    // pairs of threads, halving: the same order at any time
    part[s][r] = x;
    for (int w = kPer / 2; w; w >>= 1) {
      __syncthreads();
      if (s < w) part[s][r] = x = join(x, part[s + w][r]);
    }
    if (s) return;
  }
  if (row >= p.rows) return;
  const int64_t t = target_of(p.target, p.target_bytes, p.target_stride, p.ignore_index, p.vocab, row);
  float lse = 0.0f, loss = 0.0f;
  if (t == -2) {
    lse = loss = NAN;
  } else if (t >= 0) {
    // the sum of two terms and the difference that the loss is, in 64 bits: rounded once
    double l = x.y != x.y ? (double)NAN : fabsf(x.x) == INFINITY ? (double)x.x : ((double)x.x + (double)log2f(x.y)) * 0.69314718055994530942;
    lse = (float)l;
    loss = (float)(l - (double)ld_global(p.target_logit + row));
  }
  p.lse[row] = lse;
  p.loss[row] = loss;
}

template <class K, class P>
cudaError_t launch(K kernel, dim3 grid, int block, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
unsigned blocks_for(int64_t n, int64_t most) { return (unsigned)std::max<int64_t>(1, std::min((n + 255) / 256, most)); }

}  // namespace

cudaError_t launch_pad(const PadParams& p, int sm_count, cudaStream_t stream) {
  int64_t n = 0;
  for (int i = 0; i < p.count; ++i) n = std::max(n, p.mat[i].rows * ((p.mat[i].cols + 7) / 8));
  return launch(pad_kernel, dim3(blocks_for(n, 8 * (int64_t)sm_count), (unsigned)p.count), 256, p, stream);
}
cudaError_t launch_max(const MaxParams& p, cudaStream_t stream) { return launch(max_kernel, dim3(kScaleBlocks), 512, p, stream); }
cudaError_t launch_gated_grad(const GatedGradParams& p, int sm_count, cudaStream_t stream) {
  // (done again, as a rule it does nothing: fewer blocks begin and end sooner)
  return launch(gated_grad_kernel, dim3(blocks_for(p.rows * ((p.cols + 7) / 8), (p.again ? 8 : 32) * (int64_t)sm_count)), 256, p, stream);
}
cudaError_t launch_loss_join(const LossJoinParams& p, cudaStream_t stream) {
  if (p.rows <= 2 * kFewRows) return launch(loss_join_kernel<1>, dim3((unsigned)p.rows), kJoinThreads, p, stream);
  return launch(loss_join_kernel<8>, dim3((unsigned)((p.rows + 7) / 8)), kJoinThreads, p, stream);
}

}  // namespace mpg
