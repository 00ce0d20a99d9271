// The norm of many gradients and their scaling by it (sm_103a), and the C entry.
//
//   norm = sqrt(sum over all tensors of g^2),  out = g * min(1, max_norm / (norm + eps))
//
// Two passes over the gradients, bound by memory: 2 reads and a write of each
// (the norm has to be known before the first element is scaled).  The second
// pass walks them backwards, so that what the first one read last is still in
// L2 (129 MB).  Tensors are cut into chunks, numbered through over all of them,
// and a block takes a run of chunks; a launch's parameters hold the table of its
// tensors.  A thread has four loads of eight elements on their way.  1.0e9 bf16
// gradients take 278 us for the norm (7.3 TB/s) and 622 for the scaling (6.5).
//
// Squares: a thread sums 32 in fp32 (four sums of eight, then two additions: off by
// 10 * 2^-24 at most, so the norm by 5 * 2^-24, and 6 with its own rounding) and
// carries the sums in 64 bits (a sum of eight at a time was bound by the 64-bit
// adder: 1.0e9 bf16 gradients 483 us).
// fp32 cannot hold the square of what is below 2^-63 or above 2^64; elements
// whose sum leaves [2^-90, 2^120] are squared in 64 bits instead (all zeros
// apart, which need no sum).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "fused.cuh"
#include "outio.cuh"

namespace mpg {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipStep = kClipThreads * 8;       // elements that a block loads at once
constexpr int kClipBatch = 4;                     // such loads on their way
constexpr int kClipBlocks = 608;                  // 4 to an SM
struct ClipTensor {
  const void* g;
  void* out;
  int64_t count;
  uint32_t first;                      // number of its first chunk in this launch
  uint8_t g_type, out_type, vec, same; // same: out is g
};
template <int kMost>
struct ClipParams {
  double* partial;                     // one of each block of each launch of the first pass
  int32_t partials;                    // all of them
  int32_t count;
  uint32_t chunks;
  int32_t chunk;                       // elements of a chunk
  float max_norm, eps;
  float* norm;                         // written by this launch, or null
  ClipTensor tensor[kMost];
};
constexpr int kClipFew = 64, kClipMany = 896;
static_assert(sizeof(ClipParams<kClipMany>) <= 32764, "kernel parameters");

// The tensor of a chunk.
template <int kMost>
__device__ __forceinline__ int tensor_of(const ClipParams<kMost>& p, uint32_t chunk) {
  int lo = 0, hi = p.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.tensor[mid].first <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
// The first chunk of block b's run.
__device__ __forceinline__ uint32_t first_chunk(uint32_t chunks, uint32_t b, uint32_t blocks) {
  return (uint32_t)((uint64_t)chunks * b / blocks);
}

// Eight elements from i on (0 beyond the end).
__device__ __forceinline__ void load_eight(float (&v)[8], const void* base, int64_t i, int64_t count, int type, bool vec) {
  if (vec && i + 8 <= count) {
    if (type == kOutF32) {
      const uint4* at = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
      const uint4 a = ld_global(at), b = ld_global(at + 1);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    } else {
      const uint4 a = ld_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i));
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = unpack16(w[j], type == kOutBF16);
        v[2 * j] = y.x;
        v[2 * j + 1] = y.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = i + j < count ? out_load(base, i + j, type) : 0.0f;
  }
}

__device__ __forceinline__ void add_squares(const float (&v)[8], float (&a)[4]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j % 4] = fmaf(v[j], v[j], a[j % 4]);
}
__device__ __forceinline__ bool squares_hold(float s) { return s >= 8.0779357e-28f && s <= 1.329228e36f; }   // [2^-90, 2^120]
__device__ __forceinline__ void add_squares64(const float (&v)[8], double& d) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (v[j] != 0.0f) d = fma((double)v[j], (double)v[j], d);
}
__device__ __forceinline__ double squares(const float (&v)[8]) {
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  add_squares(v, a);
  const float s = (a[0] + a[1]) + (a[2] + a[3]);
  if (squares_hold(s)) return (double)s;
  double d = 0.0;
  add_squares64(v, d);
  return d;
}

__device__ __forceinline__ double block_sum(double x, double* warps) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
  for (int i = 0; i < kClipThreads / 32; ++i) x += warps[i];
  return x;
}

// Four times eight elements of a thread: raw 16-byte words on their way together.
template <int kType>
struct Batch {
  static constexpr int kWords = kType == kOutF32 ? 2 : 1;
  uint4 w[kClipBatch][kWords];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
#pragma unroll
    for (int j = 0; j < kClipBatch; ++j) {
      const uint4* at = kType == kOutF32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i + j * kClipStep)
                                         : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i + j * kClipStep);
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[j][k] = ld_global(at + k);
    }
  }
  __device__ __forceinline__ void values(int j, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t x[4] = {w[j][k].x, w[j][k].y, w[j][k].z, w[j][k].w};
#pragma unroll
      for (int l = 0; l < 4; ++l) {
        if constexpr (kType == kOutF32) {
          v[4 * k + l] = __uint_as_float(x[l]);
        } else {
          const float2 y = unpack16(x[l], kType == kOutBF16);
          v[2 * l] = y.x;
          v[2 * l + 1] = y.y;
        }
      }
    }
  }
};

// whole(i, v) for batches (eight elements from i on, eight from i + kClipStep ..)
// and f(i, v) for eight elements v from i on, of what lies in i0 .. end.
template <class W, class F>
__device__ __forceinline__ void for_chunk(const void* g, int type, bool vec, int64_t i0, int64_t end, W&& whole, F&& f) {
  int64_t i = i0 + (int64_t)threadIdx.x * 8;
  auto batches = [&](auto batch) {
    for (; i - threadIdx.x * 8 + kClipBatch * kClipStep <= end; i += kClipBatch * kClipStep) {
      batch.load(g, i);
      whole(i, batch);
    }
  };
  if (vec) {
    if (type == kOutF32) batches(Batch<kOutF32>());
    else if (type == kOutF16) batches(Batch<kOutF16>());
    else batches(Batch<kOutBF16>());
  }
  for (; i < end; i += kClipStep) {
    float v[8];
    load_eight(v, g, i, end, type, vec);
    f(i, v);
  }
}

template <int kMost>
__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ ClipParams<kMost> p) {
  __shared__ double warps[kClipThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  double sum = 0.0;
  uint32_t c = first_chunk(p.chunks, blockIdx.x, gridDim.x);
  const uint32_t last = first_chunk(p.chunks, blockIdx.x + 1, gridDim.x);
  for (int k = tensor_of(p, c); c < last; ++k) {
    const ClipTensor& t = p.tensor[k];
    const uint32_t next = k + 1 < p.count ? min(last, p.tensor[k + 1].first) : last;
    for_chunk(t.g, t.g_type, t.vec & 1, (int64_t)(c - t.first) * p.chunk, min(t.count, (int64_t)(next - t.first) * p.chunk),
              [&](int64_t, const auto& batch) {
                float v[8], a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < kClipBatch; ++j) {
                  batch.values(j, v);
                  add_squares(v, a);
                }
                const float s = (a[0] + a[1]) + (a[2] + a[3]);
                if (squares_hold(s)) {
                  sum += (double)s;
                  return;
                }
#pragma unroll
                for (int j = 0; j < kClipBatch; ++j) {
                  batch.values(j, v);
                  add_squares64(v, sum);
                }
              },
              [&](int64_t, const float (&v)[8]) { sum += squares(v); });
    c = next;
  }
  sum = block_sum(sum, warps);
  if (threadIdx.x == 0) p.partial[blockIdx.x] = sum;
}

template <int kMost>
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ ClipParams<kMost> p) {
  __shared__ double warps[kClipThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  // every block adds all partial sums, in the same order
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.partials; i += kClipThreads) sum += *(volatile const double*)(p.partial + i);
  sum = block_sum(sum, warps);
  const float norm = (float)sqrt(sum);
  if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = norm;
  float f = p.max_norm / (norm + p.eps);
  if (f >= 1.0f || p.max_norm == INFINITY) f = 1.0f;        // (a NaN stays)
  const uint32_t first = first_chunk(p.chunks, blockIdx.x, gridDim.x);
  uint32_t c = first_chunk(p.chunks, blockIdx.x + 1, gridDim.x);
  if (first == c) return;
  // the run backwards: chunks of the batch's length
  for (int k = tensor_of(p, c - 1); c > first; --k) {
    const ClipTensor& t = p.tensor[k];
    const void* g = t.g;
    void* out = t.out;
    const int type = t.g_type, out_type = t.out_type;
    const bool vec = t.vec & 1, out_vec = t.vec & 2;
    const int64_t count = t.count;
    const uint32_t here = max(first, t.first);
    if (t.same && f == 1.0f) {                              // nothing changes
      c = here;
      continue;
    }
    auto store = [&](int64_t i, int64_t end, float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= f;
      if (out_vec && i + 8 <= end) {
        if (out_type == kOutF32) {
          float4* to = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
          to[0] = make_float4(v[0], v[1], v[2], v[3]);
          to[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          const bool bf16 = out_type == kOutBF16;
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i) =
              make_uint4(pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16), pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (i + j < end) out_store(out, i + j, v[j], out_type);
      }
    };
    for (; c > here; --c) {
      const int64_t i0 = (int64_t)(c - 1 - t.first) * p.chunk;
      const int64_t end = min(count, i0 + p.chunk);
      for_chunk(g, type, vec, i0, end,
                [&](int64_t i, const auto& batch) {
#pragma unroll
                  for (int j = 0; j < kClipBatch; ++j) {
                    float v[8];
                    batch.values(j, v);
                    store(i + j * kClipStep, end, v);
                  }
                },
                [&](int64_t i, float (&v)[8]) { store(i, end, v); });
    }
  }
}

template <class P>
cudaError_t launch(void (*kernel)(P), unsigned blocks, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kClipThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

int type_bytes(int t) { return t == MPG_F32 ? 4 : 2; }

// Elements of a chunk: a batch of loads, or with few elements one load, so that
// more blocks share them.
int chunk_for(int64_t n, const mpg_grad* grads) {
  int64_t few = (int64_t)kClipBlocks * kClipBatch * kClipStep;
  for (int64_t i = 0; i < n && few > 0; ++i) few -= grads[i].count;
  return few > 0 ? kClipStep : kClipBatch * kClipStep;
}

// Tensors that one launch takes: as many as its table holds, below 2^31 chunks.
struct Group {
  int64_t begin, end, chunks;
};
int64_t chunks_of(int64_t count, int chunk) { return (count + chunk - 1) / chunk; }
std::vector<Group> groups_of(int64_t n, const mpg_grad* grads, int chunk) {
  std::vector<Group> r;
  Group g{0, 0, 0};
  int64_t filled = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t c = chunks_of(grads[i].count, chunk);
    if (filled == kClipMany || g.chunks + c > INT32_MAX) {
      r.push_back(g);
      g = Group{i, i, 0};
      filled = 0;
    }
    g.end = i + 1;
    g.chunks += c;
    filled += c > 0;
  }
  r.push_back(g);
  return r;
}
unsigned blocks_of(const Group& g) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(g.chunks, kClipBlocks)); }

template <int kMost>
void fill(ClipParams<kMost>& p, const mpg_grad* grads, const Group& g, int chunk) {
  p.count = 0;
  p.chunk = chunk;
  uint32_t at = 0;
  for (int64_t i = g.begin; i < g.end; ++i) {
    const mpg_grad& x = grads[i];
    if (!x.count) continue;
    ClipTensor& t = p.tensor[p.count++];
    t.g = x.g;
    t.out = x.out;
    t.count = x.count;
    t.first = at;
    t.g_type = (uint8_t)x.g_dtype;
    t.out_type = (uint8_t)x.out_dtype;
    t.vec = (uint8_t)((fused_aligned(x.g, 16) ? 1 : 0) | (fused_aligned(x.out, 16) ? 2 : 0));
    t.same = x.g == x.out;
    at += (uint32_t)chunks_of(x.count, chunk);
  }
  p.chunks = at;
}

template <int kMost>
cudaError_t run(int64_t n, const mpg_grad* grads, const std::vector<Group>& groups, int chunk, float max_norm, float eps,
                float* norm, double* partial, cudaStream_t stream) {
  // (the table is a launch's parameter: 32 KB of it stay off the caller's stack)
  static thread_local ClipParams<kMost> p;
  int32_t partials = 0;
  for (const Group& g : groups) {
    fill(p, grads, g, chunk);
    p.partial = partial + partials;
    const unsigned blocks = blocks_of(g);
    partials += (int32_t)blocks;
    const cudaError_t e = launch(clip_norm_kernel<kMost>, blocks, p, stream);
    if (e != cudaSuccess) return e;
  }
  p.partial = partial;
  p.partials = partials;
  p.max_norm = max_norm;
  p.eps = eps;
  for (size_t i = groups.size(); i-- > 0;) {
    if (groups.size() > 1) fill(p, grads, groups[i], chunk);
    p.norm = i == 0 ? norm : nullptr;
    const cudaError_t e = launch(clip_scale_kernel<kMost>, blocks_of(groups[i]), p, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

mpg_status check(int64_t n, const mpg_grad* grads) {
  if (n < 0) return fail(MPG_ERR_INVALID_ARG, "negative number of gradients");
  if (n > (1 << 20)) return fail(MPG_ERR_INVALID_ARG, "more than 2^20 gradients");
  if (n && !grads) return fail(MPG_ERR_INVALID_ARG, "NULL gradients");
  for (int64_t i = 0; i < n; ++i) {
    const mpg_grad& x = grads[i];
    if (x.count < 0 || x.count > ((int64_t)1 << 43)) return fail(MPG_ERR_INVALID_ARG, "size of gradient %lld", (long long)i);
    if ((int)x.g_dtype < 0 || (int)x.g_dtype > 2 || (int)x.out_dtype < 0 || (int)x.out_dtype > 2)
      return fail(MPG_ERR_INVALID_ARG, "unknown dtype of gradient %lld", (long long)i);
    if (!x.count) continue;
    if (!x.g || !x.out) return fail(MPG_ERR_INVALID_ARG, "NULL gradient %lld", (long long)i);
    if (!fused_aligned(x.g, (size_t)type_bytes(x.g_dtype)) || !fused_aligned(x.out, (size_t)type_bytes(x.out_dtype)))
      return fail(MPG_ERR_INVALID_ARG, "gradient %lld is not aligned to its elements", (long long)i);
    if (x.g == x.out && x.g_dtype != x.out_dtype)
      return fail(MPG_ERR_INVALID_ARG, "gradient %lld is scaled in place into another dtype", (long long)i);
  }
  return MPG_OK;
}

// Results may stand in their own gradients' places, and nowhere else in what the call reads or writes.
mpg_status check_overlap(int64_t n, const mpg_grad* grads) {
  struct Span {
    uintptr_t begin, end;
    int64_t at;
    bool out;
  };
  static thread_local std::vector<Span> spans;
  spans.clear();
  for (int64_t i = 0; i < n; ++i) {
    const mpg_grad& x = grads[i];
    if (!x.count) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(x.g), o = reinterpret_cast<uintptr_t>(x.out);
    spans.push_back(Span{o, o + (uintptr_t)x.count * type_bytes(x.out_dtype), i, true});
    if (x.g != x.out) spans.push_back(Span{g, g + (uintptr_t)x.count * type_bytes(x.g_dtype), i, false});
  }
  auto before = [](const Span& a, const Span& b) { return a.begin < b.begin; };
  if (!std::is_sorted(spans.begin(), spans.end(), before)) std::sort(spans.begin(), spans.end(), before);
  // the furthest ends of results and of gradients so far
  uintptr_t out_end = 0, any_end = 0;
  for (const Span& s : spans) {
    if (s.begin < (s.out ? any_end : out_end))
      return fail(MPG_ERR_INVALID_ARG, "the result of a gradient overlaps another tensor (gradient %lld)", (long long)s.at);
    if (s.out) out_end = std::max(out_end, s.end);
    any_end = std::max(any_end, s.end);
  }
  return MPG_OK;
}

}  // namespace
}  // namespace mpg

using namespace mpg;

extern "C" {

// (no C++ exception leaves a C function: lists of spans and launches may not find memory)
size_t mpg_clip_grad_norm_workspace_size(int64_t n, const mpg_grad* grads) {
  t_err.clear();
  if (check(n, grads) != MPG_OK) return 0;
  try {
    size_t blocks = 0;
    for (const Group& g : groups_of(n, grads, chunk_for(n, grads))) blocks += blocks_of(g);
    return align256(blocks * sizeof(double));
  } catch (const std::bad_alloc&) {
    return 0;
  }
}

mpg_status mpg_clip_grad_norm(int64_t n, const mpg_grad* grads, float max_norm, float eps, float* norm, void* workspace,
                              size_t workspace_bytes, void* stream) {
  t_err.clear();
  mpg_status s = check(n, grads);
  if (s != MPG_OK) return s;
  if (!(max_norm >= 0.0f)) return fail(MPG_ERR_INVALID_ARG, "max_norm is negative or NaN");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MPG_ERR_INVALID_ARG, "eps is negative or not finite");
  if (!norm || !fused_aligned(norm, 4)) return fail(MPG_ERR_INVALID_ARG, "NULL or misaligned norm");
  try {
    if ((s = check_overlap(n, grads)) != MPG_OK) return s;
    const int chunk = chunk_for(n, grads);
    const std::vector<Group> groups = groups_of(n, grads, chunk);
    size_t need = 0, tensors = 0;
    for (const Group& g : groups) need += blocks_of(g);
    for (int64_t i = 0; i < n; ++i) tensors += grads[i].count > 0;
    need = align256(need * sizeof(double));
    if (!workspace || workspace_bytes < need || !fused_aligned(workspace, 16))
      return fail(MPG_ERR_WORKSPACE, "%zu workspace bytes needed (16-byte aligned), got %zu", need, workspace ? workspace_bytes : (size_t)0);
    DeviceInfo* dev = nullptr;
    if ((s = get_device(&dev)) != MPG_OK) return s;
    double* partial = static_cast<double*>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = tensors <= kClipFew ? run<kClipFew>(n, grads, groups, chunk, max_norm, eps, norm, partial, st)
                                              : run<kClipMany>(n, grads, groups, chunk, max_norm, eps, norm, partial, st);
    return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "clipping launch: %s", cudaGetErrorString(e));
  } catch (const std::bad_alloc&) {
    return fail(MPG_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"
