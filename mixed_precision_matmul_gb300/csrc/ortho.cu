// Kernels of the orthogonalised update (sm_103a): X <- a X + (b S + c S S) X
// with S = X X^T, from X = G / (|G| + eps).
//
// Numbers.  The products run on the tensor cores in fp16 with fp32
// accumulation.  Every matrix of the iteration has singular values up to
// about 1.2, so fp16's 11 bits can be used without fear of its range: X is
// stored times a power of two near the root of its longer side (its entries
// then have a root mean square near 1 when X is orthogonal), S and b S + c S S
// as they are.  Where |G| is far below eps the iterates start that small and
// grow by |a| a step: a bound on their norm, |G| / (|G| + eps) taken through the
// polynomial's absolute values, gives each matrix and step a power of two of
// its own beside that one, as long as the bound is below 1.  bf16 storage would lose three bits at every rounding; rounding
// errors of X grow by up to a = 3.4 a step in the directions of small singular
// values.  With five steps on a matrix of noise and a few strong directions
// the result is off by 1.3e-3 of its norm with fp16 storage and by 1.1e-2 with
// bf16 (the rounding to a bf16 result alone is 1.7e-3).  G itself enters
// scaled by a power of two, so that 16-bit gradients are stored exactly; the
// rest of 1 / (|G| + eps) is a factor of the first step's epilogues.
//
// Work.  S and b S + c S S are symmetric: only tiles on and above the diagonal
// are computed, and stored twice.  A step costs m^2 n + m^3 + 2 m^2 n flops
// (m the shorter side) instead of 2 m^2 n + 2 m^3 + 2 m^2 n.
//
// On a GB300, five steps from a graph: 4096^2 takes 910 to 950 us (about 1500
// TFLOP/s of those flops, 0.78 of what a large library product reaches), bound by the
// tensor cores, by the last rounds of tiles (256 and 136 tiles on 76 pairs) and
// by the ways in and out of fifteen launches; 12 matrices of 2048 x 768 take
// 332 to 345 us, where those two weigh most; 1024^2 takes 116 us and 256 x 1000
// 110 us, all of it launches and latencies (seven for a product).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cluster.cuh"
#include "internal.h"
#include "ortho.h"
#include "outio.cuh"
#include "staging.cuh"
#include "tc_gemm.cuh"

namespace mpg {
namespace {

// ---------------------------------------------------------------------------
// norm and scaling
// ---------------------------------------------------------------------------
template <class XT>
__device__ __forceinline__ float as_f32(XT v);
template <>
__device__ __forceinline__ float as_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float as_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

constexpr int kScaleThreads = 256;
constexpr int kBatch = 4;   // chunks of 8 elements that a thread has in flight

// The chunks of 8 elements of a matrix that one thread takes: its index, then
// every grid's width further, as (row, chunk of the row) without divisions in
// the loop.  A matrix without gaps is one long row.
struct ChunkWalk {
  int64_t row, chunk, rows, per, step_rows, step_chunks;
  __device__ __forceinline__ ChunkWalk(const OrthoScaleParams& p, int64_t per_) : rows(p.flat ? 1 : p.rows), per(per_) {
    const int64_t i = blockIdx.x * kScaleThreads + threadIdx.x, n = gridDim.x * kScaleThreads;
    if (p.flat) {
      per = p.rows * per_;
      row = i < per ? 0 : 1;
      chunk = i;
      step_rows = 0;
      step_chunks = n;
    } else {
      row = (uint32_t)i / (uint32_t)per;
      chunk = (uint32_t)i % (uint32_t)per;
      step_rows = (uint32_t)n / (uint32_t)per;
      step_chunks = (uint32_t)n % (uint32_t)per;
    }
  }
  __device__ __forceinline__ bool inside() const { return row < rows; }
  __device__ __forceinline__ void next() {
    row += step_rows;
    chunk += step_chunks;
    if (chunk >= per) {
      chunk -= per;
      ++row;
    }
  }
};

// The thread's next kBatch chunks, their loads issued together (zeros beyond
// the matrix).
template <class XT>
__device__ __forceinline__ void read_batch(const OrthoScaleParams& p, ChunkWalk& at, const XT* g,
                                           float (&v)[kBatch][8]) {
  const int64_t cols = p.flat ? (int64_t)p.rows * p.cols : p.cols;
  const XT* line[kBatch];
  int left[kBatch];                        // elements of the line from there on, 8 at most
  bool fast = p.g_vec != 0;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    line[u] = g + at.row * p.ldg + at.chunk * 8;
    left[u] = at.inside() ? (int)max((int64_t)0, min((int64_t)8, cols - at.chunk * 8)) : 0;
    fast = fast && left[u] == 8;
    at.next();
  }
  if (fast) {
    uint4 w[kBatch][sizeof(XT) / 2];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int h = 0; h < (int)sizeof(XT) / 2; ++h) w[u][h] = ld_global(reinterpret_cast<const uint4*>(line[u]) + h);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      XT e[8];
      memcpy(e, w[u], sizeof(e));
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = as_f32<XT>(e[j]);
    }
  } else {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = j < left[u] ? as_f32<XT>(line[u][j]) : 0.0f;
  }
}

// Squares whose sum fp32 cannot hold safely, in 64 bits.  (Kept out of line:
// 64-bit arithmetic is very slow here, and inlined it was done for every
// element and discarded.)
__device__ __noinline__ void add_wide(double* wide, const float (&v)[kBatch][8]) {
  double s = 0.0;
#pragma unroll 1
  for (int j = 0; j < kBatch * 8; ++j) s += (double)v[j >> 3][j & 7] * (double)v[j >> 3][j & 7];
  *wide += s;
}

// partial[b][block] = sum of squares over the block's share of matrix b.  The
// squares of a batch of 32 elements, a thread's batches and the block's threads
// are added in fp32 where that is safe (the sum neither near overflow nor near
// underflow) and in 64 bits elsewhere, always in the same order.  With q batches
// to a thread the sum is off by at most (23 + q) 2^-24 of itself, the norm by
// half of that: 9e-7 for 4096^2 (q = 6).
template <class XT>
__global__ void __launch_bounds__(kScaleThreads) ortho_norm_kernel(const __grid_constant__ OrthoScaleParams p) {
  __shared__ float red[kScaleThreads / 32];
  __shared__ double red_wide[kScaleThreads];
  red_wide[threadIdx.x] = 0.0;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  const XT* g = reinterpret_cast<const XT*>(p.g) + (int64_t)b * p.stride_g;
  ChunkWalk at(p, (p.cols + 7) / 8);
  float sum = 0.0f;
  bool unsafe = false;
  while (at.inside()) {
    float v[kBatch][8];
    read_batch<XT>(p, at, g, v);
    float s[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) s[u] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int u = 0; u < kBatch; ++u) s[u] = fmaf(v[u][j], v[u][j], s[u]);
    const float batch = (s[0] + s[1]) + (s[2] + s[3]);
    if (batch >= 1e-28f && batch <= 1e30f) {
      sum += batch;
    } else {
      bool any = false;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int j = 0; j < 8; ++j) any = any || v[u][j] != 0.0f;
      if (any) {
        unsafe = true;
        float w[kBatch][8];                  // (a copy: only this one has an address)
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
#pragma unroll
          for (int j = 0; j < 8; ++j) w[u][j] = v[u][j];
        add_wide(&red_wide[threadIdx.x], w);
      }
    }
    if (sum > 1e30f) {
      unsafe = true;
      float w[kBatch][8] = {};
      w[0][0] = sqrtf(sum);                // a square root and its square: half a step of fp32 each
      add_wide(&red_wide[threadIdx.x], w);
      sum = 0.0f;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[warp] = sum;
  const bool wide = __syncthreads_or(unsafe) != 0;
  if (threadIdx.x == 0) {
    float f = 0.0f;
#pragma unroll
    for (int w = 0; w < kScaleThreads / 32; ++w) f += red[w];
    double s = (double)f;
    if (wide) {
#pragma unroll 1
      for (int i = 0; i < kScaleThreads; ++i) s += red_wide[i];
    }
    p.partial[(int64_t)b * kOrthoNormBlocks + blockIdx.x] = s;
  }
}

// What the sum of a matrix's squares says.  Norm and eps are held as a fraction
// in [1, 2) and an exponent, which has no limits here.
struct OrthoNorm {
  int e;             // the matrix is stored times 2^e
  float first;       // 2^-e / (norm + eps)
  float u;           // norm / (norm + eps) = u * 2^ue
  int ue;
};
__device__ __forceinline__ float split_exponent(float v, int* e) {        // v > 0
  const float f = frexpf(v, e);
  --*e;
  return 2.0f * f;
}
__device__ __forceinline__ OrthoNorm ortho_norm(const OrthoScaleParams& p, double s) {
  OrthoNorm n{0, 0.0f, 1.0f, 0};
  const uint32_t hi = (uint32_t)__double2hiint(s);
  const int exponent = (int)(hi >> 20) - 1023;                   // s = fraction * 2^exponent
  if (hi == 0u || exponent == 1024) {
    // zero (times any factor, whose square has to be finite too), 0 / 0, infinite or NaN
    n.first = hi == 0u && p.eps > 0.0f ? 0.0f : __uint_as_float(0x7FC00000u);
    return n;
  }
  const float fraction = __uint_as_float(0x3F800000u | ((hi & 0xFFFFFu) << 3) | ((uint32_t)__double2loint(s) >> 29));
  // norm = root * 2^half, root in [1, 2)
  const int half = exponent >> 1;
  const float root = sqrtf((exponent & 1) ? 2.0f * fraction : fraction);
  // norm + eps = sum * 2^top, sum in [1, 4)
  int top = half;
  float sum = root;
  if (p.eps > 0.0f) {
    int ee;
    const float ef = split_exponent(p.eps, &ee);
    top = max(half, ee);
    sum = scalbnf(root, half - top) + scalbnf(ef, ee - top);
  }
  // one factor of fp32 carries the tiniest norms of fp32 inputs only part of the way
  n.e = min(max(p.target_exp - half, -126), 127);
  n.first = scalbnf(1.0f / sum, -n.e - top);
  n.u = split_exponent(root / sum, &n.ue);
  n.ue += half - top;
  return n;
}

// The iterates' factors: later ones are stored times 2^(store_exp + extra), where
// extra brings a bound on their singular values (the polynomial of its
// coefficients' sizes, applied to u * 2^ue) to [1/2, 1) as long as it is below.
__device__ __forceinline__ void ortho_factors(const OrthoScaleParams& p, int b, OrthoNorm n) {
  p.factor[b] = n.first;
  for (int i = 1; i < p.steps; ++i) {
    if (n.ue < 0) {
      const float x = scalbnf(n.u, max(n.ue, -60)), x2 = x * x;
      const float v = n.u * (p.coeff_size[0] + x2 * (p.coeff_size[1] + x2 * p.coeff_size[2]));
      int up = 0;
      if (v > 3e38f) n.ue = 0;
      else if (v > 0.0f) n.u = split_exponent(v, &up);
      n.ue += up;
    }
    const int extra = min(max(-n.ue - 1, 0), 120 - p.store_exp);
    p.factor[(int64_t)i * p.batch + b] = scalbnf(1.0f, -p.store_exp - extra);
  }
}

// x = fp16(g * 2^e) with the power of two that brings the norm to [2^t, 2^(t+1))
// (t: target_exp).  Every block works it out from the partial sums, by a few
// additions in 64 bits and on the sum's exponent and fraction.
template <class XT>
__global__ void __launch_bounds__(kScaleThreads) ortho_scale_kernel(const __grid_constant__ OrthoScaleParams p) {
  __shared__ float scale_sh;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  OrthoNorm norm;                                                // (thread 0)
  if (threadIdx.x < 32) {
    double s = 0.0;
    for (int i = threadIdx.x; i < p.blocks; i += 32) s += p.partial[(int64_t)b * kOrthoNormBlocks + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) {
      norm = ortho_norm(p, s);
      scale_sh = scalbnf(1.0f, norm.e);
    }
  }
  __syncthreads();
  const float scale = scale_sh;
  const XT* g = reinterpret_cast<const XT*>(p.g) + (int64_t)b * p.stride_g;
  uint16_t* x = p.x + (int64_t)b * p.rows * p.ldx;
  ChunkWalk at(p, p.ldx / 8);
  while (at.inside()) {
    float v[kBatch][8];
    ChunkWalk to = at;
    read_batch<XT>(p, at, g, v);
#pragma unroll
    for (int u = 0; u < kBatch; ++u, to.next()) {
      if (!to.inside()) continue;
      *reinterpret_cast<uint4*>(x + to.row * p.ldx + to.chunk * 8) =
          make_uint4(pack_f16x2(v[u][0] * scale, v[u][1] * scale), pack_f16x2(v[u][2] * scale, v[u][3] * scale),
                     pack_f16x2(v[u][4] * scale, v[u][5] * scale), pack_f16x2(v[u][6] * scale, v[u][7] * scale));
    }
  }
  if (threadIdx.x == 0 && blockIdx.x == 0) ortho_factors(p, b, norm);
}

// ---------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------
// kPair: tiles of 256 x 256 on a cluster of two CTAs (cta_group::2), each CTA
// with 128 rows of A and 128 columns of B in shared memory and its 128 rows
// of the accumulator in TMEM.  Else tiles of 128 x 128 on one CTA.  Roles and
// hand-overs are the same: a TMA producer warp, an MMA warp (rank 0's issues
// for the pair), eight epilogue warps; two accumulators, so that the epilogue
// of a tile runs beside the products of the next.
template <bool kPair_>
struct OrthoTraits {
  static constexpr bool kPair = kPair_;
  static constexpr int kCtas = kPair ? 2 : 1;
  static constexpr int BM = 128;                    // rows of A held by one CTA
  static constexpr int kTile = kPair ? 256 : 128;
  static constexpr int kBHeld = 128;                // columns of B held by one CTA
  static constexpr int BK = 64;
  static constexpr int kRowBytes = 128;
  static constexpr uint32_t kSwizzle = kSwizzle128B;
  static constexpr int kInstrK = 16;
  static constexpr int kKSteps = BK / kInstrK;
  static constexpr int kATile = BM * kRowBytes;
  static constexpr int kStage = kATile + kBHeld * kRowBytes;
  static constexpr int kStages = 6;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;
  static constexpr int kAccBufs = 2;
  static constexpr int kTmemCols = kAccBufs * kTile;
  static constexpr int kEpiBytes = kEpiWarps * 32 * 32 * 4;
  static constexpr int kNumBars = 2 * kStages + 2 * kAccBufs + 1;
  static constexpr int kSmemBytes = 1024 + kStages * kStage + kEpiBytes + kNumBars * 8 + 16;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// ca and cz for matrix b.
struct OrthoScales {
  float ca, cz;
};
__device__ __forceinline__ OrthoScales ortho_scales(const OrthoGemmParams& p, int b) {
  float f = 1.0f, f2 = 1.0f;
  if (p.factor) f = ld_global(p.factor + b);
  // (the next iterate's is a power of two: its inverse by the exponent)
  if (p.next) f2 = __uint_as_float(0x7F000000u - __float_as_uint(ld_global(p.next + b)));
  if (p.square) f2 = f;
  return OrthoScales{p.ca * f * f2, p.cz * f * f2};
}

struct OrthoTile {
  int b, mb, nb;
};
__device__ __forceinline__ OrthoTile ortho_tile(const OrthoGemmParams& p, int t) {
  OrthoTile c;
  c.b = t / p.tiles_per_matrix;
  const int r = t - c.b * p.tiles_per_matrix;
  if (p.symmetric) {
    // column nb holds the tiles mb = 0 .. nb
    int nb = (int)((sqrtf(8.0f * (float)r + 1.0f) - 1.0f) * 0.5f);
    while ((int64_t)nb * (nb + 1) / 2 > r) --nb;
    while ((int64_t)(nb + 1) * (nb + 2) / 2 <= r) ++nb;
    c.nb = nb;
    c.mb = r - (int)((int64_t)nb * (nb + 1) / 2);
  } else {
    const int group = p.group_m * p.num_n_blk;
    const int g = r / group;
    const int first = g * p.group_m;
    const int gm = min(p.group_m, p.num_m_blk - first);
    const int within = r - g * group;
    c.mb = first + within % gm;
    c.nb = within / gm;
    if (g & 1) c.nb = p.num_n_blk - 1 - c.nb;
  }
  return c;
}

template <class T>
__global__ void __launch_bounds__(T::kThreads, 1) ortho_gemm_kernel(const __grid_constant__ OrthoGemmParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* epi_base = reinterpret_cast<float*>(smem + T::kStages * T::kStage);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(epi_base) + T::kEpiBytes);
  uint64_t* op_full = bars;
  uint64_t* op_empty = bars + T::kStages;
  uint64_t* acc_full = bars + 2 * T::kStages;
  uint64_t* acc_empty = acc_full + T::kAccBufs;
  uint64_t* done_bar = acc_empty + T::kAccBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = T::kPair ? cluster_ctarank() : 0u;
  const int worker = T::kPair ? (int)cluster_id_x() : (int)blockIdx.x;
  const int workers = T::kPair ? (int)num_clusters_x() : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(&op_full[i], 1);
      mbar_init(&op_empty[i], 1);
    }
    for (int i = 0; i < T::kAccBufs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], T::kCtas * T::kEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.map_a);
    tma_prefetch_map(&p.map_b);
  }
  if (warp == 1) {
    if constexpr (T::kPair) {
      tmem_alloc_pair(tmem_slot, T::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, T::kTmemCols);
      tmem_relinquish();
    }
    tc_fence_before_sync();
  }
  if constexpr (T::kPair) cluster_sync_all();
  else __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  WaitCtl ctl;
  ctl.abort = abort_flag;
  if constexpr (T::kPair) ctl.peer_abort = cluster_generic_ptr(const_cast<int*>(abort_flag), rank ^ 1u);
  ctl.status = p.status;
  ctl.limit_ns = p.wait_limit_ns;
  ctl.late_clock = true;
  const uint32_t op_smem = smem_addr(smem);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t full0 = T::kPair ? cluster_smem_addr(smem_addr(op_full), 0) : smem_addr(op_full);
      uint32_t it = 0;
      bool ok = true;
      for (int t = worker; t < p.num_tiles && ok; t += workers) {
        const OrthoTile tc = ortho_tile(p, t);
        const int arow = tc.mb * T::kTile + (int)rank * T::BM;
        const int bcol = tc.nb * T::kTile + (int)rank * T::kBHeld;
        for (int kb = 0; kb < p.num_k_blk; ++kb, ++it) {
          const uint32_t st = it % T::kStages;
          if (!mbar_wait(&op_empty[st], ((it / T::kStages) & 1u) ^ 1u, ctl)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(&op_full[st], T::kCtas * T::kStage);
          uint8_t* dst = smem + st * T::kStage;
          const int k0 = kb * T::BK;
          auto load = [&](const CUtensorMap* map, uint8_t* to, bool mn, int row0) {
            auto one = [&](uint8_t* d, int c0, int c1) {
              if constexpr (T::kPair) tma_load_3d_pair(d, map, full0 + st * 8u, c0, c1, tc.b);
              else tma_load_3d(d, map, &op_full[st], c0, c1, tc.b);
            };
            if (!mn) {
              one(to, k0, row0);
            } else {
#pragma unroll
              for (int g = 0; g < 2; ++g) one(to + g * T::BK * T::kRowBytes, row0 + g * T::BK, k0);
            }
          };
          load(&p.map_a, dst, p.a_mn_major != 0, arow);
          load(&p.map_b, dst + T::kATile, p.b_mn_major != 0, bcol);
        }
      }
      // a stage is released after its copies landed and were read
      const uint32_t n_drain = it < (uint32_t)T::kStages ? it : (uint32_t)T::kStages;
      for (uint32_t i = it - n_drain; i < it; ++i)
        drain_wait(&op_empty[i % T::kStages], (i / T::kStages) & 1u, p.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const bool leader = elect_one();
      const bool a_mn = p.a_mn_major != 0, b_mn = p.b_mn_major != 0;
      const uint32_t idesc = make_idesc(0u /* f16 */, a_mn, b_mn, T::kTile, T::kTile);
      // the start address sits in the descriptor's low bits, in units of 16 bytes
      const uint64_t a_desc = operand_desc<T>(op_smem, a_mn, 0), b_desc = operand_desc<T>(op_smem + T::kATile, b_mn, 0);
      const uint32_t a_step = (a_mn ? T::kInstrK * T::kRowBytes : 32) / 16, b_step = (b_mn ? T::kInstrK * T::kRowBytes : 32) / 16;
      const uint32_t d_base = __shfl_sync(0xffffffffu, tmem_base, 0);
      auto commit = [&](uint64_t* bar, uint16_t mask) {
        if constexpr (T::kPair) mma_commit_multicast(bar, mask);
        else mma_commit(bar);
      };
      uint32_t g = 0, st = 0, st_ph = 0;
      bool ok = true;
      for (int t = worker; t < p.num_tiles && ok; t += workers, ++g) {
        const uint32_t ab = g % T::kAccBufs;
        const uint32_t ph = ((g / T::kAccBufs) & 1u) ^ 1u;
        if (!(T::kPair ? warp_wait_relaxed(&acc_empty[ab], ph, ctl) : warp_wait(&acc_empty[ab], ph, ctl))) { ok = false; break; }
        tc_fence_after_sync();
        const uint32_t d0 = d_base + ab * T::kTile;
        for (int kb = 0; kb < p.num_k_blk; ++kb) {
          if (!warp_wait(&op_full[st], st_ph, ctl)) { ok = false; break; }
          tc_fence_after_sync();
          const uint64_t at = (uint64_t)(st * (T::kStage / 16));
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < T::kKSteps; ++ks) {
              const uint64_t da = a_desc + at + ks * a_step, db = b_desc + at + ks * b_step;
              const uint32_t acc = (kb > 0 || ks > 0) ? 1u : 0u;
              if constexpr (T::kPair) mma_f16_pair(d0, da, db, idesc, acc);
              else mma_f16(d0, da, db, idesc, acc);
            }
            commit(&op_empty[st], 0x3);
            if (kb + 1 == p.num_k_blk) commit(&acc_full[ab], 0x3);
          }
          __syncwarp();
          if (++st == T::kStages) {
            st = 0;
            st_ph ^= 1u;
          }
        }
      }
      // every MMA completes before TMEM is released
      if (leader) {
        commit(done_bar, 0x1);
        drain_wait(done_bar, 0, p.wait_limit_ns);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // A warp owns 32 rows (one per lane) and half of the tile's columns, in
    // chunks of 32.  Z's elements of a chunk are fetched a chunk ahead (the
    // first before the accumulator is complete): loaded where they are used,
    // their latency was most of the kernel's time at 768^2.
    const int q = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(32 * q) << 16;
    const uint32_t stg = smem_addr(epi_base + (warp - 2) * 1024);
    constexpr int kCcPer = T::kTile / 32 / (T::kEpiWarps / 4);
    const int cc0 = ((warp - 2) / 4) * kCcPer;
    const uint32_t acc_empty0 = T::kPair ? cluster_smem_addr(smem_addr(acc_empty), 0) : 0u;
    const int dt = p.d_dtype;
    const int es = dt == kOutF32 ? 4 : 2;
    uint32_t g = 0;
    for (int t = worker; t < p.num_tiles; t += workers, ++g) {
      const OrthoTile tc = ortho_tile(p, t);
      const float co = p.co;
      uint8_t* d = static_cast<uint8_t*>(p.d) + (int64_t)tc.b * p.stride_d * es;
      const uint32_t ab = g % T::kAccBufs;
      const uint32_t tacc = tmem_base + lane_off + ab * T::kTile;
      const int row_base = tc.mb * T::kTile + (int)rank * T::BM + 32 * q;
      const int row = row_base + lane;
      const bool mirror = p.symmetric && tc.mb != tc.nb;
      const uint16_t* zrow = p.z && row < p.m ? p.z + (int64_t)tc.b * p.stride_z + (int64_t)row * p.ldz : nullptr;
      uint4 z[4];
      auto fetch_z = [&](int cc) {
        const int c0 = tc.nb * T::kTile + cc * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z[i] = zrow && c0 + 8 * i < p.n ? ld_global(reinterpret_cast<const uint4*>(zrow + c0) + i) : make_uint4(0, 0, 0, 0);
      };
      fetch_z(cc0);
      const OrthoScales sc = ortho_scales(p, tc.b);
      const float ca = sc.ca, cz = sc.cz;
      if (!warp_wait(&acc_full[ab], (g / T::kAccBufs) & 1u, ctl)) break;
      tc_fence_after_sync();
#pragma unroll 1
      for (int cc = cc0; cc < cc0 + kCcPer; ++cc) {
        float v[32];
        tmem_ld_32cols(tacc + cc * 32, v);
        tmem_ld_wait();
        if (cc == cc0 + kCcPer - 1) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            // (TMEM alone is handed over: a release would wait for the stores)
            if constexpr (T::kPair) mbar_arrive_cluster_relaxed(acc_empty0 + ab * 8u);
            else mbar_arrive(&acc_empty[ab]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            __half2 h;
            memcpy(&h, &w[j], 4);
            const float2 y = __half22float2(h);
            v[8 * i + 2 * j] = fmaf(cz, y.x, ca * v[8 * i + 2 * j]);
            v[8 * i + 2 * j + 1] = fmaf(cz, y.y, ca * v[8 * i + 2 * j + 1]);
          }
        }
        if (cc + 1 < cc0 + kCcPer) fetch_z(cc + 1);
        const int col_base = tc.nb * T::kTile + cc * 32;
        if (row_base >= p.m || col_base >= p.n) continue;
        const bool whole = col_base + 32 <= p.n;
        if (dt != kOutF32 && co == 0.0f && p.vec16 && whole) {
          // 16-bit rows of 64 bytes through shared memory: chunk c of row r at
          // slot c ^ ((r / 2) & 3), which spreads both the writes (a row per
          // lane) and the reads (four lanes a row) over all banks
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[j] = dt == kOutF16 ? pack_f16x2(v[2 * j], v[2 * j + 1]) : pack_bf16x2(v[2 * j], v[2 * j + 1]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            st_shared_v4(stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), w[4 * c], w[4 * c + 1], w[4 * c + 2],
                         w[4 * c + 3]);
          if (mirror) {
            // and transposed: row j of D^T's chunk is column j here
#pragma unroll
            for (int j = 0; j < 16; ++j) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int c = 2 * j + h;
                st_shared_u16(stg + 2048 + c * 64 + (((lane >> 3) ^ ((c >> 1) & 3)) << 4) + (lane & 7) * 2,
                              (uint16_t)(w[j] >> (16 * h)));
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), c = lane & 3;
            const uint32_t at = r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
            if (row_base + r < p.m)
              *reinterpret_cast<uint4*>(d + ((int64_t)(row_base + r) * p.ldd + col_base + c * 8) * 2) =
                  ld_shared_u4(stg + at);
            if (mirror) {
              // column col_base + r, rows row_base + 8c ..
              const int row8 = row_base + c * 8;
              uint16_t* to = reinterpret_cast<uint16_t*>(d) + (int64_t)(col_base + r) * p.ldd + row8;
              const uint4 x = ld_shared_u4(stg + 2048 + at);
              if (row8 + 8 <= p.m) {
                *reinterpret_cast<uint4*>(to) = x;
              } else {
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (row8 + j < p.m) to[j] = (uint16_t)(y[j >> 1] >> (16 * (j & 1)));
              }
            }
          }
          __syncwarp();
          continue;
        }
        stage_write_row(stg, lane, v);
        __syncwarp();
        if (p.vec && whole) {
          float4 y[8];
          if (co != 0.0f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int grow = row_base + i * 4 + (lane >> 3);
              if (grow < p.m) y[i] = out_load4(d, (int64_t)grow * p.ldd + col_base + (lane & 7) * 4, dt);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int grow = row_base + i * 4 + (lane >> 3);
            float4 o = stage_read_chunk(stg, lane, i);
            if (grow < p.m) {
              if (co != 0.0f) {
                o.x = fmaf(co, y[i].x, o.x);
                o.y = fmaf(co, y[i].y, o.y);
                o.z = fmaf(co, y[i].z, o.z);
                o.w = fmaf(co, y[i].w, o.w);
              }
              out_store4(d, (int64_t)grow * p.ldd + col_base + (lane & 7) * 4, o, dt);
            }
          }
        } else {
          const int col = col_base + lane;
#pragma unroll 4
          for (int r = 0; r < 32; ++r) {
            float o = stage_read_elem(stg, lane, r);
            const int grow = row_base + r;
            if (grow < p.m && col < p.n) {
              const int64_t idx = (int64_t)grow * p.ldd + col;
              if (co != 0.0f) o = fmaf(co, out_load(d, idx, dt), o);
              out_store(d, idx, o, dt);
            }
          }
        }
        if (mirror && row < p.m) {
          // the same values at (column, row): lanes along the row of D^T
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (col_base + j < p.n) out_store(d, (int64_t)(col_base + j) * p.ldd + row, v[j], dt);
        }
        __syncwarp();
      }
    }
  }

  // neither CTA of a pair leaves while the other may address its shared memory
  __syncwarp();
  tc_fence_before_sync();
  if constexpr (T::kPair) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (T::kPair) tmem_dealloc_pair(tmem_base, T::kTmemCols);
    else tmem_dealloc(tmem_base, T::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// the product when there are few tiles
// ---------------------------------------------------------------------------
// One 128 x 128 tile per cluster of 2 or 4 CTAs, each with a range of k.  The
// ranges' sums meet in shared memory: every CTA reads its share of the tile's
// rows from all of them (in rank order: the result does not depend on timing)
// and stores it.  One launch has to fill the machine with a handful of tiles,
// and its time is that of one CTA's range and the way in and out.
struct DividedTraits {
  static constexpr int kTile = 128;
  static constexpr int BK = 64;
  static constexpr int kRowBytes = 128;
  static constexpr uint32_t kSwizzle = kSwizzle128B;
  static constexpr int kInstrK = 16;
  static constexpr int kKSteps = BK / kInstrK;
  static constexpr int kATile = kTile * kRowBytes;
  static constexpr int kStage = 2 * kATile;
  static constexpr int kStages = 6;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;
  static constexpr int kPitch = kTile + 4;                   // floats of a staged row
  static constexpr int kMirrorOffset = kTile * kPitch * 4;
  static constexpr int kZBytes = kTile * kTile * 2;          // Z's elements
  static constexpr int kNumBars = 2 * kStages + 1;
  static constexpr int kSmemBytes = 1024 + kStages * kStage + kZBytes + kNumBars * 8 + 16;
  static_assert(kMirrorOffset + kTile * kTile * 2 <= kStages * kStage, "staging reuses the operand stages");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// Where a CTA's share of the tile's rows goes.
struct DividedOut {
  uint8_t* d;            // this matrix of D
  int row0, col0;        // of the share's first row, of the tile
  float ca, cz;
  uint16_t* mir;         // staged transpose, or null
};

// Position of (column c, row r) in the staged transpose: lines of 128 16-bit
// values, chunk r / 8 at slot (r / 8) ^ ((c / 4) & 15), so that the lanes of a
// warp, four columns apart, reach eight groups of banks (unswizzled, two: the
// stores then took longer than the product).
__device__ __forceinline__ uint32_t mirror_at(int c, int r) {
  return (uint32_t)(c * 128 + (((r >> 3) ^ ((c >> 2) & 15)) << 3) + (r & 7));
}

constexpr int kDividedGroup = 4;   // rows that a warp takes at a time

// Z's elements of a warp's rows of the share, copied to shared memory beside
// the products (rows of 128 16-bit values, four a lane, zeros beyond D).
__device__ __forceinline__ void divided_fetch_z(const OrthoGemmParams& p, const DividedOut& out, int b, uint32_t zs,
                                                int r0, int rows, int rows_here, int cols_here, int lane) {
  for (int i = 0; i < rows; ++i) {
    const int r = r0 + i;
    const bool in = p.z && r < rows_here && lane * 4 < cols_here;
    const uint16_t* src =
        in ? p.z + (int64_t)b * p.stride_z + (int64_t)(out.row0 + r) * p.ldz + out.col0 + lane * 4 : p.z;
    if (p.z)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(zs + r * 256 + lane * 8), "l"(src),
                   "r"(in ? 8 : 0)
                   : "memory");
  }
}

// A warp's rows of the share (neighbours, so that two rows' values of a column
// go to the transpose in one store), four at a time; four columns a lane.  The
// ranges' sums of a group are loaded before the first is added.  The loop over
// groups stays rolled: a launch runs this code once.
// Rows beyond the matrix are not loaded: none of the CTAs may exit while a load
// from it is on its way, and only a load whose value is stored is known to have
// landed when the warp arrives at the cluster's last barrier.
template <int kSplits>
__device__ __forceinline__ void divided_rows(const OrthoGemmParams& p, const DividedOut& out, uint32_t op_smem,
                                             uint32_t zs, int ra, int rows_here, int cols_here, int warp, int lane) {
  using T = DividedTraits;
  constexpr int kRows = T::kTile / kSplits / 8;                       // of one warp
  constexpr int kAtOnce = kDividedGroup;
  static_assert(kRows % kAtOnce == 0, "rows in groups");
  uint32_t peer[kSplits];
#pragma unroll
  for (int s = 0; s < kSplits; ++s) peer[s] = cluster_smem_addr(op_smem, (uint32_t)s);
  const int c = lane * 4;
  const int dt = p.d_dtype;
#pragma unroll 1
  for (int i0 = 0; i0 < kRows; i0 += kAtOnce) {
    float4 part[kAtOnce][kSplits];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
      for (int s = 0; s < kSplits; ++s) {
        const uint32_t off = (uint32_t)((ra + warp * kRows + i0 + i) * T::kPitch + c) * 4u;
        part[i][s] = warp * kRows + i0 + i < rows_here ? ld_cluster_f4(peer[s] + off) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    uint32_t before[2];                                     // the even row's values, as fp16
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int r = warp * kRows + i0 + i;
      float4 o = part[i][0];
#pragma unroll
      for (int s = 1; s < kSplits; ++s) {
        o.x += part[i][s].x;
        o.y += part[i][s].y;
        o.z += part[i][s].z;
        o.w += part[i][s].w;
      }
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (p.z) {
        const uint2 w = ld_shared_u2(zs + r * 256 + lane * 8);
        __half2 h0, h1;
        memcpy(&h0, &w.x, 4);
        memcpy(&h1, &w.y, 4);
        const float2 y0 = __half22float2(h0), y1 = __half22float2(h1);
        y = make_float4(y0.x, y0.y, y1.x, y1.y);
      }
      o.x = fmaf(out.cz, y.x, out.ca * o.x);
      o.y = fmaf(out.cz, y.y, out.ca * o.y);
      o.z = fmaf(out.cz, y.z, out.ca * o.z);
      o.w = fmaf(out.cz, y.w, out.ca * o.w);
      if (r < rows_here && c < cols_here) {
        const int64_t idx = (int64_t)(out.row0 + r) * p.ldd + out.col0 + c;
        if (p.vec && c + 4 <= cols_here) {
          if (p.co != 0.0f) {
            const float4 y = out_load4(out.d, idx, dt);
            o.x = fmaf(p.co, y.x, o.x);
            o.y = fmaf(p.co, y.y, o.y);
            o.z = fmaf(p.co, y.z, o.z);
            o.w = fmaf(p.co, y.w, o.w);
          }
          out_store4(out.d, idx, o, dt);
        } else {
          const float e[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < cols_here)
              out_store(out.d, idx + j, p.co != 0.0f ? fmaf(p.co, out_load(out.d, idx + j, dt), e[j]) : e[j], dt);
        }
      }
      if (out.mir) {
        // (D is fp16 here: the operator's own S and B)
        const uint32_t w0 = pack_f16x2(o.x, o.y), w1 = pack_f16x2(o.z, o.w);
        if (i & 1) {
          uint32_t* m = reinterpret_cast<uint32_t*>(out.mir);
          m[mirror_at(c + 0, r - 1) / 2] = __byte_perm(before[0], w0, 0x5410);
          m[mirror_at(c + 1, r - 1) / 2] = __byte_perm(before[0], w0, 0x7632);
          m[mirror_at(c + 2, r - 1) / 2] = __byte_perm(before[1], w1, 0x5410);
          m[mirror_at(c + 3, r - 1) / 2] = __byte_perm(before[1], w1, 0x7632);
        } else {
          before[0] = w0;
          before[1] = w1;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(DividedTraits::kThreads, 1)
    ortho_divided_kernel(const __grid_constant__ OrthoGemmParams p) {
  using T = DividedTraits;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::kStages * T::kStage + T::kZBytes);
  uint64_t* op_full = bars;
  uint64_t* op_empty = bars + T::kStages;
  uint64_t* done_bar = bars + 2 * T::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const OrthoTile tc = ortho_tile(p, (int)(blockIdx.x / (uint32_t)p.splits));
  const int row0 = tc.mb * T::kTile, col0 = tc.nb * T::kTile;
  const int kb0 = (int)rank * p.kb_per_split;
  const int nkb = max(0, min(p.num_k_blk, kb0 + p.kb_per_split) - kb0);

  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(&op_full[i], 1);
      mbar_init(&op_empty[i], 1);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&p.map_a);
    tma_prefetch_map(&p.map_b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, T::kTile);
    tmem_relinquish();
    tc_fence_before_sync();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  WaitCtl ctl;
  ctl.abort = abort_flag;
  ctl.status = p.status;
  ctl.limit_ns = p.wait_limit_ns;
  ctl.late_clock = true;
  const uint32_t op_smem = smem_addr(smem);

  // this CTA's share of the tile's rows, and Z's elements there
  const int rows_per = T::kTile / p.splits;                  // (2 or 4 ranges)
  const int ra = (int)rank * rows_per;
  const int rows_here = min(rows_per, p.m - row0 - ra);
  const int cols_here = min(T::kTile, p.n - col0);
  DividedOut out;
  out.d = static_cast<uint8_t*>(p.d) + (int64_t)tc.b * p.stride_d * (p.d_dtype == kOutF32 ? 4 : 2);
  out.row0 = row0 + ra;
  out.col0 = col0;
  out.mir = p.symmetric && tc.mb != tc.nb ? reinterpret_cast<uint16_t*>(smem + T::kMirrorOffset) : nullptr;
  const uint32_t zs = op_smem + T::kStages * T::kStage;

  const OrthoScales sc = ortho_scales(p, tc.b);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int i = 0;
      for (; i < nkb; ++i) {
        const int st = i % T::kStages;
        if (!mbar_wait(&op_empty[st], ((i / T::kStages) & 1u) ^ 1u, ctl)) break;
        mbar_arrive_expect_tx(&op_full[st], T::kStage);
        uint8_t* dst = smem + st * T::kStage;
        const int k0 = (kb0 + i) * T::BK;
        auto load = [&](const CUtensorMap* map, uint8_t* to, bool mn, int r) {
          if (!mn) {
            tma_load_3d(to, map, &op_full[st], k0, r, tc.b);
          } else {
#pragma unroll
            for (int g = 0; g < 2; ++g) tma_load_3d(to + g * T::BK * T::kRowBytes, map, &op_full[st], r + g * T::BK, k0, tc.b);
          }
        };
        load(&p.map_a, dst, p.a_mn_major != 0, row0);
        load(&p.map_b, dst + T::kATile, p.b_mn_major != 0, col0);
      }
      for (int j = max(0, i - T::kStages); j < i; ++j)
        drain_wait(&op_empty[j % T::kStages], (j / T::kStages) & 1u, p.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const bool a_mn = p.a_mn_major != 0, b_mn = p.b_mn_major != 0;
    const uint32_t idesc = make_idesc(0u /* f16 */, a_mn, b_mn, T::kTile, T::kTile);
    const uint64_t a_desc = operand_desc<T>(op_smem, a_mn, 0), b_desc = operand_desc<T>(op_smem + T::kATile, b_mn, 0);
    const uint32_t a_step = (a_mn ? T::kInstrK * T::kRowBytes : 32) / 16, b_step = (b_mn ? T::kInstrK * T::kRowBytes : 32) / 16;
    const uint32_t d0 = __shfl_sync(0xffffffffu, tmem_base, 0);
    int st = 0;
    uint32_t st_ph = 0;
    for (int i = 0; i < nkb; ++i) {
      if (!warp_wait(&op_full[st], st_ph, ctl)) break;
      tc_fence_after_sync();
      const uint64_t at = (uint64_t)(st * (T::kStage / 16));
      if (leader) {
#pragma unroll
        for (int ks = 0; ks < T::kKSteps; ++ks)
          mma_f16(d0, a_desc + at + ks * a_step, b_desc + at + ks * b_step, idesc, (i > 0 || ks > 0) ? 1u : 0u);
        mma_commit(&op_empty[st]);
      }
      __syncwarp();
      if (++st == T::kStages) {
        st = 0;
        st_ph ^= 1u;
      }
    }
    if (leader) mma_commit(done_bar);
    if (!warp_wait(done_bar, 0, ctl) && leader) drain_wait(done_bar, 0, p.wait_limit_ns);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ this range's sums
    const int q = warp & 3;
    const int wc0 = ((warp - 2) / 4) * 64;
    divided_fetch_z(p, out, tc.b, zs, (warp - 2) * (rows_per / 8), rows_per / 8, rows_here, cols_here, lane);
    if (warp_wait(done_bar, 0, ctl)) {
      // every MMA is complete: the operand stages are free
      tc_fence_after_sync();
      const uint32_t t = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + wc0;
      float v[2][32];
      tmem_ld_32cols(t, v[0]);
      tmem_ld_32cols(t + 32, v[1]);
      tmem_ld_wait();
      if (nkb == 0) {                                        // an empty last range
#pragma unroll
        for (int j = 0; j < 32; ++j) v[0][j] = v[1][j] = 0.0f;
      }
      const uint32_t dst = op_smem + (uint32_t)((32 * q + lane) * T::kPitch + wc0) * 4u;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          stage_st16(dst + (h * 32 + j) * 4, v[h][j], v[h][j + 1], v[h][j + 2], v[h][j + 3]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  // ---------------------------------------------------------------- D
  tc_fence_before_sync();
  cluster_sync_all();
  const bool live = *abort_flag == 0 && rows_here > 0;
  if (live && warp >= 2) {
    out.ca = sc.ca;
    out.cz = sc.cz;
    switch (p.splits) {
      case 2: divided_rows<2>(p, out, op_smem, zs, ra, rows_here, cols_here, warp - 2, lane); break;
      default: divided_rows<4>(p, out, op_smem, zs, ra, rows_here, cols_here, warp - 2, lane); break;
    }
  }
  // The other CTAs' shared memory has been read: the value of every load from
  // it went into a store above (lane 0 stores in each row that is loaded).  Only
  // that is announced: a release waits for the stores as well, and takes 0.6 us
  // a launch even where it comes before them (1024^2: 128 us instead of 115).
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  if (out.mir) {
    __syncthreads();
    if (live) {
      // rows of D^T: 8 values (16 bytes) a thread
      const int vecs = rows_per / 8;
      for (int u = threadIdx.x; u < cols_here * vecs; u += T::kThreads) {
        const int c = u / vecs, r = (u - c * vecs) * 8;
        if (r >= rows_here) continue;
        uint16_t* to = reinterpret_cast<uint16_t*>(out.d) + (int64_t)(col0 + c) * p.ldd + row0 + ra + r;
        const uint16_t* from = out.mir + mirror_at(c, r);
        if (r + 8 <= rows_here) {
          *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
        } else {
          for (int j = 0; j < rows_here - r; ++j) to[j] = from[j];
        }
      }
    }
  }
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, T::kTile);
  }
  // no CTA exits while another may still read its shared memory
  asm volatile("barrier.cluster.wait;" ::: "memory");
}

template <class T>
void fill(OrthoKernel* out) {
  out->fn = reinterpret_cast<const void*>(&ortho_gemm_kernel<T>);
  out->block = T::kThreads;
  out->smem_bytes = T::kSmemBytes;
  out->tile = T::kTile;
  out->ctas = T::kCtas;
}

template <class XT>
cudaError_t launch_scale_type(const OrthoScaleParams& p, cudaLaunchConfig_t& cfg) {
  cudaError_t e = cudaLaunchKernelEx(&cfg, ortho_norm_kernel<XT>, p);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, ortho_scale_kernel<XT>, p);
}

}  // namespace

void ortho_lookup(OrthoForm form, OrthoKernel* out) {
  if (form == OrthoForm::kPair) {
    fill<OrthoTraits<true>>(out);
  } else if (form == OrthoForm::kOne) {
    fill<OrthoTraits<false>>(out);
  } else {
    *out = OrthoKernel{reinterpret_cast<const void*>(&ortho_divided_kernel), DividedTraits::kThreads,
                       DividedTraits::kSmemBytes, DividedTraits::kTile, 1};
  }
}

cudaError_t launch_ortho_scale(const OrthoScaleParams& p, int g_dtype, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.blocks, (unsigned)p.batch);
  cfg.blockDim = dim3(kScaleThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (g_dtype) {
    case 0: return launch_scale_type<float>(p, cfg);
    case 1: return launch_scale_type<__half>(p, cfg);
    default: return launch_scale_type<__nv_bfloat16>(p, cfg);
  }
}

}  // namespace mpg
