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
// Where lines are whole 16 bytes, a producer warp streams them to a ring in
// shared memory by bulk copies, 16 lines of 512 k a stage, over strip after strip,
// so that the memory never waits for a strip's way out; eight warps take 64 k each
// of a stage, and their sums meet in shared memory at a strip's end.  Lines in a
// stage are 64 bytes more apart than they are long: the 8 lanes of a 16-byte read
// then reach all banks once.  Other lines are read by the threads themselves.
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

// The warps' sums of a strip (one a CTA) and what becomes of them; by the
// kWarps * 32 threads of them, `sync` between.
template <int kNt>
constexpr int strips_of() { return kNt > 2 ? 2 : 1; }
template <bool kGated, int kNt, class Red, class Sync>
__device__ __forceinline__ void finish(const FewRowsParams& p, Red& red, int thread, int strip, Sync&& sync) {
  constexpr int kTokens = 8 * kNt;
  constexpr int kLines = (kGated ? 8 : 16) * strips_of<kNt>();
  const int first = strip * kLines;
  const bool bf16 = p.bf16 != 0;
  if constexpr (kGated) {
    for (int e = thread; e < kLines * kTokens; e += kWarps * 32) {
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
    for (int e = thread; e < kLines * kTokens; e += kWarps * 32) {
      const int j = e % kLines, t = e / kLines;
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l += red[w][j][t];
      red[0][j][t] = l;
    }
    sync();
    const int t = thread;
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
      p.stats[(int64_t)strip * p.rows + t] = make_float2(top, nan ? NAN : top == -INFINITY ? 0.0f : sum);
    }
  }
}

template <bool kGated, int kNt>
__global__ void __launch_bounds__(kWarps * 32) few_rows_plain_kernel(const __grid_constant__ FewRowsParams p) {
  constexpr int kStrips = strips_of<kNt>();
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
          a[u][h][s] = load8<false>(lo[s], k, p.k);
          b[u][h][s] = load8<false>(hi[s], k, p.k);
        }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + u * kWarps * 64 + h * 32 + tig * 8;
#pragma unroll
        for (int i = 0; i < kNt; ++i) {
          const uint4 x = load8<false>(xr[i], k, p.k);
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

  finish<kGated, kNt>(p, red, threadIdx.x, (int)blockIdx.x, [] { __syncthreads(); });
}

// ---------------------------------------------------------------------------
// the ring
// ---------------------------------------------------------------------------
template <int kNt>
struct RingTraits {
  static constexpr int kStrips = strips_of<kNt>();
  static constexpr int kLines = 16 * kStrips;             // of weights in a stage
  static constexpr int kWidth = 512;                      // k of a stage
  static constexpr int kPitch = kWidth * 2 + 64;
  static constexpr int kStage = kLines * kPitch;
  static constexpr int kTokens = 8 * kNt;
  using Red = float[kWarps][kLines][kTokens + 1];
  static constexpr int kStages = kNt > 2 ? 2 : 5;         // of a CTA; two CTAs on an SM
  static constexpr int kReds = kNt > 2 ? 1 : 2;           // sets of sums
  static constexpr int kSmemBytes = kStages * kStage + kReds * (int)sizeof(Red) + 2 * kStages * 8 + 16;
  static constexpr int kThreads = (kWarps + 1) * 32;
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs on an SM");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <bool kGated, int kNt>
__global__ void __launch_bounds__(RingTraits<kNt>::kThreads, 2) few_rows_kernel(const __grid_constant__ FewRowsParams p) {
  using T = RingTraits<kNt>;
  extern __shared__ __align__(128) uint8_t smem[];
  typename T::Red* red = reinterpret_cast<typename T::Red*>(smem + T::kStages * T::kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::kStages * T::kStage + T::kReds * sizeof(typename T::Red));
  uint64_t* empty = full + T::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + T::kStages);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int strips = p.strips, chunks = (p.k + T::kWidth - 1) / T::kWidth;
  if (threadIdx.x == 0) {
    for (int i = 0; i < T::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  WaitCtl ctl;
  ctl.abort = abort_flag;
  ctl.status = p.status;
  ctl.limit_ns = p.wait_limit_ns;

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer: a line a lane
    uint32_t it = 0;
    bool ok = true;
    for (int strip = blockIdx.x; strip < strips && ok; strip += gridDim.x) {
      const uint16_t* line = nullptr;
      if (lane < T::kLines) {
        const int s = lane >> 4, j = lane & 15;
        const int row = kGated ? (strip * T::kStrips + s) * 8 + (j & 7) : (strip * T::kStrips + s) * 16 + j;
        if (row < p.n)
          line = kGated && j >= 8 ? static_cast<const uint16_t*>(p.wu) + (int64_t)row * p.ldwu
                                  : static_cast<const uint16_t*>(p.w) + (int64_t)row * p.ldw;
      }
      const uint32_t lines = __popc(__ballot_sync(0xffffffffu, line != nullptr));
      for (int c = 0; c < chunks; ++c, ++it) {
        const uint32_t st = it % T::kStages;
        const bool mine = mbar_wait(&empty[st], ((it / T::kStages) & 1u) ^ 1u, ctl);
        if (!(ok = __all_sync(0xffffffffu, mine))) break;
        const int k0 = c * T::kWidth;
        const uint32_t bytes = 2u * (uint32_t)min(T::kWidth, p.k - k0);
        if (lane == 0) mbar_arrive_expect_tx(&full[st], lines * bytes);
        __syncwarp();
        if (line) bulk_load(smem_addr(smem) + st * T::kStage + lane * T::kPitch, line + k0, bytes, &full[st]);
      }
    }
    // the copies have landed before the CTA's shared memory is given up: the last
    // ones were read, or are waited for here
    const uint32_t n = it < (uint32_t)T::kStages ? it : (uint32_t)T::kStages;
    for (uint32_t i = it - n; i < it; ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_test(&full[i % T::kStages], (i / T::kStages) & 1u) && global_timer_ns() - t0 < p.wait_limit_ns) {
      }
    }
    return;
  }
  // -------------------------------------------------------------- sums
  const int g = lane >> 2, tig = lane & 3;
  const bool bf16 = p.bf16 != 0;
  const uint16_t* xr[kNt];
#pragma unroll
  for (int i = 0; i < kNt; ++i)
    xr[i] = 8 * i + g < p.rows ? static_cast<const uint16_t*>(p.x) + (int64_t)(8 * i + g) * p.ldx : nullptr;
  // X's bytes of half of a stage, fetched a stage ahead
  uint4 x[2][kNt];
  auto fetch = [&](int c, int h) {
#pragma unroll
    for (int i = 0; i < kNt; ++i) x[h][i] = load8<true>(xr[i], c * T::kWidth + warp * 64 + h * 32 + tig * 8, p.k);
  };
  fetch(0, 0);
  fetch(0, 1);
  uint32_t it = 0, n = 0;
  bool ok = true;                                    // (a CTA that gives up still meets at its barriers)
  for (int strip = blockIdx.x; strip < strips; strip += gridDim.x, ++n) {
    float c[T::kStrips][kNt][4];
#pragma unroll
    for (int s = 0; s < T::kStrips; ++s)
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[s][i][j] = 0.0f;
    for (int k = 0; k < chunks; ++k, ++it) {
      const uint32_t st = it % T::kStages;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (it / T::kStages) & 1u, ctl));
      const uint32_t at = smem_addr(smem) + st * T::kStage + g * T::kPitch + (warp * 64 + tig * 8) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (what lies beyond k in a stage is of an earlier one)
        const bool in = k * T::kWidth + warp * 64 + h * 32 + tig * 8 < p.k;
        uint4 a[T::kStrips], b[T::kStrips];
#pragma unroll
        for (int s = 0; s < T::kStrips; ++s) {
          a[s] = in ? ld_shared_16(at + s * 16 * T::kPitch + h * 64) : make_uint4(0, 0, 0, 0);
          b[s] = in ? ld_shared_16(at + (s * 16 + 8) * T::kPitch + h * 64) : make_uint4(0, 0, 0, 0);
        }
        if (h == 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
#pragma unroll
        for (int i = 0; i < kNt; ++i)
#pragma unroll
          for (int s = 0; s < T::kStrips; ++s) {
            mma_sync(c[s][i], a[s].x, b[s].x, a[s].y, b[s].y, x[h][i].x, x[h][i].y, bf16);
            mma_sync(c[s][i], a[s].z, b[s].z, a[s].w, b[s].w, x[h][i].z, x[h][i].w, bf16);
          }
        fetch(k + 1 < chunks ? k + 1 : 0, h);
      }
    }
    // (two sets of sums in turn: one barrier a strip keeps them apart)
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); };
    typename T::Red& r = red[n % T::kReds];
    if (T::kReds == 1 && n > 0) sync();
#pragma unroll
    for (int s = 0; s < T::kStrips; ++s)
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) r[warp][s * 16 + g + 8 * (j >> 1)][8 * i + 2 * tig + (j & 1)] = c[s][i][j];
    sync();
    finish<kGated, kNt>(p, r, threadIdx.x, strip, sync);
  }
}

template <bool kGated, int kNt>
mpg_status launch(DeviceInfo* dev, FewRowsParams& p, cudaStream_t stream) {
  constexpr int kLines = (kGated ? 8 : 16) * strips_of<kNt>();
  using T = RingTraits<kNt>;
  p.strips = (p.n + kLines - 1) / kLines;
  p.status = dev->status;
  p.wait_limit_ns = kDefaultWaitNs;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  cudaError_t e;
  if (p.vec) {
    const mpg_status s = allow_smem(dev, reinterpret_cast<const void*>(&few_rows_kernel<kGated, kNt>), T::kSmemBytes);
    if (s != MPG_OK) return s;
    cfg.gridDim = dim3((unsigned)std::min(p.strips, 2 * dev->sm_count));
    cfg.blockDim = dim3(T::kThreads);
    cfg.dynamicSmemBytes = T::kSmemBytes;
    e = cudaLaunchKernelEx(&cfg, few_rows_kernel<kGated, kNt>, static_cast<const FewRowsParams&>(p));
  } else {
    cfg.gridDim = dim3((unsigned)p.strips);
    cfg.blockDim = dim3(kWarps * 32);
    e = cudaLaunchKernelEx(&cfg, few_rows_plain_kernel<kGated, kNt>, static_cast<const FewRowsParams&>(p));
  }
  return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "few rows launch: %s", cudaGetErrorString(e));
}

}  // namespace

int few_rows_parts(int rows, int64_t n) {
  const int lines = rows > 16 ? 32 : 16;
  return (int)((n + lines - 1) / lines);
}

mpg_status launch_few_rows(DeviceInfo* dev, FewRowsParams& p, bool gated, cudaStream_t stream) {
  if (p.rows <= 8) return gated ? launch<true, 1>(dev, p, stream) : launch<false, 1>(dev, p, stream);
  if (p.rows <= 16) return gated ? launch<true, 2>(dev, p, stream) : launch<false, 2>(dev, p, stream);
  return gated ? launch<true, 4>(dev, p, stream) : launch<false, 4>(dev, p, stream);
}

}  // namespace mpg
