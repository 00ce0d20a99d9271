// Products of few rows (up to 16 tokens being decoded or scored): the
// weights are read once, and their bytes are all that counts (sm_103a).
//
// Weight lines are the M side of mma.sync m16n8k16 and the rows of X its N
// side, eight at a time, so that nothing but X is padded.  A strip is 16 lines:
// 8 of Wg and the same 8 of Wu (gated, and dgate and dup; c0, c1 of a thread are gates and c2, c3
// the same elements' ups), or 16 classes of a vocabulary.  The order of k inside
// a sum is free, so a thread takes 16 contiguous bytes of a line as its values
// of two instructions, and the same bytes of X's rows: fragments come straight
// from global memory, without shared memory between.
//
// A producer warp streams the lines to a ring in shared memory by bulk copies, 16
// lines of 512 k a stage, over strip after strip, so that the memory never waits
// for a strip's way out; eight warps take 64 k each of a stage, and their sums meet
// in shared memory at a strip's end.  Lines in a stage are 64 bytes more apart than
// they are long: the 8 lanes of a 16-byte read then reach all banks once.  Two CTAs
// on an SM cover each other's ways in and out.  A token through 4096 x 11008 takes
// 30 us (6.0 TB/s of 6.8; the same fragments loaded straight from global memory 41).
//
// Lines are whole 16 bytes: others are copied to such lines first, with zeros
// behind them.  (Read by the threads themselves, element by element or as two
// words and a shift, 14 rows by 16384 lines of 2140 took 62 to 66 us with the loss; copied and streamed 52.)
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

// Elements k .. k+7 of a line whose chunks of eight start on 16 bytes (0 beyond its end; null: none).
__device__ __forceinline__ uint4 load8(const uint16_t* line, int k, int end) {
  if (!line || k >= end) return make_uint4(0, 0, 0, 0);
  return ld_global(reinterpret_cast<const uint4*>(line + k));
}

constexpr bool two_of(FusedEpi e) { return e == FusedEpi::kGated || e == FusedEpi::kGatedGrad; }

// The warps' sums of a strip (one a CTA) and what becomes of them; by the
// kWarps * 32 threads of them, `sync` between.
template <FusedEpi E, int kNt, class Red, class Sync>
__device__ __forceinline__ void finish(const FewRowsParams& p, Red& red, const Scale& sc, float& top, int thread, int strip, Sync&& sync) {
  constexpr int kTokens = 8 * kNt;
  constexpr int kLines = two_of(E) ? 8 : 16;
  const int first = strip * kLines;
  const bool bf16 = p.bf16 != 0;
  auto store = [&](void* base, int64_t ld, int t, int j, uint32_t w) {
    static_cast<uint16_t*>(base)[(int64_t)t * ld + first + j] = (uint16_t)w;
  };
  if constexpr (two_of(E)) {
    for (int e = thread; e < kLines * kTokens; e += kWarps * 32) {
      const int j = e % kLines, t = e / kLines;
      float gt = 0.0f, up = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gt += red[w][j][t];
        up += red[w][j + 8][t];
      }
      if (t < p.rows && first + j < p.n) {
        float a, d;
        if constexpr (E == FusedEpi::kGatedGrad) {
          const float y = sc.mul * load16(p.dy, (int64_t)t * p.lddy + first + j, bf16);
          act_both(gt, p.act, a, d);
          const float dg = y * (up * d), du = y * a;
          top = largest_finite(largest_finite(top, dg), du);
          store(p.y, p.ldy, t, j, pack16(dg, 0.0f, bf16));
          store(p.ka, p.lda, t, j, pack16(du, 0.0f, bf16));
        } else {
          store(p.y, p.ldy, t, j, pack16(act_value(gt, p.act) * up, 0.0f, bf16));
          if (p.ka) {
            act_both(gt, p.act, a, d);
            store(p.ka, p.lda, t, j, pack_kept(a, 0.0f, bf16));
            store(p.kb, p.ldb, t, j, pack_kept(up * d, 0.0f, bf16));
          }
        }
      }
    }
  } else {
    for (int e = thread; e < kLines * kTokens; e += kWarps * 32) {
      const int j = e % kLines, t = e / kLines;
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l += red[w][j][t];
      if constexpr (E == FusedEpi::kProb) {
        if (t < p.rows && first + j < p.n) {
          const int64_t target = target_of(p.target, p.target_bytes, p.target_stride, p.ignore_index, p.vocab, t);
          const float weight = target < 0 ? (target == -1 ? 0.0f : NAN) : sc.mul * (ld_global(p.dloss + t * p.dloss_stride) / sc.div);
          const float x = ex2(fmaf(kLog2e, l, -kLog2e * ld_global(p.lse + t)));
          store(p.y, p.ldy, t, j, weight == 0.0f ? 0u : pack16(weight * (target == p.col0 + first + j ? x - 1.0f : x), 0.0f, bf16));
        }
      } else {
        red[0][j][t] = l;
      }
    }
    if constexpr (E == FusedEpi::kProb) return;
    sync();
    const int t = thread;
    if (t < p.rows) {
      const int64_t target = target_of(p.target, p.target_bytes, p.target_stride, p.ignore_index, p.vocab, t);
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

// ---------------------------------------------------------------------------
// the ring
// ---------------------------------------------------------------------------
template <int kNt>
struct RingTraits {
  static constexpr int kLines = 16;                       // of weights in a stage
  static constexpr int kWidth = 512;                      // k of a stage, 64 of each warp
  // Stages that are summed by the tensor cores at a time where the sums become a loss
  // (1024 of k in a warp): their sums are cut off towards zero, and those of 65536
  // positive products in one were off by 1.5e-5.
  static constexpr int kFold = 16;
  static constexpr int kPitch = kWidth * 2 + 64;
  static constexpr int kStage = kLines * kPitch;
  static constexpr int kTokens = 8 * kNt;
  using Red = float[kWarps][kLines][kTokens + 1];
  static constexpr int kStages = 5;                       // of a CTA; two CTAs on an SM
  static constexpr int kReds = 2;                         // sets of sums
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

template <FusedEpi E, int kNt>
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
  if (E == FusedEpi::kGatedGrad && !GradTop::needed(p, blockIdx.x == 0 && warp == 0)) return;
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
        const int row = two_of(E) ? strip * 8 + (lane & 7) : strip * 16 + lane;
        if (row < p.n)
          line = two_of(E) && lane >= 8 ? static_cast<const uint16_t*>(p.wu) + (int64_t)row * p.ldwu
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
  const Scale sc = E == FusedEpi::kGatedGrad ? GradTop::scale(p) : warp_scale(p.scale, p.scale_count, p.scale_exp, p.scale_largest != 0);
  float top = 0.0f;
  const uint16_t* xr[kNt];
#pragma unroll
  for (int i = 0; i < kNt; ++i)
    xr[i] = 8 * i + g < p.rows ? static_cast<const uint16_t*>(p.x) + (int64_t)(8 * i + g) * p.ldx : nullptr;
  // X's bytes of half of a stage, fetched a stage ahead
  uint4 x[2][kNt];
  auto fetch = [&](int c, int h) {
#pragma unroll
    for (int i = 0; i < kNt; ++i) x[h][i] = load8(xr[i], c * T::kWidth + warp * 64 + h * 32 + tig * 8, p.k);
  };
  fetch(0, 0);
  fetch(0, 1);
  uint32_t it = 0, n = 0;
  bool ok = true;                                    // (a CTA that gives up still meets at its barriers)
  for (int strip = blockIdx.x; strip < strips; strip += gridDim.x, ++n) {
    float c[kNt][4], folded[kNt][4];
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = folded[i][j] = 0.0f;
    for (int k = 0; k < chunks; ++k, ++it) {
      const uint32_t st = it % T::kStages;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&full[st], (it / T::kStages) & 1u, ctl));
      const uint32_t at = smem_addr(smem) + st * T::kStage + g * T::kPitch + (warp * 64 + tig * 8) * 2;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (what lies beyond k in a stage is of an earlier one)
        const bool in = k * T::kWidth + warp * 64 + h * 32 + tig * 8 < p.k;
        const uint4 a = in ? ld_shared_16(at + h * 64) : make_uint4(0, 0, 0, 0);
        const uint4 b = in ? ld_shared_16(at + 8 * T::kPitch + h * 64) : make_uint4(0, 0, 0, 0);
        if (h == 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }
#pragma unroll
        for (int i = 0; i < kNt; ++i) {
          mma_sync(c[i], a.x, b.x, a.y, b.y, x[h][i].x, x[h][i].y, bf16);
          mma_sync(c[i], a.z, b.z, a.w, b.w, x[h][i].z, x[h][i].w, bf16);
        }
        fetch(k + 1 < chunks ? k + 1 : 0, h);
      }
      if constexpr (E == FusedEpi::kStats) {
        if (k % T::kFold == T::kFold - 1 || k + 1 == chunks) {
#pragma unroll
          for (int i = 0; i < kNt; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              folded[i][j] += c[i][j];
              c[i][j] = 0.0f;
            }
        }
      }
    }
    if constexpr (E == FusedEpi::kStats) {
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = folded[i][j];
    }
    // (two sets of sums in turn: one barrier a strip keeps them apart)
    auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); };
    typename T::Red& r = red[n % T::kReds];
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) r[warp][g + 8 * (j >> 1)][8 * i + 2 * tig + (j & 1)] = c[i][j];
    sync();
    finish<E, kNt>(p, r, sc, top, threadIdx.x, strip, sync);
  }
  if (E == FusedEpi::kGatedGrad && p.record) {
    __syncwarp();
    GradTop::record(p.record, (int)blockIdx.x * kWarps + warp, top);
  }
}

template <FusedEpi E, int kNt>
mpg_status launch(DeviceInfo* dev, FewRowsParams& p, cudaStream_t stream) {
  constexpr int kLines = two_of(E) ? 8 : 16;
  using T = RingTraits<kNt>;
  p.strips = (p.n + kLines - 1) / kLines;
  p.status = dev->status;
  p.wait_limit_ns = kDefaultWaitNs;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  const mpg_status s = allow_smem(dev, reinterpret_cast<const void*>(&few_rows_kernel<E, kNt>), T::kSmemBytes);
  if (s != MPG_OK) return s;
  cfg.gridDim = dim3((unsigned)std::min(p.strips, 2 * dev->sm_count));
  cfg.blockDim = dim3(T::kThreads);
  cfg.dynamicSmemBytes = T::kSmemBytes;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, few_rows_kernel<E, kNt>, static_cast<const FewRowsParams&>(p));
  return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "few rows launch: %s", cudaGetErrorString(e));
}

}  // namespace

int few_rows_parts(int64_t n) {
  return (int)((n + 15) / 16);
}

namespace {
template <FusedEpi E>
mpg_status launch_rows(DeviceInfo* dev, FewRowsParams& p, cudaStream_t stream) {
  return p.rows <= 8 ? launch<E, 1>(dev, p, stream) : launch<E, 2>(dev, p, stream);
}
}  // namespace

mpg_status launch_few_rows(DeviceInfo* dev, FewRowsParams& p, FusedEpi epi, cudaStream_t stream) {
  switch (epi) {
    case FusedEpi::kGated: return launch_rows<FusedEpi::kGated>(dev, p, stream);
    case FusedEpi::kGatedGrad: return launch_rows<FusedEpi::kGatedGrad>(dev, p, stream);
    case FusedEpi::kStats: return launch_rows<FusedEpi::kStats>(dev, p, stream);
    default: return launch_rows<FusedEpi::kProb>(dev, p, stream);
  }
}

}  // namespace mpg
