// The gradients' products of the gated layer and the vocabulary, and the sums of
// their split tiles.
#include "fused_gemm.cuh"

namespace mpg {
namespace {

// ---------------------------------------------------------------------------
// split tiles
// ---------------------------------------------------------------------------
// Adds a tile's parts in the order of k, four columns a thread.  Tiles that one
// worker had whole are done already.  Every worker has a block of k at least,
// so the parts of a tile are those of consecutive workers, and only the first
// can have begun in an earlier tile (its second slot).
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) fused_join_kernel(const __grid_constant__ FusedGemmParams p, int tile, int workers) {
  griddep_wait();
  griddep_launch_dependents();
  const FusedProduct& pr = p.prod[0];
  const int64_t u0 = (int64_t)blockIdx.x * pr.num_k_blk, u1 = u0 + pr.num_k_blk;
  const int w0 = (int)(((u0 + 1) * workers - 1) / p.units);                     // the last that begins at u0 or before
  const int n = (int)((u1 * workers + p.units - 1) / p.units) - w0;             // up to the last that begins before u1
  if (n == 1) return;
  const FusedTile tc = fused_tile(pr, p.whole_tiles + (int)blockIdx.x);
  const bool second = tc.mb >= pr.mb_second;
  const int per_row = tile / 4;
  const int i = blockIdx.y * kJoinThreads + threadIdx.x;
  const int r = i / per_row, c = i % per_row * 4;
  const int row = (second ? tc.mb - pr.mb_second : tc.mb) * tile + r, col = tc.nb * tile + c;
  const Pow2 sc = warp_scale(p.scale, p.scale_exp);
  if (row >= pr.m || col >= pr.n) return;
  const int64_t slot = (int64_t)tile * tile;
  const float* at = p.slots + (int64_t)r * tile + c;
  float4 o = out_load4(at, (2 * w0 + (first_unit(p.units, w0, workers) < u0 ? 1 : 0)) * slot, kOutF32);
#pragma unroll 4
  for (int j = 1; j < n; ++j) {
    const float4 y = out_load4(at, 2 * (w0 + j) * slot, kOutF32);
    o.x += y.x;
    o.y += y.y;
    o.z += y.z;
    o.w += y.w;
  }
  o.x *= sc.inv;
  o.y *= sc.inv;
  o.z *= sc.inv;
  o.w *= sc.inv;
  void* out = pr.out[second ? 1 : 0];
  const int64_t ldo = pr.ldo[second ? 1 : 0];
  if (pr.out_vec[second ? 1 : 0] && col + 4 <= pr.n) {
    if (pr.add) {
      const float4 y = out_load4(pr.add, (int64_t)row * pr.ldadd + col, kOutF32);
      o.x += y.x;
      o.y += y.y;
      o.z += y.z;
      o.w += y.w;
    }
    out_store4(out, (int64_t)row * ldo + col, o, pr.out_dtype);
  } else {
    const float e[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < pr.n)
        out_store(out, (int64_t)row * ldo + col + j,
                  pr.add ? e[j] + out_load(pr.add, (int64_t)row * pr.ldadd + col + j, kOutF32) : e[j], pr.out_dtype);
  }
}

}  // namespace

void fused_lookup_plain(bool pair, FusedKernel* out) {
  *out = pair ? fused_describe<FusedTraits<FusedEpi::kPlain, true>>() : fused_describe<FusedTraits<FusedEpi::kPlain, false>>();
}

cudaError_t launch_fused_join(const FusedGemmParams& p, int tile, int workers, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.prod[0].num_tiles - p.whole_tiles), (unsigned)(tile * tile / 4 / kJoinThreads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, 1);
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, fused_join_kernel, p, tile, workers);
}

}  // namespace mpg
