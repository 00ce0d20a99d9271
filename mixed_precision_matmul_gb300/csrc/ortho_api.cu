// mpg_orthogonalize: argument checks, workspace layout, and the sequence of
// launches (norm, scaling, then three products a step; ortho.cu).
#include <cmath>
#include <cstring>

#include "host.h"
#include "ortho.h"

using namespace mpg;

namespace {

// the last tile's end, and a block beyond it, still fit 32 bits
constexpr int64_t kMaxExtent = 0x7FFFFFFF - 255;
constexpr int64_t kMaxBatch = 65535;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int64_t line8(int64_t n) { return (n + 7) / 8 * 8; }

struct Layout {
  int64_t side, ldx, lds;          // shorter side; leading dimensions of X and of S
  size_t partial, factor, x[2], s, b, bytes;
};
Layout layout(int64_t m, int64_t n, int64_t batch) {
  Layout l;
  l.side = std::min(m, n);
  l.ldx = line8(n);
  l.lds = line8(l.side);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align256(bytes);
    return r;
  };
  l.partial = take((size_t)batch * kOrthoNormBlocks * sizeof(double));
  l.factor = take((size_t)batch * kOrthoMaxSteps * sizeof(float));
  for (size_t& x : l.x) x = take((size_t)batch * (size_t)m * (size_t)l.ldx * 2);
  l.s = take((size_t)batch * (size_t)l.side * (size_t)l.lds * 2);
  l.b = take((size_t)batch * (size_t)l.side * (size_t)l.lds * 2);
  l.bytes = at;
  return l;
}

// One fp16 matrix of the batch, row-major.
struct Matrix {
  void* ptr;
  int64_t ld, rows;
  Operand operand() const { return Operand{ptr, ld, rows * ld, MPG_F16, MPG_ROW_MAJOR}; }
};

// rows x k operand of a product: K-major if k is the matrix's contiguous side.
mpg_status operand_map(CUtensorMap* map, const Matrix& x, bool mn_major, int64_t rows, int64_t k, int64_t batch) {
  return mn_major ? encode_map(map, x.operand(), rows, k, batch, 64, 64)
                  : encode_map(map, x.operand(), k, rows, batch, 64, 128);
}

mpg_status launch_gemm(DeviceInfo* dev, OrthoGemmParams p, cudaStream_t stream) {
  OrthoKernel one, two, div;
  ortho_lookup(OrthoForm::kOne, &one);
  ortho_lookup(OrthoForm::kPair, &two);
  ortho_lookup(OrthoForm::kDivided, &div);
  int clusters = 0;
  mpg_status s = resident_clusters(dev, two.fn, two.block, two.smem_bytes, 2, &clusters);
  if (s != MPG_OK) return s;
  if ((s = allow_smem(dev, one.fn, one.smem_bytes)) != MPG_OK) return s;
  if ((s = allow_smem(dev, div.fn, div.smem_bytes)) != MPG_OK) return s;
  auto tiles = [&](int64_t t) {
    const int64_t mb = (p.m + t - 1) / t, nb = (p.n + t - 1) / t;
    return (p.symmetric ? nb * (nb + 1) / 2 : mb * nb) * p.batch;
  };
  const int64_t t1 = tiles(one.tile), t2 = tiles(two.tile), sms = dev->sm_count;
  const int64_t kb = (p.k + 63) / 64;
  // The form that ends first, by what the forms take on a GB300 (us, from
  // their times at 64^2 .. 2048^2): a way in and out, and a time for each
  // block of 64 k in each round of tiles.  A 128 x 128 tile on one CTA is
  // bound by its operands' way to the SM; a pair's 256 x 256 tile does four
  // times the work on two SMs in hardly more time a block, but takes longer to
  // store; with few tiles k is divided among up to 4 CTAs (one to an SM), which
  // exchange their sums.
  constexpr double kOneEdge = 4.3, kDividedEdge = 5.4, kPairEdge = 7.5, kOneBlock = 0.29, kPairBlock = 0.31;
  int64_t splits = 1;
  while (splits < 4 && t1 * splits * 2 <= sms && kb / (splits * 2) >= 1) splits *= 2;   // (8: slower, 128 x 4096: 28 against 19 us a step)
  const int64_t per = (kb + splits - 1) / splits;
  const double time_one = kOneEdge + (double)((t1 + sms - 1) / sms * kb) * kOneBlock;
  const double time_div = kDividedEdge + (double)per * kOneBlock;
  const double time_pair = kPairEdge + (double)((t2 + clusters - 1) / clusters * kb) * kPairBlock;
  const bool divided = splits > 1 && time_div < std::min(time_one, time_pair);
  const bool pair = !divided && time_pair < time_one;
  const OrthoKernel& k = pair ? two : divided ? div : one;
  const int64_t all = pair ? t2 : t1;
  if (all > kMaxExtent) return fail(MPG_ERR_INVALID_ARG, "too many tiles");
  p.num_m_blk = (p.m + k.tile - 1) / k.tile;
  p.num_n_blk = (p.n + k.tile - 1) / k.tile;
  p.num_k_blk = (int32_t)kb;
  p.tiles_per_matrix = (int32_t)(all / p.batch);
  p.num_tiles = (int32_t)all;
  p.splits = divided ? (int32_t)splits : 1;
  p.kb_per_split = (int32_t)per;
  p.group_m = pair ? 8 : 16;
  p.status = dev->status;
  p.wait_limit_ns = kDefaultWaitNs;
  const int64_t ctas = divided ? all * splits : pair ? 2 * std::min<int64_t>(all, clusters) : std::min(all, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)k.block);
  cfg.dynamicSmemBytes = (size_t)k.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, divided ? (int)splits : k.ctas);
  cfg.attrs = attr;
  void* args[] = {&p};
  cudaError_t e = cudaLaunchKernelExC(&cfg, k.fn, args);
  if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "orthogonalisation product launch: %s", cudaGetErrorString(e));
  return MPG_OK;
}

}  // namespace

extern "C" {

size_t mpg_orthogonalize_workspace_size(int64_t m, int64_t n, int64_t batch) {
  if (m <= 0 || n <= 0 || batch <= 0 || m > kMaxExtent || n > kMaxExtent || batch > kMaxBatch) return 0;
  return layout(m, n, batch).bytes;
}

mpg_status mpg_orthogonalize(int64_t m, int64_t n, int64_t batch, const void* G, int64_t ldg, int64_t strideG,
                             mpg_dtype g_dtype, void* O, int64_t ldo, int64_t strideO, mpg_dtype o_dtype,
                             int32_t steps, const float* coeffs, float eps, float alpha, float beta, void* workspace,
                             size_t workspace_bytes, void* stream) {
  t_err.clear();
  if (m < 0 || n < 0 || batch < 0) return fail(MPG_ERR_INVALID_ARG, "negative size");
  if (m > kMaxExtent || n > kMaxExtent) return fail(MPG_ERR_INVALID_ARG, "size beyond 2^31-256");
  if (batch > kMaxBatch) return fail(MPG_ERR_INVALID_ARG, "more than 65535 matrices");
  if ((int)g_dtype < 0 || (int)g_dtype > 2 || (int)o_dtype < 0 || (int)o_dtype > 2)
    return fail(MPG_ERR_INVALID_ARG, "unknown dtype");
  if (steps < 1 || steps > kOrthoMaxSteps) return fail(MPG_ERR_INVALID_ARG, "steps %d outside [1, 100]", steps);
  if (!coeffs) return fail(MPG_ERR_INVALID_ARG, "NULL coefficients");
  if (!std::isfinite(coeffs[0]) || !std::isfinite(coeffs[1]) || !std::isfinite(coeffs[2]) || !std::isfinite(alpha) ||
      !std::isfinite(beta))
    return fail(MPG_ERR_INVALID_ARG, "a coefficient is not finite");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MPG_ERR_INVALID_ARG, "eps is negative or not finite");
  if (ldg < std::max<int64_t>(n, 1) || ldo < std::max<int64_t>(n, 1))
    return fail(MPG_ERR_INVALID_ARG, "leading dimension smaller than n");
  if (strideG < 0 || strideO < 0) return fail(MPG_ERR_INVALID_ARG, "negative batch stride");
  if (m == 0 || n == 0 || batch == 0) return MPG_OK;
  if (!G || !O) return fail(MPG_ERR_INVALID_ARG, "NULL operand");
  if (!aligned(G, (size_t)elem_bytes(g_dtype)) || !aligned(O, (size_t)elem_bytes(o_dtype)))
    return fail(MPG_ERR_INVALID_ARG, "operand not aligned to its element");
  if (strideG == 0) strideG = m * ldg;
  if (strideO == 0) strideO = m * ldo;
  // one after another, or side by side within the lines
  const bool apart = strideO >= (m - 1) * ldo + n || (strideO >= n && (batch - 1) * strideO + n <= ldo);
  if (batch > 1 && !apart) return fail(MPG_ERR_INVALID_ARG, "the matrices of O overlap");
  const Layout l = layout(m, n, batch);
  if (!workspace || workspace_bytes < l.bytes || !aligned(workspace, 16))
    return fail(MPG_ERR_WORKSPACE, "%zu workspace bytes needed (16-byte aligned), got %zu", l.bytes,
                workspace ? workspace_bytes : (size_t)0);
  DeviceInfo* dev = nullptr;
  mpg_status s = get_device(&dev);
  if (s != MPG_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* factor = reinterpret_cast<float*>(ws + l.factor);

  OrthoScaleParams sp;
  std::memset(&sp, 0, sizeof(sp));
  sp.g = G;
  sp.ldg = ldg;
  sp.stride_g = strideG;
  sp.rows = (int32_t)m;
  sp.cols = (int32_t)n;
  sp.batch = (int32_t)batch;
  const int64_t eg = elem_bytes(g_dtype);
  sp.g_vec = aligned(G, 16) && (ldg * eg) % 16 == 0 && (strideG * eg) % 16 == 0;
  sp.flat = ldg == n && l.ldx == n;
  sp.partial = reinterpret_cast<double*>(ws + l.partial);
  sp.x = reinterpret_cast<uint16_t*>(ws + l.x[0]);
  sp.ldx = l.ldx;
  sp.factor = factor;
  sp.steps = steps;
  for (int i = 0; i < 3; ++i) sp.coeff_size[i] = std::fabs(coeffs[i]);
  sp.store_exp = (int)std::lround(0.5 * std::log2((double)std::max(m, n)));
  // a norm near sqrt(m n) gives entries near 1; below 2^15, so that even a
  // single entry that holds the whole norm stays within fp16
  sp.target_exp = std::min((int)std::floor(0.5 * std::log2((double)m * (double)n)), 14);
  sp.eps = eps;
  // blocks that fill the machine (8 to an SM), of two chunks a thread at least
  const int64_t chunks = m * (l.ldx / 8);
  const int64_t fill = (8 * (int64_t)dev->sm_count + batch - 1) / batch;
  sp.blocks = (int32_t)std::max<int64_t>(1, std::min(std::min((chunks + 511) / 512, fill), (int64_t)kOrthoNormBlocks));
  cudaError_t e = launch_ortho_scale(sp, (int)g_dtype, st);
  if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "scaling launch: %s", cudaGetErrorString(e));

  const bool wide = m <= n;
  const int64_t side = l.side, length = std::max(m, n);
  const Matrix S{ws + l.s, l.lds, side}, B{ws + l.b, l.lds, side};
  for (int i = 0; i < steps; ++i) {
    const bool last = i == steps - 1;
    const float* here = factor + (int64_t)i * batch;
    const Matrix X{ws + l.x[i & 1], l.ldx, m}, Y{ws + l.x[(i & 1) ^ 1], l.ldx, m};
    OrthoGemmParams p;
    // S = X X^T (tall X: X^T X)
    std::memset(&p, 0, sizeof(p));
    p.batch = (int32_t)batch;
    p.m = p.n = (int32_t)side;
    p.k = (int32_t)length;
    p.a_mn_major = p.b_mn_major = !wide;
    if ((s = operand_map(&p.map_a, X, !wide, side, length, batch)) != MPG_OK) return s;
    p.map_b = p.map_a;
    p.symmetric = 1;
    p.d = S.ptr;
    p.ldd = S.ld;
    p.stride_d = side * S.ld;
    p.d_dtype = MPG_F16;
    p.vec = p.vec16 = 1;
    p.ca = 1.0f;
    p.factor = here;
    p.square = 1;
    if ((s = launch_gemm(dev, p, st)) != MPG_OK) return s;
    // B = b S + c S S
    std::memset(&p, 0, sizeof(p));
    p.batch = (int32_t)batch;
    p.m = p.n = p.k = (int32_t)side;
    if ((s = operand_map(&p.map_a, S, false, side, side, batch)) != MPG_OK) return s;
    p.map_b = p.map_a;
    p.symmetric = 1;
    p.z = static_cast<const uint16_t*>(S.ptr);
    p.ldz = S.ld;
    p.stride_z = side * S.ld;
    p.d = B.ptr;
    p.ldd = B.ld;
    p.stride_d = side * B.ld;
    p.d_dtype = MPG_F16;
    p.vec = p.vec16 = 1;
    p.ca = coeffs[2];
    p.cz = coeffs[1];
    if ((s = launch_gemm(dev, p, st)) != MPG_OK) return s;
    // X = a X + B X (tall X: X B)
    std::memset(&p, 0, sizeof(p));
    p.batch = (int32_t)batch;
    p.m = (int32_t)m;
    p.n = (int32_t)n;
    p.k = (int32_t)side;
    if (wide) {
      if ((s = operand_map(&p.map_a, B, false, m, side, batch)) != MPG_OK) return s;
      if ((s = operand_map(&p.map_b, X, true, n, side, batch)) != MPG_OK) return s;
      p.b_mn_major = 1;
    } else {
      if ((s = operand_map(&p.map_a, X, false, m, side, batch)) != MPG_OK) return s;
      if ((s = operand_map(&p.map_b, B, false, n, side, batch)) != MPG_OK) return s;
    }
    p.z = static_cast<const uint16_t*>(X.ptr);
    p.ldz = X.ld;
    p.stride_z = m * X.ld;
    p.ca = last ? alpha : 1.0f;
    p.cz = coeffs[0] * p.ca;
    p.factor = here;
    p.next = last ? nullptr : here + batch;
    if (last) {
      p.d = O;
      p.ldd = ldo;
      p.stride_d = strideO;
      p.d_dtype = (int32_t)o_dtype;
      p.co = beta;
      const size_t chunk = o_dtype == MPG_F32 ? 16 : 8;
      p.vec = aligned(O, chunk) && ldo % 4 == 0 && strideO % 4 == 0;
      p.vec16 = aligned(O, 16) && ldo % 8 == 0 && strideO % 8 == 0;
    } else {
      p.d = Y.ptr;
      p.ldd = Y.ld;
      p.stride_d = m * Y.ld;
      p.d_dtype = MPG_F16;
      p.vec = p.vec16 = 1;
    }
    if ((s = launch_gemm(dev, p, st)) != MPG_OK) return s;
  }
  return MPG_OK;
}

}  // extern "C"
