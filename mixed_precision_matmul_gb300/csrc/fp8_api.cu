// mpg_fp8_quantize and mpg_gemm_fp8: argument checks, the choice of the
// product's kernel and of its division along k, aligned copies of operands
// that TMA cannot describe, and the launches (fp8_quant.cu, fp8_gemm.cu).
#include <cstring>

#include "fp8.h"
#include "host.h"

using namespace mpg;

namespace {

// the last tile's end, and a block beyond it, still fit 32 bits
constexpr int64_t kMaxExtent = 0x7FFFFFFF - 255;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

bool tma_ok_bytes(const mpg_fp8_operand& x) {
  return aligned(x.data, 16) && x.ld % 16 == 0 && x.ld < (int64_t(1) << 40);
}

// A single line has no use for its leading dimension: any value will do.
mpg_fp8_operand one_line(mpg_fp8_operand x, int64_t rows, int64_t k) {
  if (rows == 1) x.ld = (k + 15) / 16 * 16;
  return x;
}

mpg_status check_operand(const mpg_fp8_operand* x, const char* name, int64_t rows, int64_t k) {
  if ((int)x->format < 0 || (int)x->format > 1)
    return fail(MPG_ERR_UNSUPPORTED, "%s: unknown 8-bit format %d", name, (int)x->format);
  if (x->scale_rows != 1 && x->scale_rows != kFp8Block)
    return fail(MPG_ERR_UNSUPPORTED, "%s: scale_rows %d is neither 1 nor 128", name, x->scale_rows);
  if (x->ld < k || x->ld < 1) return fail(MPG_ERR_INVALID_ARG, "%s: leading dimension smaller than k", name);
  if (x->scale_row_stride < 0 || x->scale_k_stride < 0)
    return fail(MPG_ERR_INVALID_ARG, "%s: negative scale stride", name);
  if (rows > 0 && k > 0) {
    if (!x->data || !x->scale) return fail(MPG_ERR_INVALID_ARG, "%s: NULL data or scale", name);
    if (!aligned(x->scale, 4)) return fail(MPG_ERR_INVALID_ARG, "%s: scale not aligned to 4 bytes", name);
  }
  return MPG_OK;
}

struct Copies {
  bool a = false, b = false;
  int64_t ld = 0;
  size_t off_b = 0, bytes = 0;
};
Copies plan_copies(int64_t m, int64_t n, int64_t k, const mpg_fp8_operand& A, const mpg_fp8_operand& B) {
  Copies c;
  c.a = !tma_ok_bytes(A);
  c.b = !tma_ok_bytes(B);
  c.ld = (k + 15) / 16 * 16;
  c.off_b = c.a ? align256((size_t)m * (size_t)c.ld) : 0;
  c.bytes = c.off_b + (c.b ? align256((size_t)n * (size_t)c.ld) : 0);
  return c;
}

// The product's tile and its division along k.
struct Fp8Plan {
  bool pair = false;      // 256 x 256 tiles on CTA pairs
  bool swapped = false;
  int bn = 128;
  int splits = 1;
};

struct FormCost {
  int64_t round, block;
};
constexpr int64_t kExchange = 7, kNarrowExchange = 4;   // blocks of k

// col_vec: a scale for each column (row of B).  room(s): clusters of s CTAs
// that find an SM for each CTA at a time.
template <class Room>
Fp8Plan plan_product(int64_t m, int64_t n, int64_t k, const mpg_options& o, bool col_vec, int sm_count, int clusters,
                     Room room) {
  Fp8Plan p;
  // Few tokens: the weights' rows fill the tensor core's 128 rows.
  p.swapped = m <= 64;
  p.bn = !p.swapped ? 128 : m <= 16 ? 16 : m <= 32 ? 32 : 64;
  if (o.tile_n) {
    p.swapped = o.tile_n < 128;
    p.bn = o.tile_n;
  }
  const int64_t rows = p.swapped ? n : m, cols = p.swapped ? m : n;
  const int64_t tiles = (rows + 127) / 128 * ((cols + p.bn - 1) / p.bn);
  const int64_t kb = blocks_of(k);
  int64_t s = 1;
  if (o.splitk > 0) {
    s = o.splitk;
  } else {
    // As many ranges as keep every CTA on an SM of its own, of two blocks at
    // least: 64 x 4096 x 4096 takes 17.9, 12.3, 9.6, 7.9 us with 1 .. 4 ranges
    // (128 CTAs) and 12.0 with 5 (160).  Of 128 x 128 tiles the exchange takes
    // as long as kExchange blocks: 256 x 4096 x 512 takes 7.1 us with two
    // ranges of two blocks and 5.2 with one, 256 x 4096 x 4096 12.0 and 14.6.
    // Of narrow tiles it takes about four: 1 x 8192 x 1024 4.6 and 4.7 us, 1 x
    // 8192 x 512 4.0 and 3.6, 1 x 8192 x 4096 7.7 and 11.3.
    // Clusters lie within a group of SMs, so large ones leave some unused: 64 x
    // 2048 x 8192 (16 tiles) takes 9.9 us with six ranges, 12.1 with eight.
    while (s < 8 && tiles * (s + 1) <= sm_count && kb / (s + 1) >= 2 && tiles <= room((int)s + 1)) ++s;
    if (kb - (kb + s - 1) / s <= (p.swapped ? kNarrowExchange : kExchange)) s = 1;
  }
  s = std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(s, 8), kb));
  const int64_t per = (kb + s - 1) / s;
  p.splits = (int)((kb + per - 1) / per);
  // The form that ends first, by what the forms take on a GB300 (ns): each
  // round of tiles, and each block of k in it.  One CTA's 128 x 128 tile keeps
  // the way to its SM busy for a block of k as long as a pair's 256 x 256 tile
  // does (32 KB either way), but a pair's SM has twice the additions to do, and
  // with a scale for each column those take longest.  With a scale for 128
  // columns 4096^3 takes 71 us on pairs and 86 on single CTAs, 4096 x 4096 x
  // 512 22 and 21; with one for each column (fp32 C) 125 and 117, 39 and 32.
  const int64_t pair_rounds = ((m + 255) / 256 * ((n + 255) / 256) + clusters - 1) / clusters;
  const int64_t rounds = (tiles * p.splits + sm_count - 1) / sm_count;
  const FormCost one = col_vec ? FormCost{1900, 460} : FormCost{1150, 355};
  const FormCost two = col_vec ? FormCost{5750, 730} : FormCost{3000, 420};
  const int64_t one_time = rounds * (one.round + one.block * (per + (p.splits > 1 ? kExchange : 0)));
  const int64_t pair_time = pair_rounds * (two.round + two.block * kb);
  if (o.cta_pair == 1 || (o.cta_pair == 0 && o.tile_n == 0 && o.splitk == 0 && !p.swapped && pair_time < one_time)) {
    p.pair = true;
    p.swapped = false;
    p.splits = 1;
  }
  return p;
}

mpg_status check_options(const mpg_options& o) {
  if (o.tile_n != 0 && o.tile_n != 16 && o.tile_n != 32 && o.tile_n != 64 && o.tile_n != 128)
    return fail(MPG_ERR_INVALID_ARG, "tile_n %d: 0, 16, 32, 64 or 128 for 8-bit operands", o.tile_n);
  if (o.cta_pair < -1 || o.cta_pair > 1) return fail(MPG_ERR_INVALID_ARG, "cta_pair %d outside [-1, 1]", o.cta_pair);
  if (o.cta_pair == 1 && (o.tile_n != 0 || o.splitk > 1))
    return fail(MPG_ERR_INVALID_ARG, "cta_pair 1 has 256 x 256 tiles and one range of k");
  if (o.splitk < 0 || o.splitk > 8) return fail(MPG_ERR_INVALID_ARG, "splitk %d outside [0, 8]", o.splitk);
  if (o.c_dtype < 0 || o.c_dtype > 2) return fail(MPG_ERR_INVALID_ARG, "unknown c_dtype %d", o.c_dtype);
  if (o.wait_timeout_ns < 0) return fail(MPG_ERR_INVALID_ARG, "negative wait_timeout_ns");
  return MPG_OK;
}

mpg_status launch_product(DeviceInfo* dev, int64_t m, int64_t n, int64_t k, const mpg_fp8_operand& A,
                          const mpg_fp8_operand& B, void* C, int64_t ldc, float alpha, float beta,
                          const mpg_options& o, cudaStream_t stream) {
  Fp8Kernel kern;
  fp8_lookup_pair(B.scale_rows == 1, &kern);
  int clusters = 0;
  mpg_status s = resident_clusters(dev, kern.fn, kern.block, kern.smem_bytes, 2, &clusters);
  if (s != MPG_OK) return s;
  // (the divided form of wide tiles has one CTA to an SM)
  Fp8Kernel wide;
  fp8_lookup(128, false, true, false, &wide);
  auto room = [&](int size) {
    int fit = 0;
    return resident_clusters(dev, wide.fn, wide.block, wide.smem_bytes, size, &fit) == MPG_OK ? fit : 0;
  };
  const Fp8Plan plan = plan_product(m, n, k, o, B.scale_rows == 1, dev->sm_count, clusters, room);
  const mpg_fp8_operand& R = plan.swapped ? B : A;
  const mpg_fp8_operand& S = plan.swapped ? A : B;
  if (!plan.pair) {
    if (!fp8_lookup(plan.bn, plan.swapped, plan.swapped || S.scale_rows == 1, !plan.swapped && plan.splits == 1, &kern))
      return fail(MPG_ERR_UNSUPPORTED, "no 8-bit kernel for tile_n %d", plan.bn);
    if ((s = allow_smem(dev, kern.fn, kern.smem_bytes)) != MPG_OK) return s;
  }
  Fp8GemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = (int32_t)(plan.swapped ? n : m);
  p.cols = (int32_t)(plan.swapped ? m : n);
  // (each CTA of a pair holds half of the tile's rows and half of its columns)
  s = encode_map_bytes(&p.map_r, R.data, R.ld, k, p.rows, kFp8Block, kern.tile_rows / (plan.pair ? 2 : 1));
  if (s != MPG_OK) return s;
  s = encode_map_bytes(&p.map_c, S.data, S.ld, k, p.cols, kFp8Block, kern.tile_cols / (plan.pair ? 2 : 1));
  if (s != MPG_OK) return s;
  p.sr = R.scale;
  p.sr_row = R.scale_row_stride;
  p.sr_k = R.scale_k_stride;
  p.sr_shift = R.scale_rows == 1 ? 0 : 7;
  p.sc = S.scale;
  p.sc_row = S.scale_row_stride;
  p.sc_k = S.scale_k_stride;
  p.sc_shift = S.scale_rows == 1 ? 0 : 7;
  p.out = C;
  p.ld_out = ldc;
  p.out_dtype = o.c_dtype;
  p.out_vec = aligned(C, o.c_dtype == MPG_F32 ? 16 : 8) && ldc % 4 == 0;
  p.out_vec16 = aligned(C, 16) && (ldc * elem_bytes((mpg_dtype)o.c_dtype)) % 16 == 0;
  p.num_r_blk = (p.rows + kern.tile_rows - 1) / kern.tile_rows;
  p.num_c_blk = (p.cols + kern.tile_cols - 1) / kern.tile_cols;
  p.num_k_blk = (int32_t)blocks_of(k);
  p.splits = plan.splits;
  p.kb_per_split = (p.num_k_blk + plan.splits - 1) / plan.splits;
  p.fmt_bits = ((uint32_t)R.format << 7) | ((uint32_t)S.format << 10);
  p.alpha = alpha;
  p.beta = beta;
  p.status = dev->status;
  p.wait_limit_ns = o.wait_timeout_ns ? (uint64_t)o.wait_timeout_ns : kDefaultWaitNs;
  const int64_t tiles = (int64_t)p.num_r_blk * p.num_c_blk;
  if (tiles * p.splits > kMaxExtent) return fail(MPG_ERR_INVALID_ARG, "too many tiles");
  p.num_tiles = (int32_t)tiles;
  p.group = 8;
  const int64_t ctas = plan.pair ? 2 * std::min<int64_t>(tiles, clusters)
                       : !plan.swapped && p.splits == 1 ? std::min<int64_t>(tiles, dev->sm_count) : tiles * p.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)kern.block);
  cfg.dynamicSmemBytes = (size_t)kern.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = (unsigned)launch_attributes(attr, plan.pair ? 2 : p.splits);
  cfg.attrs = attr;
  void* args[] = {&p};
  cudaError_t e = cudaLaunchKernelExC(&cfg, kern.fn, args);
  if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "8-bit product launch: %s", cudaGetErrorString(e));
  return MPG_OK;
}

}  // namespace

extern "C" {

mpg_status mpg_fp8_quantize(int64_t rows, int64_t cols, const void* X, int64_t ldx, mpg_dtype x_dtype,
                            mpg_fp8_format format, int32_t scale_rows, void* Q, int64_t ldq, float* S,
                            int64_t s_row_stride, int64_t s_k_stride, void* QT, int64_t ldqt, float* ST,
                            int64_t st_row_stride, int64_t st_k_stride, void* stream) {
  t_err.clear();
  if (rows < 0 || cols < 0) return fail(MPG_ERR_INVALID_ARG, "negative size");
  if (rows > kMaxExtent || cols > kMaxExtent) return fail(MPG_ERR_INVALID_ARG, "size beyond 2^31-256");
  if ((int)x_dtype < 0 || (int)x_dtype > 2) return fail(MPG_ERR_INVALID_ARG, "unknown dtype %d", (int)x_dtype);
  if ((int)format < 0 || (int)format > 1) return fail(MPG_ERR_UNSUPPORTED, "unknown 8-bit format %d", (int)format);
  if (scale_rows != 1 && scale_rows != kFp8Block)
    return fail(MPG_ERR_UNSUPPORTED, "scale_rows %d is neither 1 nor 128", scale_rows);
  if (ldx < cols) return fail(MPG_ERR_INVALID_ARG, "ldx smaller than cols");
  if (!Q && !QT) return fail(MPG_ERR_INVALID_ARG, "neither Q nor QT given");
  if (Q && (!S || ldq < cols)) return fail(MPG_ERR_INVALID_ARG, "Q needs S and ldq >= cols");
  if (QT && (!ST || ldqt < rows)) return fail(MPG_ERR_INVALID_ARG, "QT needs ST and ldqt >= rows");
  if ((Q && (s_row_stride < 0 || s_k_stride < 0)) || (QT && (st_row_stride < 0 || st_k_stride < 0)))
    return fail(MPG_ERR_INVALID_ARG, "negative scale stride");
  if (rows == 0 || cols == 0) return MPG_OK;
  if (!X) return fail(MPG_ERR_INVALID_ARG, "NULL operand");
  if (!aligned(X, (size_t)elem_bytes(x_dtype)) || !aligned(S, 4) || !aligned(ST, 4))
    return fail(MPG_ERR_INVALID_ARG, "pointer not aligned to its element");
  if (blocks_of(rows) * blocks_of(cols) > kMaxExtent) return fail(MPG_ERR_INVALID_ARG, "too many blocks");
  DeviceInfo* dev = nullptr;
  mpg_status s = get_device(&dev);
  if (s != MPG_OK) return s;
  Fp8QuantParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = X;
  p.ldx = ldx;
  p.rows = (int32_t)rows;
  p.cols = (int32_t)cols;
  p.x_align = 16;
  while (p.x_align > 2 && (!aligned(X, (size_t)p.x_align) || (ldx * elem_bytes(x_dtype)) % p.x_align != 0)) p.x_align /= 2;
  p.q = static_cast<uint8_t*>(Q);
  p.ldq = ldq;
  p.q_vec = aligned(Q, 8) && ldq % 8 == 0;
  p.s = S;
  p.s_row = s_row_stride;
  p.s_k = s_k_stride;
  p.qt = static_cast<uint8_t*>(QT);
  p.ldqt = ldqt;
  p.qt_vec = aligned(QT, 16) && ldqt % 16 == 0;
  p.st = ST;
  p.st_row = st_row_stride;
  p.st_k = st_k_stride;
  cudaError_t e = launch_fp8_quantize(p, (int)x_dtype, (int)format, scale_rows, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "quantiser launch: %s", cudaGetErrorString(e));
  return MPG_OK;
}

size_t mpg_gemm_fp8_workspace_size(int64_t m, int64_t n, int64_t k, const mpg_fp8_operand* A,
                                   const mpg_fp8_operand* B) {
  if (m <= 0 || n <= 0 || k <= 0 || m > kMaxExtent || n > kMaxExtent || k > kMaxExtent || !A || !B) return 0;
  return plan_copies(m, n, k, one_line(*A, m, k), one_line(*B, n, k)).bytes;
}

mpg_status mpg_gemm_fp8(int64_t m, int64_t n, int64_t k, const mpg_fp8_operand* A, const mpg_fp8_operand* B, void* C,
                        int64_t ldc, float alpha, float beta, void* workspace, size_t workspace_bytes, void* stream,
                        const mpg_options* opt) {
  t_err.clear();
  if (m < 0 || n < 0 || k < 0) return fail(MPG_ERR_INVALID_ARG, "negative size");
  if (m > kMaxExtent || n > kMaxExtent || k > kMaxExtent) return fail(MPG_ERR_INVALID_ARG, "size beyond 2^31-256");
  if (!A || !B) return fail(MPG_ERR_INVALID_ARG, "NULL operand description");
  mpg_options o;
  resolve_options(opt, &o);
  mpg_status s = check_options(o);
  if (s != MPG_OK) return s;
  if ((s = check_operand(A, "A", m, k)) != MPG_OK) return s;
  if ((s = check_operand(B, "B", n, k)) != MPG_OK) return s;
  if (ldc < n || ldc < 1) return fail(MPG_ERR_INVALID_ARG, "ldc smaller than n");
  if (m == 0 || n == 0) return MPG_OK;
  if (!C) return fail(MPG_ERR_INVALID_ARG, "NULL operand");
  if (!aligned(C, (size_t)elem_bytes((mpg_dtype)o.c_dtype)))
    return fail(MPG_ERR_INVALID_ARG, "C not aligned to its element");
  DeviceInfo* dev = nullptr;
  s = get_device(&dev);
  if (s != MPG_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (k == 0 || alpha == 0.0f) {
    cudaError_t e = launch_scale_c(C, o.c_dtype, ldc, m * ldc, (int32_t)m, (int32_t)n, 1, beta, st);
    if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "scale launch: %s", cudaGetErrorString(e));
    return MPG_OK;
  }
  mpg_fp8_operand Ax = one_line(*A, m, k), Bx = one_line(*B, n, k);
  const Copies cp = plan_copies(m, n, k, Ax, Bx);
  if (cp.bytes && (!workspace || workspace_bytes < cp.bytes || !aligned(workspace, 16)))
    return fail(MPG_ERR_WORKSPACE, "operands whose base or leading dimension is no multiple of 16 bytes need %zu "
                "workspace bytes (16-byte aligned), got %zu", cp.bytes, workspace ? workspace_bytes : (size_t)0);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (cp.a || cp.b) {
    auto copy = [&](bool wanted, mpg_fp8_operand& x, int64_t rows, uint8_t* to) {
      Fp8AlignJob j;
      std::memset(&j, 0, sizeof(j));
      if (!wanted) return j;
      j = Fp8AlignJob{static_cast<const uint8_t*>(x.data), x.ld, rows, k, cp.ld / 16, to, cp.ld};
      x.data = to;
      x.ld = cp.ld;
      return j;
    };
    const Fp8AlignJob ja = copy(cp.a, Ax, m, ws), jb = copy(cp.b, Bx, n, ws + cp.off_b);
    cudaError_t e = launch_fp8_align(ja, jb, dev->sm_count, st);
    if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "alignment copy launch: %s", cudaGetErrorString(e));
  }
  return launch_product(dev, m, n, k, Ax, Bx, C, ldc, alpha, beta, o, st);
}

}  // extern "C"
