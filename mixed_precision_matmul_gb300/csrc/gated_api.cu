// mpg_gated_gemm and mpg_gated_gemm_backward: argument checks, workspace
// layout, and the sequence of launches.
#include <algorithm>
#include <cstring>

#include "fused.h"

using namespace mpg;

namespace {

mpg_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t element, const char* name) {
  if (!p) return fail(MPG_ERR_INVALID_ARG, "NULL %s", name);
  if (!fused_aligned(p, element)) return fail(MPG_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  if (rows > 1 && ld < cols) return fail(MPG_ERR_INVALID_ARG, "leading dimension of %s smaller than its lines", name);
  return MPG_OK;
}

bool empty(const mpg_gated_layer* l) { return l->tokens == 0 || l->hidden == 0 || l->inner == 0; }

mpg_status check_layer(const mpg_gated_layer* l) {
  if (!l) return fail(MPG_ERR_INVALID_ARG, "NULL layer");
  if (l->tokens < 0 || l->hidden < 0 || l->inner < 0) return fail(MPG_ERR_INVALID_ARG, "negative size");
  if (l->tokens > kFusedMaxExtent || l->hidden > kFusedMaxExtent || l->inner > kFusedMaxExtent)
    return fail(MPG_ERR_INVALID_ARG, "size beyond 2^31-256");
  if (l->dtype != MPG_F16 && l->dtype != MPG_BF16) return fail(MPG_ERR_INVALID_ARG, "dtype must be fp16 or bf16");
  if ((int)l->act < 0 || (int)l->act > 2) return fail(MPG_ERR_INVALID_ARG, "unknown activation");
  if (empty(l)) return MPG_OK;
  mpg_status s;
  if ((s = check_matrix(l->x, l->ldx, l->tokens, l->hidden, 2, "X")) != MPG_OK) return s;
  if ((s = check_matrix(l->wg, l->ldwg, l->inner, l->hidden, 2, "Wg")) != MPG_OK) return s;
  return check_matrix(l->wu, l->ldwu, l->inner, l->hidden, 2, "Wu");
}

// An operand and the copy that stands for it where TMA cannot describe it.
struct Source {
  const void* ptr;
  int64_t ld, rows, cols;
  bool copy;
  size_t at;
};
Source source(const void* ptr, int64_t ld, int64_t rows, int64_t cols) {
  Source s{ptr, ld, rows, cols, false, 0};
  if (rows == 1) s.ld = fused_line(cols);           // (one line: no distance to the next)
  s.copy = !fused_lines_ok(ptr, s.ld);
  return s;
}

struct Layout {
  Source x, wg, wu;
  size_t dg, du, partial, top, slots, bytes;
  int64_t ldd;
};
FusedLaunch product(FusedEpi epi, int64_t m, int64_t n, int64_t k) {
  FusedLaunch l;
  l.epi = epi;
  l.m = m;
  l.n = n;
  l.k = k;
  return l;
}
FusedLaunch input_gradient(const mpg_gated_layer* l) {
  FusedLaunch g = product(FusedEpi::kPlain, l->tokens, l->hidden, l->inner);
  g.second_k = true;
  return g;
}
FusedLaunch weight_gradient(const mpg_gated_layer* l) {
  FusedLaunch g = product(FusedEpi::kPlain, l->inner, l->hidden, l->tokens);
  g.second_m = true;
  return g;
}
Layout layout(const mpg_gated_layer* l, bool backward) {
  Layout o;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align256(bytes);
    return r;
  };
  o.x = source(l->x, l->ldx, l->tokens, l->hidden);
  o.wg = source(l->wg, l->ldwg, l->inner, l->hidden);
  o.wu = source(l->wu, l->ldwu, l->inner, l->hidden);
  o.dg = o.du = o.partial = o.top = o.slots = 0;
  o.ldd = fused_wide_line(l->inner);
  // (few rows are multiplied in whole chunks of eight: zeros behind all of them, or none needed)
  const bool all = !backward && l->tokens <= kFewRows && l->hidden % 8 != 0;
  for (Source* s : {&o.x, &o.wg, &o.wu}) {
    s->copy = s->copy || all;
    if (s->copy) s->at = take((size_t)s->rows * (size_t)fused_wide_line(s->cols) * 2);
  }
  if (backward) {
    o.dg = take((size_t)l->tokens * (size_t)o.ldd * 2);
    o.du = take((size_t)l->tokens * (size_t)o.ldd * 2);
    o.partial = take(kScaleBlocks * sizeof(float));
    o.top = take((kTopParts + 1) * sizeof(float));
  }
  if (backward) {
    const FusedLaunch to_x = input_gradient(l), to_w = weight_gradient(l);
    o.slots = take(std::max(fused_slot_bytes(to_x, &to_w), fused_slot_bytes(product(FusedEpi::kGatedGrad, l->tokens, l->inner, l->hidden))));
  } else if (l->tokens > kFewRows)
    o.slots = take(fused_slot_bytes(product(FusedEpi::kGated, l->tokens, l->inner, l->hidden)));
  o.bytes = at;
  return o;
}

// Copies what has to be copied and puts the copies in place.
mpg_status make_copies(DeviceInfo* dev, std::initializer_list<Source*> list, uint8_t* ws, cudaStream_t stream) {
  PadParams p;
  std::memset(&p, 0, sizeof(p));
  for (Source* s : list) {
    if (!s->copy) continue;
    const int64_t ld = fused_wide_line(s->cols);
    p.mat[p.count++] = PadParams::Matrix{static_cast<const uint16_t*>(s->ptr), reinterpret_cast<uint16_t*>(ws + s->at), s->ld,
                                         ld, s->rows, s->cols};
    s->ptr = ws + s->at;
    s->ld = ld;
  }
  if (!p.count) return MPG_OK;
  const cudaError_t e = launch_pad(p, dev->sm_count, stream);
  return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "copy launch: %s", cudaGetErrorString(e));
}

mpg_status check_workspace(const Layout& o, const void* ws, size_t bytes) {
  if (o.bytes && (!ws || bytes < o.bytes || !fused_aligned(ws, 16)))
    return fail(MPG_ERR_WORKSPACE, "%zu workspace bytes needed (16-byte aligned), got %zu", o.bytes, ws ? bytes : (size_t)0);
  return MPG_OK;
}

}  // namespace

extern "C" {

size_t mpg_gated_gemm_workspace_size(const mpg_gated_layer* layer) {
  t_err.clear();
  if (check_layer(layer) != MPG_OK || empty(layer)) return 0;
  return layout(layer, false).bytes;
}

mpg_status mpg_gated_gemm(const mpg_gated_layer* layer, void* Y, int64_t ldy, void* A, int64_t lda, void* B, int64_t ldb,
                          void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  mpg_status s = check_layer(layer);
  if (s != MPG_OK) return s;
  const mpg_gated_layer& l = *layer;
  if ((A == nullptr) != (B == nullptr)) return fail(MPG_ERR_INVALID_ARG, "A and B are kept together");
  if (l.tokens == 0 || l.inner == 0) return MPG_OK;
  if ((s = check_matrix(Y, ldy, l.tokens, l.inner, 2, "Y")) != MPG_OK) return s;
  if (A && (s = check_matrix(A, lda, l.tokens, l.inner, 2, "A")) != MPG_OK) return s;
  if (B && (s = check_matrix(B, ldb, l.tokens, l.inner, 2, "B")) != MPG_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (l.hidden == 0) {
    // sums of nothing: act(0) * 0
    DeviceInfo* dev = nullptr;
    if ((s = get_device(&dev)) != MPG_OK) return s;
    const struct { void* p; int64_t ld; } out[3] = {{Y, ldy}, {A, lda}, {B, ldb}};
    for (const auto& o : out) {
      if (!o.p) continue;
      const cudaError_t e = cudaMemset2DAsync(o.p, (size_t)(l.tokens > 1 ? o.ld : l.inner) * 2, 0, (size_t)l.inner * 2,
                                              (size_t)l.tokens, st);
      if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "zero fill: %s", cudaGetErrorString(e));
    }
    return MPG_OK;
  }
  Layout o = layout(layer, false);
  if ((s = check_workspace(o, workspace, workspace_bytes)) != MPG_OK) return s;
  DeviceInfo* dev = nullptr;
  if ((s = get_device(&dev)) != MPG_OK) return s;

  if ((s = make_copies(dev, {&o.x, &o.wg, &o.wu}, static_cast<uint8_t*>(workspace), st)) != MPG_OK) return s;
  if (l.tokens <= kFewRows) {
    FewRowsParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = o.x.ptr;
    p.ldx = o.x.ld;
    p.w = o.wg.ptr;
    p.ldw = o.wg.ld;
    p.wu = o.wu.ptr;
    p.ldwu = o.wu.ld;
    p.bf16 = l.dtype == MPG_BF16;
    p.rows = (int32_t)l.tokens;
    p.n = (int32_t)l.inner;
    p.k = (int32_t)fused_line(l.hidden);
    p.act = (int32_t)l.act;
    p.y = Y;
    p.ldy = ldy;
    p.ka = A;
    p.lda = lda;
    p.kb = B;
    p.ldb = ldb;
    return launch_few_rows(dev, p, FusedEpi::kGated, st);
  }

  FusedGemmParams p;
  std::memset(&p, 0, sizeof(p));
  if ((s = fused_map(&p.prod[0].map_a[0], o.x.ptr, o.x.ld, l.dtype, false, l.tokens, l.hidden)) != MPG_OK) return s;
  if ((s = fused_map(&p.prod[0].map_b[0], o.wg.ptr, o.wg.ld, l.dtype, false, l.inner, l.hidden)) != MPG_OK) return s;
  if ((s = fused_map(&p.prod[0].map_b[1], o.wu.ptr, o.wu.ld, l.dtype, false, l.inner, l.hidden)) != MPG_OK) return s;
  p.bf16 = l.dtype == MPG_BF16;
  p.act = (int32_t)l.act;
  void* const out[3] = {Y, A, B};
  const int64_t ld[3] = {ldy, lda, ldb};
  for (int i = 0; i < 3; ++i) {
    p.prod[0].out[i] = out[i];
    p.prod[0].ldo[i] = ld[i];
    p.prod[0].out_vec[i] = fused_lines_ok(out[i], ld[i]);
  }
  return launch_fused(dev, product(FusedEpi::kGated, l.tokens, l.inner, l.hidden), p,
                      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + o.slots), st);
}

size_t mpg_gated_gemm_backward_workspace_size(const mpg_gated_layer* layer) {
  t_err.clear();
  if (check_layer(layer) != MPG_OK || empty(layer)) return 0;
  return layout(layer, true).bytes;
}

mpg_status mpg_gated_gemm_backward(const mpg_gated_layer* layer, const void* dY, int64_t lddy, const void* A, int64_t lda,
                                   const void* B, int64_t ldb, void* dX, int64_t lddx, void* dWg, int64_t lddwg, void* dWu,
                                   int64_t lddwu, void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  mpg_status s = check_layer(layer);
  if (s != MPG_OK) return s;
  const mpg_gated_layer& l = *layer;
  if ((A == nullptr) != (B == nullptr)) return fail(MPG_ERR_INVALID_ARG, "A and B are kept together");
  if ((dWg == nullptr) != (dWu == nullptr)) return fail(MPG_ERR_INVALID_ARG, "dWg and dWu are made together");
  if (l.hidden == 0) return MPG_OK;                 // (gradients without elements)
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dX && l.tokens && (s = check_matrix(dX, lddx, l.tokens, l.hidden, 2, "dX")) != MPG_OK) return s;
  if (dWg && l.inner && (s = check_matrix(dWg, lddwg, l.inner, l.hidden, 2, "dWg")) != MPG_OK) return s;
  if (dWu && l.inner && (s = check_matrix(dWu, lddwu, l.inner, l.hidden, 2, "dWu")) != MPG_OK) return s;
  if (!dX && !dWg) return MPG_OK;
  DeviceInfo* dev = nullptr;
  if (empty(layer)) {
    // no tokens or no inner values: the gradients are sums of nothing
    if ((s = get_device(&dev)) != MPG_OK) return s;
    const struct { void* p; int64_t ld, rows; } out[3] = {{dX, lddx, l.tokens}, {dWg, lddwg, l.inner}, {dWu, lddwu, l.inner}};
    for (const auto& o : out) {
      if (!o.p || !o.rows) continue;
      const cudaError_t e = cudaMemset2DAsync(o.p, (size_t)(o.rows > 1 ? o.ld : l.hidden) * 2, 0, (size_t)l.hidden * 2,
                                              (size_t)o.rows, st);
      if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "zero fill: %s", cudaGetErrorString(e));
    }
    return MPG_OK;
  }
  if ((s = check_matrix(dY, lddy, l.tokens, l.inner, 2, "dY")) != MPG_OK) return s;
  if (A && (s = check_matrix(A, lda, l.tokens, l.inner, 2, "A")) != MPG_OK) return s;
  if (B && (s = check_matrix(B, ldb, l.tokens, l.inner, 2, "B")) != MPG_OK) return s;
  Layout o = layout(layer, true);
  if ((s = check_workspace(o, workspace, workspace_bytes)) != MPG_OK) return s;
  if ((s = get_device(&dev)) != MPG_OK) return s;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* partial = reinterpret_cast<float*>(ws + o.partial);
  float* top = reinterpret_cast<float*>(ws + o.top);
  float* slots = reinterpret_cast<float*>(ws + o.slots);
  uint16_t* dg = reinterpret_cast<uint16_t*>(ws + o.dg);
  uint16_t* du = reinterpret_cast<uint16_t*>(ws + o.du);
  if ((s = make_copies(dev, {&o.x, &o.wg, &o.wu}, ws, st)) != MPG_OK) return s;

  // fp16: dgate and dup carry a power of two that brings the largest of dY to
  // [2^4, 2^5), which leaves 2^11 above for what they are multiplied by, and 18 bits
  // below before values lose precision.  Where the largest of them leaves fp16
  // (or all are small) they are made again with a scale from themselves (see GradTop):
  // a second launch, which ends at once where nothing is to be done: 1 to 5 us
  // (17 x 2048 x 5632 recomputed 47 -> 50, 2048 x 2048 x 5504 186 -> 188).  A bound
  // beforehand costs two more reads of what was kept, or a read of the operands.
  const bool half = l.dtype == MPG_F16;
  constexpr int kExp = 4;
  if (half) {
    MaxParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = dY;
    p.ld = lddy;
    p.rows = l.tokens;
    p.cols = l.inner;
    p.vec = fused_lines_ok(dY, l.tokens > 1 ? lddy : 0);
    p.flat = p.vec && l.inner % 8 == 0 && (lddy == l.inner || l.tokens == 1);
    p.partial = partial;
    p.top = top;
    const cudaError_t e = launch_max(p, st);
    if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "maximum launch: %s", cudaGetErrorString(e));
  }
  for (int pass = 0; pass < (half ? 2 : 1); ++pass) {
    float* record = half && !pass ? top : nullptr;
    float* again = pass ? top : nullptr;
    if (A) {
      GatedGradParams p;
      std::memset(&p, 0, sizeof(p));
      p.dy = dY;
      p.lddy = lddy;
      p.a = A;
      p.lda = lda;
      p.b = B;
      p.ldb = ldb;
      p.dg = dg;
      p.du = du;
      p.ldd = o.ldd;
      p.rows = l.tokens;
      p.cols = l.inner;
      p.vec = fused_lines_ok(dY, lddy) && fused_lines_ok(A, lda) && fused_lines_ok(B, ldb);
      p.bf16 = l.dtype == MPG_BF16;
      p.scale = half ? partial : nullptr;
      p.scale_count = kScaleBlocks;
      p.scale_exp = kExp;
      p.record = record;
      p.again = again;
      const cudaError_t e = launch_gated_grad(p, dev->sm_count, st);
      if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "gradient launch: %s", cudaGetErrorString(e));
    } else if (l.tokens <= kFewRows && (l.hidden % 8 == 0 || (o.x.copy && o.wg.copy && o.wu.copy))) {
      // (lines of whole chunks of eight, or copies with zeros behind them)
      FewRowsParams p;
      std::memset(&p, 0, sizeof(p));
      p.x = o.x.ptr;
      p.ldx = o.x.ld;
      p.w = o.wg.ptr;
      p.ldw = o.wg.ld;
      p.wu = o.wu.ptr;
      p.ldwu = o.wu.ld;
      p.bf16 = !half;
      p.rows = (int32_t)l.tokens;
      p.n = (int32_t)l.inner;
      p.k = (int32_t)fused_line(l.hidden);
      p.act = (int32_t)l.act;
      p.y = dg;
      p.ka = du;
      p.ldy = p.lda = o.ldd;
      p.dy = dY;
      p.lddy = lddy;
      p.scale = half ? partial : nullptr;
      p.scale_count = kScaleBlocks;
      p.scale_exp = kExp;
      p.record = record;
      p.again = again;
      if ((s = launch_few_rows(dev, p, FusedEpi::kGatedGrad, st)) != MPG_OK) return s;
    } else {
      FusedGemmParams p;
      std::memset(&p, 0, sizeof(p));
      if ((s = fused_map(&p.prod[0].map_a[0], o.x.ptr, o.x.ld, l.dtype, false, l.tokens, l.hidden)) != MPG_OK) return s;
      if ((s = fused_map(&p.prod[0].map_b[0], o.wg.ptr, o.wg.ld, l.dtype, false, l.inner, l.hidden)) != MPG_OK) return s;
      if ((s = fused_map(&p.prod[0].map_b[1], o.wu.ptr, o.wu.ld, l.dtype, false, l.inner, l.hidden)) != MPG_OK) return s;
      p.bf16 = l.dtype == MPG_BF16;
      p.act = (int32_t)l.act;
      p.prod[0].out[0] = dg;
      p.prod[0].out[1] = du;
      p.prod[0].ldo[0] = p.prod[0].ldo[1] = o.ldd;
      p.prod[0].out_vec[0] = p.prod[0].out_vec[1] = 1;
      p.dy = dY;
      p.lddy = lddy;
      p.dy_vec = fused_lines_ok(dY, lddy);
      p.scale = half ? partial : nullptr;
      p.scale_count = kScaleBlocks;
      p.scale_exp = kExp;
      p.record = record;
      p.again = again;
      if ((s = launch_fused(dev, product(FusedEpi::kGatedGrad, l.tokens, l.inner, l.hidden), p, slots, st)) != MPG_OK) return s;
    }
  }
  FusedGemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.bf16 = !half;
  // (the factor that dgate and dup carry, as it was left)
  const float* factor = half ? top + kTopParts : nullptr;
  p.scale = factor;
  p.scale_count = p.scale_largest = 1;
  const void* const d[2] = {dg, du};
  int count = 0;
  if (dX) {
    // dX = dgate Wg + dup Wu
    FusedProduct& x = p.prod[count++];
    const Source* const w[2] = {&o.wg, &o.wu};
    for (int i = 0; i < 2; ++i) {
      if ((s = fused_map(&x.map_a[i], d[i], o.ldd, l.dtype, false, l.tokens, l.inner)) != MPG_OK) return s;
      if ((s = fused_map(&x.map_b[i], w[i]->ptr, w[i]->ld, l.dtype, true, l.hidden, l.inner)) != MPG_OK) return s;
    }
    x.b_mn_major = 1;
    x.out[0] = dX;
    x.ldo[0] = lddx;
    x.out_vec[0] = fused_lines_ok(dX, lddx);
    x.out_dtype = (int32_t)l.dtype;
  }
  // (elements of lines off 16 bytes are written faster by the tiles' epilogue)
  const bool few = dWg && l.tokens <= kFewGradTokens && l.inner <= kFewGradRows && fused_lines_ok(dWg, lddwg) && fused_lines_ok(dWu, lddwu);
  if (dWg && !few) {
    // dWg = dgate^T X, dWu = dup^T X
    FusedProduct& w = p.prod[count++];
    for (int i = 0; i < 2; ++i)
      if ((s = fused_map(&w.map_a[i], d[i], o.ldd, l.dtype, true, l.inner, l.tokens)) != MPG_OK) return s;
    if ((s = fused_map(&w.map_b[0], o.x.ptr, o.x.ld, l.dtype, true, l.hidden, l.tokens)) != MPG_OK) return s;
    w.a_mn_major = w.b_mn_major = 1;
    w.out[0] = dWg;
    w.out[1] = dWu;
    w.ldo[0] = lddwg;
    w.ldo[1] = lddwu;
    w.out_vec[0] = fused_lines_ok(dWg, lddwg);
    w.out_vec[1] = fused_lines_ok(dWu, lddwu);
    w.out_dtype = (int32_t)l.dtype;
  }
  if (few) {
    if (dX && (s = launch_fused(dev, input_gradient(layer), p, slots, st)) != MPG_OK) return s;
    FewGradParams w;
    std::memset(&w, 0, sizeof(w));
    w.d[0] = dg;
    w.d[1] = du;
    w.x = static_cast<const uint16_t*>(o.x.ptr);
    w.ldd = o.ldd;
    w.ldx = o.x.ld;
    w.tokens = (int32_t)l.tokens;
    w.rows = (int32_t)l.inner;
    w.cols = (int32_t)l.hidden;
    w.count = 2;
    w.bf16 = !half;
    w.out[0] = dWg;
    w.out[1] = dWu;
    w.ldo[0] = lddwg;
    w.ldo[1] = lddwu;
    w.scale = factor;
    w.scale_count = w.scale_largest = 1;
    const cudaError_t e = launch_few_grad(w, st);
    return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "weight gradient launch: %s", cudaGetErrorString(e));
  }
  if (count == 2) return launch_fused_two(dev, input_gradient(layer), weight_gradient(layer), p, slots, st);
  return launch_fused(dev, dX ? input_gradient(layer) : weight_gradient(layer), p, slots, st);
}

}  // extern "C"
