// mpg_linear_cross_entropy and mpg_linear_cross_entropy_backward: argument
// checks, workspace layout, and the sequence of launches.
#include <algorithm>
#include <cstring>

#include "fused.h"

using namespace mpg;

namespace {

// Bytes of the logits' gradient that is held at a time.  More and smaller pieces
// cost the fp32 sums of dX another way through memory each, fewer and larger
// ones memory.
constexpr int64_t kPieceBytes = 512ll << 20;

mpg_status check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, const char* name) {
  if (!p) return fail(MPG_ERR_INVALID_ARG, "NULL %s", name);
  if (!fused_aligned(p, 2)) return fail(MPG_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
  if (rows > 1 && ld < cols) return fail(MPG_ERR_INVALID_ARG, "leading dimension of %s smaller than its lines", name);
  return MPG_OK;
}

mpg_status check_loss(const mpg_vocab_loss* l) {
  if (!l) return fail(MPG_ERR_INVALID_ARG, "NULL description");
  if (l->tokens < 0 || l->hidden < 0 || l->vocab < 0) return fail(MPG_ERR_INVALID_ARG, "negative size");
  if (l->tokens > kFusedMaxExtent || l->hidden > kFusedMaxExtent || l->vocab > kFusedMaxExtent)
    return fail(MPG_ERR_INVALID_ARG, "size beyond 2^31-256");
  if (l->dtype != MPG_F16 && l->dtype != MPG_BF16) return fail(MPG_ERR_INVALID_ARG, "dtype must be fp16 or bf16");
  if (l->target_bytes != 4 && l->target_bytes != 8) return fail(MPG_ERR_INVALID_ARG, "targets have 4 or 8 bytes");
  if (l->hidden == 0 || l->vocab == 0) return fail(MPG_ERR_INVALID_ARG, "logits need a hidden size and classes");
  if (l->tokens == 0) return MPG_OK;
  if (!l->target || !fused_aligned(l->target, (size_t)l->target_bytes)) return fail(MPG_ERR_INVALID_ARG, "NULL or misaligned targets");
  mpg_status s;
  if ((s = check_matrix(l->x, l->ldx, l->tokens, l->hidden, "X")) != MPG_OK) return s;
  return check_matrix(l->w, l->ldw, l->vocab, l->hidden, "W");
}

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
  Source x, w;
  size_t stats, target_logit, grad, sum, partial, slots, bytes;
  int64_t piece, pieces, ldsum;
};
FusedLaunch product(FusedEpi epi, int64_t m, int64_t n, int64_t k) {
  FusedLaunch l;
  l.epi = epi;
  l.m = m;
  l.n = n;
  l.k = k;
  return l;
}
Layout layout(const mpg_vocab_loss* l, bool backward) {
  Layout o;
  std::memset(static_cast<void*>(&o), 0, sizeof(o));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align256(bytes);
    return r;
  };
  const int64_t t = l->tokens;
  o.x = source(l->x, l->ldx, t, l->hidden);
  o.w = source(l->w, l->ldw, l->vocab, l->hidden);
  // (few rows are multiplied in whole chunks of eight: zeros behind all of them, or none needed)
  const bool all = !backward && t <= kFewRows && l->hidden % 8 != 0;
  for (Source* s : {&o.x, &o.w}) {
    s->copy = s->copy || all;
    if (s->copy) s->at = take((size_t)s->rows * (size_t)fused_wide_line(s->cols) * 2);
  }
  if (!backward) {
    const int64_t parts = t <= kFewRows ? few_rows_parts(l->vocab) : 2 * ((l->vocab + 127) / 128);
    o.stats = take((size_t)parts * (size_t)t * sizeof(float2));
    o.target_logit = take((size_t)t * sizeof(float));
    if (t > kFewRows) o.slots = take(fused_slot_bytes(product(FusedEpi::kStats, t, l->vocab, l->hidden)));
  } else {
    int64_t piece = std::max<int64_t>(256, kPieceBytes / 2 / t / 256 * 256);
    o.pieces = (l->vocab + piece - 1) / piece;
    piece = ((l->vocab + o.pieces - 1) / o.pieces + 255) / 256 * 256;
    o.pieces = (l->vocab + piece - 1) / piece;
    o.piece = std::min(piece, fused_wide_line(l->vocab));
    o.grad = take((size_t)t * (size_t)o.piece * 2);
    o.ldsum = (l->hidden + 3) / 4 * 4;
    if (o.pieces > 1) o.sum = take((size_t)t * (size_t)o.ldsum * sizeof(float));
    o.partial = take(kScaleBlocks * sizeof(float));
    const FusedLaunch to_x = product(FusedEpi::kPlain, t, l->hidden, o.piece), to_w = product(FusedEpi::kPlain, o.piece, l->hidden, t);
    o.slots = take(std::max(fused_slot_bytes(to_x, &to_w), fused_slot_bytes(product(FusedEpi::kProb, t, o.piece, l->hidden))));
  }
  o.bytes = at;
  return o;
}

mpg_status make_copies(DeviceInfo* dev, Layout& o, uint8_t* ws, cudaStream_t stream) {
  PadParams p;
  std::memset(&p, 0, sizeof(p));
  for (Source* s : {&o.x, &o.w}) {
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
  if (!ws || bytes < o.bytes || !fused_aligned(ws, 16))
    return fail(MPG_ERR_WORKSPACE, "%zu workspace bytes needed (16-byte aligned), got %zu", o.bytes, ws ? bytes : (size_t)0);
  return MPG_OK;
}

}  // namespace

extern "C" {

size_t mpg_linear_cross_entropy_workspace_size(const mpg_vocab_loss* loss) {
  t_err.clear();
  if (check_loss(loss) != MPG_OK || loss->tokens == 0) return 0;
  return layout(loss, false).bytes;
}

mpg_status mpg_linear_cross_entropy(const mpg_vocab_loss* desc, float* loss, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  t_err.clear();
  mpg_status s = check_loss(desc);
  if (s != MPG_OK) return s;
  const mpg_vocab_loss& l = *desc;
  if (l.tokens == 0) return MPG_OK;
  if (!loss || !lse || !fused_aligned(loss, 4) || !fused_aligned(lse, 4))
    return fail(MPG_ERR_INVALID_ARG, "NULL or misaligned loss or lse");
  Layout o = layout(desc, false);
  if ((s = check_workspace(o, workspace, workspace_bytes)) != MPG_OK) return s;
  DeviceInfo* dev = nullptr;
  if ((s = get_device(&dev)) != MPG_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float2* stats = reinterpret_cast<float2*>(ws + o.stats);
  float* target_logit = reinterpret_cast<float*>(ws + o.target_logit);
  LossJoinParams j;
  std::memset(&j, 0, sizeof(j));

  if ((s = make_copies(dev, o, ws, st)) != MPG_OK) return s;
  if (l.tokens <= kFewRows) {
    FewRowsParams p;
    std::memset(&p, 0, sizeof(p));
    p.x = o.x.ptr;
    p.ldx = o.x.ld;
    p.w = o.w.ptr;
    p.ldw = o.w.ld;
    p.bf16 = l.dtype == MPG_BF16;
    p.rows = (int32_t)l.tokens;
    p.n = (int32_t)l.vocab;
    p.k = (int32_t)fused_line(l.hidden);
    p.target = l.target;
    p.target_bytes = l.target_bytes;
    p.target_stride = l.target_stride;
    p.ignore_index = l.ignore_index;
    p.vocab = (int32_t)l.vocab;
    p.stats = stats;
    p.target_logit = target_logit;
    if ((s = launch_few_rows(dev, p, FusedEpi::kStats, st)) != MPG_OK) return s;
    j.parts = few_rows_parts(l.vocab);
  } else {
    FusedGemmParams p;
    std::memset(&p, 0, sizeof(p));
    if ((s = fused_map(&p.prod[0].map_a[0], o.x.ptr, o.x.ld, l.dtype, false, l.tokens, l.hidden)) != MPG_OK) return s;
    if ((s = fused_map(&p.prod[0].map_b[0], o.w.ptr, o.w.ld, l.dtype, false, l.vocab, l.hidden)) != MPG_OK) return s;
    p.bf16 = l.dtype == MPG_BF16;
    p.target = l.target;
    p.target_bytes = l.target_bytes;
    p.target_stride = l.target_stride;
    p.ignore_index = l.ignore_index;
    p.vocab = (int32_t)l.vocab;
    p.stats = stats;
    p.target_logit = target_logit;
    if ((s = launch_fused(dev, product(FusedEpi::kStats, l.tokens, l.vocab, l.hidden), p,
                          reinterpret_cast<float*>(ws + o.slots), st)) != MPG_OK) return s;
    j.parts = 2 * p.prod[0].num_n_blk;
  }
  j.stats = stats;
  j.rows = l.tokens;
  j.target_logit = target_logit;
  j.target = l.target;
  j.target_bytes = l.target_bytes;
  j.target_stride = l.target_stride;
  j.ignore_index = l.ignore_index;
  j.vocab = l.vocab;
  j.loss = loss;
  j.lse = lse;
  const cudaError_t e = launch_loss_join(j, st);
  return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "loss launch: %s", cudaGetErrorString(e));
}

size_t mpg_linear_cross_entropy_backward_workspace_size(const mpg_vocab_loss* loss) {
  t_err.clear();
  if (check_loss(loss) != MPG_OK || loss->tokens == 0) return 0;
  return layout(loss, true).bytes;
}

mpg_status mpg_linear_cross_entropy_backward(const mpg_vocab_loss* desc, const float* lse, const float* dloss,
                                             int64_t dloss_stride, void* dX, int64_t lddx, void* dW, int64_t lddw,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  mpg_status s = check_loss(desc);
  if (s != MPG_OK) return s;
  const mpg_vocab_loss& l = *desc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dX && l.tokens && (s = check_matrix(dX, lddx, l.tokens, l.hidden, "dX")) != MPG_OK) return s;
  if (dW && (s = check_matrix(dW, lddw, l.vocab, l.hidden, "dW")) != MPG_OK) return s;
  if (!dX && !dW) return MPG_OK;
  DeviceInfo* dev = nullptr;
  if (l.tokens == 0) {
    // a gradient of W without tokens is a sum of nothing
    if (!dW) return MPG_OK;
    if ((s = get_device(&dev)) != MPG_OK) return s;
    const cudaError_t e = cudaMemset2DAsync(dW, (size_t)(l.vocab > 1 ? lddw : l.hidden) * 2, 0, (size_t)l.hidden * 2,
                                            (size_t)l.vocab, st);
    return e == cudaSuccess ? MPG_OK : fail(MPG_ERR_CUDA, "zero fill: %s", cudaGetErrorString(e));
  }
  if (!lse || !dloss || !fused_aligned(lse, 4) || !fused_aligned(dloss, 4))
    return fail(MPG_ERR_INVALID_ARG, "NULL or misaligned lse or dloss");
  Layout o = layout(desc, true);
  if ((s = check_workspace(o, workspace, workspace_bytes)) != MPG_OK) return s;
  if ((s = get_device(&dev)) != MPG_OK) return s;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* partial = reinterpret_cast<float*>(ws + o.partial);
  float* slots = reinterpret_cast<float*>(ws + o.slots);
  float* sum = reinterpret_cast<float*>(ws + o.sum);
  uint16_t* grad = reinterpret_cast<uint16_t*>(ws + o.grad);
  if ((s = make_copies(dev, o, ws, st)) != MPG_OK) return s;

  // The logits' gradient is divided by the largest dloss; in fp16 it is multiplied
  // by 2^14 too: no element is larger, and a probability of 2^-28 is still a normal
  // number.
  const bool half = l.dtype == MPG_F16;
  const int exp = half ? 14 : 0;
  // (one weight for all tokens is the largest: ignored ones have no gradient at all)
  const bool same = dloss_stride == 0 || l.tokens == 1;
  const float* scale = same ? dloss : partial;
  if (!same) {
    MaxParams p;
    std::memset(&p, 0, sizeof(p));
    p.rows = l.tokens;
    p.dloss = dloss;
    p.dloss_stride = dloss_stride;
    p.target = l.target;
    p.target_bytes = l.target_bytes;
    p.target_stride = l.target_stride;
    p.ignore_index = l.ignore_index;
    p.partial = partial;
    const cudaError_t e = launch_max(p, st);
    if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "maximum launch: %s", cudaGetErrorString(e));
  }
  for (int64_t i = 0; i < o.pieces; ++i) {
    const int64_t c0 = i * o.piece, cols = std::min(o.piece, l.vocab - c0);
    const uint16_t* w = static_cast<const uint16_t*>(o.w.ptr) + c0 * o.w.ld;
    FusedGemmParams p;
    std::memset(&p, 0, sizeof(p));
    if (l.tokens <= kFewRows && (l.hidden % 8 == 0 || (o.x.copy && o.w.copy))) {
      // (lines of whole chunks of eight, or copies with zeros behind them)
      FewRowsParams r;
      std::memset(&r, 0, sizeof(r));
      r.x = o.x.ptr;
      r.ldx = o.x.ld;
      r.w = w;
      r.ldw = o.w.ld;
      r.bf16 = !half;
      r.rows = (int32_t)l.tokens;
      r.n = (int32_t)cols;
      r.k = (int32_t)fused_line(l.hidden);
      r.y = grad;
      r.ldy = o.piece;
      r.target = l.target;
      r.target_bytes = l.target_bytes;
      r.target_stride = l.target_stride;
      r.ignore_index = l.ignore_index;
      r.col0 = (int32_t)c0;
      r.vocab = (int32_t)l.vocab;
      r.lse = lse;
      r.dloss = dloss;
      r.dloss_stride = dloss_stride;
      r.scale = scale;
      r.scale_count = same ? 1 : kScaleBlocks;
      r.scale_exp = exp;
      r.scale_largest = 1;
      if ((s = launch_few_rows(dev, r, FusedEpi::kProb, st)) != MPG_OK) return s;
    } else {
      if ((s = fused_map(&p.prod[0].map_a[0], o.x.ptr, o.x.ld, l.dtype, false, l.tokens, l.hidden)) != MPG_OK) return s;
      if ((s = fused_map(&p.prod[0].map_b[0], w, o.w.ld, l.dtype, false, cols, l.hidden)) != MPG_OK) return s;
      p.bf16 = !half;
      p.prod[0].out[0] = grad;
      p.prod[0].ldo[0] = o.piece;
      p.prod[0].out_vec[0] = 1;
      p.target = l.target;
      p.target_bytes = l.target_bytes;
      p.target_stride = l.target_stride;
      p.ignore_index = l.ignore_index;
      p.col0 = (int32_t)c0;
      p.vocab = (int32_t)l.vocab;
      p.lse = lse;
      p.dloss = dloss;
      p.dloss_stride = dloss_stride;
      p.scale = scale;
      p.scale_count = same ? 1 : kScaleBlocks;
      p.scale_exp = exp;
      p.scale_largest = 1;
      if ((s = launch_fused(dev, product(FusedEpi::kProb, l.tokens, cols, l.hidden), p, slots, st)) != MPG_OK) return s;
    }
    std::memset(&p, 0, sizeof(p));
    p.bf16 = !half;
    p.scale = scale;
    p.scale_count = same ? 1 : kScaleBlocks;
    p.scale_exp = exp;
    p.scale_largest = 1;
    int count = 0;
    const FusedLaunch to_x = product(FusedEpi::kPlain, l.tokens, l.hidden, cols);
    const FusedLaunch to_w = product(FusedEpi::kPlain, cols, l.hidden, l.tokens);
    if (dX) {
      const bool last = i + 1 == o.pieces;
      FusedProduct& x = p.prod[count++];
      if ((s = fused_map(&x.map_a[0], grad, o.piece, l.dtype, false, l.tokens, cols)) != MPG_OK) return s;
      if ((s = fused_map(&x.map_b[0], w, o.w.ld, l.dtype, true, l.hidden, cols)) != MPG_OK) return s;
      x.b_mn_major = 1;
      x.out[0] = last ? dX : sum;
      x.ldo[0] = last ? lddx : o.ldsum;
      x.out_dtype = last ? (int32_t)l.dtype : (int32_t)MPG_F32;
      x.out_vec[0] = last ? fused_lines_ok(dX, lddx) : 1;
      x.add = i > 0 ? sum : nullptr;
      x.ldadd = o.ldsum;
    }
    // (elements of lines off 16 bytes are written faster by the tiles' epilogue)
    const bool few = dW && l.tokens <= kFewGradTokens && cols <= kFewGradRows && fused_lines_ok(dW, lddw);
    if (dW && !few) {
      FusedProduct& y = p.prod[count++];
      if ((s = fused_map(&y.map_a[0], grad, o.piece, l.dtype, true, cols, l.tokens)) != MPG_OK) return s;
      if ((s = fused_map(&y.map_b[0], o.x.ptr, o.x.ld, l.dtype, true, l.hidden, l.tokens)) != MPG_OK) return s;
      y.a_mn_major = y.b_mn_major = 1;
      y.out[0] = static_cast<uint16_t*>(dW) + c0 * lddw;
      y.ldo[0] = lddw;
      y.out_dtype = (int32_t)l.dtype;
      y.out_vec[0] = fused_lines_ok(y.out[0], lddw);
    }
    if (few) {
      if (dX && (s = launch_fused(dev, to_x, p, slots, st)) != MPG_OK) return s;
      FewGradParams y;
      std::memset(&y, 0, sizeof(y));
      y.d[0] = grad;
      y.x = static_cast<const uint16_t*>(o.x.ptr);
      y.ldd = o.piece;
      y.ldx = o.x.ld;
      y.tokens = (int32_t)l.tokens;
      y.rows = (int32_t)cols;
      y.cols = (int32_t)l.hidden;
      y.count = 1;
      y.bf16 = !half;
      y.out[0] = static_cast<uint16_t*>(dW) + c0 * lddw;
      y.ldo[0] = lddw;
      y.scale = scale;
      y.scale_count = same ? 1 : kScaleBlocks;
      y.scale_exp = exp;
      y.scale_largest = 1;
      const cudaError_t e = launch_few_grad(y, st);
      if (e != cudaSuccess) return fail(MPG_ERR_CUDA, "weight gradient launch: %s", cudaGetErrorString(e));
      continue;
    }
    s = count == 2 ? launch_fused_two(dev, to_x, to_w, p, slots, st) : launch_fused(dev, dX ? to_x : to_w, p, slots, st);
    if (s != MPG_OK) return s;
  }
  return MPG_OK;
}

}  // extern "C"
