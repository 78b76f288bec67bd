// The C entry points round the layer in a training step (include/moe.h): dropout,
// the block joint and the cross entropy.  Argument checks and launches.
#include <math.h>
#include <stdint.h>

#include "api.h"
#include "moe.h"
#include "philox.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 32;   // (a row's index is 32 bits of the counter)
constexpr int kMaxD = 1 << 30;                   // (columns are counted in int, rounded up)
constexpr int kMaxTokens = 1 << 20, kMaxVocab = 1 << 24, kMaxWidth = 1 << 16;   // of the loss

bool ok_or_null(const void *p) { return p == nullptr || aligned(p, 16); }

moe_status check_rows(int64_t rows, int32_t d, int32_t dtype, int32_t reserved) {
  if (rows < 0 || d < 1 || reserved != 0) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  return rows > kMaxRows || d > kMaxD ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// A leading dimension: 0 stands for d.
bool ok_ld(int64_t ld, int64_t rows, int32_t d) {
  return ld == 0 || (ld >= d && ld <= INT64_MAX / 4 / (rows > 0 ? rows : 1));
}
int64_t dense(int64_t ld, int32_t d) { return ld == 0 ? d : ld; }

// The generator's state is needed where something may be dropped.
bool ok_rng(const uint64_t *rng, int threshold) {
  return rng == nullptr ? threshold == 0 : aligned(rng, 8);
}

moe_status check_join(const moe_join_config *c, int &threshold) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_rows(c->rows, c->d, c->dtype, c->reserved));
  for (int32_t kind : {c->post, c->pre})
    if (kind != MOE_NORM_NONE && kind != MOE_NORM_RMS && kind != MOE_NORM_LAYER)
      return MOE_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f) || !isfinite(c->eps) || !isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
  threshold = dropout_threshold(c->dropout);
  if (threshold < 0) return MOE_ERR_INVALID_ARG;
  for (int64_t ld : {c->ldx, c->ldb, c->ldr, c->ldy, c->lddx, c->lddb, c->lddr, c->lddy})
    if (!ok_ld(ld, c->rows, c->d)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_join_params(const moe_join_config &c, const moe_join_params *w) {
  if (w == nullptr || !ok_or_null(w->gate)) return MOE_ERR_INVALID_ARG;
  auto side = [](int32_t kind, const void *gamma, const void *beta) {
    if (kind == MOE_NORM_NONE ? gamma != nullptr : !ok_ptr(gamma)) return MOE_ERR_INVALID_ARG;
    if (kind != MOE_NORM_LAYER && beta != nullptr) return MOE_ERR_INVALID_ARG;
    return ok_or_null(beta) ? MOE_OK : MOE_ERR_INVALID_ARG;
  };
  MOE_TRY(side(c.post, w->post_gamma, w->post_beta));
  return side(c.pre, w->pre_gamma, w->pre_beta);
}

moe_join_config dense(const moe_join_config &c) {
  moe_join_config r = c;
  for (int64_t *ld : {&r.ldx, &r.ldb, &r.ldr, &r.ldy, &r.lddx, &r.lddb, &r.lddr, &r.lddy})
    *ld = dense(*ld, r.d);
  return r;
}

moe_status check_loss(const moe_loss_config *c) {
  if (c == nullptr || c->n < 0 || c->d < 1 || c->vocab < 1 || c->reserved != 0)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(c->z_loss >= 0.f) || !isfinite(c->z_loss)) return MOE_ERR_INVALID_ARG;
  if (c->n > kMaxTokens || c->vocab > kMaxVocab || c->d > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  return c->d % (c->dtype == MOE_F32 ? 4 : 8) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_loss_ws(const moe_loss_config &c, const void *ws, size_t ws_bytes) {
  if (ws == nullptr || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < loss_workspace(c) ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_dropout(const moe_dropout_config *cfg, const void *x, const uint64_t *rng, void *y,
                       void *stream) {
  if (cfg == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_rows(cfg->rows, cfg->d, cfg->dtype, cfg->reserved));
  const int threshold = dropout_threshold(cfg->p);
  if (threshold < 0 || !ok_rng(rng, threshold)) return MOE_ERR_INVALID_ARG;
  if (!ok_ld(cfg->ldx, cfg->rows, cfg->d) || !ok_ld(cfg->ldy, cfg->rows, cfg->d))
    return MOE_ERR_INVALID_ARG;
  if (cfg->rows == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
  moe_dropout_config c = *cfg;
  c.ldx = dense(c.ldx, c.d);
  c.ldy = dense(c.ldy, c.d);
  if (x == y && c.ldx != c.ldy && c.rows > 1) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_dropout(c, threshold, x, rng, y, as_stream(stream)));
}

moe_status moe_block_join(const moe_join_config *cfg, const void *x, const void *b,
                          const moe_join_params *w, const uint64_t *rng, void *r, void *y,
                          float *stats, void *stream) {
  int threshold;
  MOE_TRY(check_join(cfg, threshold));
  MOE_TRY(check_join_params(*cfg, w));
  if (!ok_rng(rng, threshold) || !ok_or_null(stats)) return MOE_ERR_INVALID_ARG;
  if (cfg->pre == MOE_NORM_NONE && y != nullptr) return MOE_ERR_INVALID_ARG;
  if (cfg->rows == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(b) || !ok_ptr(r)) return MOE_ERR_INVALID_ARG;
  if (cfg->pre != MOE_NORM_NONE && !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
  const moe_join_config c = dense(*cfg);
  if (r == x && c.ldr != c.ldx && c.rows > 1) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_join(c, threshold, JoinForward{x, b, *w, rng, r, y, stats},
                                 as_stream(stream)));
}

moe_status moe_block_join_workspace_size(const moe_join_config *cfg, size_t *bytes) {
  int threshold;
  MOE_TRY(check_join(cfg, threshold));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = align_up(join_backward_scratch(dense(*cfg)));
  return MOE_OK;
}

moe_status moe_block_join_backward(const moe_join_config *cfg, const void *b, const void *r,
                                   const float *stats, const moe_join_params *w,
                                   const uint64_t *rng, const void *dr, const void *dy, void *dx,
                                   void *db, const moe_join_grads *grads, void *ws,
                                   size_t ws_bytes, void *stream) {
  int threshold;
  MOE_TRY(check_join(cfg, threshold));
  MOE_TRY(check_join_params(*cfg, w));
  if (grads == nullptr || !ok_rng(rng, threshold)) return MOE_ERR_INVALID_ARG;
  const moe_join_grads &g = *grads;
  for (const float *p : {g.gate, g.post_gamma, g.post_beta, g.pre_gamma, g.pre_beta})
    if (!ok_or_null(p)) return MOE_ERR_INVALID_ARG;
  if (g.gate && !w->gate) return MOE_ERR_INVALID_ARG;
  if ((g.post_gamma && cfg->post == MOE_NORM_NONE) || (g.pre_gamma && cfg->pre == MOE_NORM_NONE) ||
      (g.post_beta && cfg->post != MOE_NORM_LAYER) || (g.pre_beta && cfg->pre != MOE_NORM_LAYER))
    return MOE_ERR_INVALID_ARG;
  if (cfg->pre == MOE_NORM_NONE && dy != nullptr) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  const moe_join_config c = dense(*cfg);
  if (c.rows == 0) {
    for (float *p : {g.gate, g.post_gamma, g.post_beta, g.pre_gamma, g.pre_beta})
      if (p) MOE_TRY(cuda_status(cudaMemsetAsync(p, 0, (size_t)c.d * 4, s)));
    return MOE_OK;
  }
  // b is read with a post norm or for the gate's gradient, r and the statistics
  // with a norm
  const bool need_b = c.post != MOE_NORM_NONE || g.gate != nullptr;
  const bool need_r = c.pre != MOE_NORM_NONE && dy != nullptr;
  if (need_b ? !ok_ptr(b) : !ok_or_null(b)) return MOE_ERR_INVALID_ARG;
  if (need_r ? !ok_ptr(r) : !ok_or_null(r)) return MOE_ERR_INVALID_ARG;
  if (need_r || c.post != MOE_NORM_NONE ? !ok_ptr(stats) : !ok_or_null(stats))
    return MOE_ERR_INVALID_ARG;
  if (!ok_or_null(dr) || !ok_or_null(dy) || !ok_or_null(dx) || !ok_or_null(db))
    return MOE_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < join_backward_scratch(c)) return MOE_ERR_WORKSPACE;
  return cuda_status(launch_join_backward(
      c, threshold, JoinBackward{b, r, stats, *w, rng, dr, dy, dx, db, g}, ws, s));
}

moe_status moe_cross_entropy_workspace_size(const moe_loss_config *cfg, size_t *bytes) {
  MOE_TRY(check_loss(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = loss_workspace(*cfg);
  return MOE_OK;
}

moe_status moe_cross_entropy(const moe_loss_config *cfg, const void *x, const void *W,
                             const int32_t *targets, float *loss, float *lse, void *ws,
                             size_t ws_bytes, void *stream) {
  MOE_TRY(check_loss(cfg));
  if (!ok_ptr(W)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_loss_ws(*cfg, ws, ws_bytes));
  if (cfg->n == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(targets) || !ok_ptr(loss) || !ok_ptr(lse)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_loss(*cfg, x, W, targets, loss, lse, ws, as_stream(stream)));
}

moe_status moe_cross_entropy_backward(const moe_loss_config *cfg, const void *x, const void *W,
                                      const int32_t *targets, const float *lse,
                                      const float *dloss, void *dx, void *dW, void *ws,
                                      size_t ws_bytes, void *stream) {
  MOE_TRY(check_loss(cfg));
  const moe_loss_config &c = *cfg;
  if (!ok_ptr(W) || !ok_or_null(dx) || !ok_or_null(dW)) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_loss_ws(c, ws, ws_bytes));
  cudaStream_t s = as_stream(stream);
  if (c.n == 0) {
    const size_t bytes = (size_t)c.vocab * c.d * (c.dtype == MOE_F32 ? 4 : 2);
    return dW ? cuda_status(cudaMemsetAsync(dW, 0, bytes, s)) : MOE_OK;
  }
  if (!ok_ptr(x) || !ok_ptr(targets) || !ok_ptr(lse) || !ok_ptr(dloss)) return MOE_ERR_INVALID_ARG;
  if (!dx && !dW) return MOE_OK;
  return cuda_status(launch_loss_backward(c, x, W, targets, lse, dloss, dx, dW, ws, s));
}

}  // extern "C"
