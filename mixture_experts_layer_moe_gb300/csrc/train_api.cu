// The C entry points that train the layer (include/moe.h): argument checks,
// the training workspace and the launch sequences.
#include <stdint.h>

#include "api.h"
#include "launch.h"
#include "moe.h"
#include "train.h"

namespace moe {
namespace {

// The layer's workspace, then the scratch of the gradients.
struct TrainLayout {
  size_t status, dg, du, dl, bias_parts, parts, total;
};

// dl's rows are padded to whole 16-byte vectors of bf16.
int dl_pitch(const moe_config &c) { return (c.n_experts + 7) / 8 * 8; }

// Whether a bf16 product is small enough for the CUDA cores: setting up the
// pair kernels (clusters, tensor memory, tensor maps) takes about 6 us a launch,
// so a short reduction and few products are faster without.  Forward and
// gradient in us, CUDA cores / tensor cores: 53 rows, d 80, d_ff 24, 3 experts
// 9, 10 / 13, 25;  1024 rows, d = d_ff = 128, 8 experts 15, 23 / 19, 35;  256
// rows, d = d_ff = 256 17, 25 / 20, 41;  400 rows, d 256, d_ff 384, 8 experts 31,
// 49 / 18, 35;  16 rows, d = d_ff = 512, 4 experts 28, 48 / 17, 33.
bool small_product(int64_t macs, int reduction) {
  return macs <= kSmallProducts && reduction <= 256;
}

bool on_cuda_cores(const RowsProduct &p) {
  return p.dtype == MOE_F32 || small_product((int64_t)p.rows * p.N * p.K, p.K);
}

// The weight gradients of the experts and of the router (operands unset).
void expert_grads_of(const moe_config &c, const int32_t *offsets, GradProduct (&p)[3]) {
  const int M[3] = {c.d, c.d_ff, c.d_ff}, N[3] = {c.d_ff, c.d, c.d};   // W2, W1, W3
  for (int i = 0; i < 3; ++i) {
    p[i] = GradProduct{};
    p[i].dtype = c.act_dtype;
    p[i].offsets = offsets;
    p[i].num_experts = c.n_experts;
    p[i].rows = c.n * c.top_k;
    p[i].M = M[i];
    p[i].N = N[i];
  }
}
GradProduct router_grad_of(const moe_config &c) {
  GradProduct p{};
  p.dtype = c.act_dtype;
  p.num_experts = 1;
  p.rows = c.n;
  p.M = c.n_experts;
  p.N = c.d;
  p.lda = dl_pitch(c);
  return p;
}
// The row products of the experts (operands unset): the two projections, dg and
// du, and dx.
enum RowsKind { kUp, kDown, kGateGrad, kInputGrad };
RowsProduct rows_of(const moe_config &c, RowsKind kind) {
  const bool gated = c.act == MOE_ACT_SWIGLU;
  RowsProduct p{};
  p.dtype = c.act_dtype;
  p.epi = kind == kUp ? (gated ? kRowsSwiglu : kRowsRelu)
          : kind == kGateGrad ? (gated ? kRowsSwigluGrad : kRowsReluGrad)
                              : kRowsPlain;
  p.b_rows = kind == kGateGrad || kind == kInputGrad;
  p.num_experts = c.n_experts;
  p.rows = c.n * c.top_k;
  const bool wide = kind == kUp || kind == kGateGrad;   // d -> d_ff
  p.K = wide ? c.d : c.d_ff;
  p.N = wide ? c.d_ff : c.d;
  // (shapes alone; the callers set the operands)
  p.offsets = reinterpret_cast<const int32_t *>(16);
  if (kind == kInputGrad && gated) p.A2 = reinterpret_cast<const void *>(16);
  return p;
}
int expert_problems(const moe_config &c) { return c.act == MOE_ACT_SWIGLU ? 3 : 2; }
// The router's share of the rows' gradient, dl Wg (operands unset).
RowsProduct router_rows_of(const moe_config &c) {
  RowsProduct r{};
  r.dtype = c.act_dtype;
  r.epi = kRowsPlain;
  r.b_rows = 1;
  r.num_experts = 1;
  r.rows = c.n;
  r.K = c.n_experts;
  r.N = c.d;
  r.lda = dl_pitch(c);
  return r;
}

// dg and du, or dl, are rounded to bf16 where tensor cores multiply them.  A
// small layer, where every product that takes them runs on the CUDA cores, keeps
// them in fp32: with few rows that rounding is not averaged out (one token, d
// 2776, d_ff 104: dW1 off by 3.1e-3 of its norm, 1.7e-3 without).  The product
// that forms dg and du may run on the tensor cores all the same (a long
// reduction over d), as partial sums (rows_split.cu): their second launch costs
// 1 to 2 us where the reduction was not cut anyway (53 rows of 2 experts, d 520,
// d_ff 248 24.8 us for the backward, 22.9 with the rounding).
bool wide_expert_grads(const moe_config &c) {
  GradProduct p[3];
  expert_grads_of(c, reinterpret_cast<const int32_t *>(16), p);
  return grads_small(p, expert_problems(c)) && on_cuda_cores(rows_of(c, kInputGrad));
}
bool wide_router_grads(const moe_config &c) {
  const GradProduct p = router_grad_of(c);
  return grads_small(&p, 1) && on_cuda_cores(router_rows_of(c));
}

TrainLayout train_layout_of(const moe_config &c) {
  moe_config c1 = c;
  c1.d_ff_shared = 0;
  const Layout base = layout_of(c1);
  const size_t P = (size_t)c.n * c.top_k, z = act_size(c);
  TrainLayout L{};
  L.status = base.status;
  size_t off = layout_of(c).total;
  auto take = [&](size_t bytes) {
    const size_t a = off;
    off += align_up(bytes);
    return a;
  };
  const bool wide = wide_expert_grads(c);   // (fp32 dg and du)
  L.dg = wide && z < 4 ? take(P * c.d_ff * 4) : base.h;   // [P][d_ff]
  L.du = take(P * c.d_ff * (wide ? 4 : z));
  L.dl = take((size_t)c.n * dl_pitch(c) * (wide_router_grads(c) ? 4 : z));
  L.bias_parts = take(route_grad_scratch(c));
  GradProduct experts[3];
  expert_grads_of(c, reinterpret_cast<const int32_t *>(16), experts);   // (shapes alone)
  const GradProduct router = router_grad_of(c);
  const size_t ge = grad_scratch(experts, expert_problems(c)), gr = grad_scratch(&router, 1);
  size_t parts = ge > gr ? ge : gr;   // (used by one launch after the other)
  for (RowsKind kind : {kUp, kDown, kGateGrad, kInputGrad}) {
    RowsProduct r = rows_of(c, kind);
    r.out_f32 = wide && z < 4 && kind == kGateGrad;
    const size_t bytes = on_cuda_cores(r) ? 0 : rows_scratch(r);
    if (bytes > parts) parts = bytes;
  }
  L.parts = take(parts);
  L.total = off;
  return L;
}

moe_status check_train_config(const moe_config *c) {
  MOE_TRY(check_config(c));
  if (c->weight_dtype != c->act_dtype) return MOE_ERR_UNSUPPORTED;   // (MXFP4, NVFP4)
  return MOE_OK;
}

// Checks the workspace and lays it out.
moe_status check_train_ws(const moe_config &c, const void *ws, size_t ws_bytes, TrainLayout &L) {
  if (ws == nullptr || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
  L = train_layout_of(c);
  return ws_bytes < L.total ? MOE_ERR_WORKSPACE : MOE_OK;
}

// The routed experts' weights alone (shared-expert weights are not read here).
moe_status check_routed_weights(const moe_config &c, const moe_weights *w) {
  moe_config c1 = c;
  c1.d_ff_shared = 0;
  moe_weights w1 = w ? *w : moe_weights{};
  w1.Ws1 = w1.Ws2 = w1.Ws3 = nullptr;
  return check_expert_weights(c1, &w1);
}

bool ok_or_null(const void *p) { return p == nullptr || aligned(p, 16); }

// bf16 rows run on the tensor cores (SM pairs), fp32 rows on the CUDA cores.
// parts: rows_scratch(p) bytes.
cudaError_t launch_rows(const RowsProduct &p, float *parts, int *status, cudaStream_t s) {
  if (on_cuda_cores(p)) return launch_rows_simt(p, status, s);
  if (gemm_router_rows_supported(p)) return launch_gemm_router_rows(p, status, s);
  if (p.add) return cudaErrorNotSupported;
  constexpr int epi[] = {0, 1, kEpiSwigluKeep, kEpiReluGrad, kEpiSwigluGrad};   // by kRows*
  GemmStage g{};
  g.a_dtype = g.b_dtype = g.out_dtype = MOE_BF16;
  g.epi = epi[p.epi];
  g.w_rows = p.b_rows;
  g.offsets = p.offsets;
  g.num_experts = p.num_experts;
  g.rows = p.rows;
  g.K = p.K;
  g.N = p.N;
  g.lda = p.lda;
  g.A = p.A;
  g.A2 = p.A2;
  g.B = p.B;
  g.B3 = p.B2;
  g.out = p.out;
  g.out_g = p.out_g;
  g.out_u = p.out_u;
  g.kept_g = p.g;
  g.kept_u = p.u;
  g.kept_h = p.h;
  g.beside = p.beside;
  if (!gemm_t2_supported(g)) return cudaErrorNotSupported;
  // (fp32 outputs: the pair kernel's epilogues store bf16)
  const int splits = rows_splits(p);
  return splits > 1 || p.out_f32 ? launch_rows_split(p, g, splits, parts, status, s)
                                 : launch_gemm_t2(g, status, s);
}

// Weight gradients over the same segments, in one launch.  splits, parts: as
// grad_splits and grad_scratch of all the layer's problems say, whichever of
// them are wanted (so that a gradient has the same bits alone and with the
// others).
cudaError_t launch_grads(const GradProduct *p, int count, int splits, float *parts, int beside,
                         int *status, cudaStream_t s) {
  if (count == 0) return cudaSuccess;
  if (grads_small(p, count)) return launch_grad_simt(p, count, splits, parts, status, s);
  for (int i = 0; i < count; ++i)
    if (!gemm_grad_supported(p[i])) return cudaErrorNotSupported;
  return launch_gemm_grad(p, count, splits, parts, beside, status, s);
}

// Whether the backward of the expert FFNs runs its launches in two pairs, dW2
// with dg and du, then dW1 and dW3 with dx, each launch on a share of the SMs.  With few
// rows per expert the one of a pair writes matrices and the other reads them:
// together HBM moves both ways, and the two share one ramp and one tail.
// A pass in us, one after the other / in pairs (46 SM pairs write, 30 read):
//   18 rows of 32 experts (d 7168, d_ff 2048) 1109 / 1043, 32 of 32 (2880, 2880)
//   712 / 647, 64 of 128 (2048, 768) 563 / 505, 128 of 16 (1024, 2048) 142 / 131,
//   128 of 8 (4096, 14336) 1200 / 1190;  with 256 rows 1443 / 1462 and 724 / 770
//   of the first and third, with 1024 4141 / 4410 of the first.
// (The first with 38 pairs each 1246, with 43 and 33 1111.)
bool side_by_side(const moe_config &c, int splits, const RowsProduct &r, const RowsProduct &x) {
  GradProduct p[3];
  expert_grads_of(c, r.offsets, p);
  return c.act_dtype == MOE_BF16 && splits == 1 && !grads_small(p, expert_problems(c)) &&
         !on_cuda_cores(r) && !on_cuda_cores(x) && rows_splits(r) == 1 && rows_splits(x) == 1 &&
         r.rows <= 128 * (int64_t)c.n_experts;
}

moe_status check_norm(const moe_norm_config *c) {
  if (c == nullptr || c->rows < 0 || c->d < 1 || c->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(c->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  for (int64_t ld : {c->ldx, c->ldy, c->lddx, c->lddy})
    if (ld != 0 && (ld < c->d || ld > INT64_MAX / 4 / (c->rows > 0 ? c->rows : 1)))
      return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Leading dimensions of 0 stand for d.
moe_norm_config dense(const moe_norm_config &c) {
  moe_norm_config r = c;
  for (int64_t *ld : {&r.ldx, &r.ldy, &r.lddx, &r.lddy})
    if (*ld == 0) *ld = r.d;
  return r;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_train_workspace_size(const moe_config *cfg, size_t *bytes) {
  MOE_TRY(check_train_config(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = train_layout_of(*cfg).total;
  return MOE_OK;
}

moe_status moe_layernorm(const moe_norm_config *cfg, const void *x, const void *gamma,
                         const void *beta, void *y, float *mean, float *rstd, void *stream) {
  MOE_TRY(check_norm(cfg));
  if (!ok_ptr(gamma) || !ok_or_null(beta) || (mean == nullptr) != (rstd == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!ok_or_null(mean) || !ok_or_null(rstd)) return MOE_ERR_INVALID_ARG;
  if (cfg->rows == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(y)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_norm(dense(*cfg), x, gamma, beta, y, mean, rstd, as_stream(stream)));
}

moe_status moe_layernorm_workspace_size(const moe_norm_config *cfg, size_t *bytes) {
  MOE_TRY(check_norm(cfg));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = align_up(norm_backward_scratch(dense(*cfg)));
  return MOE_OK;
}

moe_status moe_layernorm_backward(const moe_norm_config *cfg, const void *x, const void *gamma,
                                  const float *mean, const float *rstd, const void *dy, void *dx,
                                  float *dgamma, float *dbeta, void *ws, size_t ws_bytes,
                                  void *stream) {
  MOE_TRY(check_norm(cfg));
  if (!ok_ptr(gamma) || !ok_or_null(dgamma) || !ok_or_null(dbeta)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  const moe_norm_config c = dense(*cfg);
  if (c.rows == 0) {
    if (dgamma) MOE_TRY(cuda_status(cudaMemsetAsync(dgamma, 0, (size_t)c.d * 4, s)));
    if (dbeta) MOE_TRY(cuda_status(cudaMemsetAsync(dbeta, 0, (size_t)c.d * 4, s)));
    return MOE_OK;
  }
  if (!ok_ptr(x) || !ok_ptr(mean) || !ok_ptr(rstd) || !ok_ptr(dy) || !ok_ptr(dx))
    return MOE_ERR_INVALID_ARG;
  if (ws == nullptr || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < norm_backward_scratch(c)) return MOE_ERR_WORKSPACE;
  return cuda_status(
      launch_norm_backward(c, x, gamma, mean, rstd, dy, dx, dgamma, dbeta, ws, s));
}

moe_status moe_expert_ffn_train(const moe_config *cfg, const void *x_perm, const int32_t *offsets,
                                const moe_weights *w, void *g, void *u, void *h, void *y_perm,
                                void *ws, size_t ws_bytes, void *stream) {
  MOE_TRY(check_train_config(cfg));
  const moe_config &c = *cfg;
  MOE_TRY(check_routed_weights(c, w));
  if (!ok_ptr(x_perm) || !ok_ptr(offsets) || !ok_ptr(h) || !ok_ptr(y_perm))
    return MOE_ERR_INVALID_ARG;
  const bool gated = c.act == MOE_ACT_SWIGLU;
  if (gated ? !ok_ptr(g) || !ok_ptr(u) : g != nullptr || u != nullptr) return MOE_ERR_INVALID_ARG;
  TrainLayout L;
  MOE_TRY(check_train_ws(c, ws, ws_bytes, L));
  int *status = at<int>(ws, L.status);
  cudaStream_t s = as_stream(stream);
  float *parts = at<float>(ws, L.parts);
  RowsProduct up = rows_of(c, kUp);
  up.offsets = offsets;
  up.A = x_perm;
  up.B = w->W1;
  up.B2 = w->W3;
  up.out = h;
  up.out_g = g;
  up.out_u = u;
  MOE_TRY(cuda_status(launch_rows(up, parts, status, s)));
  RowsProduct dn = rows_of(c, kDown);
  dn.offsets = offsets;
  dn.A = h;
  dn.B = w->W2;
  dn.out = y_perm;
  return cuda_status(launch_rows(dn, parts, status, s));
}

moe_status moe_expert_ffn_backward(const moe_config *cfg, const void *x_perm,
                                   const int32_t *offsets, const moe_weights *w, const void *g,
                                   const void *u, const void *h, const void *dy_perm,
                                   void *dx_perm, const moe_expert_grads *grads, void *ws,
                                   size_t ws_bytes, void *stream) {
  MOE_TRY(check_train_config(cfg));
  const moe_config &c = *cfg;
  MOE_TRY(check_routed_weights(c, w));
  if (!ok_ptr(x_perm) || !ok_ptr(offsets) || !ok_ptr(h) || !ok_ptr(dy_perm) ||
      !ok_or_null(dx_perm) || grads == nullptr)
    return MOE_ERR_INVALID_ARG;
  const bool gated = c.act == MOE_ACT_SWIGLU;
  if (gated ? !ok_ptr(g) || !ok_ptr(u) : g != nullptr || u != nullptr) return MOE_ERR_INVALID_ARG;
  if (!ok_or_null(grads->W1) || !ok_or_null(grads->W3) || !ok_or_null(grads->W2))
    return MOE_ERR_INVALID_ARG;
  if (!gated && grads->W3) return MOE_ERR_INVALID_ARG;
  TrainLayout L;
  MOE_TRY(check_train_ws(c, ws, ws_bytes, L));
  int *status = at<int>(ws, L.status);
  cudaStream_t s = as_stream(stream);
  const int P = c.n * c.top_k;
  void *dg = at<void>(ws, L.dg), *du = at<void>(ws, L.du);

  GradProduct all[3], gw[kMaxGradProblems];
  expert_grads_of(c, offsets, all);
  const int splits = grad_splits(all, expert_problems(c));
  float *parts = at<float>(ws, L.parts);
  const void *left[3] = {dy_perm, dg, du}, *right[3] = {h, x_perm, x_perm};
  const int wide = c.act_dtype == MOE_BF16 && wide_expert_grads(c);
  void *out[3] = {grads->W2, grads->W1, grads->W3};
  int n_gw = 0;
  for (int i = 0; i < 3; ++i) {
    if (!out[i]) continue;
    gw[n_gw] = all[i];
    gw[n_gw].A = left[i];
    gw[n_gw].B = right[i];
    gw[n_gw].out = out[i];
    gw[n_gw].a_f32 = i > 0 && wide;
    ++n_gw;
  }
  if (!dx_perm && !grads->W1 && !grads->W3)
    return cuda_status(launch_grads(gw, n_gw, splits, parts, 0, status, s));
  RowsProduct r = rows_of(c, kGateGrad);
  r.offsets = offsets;
  r.A = dy_perm;
  r.B = w->W2;
  r.g = g;
  r.u = u;
  r.h = h;
  r.out = dg;
  r.out_u = gated ? du : nullptr;
  r.out_f32 = wide;
  RowsProduct x = rows_of(c, kInputGrad);
  x.offsets = offsets;
  x.A = dg;
  x.B = w->W1;
  x.A2 = gated ? du : nullptr;
  x.B2 = w->W3;
  x.out = dx_perm;
  x.a_f32 = wide;
  // SM pairs that write gradients while the others read weights (0: each launch
  // has them all)
  const int all_pairs = num_sms() / 2;
  const int writing = side_by_side(c, splits, r, x) ? (3 * all_pairs + 4) / 5 : 0;
  const int first = writing && grads->W2 ? 1 : 0, rest = n_gw - first;
  if (first) {
    r.beside = all_pairs - writing;
    MOE_TRY(cuda_status(launch_grads(gw, 1, splits, parts, writing, status, s)));
  }
  MOE_TRY(cuda_status(launch_rows(r, parts, status, s)));
  const bool both = writing && dx_perm && rest;
  if (both) x.beside = all_pairs - writing;
  MOE_TRY(cuda_status(launch_grads(gw + first, rest, splits, parts, both ? writing : 0, status, s)));
  return dx_perm ? cuda_status(launch_rows(x, parts, status, s)) : MOE_OK;
}

moe_status moe_combine_backward(const moe_config *cfg, const void *dy, const void *y_perm,
                                const int32_t *inv_perm, const float *topk_gate, void *dy_perm,
                                float *dgate, void *ws, size_t ws_bytes, void *stream) {
  MOE_TRY(check_train_config(cfg));
  const moe_config &c = *cfg;
  if (!ok_ptr(dy) || !ok_ptr(inv_perm) || !ok_ptr(topk_gate) || !ok_ptr(dy_perm))
    return MOE_ERR_INVALID_ARG;
  if ((y_perm == nullptr) != (dgate == nullptr) || !ok_or_null(y_perm) || !ok_or_null(dgate))
    return MOE_ERR_INVALID_ARG;
  TrainLayout L;
  MOE_TRY(check_train_ws(c, ws, ws_bytes, L));
  return cuda_status(launch_combine_backward(c.act_dtype, dy, y_perm, inv_perm, topk_gate, dy_perm,
                                             dgate, c.n, c.top_k, c.d,
                                             at<int>(ws, L.status),
                                             as_stream(stream)));
}

moe_status moe_route_backward(const moe_config *cfg, const void *x, const moe_weights *w,
                              const float *probs, const int32_t *topk_idx, const float *topk_gate,
                              const float *dgate, const float *f, float aux,
                              const int32_t *inv_perm, const void *dx_perm, void *dx, void *dWg,
                              float *dbias, void *ws, size_t ws_bytes, void *stream) {
  MOE_TRY(check_train_config(cfg));
  const moe_config &c = *cfg;
  MOE_TRY(check_router_weights(c, w));
  if (!ok_ptr(topk_idx) || !ok_ptr(topk_gate) || !ok_ptr(dgate)) return MOE_ERR_INVALID_ARG;
  if (!ok_or_null(probs) || !ok_or_null(f) || !ok_or_null(inv_perm) || !ok_or_null(dx_perm) ||
      !ok_or_null(dx) || !ok_or_null(dWg) || !ok_or_null(dbias))
    return MOE_ERR_INVALID_ARG;
  if ((c.gate == MOE_GATE_TOP_PROB || f) && probs == nullptr) return MOE_ERR_INVALID_ARG;
  if ((inv_perm == nullptr) != (dx_perm == nullptr)) return MOE_ERR_INVALID_ARG;
  if (dx_perm && !dx) return MOE_ERR_INVALID_ARG;
  if (dWg && !ok_ptr(x)) return MOE_ERR_INVALID_ARG;
  TrainLayout L;
  MOE_TRY(check_train_ws(c, ws, ws_bytes, L));
  int *status = at<int>(ws, L.status);
  cudaStream_t s = as_stream(stream);
  const int pitch = dl_pitch(c);
  const bool wide = wide_router_grads(c);
  const bool rows = dx && route_rows_supported(c, f);   // dx without dl
  void *dl = (dx && !rows) || dWg ? at<void>(ws, L.dl) : nullptr;
  if (dl || dbias)
    MOE_TRY(cuda_status(launch_route_grad(c, probs, topk_idx, topk_gate, dgate, f, aux,
                                          dx && !rows ? inv_perm : nullptr, dl, wide, pitch, dbias,
                                          at<float>(ws, L.bias_parts), status, s)));
  if (dWg) {
    GradProduct gw = router_grad_of(c);
    gw.A = dl;
    gw.B = x;
    gw.out = dWg;
    gw.a_f32 = c.act_dtype == MOE_BF16 && wide;
    MOE_TRY(cuda_status(launch_grads(&gw, 1, grad_splits(&gw, 1), at<float>(ws, L.parts),
                                     0, status, s)));
  }
  if (rows) {
    MOE_TRY(cuda_status(launch_route_rows(c, w->Wg, topk_idx, topk_gate, dgate, inv_perm, dx_perm,
                                          dx, status, s)));
  } else if (dx) {
    RowsProduct r = router_rows_of(c);
    r.A = dl;
    r.B = w->Wg;
    r.a_f32 = c.act_dtype == MOE_BF16 && wide;
    // (the sum of the expert rows in the product's epilogue, in fp32)
    r.add = dx_perm;
    r.add_inv = inv_perm;
    r.add_k = c.top_k;
    r.out = dx;
    MOE_TRY(cuda_status(launch_rows(r, nullptr, status, s)));
  }
  return MOE_OK;
}

}  // extern "C"
