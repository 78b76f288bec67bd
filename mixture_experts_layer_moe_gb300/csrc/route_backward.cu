// Gradient of the gates, the softmax and the load-balancing loss with respect
// to the router's logits.
//   RENORM    dl_e = g_j (dgate_j - sum_i g_i dgate_i) for the chosen e
//   TOP_PROB  dl_e = [e chosen] g_j dgate_j - p_e sum_i g_i dgate_i
//   loss      dl_e += aux (E / n) p_e (f_e - sum_i f_i p_i)
// One warp per token (lane l holds experts l, l + 32, ...); the products with
// the router's weights and with x run on the grouped-product kernels.  The
// bias gradient is the column sum: each warp adds the rows it meets in
// registers, each CTA its warps in order, and a second launch the CTAs in
// order, so the result does not depend on timing.
#include "common.cuh"
#include "launch.h"
#include "train.h"

namespace moe {
namespace {

constexpr int RB_WARPS = 8;
constexpr int RB_MAX_CTAS = 304;
constexpr int RB_SLOTS = 8;   // experts per lane at most (E <= 256)

template <typename T>
__global__ void __launch_bounds__(32 * RB_WARPS)
route_grad_kernel(const float *__restrict__ probs, const int32_t *__restrict__ topk_idx,
                  const float *__restrict__ gates, const float *__restrict__ dgate,
                  const float *__restrict__ f, float aux_scale, int renorm, int n, int E, int k,
                  T *__restrict__ dl, int pitch, float *__restrict__ bias_parts, int *status) {
  __shared__ float s_sum[RB_WARPS][RB_SLOTS * 32];
  pdl_launch_dependents();
  pdl_wait();
  if (status_failed(status)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float fe[RB_SLOTS], col[RB_SLOTS];
#pragma unroll
  for (int i = 0; i < RB_SLOTS; ++i) {
    const int e = lane + 32 * i;
    col[i] = 0.f;
    fe[i] = (f && e < E) ? f[e] : 0.f;
  }
  for (int t = blockIdx.x * RB_WARPS + warp; t < n; t += gridDim.x * RB_WARPS) {
    float p[RB_SLOTS], v[RB_SLOTS], fp = 0.f;
#pragma unroll
    for (int i = 0; i < RB_SLOTS; ++i) {
      const int e = lane + 32 * i;
      p[i] = (probs && e < E) ? probs[(int64_t)t * E + e] : 0.f;
      v[i] = 0.f;
      fp = fmaf(fe[i], p[i], fp);
    }
    // the token's choices, 32 slots at a time, one per lane; first the sum over
    // the chosen experts of gate * dgate, then each choice's term to the lane
    // that holds its expert
    float sum = 0.f;
    int e_l = -1;
    float g_l = 0.f, dg_l = 0.f;
    auto choices = [&](int j0) {
      const int j = j0 + lane;
      e_l = -1;
      if (j < k) {
        e_l = topk_idx[(int64_t)t * k + j];
        g_l = gates[(int64_t)t * k + j];
        dg_l = dgate[(int64_t)t * k + j];
        if (e_l < 0 || e_l >= E) {
          set_status(status, MOE_ERR_BAD_INDEX, t * k + j);
          e_l = -1;
        }
      }
    };
    for (int j0 = 0; j0 < k; j0 += 32) {
      choices(j0);
      if (e_l >= 0) sum = fmaf(g_l, dg_l, sum);
    }
    sum = warp_sum_xor(sum);
    for (int j0 = 0; j0 < k; j0 += 32) {
      if (k > 32) choices(j0);
      const float term = renorm ? g_l * (dg_l - sum) : g_l * dg_l;
      for (int j = 0; j < min(32, k - j0); ++j) {
        const int e = __shfl_sync(0xffffffffu, e_l, j);
        const float add = __shfl_sync(0xffffffffu, term, j);
#pragma unroll
        for (int i = 0; i < RB_SLOTS; ++i)
          if (e == lane + 32 * i) v[i] += add;
      }
    }
    if (f) fp = warp_sum_xor(fp);
#pragma unroll
    for (int i = 0; i < RB_SLOTS; ++i) {
      const int e = lane + 32 * i;
      if (!renorm) v[i] = fmaf(-p[i], sum, v[i]);
      if (f) v[i] = fmaf(aux_scale * p[i], fe[i] - fp, v[i]);
      if (e >= E) v[i] = 0.f;
      col[i] += v[i];
      if (dl && e < pitch) dl[(int64_t)t * pitch + e] = Elem<T>::from_f(v[i]);
    }
  }
  if (bias_parts == nullptr) return;
#pragma unroll
  for (int i = 0; i < RB_SLOTS; ++i) s_sum[warp][lane + 32 * i] = col[i];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < RB_WARPS; ++w) a += s_sum[w][e];
    bias_parts[(int64_t)blockIdx.x * E + e] = a;
  }
}

int grid_of(int n) {
  const int want = (n + RB_WARPS - 1) / RB_WARPS;
  return want < RB_MAX_CTAS ? want : RB_MAX_CTAS;
}

}  // namespace

size_t route_grad_scratch(const moe_config &c) { return (size_t)grid_of(c.n) * c.n_experts * 4; }

cudaError_t launch_route_grad(const moe_config &c, const float *probs, const int32_t *topk_idx,
                              const float *gates, const float *dgate, const float *f, float aux,
                              void *dl, int pitch, float *dbias, float *scratch, int *status,
                              cudaStream_t s) {
  const int grid = grid_of(c.n), E = c.n_experts;
  const int renorm = c.gate == MOE_GATE_RENORM;
  const float scale = aux * (float)E / (float)c.n;
  // one CTA's sums are the result
  float *parts = dbias == nullptr ? nullptr : grid == 1 ? dbias : scratch;
  const dim3 blocks(grid), threads(32 * RB_WARPS);
  cudaError_t e;
  if (c.act_dtype == MOE_F32)
    e = launch_pdl(route_grad_kernel<float>, blocks, threads, 0, s, probs, topk_idx, gates, dgate, f,
                   scale, renorm, c.n, E, c.top_k, (float *)dl, pitch, parts, status);
  else
    e = launch_pdl(route_grad_kernel<__nv_bfloat16>, blocks, threads, 0, s, probs, topk_idx, gates,
                   dgate, f, scale, renorm, c.n, E, c.top_k, (__nv_bfloat16 *)dl, pitch, parts,
                   status);
  if (e == cudaSuccess && dbias && grid > 1)
    e = launch_column_sum(scratch, nullptr, grid, E, dbias, nullptr, status, s);
  return e;
}

}  // namespace moe
