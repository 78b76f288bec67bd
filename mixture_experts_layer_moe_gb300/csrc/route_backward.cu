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
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int RB_WARPS = 8;
constexpr int RB_MAX_CTAS = 304;
constexpr int RB_SLOTS = 8;   // experts per lane at most (E <= 256)

template <typename T>
__global__ void __launch_bounds__(32 * RB_WARPS)
route_grad_kernel(const float *__restrict__ probs, const int32_t *__restrict__ topk_idx,
                  const float *__restrict__ gates, const float *__restrict__ dgate,
                  const float *__restrict__ f, const int32_t *__restrict__ inv_perm,
                  float aux_scale, int renorm, int n, int E, int k, T *__restrict__ dl, int pitch,
                  float *__restrict__ bias_parts, int *status) {
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
        if (inv_perm) {
          const int q = inv_perm[(int64_t)t * k + j];
          if (q < 0 || q >= n * k) set_status(status, MOE_ERR_BAD_INDEX, t * k + j);
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

// The rows' gradient where dl has entries at the token's k choices alone (RENORM
// without the loss):
//   dx[t] = sum_j (dx_perm[q_j] + c_j Wg[e_j]),   c_j = g_j (dgate_j - sum g dgate),
// in one pass: the k router rows of a token come from L2 (Wg is a few MB), so
// the launch moves what the sum of the expert rows moves, and neither dl nor
// a rounding of it is kept.  CTA (t, c) takes vectors [c * 256 VB, ...) of
// token t's row; four slots' rows are in flight per thread, and the sum runs in
// slot order.  (blockDim.x: 256, or fewer for a row of fewer vectors.)
constexpr int RR_SLOTS = 4;
__device__ __forceinline__ uint4 load_now(const uint4 *p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <typename T, int VB>
__global__ void __launch_bounds__(256)
route_rows_kernel(const uint4 *__restrict__ dx_perm, const int32_t *__restrict__ inv_perm,
                  const int32_t *__restrict__ topk_idx, const float *__restrict__ gates,
                  const float *__restrict__ dgate, const uint4 *__restrict__ Wg,
                  uint4 *__restrict__ dx, int n, int E, int k, int vpr, int *status) {
  constexpr int V = Vec16<T>::N;
  __shared__ int s_q[kRouteRowsMaxK], s_e[kRouteRowsMaxK];
  __shared__ float s_c[kRouteRowsMaxK];
  pdl_launch_dependents();
  pdl_wait();
  // (other CTAs of this launch may set the status meanwhile, so the threads of a
  // CTA need not agree on it: all of them reach the barrier, and none reads
  // indexes that warp 0 did not write)
  const bool failed = status_failed(status);
  const int t = blockIdx.x, P = n * k;
  if (threadIdx.x < 32) {
    // (k <= 32: one slot per lane)
    const int j = threadIdx.x;
    int q = -1, e = -1;
    float g = 0.f, dg = 0.f;
    if (j < k) {
      const int64_t pair = (int64_t)t * k + j;
      e = topk_idx[pair];
      if (e < 0 || e >= E) {
        if (blockIdx.y == 0) set_status(status, MOE_ERR_BAD_INDEX, (int)pair);
        e = -1;
      } else {
        g = gates[pair];
        dg = dgate[pair];
      }
      if (dx_perm) {
        q = inv_perm[pair];
        if (q < 0 || q >= P) {
          if (blockIdx.y == 0) set_status(status, MOE_ERR_BAD_INDEX, (int)pair);
          q = -1;
        }
      }
    }
    const float sum = warp_sum_xor(g * dg);
    if (j < kRouteRowsMaxK) {
      s_q[j] = q;
      s_e[j] = e;
      s_c[j] = g * (dg - sum);
    }
  }
  __syncthreads();
  if (failed) return;
  const int v0 = blockIdx.y * blockDim.x * VB + threadIdx.x;
  float acc[VB][V];
#pragma unroll
  for (int b = 0; b < VB; ++b)
#pragma unroll
    for (int c = 0; c < V; ++c) acc[b][c] = 0.f;
  // (a slot or a vector that is not there reads a valid one and drops it, so
  // that all loads of a round are issued before the first is used)
  int at[VB];
#pragma unroll
  for (int b = 0; b < VB; ++b) at[b] = min(v0 + b * (int)blockDim.x, vpr - 1);
  const uint4 *rows = dx_perm ? dx_perm : Wg;
  for (int j0 = 0; j0 < k; j0 += RR_SLOTS) {
    uint4 r[RR_SLOTS][VB], w[RR_SLOTS][VB];
    int q[RR_SLOTS], e[RR_SLOTS];
#pragma unroll
    for (int u = 0; u < RR_SLOTS; ++u) {
      const int j = min(j0 + u, k - 1);
      q[u] = s_q[j];
      e[u] = s_e[j];
#pragma unroll
      for (int b = 0; b < VB; ++b) {
        r[u][b] = load_now(rows + (int64_t)max(q[u], 0) * vpr + at[b]);
        w[u][b] = load_now(Wg + (int64_t)max(e[u], 0) * vpr + at[b]);
      }
    }
#pragma unroll
    for (int u = 0; u < RR_SLOTS; ++u) {
      if (j0 + u >= k) break;
      const float c = s_c[j0 + u];
#pragma unroll
      for (int b = 0; b < VB; ++b) {
        float f[V], g[V];
        unpack16<T>(r[u][b], f);
        unpack16<T>(w[u][b], g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (q[u] >= 0) acc[b][i] += f[i];
          if (e[u] >= 0) acc[b][i] = fmaf(c, g[i], acc[b][i]);
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < VB; ++b)
    if (v0 + b * (int)blockDim.x < vpr) dx[(int64_t)t * vpr + at[b]] = pack16<T>(acc[b]);
}

int grid_of(int n) {
  const int want = (n + RB_WARPS - 1) / RB_WARPS;
  return want < RB_MAX_CTAS ? want : RB_MAX_CTAS;
}

}  // namespace

size_t route_grad_scratch(const moe_config &c) { return (size_t)grid_of(c.n) * c.n_experts * 4; }

cudaError_t launch_route_grad(const moe_config &c, const float *probs, const int32_t *topk_idx,
                              const float *gates, const float *dgate, const float *f, float aux,
                              const int32_t *inv_perm, void *dl, bool dl_f32, int pitch,
                              float *dbias, float *scratch, int *status, cudaStream_t s) {
  const int grid = grid_of(c.n), E = c.n_experts;
  const int renorm = c.gate == MOE_GATE_RENORM;
  const float scale = aux * (float)E / (float)c.n;
  // one CTA's sums are the result
  float *parts = dbias == nullptr ? nullptr : grid == 1 ? dbias : scratch;
  const dim3 blocks(grid), threads(32 * RB_WARPS);
  cudaError_t e;
  if (dl_f32)
    e = launch_pdl(route_grad_kernel<float>, blocks, threads, 0, s, probs, topk_idx, gates, dgate, f,
                   inv_perm, scale, renorm, c.n, E, c.top_k, (float *)dl, pitch, parts, status);
  else
    e = launch_pdl(route_grad_kernel<__nv_bfloat16>, blocks, threads, 0, s, probs, topk_idx, gates,
                   dgate, f, inv_perm, scale, renorm, c.n, E, c.top_k, (__nv_bfloat16 *)dl, pitch,
                   parts, status);
  if (e == cudaSuccess && dbias && grid > 1)
    e = launch_column_sum(scratch, nullptr, grid, E, dbias, nullptr, status, s);
  return e;
}

// Against dl in a launch of its own and the product dl Wg with the rows added in
// its epilogue, the whole gradient of a bf16 router took (us, this / the product):
//   n 16384, d 7168, 256 experts: k = 2 299 / 254, k = 4 380 / 328, k = 8 572 / 488
//   n 4096, d 4096, 64 experts, k = 2 57 / 59;  n 2048, d 7168, k = 8 100 / 88
//   n 1024, d 1024, k = 8 23 / 27;  n 1, k = 8 14 / 21
// Long rows of many choices take the product: the reads of Wg's rows from L2 are
// what this sum waits for.  Few choices stay here although the product is the
// faster on large batches: it rounds dl to bf16 as its operand, this sum
// does not.  (fp32: 2048 tokens, d 1024, 256 experts, k = 8 59 / 93.)
bool route_rows_supported(const moe_config &c, const float *f) {
  if (c.gate != MOE_GATE_RENORM || f != nullptr || c.top_k > kRouteRowsMaxK) return false;
  return c.act_dtype == MOE_F32 || c.top_k <= 4 || (int64_t)c.n * c.d <= 1 << 23;
}

cudaError_t launch_route_rows(const moe_config &c, const void *Wg, const int32_t *topk_idx,
                              const float *gates, const float *dgate, const int32_t *inv_perm,
                              const void *dx_perm, void *dx, int *status, cudaStream_t s) {
  const int vpr = c.d / (c.act_dtype == MOE_F32 ? 4 : 8);
  // two vectors per thread where that still leaves two CTAs per SM
  const bool two = vpr > 256 && (int64_t)c.n * ((vpr + 511) / 512) >= 2 * 152;
  const int threads = vpr < 256 ? (vpr + 31) / 32 * 32 : 256, per_cta = threads * (two ? 2 : 1);
  const dim3 grid(c.n, (vpr + per_cta - 1) / per_cta);
  auto with = c.act_dtype == MOE_F32
                  ? (two ? route_rows_kernel<float, 2> : route_rows_kernel<float, 1>)
                  : (two ? route_rows_kernel<__nv_bfloat16, 2> : route_rows_kernel<__nv_bfloat16, 1>);
  return launch_pdl(with, grid, dim3(threads), 0, s, (const uint4 *)dx_perm, inv_perm, topk_idx, gates,
                    dgate, (const uint4 *)Wg, (uint4 *)dx, c.n, c.n_experts, c.top_k, vpr, status);
}

}  // namespace moe
