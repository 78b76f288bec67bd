// Gradient of the combine: the gate-scaled copy of dy to expert order, and the
// gates' gradient.
//   dy_perm[q] = g[t][j] dy[t],   dgate[t][j] = sum_i dy[t][i] y_perm[q][i],
//   q = inv_perm[t * k + j].
// One warp per (token, slot), or a part of one where a row is shorter than 32
// vectors: neighbouring pairs share a CTA, so that the k reads of a dy row meet
// in L1.  The dot product sums fp32 products of the lane's vectors in order,
// then over the lanes by a butterfly.
// A stream: 16384 tokens, 8 slots, d 7168 bf16 move 3.99 GB in 590 us = 6.77
// TB/s, the rate of a plain copy.
#include "common.cuh"
#include "launch.h"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

template <typename T, bool DOT, int LANES>
__global__ void __launch_bounds__(256)
combine_backward_kernel(const uint4 *__restrict__ dy, const uint4 *__restrict__ y_perm,
                        const int32_t *__restrict__ inv_perm, const float *__restrict__ gates,
                        uint4 *__restrict__ dy_perm, float *__restrict__ dgate, int P, int k,
                        int vpr, int *status) {
  constexpr int V = Vec16<T>::N;
  if (status_failed(status)) return;
  const int pair = blockIdx.x * (256 / LANES) + threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const bool inside = pair < P;
  const int q = inside ? inv_perm[pair] : -1;
  const bool ok = q >= 0 && q < P;
  if (inside && !ok && lane == 0) set_status(status, MOE_ERR_BAD_INDEX, pair);
  const float g = ok ? gates[pair] : 0.f;
  const uint4 *src = dy + (int64_t)(ok ? pair / k : 0) * vpr;
  const uint4 *yr = y_perm + (int64_t)(ok ? q : 0) * vpr;
  uint4 *dst = dy_perm + (int64_t)(ok ? q : 0) * vpr;
  float dot = 0.f;
  for (int v = ok ? lane : vpr; v < vpr; v += LANES) {
    float a[V], b[V];
    unpack16<T>(src[v], a);
    if (DOT) {
      unpack16<T>(yr[v], b);
#pragma unroll
      for (int i = 0; i < V; ++i) dot = fmaf(a[i], b[i], dot);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] *= g;
    dst[v] = pack16<T>(a);
  }
  if (DOT) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (inside && lane == 0) dgate[pair] = dot;
  }
}

template <typename T, int LANES>
cudaError_t launch_lanes(const void *dy, const void *y_perm, const int32_t *inv_perm,
                         const float *gates, void *dy_perm, float *dgate, int P, int k, int vpr,
                         int *status, cudaStream_t s) {
  constexpr int PAIRS = 256 / LANES;
  const unsigned grid = (unsigned)(((int64_t)P + PAIRS - 1) / PAIRS);
  if (dgate)
    combine_backward_kernel<T, true, LANES><<<grid, 256, 0, s>>>(
        (const uint4 *)dy, (const uint4 *)y_perm, inv_perm, gates, (uint4 *)dy_perm, dgate, P, k,
        vpr, status);
  else
    combine_backward_kernel<T, false, LANES><<<grid, 256, 0, s>>>(
        (const uint4 *)dy, nullptr, inv_perm, gates, (uint4 *)dy_perm, nullptr, P, k, vpr, status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch(const void *dy, const void *y_perm, const int32_t *inv_perm, const float *gates,
                   void *dy_perm, float *dgate, int P, int k, int vpr, int *status,
                   cudaStream_t s) {
  auto with = vpr > 8 ? launch_lanes<T, 32> : vpr > 2 ? launch_lanes<T, 8> : launch_lanes<T, 2>;
  return with(dy, y_perm, inv_perm, gates, dy_perm, dgate, P, k, vpr, status, s);
}

}  // namespace

cudaError_t launch_combine_backward(int dtype, const void *dy, const void *y_perm,
                                    const int32_t *inv_perm, const float *gates, void *dy_perm,
                                    float *dgate, int n, int k, int d, int *status,
                                    cudaStream_t s) {
  const int P = n * k;
  if (dtype == MOE_F32)
    return launch<float>(dy, y_perm, inv_perm, gates, dy_perm, dgate, P, k, d / 4, status, s);
  return launch<__nv_bfloat16>(dy, y_perm, inv_perm, gates, dy_perm, dgate, P, k, d / 8, status, s);
}

}  // namespace moe
