// Gradient of the combine: the gate-scaled copy of dy to expert order, and the
// gates' gradient.
//   dy_perm[q] = g[t][j] dy[t],   dgate[t][j] = sum_i dy[t][i] y_perm[q][i],
//   q = inv_perm[t * k + j].
// One warp per (token, slot): eight neighbouring pairs share a CTA, so that
// the k reads of a dy row meet in L1.  The dot product sums fp32 products of
// the lane's vectors in order, then over the warp by a butterfly.
#include "common.cuh"
#include "launch.h"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

template <typename T, bool DOT>
__global__ void __launch_bounds__(256)
combine_backward_kernel(const uint4 *__restrict__ dy, const uint4 *__restrict__ y_perm,
                        const int32_t *__restrict__ inv_perm, const float *__restrict__ gates,
                        uint4 *__restrict__ dy_perm, float *__restrict__ dgate, int P, int k,
                        int vpr, int *status) {
  constexpr int V = Vec16<T>::N;
  if (status_failed(status)) return;
  const int pair = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (pair >= P) return;
  const int q = inv_perm[pair];
  if (q < 0 || q >= P) {
    if (lane == 0) {
      set_status(status, MOE_ERR_BAD_INDEX, pair);
      if (DOT) dgate[pair] = 0.f;
    }
    return;
  }
  const float g = gates[pair];
  const uint4 *src = dy + (int64_t)(pair / k) * vpr, *yr = y_perm + (int64_t)q * vpr;
  uint4 *dst = dy_perm + (int64_t)q * vpr;
  float dot = 0.f;
  for (int v = lane; v < vpr; v += 32) {
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
    dot = warp_sum_xor(dot);
    if (lane == 0) dgate[pair] = dot;
  }
}

template <typename T>
cudaError_t launch(const void *dy, const void *y_perm, const int32_t *inv_perm, const float *gates,
                   void *dy_perm, float *dgate, int P, int k, int vpr, int *status,
                   cudaStream_t s) {
  const unsigned grid = (unsigned)((P + 7) / 8);
  if (dgate)
    combine_backward_kernel<T, true><<<grid, 256, 0, s>>>(
        (const uint4 *)dy, (const uint4 *)y_perm, inv_perm, gates, (uint4 *)dy_perm, dgate, P, k,
        vpr, status);
  else
    combine_backward_kernel<T, false><<<grid, 256, 0, s>>>(
        (const uint4 *)dy, nullptr, inv_perm, gates, (uint4 *)dy_perm, nullptr, P, k, vpr, status);
  return cudaGetLastError();
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
