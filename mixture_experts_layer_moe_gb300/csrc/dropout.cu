// Dropout of rows: y = x / (1 - q) where element (r, c) is kept, else 0 (philox.cuh).
#include "common.cuh"
#include "launch.h"
#include "philox.cuh"
#include "step.h"
#include "vec16.cuh"

namespace moe {
namespace {

// One thread per block of eight elements of a row.
template <typename T>
__global__ void __launch_bounds__(256)
dropout_kernel(moe_dropout_config c, const T *x, const RngState *rng, T *y, int threshold,
               float factor) {
  const RngState st = threshold ? *rng : RngState{0, 0};
  const int blocks = (c.d + 7) / 8;
  const int64_t total = c.rows * blocks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / blocks;
    const int k = (int)(i - r * blocks);
    const uint32_t keep = dropout_keep(st, k, (uint32_t)r, threshold);
    const T *from = x + r * c.ldx + k * 8;
    T *to = y + r * c.ldy + k * 8;
    const int n = min(8, c.d - k * 8);
    for (int j = 0; j < n; ++j)
      to[j] = Elem<T>::from_f(keep >> j & 1 ? Elem<T>::load(from + j) * factor : 0.f);
  }
}

}  // namespace

cudaError_t launch_dropout(const moe_dropout_config &c, int threshold, const void *x,
                           const uint64_t *rng, void *y, cudaStream_t s) {
  const int64_t blocks = (c.rows * ((c.d + 7) / 8) + 255) / 256, most = (int64_t)num_sms() * 8;
  const dim3 grid((unsigned)(blocks < most ? blocks : most));
  const RngState *st = reinterpret_cast<const RngState *>(rng);
  const float f = dropout_factor(threshold);
  if (c.dtype == MOE_F32)
    dropout_kernel<float><<<grid, 256, 0, s>>>(c, (const float *)x, st, (float *)y, threshold, f);
  else
    dropout_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        c, (const __nv_bfloat16 *)x, st, (__nv_bfloat16 *)y, threshold, f);
  return cudaGetLastError();
}

}  // namespace moe
