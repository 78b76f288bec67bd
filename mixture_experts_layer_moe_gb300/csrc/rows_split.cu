// Row products whose tiles are too few to fill the SM pairs (few rows and a
// narrow result of a long reduction: a dense block's down projection of some
// tokens, or its dx): the reduction is cut into ranges, whose products run side
// by side on the pair kernel (kEpiPartial) and leave fp32 partial sums; a second
// launch adds them in order and applies the epilogue that the whole product
// would have had.  A gradient whose dg and du are to stay in fp32 takes this path
// uncut too (one range): the pair kernel's own epilogues store bf16.
#include "api.h"
#include "common.cuh"
#include "gate_math.cuh"
#include "launch.h"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int RS_PAIRS = 76;   // SM pairs that the plan counts on

struct FinishArgs {
  const float *parts;        // [mat][split][rows][N]
  const int32_t *offsets;    // nullptr: all rows
  int num_experts, rows, N, splits;
  const uint4 *g, *u, *h;    // kept rows
  void *out, *out_g, *out_u;
  int *status;
};

// Eight outputs: the sum over the ranges, in order.
__device__ __forceinline__ void sum_parts(const float *p, size_t plane, int splits, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 a = *reinterpret_cast<const float4 *>(p + s * plane);
    const float4 b = *reinterpret_cast<const float4 *>(p + s * plane + 4);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
}

// Vector i of 8 outputs.
template <typename T>
__device__ __forceinline__ void store8(void *out, size_t i, const float (&v)[8]) {
  constexpr int N = Vec16<T>::N;
#pragma unroll
  for (int q = 0; q < 8 / N; ++q)
    static_cast<uint4 *>(out)[i * (8 / N) + q] = pack16<T>(v + q * N);
}

// TO: the type of a gradient's outputs.
template <int EPI, typename TO = __nv_bfloat16>
__global__ void __launch_bounds__(256) rows_finish_kernel(FinishArgs a) {
  pdl_wait();
  if (status_failed(a.status)) return;
  // the segments' rows (rows outside them are not written)
  const int first = a.offsets ? a.offsets[0] : 0;
  const int last = a.offsets ? a.offsets[a.num_experts] : a.rows;
  const size_t plane = (size_t)a.rows * a.N;
  const size_t begin = (size_t)first * a.N / 8, end = (size_t)last * a.N / 8;   // (N % 8 == 0)
  for (size_t i = begin + (size_t)blockIdx.x * 256 + threadIdx.x; i < end;
       i += (size_t)gridDim.x * 256) {
    float v[8];
    sum_parts(a.parts + i * 8, plane, a.splits, v);
    if constexpr (EPI == kRowsRelu) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = relu(v[j]);
    } else if constexpr (EPI == kRowsSwiglu) {
      float u[8];
      sum_parts(a.parts + a.splits * plane + i * 8, plane, a.splits, u);
      store8<__nv_bfloat16>(a.out_g, i, v);
      store8<__nv_bfloat16>(a.out_u, i, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = silu_mul(v[j], u[j]);
    } else if constexpr (EPI == kRowsReluGrad) {
      float h[8];
      unpack16<__nv_bfloat16>(a.h[i], h);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = h[j] > 0.f ? v[j] : 0.f;
    } else if constexpr (EPI == kRowsSwigluGrad) {
      float g[8], u[8], du[8];
      unpack16<__nv_bfloat16>(a.g[i], g);
      unpack16<__nv_bfloat16>(a.u[i], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) swiglu_grad(v[j], g[j], u[j], v[j], du[j]);
      store8<TO>(a.out_u, i, du);
    }
    store8<TO>(a.out, i, v);
  }
}

int matrices_of(const RowsProduct &p) { return p.epi == kRowsSwiglu ? 2 : 1; }

}  // namespace

// The number of ranges with the least estimated time, where that is a fifth
// below the whole product's: rounds of tiles of 2.5 us and 0.4 us per k-block
// each, and with more than one range 4 us for the second launch and the partial
// sums written and read at 6 TB/s.  (bf16, whole / cut: one expert of 64 tokens,
// d 4096, d_ff 14336, forward 119 / 85 us; of 145 tokens, d 376, d_ff 10632,
// gradient 169 / 62; of 256 tokens, d 7168, d_ff 2048, forward 59 / 49.  Four
// experts of one token, d = d_ff = 2880, stay whole: 160 us for the gradient,
// 190 cut.)
int rows_splits(const RowsProduct &p) {
  if (p.dtype != MOE_BF16) return 1;
  const int E = p.offsets ? p.num_experts : 1;
  const int used = p.rows < E ? p.rows : E;   // experts with rows, at most
  const int64_t blocks = ((int64_t)p.rows + (int64_t)used * 256 - 1) / ((int64_t)used * 256);
  const int64_t tiles = used * blocks * ((p.N + 255) / 256) * matrices_of(p);
  const int64_t kb = (int64_t)((p.K + 63) / 64) * (p.A2 ? 2 : 1);
  if (tiles >= RS_PAIRS) return 1;
  const double whole = 2.5 + (double)kb * 0.4;   // (one round)
  int best = 1;
  double least = 0.8 * whole;
  // (no more than two rounds)
  for (int n = 2; n * tiles <= 2 * RS_PAIRS && n <= kb; ++n) {
    const int64_t each = (kb + n - 1) / n;
    if ((kb + each - 1) / each != n) continue;   // (a range would be empty)
    const double us = (double)((tiles * n + RS_PAIRS - 1) / RS_PAIRS) * (2.5 + each * 0.4) + 4 +
                      8e-6 / 6 * n * matrices_of(p) * (double)p.rows * p.N;
    if (us < least) {
      best = n;
      least = us;
    }
  }
  return best;
}

size_t rows_scratch(const RowsProduct &p) {
  const int splits = rows_splits(p);
  return splits > 1 || p.out_f32 ? (size_t)matrices_of(p) * splits * p.rows * p.N * 4 : 0;
}

cudaError_t launch_rows_split(const RowsProduct &p, const GemmStage &whole, int splits,
                              float *parts, int *status, cudaStream_t s) {
  GemmStage g = whole;
  g.epi = kEpiPartial;
  g.parts = parts;
  g.splits = splits;
  g.mats = matrices_of(p);
  const cudaError_t e = launch_gemm_t2(g, status, s);
  if (e != cudaSuccess) return e;
  FinishArgs a{};
  a.parts = parts;
  a.offsets = p.offsets;
  a.num_experts = p.num_experts;
  a.rows = p.rows;
  a.N = p.N;
  a.splits = splits;
  a.g = (const uint4 *)p.g;
  a.u = (const uint4 *)p.u;
  a.h = (const uint4 *)p.h;
  a.out = p.out;
  a.out_g = p.out_g;
  a.out_u = p.out_u;
  a.status = status;
  const int64_t blocks = ((int64_t)p.rows * p.N / 8 + 255) / 256;
  const dim3 grid((unsigned)(blocks < 1216 ? blocks : 1216));
  if (p.out_f32) {
    auto wide = p.epi == kRowsReluGrad ? rows_finish_kernel<kRowsReluGrad, float>
                                       : rows_finish_kernel<kRowsSwigluGrad, float>;
    return launch_pdl(wide, grid, dim3(256), 0, s, a);
  }
  auto with = p.epi == kRowsPlain      ? rows_finish_kernel<kRowsPlain>
              : p.epi == kRowsRelu     ? rows_finish_kernel<kRowsRelu>
              : p.epi == kRowsSwiglu   ? rows_finish_kernel<kRowsSwiglu>
              : p.epi == kRowsReluGrad ? rows_finish_kernel<kRowsReluGrad>
                                       : rows_finish_kernel<kRowsSwigluGrad>;
  return launch_pdl(with, grid, dim3(256), 0, s, a);
}

}  // namespace moe
