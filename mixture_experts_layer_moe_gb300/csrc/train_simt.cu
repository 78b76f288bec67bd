// The grouped products of training on CUDA cores (fp32 FMA accumulation).
//
// The path of fp32 layers (tensor cores multiply fp32 operands in fewer
// bits), written for their sizes: a layer of a few hundred rows, whose
// launches cost as much as its products.
// A CTA computes a 64 x 64 tile of one segment's rows (RowsProduct) or of one
// expert's gradient (GradProduct), 4 x 4 outputs per thread, over steps of 16
// along the reduction.  The three storage orders of the operands differ in
// how a tile is staged only: in shared memory both operands lie reduction
// index first, so that a thread reads its 4 + 4 values as two float4.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "train.h"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64, TK = 16, T_THREADS = 256, T_LD = TM + 4;

// Stages a TK x 64 tile: element (kk, i) is src[i * ld + kk] (K_FAST) or
// src[kk * ld + i]; zero outside i < ni, kk < nk.
template <typename T, bool K_FAST>
__device__ __forceinline__ void stage(float (*dst)[T_LD], const T *src, int64_t ld, int ni, int nk) {
#pragma unroll
  for (int c = 0; c < TM * TK / T_THREADS; ++c) {
    const int l = threadIdx.x + c * T_THREADS;
    const int kk = K_FAST ? l % TK : l / TM;
    const int i = K_FAST ? l / TK : l % TM;
    float v = 0.f;
    if (i < ni && kk < nk) v = Elem<T>::load(src + (K_FAST ? i * ld + kk : kk * ld + i));
    dst[kk][i] = v;
  }
}

__device__ __forceinline__ void tile_fma(float (&acc)[4][4], const float (*as)[T_LD],
                                         const float (*bs)[T_LD], int tx, int ty) {
#pragma unroll
  for (int kk = 0; kk < TK; ++kk) {
    const float4 a4 = *reinterpret_cast<const float4 *>(&as[kk][ty * 4]);
    const float4 b4 = *reinterpret_cast<const float4 *>(&bs[kk][tx * 4]);
    const float a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
  }
}

// Expert and row range of this CTA's tile; false when there is none.
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int E, int rows, int tile, int &e,
                                          int &row0, int &end, int *status) {
  if (offsets == nullptr) {
    e = 0;
    row0 = tile * TM;
    end = rows;
    return row0 < end;
  }
  int acc = 0;
  for (int x = 0; x < E; ++x) {
    const int a = offsets[x], b = offsets[x + 1];
    if (a < 0 || b < a || b > rows) {
      if (threadIdx.x == 0) set_status(status, MOE_ERR_BAD_INDEX, x);
      return false;
    }
    const int nt = (b - a + TM - 1) / TM;
    if (tile < acc + nt) {
      e = x;
      row0 = a + (tile - acc) * TM;
      end = b;
      return true;
    }
    acc += nt;
  }
  return false;
}

template <typename T, int EPI, bool B_ROWS>
__global__ void __launch_bounds__(T_THREADS) rows_simt_kernel(RowsProduct p, int *status) {
  constexpr bool DUAL = EPI == kRowsSwiglu;
  __shared__ __align__(16) float as[TK][T_LD], bs[TK][T_LD], b2s[DUAL ? TK : 1][T_LD];
  if (status_failed(status)) return;
  int e, row0, end;
  if (!find_tile(p.offsets, p.num_experts, p.rows, blockIdx.x, e, row0, end, status)) return;
  const int n0 = blockIdx.y * TN, N = p.N, K = p.K;
  const int64_t lda = p.lda ? p.lda : K;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {}, acc2[4][4] = {};
  for (int half = 0; half < (EPI == kRowsPlain && p.A2 ? 2 : 1); ++half) {
    const T *A = static_cast<const T *>(half ? p.A2 : p.A) + row0 * lda;
    const int64_t base = (int64_t)e * N * K + (B_ROWS ? (int64_t)n0 : (int64_t)n0 * K);
    const T *B = static_cast<const T *>(half ? p.B2 : p.B) + base;
    for (int k0 = 0; k0 < K; k0 += TK) {
      stage<T, true>(as, A + k0, lda, end - row0, K - k0);
      if constexpr (B_ROWS) stage<T, false>(bs, B + (int64_t)k0 * N, N, N - n0, K - k0);
      else stage<T, true>(bs, B + k0, K, N - n0, K - k0);
      if constexpr (DUAL)
        stage<T, true>(b2s, static_cast<const T *>(p.B2) + base + k0, K, N - n0, K - k0);
      __syncthreads();
      tile_fma(acc, as, bs, tx, ty);
      if constexpr (DUAL) tile_fma(acc2, as, b2s, tx, ty);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + ty * 4 + i;
    if (r >= end) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + tx * 4 + j;
      if (c >= N) continue;
      const int64_t at = (int64_t)r * N + c;
      float v = acc[i][j];
      if constexpr (EPI == kRowsRelu) v = v < 0.f ? 0.f : v;
      if constexpr (EPI == kRowsSwiglu) {
        static_cast<T *>(p.out_g)[at] = Elem<T>::from_f(v);
        static_cast<T *>(p.out_u)[at] = Elem<T>::from_f(acc2[i][j]);
        v = v / (1.f + expf(-v)) * acc2[i][j];
      }
      if constexpr (EPI == kRowsReluGrad)
        v = Elem<T>::load(static_cast<const T *>(p.h) + at) > 0.f ? v : 0.f;
      if constexpr (EPI == kRowsSwigluGrad) {
        const float g = Elem<T>::load(static_cast<const T *>(p.g) + at);
        const float u = Elem<T>::load(static_cast<const T *>(p.u) + at);
        const float s = 1.f / (1.f + expf(-g));
        static_cast<T *>(p.out_u)[at] = Elem<T>::from_f(v * g * s);
        v = v * u * s * (1.f + g * (1.f - s));
      }
      static_cast<T *>(p.out)[at] = Elem<T>::from_f(v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(T_THREADS) grad_simt_kernel(GradProduct p, int *status) {
  __shared__ __align__(16) float as[TK][T_LD], bs[TK][T_LD];
  if (status_failed(status)) return;
  const int e = blockIdx.z, m0 = blockIdx.y * TM, n0 = blockIdx.x * TN, M = p.M, N = p.N;
  const int beg = p.offsets ? p.offsets[e] : 0, end = p.offsets ? p.offsets[e + 1] : p.rows;
  if (beg < 0 || end < beg || end > p.rows) {
    if (threadIdx.x == 0) set_status(status, MOE_ERR_BAD_INDEX, e);
    return;
  }
  const int64_t lda = p.lda ? p.lda : M;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  const T *A = static_cast<const T *>(p.A) + m0, *B = static_cast<const T *>(p.B) + n0;
  for (int q = beg; q < end; q += TK) {
    stage<T, false>(as, A + q * lda, lda, M - m0, end - q);
    stage<T, false>(bs, B + (int64_t)q * N, N, N - n0, end - q);
    __syncthreads();
    tile_fma(acc, as, bs, tx, ty);
    __syncthreads();
  }
  T *out = static_cast<T *>(p.out) + (int64_t)e * M * N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + ty * 4 + i;
    if (m >= M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = n0 + tx * 4 + j;
      if (c < N) out[(int64_t)m * N + c] = Elem<T>::from_f(acc[i][j]);
    }
  }
}

template <typename T>
cudaError_t launch_rows(const RowsProduct &p, int *status, cudaStream_t s) {
  const int mt = (p.rows + TM - 1) / TM + (p.offsets ? p.num_experts : 0);
  const dim3 grid(mt, (p.N + TN - 1) / TN);
  if (p.epi == kRowsPlain && p.b_rows)
    rows_simt_kernel<T, kRowsPlain, true><<<grid, T_THREADS, 0, s>>>(p, status);
  else if (p.epi == kRowsPlain)
    rows_simt_kernel<T, kRowsPlain, false><<<grid, T_THREADS, 0, s>>>(p, status);
  else if (p.epi == kRowsRelu)
    rows_simt_kernel<T, kRowsRelu, false><<<grid, T_THREADS, 0, s>>>(p, status);
  else if (p.epi == kRowsSwiglu)
    rows_simt_kernel<T, kRowsSwiglu, false><<<grid, T_THREADS, 0, s>>>(p, status);
  else if (p.epi == kRowsReluGrad)
    rows_simt_kernel<T, kRowsReluGrad, true><<<grid, T_THREADS, 0, s>>>(p, status);
  else
    rows_simt_kernel<T, kRowsSwigluGrad, true><<<grid, T_THREADS, 0, s>>>(p, status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_simt(const RowsProduct &p, int *status, cudaStream_t s) {
  return p.dtype == MOE_F32 ? launch_rows<float>(p, status, s)
                            : launch_rows<__nv_bfloat16>(p, status, s);
}

cudaError_t launch_grad_simt(const GradProduct &p, int *status, cudaStream_t s) {
  const dim3 grid((p.N + TN - 1) / TN, (p.M + TM - 1) / TM, p.offsets ? p.num_experts : 1);
  if (p.dtype == MOE_F32) grad_simt_kernel<float><<<grid, T_THREADS, 0, s>>>(p, status);
  else grad_simt_kernel<__nv_bfloat16><<<grid, T_THREADS, 0, s>>>(p, status);
  return cudaGetLastError();
}

}  // namespace moe
