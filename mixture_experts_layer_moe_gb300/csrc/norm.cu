// Layer norm and its gradient.
//   y_i = (x_i - mean) rstd gamma_i + beta_i
//   dx_i = rstd (w_i - sum w / d - xh_i sum w xh / d),   w_i = dy_i gamma_i
//   dgamma_i = sum_rows dy_i xh_i,   dbeta_i = sum_rows dy_i
// Both are streams through HBM: the forward reads and writes each row once,
// the gradient reads x and dy once and writes dx.  A row lives in the
// registers of a group of threads (a warp for short rows, else the CTA), so
// the variance is summed around the mean without a second read.  Groups walk
// the rows with a grid stride, with the next row's loads in flight while the
// current one is reduced.  In the gradient a thread owns the same columns of
// every row it meets, so the column sums grow in its registers; each CTA
// writes one partial row and a second launch adds the partials in order (no
// atomics: the result does not depend on timing).
// All statistics and sums are fp32.
#include "common.cuh"
#include "launch.h"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int N_MAX_THREADS = 512;
constexpr int N_MAX_PARTS = 304;   // partial rows of the column sums (two CTAs per SM)

// VEC elements as they lie in memory: 16 bytes, or one element.
template <typename T, int VEC>
struct Raw {
  uint4 v;
  __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float *f) const { unpack16<T>(v, f); }
  static __device__ __forceinline__ void put(T *p, const float *f) {
    *reinterpret_cast<uint4 *>(p) = pack16<T>(f);
  }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T *p) { v = *p; }
  __device__ __forceinline__ void get(float *f) const { f[0] = Elem<T>::to_f(v); }
  static __device__ __forceinline__ void put(T *p, const float *f) { *p = Elem<T>::from_f(f[0]); }
};

// Sum over the group: the warp, or the CTA through one of two alternating
// buffers (a buffer is written again only after the barrier of the sum in
// between, which every reader of it has reached).
template <bool WARP>
__device__ __forceinline__ float2 group_sum(float a, float b, float2 (*buf)[32], int &turn) {
  a = warp_sum_xor(a);
  b = warp_sum_xor(b);
  if (WARP) return make_float2(a, b);
  float2 *s = buf[turn];
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 r = s[0];
  const int nw = blockDim.x >> 5;
  for (int w = 1; w < nw; ++w) {
    r.x += s[w].x;
    r.y += s[w].y;
  }
  return r;
}

template <typename T, int VEC, int VPT, bool WARP>
__global__ void __launch_bounds__(N_MAX_THREADS)
norm_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
            const T *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
            float *__restrict__ rstd_out) {
  __shared__ float2 buf[2][32];
  const int tpr = WARP ? 32 : blockDim.x, tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = WARP ? blockDim.x >> 5 : 1, group = WARP ? threadIdx.x >> 5 : 0;
  const int d = c.d;
  const float df = (float)d;
  int turn = 0;
  Raw<T, VEC> raw[VPT], ga[VPT], be[VPT];
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t r = (int64_t)blockIdx.x * groups + group;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (tid + i * tpr) * VEC;
    if (col < d) {
      if (r < c.rows) raw[i].load(x + r * c.ldx + col);
      ga[i].load(gamma + col);
      if (beta) be[i].load(beta + col);
    }
  }
  for (; r < c.rows; r += step) {
    float v[VPT][VEC];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (tid + i * tpr) * VEC;
      if (col < d) {
        raw[i].get(v[i]);
        if (r + step < c.rows) raw[i].load(x + (r + step) * c.ldx + col);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += v[i][j];
      }
    }
    const float mean = group_sum<WARP>(sum, 0.f, buf, turn).x / df;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if ((tid + i * tpr) * VEC < d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] -= mean;
          sq = fmaf(v[i][j], v[i][j], sq);
        }
      }
    }
    const float rstd = 1.f / sqrtf(group_sum<WARP>(sq, 0.f, buf, turn).x / df + c.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (tid + i * tpr) * VEC;
      if (col < d) {
        float g[VEC], b[VEC];
        ga[i].get(g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) b[j] = 0.f;
        if (beta) be[i].get(b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = fmaf(v[i][j] * rstd, g[j], b[j]);
        Raw<T, VEC>::put(y + r * c.ldy + col, v[i]);
      }
    }
    if (mean_out && tid == 0) {
      mean_out[r] = mean;
      rstd_out[r] = rstd;
    }
  }
}

// pg, pb: [gridDim.x][d] partial column sums (or the results themselves when
// there is one CTA); either may be nullptr.
template <typename T, int VEC, int VPT, bool WARP>
__global__ void __launch_bounds__(N_MAX_THREADS)
norm_backward_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
                     const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                     const T *__restrict__ dy, T *__restrict__ dx, float *__restrict__ pg,
                     float *__restrict__ pb) {
  __shared__ float2 buf[2][32];
  __shared__ float cols[WARP ? 8 * 32 * VPT * VEC : 1];
  const int tpr = WARP ? 32 : blockDim.x, tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int groups = WARP ? blockDim.x >> 5 : 1, group = WARP ? threadIdx.x >> 5 : 0;
  const int d = c.d;
  const float df = (float)d;
  int turn = 0;
  Raw<T, VEC> rx[VPT], ry[VPT], ga[VPT];
  float ag[VPT][VEC], ab[VPT][VEC];
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t r = (int64_t)blockIdx.x * groups + group;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int col = (tid + i * tpr) * VEC;
    if (col < d) {
      if (r < c.rows) {
        rx[i].load(x + r * c.ldx + col);
        ry[i].load(dy + r * c.lddy + col);
      }
      ga[i].load(gamma + col);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) ag[i][j] = ab[i][j] = 0.f;
  }
  for (; r < c.rows; r += step) {
    const float mean = mean_in[r], rstd = rstd_in[r];
    float xh[VPT][VEC], w[VPT][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (tid + i * tpr) * VEC;
      if (col < d) {
        float g[VEC];
        rx[i].get(xh[i]);
        ry[i].get(w[i]);
        ga[i].get(g);
        if (r + step < c.rows) {
          rx[i].load(x + (r + step) * c.ldx + col);
          ry[i].load(dy + (r + step) * c.lddy + col);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[i][j] = (xh[i][j] - mean) * rstd;
          ag[i][j] = fmaf(w[i][j], xh[i][j], ag[i][j]);
          ab[i][j] += w[i][j];
          w[i][j] *= g[j];
          s1 += w[i][j];
          s2 = fmaf(w[i][j], xh[i][j], s2);
        }
      }
    }
    const float2 s = group_sum<WARP>(s1, s2, buf, turn);
    const float m1 = s.x / df, m2 = s.y / df;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int col = (tid + i * tpr) * VEC;
      if (col < d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[i][j] = rstd * (w[i][j] - m1 - xh[i][j] * m2);
        Raw<T, VEC>::put(dx + r * c.lddx + col, w[i]);
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *part = which ? pb : pg;
    if (part == nullptr) continue;
    part += (int64_t)blockIdx.x * d;
    if (WARP) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          cols[group * 32 * VPT * VEC + (tid + i * 32) * VEC + j] = which ? ab[i][j] : ag[i][j];
      __syncthreads();
      for (int col = threadIdx.x; col < d; col += blockDim.x) {
        float a = 0.f;
        for (int g = 0; g < groups; ++g) a += cols[g * 32 * VPT * VEC + col];
        part[col] = a;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int col = (tid + i * tpr) * VEC;
        if (col < d) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) part[col + j] = which ? ab[i][j] : ag[i][j];
        }
      }
    }
  }
}

// out[which][col] = sum over count partial rows, in a fixed order: warp w of
// eight adds rows w, w + 8, ..., then the eight sums are added.
__global__ void __launch_bounds__(256)
column_sum_kernel(const float *__restrict__ pg, const float *__restrict__ pb, int count, int d,
                  float *__restrict__ dgamma, float *__restrict__ dbeta) {
  __shared__ float s[8][33];
  const float *part = blockIdx.y ? pb : pg;
  float *out = blockIdx.y ? dbeta : dgamma;
  pdl_wait();
  if (out == nullptr) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int r = warp; r < count; r += 8) a += part[(int64_t)r * d + col];
  }
  s[warp][lane] = a;
  __syncthreads();
  if (warp == 0 && col < d) {
#pragma unroll
    for (int w = 1; w < 8; ++w) a += s[w][lane];
    out[col] = a;
  }
}

// Rows wider than a CTA holds in registers: one CTA per row, reading it again
// (from L2) for each pass.
template <typename T>
__global__ void __launch_bounds__(512)
norm_wide_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
                 const T *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
                 float *__restrict__ rstd_out) {
  __shared__ float2 buf[2][32];
  int turn = 0;
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const T *xr = x + r * c.ldx;
    float sum = 0.f, sq = 0.f;
    for (int i = threadIdx.x; i < c.d; i += blockDim.x) sum += Elem<T>::load(xr + i);
    const float mean = group_sum<false>(sum, 0.f, buf, turn).x / (float)c.d;
    for (int i = threadIdx.x; i < c.d; i += blockDim.x) {
      const float v = Elem<T>::load(xr + i) - mean;
      sq = fmaf(v, v, sq);
    }
    const float rstd =
        1.f / sqrtf(group_sum<false>(sq, 0.f, buf, turn).x / (float)c.d + c.eps);
    for (int i = threadIdx.x; i < c.d; i += blockDim.x)
      y[r * c.ldy + i] = Elem<T>::from_f(
          fmaf((Elem<T>::load(xr + i) - mean) * rstd, Elem<T>::load(gamma + i),
               beta ? Elem<T>::load(beta + i) : 0.f));
    if (mean_out && threadIdx.x == 0) {
      mean_out[r] = mean;
      rstd_out[r] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(512)
norm_backward_wide_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
                          const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                          const T *__restrict__ dy, T *__restrict__ dx) {
  __shared__ float2 buf[2][32];
  int turn = 0;
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const T *xr = x + r * c.ldx, *yr = dy + r * c.lddy;
    const float mean = mean_in[r], rstd = rstd_in[r];
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < c.d; i += blockDim.x) {
      const float w = Elem<T>::load(yr + i) * Elem<T>::load(gamma + i);
      s1 += w;
      s2 = fmaf(w, (Elem<T>::load(xr + i) - mean) * rstd, s2);
    }
    const float2 s = group_sum<false>(s1, s2, buf, turn);
    const float m1 = s.x / (float)c.d, m2 = s.y / (float)c.d;
    for (int i = threadIdx.x; i < c.d; i += blockDim.x) {
      const float w = Elem<T>::load(yr + i) * Elem<T>::load(gamma + i);
      const float xh = (Elem<T>::load(xr + i) - mean) * rstd;
      dx[r * c.lddx + i] = Elem<T>::from_f(rstd * (w - m1 - xh * m2));
    }
  }
}

// Column sums of wide rows: CTA (a, b) takes columns 32 a .. + 31 of the rows
// b * 8 + warp, + 8 gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256)
norm_columns_kernel(moe_norm_config c, const T *__restrict__ x, const float *__restrict__ mean_in,
                    const float *__restrict__ rstd_in, const T *__restrict__ dy,
                    float *__restrict__ pg, float *__restrict__ pb) {
  __shared__ float s[2][8][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  float ag = 0.f, ab = 0.f;
  if (col < c.d) {
    for (int64_t r = (int64_t)blockIdx.y * 8 + warp; r < c.rows; r += (int64_t)gridDim.y * 8) {
      const float g = Elem<T>::load(dy + r * c.lddy + col);
      ag = fmaf(g, (Elem<T>::load(x + r * c.ldx + col) - mean_in[r]) * rstd_in[r], ag);
      ab += g;
    }
  }
  s[0][warp][lane] = ag;
  s[1][warp][lane] = ab;
  __syncthreads();
  if (warp < 2 && col < c.d) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) a += s[warp][w][lane];
    float *part = warp ? pb : pg;
    if (part) part[(int64_t)blockIdx.y * c.d + col] = a;
  }
}

// ------------------------------------------------------------------- launch
// Threads per row for rows of d elements held as vpt pieces of vec per thread
// (0: too wide).
int threads_of(int d, int vec, int vpt) {
  const int64_t per_warp = (int64_t)32 * vec * vpt;
  const int64_t warps = (d + per_warp - 1) / per_warp;
  return warps * 32 <= N_MAX_THREADS ? (int)warps * 32 : 0;
}

constexpr int kScalarPieces = 16;
template <typename T> constexpr int fwd_pieces() { return 4; }
// the gradient's column sums take two registers per element: at most 16
// elements per thread
template <typename T> constexpr int bwd_pieces() { return sizeof(T) == 2 ? 2 : 4; }

bool by_vectors(const moe_norm_config &c, int vec, bool backward) {
  return c.d % vec == 0 && c.ldx % vec == 0 &&
         (backward ? c.lddy % vec == 0 && c.lddx % vec == 0 : c.ldy % vec == 0);
}

// CTAs that walk the rows: `ctas_per_sm` per SM at most.
unsigned grid_of(int64_t rows, int groups, int most) {
  const int64_t want = (rows + groups - 1) / groups;
  return (unsigned)(want < most ? want : most);
}

// Partial rows of the column sums.
struct BwdPlan {
  int vec, threads;   // threads per row, 0: the wide kernels
  int groups, parts;
};
BwdPlan plan_backward(const moe_norm_config &c) {
  BwdPlan p;
  const int v16 = c.dtype == MOE_F32 ? 4 : 8;
  p.vec = by_vectors(c, v16, true) ? v16 : 1;
  const int pieces = p.vec == 1 ? kScalarPieces : c.dtype == MOE_F32 ? bwd_pieces<float>()
                                                                     : bwd_pieces<__nv_bfloat16>();
  p.threads = threads_of(c.d, p.vec, pieces);
  p.groups = p.threads == 32 ? 8 : 1;
  if (p.threads) {
    p.parts = (int)grid_of(c.rows, p.groups, N_MAX_PARTS);
  } else {
    p.parts = (int)grid_of(c.rows, 64, N_MAX_PARTS);
  }
  return p;
}

template <typename T, int VEC, int VPT>
cudaError_t fwd(const moe_norm_config &c, const T *x, const T *gamma, const T *beta, T *y,
                float *mean, float *rstd, int threads, cudaStream_t s) {
  if (threads == 32) {
    norm_kernel<T, VEC, VPT, true><<<grid_of(c.rows, 8, num_sms() * 4), 256, 0, s>>>(
        c, x, gamma, beta, y, mean, rstd);
  } else {
    const int per_sm = threads > 1024 / 2 ? 1 : 1024 / threads;
    norm_kernel<T, VEC, VPT, false><<<grid_of(c.rows, 1, num_sms() * per_sm), threads, 0, s>>>(
        c, x, gamma, beta, y, mean, rstd);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_typed(const moe_norm_config &c, const void *xv, const void *gv, const void *bv,
                      void *yv, float *mean, float *rstd, cudaStream_t s) {
  const T *x = (const T *)xv, *gamma = (const T *)gv, *beta = (const T *)bv;
  T *y = (T *)yv;
  constexpr int V = Vec16<T>::N;
  const bool vec = by_vectors(c, V, false);
  const int threads = threads_of(c.d, vec ? V : 1, vec ? fwd_pieces<T>() : kScalarPieces);
  if (threads == 0) {
    norm_wide_kernel<T><<<grid_of(c.rows, 1, num_sms() * 4), 512, 0, s>>>(c, x, gamma, beta, y,
                                                                          mean, rstd);
    return cudaGetLastError();
  }
  if (vec) return fwd<T, V, fwd_pieces<T>()>(c, x, gamma, beta, y, mean, rstd, threads, s);
  return fwd<T, 1, kScalarPieces>(c, x, gamma, beta, y, mean, rstd, threads, s);
}

template <typename T, int VEC, int VPT>
void bwd(const moe_norm_config &c, const BwdPlan &p, const T *x, const T *gamma, const float *mean,
         const float *rstd, const T *dy, T *dx, float *pg, float *pb, cudaStream_t s) {
  if (p.threads == 32)
    norm_backward_kernel<T, VEC, VPT, true><<<p.parts, 256, 0, s>>>(c, x, gamma, mean, rstd, dy, dx,
                                                                    pg, pb);
  else
    norm_backward_kernel<T, VEC, VPT, false><<<p.parts, p.threads, 0, s>>>(c, x, gamma, mean, rstd,
                                                                           dy, dx, pg, pb);
}

template <typename T>
cudaError_t bwd_typed(const moe_norm_config &c, const void *xv, const void *gv, const float *mean,
                      const float *rstd, const void *dyv, void *dxv, float *dgamma, float *dbeta,
                      void *scratch, cudaStream_t s) {
  const T *x = (const T *)xv, *gamma = (const T *)gv, *dy = (const T *)dyv;
  T *dx = (T *)dxv;
  const BwdPlan p = plan_backward(c);
  float *pg = nullptr, *pb = nullptr;
  const bool direct = p.parts == 1;
  if (dgamma) pg = direct ? dgamma : (float *)scratch;
  if (dbeta) pb = direct ? dbeta : (float *)scratch + (int64_t)p.parts * c.d;
  if (p.threads == 0) {
    norm_backward_wide_kernel<T><<<grid_of(c.rows, 1, num_sms() * 4), 512, 0, s>>>(
        c, x, gamma, mean, rstd, dy, dx);
    if (pg || pb)
      norm_columns_kernel<T><<<dim3((c.d + 31) / 32, p.parts), 256, 0, s>>>(c, x, mean, rstd, dy,
                                                                            pg, pb);
  } else if (p.vec > 1) {
    bwd<T, Vec16<T>::N, bwd_pieces<T>()>(c, p, x, gamma, mean, rstd, dy, dx, pg, pb, s);
  } else {
    bwd<T, 1, kScalarPieces>(c, p, x, gamma, mean, rstd, dy, dx, pg, pb, s);
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && !direct && (pg || pb))
    e = launch_pdl(column_sum_kernel, dim3((c.d + 31) / 32, 2), dim3(256), 0, s,
                   (const float *)pg, (const float *)pb, p.parts, (int)c.d, dgamma, dbeta);
  return e;
}

}  // namespace

cudaError_t launch_norm(const moe_norm_config &c, const void *x, const void *gamma,
                        const void *beta, void *y, float *mean, float *rstd, cudaStream_t s) {
  return c.dtype == MOE_F32 ? fwd_typed<float>(c, x, gamma, beta, y, mean, rstd, s)
                            : fwd_typed<__nv_bfloat16>(c, x, gamma, beta, y, mean, rstd, s);
}

size_t norm_backward_scratch(const moe_norm_config &c) {
  return c.rows > 0 ? (size_t)plan_backward(c).parts * 2 * c.d * 4 : 0;
}

cudaError_t launch_norm_backward(const moe_norm_config &c, const void *x, const void *gamma,
                                 const float *mean, const float *rstd, const void *dy, void *dx,
                                 float *dgamma, float *dbeta, void *scratch, cudaStream_t s) {
  return c.dtype == MOE_F32
             ? bwd_typed<float>(c, x, gamma, mean, rstd, dy, dx, dgamma, dbeta, scratch, s)
             : bwd_typed<__nv_bfloat16>(c, x, gamma, mean, rstd, dy, dx, dgamma, dbeta, scratch, s);
}

}  // namespace moe
