// The joint of a block with the residual stream, and its gradient (moe.h has
// the formulas).
#include "common.cuh"
#include "launch.h"
#include "philox.cuh"
#include "rows_common.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int J_PARTS = 152;   // partial rows of the column sums, at most
constexpr int J_SUMS = 4;      // sum u bh, sum u, sum dy rh, sum dy

template <typename T>
struct Fwd {
  moe_join_config c;
  const T *x, *b, *gate, *post_gamma, *post_beta, *pre_gamma, *pre_beta;
  const RngState *rng;
  T *r, *y;
  float *stats;
  int threshold;
  float factor;
};
template <typename T>
struct Bwd {
  moe_join_config c;
  const T *b, *r, *gate, *post_gamma, *post_beta, *pre_gamma, *pre_beta;
  const float *stats;
  const RngState *rng;
  const T *dr, *dy;
  T *dx, *db;
  int threshold;
  float factor;
  int has_b;          // b is there: a post norm, or the gate's gradient is wanted
  float2 *means;      // wide rows: the pre norm's two means of each row
  float *parts;       // [part][J_SUMS][d]
  int sums;           // bit i: column sum i is wanted
};

template <typename T>
__device__ __forceinline__ float at_or(const T *v, int i, float other) {
  return v ? Elem<T>::load(v + i) : other;
}

// ------------------------------------------------- rows of any width, in passes
// One CTA per row, which reads it again (from L2) for each pass; a thread takes
// blocks of eight elements, as the generator gives its bits.
constexpr int J_WIDE = 512;

// Element i of the joined row, in fp32.
template <typename T>
__device__ __forceinline__ float joined(const Fwd<T> &a, const T *xr, const T *br, int i,
                                        float mean, float rstd, bool keep) {
  float z = Elem<T>::load(br + i);
  if (a.c.post != MOE_NORM_NONE)
    z = fmaf((z - mean) * rstd, Elem<T>::load(a.post_gamma + i), at_or(a.post_beta, i, 0.f));
  z = keep ? z * a.factor : 0.f;
  return fmaf(a.c.scale, Elem<T>::load(xr + i), z * at_or(a.gate, i, 1.f));
}

template <typename T>
__global__ void __launch_bounds__(J_WIDE) join_wide_kernel(const __grid_constant__ Fwd<T> a) {
  __shared__ float buf[2][32];
  const moe_join_config &c = a.c;
  const int warps = J_WIDE / 32, blocks = (c.d + 7) / 8;
  const RngState st = a.threshold ? *a.rng : RngState{0, 0};
  int turn = 0;
  auto sum = [&](float v) { return group_sum<false>(v, buf, turn, warps); };
  for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x) {
    const T *xr = a.x + row * c.ldx, *br = a.b + row * c.ldb;
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f, s;
    if (c.post == MOE_NORM_LAYER) {
      s = 0.f;
      for (int i = threadIdx.x; i < c.d; i += J_WIDE) s += Elem<T>::load(br + i);
      mean1 = sum(s) / (float)c.d;
    }
    if (c.post != MOE_NORM_NONE) {
      s = 0.f;
      for (int i = threadIdx.x; i < c.d; i += J_WIDE) {
        const float v = Elem<T>::load(br + i) - mean1;
        s = fmaf(v, v, s);
      }
      rstd1 = 1.f / sqrtf(sum(s) / (float)c.d + c.eps);
    }
    auto each = [&](auto &&f) {
      for (int k = threadIdx.x; k < blocks; k += J_WIDE) {
        const uint32_t keep =
            a.threshold ? dropout_keep(st, k, (uint32_t)row, a.threshold) : 0xffu;
        for (int i = k * 8; i < min(c.d, k * 8 + 8); ++i)
          f(i, joined(a, xr, br, i, mean1, rstd1, keep >> (i & 7) & 1));
      }
    };
    if (c.pre == MOE_NORM_LAYER) {
      s = 0.f;
      each([&](int, float v) { s += v; });
      mean2 = sum(s) / (float)c.d;
    }
    if (c.pre != MOE_NORM_NONE) {
      s = 0.f;
      each([&](int, float v) { s = fmaf(v - mean2, v - mean2, s); });
      rstd2 = 1.f / sqrtf(sum(s) / (float)c.d + c.eps);
    }
    each([&](int i, float v) {
      a.r[row * c.ldr + i] = Elem<T>::from_f(v);
      if (c.pre != MOE_NORM_NONE)
        a.y[row * c.ldy + i] = Elem<T>::from_f(fmaf(
            (v - mean2) * rstd2, Elem<T>::load(a.pre_gamma + i), at_or(a.pre_beta, i, 0.f)));
    });
    if (a.stats && threadIdx.x == 0) {
      const float v[4] = {mean1, rstd1, mean2, rstd2};
      for (int i = 0; i < 4; ++i) a.stats[i * c.rows + row] = v[i];
    }
  }
}

// The statistics of a row as the forward left them.
template <typename T>
__device__ __forceinline__ float4 stats_of(const Bwd<T> &a, int64_t row) {
  float4 v = make_float4(0.f, 1.f, 0.f, 1.f);
  if (a.c.post != MOE_NORM_NONE) {
    v.x = a.stats[row];
    v.y = a.stats[a.c.rows + row];
  }
  if (a.c.pre != MOE_NORM_NONE && a.dy) {
    v.z = a.stats[2 * a.c.rows + row];
    v.w = a.stats[3 * a.c.rows + row];
  }
  return v;
}

// The stream's gradient R at element i, from the pre norm's means m.
template <typename T>
__device__ __forceinline__ float stream_grad(const Bwd<T> &a, int64_t row, int i, float4 st,
                                             float2 m) {
  float g = a.dr ? Elem<T>::load(a.dr + row * a.c.lddr + i) : 0.f;
  if (a.dy) {
    const float w = Elem<T>::load(a.dy + row * a.c.lddy + i) * Elem<T>::load(a.pre_gamma + i);
    const float rh = (Elem<T>::load(a.r + row * a.c.ldr + i) - st.z) * st.w;
    g = fmaf(st.w, w - m.x - rh * m.y, g);
  }
  return g;
}

template <typename T>
__global__ void __launch_bounds__(J_WIDE)
join_backward_wide_kernel(const __grid_constant__ Bwd<T> a) {
  __shared__ float2 buf[2][32];
  const moe_join_config &c = a.c;
  const int warps = J_WIDE / 32, blocks = (c.d + 7) / 8;
  const float inv_d = 1.f / (float)c.d;
  const RngState rng = a.threshold ? *a.rng : RngState{0, 0};
  int turn = 0;
  for (int64_t row = blockIdx.x; row < c.rows; row += gridDim.x) {
    const float4 st = stats_of(a, row);
    float2 m = make_float2(0.f, 0.f), q = m;
    if (a.dy) {
      float s1 = 0.f, s2 = 0.f;
      for (int i = threadIdx.x; i < c.d; i += J_WIDE) {
        const float w = Elem<T>::load(a.dy + row * c.lddy + i) * Elem<T>::load(a.pre_gamma + i);
        s1 += w;
        s2 = fmaf(w, (Elem<T>::load(a.r + row * c.ldr + i) - st.z) * st.w, s2);
      }
      m = group_sum2<false>(s1, s2, buf, turn, 0, warps);
      m = make_float2(c.pre == MOE_NORM_LAYER ? m.x * inv_d : 0.f, m.y * inv_d);
    }
    if (a.means && threadIdx.x == 0) a.means[row] = m;
    // f(i, R, the gradient of the post norm's output times its gamma, bh)
    auto each = [&](auto &&f) {
      for (int k = threadIdx.x; k < blocks; k += J_WIDE) {
        const uint32_t keep =
            a.threshold ? dropout_keep(rng, k, (uint32_t)row, a.threshold) : 0xffu;
        for (int i = k * 8; i < min(c.d, k * 8 + 8); ++i) {
          const float g = stream_grad(a, row, i, st, m);
          const float u = keep >> (i & 7) & 1 ? g * a.factor : 0.f;
          float bh = 0.f, w = u * at_or(a.gate, i, 1.f);
          if (c.post != MOE_NORM_NONE) {
            bh = (Elem<T>::load(a.b + row * c.ldb + i) - st.x) * st.y;
            w *= Elem<T>::load(a.post_gamma + i);
          }
          f(i, g, w, bh);
        }
      }
    };
    if (c.post != MOE_NORM_NONE && a.db) {
      float s1 = 0.f, s2 = 0.f;
      each([&](int, float, float w, float bh) {
        s1 += w;
        s2 = fmaf(w, bh, s2);
      });
      q = group_sum2<false>(s1, s2, buf, turn, 0, warps);
      q = make_float2(c.post == MOE_NORM_LAYER ? q.x * inv_d : 0.f, q.y * inv_d);
    }
    if (a.dx || a.db)
      each([&](int i, float g, float w, float bh) {
        if (a.dx) a.dx[row * c.lddx + i] = Elem<T>::from_f(c.scale * g);
        if (a.db) a.db[row * c.lddb + i] = Elem<T>::from_f(st.y * (w - q.x - bh * q.y));
      });
  }
}

// Column sums of wide rows: CTA (a, b) takes columns 32 a .. + 31 of the rows
// 8 b + warp, + 8 gridDim.y, ...
template <typename T>
__global__ void __launch_bounds__(256) join_columns_kernel(const __grid_constant__ Bwd<T> a) {
  __shared__ float s[J_SUMS][8][33];
  const moe_join_config &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  const RngState rng = a.threshold ? *a.rng : RngState{0, 0};
  float v[J_SUMS] = {};
  if (col < c.d) {
    for (int64_t row = (int64_t)blockIdx.y * 8 + warp; row < c.rows;
         row += (int64_t)gridDim.y * 8) {
      const float4 st = stats_of(a, row);
      const float g = stream_grad(a, row, col, st, a.means[row]);
      const bool keep =
          !a.threshold ||
          (dropout_keep(rng, col >> 3, (uint32_t)row, a.threshold) >> (col & 7) & 1);
      const float u = keep ? g * a.factor : 0.f;
      if (a.has_b) v[0] = fmaf(u, (Elem<T>::load(a.b + row * c.ldb + col) - st.x) * st.y, v[0]);
      v[1] += u;
      if (a.dy) {
        const float dy = Elem<T>::load(a.dy + row * c.lddy + col);
        v[2] = fmaf(dy, (Elem<T>::load(a.r + row * c.ldr + col) - st.z) * st.w, v[2]);
        v[3] += dy;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < J_SUMS; ++i) s[i][warp][lane] = v[i];
  __syncthreads();
  if (warp < J_SUMS && col < c.d) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s[warp][w][lane];
    a.parts[((int64_t)blockIdx.y * J_SUMS + warp) * c.d + col] = t;
  }
}

// The vectors' gradients from the partial column sums, added in a fixed order:
// with A, B, C, E the sums of u bh, u, dy rh and dy,
//   dgate = gamma1 A + beta1 B,  dgamma1 = gate A,  dbeta1 = gate B,  dgamma2 = C,  dbeta2 = E.
// Warp w of 32 adds part rows w, w + 32, ...; a butterfly adds the warps' sums.
template <typename T>
struct FinishArgs {
  const float *parts;
  int count, d, sums;
  const T *gate, *post_gamma, *post_beta;
  moe_join_grads g;
};
template <typename T>
__global__ void __launch_bounds__(1024) join_finish_kernel(const __grid_constant__ FinishArgs<T> a) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = blockIdx.x * 32 + lane, out = blockIdx.x * 32 + warp;
  float total[J_SUMS];
  pdl_wait();
#pragma unroll
  for (int i = 0; i < J_SUMS; ++i) {
    total[i] = 0.f;
    if (!(a.sums >> i & 1)) continue;
    float v = 0.f;
    if (mine < a.d) {
#pragma unroll 5
      for (int p = warp; p < a.count; p += 32)
        v += a.parts[((int64_t)p * J_SUMS + i) * a.d + mine];
    }
    s[warp][lane] = v;
    __syncthreads();
    total[i] = warp_sum_xor(s[lane][warp]);
    __syncthreads();
  }
  if (lane != 0 || out >= a.d) return;
  const float gate = at_or(a.gate, out, 1.f);
  if (a.g.gate)
    a.g.gate[out] =
        fmaf(at_or(a.post_gamma, out, 1.f), total[0], at_or(a.post_beta, out, 0.f) * total[1]);
  if (a.g.post_gamma) a.g.post_gamma[out] = gate * total[0];
  if (a.g.post_beta) a.g.post_beta[out] = gate * total[1];
  if (a.g.pre_gamma) a.g.pre_gamma[out] = total[2];
  if (a.g.pre_beta) a.g.pre_beta[out] = total[3];
}

int grid_of(int64_t rows, int64_t most) { return (int)(rows < most ? rows : most); }

template <typename T>
cudaError_t forward(const moe_join_config &c, int threshold, const JoinForward &f, cudaStream_t s) {
  Fwd<T> a{};
  a.c = c;
  a.x = (const T *)f.x;
  a.b = (const T *)f.b;
  a.gate = (const T *)f.w.gate;
  a.post_gamma = (const T *)f.w.post_gamma;
  a.post_beta = (const T *)f.w.post_beta;
  a.pre_gamma = (const T *)f.w.pre_gamma;
  a.pre_beta = (const T *)f.w.pre_beta;
  a.rng = reinterpret_cast<const RngState *>(f.rng);
  a.r = (T *)f.r;
  a.y = (T *)f.y;
  a.stats = f.stats;
  a.threshold = threshold;
  a.factor = dropout_factor(threshold);
  join_wide_kernel<T><<<grid_of(c.rows, (int64_t)num_sms() * 4), J_WIDE, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const moe_join_config &c, int threshold, const JoinBackward &f, void *scratch,
                     cudaStream_t s) {
  const moe_join_grads &g = f.grads;
  Bwd<T> a{};
  a.c = c;
  a.b = (const T *)f.b;
  a.r = (const T *)f.r;
  a.gate = (const T *)f.w.gate;
  a.post_gamma = (const T *)f.w.post_gamma;
  a.post_beta = (const T *)f.w.post_beta;
  a.pre_gamma = (const T *)f.w.pre_gamma;
  a.pre_beta = (const T *)f.w.pre_beta;
  a.stats = f.stats;
  a.rng = reinterpret_cast<const RngState *>(f.rng);
  a.dr = (const T *)f.dr;
  a.dy = (const T *)f.dy;
  a.dx = (T *)f.dx;
  a.db = (T *)f.db;
  a.threshold = threshold;
  a.factor = dropout_factor(threshold);
  a.has_b = c.post != MOE_NORM_NONE || g.gate;
  a.sums = (g.gate || g.post_gamma ? 1 : 0) | ((g.gate && f.w.post_beta) || g.post_beta ? 2 : 0) |
           (g.pre_gamma ? 4 : 0) | (g.pre_beta ? 8 : 0);
  const int parts = grid_of((c.rows + 7) / 8, 64);
  a.parts = (float *)scratch;
  a.means = (float2 *)((char *)scratch + (size_t)J_PARTS * J_SUMS * c.d * 4);
  join_backward_wide_kernel<T><<<grid_of(c.rows, (int64_t)num_sms() * 4), J_WIDE, 0, s>>>(a);
  if (a.sums)
    join_columns_kernel<T><<<dim3((c.d + 31) / 32, parts), 256, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.sums) return e;
  FinishArgs<T> fin{a.parts, parts, c.d, a.sums, a.gate, a.post_gamma, a.post_beta, g};
  return launch_pdl(join_finish_kernel<T>, dim3((c.d + 31) / 32), dim3(1024), 0, s, fin);
}

}  // namespace

cudaError_t launch_join(const moe_join_config &c, int threshold, const JoinForward &f,
                        cudaStream_t s) {
  return c.dtype == MOE_F32 ? forward<float>(c, threshold, f, s)
                            : forward<__nv_bfloat16>(c, threshold, f, s);
}

size_t join_backward_scratch(const moe_join_config &c) {
  return c.rows > 0 ? (size_t)J_PARTS * J_SUMS * c.d * 4 + (size_t)c.rows * sizeof(float2) : 0;
}

cudaError_t launch_join_backward(const moe_join_config &c, int threshold, const JoinBackward &f,
                                 void *scratch, cudaStream_t s) {
  return c.dtype == MOE_F32 ? backward<float>(c, threshold, f, scratch, s)
                            : backward<__nv_bfloat16>(c, threshold, f, scratch, s);
}

}  // namespace moe
