// The cross entropy of a few tokens, and in fp32 its gradient: as many streams over the
// vocabulary's rows W [entries][d] as there are warps.
//
//   loss_stream_kernel   l[t][v] = sum_k x[t][k] W[v][k], reduced to a maximum and a sum of
//                        exponentials per token, or (GRAD) turned into its gradient dl [v][pitch];
//   loss_stream_grads_kernel   dx[t] = sum_v dl[v][t] W[v] and dW[v] = sum_t dl[v][t] x[t] in one
//                        pass, W read once and dW written once.
// Bytes bound both: a value of W serves at most 8 tokens.  In bf16 the tensor cores' kernel
// is as fast from 4 tokens on.  It / the streams, us, d 2880, 131072 entries: one token 130 / 117
// (6.5 TB/s), 2 130 / 120, 3 130 / 131, 5 130 / 229; d 4096, 32000 entries, 3 tokens 53 / 50; d 8192,
// 8192 entries 45 / 28.  In fp32 a tile of 32 x 32 outputs reads and multiplies for 32 tokens
// whatever their number.  Tiles / streams, us: one token,
// d 4096, 50000 entries 812 / 127 (6.5 TB/s) and its gradient 1648 / 399; 8 tokens 816 / 153 and
// 1669 / 479; d 512, 8192 entries, 8 tokens 20.8 / 11.0 and 42.7 / 28.5; d 64 12.2 / 10.0 and
// 22.9 / 17.8; d 8 10.6 / 10.8 and 21.2 / 28.7.
#include <math.h>

#include "common.cuh"
#include "fp32x2.cuh"
#include "launch.h"
#include "loss.h"
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int S_THREADS = 512, S_WARPS = S_THREADS / 32;
constexpr int S_X = 48 * 1024;      // floats of the tokens' rows in shared memory at most
constexpr int S_GRADS = 256;        // threads of the second kernel
constexpr int S_DL = 256;           // entries whose dl it holds
constexpr int S_TOKENS = 8, S_TOKENS_BF16 = 4;   // at most
constexpr int S_MIN_D = 64;

struct StreamArgs {
  LossProduct p;
  float *dl;
  int *status;
};

// Sums of V values over a warp (V a power of two, 32 at most): lane l ends with that of
// value l / (32 / V).
template <int V>
__device__ __forceinline__ float spread_sums(float (&v)[V]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int s = V / 2; s >= 1; s /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < s; ++i)
      v[i] = (upper ? v[i + s] : v[i]) + __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i + s], o);
  }
  for (; o >= 1; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

// Entries that a warp takes at a time.  (8 tokens, 4 of them: registers spill, 175 us for 153 at
// d 4096, 50000 entries.)
__host__ __device__ constexpr int entries_of(int tokens) { return tokens > 4 ? 2 : 4; }

// Columns of a token's row in shared memory.
template <typename T>
__host__ __device__ constexpr int whole_steps(int d) {
  constexpr int STEP = 32 * Vec16<T>::N;
  return (d + STEP - 1) / STEP * STEP;
}

// A warp takes R neighbouring entries at a time, whose sums for NT tokens it spreads
// over its lanes; a lane goes on with one of them.
template <typename T, int NT, bool GRAD>
__global__ void __launch_bounds__(S_THREADS, 1) loss_stream_kernel(const __grid_constant__ StreamArgs a) {
  constexpr int R = entries_of(NT), V = R * NT, EACH = 32 / V;
  constexpr int N = Vec16<T>::N, STEP = 32 * N;   // columns of a lane, and of a warp
  extern __shared__ __align__(16) float xs[];     // [NT][d rounded up to whole steps]
  __shared__ float2 pairs[S_WARPS][32];
  const LossProduct &p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = p.d, entries = p.entries;
  pdl_wait();
  if (status_failed(a.status)) return;
  const int count = GRAD ? min(max(p.range[1], 0), p.n) : p.n;
  // (a step's first four columns of every lane, then in bf16 the other four)
  const int pitch = whole_steps<T>(d);
  for (int i = threadIdx.x; i < NT * (d / N); i += S_THREADS) {
    const int k = i / (d / N), c = i - k * (d / N);
    float f[N] = {};
    if (k < p.n) unpack16<T>(static_cast<const uint4 *>(p.x)[i], f);
    float *to = xs + k * pitch + c / 32 * STEP + c % 32 * 4;
#pragma unroll
    for (int h = 0; h < N / 4; ++h)
      *reinterpret_cast<float4 *>(to + h * 128) =
          make_float4(f[h * 4], f[h * 4 + 1], f[h * 4 + 2], f[h * 4 + 3]);
  }
  // this lane's token and entry of the R
  const int q = lane / EACH, t = q % NT, r = q / NT;
  const bool lead = lane % EACH == 0, there = t < count;
  const int target = there ? p.target[t] - p.v0 : -1;
  float lse = 0.f, dloss = 0.f, slope = 0.f;
  if (GRAD && there) {
    lse = p.lse[t];
    dloss = p.dloss[t];
    slope = fmaf(2.f * p.z_loss, lse, 1.f);
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int e0 = ((int)blockIdx.x * S_WARPS + warp) * R; e0 < entries;
       e0 += (int)gridDim.x * S_WARPS * R) {
    const T *row[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      row[i] = static_cast<const T *>(p.W) + (int64_t)min(e0 + i, entries - 1) * d;
    float2 acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = both(0.f);
#pragma unroll 2
    for (int c = lane * N, at = lane * 4; c < d; c += STEP, at += STEP) {
      float w[R][N];
#pragma unroll
      for (int i = 0; i < R; ++i) unpack16<T>(__ldcs(reinterpret_cast<const uint4 *>(row[i] + c)), w[i]);
#pragma unroll
      for (int k = 0; k < NT; ++k) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const float4 v = *reinterpret_cast<const float4 *>(xs + k * pitch + at + h * 128);
#pragma unroll
          for (int i = 0; i < R; ++i) {
            float2 &s = acc[i * NT + k];
            s = fma2(make_float2(w[i][h * 4], w[i][h * 4 + 1]), make_float2(v.x, v.y), s);
            s = fma2(make_float2(w[i][h * 4 + 2], w[i][h * 4 + 3]), make_float2(v.z, v.w), s);
          }
        }
      }
    }
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = acc[i].x + acc[i].y;
    const float l = spread_sums<V>(v);
    const int e = e0 + r;
    if (e >= entries || !lead) continue;
    if constexpr (GRAD) {
      float g = 0.f;
      if (there) {
        const float prob = expf(l - lse) * slope;
        g = dloss * (target == e ? prob - 1.f : prob);
      }
      float *to = a.dl + (int64_t)e * p.pitch;
      if (t < p.pitch) to[t] = g;
      if (t == NT - 1)
        for (int k = NT; k < p.pitch; ++k) to[k] = 0.f;
    } else {
      const float up = fmaxf(top, l), shift = shift_of(up);
      sum = sum * expf(top - shift) + expf(l - shift);
      top = up;
      if (there && e == target) p.at[t] = l;
    }
  }
  pdl_launch_dependents();
  if constexpr (!GRAD) {
    // the CTA's pairs of a token, by a warp
    pairs[warp][lane] = make_float2(top, sum);
    __syncthreads();
    for (int k = warp; k < p.n; k += S_WARPS) {
      float most = -INFINITY;
      for (int i = lane; i < S_WARPS * R; i += 32)
        most = fmaxf(most, pairs[i / R][(i % R * NT + k) * EACH].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      float s = 0.f;
      for (int i = lane; i < S_WARPS * R; i += 32) {
        const float2 v = pairs[i / R][(i % R * NT + k) * EACH];
        s += v.y * expf(v.x - shift_of(most));
      }
      s = warp_sum_xor(s);
      if (lane == 0) p.sums[(int64_t)k * p.chunks + blockIdx.x] = make_float2(most, s);
    }
  }
}

struct StreamGrads {
  LossProduct p;
  const float *dl;
  float *dW;        // or nullptr
  int want_dx, tx;  // threads across the columns, four each; the others take entries in turn
  int *status;
};
// A CTA takes 4 tx columns of a range of the entries, whose dl it stages S_DL entries at a time.
template <int NT>
__global__ void __launch_bounds__(S_GRADS) loss_stream_grads_kernel(const __grid_constant__ StreamGrads a) {
  constexpr int U = NT == 8 ? 4 : 8;   // entries whose rows of W are loaded together
  __shared__ __align__(16) float dl[S_DL][NT];
  __shared__ float4 part[S_GRADS];
  const LossProduct &p = a.p;
  const int tx = threadIdx.x % a.tx, ty = threadIdx.x / a.tx, rows = S_GRADS / a.tx;
  const int col = (blockIdx.x * a.tx + tx) * 4;
  pdl_wait();
  if (status_failed(a.status)) return;
  const int each = (p.entries + (int)gridDim.y - 1) / (int)gridDim.y;
  const int end = min(p.entries, ((int)blockIdx.y + 1) * each);
  const bool active = col < p.d;
  float4 x[NT], dx[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    dx[t] = x[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (active && t < p.n)
      x[t] = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + (int64_t)t * p.d + col);
  }
  for (int e0 = blockIdx.y * each; e0 < end; e0 += S_DL) {
    const int here = min(S_DL, end - e0);
    __syncthreads();
    for (int i = threadIdx.x; i < here * NT; i += S_GRADS)
      dl[i / NT][i % NT] = i % NT < p.n ? a.dl[(int64_t)(e0 + i / NT) * p.pitch + i % NT] : 0.f;
    __syncthreads();
    if (!active) continue;
    const int64_t at = (int64_t)e0 * p.d + col;
    const float *W = static_cast<const float *>(p.W) + at;
    float *dW = a.dW ? a.dW + at : nullptr;
    for (int k0 = ty; k0 < here; k0 += U * rows) {
      float4 w[U];
      if (a.want_dx) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = k0 + u * rows;
          if (k < here) w[u] = __ldcs(reinterpret_cast<const float4 *>(W + (int64_t)k * p.d));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * rows;
        if (k >= here) break;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float g = dl[k][t];
          if (a.want_dx)
            dx[t] = make_float4(fmaf(g, w[u].x, dx[t].x), fmaf(g, w[u].y, dx[t].y),
                                fmaf(g, w[u].z, dx[t].z), fmaf(g, w[u].w, dx[t].w));
          s = make_float4(fmaf(g, x[t].x, s.x), fmaf(g, x[t].y, s.y), fmaf(g, x[t].z, s.z),
                          fmaf(g, x[t].w, s.w));
        }
        if (dW) __stcs(reinterpret_cast<float4 *>(dW + (int64_t)k * p.d), s);
      }
    }
  }
  pdl_launch_dependents();
  if (!a.want_dx) return;
  // the sums over this CTA's entries, in order
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t >= p.n) break;
    __syncthreads();
    part[threadIdx.x] = dx[t];
    __syncthreads();
    if (ty != 0 || !active) continue;
    float4 s = part[tx];
    for (int k = 1; k < rows; ++k) {
      const float4 v = part[k * a.tx + tx];
      s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    *reinterpret_cast<float4 *>(p.planes + ((int64_t)blockIdx.y * p.n + t) * p.d + col) = s;
  }
}

// Threads across the columns in the second kernel.
int across(int d) {
  int tx = 1;
  while (tx < S_GRADS && tx * 4 < d) tx *= 2;
  return tx;
}

template <typename T, int NT, bool GRAD>
cudaError_t launch(const StreamArgs &a, int grid, cudaStream_t s) {
  static bool set = false;
  if (!set) {
    const cudaError_t e = cudaFuncSetAttribute(
        loss_stream_kernel<T, NT, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_X * 4);
    if (e != cudaSuccess) return e;
    set = true;
  }
  return launch_pdl(loss_stream_kernel<T, NT, GRAD>, dim3(grid), dim3(S_THREADS),
                    (size_t)NT * whole_steps<T>(a.p.d) * 4, s, a);
}

int tokens_of(int n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : S_TOKENS; }

}  // namespace

bool loss_stream_supported(const moe_loss_config &c) {
  const int64_t row = c.dtype == MOE_F32 ? whole_steps<float>(c.d) : whole_steps<__nv_bfloat16>(c.d);
  return c.n >= 1 && c.n <= (c.dtype == MOE_F32 ? S_TOKENS : S_TOKENS_BF16) && c.d >= S_MIN_D && tokens_of(c.n) * row <= S_X;
}

int loss_stream_chunks(const moe_loss_config &c) {
  const int each = S_WARPS * entries_of(c.n), want = (c.vocab + each - 1) / each;
  return want < num_sms() ? want : num_sms();
}

int loss_stream_splits(int d, int entries, int most) {
  const int tx = across(d), columns = (d + 4 * tx - 1) / (4 * tx);
  const int by_rows = entries / (16 * (S_GRADS / tx));
  int s = 608 / columns;
  if (s > most) s = most;
  if (s > by_rows) s = by_rows;
  return s < 1 ? 1 : s;
}

template <typename T, bool GRAD>
static cudaError_t launch_tokens(const StreamArgs &a, int grid, cudaStream_t s) {
  switch (tokens_of(a.p.n)) {
    case 1: return launch<T, 1, GRAD>(a, grid, s);
    case 2: return launch<T, 2, GRAD>(a, grid, s);
    case 4: return launch<T, 4, GRAD>(a, grid, s);
    default: return launch<T, sizeof(T) == 4 ? S_TOKENS : S_TOKENS_BF16, GRAD>(a, grid, s);
  }
}
cudaError_t launch_loss_stream_sums(int dtype, const LossProduct &p, int grid, int *status,
                                    cudaStream_t s) {
  const StreamArgs a{p, nullptr, status};
  return dtype == MOE_F32 ? launch_tokens<float, false>(a, grid, s)
                          : launch_tokens<__nv_bfloat16, false>(a, grid, s);
}
cudaError_t launch_loss_stream_logit_grad(const LossProduct &p, float *dl, int grid, int *status,
                                          cudaStream_t s) {
  return launch_tokens<float, true>(StreamArgs{p, dl, status}, grid, s);
}

cudaError_t launch_loss_stream_grads(const LossProduct &p, const float *dl, float *dW, bool want_dx,
                                     int *status, cudaStream_t s) {
  const StreamGrads a{p, dl, dW, want_dx, across(p.d), status};
  const dim3 grid((p.d + 4 * a.tx - 1) / (4 * a.tx), p.splits);
  switch (tokens_of(p.n)) {
    case 1: return launch_pdl(loss_stream_grads_kernel<1>, grid, dim3(S_GRADS), 0, s, a);
    case 2: return launch_pdl(loss_stream_grads_kernel<2>, grid, dim3(S_GRADS), 0, s, a);
    case 4: return launch_pdl(loss_stream_grads_kernel<4>, grid, dim3(S_GRADS), 0, s, a);
    default: return launch_pdl(loss_stream_grads_kernel<S_TOKENS>, grid, dim3(S_GRADS), 0, s, a);
  }
}

}  // namespace moe
