// Layer norm and its gradient.
//   y_i = (x_i - mean) rstd gamma_i + beta_i
//   dx_i = rstd (w_i - sum w / d - xh_i sum w xh / d),   w_i = dy_i gamma_i
//   dgamma_i = sum_rows dy_i xh_i,   dbeta_i = sum_rows dy_i
// Both are streams through HBM: the forward reads and writes each row once,
// the gradient reads x and dy once and writes dx.  A row lives in the
// registers of a group of threads (a warp for short rows, else up to a CTA),
// so the variance is summed around the mean without a second read.  Groups
// walk the rows with a grid stride.  Rows of 16-byte vectors arrive through a
// ring in shared memory that each thread fills for itself, several rows ahead
// (cp.async; no other thread reads its part, so no barrier guards the ring):
// with one row ahead in registers the gradient's one CTA per SM waited for
// memory (the kernel at 16384 x 7168 bf16 285 us, 130 now; 135 the whole call).
// The sums use two fp32 values per instruction: the norms are bound by
// instruction issue before they are by HBM.
// In the gradient a thread owns the same columns of every row it meets, so the
// column sums grow in its registers; each CTA writes one partial row and a
// second launch adds the partials in order (no atomics: the result does not
// depend on timing).  All statistics and sums are fp32.
#include "common.cuh"
#include "fp32x2.cuh"
#include "launch.h"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int N_MAX_PARTS = 152;   // partial rows of the column sums: one CTA per SM
constexpr int N_FWD_THREADS = 512, N_BWD_THREADS = 512;
constexpr int N_FWD_STAGES = 3;
constexpr int N_SMEM = 208 * 1024;   // dynamic shared memory of a CTA at most
// rows in a thread's ring: 512 threads hold 192 KB of them
constexpr int bwd_stages(int vpt) { return vpt == 2 ? 6 : 3; }

// How a thread's share of a row is cut: chunks of 16 bytes, or (rows that are
// not whole vectors) two elements tpr apart.  H pairs per chunk.
template <typename T, int VEC>
struct Chunk {
  static constexpr int H = VEC / 2, SPAN = VEC;
  static __device__ __forceinline__ void unpack(uint4 raw, float2 *p) {
    unpack16<T>(raw, reinterpret_cast<float *>(p));
  }
  static __device__ __forceinline__ void load(const T *row, int col, int, int, float2 *p) {
    unpack(*reinterpret_cast<const uint4 *>(row + col), p);
  }
  static __device__ __forceinline__ void store(T *row, int col, int, int, const float2 *p) {
    *reinterpret_cast<uint4 *>(row + col) = pack16<T>(reinterpret_cast<const float *>(p));
  }
  static __device__ __forceinline__ void mask(int, int, int, float2 *) {}
};
template <typename T>
struct Chunk<T, 1> {
  static constexpr int H = 1, SPAN = 2;
  static __device__ __forceinline__ void load(const T *row, int col, int tpr, int d, float2 *p) {
    p->x = Elem<T>::load(row + col);
    p->y = col + tpr < d ? Elem<T>::load(row + col + tpr) : 0.f;
  }
  static __device__ __forceinline__ void store(T *row, int col, int tpr, int d, const float2 *p) {
    row[col] = Elem<T>::from_f(p->x);
    if (col + tpr < d) row[col + tpr] = Elem<T>::from_f(p->y);
  }
  // clears the second element where there is none
  static __device__ __forceinline__ void mask(int col, int tpr, int d, float2 *p) {
    if (col + tpr >= d) p->y = 0.f;
  }
};

__device__ __forceinline__ void copy16_async(uint4 *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows that are not whole vectors arrive as the aligned 16-byte pieces that
// cover them, in a slot of their group's own: copies a row of d elements into
// slot, whose first element then lies (address of src) % 16 bytes into it.
// `end`: past the last element of the tensor; a piece that reaches over it is
// copied element by element.  The group's threads read one another's pieces.
__host__ __device__ constexpr int slot_bytes(int d, int elem) { return (d * elem + 15) / 16 * 16 + 16; }
template <typename T>
__device__ __forceinline__ int head_of(const T *src) {
  return (int)(reinterpret_cast<uintptr_t>(src) & 15);
}
template <typename T>
__device__ __forceinline__ void copy_row(uint8_t *slot, const T *src, int d, const T *end, int tid,
                                         int tpr) {
  const int head = head_of(src);
  const uint8_t *base = reinterpret_cast<const uint8_t *>(src) - head;
  const int pieces = (head + d * (int)sizeof(T) + 15) >> 4;
  for (int v = tid; v < pieces; v += tpr) {
    const uint8_t *p = base + v * 16;
    if (p + 16 <= reinterpret_cast<const uint8_t *>(end)) {
      copy16_async(reinterpret_cast<uint4 *>(slot + v * 16), p);
    } else {
      const T *from = reinterpret_cast<const T *>(p);
      T *to = reinterpret_cast<T *>(slot + v * 16);
      for (int i = 0; from + i < end; ++i) to[i] = from[i];
    }
  }
}

// Sum over the group of `warps` warps this warp belongs to (its warps are
// neighbours; every thread of the CTA takes part): a butterfly, then one over
// the warps' sums, which pass through one of two alternating buffers (a buffer
// is written again only after the barrier of the sum in between, which every
// reader of it has reached).
template <bool WARP>
__device__ __forceinline__ float group_sum(float a, float (*buf)[32], int &turn, int warps) {
  a = warp_sum_xor(a);
  if (WARP) return a;
  float *s = buf[turn];
  turn ^= 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s[warp] = a;
  __syncthreads();
  return warp_sum_xor(lane < warps ? s[warp / warps * warps + lane] : 0.f);
}
// Two sums at once: after one exchange the lower half warp carries a and the
// upper one b, so that two butterflies cost the shuffles of one.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <bool WARP>
__device__ __forceinline__ float2 group_sum2(float a, float b, float2 (*buf)[32], int &turn,
                                             int first, int warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool upper = lane >= 16;
  float v = half_sum((upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16));
  if (!WARP) {
    float *s = reinterpret_cast<float *>(buf[turn]);   // [which][warp]
    turn ^= 1;
    if ((lane & 15) == 0) s[(lane & 16) * 2 + warp] = v;
    __syncthreads();
    const float *mine = s + (lane & 16) * 2 + first;
    const int i = lane & 15;
    v = half_sum((i < warps ? mine[i] : 0.f) + (i + 16 < warps ? mine[i + 16] : 0.f));
  }
  const float other = __shfl_xor_sync(0xffffffffu, v, 16);
  return upper ? make_float2(other, v) : make_float2(v, other);
}

template <bool WARP>
__device__ __forceinline__ void group_barrier() {
  if (WARP) __syncwarp();
  else __syncthreads();
}

// Rows of a CTA: `groups` groups of tpr threads take neighbouring rows.
template <typename T, int VEC, int VPT, bool WARP>
__global__ void __launch_bounds__(N_FWD_THREADS, 2)
norm_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
            const T *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
            float *__restrict__ rstd_out, int tpr, int groups) {
  // [stage][chunk][thread], or [stage][group] slots of whole rows
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float buf[2][32];
  using C = Chunk<T, VEC>;
  constexpr bool RING = VEC > 1;
  constexpr int NC = VPT * VEC / C::SPAN, H = C::H;
  const int group = WARP ? threadIdx.x >> 5 : threadIdx.x / tpr;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x - group * tpr;
  const int d = c.d, nthr = blockDim.x, warps = tpr >> 5;
  const float inv_d = 1.f / (float)d;
  int turn = 0, stage = 0;
  const int64_t step = (int64_t)gridDim.x * groups;
  const int64_t first = (int64_t)blockIdx.x * groups;
  auto col_of = [&](int i) { return VEC > 1 ? (tid + i * tpr) * VEC : tid + 2 * i * tpr; };
  const int slot = slot_bytes(d, sizeof(T));
  const T *x_end = x + (c.rows - 1) * c.ldx + d;
  auto slot_of = [&](int st) {
    return reinterpret_cast<uint8_t *>(ring) + (st * groups + group) * slot;
  };
  auto fill = [&](int64_t r, int st) {
    if (r < c.rows) {
      const T *row = x + r * c.ldx;
      if constexpr (RING) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (col_of(i) < d)
            copy16_async(&ring[(st * NC + i) * nthr + threadIdx.x], row + col_of(i));
      } else {
        copy_row(slot_of(st), row, d, x_end, tid, tpr);
      }
    }
    copy_commit();
  };
  for (int st = 0; st < N_FWD_STAGES - 1; ++st) fill(first + group + st * step, st);
  for (int64_t r0 = first; r0 < c.rows; r0 += step) {
    const int64_t r = r0 + group;
    const bool live = r < c.rows;
    float2 v[NC][H], sum = both(0.f), sq = both(0.f);
    // the stage being filled was read in the iteration before: by this thread,
    // or by the group's, which have all reached the barrier since
    if (!RING) {
      copy_wait<N_FWD_STAGES - 2>();
      group_barrier<WARP>();
    }
    fill(r + (N_FWD_STAGES - 1) * step, stage == 0 ? N_FWD_STAGES - 1 : stage - 1);
    if (RING) copy_wait<N_FWD_STAGES - 1>();
    const T *row = nullptr;
    if (!RING && live)
      row = reinterpret_cast<const T *>(slot_of(stage) + head_of(x + r * c.ldx));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (live && col_of(i) < d) {
        if constexpr (RING) C::unpack(ring[(stage * NC + i) * nthr + threadIdx.x], v[i]);
        else C::load(row, col_of(i), tpr, d, v[i]);
#pragma unroll
        for (int h = 0; h < H; ++h) sum = add2(sum, v[i][h]);
      } else {
#pragma unroll
        for (int h = 0; h < H; ++h) v[i][h] = both(0.f);
      }
    }
    stage = stage + 1 == N_FWD_STAGES ? 0 : stage + 1;
    const float mean = group_sum<WARP>(sum.x + sum.y, buf, turn, warps) * inv_d;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (col_of(i) < d) {
#pragma unroll
        for (int h = 0; h < H; ++h) v[i][h] = add2(v[i][h], both(-mean));
        C::mask(col_of(i), tpr, d, v[i]);
#pragma unroll
        for (int h = 0; h < H; ++h) sq = fma2(v[i][h], v[i][h], sq);
      }
    }
    const float var = group_sum<WARP>(sq.x + sq.y, buf, turn, warps) * inv_d;
    const float rstd = rsqrtf(var + c.eps);
    if (!live) continue;
    T *out = y + r * c.ldy;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (col_of(i) < d) {
        // (gamma and beta come from L1: held in registers they would cost
        // resident CTAs)
        float2 g[H], b[H];
        C::load(gamma, col_of(i), tpr, d, g);
#pragma unroll
        for (int h = 0; h < H; ++h) b[h] = both(0.f);
        if (beta) C::load(beta, col_of(i), tpr, d, b);
#pragma unroll
        for (int h = 0; h < H; ++h) v[i][h] = fma2(mul2(v[i][h], both(rstd)), g[h], b[h]);
        C::store(out, col_of(i), tpr, d, v[i]);
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
__global__ void __launch_bounds__(N_BWD_THREADS)
norm_backward_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
                     const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                     const T *__restrict__ dy, T *__restrict__ dx, float *__restrict__ pg,
                     float *__restrict__ pb, int tpr, int groups) {
  // [stage][chunk][x, dy][thread], or [stage][group][x, dy] slots of whole rows
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float2 buf[2][32];
  using C = Chunk<T, VEC>;
  constexpr bool RING = VEC > 1;
  constexpr int STAGES = bwd_stages(VPT);
  constexpr int NC = VPT * VEC / C::SPAN, H = C::H;
  const int group = WARP ? threadIdx.x >> 5 : threadIdx.x / tpr;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x - group * tpr;
  const int d = c.d, nthr = blockDim.x, warps = tpr >> 5, first_warp = group * warps;
  const float inv_d = 1.f / (float)d;
  int turn = 0, stage = 0;
  pdl_launch_dependents();   // (the column sums wait for this grid to end)
  float2 ga[NC][H], ag[NC][H], ab[NC][H];
  auto col_of = [&](int i) { return VEC > 1 ? (tid + i * tpr) * VEC : tid + 2 * i * tpr; };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (col_of(i) < d) C::load(gamma, col_of(i), tpr, d, ga[i]);
#pragma unroll
    for (int h = 0; h < H; ++h) ag[i][h] = ab[i][h] = both(0.f);
  }
  const int64_t step = (int64_t)gridDim.x * groups;
  const int64_t first = (int64_t)blockIdx.x * groups;
  // rows still to come, and where the next copies and the next result go
  int64_t ahead = first + group;
  const T *rx = x + ahead * c.ldx, *ry = dy + ahead * c.lddy;
  T *out = dx + ahead * c.lddx;
  const int64_t sx = step * c.ldx, sy = step * c.lddy, so = step * c.lddx;
  const int slot = slot_bytes(d, sizeof(T));
  const T *x_end = x + (c.rows - 1) * c.ldx + d, *y_end = dy + (c.rows - 1) * c.lddy + d;
  auto slot_of = [&](int st) {
    return reinterpret_cast<uint8_t *>(ring) + (st * groups + group) * 2 * slot;
  };
  auto fill = [&](int st) {
    if (ahead < c.rows) {
      if constexpr (RING) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (col_of(i) < d) {
            uint4 *at = &ring[(st * NC + i) * 2 * nthr + threadIdx.x];
            copy16_async(at, rx + col_of(i));
            copy16_async(at + nthr, ry + col_of(i));
          }
        }
      } else {
        copy_row(slot_of(st), rx, d, x_end, tid, tpr);
        copy_row(slot_of(st) + slot, ry, d, y_end, tid, tpr);
      }
    }
    copy_commit();
    ahead += step;
    rx += sx;
    ry += sy;
  };
  for (int st = 0; st < STAGES - 1; ++st) fill(st);
  float mean = 0.f, rstd = 0.f;
  if (first + group < c.rows) {
    mean = mean_in[first + group];
    rstd = rstd_in[first + group];
  }
  for (int64_t r0 = first; r0 < c.rows; r0 += step) {
    const int64_t r = r0 + group;
    const bool live = r < c.rows;
    float2 xh[NC][H], w[NC][H], s1 = both(0.f), s2 = both(0.f);
    if (!RING) {
      copy_wait<STAGES - 2>();
      group_barrier<WARP>();
    }
    fill(stage == 0 ? STAGES - 1 : stage - 1);
    if (RING) copy_wait<STAGES - 1>();
    const T *row_x = nullptr, *row_y = nullptr;
    if (!RING && live) {
      row_x = reinterpret_cast<const T *>(slot_of(stage) + head_of(x + r * c.ldx));
      row_y = reinterpret_cast<const T *>(slot_of(stage) + slot + head_of(dy + r * c.lddy));
    }
    float next_mean = 0.f, next_rstd = 0.f;
    if (r + step < c.rows) {
      next_mean = mean_in[r + step];
      next_rstd = rstd_in[r + step];
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (live && col_of(i) < d) {
        if constexpr (RING) {
          const uint4 *at = &ring[(stage * NC + i) * 2 * nthr + threadIdx.x];
          C::unpack(at[0], xh[i]);
          C::unpack(at[nthr], w[i]);
        } else {
          C::load(row_x, col_of(i), tpr, d, xh[i]);
          C::load(row_y, col_of(i), tpr, d, w[i]);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          // (an element that is not there has dy = 0)
          xh[i][h] = mul2(add2(xh[i][h], both(-mean)), both(rstd));
          ag[i][h] = fma2(w[i][h], xh[i][h], ag[i][h]);
          ab[i][h] = add2(ab[i][h], w[i][h]);
          w[i][h] = mul2(w[i][h], ga[i][h]);
          s1 = add2(s1, w[i][h]);
          s2 = fma2(w[i][h], xh[i][h], s2);
        }
      }
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    const float2 s = group_sum2<WARP>(s1.x + s1.y, s2.x + s2.y, buf, turn, first_warp, warps);
    const float2 m1 = both(-s.x * inv_d), m2 = both(-s.y * inv_d);
    if (live) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (col_of(i) < d) {
#pragma unroll
          for (int h = 0; h < H; ++h)
            w[i][h] = mul2(fma2(xh[i][h], m2, add2(w[i][h], m1)), both(rstd));
          C::store(out, col_of(i), tpr, d, w[i]);
        }
      }
    }
    out += so;
    mean = next_mean;
    rstd = next_rstd;
  }
  // the groups of the CTA meet in shared memory (the ring's, now read; no copy
  // is in flight: the ones issued past the last row were empty)
  copy_wait<0>();
  float *cols = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *part = which ? pb : pg;
    if (part == nullptr) continue;
    part += (int64_t)blockIdx.x * d;
    const int width = tpr * VPT * VEC;
    float *to = groups == 1 ? part : cols + group * width;
    if (groups > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (col_of(i) < d) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float2 a = which ? ab[i][h] : ag[i][h];
          to[col_of(i) + (VEC > 1 ? 2 * h : 0)] = a.x;
          const int second = col_of(i) + (VEC > 1 ? 2 * h + 1 : tpr);
          if (VEC > 1 || second < d) to[second] = a.y;
        }
      }
    }
    if (groups == 1) continue;
    __syncthreads();
    for (int col = threadIdx.x; col < d; col += nthr) {
      float a = 0.f;
      for (int g = 0; g < groups; ++g) a += cols[g * width + col];
      part[col] = a;
    }
  }
}

// out[which][col] = sum over count partial rows, in a fixed order: warp w of 32
// adds rows w, w + 32, ..., then a butterfly adds the warps' sums.
__global__ void __launch_bounds__(1024)
column_sum_kernel(const float *__restrict__ pg, const float *__restrict__ pb, int count, int d,
                  float *__restrict__ dgamma, float *__restrict__ dbeta, const int *status) {
  __shared__ float s[32][33];
  const float *part = blockIdx.y ? pb : pg;
  float *out = blockIdx.y ? dbeta : dgamma;
  pdl_wait();
  if (out == nullptr || status_failed(status)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (col < d) {
#pragma unroll 8
    for (int r = warp; r < count; r += 32) a += part[(int64_t)r * d + col];
  }
  s[warp][lane] = a;
  __syncthreads();
  a = warp_sum_xor(s[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < d) out[blockIdx.x * 32 + warp] = a;
}

// Rows wider than a CTA holds in registers: one CTA per row, reading it again
// (from L2) for each pass.
template <typename T>
__global__ void __launch_bounds__(512)
norm_wide_kernel(moe_norm_config c, const T *__restrict__ x, const T *__restrict__ gamma,
                 const T *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
                 float *__restrict__ rstd_out) {
  __shared__ float buf[2][32];
  int turn = 0;
  for (int64_t r = blockIdx.x; r < c.rows; r += gridDim.x) {
    const T *xr = x + r * c.ldx;
    float sum = 0.f, sq = 0.f;
    for (int i = threadIdx.x; i < c.d; i += blockDim.x) sum += Elem<T>::load(xr + i);
    const float mean = group_sum<false>(sum, buf, turn, blockDim.x >> 5) / (float)c.d;
    for (int i = threadIdx.x; i < c.d; i += blockDim.x) {
      const float v = Elem<T>::load(xr + i) - mean;
      sq = fmaf(v, v, sq);
    }
    const float rstd =
        1.f / sqrtf(group_sum<false>(sq, buf, turn, blockDim.x >> 5) / (float)c.d + c.eps);
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
    const float2 s = group_sum2<false>(s1, s2, buf, turn, 0, blockDim.x >> 5);
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
// Pieces per thread.  The gradient keeps five values per element (two of the
// row, gamma, two column sums): 16 elements in 128 registers of 512 threads.
// (8 elements in 64 registers of 1024 threads pay the sums over the row twice
// as often: before the ring 177 us against 148 at 16384 x 7168 bf16.)
// The forward with four pieces of 16 bytes in 64 registers: 88 us at 16384 x
// 7168 bf16; with two pieces 98, with one 124, with 96 registers 108.
constexpr int fwd_vpt(int vec) { return vec == 1 ? 16 : 4; }
constexpr int bwd_vpt(int vec) { return 16 / vec; }

// Threads per row for rows of d elements held as vpt pieces of vec per thread
// (0: wider than `most` threads hold).
int threads_of(int d, int vec, int vpt, int most) {
  const int64_t per_warp = (int64_t)32 * vec * vpt;
  const int64_t warps = (d + per_warp - 1) / per_warp;
  return warps * 32 <= most ? (int)warps * 32 : 0;
}

bool by_vectors(const moe_norm_config &c, int vec, bool backward) {
  return c.d % vec == 0 && c.ldx % vec == 0 &&
         (backward ? c.lddy % vec == 0 && c.lddx % vec == 0 : c.ldy % vec == 0);
}

// CTAs that walk the rows, `most` at most.
int grid_of(int64_t rows, int groups, int64_t most) {
  const int64_t want = (rows + groups - 1) / groups;
  return (int)(want < most ? want : most);
}

// How the gradient covers the rows.  Short rows share a CTA of up to 512
// threads, fewer where there are SMs to spare.
struct BwdPlan {
  int vec, tpr;   // threads per row, 0: the wide kernels
  int groups, parts;
};
BwdPlan plan_backward(const moe_norm_config &c) {
  BwdPlan p;
  const int v16 = c.dtype == MOE_F32 ? 4 : 8;
  p.vec = by_vectors(c, v16, true) ? v16 : 1;
  p.tpr = threads_of(c.d, p.vec, bwd_vpt(p.vec), N_BWD_THREADS);
  p.groups = p.tpr == 0 ? 64 : N_BWD_THREADS / p.tpr;
  while (p.tpr && p.groups > 1 && c.rows <= (int64_t)(p.groups / 2) * N_MAX_PARTS) p.groups /= 2;
  p.parts = grid_of(c.rows, p.groups, N_MAX_PARTS);
  return p;
}

template <typename T, int VEC, int VPT, bool WARP>
cudaError_t fwd(const moe_norm_config &c, const T *x, const T *gamma, const T *beta, T *y,
                float *mean, float *rstd, int tpr, cudaStream_t s) {
  auto kernel = norm_kernel<T, VEC, VPT, WARP>;
  const int groups = tpr <= 256 ? 256 / tpr : 1, threads = tpr * groups;
  const size_t smem = VEC > 1 ? (size_t)N_FWD_STAGES * VPT * threads * 16
                              : (size_t)N_FWD_STAGES * groups * slot_bytes(c.d, sizeof(T));
  // CTAs per SM by warps per CTA.  (The ring's size varies with d too where rows are
  // not whole vectors, but 64 registers a thread are the tighter bound for each.)
  static int resident[N_FWD_THREADS / 32 + 1] = {};
  int &ctas = resident[threads / 32];
  if (ctas == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         N_SMEM);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    if (ctas < 1) ctas = 1;
  }
  kernel<<<grid_of(c.rows, groups, (int64_t)num_sms() * ctas), threads, smem, s>>>(
      c, x, gamma, beta, y, mean, rstd, tpr, groups);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t fwd_vec(const moe_norm_config &c, const T *x, const T *gamma, const T *beta, T *y,
                    float *mean, float *rstd, cudaStream_t s) {
  constexpr int VPT = fwd_vpt(VEC);
  const int tpr = threads_of(c.d, VEC, VPT, N_FWD_THREADS);
  if (tpr == 0) {
    norm_wide_kernel<T><<<grid_of(c.rows, 1, (int64_t)num_sms() * 4), 512, 0, s>>>(
        c, x, gamma, beta, y, mean, rstd);
    return cudaGetLastError();
  }
  return tpr == 32 ? fwd<T, VEC, VPT, true>(c, x, gamma, beta, y, mean, rstd, tpr, s)
                   : fwd<T, VEC, VPT, false>(c, x, gamma, beta, y, mean, rstd, tpr, s);
}

template <typename T>
cudaError_t fwd_typed(const moe_norm_config &c, const void *xv, const void *gv, const void *bv,
                      void *yv, float *mean, float *rstd, cudaStream_t s) {
  const T *x = (const T *)xv, *gamma = (const T *)gv, *beta = (const T *)bv;
  T *y = (T *)yv;
  constexpr int V = Vec16<T>::N;
  return by_vectors(c, V, false) ? fwd_vec<T, V>(c, x, gamma, beta, y, mean, rstd, s)
                                 : fwd_vec<T, 1>(c, x, gamma, beta, y, mean, rstd, s);
}

template <typename T, int VEC, bool WARP>
cudaError_t bwd(const moe_norm_config &c, const BwdPlan &p, const T *x, const T *gamma,
                const float *mean, const float *rstd, const T *dy, T *dx, float *pg, float *pb,
                cudaStream_t s) {
  constexpr int VPT = bwd_vpt(VEC);
  auto kernel = norm_backward_kernel<T, VEC, VPT, WARP>;
  const int threads = p.tpr * p.groups;
  const size_t ring = VEC > 1
                          ? (size_t)bwd_stages(VPT) * VPT * 2 * threads * 16
                          : (size_t)bwd_stages(VPT) * p.groups * 2 * slot_bytes(c.d, sizeof(T));
  const size_t cols = p.groups > 1 ? (size_t)threads * VPT * VEC * 4 : 0;
  static bool set = false;
  if (!set) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, N_SMEM);
    if (e != cudaSuccess) return e;
    set = true;
  }
  kernel<<<p.parts, threads, ring > cols ? ring : cols, s>>>(c, x, gamma, mean, rstd, dy, dx, pg,
                                                             pb, p.tpr, p.groups);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd_vec(const moe_norm_config &c, const BwdPlan &p, const T *x, const T *gamma,
                    const float *mean, const float *rstd, const T *dy, T *dx, float *pg, float *pb,
                    cudaStream_t s) {
  return p.tpr == 32 ? bwd<T, VEC, true>(c, p, x, gamma, mean, rstd, dy, dx, pg, pb, s)
                     : bwd<T, VEC, false>(c, p, x, gamma, mean, rstd, dy, dx, pg, pb, s);
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
  cudaError_t e;
  if (p.tpr == 0) {
    norm_backward_wide_kernel<T><<<grid_of(c.rows, 1, (int64_t)num_sms() * 4), 512, 0, s>>>(
        c, x, gamma, mean, rstd, dy, dx);
    if (pg || pb)
      norm_columns_kernel<T><<<dim3((c.d + 31) / 32, p.parts), 256, 0, s>>>(c, x, mean, rstd, dy,
                                                                            pg, pb);
    e = cudaGetLastError();
  } else if (p.vec > 1) {
    e = bwd_vec<T, Vec16<T>::N>(c, p, x, gamma, mean, rstd, dy, dx, pg, pb, s);
  } else {
    e = bwd_vec<T, 1>(c, p, x, gamma, mean, rstd, dy, dx, pg, pb, s);
  }
  if (e == cudaSuccess && !direct && (pg || pb))
    e = launch_column_sum(pg, pb, p.parts, c.d, dgamma, dbeta, nullptr, s);
  return e;
}

}  // namespace

cudaError_t launch_column_sum(const float *pa, const float *pb, int count, int d, float *a,
                              float *b, const int *status, cudaStream_t s) {
  return launch_pdl(column_sum_kernel, dim3((d + 31) / 32, b ? 2 : 1), dim3(1024), 0, s, pa, pb,
                    count, d, a, b, status);
}

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
