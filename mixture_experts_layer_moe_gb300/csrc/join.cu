// The joint of a block with the residual stream, and its gradient:
//   z = post(b),  r = scale x + gate . D(z),  y = pre(r)
// (moe.h has the gradient's formulas).  Both are streams through HBM: the forward
// reads x and b and writes r and y, the gradient reads b, r, dr and dy once and
// writes dx and db.
//
// A row belongs to a group of threads (a warp for short rows, else up to a CTA)
// and stays in a ring in shared memory, where it arrives some rows ahead
// (cp.async; a thread reads its own copies alone where rows are whole vectors).
// The norms' sums are joined over the group, two for an RMS and two or three for a
// layer norm's pair, and each pass over the row between them reads the ring
// again: that leaves registers for the values that pass on (the joined row; in
// the gradient post's input) and for the column sums, which grow in a thread's
// registers as it owns the same columns of every row.  Each CTA writes one partial
// row of these and a second launch adds them in order.  The dropout mask is made
// again in each direction (philox.cuh).
#include <initializer_list>

#include "common.cuh"
#include "fp32x2.cuh"
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

// ------------------------------------------------------- rows held in a ring
constexpr int J_THREADS = 512;
constexpr int J_SMEM = 208 * 1024;   // dynamic shared memory of a CTA at most

// Waits until at most `ahead` of this thread's groups of copies are in flight.
__device__ __forceinline__ void copies_wait(int ahead) {
  if (ahead >= 2) copy_wait<2>();
  else if (ahead == 1) copy_wait<1>();
  else copy_wait<0>();
}

// Where the rows of a ring's tensors lie for a thread.  Vectors: [stage][chunk]
// [tensor][thread], each thread's own; else [stage][group][tensor] slots of whole
// rows.
template <typename T, int VEC, int VPT>
struct Ring {
  using C = Chunk<T, VEC>;
  static constexpr bool OWN = VEC > 1;
  static constexpr int NC = VPT * VEC / C::SPAN;
  uint8_t *base;
  int tid, tpr, group, groups, tensors, d, slot;

  __device__ __forceinline__ int col(int i) const {
    return OWN ? (tid + i * tpr) * VEC : tid + 2 * i * tpr;
  }
  __device__ __forceinline__ uint4 *piece(int stage, int i, int t) const {
    return reinterpret_cast<uint4 *>(base) +
           ((stage * NC + i) * tensors + t) * (int)blockDim.x + threadIdx.x;
  }
  __device__ __forceinline__ uint8_t *row(int stage, int t) const {
    return base + (int64_t)((stage * groups + group) * tensors + t) * slot;
  }
  __device__ __forceinline__ void copy(int stage, int t, const T *src, const T *end) const {
    if constexpr (OWN) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (col(i) < d) copy16_async(piece(stage, i, t), src + col(i));
    } else {
      copy_row(row(stage, t), src, d, end, tid, tpr);
    }
  }
  // chunk i of tensor t, whose row src was copied
  __device__ __forceinline__ void get(int stage, int i, int t, const T *src, float2 *p) const {
    if constexpr (OWN) C::unpack(*piece(stage, i, t), p);
    else C::load(reinterpret_cast<const T *>(row(stage, t) + head_of(src)), col(i), tpr, d, p);
  }
};

__host__ __device__ constexpr int mask_bytes(int d) { return ((d + 7) / 8 + 15) / 16 * 16; }

// The dropout masks of a thread's share of a row.  Vectors: VEC bits per chunk, made
// by the thread; else from a row of bytes in shared memory that the group makes.
template <typename T, int VEC, int VPT>
struct Masks {
  using R = Ring<T, VEC, VPT>;
  uint32_t bits[(R::NC * VEC + 31) / 32];
  const uint8_t *bytes;

  __device__ __forceinline__ void make(const R &ring, const RngState &st, int64_t row,
                                       int threshold, uint8_t *space) {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int w = 0; w < (int)(sizeof(bits) / 4); ++w) bits[w] = 0;
#pragma unroll
      for (int i = 0; i < R::NC; ++i) {
        if (ring.col(i) >= ring.d) continue;
        const uint32_t keep = dropout_keep(st, ring.col(i) >> 3, (uint32_t)row, threshold) >>
                              (VEC == 8 ? 0 : ring.col(i) & 4);
        bits[i * VEC / 32] |= (keep & ((1u << VEC) - 1)) << (i * VEC % 32);
      }
    } else {
      for (int k = ring.tid; k < (ring.d + 7) / 8; k += ring.tpr)
        space[k] = (uint8_t)dropout_keep(st, k, (uint32_t)row, threshold);
      bytes = space;   // (read after the group's next barrier)
    }
  }
  // both elements of pair h of chunk i: kept ones times factor, others 0
  __device__ __forceinline__ float2 apply(const R &ring, int i, int h, float2 v, float factor) const {
    bool x, y;
    if constexpr (VEC > 1) {
      const uint32_t b = bits[i * VEC / 32] >> (i * VEC % 32 + 2 * h);
      x = b & 1;
      y = b & 2;
    } else {
      const int c0 = ring.col(i), c1 = c0 + ring.tpr;
      x = bytes[c0 >> 3] >> (c0 & 7) & 1;
      y = c1 < ring.d && (bytes[c1 >> 3] >> (c1 & 7) & 1);
    }
    return make_float2(x ? v.x * factor : 0.f, y ? v.y * factor : 0.f);
  }
};

// Chunk i of a vector of d parameters, or `other` where there is none.
template <typename T, int VEC, int VPT>
__device__ __forceinline__ void params(const Ring<T, VEC, VPT> &ring, const T *v, int i, float other,
                                       float2 (&p)[Chunk<T, VEC>::H]) {
#pragma unroll
  for (int h = 0; h < Chunk<T, VEC>::H; ++h) p[h] = both(other);
  if (v) Chunk<T, VEC>::load(v, ring.col(i), ring.tpr, ring.d, p);
}

// Rows of a CTA: `groups` groups of tpr threads take neighbouring rows.
template <typename T, int VEC, int VPT, bool WARP, bool DROP>
__global__ void __launch_bounds__(J_THREADS, 2)
join_kernel(const __grid_constant__ Fwd<T> a, int tpr, int groups, int stages) {
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ float buf[2][32];
  using C = Chunk<T, VEC>;
  using R = Ring<T, VEC, VPT>;
  constexpr int NC = R::NC, H = C::H;
  const moe_join_config &c = a.c;
  const int d = c.d, warps = tpr >> 5;
  const int group = WARP ? threadIdx.x >> 5 : threadIdx.x / tpr;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x - group * tpr;
  const R ring{reinterpret_cast<uint8_t *>(dyn), tid, tpr, group, groups, 2, d,
               slot_bytes(d, sizeof(T))};
  // (the masks of rows that are not whole vectors, behind the ring)
  uint8_t *space = reinterpret_cast<uint8_t *>(dyn) +
                   (int64_t)stages * groups * 2 * ring.slot + (int64_t)group * 2 * mask_bytes(d);
  const float inv_d = 1.f / (float)d;
  const RngState st = DROP ? *a.rng : RngState{0, 0};
  int turn = 0, stage = 0, parity = 0;
  const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups;
  const T *x_end = a.x + (c.rows - 1) * c.ldx + d, *b_end = a.b + (c.rows - 1) * c.ldb + d;
  auto fill = [&](int64_t row, int to) {
    if (row < c.rows) {
      ring.copy(to, 0, a.b + row * c.ldb, b_end);
      ring.copy(to, 1, a.x + row * c.ldx, x_end);
    }
    copy_commit();
  };
  auto sum = [&](float2 v) { return group_sum<WARP>(v.x + v.y, buf, turn, warps); };
  for (int i = 0; i < stages - 1; ++i) fill(first + group + i * step, i);
  for (int64_t r0 = first; r0 < c.rows; r0 += step) {
    const int64_t row = r0 + group;
    const bool live = row < c.rows;
    const int64_t ahead = row + (stages - 1) * step;
    const int next = stage == 0 ? stages - 1 : stage - 1;   // (read in the iteration before)
    Masks<T, VEC, VPT> masks;
    if (R::OWN) {
      fill(ahead, next);
      if (DROP) masks.make(ring, st, row, a.threshold, nullptr);
      copies_wait(stages - 1);
    } else {
      if (DROP) masks.make(ring, st, row, a.threshold, space + parity * mask_bytes(d));
      parity ^= 1;
      if (stages == 1) {
        group_barrier<WARP>();
        fill(ahead, next);
        copy_wait<0>();
        group_barrier<WARP>();
      } else {
        copies_wait(stages - 2);
        group_barrier<WARP>();
        fill(ahead, next);
      }
    }
    const T *b_row = a.b + row * c.ldb, *x_row = a.x + row * c.ldx;
    auto there = [&](int i) { return live && ring.col(i) < d; };
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
    if (c.post == MOE_NORM_LAYER) {
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!there(i)) continue;
        float2 v[H];
        ring.get(stage, i, 0, b_row, v);
#pragma unroll
        for (int h = 0; h < H; ++h) s = add2(s, v[h]);
      }
      mean1 = sum(s) * inv_d;
    }
    if (c.post != MOE_NORM_NONE) {
      float2 s = both(0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!there(i)) continue;
        float2 v[H];
        ring.get(stage, i, 0, b_row, v);
#pragma unroll
        for (int h = 0; h < H; ++h) v[h] = add2(v[h], both(-mean1));
        C::mask(ring.col(i), tpr, d, v);
#pragma unroll
        for (int h = 0; h < H; ++h) s = fma2(v[h], v[h], s);
      }
      rstd1 = rsqrtf(sum(s) * inv_d + c.eps);
    }
    // the joined row, and the sum that the next norm takes of it
    float2 v[NC][H], s = both(0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!there(i)) {
#pragma unroll
        for (int h = 0; h < H; ++h) v[i][h] = both(0.f);
        continue;
      }
      float2 z[H], q[H], t[H];
      ring.get(stage, i, 0, b_row, z);
      if (c.post != MOE_NORM_NONE) {
        params(ring, a.post_gamma, i, 1.f, q);
        params(ring, a.post_beta, i, 0.f, t);
#pragma unroll
        for (int h = 0; h < H; ++h)
          z[h] = fma2(mul2(add2(z[h], both(-mean1)), both(rstd1)), q[h], t[h]);
      }
      if (DROP) {
#pragma unroll
        for (int h = 0; h < H; ++h) z[h] = masks.apply(ring, i, h, z[h], a.factor);
      }
      if (a.gate) {
        params(ring, a.gate, i, 1.f, q);
#pragma unroll
        for (int h = 0; h < H; ++h) z[h] = mul2(z[h], q[h]);
      }
      ring.get(stage, i, 1, x_row, q);
#pragma unroll
      for (int h = 0; h < H; ++h) v[i][h] = fma2(both(c.scale), q[h], z[h]);
      C::mask(ring.col(i), tpr, d, v[i]);
#pragma unroll
      for (int h = 0; h < H; ++h)
        s = c.pre == MOE_NORM_LAYER ? add2(s, v[i][h]) : fma2(v[i][h], v[i][h], s);
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
    if (c.pre == MOE_NORM_LAYER) {
      mean2 = sum(s) * inv_d;
      s = both(0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!there(i)) continue;
        float2 t[H];
#pragma unroll
        for (int h = 0; h < H; ++h) t[h] = add2(v[i][h], both(-mean2));
        C::mask(ring.col(i), tpr, d, t);
#pragma unroll
        for (int h = 0; h < H; ++h) s = fma2(t[h], t[h], s);
      }
    }
    if (c.pre != MOE_NORM_NONE) rstd2 = rsqrtf(sum(s) * inv_d + c.eps);
    if (!live) continue;
    T *r_row = a.r + row * c.ldr, *y_row = a.y + row * c.ldy;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (ring.col(i) >= d) continue;
      C::store(r_row, ring.col(i), tpr, d, v[i]);
      if (c.pre == MOE_NORM_NONE) continue;
      float2 q[H], t[H];
      params(ring, a.pre_gamma, i, 1.f, q);
      params(ring, a.pre_beta, i, 0.f, t);
#pragma unroll
      for (int h = 0; h < H; ++h)
        t[h] = fma2(mul2(add2(v[i][h], both(-mean2)), both(rstd2)), q[h], t[h]);
      C::store(y_row, ring.col(i), tpr, d, t);
    }
    if (a.stats && tid == 0) {
      a.stats[row] = mean1;
      a.stats[c.rows + row] = rstd1;
      a.stats[2 * c.rows + row] = mean2;
      a.stats[3 * c.rows + row] = rstd2;
    }
  }
}

// BETAS: the sums of u and dy are wanted too.
template <typename T, int VEC, int VPT, bool WARP, bool DROP, bool BETAS>
__global__ void __launch_bounds__(J_THREADS, 1)
join_backward_kernel(const __grid_constant__ Bwd<T> a, int tpr, int groups, int stages, int tensors) {
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ float2 buf[2][32];
  using C = Chunk<T, VEC>;
  using R = Ring<T, VEC, VPT>;
  constexpr int NC = R::NC, H = C::H;
  const moe_join_config &c = a.c;
  const int d = c.d, warps = tpr >> 5;
  const int group = WARP ? threadIdx.x >> 5 : threadIdx.x / tpr;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x - group * tpr;
  const int first_warp = group * warps;
  const R ring{reinterpret_cast<uint8_t *>(dyn), tid, tpr, group, groups, tensors, d,
               slot_bytes(d, sizeof(T))};
  uint8_t *space = reinterpret_cast<uint8_t *>(dyn) +
                   (int64_t)stages * groups * tensors * ring.slot + (int64_t)group * 2 * mask_bytes(d);
  // where the tensors lie in a stage of the ring
  const bool has_dr = a.dr != nullptr, has_dy = a.dy != nullptr, has_b = a.has_b;
  const int at_dr = 0, at_b = has_dr, at_dy = at_b + has_b, at_r = at_dy + 1;
  const float inv_d = 1.f / (float)d;
  const RngState st = DROP ? *a.rng : RngState{0, 0};
  int turn = 0, stage = 0, parity = 0;
  pdl_launch_dependents();   // (the column sums wait for this grid to end)
  const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups;
  const int64_t last = c.rows - 1;
  auto fill = [&](int64_t row, int to) {
    if (row < c.rows) {
      if (has_dy) {
        ring.copy(to, at_dy, a.dy + row * c.lddy, a.dy + last * c.lddy + d);
        ring.copy(to, at_r, a.r + row * c.ldr, a.r + last * c.ldr + d);
      }
      if (has_dr) ring.copy(to, at_dr, a.dr + row * c.lddr, a.dr + last * c.lddr + d);
      if (has_b) ring.copy(to, at_b, a.b + row * c.ldb, a.b + last * c.ldb + d);
    }
    copy_commit();
  };
  // sums of u bh and dy rh, and of u and dy
  float2 sum_a[NC][H], sum_c[NC][H], sum_b[BETAS ? NC : 1][H], sum_e[BETAS ? NC : 1][H];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      sum_a[i][h] = sum_c[i][h] = both(0.f);
      if (BETAS) sum_b[i][h] = sum_e[i][h] = both(0.f);
    }
  }
  for (int i = 0; i < stages - 1; ++i) fill(first + group + i * step, i);
  for (int64_t r0 = first; r0 < c.rows; r0 += step) {
    const int64_t row = r0 + group;
    const bool live = row < c.rows;
    const int64_t ahead = row + (stages - 1) * step;
    const int next = stage == 0 ? stages - 1 : stage - 1;
    Masks<T, VEC, VPT> masks;
    float4 stat = make_float4(0.f, 1.f, 0.f, 1.f);
    if (live) stat = stats_of(a, row);
    if (R::OWN) {
      fill(ahead, next);
      if (DROP) masks.make(ring, st, row, a.threshold, nullptr);
      copies_wait(stages - 1);
    } else {
      if (DROP) masks.make(ring, st, row, a.threshold, space + parity * mask_bytes(d));
      parity ^= 1;
      if (stages == 1) {
        group_barrier<WARP>();
        fill(ahead, next);
        copy_wait<0>();
        group_barrier<WARP>();
      } else {
        copies_wait(stages - 2);
        group_barrier<WARP>();
        fill(ahead, next);
      }
    }
    const T *b_row = a.b + row * c.ldb, *dr_row = a.dr + row * c.lddr;
    const T *dy_row = a.dy + row * c.lddy, *r_row = a.r + row * c.ldr;
    auto there = [&](int i) { return live && ring.col(i) < d; };
    // dy and rh of chunk i
    auto pre = [&](int i, float2 (&dy)[H], float2 (&rh)[H]) {
      ring.get(stage, i, at_dy, dy_row, dy);
      ring.get(stage, i, at_r, r_row, rh);
#pragma unroll
      for (int h = 0; h < H; ++h) rh[h] = mul2(add2(rh[h], both(-stat.z)), both(stat.w));
    };
    auto post = [&](int i, float2 (&bh)[H]) {
      ring.get(stage, i, at_b, b_row, bh);
      if (c.post != MOE_NORM_NONE) {
#pragma unroll
        for (int h = 0; h < H; ++h) bh[h] = mul2(add2(bh[h], both(-stat.x)), both(stat.y));
      }
    };
    float2 m = both(0.f);
    if (has_dy) {
      float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!there(i)) continue;
        float2 dy[H], rh[H], q[H];
        pre(i, dy, rh);
        params(ring, a.pre_gamma, i, 1.f, q);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          // (an element that is not there has dy = 0)
          sum_c[i][h] = fma2(dy[h], rh[h], sum_c[i][h]);
          if (BETAS) sum_e[i][h] = add2(sum_e[i][h], dy[h]);
          const float2 w = mul2(dy[h], q[h]);
          s1 = add2(s1, w);
          s2 = fma2(w, rh[h], s2);
        }
      }
      m = group_sum2<WARP>(s1.x + s1.y, s2.x + s2.y, buf, turn, first_warp, warps);
      m = make_float2(c.pre == MOE_NORM_LAYER ? -m.x * inv_d : 0.f, -m.y * inv_d);
    }
    float2 w[NC][H], s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!there(i)) {
#pragma unroll
        for (int h = 0; h < H; ++h) w[i][h] = both(0.f);
        continue;
      }
      float2 g[H], q[H], t[H];
#pragma unroll
      for (int h = 0; h < H; ++h) g[h] = both(0.f);
      if (has_dr) ring.get(stage, i, at_dr, dr_row, g);
      if (has_dy) {
        float2 dy[H], rh[H];
        pre(i, dy, rh);
        params(ring, a.pre_gamma, i, 1.f, q);
#pragma unroll
        for (int h = 0; h < H; ++h)
          g[h] = fma2(both(stat.w), fma2(rh[h], both(m.y), fma2(dy[h], q[h], both(m.x))), g[h]);
        C::mask(ring.col(i), tpr, d, g);
      }
      if (a.dx) {
#pragma unroll
        for (int h = 0; h < H; ++h) t[h] = mul2(both(c.scale), g[h]);
        C::store(a.dx + row * c.lddx, ring.col(i), tpr, d, t);
      }
      if (DROP) {
#pragma unroll
        for (int h = 0; h < H; ++h) g[h] = masks.apply(ring, i, h, g[h], a.factor);
      }
      if (has_b) post(i, t);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (has_b) sum_a[i][h] = fma2(g[h], t[h], sum_a[i][h]);
        if (BETAS) sum_b[i][h] = add2(sum_b[i][h], g[h]);
      }
      if (a.gate) {
        params(ring, a.gate, i, 1.f, q);
#pragma unroll
        for (int h = 0; h < H; ++h) g[h] = mul2(g[h], q[h]);
      }
      if (c.post != MOE_NORM_NONE) {
        params(ring, a.post_gamma, i, 1.f, q);
#pragma unroll
        for (int h = 0; h < H; ++h) {
          g[h] = mul2(g[h], q[h]);
          s1 = add2(s1, g[h]);
          s2 = fma2(g[h], t[h], s2);
        }
      } else if (a.db) {
        C::store(a.db + row * c.lddb, ring.col(i), tpr, d, g);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) w[i][h] = g[h];
    }
    if (c.post != MOE_NORM_NONE && a.db) {
      float2 q = group_sum2<WARP>(s1.x + s1.y, s2.x + s2.y, buf, turn, first_warp, warps);
      q = make_float2(c.post == MOE_NORM_LAYER ? -q.x * inv_d : 0.f, -q.y * inv_d);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!there(i)) continue;
        float2 t[H];
        post(i, t);
#pragma unroll
        for (int h = 0; h < H; ++h)
          t[h] = mul2(both(stat.y), fma2(t[h], both(q.y), add2(w[i][h], both(q.x))));
        C::store(a.db + row * c.lddb, ring.col(i), tpr, d, t);
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  // the groups of the CTA meet in shared memory (the ring's, now read; no copy
  // is in flight: the ones issued past the last row were empty)
  copy_wait<0>();
  float *cols = reinterpret_cast<float *>(dyn);
  const int width = tpr * VPT * VEC;
#pragma unroll
  for (int which = 0; which < J_SUMS; ++which) {
    if (!(a.sums >> which & 1) || (!BETAS && (which & 1))) continue;
    float *part = a.parts + ((int64_t)blockIdx.x * J_SUMS + which) * d;
    float *to = groups == 1 ? part : cols + group * width;
    if (groups > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (ring.col(i) >= d) continue;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int k = BETAS ? i : 0;
        const float2 v = which == 0 ? sum_a[i][h] : which == 1 ? sum_b[k][h]
                         : which == 2 ? sum_c[i][h] : sum_e[k][h];
        to[ring.col(i) + (VEC > 1 ? 2 * h : 0)] = v.x;
        const int second = ring.col(i) + (VEC > 1 ? 2 * h + 1 : tpr);
        if (VEC > 1 || second < d) to[second] = v.y;
      }
    }
    if (groups == 1) continue;
    __syncthreads();
    for (int col = threadIdx.x; col < d; col += blockDim.x) {
      float t = 0.f;
      for (int g = 0; g < groups; ++g) t += cols[g * width + col];
      part[col] = t;
    }
  }
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

int64_t grid_of(int64_t rows, int groups, int64_t most) {
  const int64_t want = (rows + groups - 1) / groups;
  return want < most ? want : most;
}

// Threads per row for rows of d elements, `each` per thread (0: wider than a CTA
// holds).
int threads_of(int d, int each) {
  const int64_t per_warp = (int64_t)32 * each, warps = (d + per_warp - 1) / per_warp;
  return warps * 32 <= J_THREADS ? (int)warps * 32 : 0;
}

// Bytes of a stage of the ring, and of the masks behind it.
template <typename T, int VEC, int VPT>
size_t stage_bytes(int d, int threads, int groups, int tensors) {
  return VEC > 1 ? (size_t)VPT * 16 * threads * tensors
                 : (size_t)groups * tensors * slot_bytes(d, sizeof(T));
}
template <int VEC>
size_t masks_bytes(int d, int groups, bool drop) {
  return VEC == 1 && drop ? (size_t)groups * 2 * mask_bytes(d) : 0;
}

template <typename T, int VEC, int VPT, bool WARP, bool DROP>
cudaError_t run_forward(const Fwd<T> &a, int tpr, cudaStream_t s) {
  auto kernel = join_kernel<T, VEC, VPT, WARP, DROP>;
  const int groups = tpr <= 256 ? 256 / tpr : 1, threads = tpr * groups;
  const size_t stage = stage_bytes<T, VEC, VPT>(a.c.d, threads, groups, 2);
  const size_t masks = masks_bytes<VEC>(a.c.d, groups, DROP);
  int stages = 3;
  while (stages > 1 && stages * stage + masks > J_SMEM) --stages;
  const size_t smem = stages * stage + masks;
  // CTAs per SM by warps per CTA and 4 KB of shared memory
  static int8_t resident[J_THREADS / 32 + 1][J_SMEM / 4096 + 2] = {};
  int8_t &ctas = resident[threads / 32][smem / 4096];
  if (ctas == 0) {
    int n = 0;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, J_SMEM);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    ctas = (int8_t)(n < 1 ? 1 : n);
  }
  kernel<<<(unsigned)grid_of(a.c.rows, groups, (int64_t)num_sms() * ctas), threads, smem, s>>>(
      a, tpr, groups, stages);
  return cudaGetLastError();
}

template <typename T, int VEC, int VPT>
cudaError_t forward_vec(const Fwd<T> &a, int tpr, cudaStream_t s) {
  if (a.threshold)
    return tpr == 32 ? run_forward<T, VEC, VPT, true, true>(a, tpr, s)
                     : run_forward<T, VEC, VPT, false, true>(a, tpr, s);
  return tpr == 32 ? run_forward<T, VEC, VPT, true, false>(a, tpr, s)
                   : run_forward<T, VEC, VPT, false, false>(a, tpr, s);
}

// Partial rows of the column sums, at most one CTA per SM; short rows share a CTA
// of up to 512 threads, fewer where there are SMs to spare.
template <typename T, int VEC, int VPT, bool WARP, bool DROP, bool BETAS>
cudaError_t run_backward(const Bwd<T> &a, int tpr, int &parts, cudaStream_t s) {
  auto kernel = join_backward_kernel<T, VEC, VPT, WARP, DROP, BETAS>;
  int groups = J_THREADS / tpr;
  while (groups > 1 && a.c.rows <= (int64_t)(groups / 2) * J_PARTS) groups /= 2;
  const int threads = tpr * groups, tensors = (a.dr ? 1 : 0) + (a.has_b ? 1 : 0) + (a.dy ? 2 : 0);
  const size_t stage = stage_bytes<T, VEC, VPT>(a.c.d, threads, groups, tensors);
  const size_t masks = masks_bytes<VEC>(a.c.d, groups, DROP);
  int stages = 3;
  while (stages > 1 && stages * stage + masks > J_SMEM) --stages;
  const size_t ring = stages * stage + masks;
  const size_t cols = groups > 1 ? (size_t)threads * VPT * VEC * 4 : 0;
  static bool set = false;
  if (!set) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, J_SMEM);
    if (e != cudaSuccess) return e;
    set = true;
  }
  parts = (int)grid_of(a.c.rows, groups, J_PARTS);
  kernel<<<parts, threads, ring > cols ? ring : cols, s>>>(a, tpr, groups, stages, tensors);
  return cudaGetLastError();
}

template <typename T, int VEC, int VPT>
cudaError_t backward_vec(const Bwd<T> &a, int tpr, int &parts, cudaStream_t s) {
  const bool betas = a.sums & 10;
  auto pick = [&](auto run_warp, auto run_cta) {
    return tpr == 32 ? run_warp(a, tpr, parts, s) : run_cta(a, tpr, parts, s);
  };
  if (a.threshold)
    return betas ? pick(run_backward<T, VEC, VPT, true, true, true>,
                        run_backward<T, VEC, VPT, false, true, true>)
                 : pick(run_backward<T, VEC, VPT, true, true, false>,
                        run_backward<T, VEC, VPT, false, true, false>);
  return betas ? pick(run_backward<T, VEC, VPT, true, false, true>,
                      run_backward<T, VEC, VPT, false, false, true>)
               : pick(run_backward<T, VEC, VPT, true, false, false>,
                      run_backward<T, VEC, VPT, false, false, false>);
}

// Whether rows this far apart start on a vector.
template <typename T>
bool whole_vectors(const moe_join_config &c, std::initializer_list<int64_t> lds) {
  if (c.d % 8 != 0) return false;
  for (int64_t ld : lds)
    if (c.rows > 1 && ld % Vec16<T>::N != 0) return false;
  return true;
}

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
  constexpr int V = Vec16<T>::N;
  const bool vectors = whole_vectors<T>(c, {c.ldx, c.ldb, c.ldr, c.ldy});
  const int tpr = threads_of(c.d, vectors ? 4 * V : 16);
  if (tpr) return vectors ? forward_vec<T, V, 4>(a, tpr, s) : forward_vec<T, 1, 16>(a, tpr, s);
  join_wide_kernel<T><<<(unsigned)grid_of(c.rows, 1, (int64_t)num_sms() * 4), J_WIDE, 0, s>>>(a);
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
  a.parts = (float *)scratch;
  constexpr int V = Vec16<T>::N;
  const bool vectors = whole_vectors<T>(c, {c.ldb, c.ldr, c.lddr, c.lddy, c.lddx, c.lddb});
  const int tpr = threads_of(c.d, 16);
  int parts = 0;
  cudaError_t e;
  if (tpr) {
    e = vectors ? backward_vec<T, V, 16 / V>(a, tpr, parts, s)
                : backward_vec<T, 1, 16>(a, tpr, parts, s);
  } else {
    parts = (int)grid_of(c.rows, 8, 64);
    a.means = (float2 *)((char *)scratch + (size_t)J_PARTS * J_SUMS * c.d * 4);
    join_backward_wide_kernel<T>
        <<<(unsigned)grid_of(c.rows, 1, (int64_t)num_sms() * 4), J_WIDE, 0, s>>>(a);
    if (a.sums) join_columns_kernel<T><<<dim3((c.d + 31) / 32, parts), 256, 0, s>>>(a);
    e = cudaGetLastError();
  }
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
