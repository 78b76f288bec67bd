// The block joint's gradient (join.cu has the formulas and the design).
#include "join_common.cuh"

namespace moe {
namespace {

using namespace join;

constexpr int J_PARTS = 152;   // partial rows of the column sums, at most
constexpr int J_SUMS = 4;      // sum u bh, sum u, sum dy rh, sum dy

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


// The statistics of a row as the forward left them: the post norm's mean and 1 /
// deviation, then the pre norm's (MEANS: the means are read).
template <typename T, bool MEANS = true>
__device__ __forceinline__ float4 stats_of(const Bwd<T> &a, int64_t row) {
  float4 v = make_float4(0.f, 1.f, 0.f, 1.f);
  if (a.c.post != MOE_NORM_NONE) {
    if (MEANS) v.x = a.stats[row];
    v.y = a.stats[a.c.rows + row];
  }
  if (a.dy) {
    if (MEANS) v.z = a.stats[2 * a.c.rows + row];
    v.w = a.stats[3 * a.c.rows + row];
  }
  return v;
}

// A column sum's partial row of this CTA: put(to) writes a group's sums to to[column];
// the groups meet in shared memory (the ring's, which is read by then).
template <typename T, typename Put>
__device__ __forceinline__ void store_columns(const Bwd<T> &a, float *cols, int width, int group,
                                              int groups, int which, Put &&put) {
  float *part = a.parts + ((int64_t)blockIdx.x * J_SUMS + which) * a.c.d;
  if (groups == 1) {
    put(part);
    return;
  }
  __syncthreads();
  put(cols + group * width);
  __syncthreads();
  for (int col = threadIdx.x; col < a.c.d; col += blockDim.x) {
    float t = 0.f;
    for (int g = 0; g < groups; ++g) t += cols[g * width + col];
    part[col] = t;
  }
}

// Rows of whole vectors, as the forward's kernel takes them.  With rc = r - mean2, bc = b
// - mean1 (the rows themselves without a layer norm, which CENTRED says there is):
//   g = dr + rstd2 dy gamma2 + c2 rc + e2,   c2 = -rstd2^2 mean(w rh),  e2 = -rstd2 mean(w),
//   h = D(g) rstd1 gate gamma1,   db = h + c1 bc + e1  likewise,
// so that neither rh nor bh is formed for itself.
template <typename T, int NB, bool WARP, bool DROP, bool CENTRED>
__global__ void __launch_bounds__(512, 1)
join_backward_vec_kernel(const __grid_constant__ Bwd<T> a, int tpr, int groups, int stages) {
  extern __shared__ __align__(16) uint4 dyn[];   // [stage][block][dr, dy, r, b][vector][thread]
  __shared__ float2 buf[2][32];
  using V = Vec8<T>;
  constexpr int PIECE = V8_PIECE, STAGE = NB * 4 * V::Q * PIECE;
  enum { DR, DY, RR, BB };
  const moe_join_config &c = a.c;
  const int d = c.d, warps = tpr >> 5, warp = threadIdx.x >> 5;
  const int group = WARP ? warp : warp / warps, tid = threadIdx.x - group * tpr;
  const int first_warp = group * warps;
  const bool has_dr = a.dr != nullptr, has_dy = a.dy != nullptr, has_b = a.has_b;
  const bool norm1 = c.post != MOE_NORM_NONE;
  const bool layer1 = CENTRED && c.post == MOE_NORM_LAYER, layer2 = CENTRED && c.pre == MOE_NORM_LAYER;
  const float inv_d = 1.f / (float)d;
  const RngState st = load_state(DROP ? a.rng : nullptr);
  const uint32_t cut = (uint32_t)a.threshold << 16;
  int turn = 0;
  pdl_launch_dependents();   // (the column sums wait for this grid to end)
  const int apart = tpr * 8 * (int)sizeof(T);
  bool on[NB];
  // what D's kept elements and dy are multiplied by; the column sums of u bh, dy rh, u
  // and dy, those of u without dropout's factor
  Block8 p1[NB], p2[NB], sum_a[NB], sum_c[NB], sum_b[CENTRED ? NB : 1], sum_e[CENTRED ? NB : 1];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int col = (tid + n * tpr) * 8;
    on[n] = col < d;
    p1[n] = p2[n] = sum_a[n] = sum_c[n] = fill8(0.f);
    if (CENTRED) sum_b[n] = sum_e[n] = fill8(0.f);
    if (!on[n]) continue;
    p1[n] = V::param(a.gate, col, 1.f);
    p2[n] = V::param(a.pre_gamma, col, 1.f);
    const Block8 g = V::param(a.post_gamma, col, 1.f);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      p1[n].v[h] = mul2(p1[n].v[h], g.v[h]);
      if (DROP) p1[n].v[h] = mul2(p1[n].v[h], both(a.factor));
    }
  }
  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + group, ahead = row;
  uint8_t *const mine = reinterpret_cast<uint8_t *>(dyn) + threadIdx.x * 16;
  uint8_t *const ring_end = mine + stages * STAGE;
  auto bytes = [](int64_t elements) { return elements * (int64_t)sizeof(T); };
  auto start = [&](const T *p, int64_t ld) {
    return reinterpret_cast<const char *>(p + row * ld + tid * 8);
  };
  const char *dr_ahead = start(a.dr, c.lddr), *dy_ahead = start(a.dy, c.lddy);
  const char *r_ahead = start(a.r, c.ldr), *b_ahead = start(a.b, c.ldb);
  char *dx_out = const_cast<char *>(start(a.dx, c.lddx));
  char *db_out = const_cast<char *>(start(a.db, c.lddb));
  auto fill = [&](uint8_t *to) {
    if (ahead < c.rows) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!on[n]) continue;
        if (has_dy) {
          V::template copy<PIECE>(to, n * 4 + DY, dy_ahead + n * apart);
          V::template copy<PIECE>(to, n * 4 + RR, r_ahead + n * apart);
        }
        if (has_dr) V::template copy<PIECE>(to, n * 4 + DR, dr_ahead + n * apart);
        if (has_b) V::template copy<PIECE>(to, n * 4 + BB, b_ahead + n * apart);
      }
    }
    copy_commit();
    ahead += step;
    dr_ahead += bytes(step * c.lddr);
    dy_ahead += bytes(step * c.lddy);
    r_ahead += bytes(step * c.ldr);
    b_ahead += bytes(step * c.ldb);
  };
  for (int i = 0; i < stages - 1; ++i) fill(mine + i * STAGE);
  uint8_t *now = mine, *next = mine + (stages - 1) * STAGE;
  float4 next_stat = make_float4(0.f, 1.f, 0.f, 1.f);
  if (row < c.rows) next_stat = stats_of<T, CENTRED>(a, row);
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < c.rows; r0 += step) {
    const bool live = row < c.rows;
    // (the stage being filled was read by this thread in the iteration before)
    fill(next);
    const float4 stat = next_stat;
    if (row + step < c.rows) next_stat = stats_of<T, CENTRED>(a, row + step);
    copies_wait(stages - 1);
    auto get = [&](int n, int t) { return V::template ring<PIECE>(now, n * 4 + t); };
    auto centred = [&](int n, int t, float mean) {
      Block8 b = get(n, t);
      if (CENTRED) {
#pragma unroll
        for (int h = 0; h < 4; ++h) b.v[h] = add2(b.v[h], both(-mean));
      }
      return b;
    };
    float c2 = 0.f, e2 = 0.f;
    if (has_dy) {
      float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!live || !on[n]) continue;
        const Block8 dy = get(n, DY), rc = centred(n, RR, stat.z);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float2 w = mul2(dy.v[h], p2[n].v[h]);
          if (CENTRED) s1 = add2(s1, w);
          s2 = fma2(w, rc.v[h], s2);
        }
      }
      if (CENTRED) {
        const float2 t = group_sum2<WARP>(s1.x + s1.y, s2.x + s2.y, buf, turn, first_warp, warps);
        e2 = layer2 ? -stat.w * t.x * inv_d : 0.f;
        c2 = -stat.w * stat.w * stat.w * t.y * inv_d;
      } else {
        const float t = group_sum<WARP>(s2.x + s2.y, reinterpret_cast<float (*)[32]>(buf), turn, warps);
        c2 = -stat.w * stat.w * stat.w * t * inv_d;
      }
    }
    Block8 w[NB];
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      w[n] = fill8(0.f);
      if (!live || !on[n]) continue;
      Block8 g = has_dr ? get(n, DR) : fill8(0.f);
      if (has_dy) {
        const Block8 rc = centred(n, RR, stat.z);
        Block8 dy = get(n, DY);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (CENTRED) {
            sum_e[n].v[h] = add2(sum_e[n].v[h], dy.v[h]);
            g.v[h] = add2(g.v[h], both(e2));
          }
          dy.v[h] = mul2(dy.v[h], both(stat.w));
          sum_c[n].v[h] = fma2(dy.v[h], rc.v[h], sum_c[n].v[h]);
          g.v[h] = fma2(dy.v[h], p2[n].v[h], fma2(rc.v[h], both(c2), g.v[h]));
        }
      }
      if (a.dx) {
        Block8 t;
#pragma unroll
        for (int h = 0; h < 4; ++h) t.v[h] = mul2(both(c.scale), g.v[h]);
        V::store(dx_out + n * apart, t);
      }
      if (DROP) drop8(g, dropout_bits(st, tid + n * tpr, (uint32_t)row), cut);
      if (CENTRED) {
#pragma unroll
        for (int h = 0; h < 4; ++h) sum_b[n].v[h] = add2(sum_b[n].v[h], g.v[h]);
      }
      if (norm1) {
#pragma unroll
        for (int h = 0; h < 4; ++h) g.v[h] = mul2(g.v[h], both(stat.y));
      }
      if (has_b) {
        const Block8 bc = centred(n, BB, stat.x);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          sum_a[n].v[h] = fma2(g.v[h], bc.v[h], sum_a[n].v[h]);
          w[n].v[h] = mul2(g.v[h], p1[n].v[h]);
          if (CENTRED) s1 = add2(s1, w[n].v[h]);
          s2 = fma2(w[n].v[h], bc.v[h], s2);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) w[n].v[h] = mul2(g.v[h], p1[n].v[h]);
      }
    }
    if (a.db) {
      // (w is rstd1 times the gradient of the normed row)
      float c1 = 0.f, e1 = 0.f;
      if (norm1 && CENTRED) {
        const float2 t = group_sum2<WARP>(s1.x + s1.y, s2.x + s2.y, buf, turn, first_warp, warps);
        e1 = layer1 ? -t.x * inv_d : 0.f;
        c1 = -stat.y * stat.y * t.y * inv_d;
      } else if (norm1) {
        const float t = group_sum<WARP>(s2.x + s2.y, reinterpret_cast<float (*)[32]>(buf), turn, warps);
        c1 = -stat.y * stat.y * t * inv_d;
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!live || !on[n]) continue;
        if (norm1) {
          const Block8 bc = centred(n, BB, stat.x);
#pragma unroll
          for (int h = 0; h < 4; ++h)
            w[n].v[h] = fma2(bc.v[h], both(c1), CENTRED ? add2(w[n].v[h], both(e1)) : w[n].v[h]);
        }
        V::store(db_out + n * apart, w[n]);
      }
    }
    next = now;
    now = now + STAGE == ring_end ? mine : now + STAGE;
    row += step;
    dx_out += bytes(step * c.lddx);
    db_out += bytes(step * c.lddb);
  }
  copy_wait<0>();   // (none is in flight: the ones past the last row were empty)
#pragma unroll
  for (int which = 0; which < J_SUMS; ++which) {
    if (!(a.sums >> which & 1) || (!CENTRED && (which & 1))) continue;
    const float factor = DROP && which < 2 ? a.factor : 1.f;
    store_columns(a, reinterpret_cast<float *>(dyn), tpr * 8 * NB, group, groups, which,
                  [&](float *to) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!on[n]) continue;
        const int e = CENTRED ? n : 0;
        const Block8 &s = which == 0 ? sum_a[n] : which == 1 ? sum_b[e] : which == 2 ? sum_c[n] : sum_e[e];
#pragma unroll
        for (int h = 0; h < 4; h += 2)
          *reinterpret_cast<float4 *>(to + (tid + n * tpr) * 8 + 2 * h) =
              make_float4(s.v[h].x * factor, s.v[h].y * factor, s.v[h + 1].x * factor,
                          s.v[h + 1].y * factor);
      }
    });
  }
}

// Rows that are not whole vectors.
template <typename T, bool WARP>
__global__ void __launch_bounds__(J_THREADS, 1)
join_backward_odd_kernel(const __grid_constant__ Bwd<T> a, int tpr, int groups, int stages, int tensors) {
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ float2 buf[2][32];
  using C = Chunk<T, 1>;
  using R = Ring<T>;
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
  const bool dropping = a.threshold != 0;
  const RngState st = load_state(dropping ? a.rng : nullptr);
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
  float2 sum_a[NC][H], sum_c[NC][H], sum_b[NC][H], sum_e[NC][H];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      sum_a[i][h] = sum_b[i][h] = sum_c[i][h] = sum_e[i][h] = both(0.f);
    }
  }
  for (int i = 0; i < stages - 1; ++i) fill(first + group + i * step, i);
  for (int64_t r0 = first; r0 < c.rows; r0 += step) {
    const int64_t row = r0 + group;
    const bool live = row < c.rows;
    const int64_t ahead = row + (stages - 1) * step;
    const int next = stage == 0 ? stages - 1 : stage - 1;
    float4 stat = make_float4(0.f, 1.f, 0.f, 1.f);
    if (live) stat = stats_of(a, row);
    uint8_t *masks = space + parity * mask_bytes(d);
    if (dropping) make_masks(ring, st, (uint32_t)row, a.threshold, masks);
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
          sum_e[i][h] = add2(sum_e[i][h], dy[h]);
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
          g[h] = fma2(both(stat.w),
                      fma2(rh[h], both(m.y), fma2(dy[h], q[h], both(m.x))),
                      g[h]);
        C::mask(ring.col(i), tpr, d, g);
      }
      if (a.dx) {
#pragma unroll
        for (int h = 0; h < H; ++h) t[h] = mul2(both(c.scale), g[h]);
        C::store(a.dx + row * c.lddx, ring.col(i), tpr, d, t);
      }
      if (dropping) g[0] = drop_pair(ring, masks, i, g[0], a.factor);
      if (has_b) post(i, t);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        if (has_b) sum_a[i][h] = fma2(g[h], t[h], sum_a[i][h]);
        sum_b[i][h] = add2(sum_b[i][h], g[h]);
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
          t[h] = mul2(both(stat.y),
                      fma2(t[h], both(q.y), add2(w[i][h], both(q.x))));
        C::store(a.db + row * c.lddb, ring.col(i), tpr, d, t);
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
  }
  copy_wait<0>();   // (none is in flight: the ones past the last row were empty)
  float *cols = reinterpret_cast<float *>(dyn);
  const int width = tpr * 16;
#pragma unroll
  for (int which = 0; which < J_SUMS; ++which) {
    if (!(a.sums >> which & 1)) continue;
    store_columns(a, cols, width, group, groups, which, [&](float *to) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (ring.col(i) >= d) continue;
        const float2 v = which == 0 ? sum_a[i][0] : which == 1 ? sum_b[i][0]
                         : which == 2 ? sum_c[i][0] : sum_e[i][0];
        to[ring.col(i)] = v.x;
        if (ring.col(i) + tpr < d) to[ring.col(i) + tpr] = v.y;
      }
    });
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
  const RngState rng = load_state(a.threshold ? a.rng : nullptr);
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
  const RngState rng = load_state(a.threshold ? a.rng : nullptr);
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

// Groups of tpr threads in a CTA of up to 512 threads, fewer where there are SMs to
// spare (one CTA per SM leaves a partial row of each column sum), and the stages
// of a ring whose stage takes `fixed` bytes and `each` per group.  The column sums
// (`columns` bytes of a group) take the ring's place at the end.
struct BwdPlan {
  int groups, stages, parts;
  size_t smem;
};
template <typename T>
BwdPlan plan(const Bwd<T> &a, int tpr, size_t fixed, size_t each, size_t masks, size_t columns) {
  BwdPlan p;
  p.groups = J_THREADS / tpr;
  while (p.groups > 1 && a.c.rows <= (int64_t)(p.groups / 2) * J_PARTS) p.groups /= 2;
  const size_t stage = fixed + p.groups * each;
  p.stages = 3;
  while (p.stages > 1 && p.stages * stage + p.groups * masks > J_SMEM) --p.stages;
  p.smem = p.stages * stage + p.groups * masks;
  if (p.groups > 1 && p.smem < p.groups * columns) p.smem = p.groups * columns;
  p.parts = (int)grid_of(a.c.rows, p.groups, J_PARTS);
  return p;
}

template <typename K>
cudaError_t allow_smem(K kernel, bool &set) {
  if (set) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, J_SMEM);
  set = e == cudaSuccess;
  return e;
}

template <typename T, bool WARP>
cudaError_t run_odd(const Bwd<T> &a, int tpr, int &parts, cudaStream_t s) {
  auto kernel = join_backward_odd_kernel<T, WARP>;
  const int tensors = (a.dr ? 1 : 0) + (a.has_b ? 1 : 0) + (a.dy ? 2 : 0);
  const BwdPlan p = plan(a, tpr, 0, (size_t)tensors * slot_bytes(a.c.d, sizeof(T)),
                         2 * mask_bytes(a.c.d), (size_t)tpr * 16 * 4);
  static bool set = false;
  const cudaError_t e = allow_smem(kernel, set);
  if (e != cudaSuccess) return e;
  parts = p.parts;
  kernel<<<parts, tpr * p.groups, p.smem, s>>>(a, tpr, p.groups, p.stages, tensors);
  return cudaGetLastError();
}

template <typename T, int NB, bool WARP, bool DROP, bool CENTRED>
cudaError_t run_vec(const Bwd<T> &a, int tpr, int &parts, cudaStream_t s) {
  auto kernel = join_backward_vec_kernel<T, NB, WARP, DROP, CENTRED>;
  const BwdPlan p = plan(a, tpr, (size_t)NB * 4 * Vec8<T>::Q * V8_PIECE, 0, 0, (size_t)tpr * NB * 32);
  static bool set = false;
  const cudaError_t e = allow_smem(kernel, set);
  if (e != cudaSuccess) return e;
  parts = p.parts;
  kernel<<<parts, tpr * p.groups, p.smem, s>>>(a, tpr, p.groups, p.stages);
  return cudaGetLastError();
}
template <typename T, int NB, bool WARP>
cudaError_t vec_kinds(const Bwd<T> &a, int tpr, int &parts, cudaStream_t s) {
  const bool centred = a.c.post == MOE_NORM_LAYER || a.c.pre == MOE_NORM_LAYER;
  if (a.threshold)
    return centred ? run_vec<T, NB, WARP, true, true>(a, tpr, parts, s)
                   : run_vec<T, NB, WARP, true, false>(a, tpr, parts, s);
  return centred ? run_vec<T, NB, WARP, false, true>(a, tpr, parts, s)
                 : run_vec<T, NB, WARP, false, false>(a, tpr, parts, s);
}
template <typename T, int NB>
cudaError_t vec_rows(const Bwd<T> &a, int &parts, cudaStream_t s) {
  const int tpr = ((a.c.d + 8 * NB - 1) / (8 * NB) + 31) / 32 * 32;
  return tpr == 32 ? vec_kinds<T, NB, true>(a, tpr, parts, s)
                   : vec_kinds<T, NB, false>(a, tpr, parts, s);
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
  const bool vectors = whole_vectors<T>(c, {c.ldb, c.ldr, c.lddr, c.lddy, c.lddx, c.lddb});
  const int tpr = threads_of(c.d, 16);
  int parts = 0;
  cudaError_t e;
  if (tpr && vectors) {
    // (fp32: one block per thread where that is enough, so that three rows fit the ring)
    e = sizeof(T) == 4 && c.d <= 4096 ? vec_rows<T, 1>(a, parts, s) : vec_rows<T, 2>(a, parts, s);
  } else if (tpr) {
    e = tpr == 32 ? run_odd<T, true>(a, tpr, parts, s) : run_odd<T, false>(a, tpr, parts, s);
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

size_t join_backward_scratch(const moe_join_config &c) {
  return c.rows > 0 ? (size_t)J_PARTS * J_SUMS * c.d * 4 + (size_t)c.rows * sizeof(float2) : 0;
}

cudaError_t launch_join_backward(const moe_join_config &c, int threshold, const JoinBackward &f,
                                 void *scratch, cudaStream_t s) {
  return c.dtype == MOE_F32 ? backward<float>(c, threshold, f, scratch, s)
                            : backward<__nv_bfloat16>(c, threshold, f, scratch, s);
}

}  // namespace moe
