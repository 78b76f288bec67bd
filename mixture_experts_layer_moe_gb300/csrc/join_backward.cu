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
  const T *b, *r, *gate, *post_gamma, *post_beta, *pre_gamma;
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


// A load that stays where it is written, among the copies that it follows: a row ahead
// of its use (moved down to the use by the compiler, its latency was exposed in
// every row: 378 us for 301 at 16384 x 7168 bf16).
__device__ __forceinline__ float load_early(const float *p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// The statistics of a row as the forward left them: the post norm's mean and 1 /
// deviation, then the pre norm's (MEANS: the means are read).
template <typename T, bool MEANS = true>
__device__ __forceinline__ float4 stats_of(const Bwd<T> &a, int64_t row) {
  float4 v = make_float4(0.f, 1.f, 0.f, 1.f);
  if (a.c.post != MOE_NORM_NONE) {
    if (MEANS) v.x = load_early(a.stats + row);
    v.y = load_early(a.stats + a.c.rows + row);
  }
  if (a.dy) {
    if (MEANS) v.z = load_early(a.stats + 2 * a.c.rows + row);
    v.w = load_early(a.stats + 3 * a.c.rows + row);
  }
  return v;
}

// What an iteration moves on by: rows, and bytes of each tensor.
struct BwdSteps {
  int64_t rows, dr, dy, r, b, dx, db;
};

template <typename T, int NB, bool CENTRED, bool ODD>
struct BwdRing {
  static constexpr int STAGE = NB * 4 * Blocks<T, J_THREADS, ODD>::BYTES;
  static constexpr int OWN = NB * (CENTRED ? 3 : 1) * Own8<J_THREADS>::BYTES;
  static constexpr int STAGES = stages_of(STAGE, OWN);
  // The pre norm's sums over a row are formed with the post norm's over the row before, so
  // that one barrier serves both: 287 us for 243 (16384 x 7168 bf16).  A row must have
  // landed sooner for it, which loses with two stages (layer norms 368 / 402).
  static constexpr bool AHEAD = STAGES > 2;
  static_assert(!(AHEAD && CENTRED), "two sums at once");
};

// As the forward's kernel.  With rc = r - mean2, bc = b - mean1 (the rows themselves
// without a layer norm, which CENTRED says there is):
//   g = dr + rstd2 dy gamma2 + c2 rc + e2,   c2 = -rstd2^2 mean(w rh),  e2 = -rstd2 mean(w),
//   h = D(g) rstd1 gate gamma1,   db = h + c1 bc + e1  likewise,
// so that neither rh nor bh is formed for itself.
// One row at a time: the column sums take the registers that two would need.  gate
// gamma1 lies in shared memory, with a layer norm the sums of u and dy too: with a few
// values spilled instead, a row waits for the slowest warp's (378 us for 301 at 16384 x
// 7168 bf16).
template <typename T, int NB, bool DROP, bool CENTRED, bool ODD>
__global__ void __launch_bounds__(J_THREADS, 1)
join_backward_kernel(const __grid_constant__ Bwd<T> a, const __grid_constant__ BwdSteps by, int tpr,
                     int groups) {
  extern __shared__ __align__(16) uint8_t dyn[];   // [stage][block][dr, dy, r, b], own values
  __shared__ float2 buf[2][32];
  using B = Blocks<T, J_THREADS, ODD>;
  using Own = Own8<J_THREADS>;
  using R = BwdRing<T, NB, CENTRED, ODD>;
  enum { DR, DY, RR, BB };
  constexpr int STAGE = R::STAGE, STAGES = R::STAGES, SIZE = (int)sizeof(T);
  constexpr bool AHEAD = R::AHEAD;
  const moe_join_config &c = a.c;
  const int d = c.d, warps = tpr >> 5, warp = threadIdx.x >> 5;
  const int group = warp / warps, tid = threadIdx.x - group * tpr, first_warp = group * warps;
  const bool has_dr = a.dr != nullptr, has_dy = a.dy != nullptr, has_b = a.has_b;
  const bool norm1 = c.post != MOE_NORM_NONE;
  const bool layer1 = CENTRED && c.post == MOE_NORM_LAYER, layer2 = CENTRED && c.pre == MOE_NORM_LAYER;
  const float inv_d = 1.f / (float)d;
  const RngState st = load_state(DROP ? a.rng : nullptr);
  const uint32_t cut = (uint32_t)a.threshold << 16;
  int turn = 0;
  pdl_launch_dependents();   // (the column sums wait for this grid to end)
  const int apart = tpr * 8 * SIZE;
  bool active[NB];
  int valid[NB], left[NB];
  // what dy is multiplied by; the column sums of u bh and dy rh, the former without
  // dropout's factor.  In shared memory: what D's kept elements are multiplied by,
  // and the sums of u (without the factor) and dy
  Block8 p2[NB], sum_a[NB], sum_c[NB];
  uint8_t *const own = dyn + STAGES * STAGE;
  auto p1 = [&](int n) { return Own(own + n * Own::BYTES); };
  auto sum_b = [&](int n) { return Own(own + (NB + n) * Own::BYTES); };
  auto sum_e = [&](int n) { return Own(own + (2 * NB + n) * Own::BYTES); };
  auto grow = [](const Own &sum, const Block8 &by) {
    Block8 s = sum.get();
#pragma unroll
    for (int h = 0; h < 4; ++h) s.v[h] = add2(s.v[h], by.v[h]);
    sum.set(s);
  };
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int col = (tid + n * tpr) * 8;
    left[n] = (d - col) * SIZE;
    valid[n] = min(max(d - col, 0), 8);
    active[n] = ODD ? col - (int)(threadIdx.x & 31) * 8 < d : col < d;
    sum_a[n] = sum_c[n] = fill8(0.f);
    p2[n] = param8(a.pre_gamma, col, valid[n], 1.f);
    Block8 p = param8(a.gate, col, valid[n], 1.f);
    const Block8 g = param8(a.post_gamma, col, valid[n], 1.f);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      p.v[h] = mul2(p.v[h], g.v[h]);
      if (DROP) p.v[h] = mul2(p.v[h], both(a.factor));
    }
    p1(n).set(p);
    if (CENTRED) {
      sum_b(n).set(fill8(0.f));
      sum_e(n).set(fill8(0.f));
    }
  }
  int64_t row = (int64_t)blockIdx.x * groups + group, ahead = row;
  uint8_t *const mine = dyn + B::place(), *const ring_end = mine + STAGES * STAGE;
  auto start = [&](const T *p, int64_t ld) {
    return reinterpret_cast<const char *>(p + row * ld + tid * 8);
  };
  const char *dr_ahead = start(a.dr, c.lddr), *dy_ahead = start(a.dy, c.lddy);
  const char *r_ahead = start(a.r, c.ldr), *b_ahead = start(a.b, c.ldb);
  char *dx_out = const_cast<char *>(start(a.dx, c.lddx));
  char *db_out = const_cast<char *>(start(a.db, c.lddb));
  auto at = [&](uint8_t *stage, int n, int t) { return stage + (n * 4 + t) * B::BYTES; };
  auto fill = [&](uint8_t *to) {
    if (ahead < c.rows) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!active[n]) continue;
        if (has_dy) {
          B::copy(at(to, n, DY), dy_ahead + n * apart, left[n]);
          B::copy(at(to, n, RR), r_ahead + n * apart, left[n]);
        }
        if (has_dr) B::copy(at(to, n, DR), dr_ahead + n * apart, left[n]);
        if (has_b) B::copy(at(to, n, BB), b_ahead + n * apart, left[n]);
      }
    }
    copy_commit();
    ahead += by.rows;
    dr_ahead += by.dr;
    dy_ahead += by.dy;
    r_ahead += by.r;
    b_ahead += by.b;
  };
  // the elements of a row that landed, where its threads read them
  auto align = [&](uint8_t *stage, int64_t row) {
    if (!ODD) return;
    __syncwarp();
    if (row >= c.rows) return;
    auto head = [&](const T *p, int64_t ld) {
      return (int)((uint32_t)reinterpret_cast<uintptr_t>(p) + (uint32_t)row * (uint32_t)ld * SIZE) & 15;
    };
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (!active[n]) continue;
      if (has_dy) {
        B::realign(at(stage, n, DY), head(a.dy, c.lddy));
        B::realign(at(stage, n, RR), head(a.r, c.ldr));
      }
      if (has_dr) B::realign(at(stage, n, DR), head(a.dr, c.lddr));
      if (has_b) B::realign(at(stage, n, BB), head(a.b, c.ldb));
    }
  };
  auto centred = [&](uint8_t *at, float mean) {
    Block8 b = B::load(at);
    if (CENTRED) {
#pragma unroll
      for (int h = 0; h < 4; ++h) b.v[h] = add2(b.v[h], both(-mean));
    }
    return b;
  };
  // this thread's share of the sums of w and w rc (a column that is not there has gamma 0)
  auto pre_sums = [&](uint8_t *stage, int64_t row, float mean) {
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (row >= c.rows || !active[n]) continue;
      const Block8 dy = B::load(at(stage, n, DY)), rc = centred(at(stage, n, RR), mean);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float2 w = mul2(dy.v[h], p2[n].v[h]);
        if (CENTRED) s1 = add2(s1, w);
        s2 = fma2(w, rc.v[h], s2);
      }
    }
    return make_float2(s1.x + s1.y, s2.x + s2.y);
  };
  for (int i = 0; i < STAGES - 1; ++i) fill(mine + i * STAGE);
  uint8_t *now = mine, *next = mine + (STAGES - 1) * STAGE;
  float4 next_stat = make_float4(0.f, 1.f, 0.f, 1.f);
  if (row < c.rows) next_stat = stats_of<T, CENTRED>(a, row);
  // a norm's sums over the group
  auto join = [&](float2 v) {
    if (CENTRED) return row_sum2(v.x, v.y, buf, turn, first_warp, warps);
    return make_float2(0.f, row_sum(v.y, buf, turn, warps));
  };
  float2 pre = both(0.f);   // AHEAD: those of the pre norm over the coming row
  if (AHEAD) {
    copies_wait(STAGES - 2);
    align(now, row);
    if (has_dy) pre = join(pre_sums(now, row, next_stat.z));
  }
  const bool norm_b = norm1 && a.db != nullptr;
  for (int64_t r0 = (int64_t)blockIdx.x * groups; r0 < c.rows; r0 += by.rows) {
    const bool live = row < c.rows;
    // (the stage being filled was read in the iteration before, by this thread or its warp)
    if (ODD) __syncwarp();
    if (STAGES == 1) fill(next);
    const float4 stat = next_stat;
    if (row + by.rows < c.rows) next_stat = stats_of<T, CENTRED>(a, row + by.rows);
    if (!AHEAD) {
      copies_wait(STAGES - 2);
      align(now, row);
      if (has_dy) pre = pre_sums(now, row, stat.z);
      if (STAGES > 1) fill(next);
      if (has_dy) pre = join(pre);
    }
    // (1 / deviation meets the sum before itself: its cube alone leaves fp32's range for rows of
    // a root mean square above 4e12 or below 1e-13)
    const float c2 = -stat.w * (stat.w * (stat.w * pre.y * inv_d));
    const float e2 = layer2 ? -stat.w * pre.x * inv_d : 0.f;
    auto get = [&](int n, int t) { return B::load(at(now, n, t)); };
    Block8 w[NB];
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      w[n] = fill8(0.f);
      if (!live || !active[n]) continue;
      Block8 g = has_dr ? get(n, DR) : fill8(0.f);
      if (has_dy) {
        const Block8 rc = centred(at(now, n, RR), stat.z);
        Block8 dy = get(n, DY);
        if (CENTRED) grow(sum_e(n), dy);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (CENTRED) g.v[h] = add2(g.v[h], both(e2));
          dy.v[h] = mul2(dy.v[h], both(stat.w));
          sum_c[n].v[h] = fma2(dy.v[h], rc.v[h], sum_c[n].v[h]);
          g.v[h] = fma2(dy.v[h], p2[n].v[h], fma2(rc.v[h], both(c2), g.v[h]));
        }
      }
      if (a.dx) {
        Block8 t;
#pragma unroll
        for (int h = 0; h < 4; ++h) t.v[h] = mul2(both(c.scale), g.v[h]);
        B::store(at(now, n, DR), dx_out + n * apart, left[n], t);
      }
      if (DROP) drop8(g, dropout_bits(st, tid + n * tpr, (uint32_t)row), cut);
      if (CENTRED) grow(sum_b(n), g);
      if (norm1) {
#pragma unroll
        for (int h = 0; h < 4; ++h) g.v[h] = mul2(g.v[h], both(stat.y));
      }
      const Block8 p = p1(n).get();
#pragma unroll
      for (int h = 0; h < 4; ++h) w[n].v[h] = mul2(g.v[h], p.v[h]);
      if (has_b) {
        const Block8 bc = centred(at(now, n, BB), stat.x);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          sum_a[n].v[h] = fma2(g.v[h], bc.v[h], sum_a[n].v[h]);
          if (CENTRED) s1 = add2(s1, w[n].v[h]);
          s2 = fma2(w[n].v[h], bc.v[h], s2);
        }
      }
    }
    uint8_t *const then = now + STAGE == ring_end ? mine : now + STAGE;
    float2 post = make_float2(s1.x + s1.y, s2.x + s2.y);
    if (AHEAD) {
      fill(next);   // (here: before the row's work 233 us for 219 without a post norm)
      copies_wait(STAGES - 2);
      align(then, row + by.rows);
      if (has_dy) pre = pre_sums(then, row + by.rows, next_stat.z);
      if (norm_b || has_dy) {
        const float2 t = row_sum2(post.y, pre.y, buf, turn, first_warp, warps);
        post.y = t.x;
        pre.y = t.y;
      }
    } else if (norm_b) {
      post = join(post);
    }
    if (a.db) {
      // (w is rstd1 times the gradient of the normed row)
      const float c1 = -stat.y * (stat.y * post.y * inv_d), e1 = layer1 ? -post.x * inv_d : 0.f;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!live || !active[n]) continue;
        if (norm1) {
          const Block8 bc = centred(at(now, n, BB), stat.x);
#pragma unroll
          for (int h = 0; h < 4; ++h)
            w[n].v[h] = fma2(bc.v[h], both(c1), CENTRED ? add2(w[n].v[h], both(e1)) : w[n].v[h]);
        }
        B::store(at(now, n, DY), db_out + n * apart, left[n], w[n]);
      }
    }
    next = now;
    now = then;
    row += by.rows;
    dx_out += by.dx;
    db_out += by.db;
  }
  // each group's sums, and where there are several their sum through shared memory
  // (the ring's, now read; no copy is in flight: the ones past the last row were
  // empty)
  copy_wait<0>();
  float *const cols = reinterpret_cast<float *>(dyn);
  const int width = tpr * 8 * NB;
#pragma unroll
  for (int which = 0; which < J_SUMS; ++which) {
    if (!(a.sums >> which & 1) || (!CENTRED && (which & 1))) continue;
    const float factor = DROP && which < 2 ? a.factor : 1.f;
    float *part = a.parts + ((int64_t)blockIdx.x * J_SUMS + which) * d;
    float *to = groups == 1 ? part : cols + group * width;
    if (groups > 1) __syncthreads();
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const Block8 s = which == 0 ? sum_a[n] : which == 1 ? sum_b(n).get()
                       : which == 2 ? sum_c[n] : sum_e(n).get();
      const float *f = reinterpret_cast<const float *>(s.v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < valid[n]) to[(tid + n * tpr) * 8 + i] = f[i] * factor;
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
  __shared__ float s[J_SUMS][32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = blockIdx.x * 32 + lane, out = blockIdx.x * 32 + warp;
  constexpr int EACH = (J_PARTS + 31) / 32;
  float v[J_SUMS][EACH] = {}, total[J_SUMS];
  pdl_wait();
  // (all loads first: the sums one after the other took 9 to 12 us)
#pragma unroll
  for (int i = 0; i < J_SUMS; ++i) {
    if (!(a.sums >> i & 1)) continue;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int p = warp + 32 * k;
      if (mine < a.d && p < a.count) v[i][k] = a.parts[((int64_t)p * J_SUMS + i) * a.d + mine];
    }
  }
#pragma unroll
  for (int i = 0; i < J_SUMS; ++i) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < EACH; ++k) t += v[i][k];
    s[i][warp][lane] = t;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < J_SUMS; ++i) total[i] = warp_sum_xor(s[i][lane][warp]);
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

// (one CTA per SM at most: each leaves a partial row of the column sums, which meet in
// the ring's place)
template <typename T, int NB, bool DROP, bool CENTRED, bool ODD>
cudaError_t run(const Bwd<T> &a, int &parts, cudaStream_t s) {
  auto kernel = join_backward_kernel<T, NB, DROP, CENTRED, ODD>;
  const moe_join_config &c = a.c;
  const int tpr = threads_of(c.d, NB), groups = groups_of(c.rows, 1, tpr, J_THREADS, J_PARTS);
  using R = BwdRing<T, NB, CENTRED, ODD>;
  static_assert(R::STAGE >= J_THREADS * NB * 32, "the groups' column sums fit a stage");
  static bool set = false;
  if (!set) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, J_SMEM);
    if (e != cudaSuccess) return e;
    set = true;
  }
  parts = (int)grid_of(c.rows, groups, J_PARTS);
  const int64_t rows = (int64_t)parts * groups, bytes = rows * sizeof(T);
  const BwdSteps by{rows,          bytes * c.lddr, bytes * c.lddy, bytes * c.ldr,
                    bytes * c.ldb, bytes * c.lddx, bytes * c.lddb};
  kernel<<<parts, tpr * groups, R::STAGES * R::STAGE + R::OWN, s>>>(a, by, tpr, groups);
  return cudaGetLastError();
}
template <typename T, int NB, bool ODD>
cudaError_t kinds(const Bwd<T> &a, int &parts, cudaStream_t s) {
  const bool centred = a.c.post == MOE_NORM_LAYER || a.c.pre == MOE_NORM_LAYER;
  if (a.threshold)
    return centred ? run<T, NB, true, true, ODD>(a, parts, s) : run<T, NB, true, false, ODD>(a, parts, s);
  return centred ? run<T, NB, false, true, ODD>(a, parts, s) : run<T, NB, false, false, ODD>(a, parts, s);
}
// fp32: one block per thread where that is enough, so that several rows fit the ring.
template <typename T, bool ODD>
cudaError_t backward_ring(const Bwd<T> &a, int &parts, cudaStream_t s) {
  return sizeof(T) == 4 && a.c.d <= J_MAX_D / 2 ? kinds<T, sizeof(T) == 4 ? 1 : 2, ODD>(a, parts, s)
                                                : kinds<T, 2, ODD>(a, parts, s);
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
  int parts = 0;
  cudaError_t e;
  if (c.d <= J_MAX_D) {
    e = vectors ? backward_ring<T, sizeof(T) == 4>(a, parts, s) : backward_ring<T, true>(a, parts, s);
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
