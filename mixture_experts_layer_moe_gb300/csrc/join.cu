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
#include "join_common.cuh"

namespace moe {
namespace {

using namespace join;

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

// Rows of whole vectors.  `groups` groups of tpr threads take R neighbouring rows each,
// whose sums are joined together; NB blocks of eight columns per thread.  CENTRED:
// a layer norm is among the norms.
template <typename T, int NB, int R, bool WARP, bool DROP, bool CENTRED>
__global__ void __launch_bounds__(NB == 1 ? 1024 : 512, 1)
join_vec_kernel(const __grid_constant__ Fwd<T> a, int tpr, int groups, int stages) {
  extern __shared__ __align__(16) uint4 dyn[];   // [stage][row][block][b, x][vector][thread]
  __shared__ float2 buf[2][32];
  using V = Vec8<T>;
  constexpr int PIECE = NB == 1 ? 2 * V8_PIECE : V8_PIECE, STAGE = R * NB * 2 * V::Q * PIECE;
  const moe_join_config &c = a.c;
  const int d = c.d, warps = tpr >> 5, warp = threadIdx.x >> 5;
  const int group = WARP ? warp : warp / warps, tid = threadIdx.x - group * tpr;
  const int first_warp = group * warps;
  const float inv_d = 1.f / (float)d;
  const RngState st = load_state(DROP ? a.rng : nullptr);
  const uint32_t cut = (uint32_t)a.threshold << 16;
  const bool layer1 = CENTRED && c.post == MOE_NORM_LAYER, layer2 = CENTRED && c.pre == MOE_NORM_LAYER;
  const bool norm1 = c.post != MOE_NORM_NONE, norm2 = c.pre != MOE_NORM_NONE;
  int turn = 0;
  // blocks of this thread: the first from column 8 tid on, `apart` bytes between them
  const int apart = tpr * 8 * (int)sizeof(T);
  bool on[NB];
  // what the block's output and the joined row are multiplied by, and shifted
  Block8 p1[NB], p2[NB], q1[CENTRED ? NB : 1], q2[CENTRED ? NB : 1];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int col = (tid + n * tpr) * 8;
    on[n] = col < d;
    p1[n] = p2[n] = fill8(0.f);
    if (CENTRED) q1[n] = q2[n] = fill8(0.f);
    if (!on[n]) continue;
    p1[n] = V::param(a.gate, col, 1.f);
    const Block8 g = V::param(a.post_gamma, col, 1.f);
    p2[n] = V::param(a.pre_gamma, col, 1.f);
    if (CENTRED) {
      q1[n] = V::param(a.post_beta, col, 0.f);
      q2[n] = V::param(a.pre_beta, col, 0.f);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (DROP) p1[n].v[h] = mul2(p1[n].v[h], both(a.factor));
      if (CENTRED) q1[n].v[h] = mul2(q1[n].v[h], p1[n].v[h]);
      p1[n].v[h] = mul2(p1[n].v[h], g.v[h]);
    }
  }
  const int64_t step = (int64_t)gridDim.x * groups * R;
  int64_t row = ((int64_t)blockIdx.x * groups + group) * R, ahead = row;
  uint8_t *const mine = reinterpret_cast<uint8_t *>(dyn) + threadIdx.x * 16;
  uint8_t *const ring_end = mine + stages * STAGE;
  auto bytes = [](int64_t elements) { return elements * (int64_t)sizeof(T); };
  auto start = [&](const T *p, int64_t ld) {
    return reinterpret_cast<const char *>(p + row * ld + tid * 8);
  };
  const char *b_ahead = start(a.b, c.ldb), *x_ahead = start(a.x, c.ldx);
  char *r_out = const_cast<char *>(start(a.r, c.ldr)), *y_out = const_cast<char *>(start(a.y, c.ldy));
  auto fill = [&](uint8_t *to) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (ahead + k >= c.rows) break;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!on[n]) continue;
        V::template copy<PIECE>(to, (k * NB + n) * 2, b_ahead + k * bytes(c.ldb) + n * apart);
        V::template copy<PIECE>(to, (k * NB + n) * 2 + 1, x_ahead + k * bytes(c.ldx) + n * apart);
      }
    }
    copy_commit();
    ahead += step;
    b_ahead += bytes(step * c.ldb);
    x_ahead += bytes(step * c.ldx);
  };
  // the rows' sums over their group
  auto sums = [&](float2 (&s)[R]) {
    if constexpr (R == 1) {
      s[0].x = group_sum<WARP>(s[0].x + s[0].y, reinterpret_cast<float (*)[32]>(buf), turn, warps);
    } else {
      const float2 t = group_sum2<WARP>(s[0].x + s[0].y, s[R - 1].x + s[R - 1].y, buf, turn,
                                        first_warp, warps);
      s[0].x = t.x;
      s[R - 1].x = t.y;
    }
  };
  for (int i = 0; i < stages - 1; ++i) fill(mine + i * STAGE);
  uint8_t *now = mine, *next = mine + (stages - 1) * STAGE;
  for (int64_t r0 = (int64_t)blockIdx.x * groups * R; r0 < c.rows; r0 += step) {
    // (the stage being filled was read by this thread in the iteration before)
    fill(next);
    copies_wait(stages - 1);
    Block8 v[R][NB];
    float mean1[R], rstd1[R], mean2[R], rstd2[R];
    float2 s[R];
    auto there = [&](int k, int n) { return on[n] && row + k < c.rows; };
#pragma unroll
    for (int k = 0; k < R; ++k) {
      s[k] = both(0.f);
      mean1[k] = mean2[k] = 0.f;
      rstd1[k] = rstd2[k] = 1.f;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        v[k][n] = there(k, n) ? V::template ring<PIECE>(now, (k * NB + n) * 2) : fill8(0.f);
        if (layer1) {
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = add2(s[k], v[k][n].v[h]);
        }
      }
    }
    if (layer1) {
      sums(s);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        mean1[k] = s[k].x * inv_d;
        s[k] = both(0.f);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if (!on[n]) continue;
#pragma unroll
          for (int h = 0; h < 4; ++h) v[k][n].v[h] = add2(v[k][n].v[h], both(-mean1[k]));
        }
      }
    }
    if (norm1) {
#pragma unroll
      for (int k = 0; k < R; ++k)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = fma2(v[k][n].v[h], v[k][n].v[h], s[k]);
      sums(s);
#pragma unroll
      for (int k = 0; k < R; ++k) rstd1[k] = rsqrtf(s[k].x * inv_d + c.eps);
    }
    // the joined rows, and the sum that the next norm takes of them
#pragma unroll
    for (int k = 0; k < R; ++k) {
      s[k] = both(0.f);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!there(k, n)) {
          v[k][n] = fill8(0.f);
          continue;
        }
        Block8 &z = v[k][n];
        const Block8 x = V::template ring<PIECE>(now, (k * NB + n) * 2 + 1);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          z.v[h] = mul2(z.v[h], both(rstd1[k]));
          z.v[h] = CENTRED ? fma2(z.v[h], p1[n].v[h], q1[n].v[h]) : mul2(z.v[h], p1[n].v[h]);
        }
        if (DROP) drop8(z, dropout_bits(st, tid + n * tpr, (uint32_t)(row + k)), cut);
#pragma unroll
        for (int h = 0; h < 4; ++h) z.v[h] = fma2(both(c.scale), x.v[h], z.v[h]);
        V::store(r_out + k * bytes(c.ldr) + n * apart, z);
        if (layer2) {
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = add2(s[k], z.v[h]);
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = fma2(z.v[h], z.v[h], s[k]);
        }
      }
    }
    next = now;
    now = now + STAGE == ring_end ? mine : now + STAGE;
    if (norm2) {
      sums(s);
      if (layer2) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
          mean2[k] = s[k].x * inv_d;
          s[k] = both(0.f);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if (!on[n]) continue;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              v[k][n].v[h] = add2(v[k][n].v[h], both(-mean2[k]));
              s[k] = fma2(v[k][n].v[h], v[k][n].v[h], s[k]);
            }
          }
        }
        sums(s);
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        rstd2[k] = rsqrtf(s[k].x * inv_d + c.eps);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if (!there(k, n)) continue;
          Block8 &z = v[k][n];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            z.v[h] = mul2(z.v[h], both(rstd2[k]));
            z.v[h] = CENTRED ? fma2(z.v[h], p2[n].v[h], q2[n].v[h]) : mul2(z.v[h], p2[n].v[h]);
          }
          V::store(y_out + k * bytes(c.ldy) + n * apart, z);
        }
      }
    }
    if (a.stats && tid == 0) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (row + k >= c.rows) break;
        a.stats[row + k] = mean1[k];
        a.stats[c.rows + row + k] = rstd1[k];
        a.stats[2 * c.rows + row + k] = mean2[k];
        a.stats[3 * c.rows + row + k] = rstd2[k];
      }
    }
    row += step;
    r_out += bytes(step * c.ldr);
    y_out += bytes(step * c.ldy);
  }
}

// Rows that are not whole vectors: the aligned pieces that cover a row, in a slot
// that the group reads.
template <typename T, bool WARP>
__global__ void __launch_bounds__(J_THREADS, 2)
join_odd_kernel(const __grid_constant__ Fwd<T> a, int tpr, int groups, int stages) {
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ float buf[2][32];
  using C = Chunk<T, 1>;
  using R = Ring<T>;
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
  const bool dropping = a.threshold != 0;
  const RngState st = load_state(dropping ? a.rng : nullptr);
  const bool layer1 = c.post == MOE_NORM_LAYER, layer2 = c.pre == MOE_NORM_LAYER;
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
    const T *b_row = a.b + row * c.ldb, *x_row = a.x + row * c.ldx;
    auto there = [&](int i) { return live && ring.col(i) < d; };
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f;
    if (layer1) {
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
        for (int h = 0; h < H; ++h)
          v[h] = add2(v[h], both(-mean1));
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
      if (dropping) z[0] = drop_pair(ring, masks, i, z[0], a.factor);
      if (a.gate) {
        params(ring, a.gate, i, 1.f, q);
#pragma unroll
        for (int h = 0; h < H; ++h) z[h] = mul2(z[h], q[h]);
      }
      ring.get(stage, i, 1, x_row, q);
#pragma unroll
      for (int h = 0; h < H; ++h) v[i][h] = fma2(both(c.scale), q[h], z[h]);
      C::mask(ring.col(i), tpr, d, v[i]);
      if (layer2) {
#pragma unroll
        for (int h = 0; h < H; ++h) s = add2(s, v[i][h]);
      } else {
#pragma unroll
        for (int h = 0; h < H; ++h) s = fma2(v[i][h], v[i][h], s);
      }
    }
    stage = stage + 1 == stages ? 0 : stage + 1;
    if (layer2) {
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

// ------------------------------------------------- rows of any width, in passes
// One CTA per row, which reads it again (from L2) for each pass; a thread takes
// blocks of eight elements, as the generator gives its bits.

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
  const RngState st = load_state(a.threshold ? a.rng : nullptr);
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

template <typename T, bool WARP>
cudaError_t run_odd(const Fwd<T> &a, int tpr, cudaStream_t s) {
  auto kernel = join_odd_kernel<T, WARP>;
  const int groups = tpr <= 256 ? 256 / tpr : 1, threads = tpr * groups;
  const size_t stage = (size_t)groups * 2 * slot_bytes(a.c.d, sizeof(T));
  const size_t masks = (size_t)groups * 2 * mask_bytes(a.c.d);
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

// Rows of whole vectors: threads per row, and CTAs as the SMs hold.
template <typename T, int NB, int R, bool WARP, bool DROP, bool CENTRED>
cudaError_t run_vec(const Fwd<T> &a, int tpr, cudaStream_t s) {
  auto kernel = join_vec_kernel<T, NB, R, WARP, DROP, CENTRED>;
  int groups = tpr < 512 ? 512 / tpr : 1;
  while (groups > 1 && a.c.rows <= (int64_t)(groups / 2) * R * num_sms()) groups /= 2;
  const int threads = tpr * groups;
  const size_t stage = (size_t)R * NB * 2 * Vec8<T>::Q * (NB == 1 ? 2 * V8_PIECE : V8_PIECE);
  int stages = 3;
  while (stages > 1 && stages * stage > J_SMEM) --stages;
  const size_t smem = stages * stage;
  static int8_t resident[1024 / 32 + 1] = {};   // CTAs per SM by warps per CTA
  int8_t &ctas = resident[threads / 32];
  if (ctas == 0) {
    int n = 0;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, J_SMEM);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    ctas = (int8_t)(n < 1 ? 1 : n);
  }
  kernel<<<(unsigned)grid_of(a.c.rows, groups * R, (int64_t)num_sms() * ctas), threads, smem, s>>>(
      a, tpr, groups, stages);
  return cudaGetLastError();
}
template <typename T, int NB, int R, bool WARP>
cudaError_t vec_kinds(const Fwd<T> &a, int tpr, cudaStream_t s) {
  const bool centred = a.c.post == MOE_NORM_LAYER || a.c.pre == MOE_NORM_LAYER;
  if (a.threshold)
    return centred ? run_vec<T, NB, R, WARP, true, true>(a, tpr, s)
                   : run_vec<T, NB, R, WARP, true, false>(a, tpr, s);
  return centred ? run_vec<T, NB, R, WARP, false, true>(a, tpr, s)
                 : run_vec<T, NB, R, WARP, false, false>(a, tpr, s);
}

template <typename T, int NB, int R>
cudaError_t vec_rows(const Fwd<T> &a, cudaStream_t s) {
  const int tpr = ((a.c.d + 8 * NB - 1) / (8 * NB) + 31) / 32 * 32;
  return tpr == 32 ? vec_kinds<T, NB, R, true>(a, tpr, s) : vec_kinds<T, NB, R, false>(a, tpr, s);
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
  const bool vectors = whole_vectors<T>(c, {c.ldx, c.ldb, c.ldr, c.ldy});
  if (vectors && c.d <= 8192) {
    // few rows: as many threads on each as there can be
    constexpr int R = sizeof(T) == 2 ? 2 : 1;
    return c.rows <= num_sms() ? vec_rows<T, 1, 1>(a, s) : vec_rows<T, 2, R>(a, s);
  }
  const int tpr = threads_of(c.d, 16);
  if (tpr && !vectors) return tpr == 32 ? run_odd<T, true>(a, tpr, s) : run_odd<T, false>(a, tpr, s);
  join_wide_kernel<T><<<(unsigned)grid_of(c.rows, 1, (int64_t)num_sms() * 4), J_WIDE, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_join(const moe_join_config &c, int threshold, const JoinForward &f,
                        cudaStream_t s) {
  return c.dtype == MOE_F32 ? forward<float>(c, threshold, f, s)
                            : forward<__nv_bfloat16>(c, threshold, f, s);
}

}  // namespace moe
