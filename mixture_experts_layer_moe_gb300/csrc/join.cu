// The joint of a block with the residual stream, and its gradient:
//   z = post(b),  r = scale x + gate . D(z),  y = pre(r)
// (moe.h has the gradient's formulas).  Both are streams through HBM: the forward
// reads x and b and writes r and y, the gradient reads b, r, dr and dy once and
// writes dx and db.
//
// A row belongs to a group of threads (a warp for short rows, else up to a CTA)
// and stays in a ring in shared memory, where it arrives some rows ahead
// (cp.async; what a thread reads it or its warp copied, so no barrier guards the
// ring).  The norms' sums are joined over the group, two for a pair of RMS norms and
// four for layer norms, those of two rows at a time in bf16.  Parameters are
// multiplied together once per CTA (gate, post's gamma, dropout's factor) and stay in
// registers in fp32.  The dropout mask is made again in each direction (philox.cuh).
// In the gradient a thread owns the same columns of every row, so the column sums
// grow in its registers; each CTA writes one partial row of them and a second
// launch adds them in order.
//
// What bounds it is issue before it is HBM: about 30 instructions per element here, 11
// of them for dropout.  16384 x 7168 bf16, two RMS norms, gate and dropout: 160 us,
// 5.9 TB/s; the gradient 243 us, 5.8 TB/s.  (Blocks per thread and rows at a time: 1, 1 223 us; 1, 2 191; 2, 1 198;
// 2, 2 178; 4, 1 208; 4, 2 195, all before the ring's offsets were constants.)
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

// What an iteration moves on by: rows, and bytes of each tensor.  (Computed here: in
// the kernel they would be multiplied out again in every iteration.)
struct FwdSteps {
  int64_t rows, b, x, r, y;
};

// CTAs of few rows hold more threads, of one block each.
constexpr int fwd_threads(int NB) { return NB == 1 ? 2 * J_THREADS : J_THREADS; }

// `groups` groups of tpr threads take R neighbouring rows each, whose sums are joined
// together; NB blocks of eight columns per thread.  CENTRED: a layer norm is
// among the norms.  ODD: rows that are not whole vectors.
template <typename T, int NB, int R, bool DROP, bool CENTRED, bool ODD>
__global__ void __launch_bounds__(fwd_threads(NB), 1)
join_kernel(const __grid_constant__ Fwd<T> a, const __grid_constant__ FwdSteps by, int tpr,
            int groups, int stages) {
  extern __shared__ __align__(16) uint8_t dyn[];   // [stage][row][block][b, x]
  __shared__ float2 buf[2][32];
  constexpr int THREADS = fwd_threads(NB);
  using B = Blocks<T, THREADS, ODD>;
  using Own = Own8<THREADS>;
  constexpr int STAGE = R * NB * 2 * B::BYTES, SIZE = (int)sizeof(T);
  const moe_join_config &c = a.c;
  const int d = c.d, warps = tpr >> 5, warp = threadIdx.x >> 5;
  const int group = warp / warps, tid = threadIdx.x - group * tpr, first_warp = group * warps;
  const float inv_d = 1.f / (float)d;
  const RngState st = load_state(DROP ? a.rng : nullptr);
  const uint32_t cut = (uint32_t)a.threshold << 16;
  const bool layer1 = CENTRED && c.post == MOE_NORM_LAYER, layer2 = CENTRED && c.pre == MOE_NORM_LAYER;
  const bool norm1 = c.post != MOE_NORM_NONE, norm2 = c.pre != MOE_NORM_NONE;
  int turn = 0;
  // blocks of this thread: the first from column 8 tid on, `apart` bytes between them;
  // `left` bytes of a row from a block on.  An active block is there, or (ODD) its
  // warp's first one is.
  const int apart = tpr * 8 * SIZE;
  bool active[NB];
  int valid[NB], left[NB];
  // what the block's output and the joined row are multiplied by, and shifted
  Block8 p1[NB], p2[NB];
  uint8_t *const own = dyn + stages * STAGE;
  auto shift1 = [&](int n) { return Own(own + (2 * n) * Own::BYTES); };
  auto shift2 = [&](int n) { return Own(own + (2 * n + 1) * Own::BYTES); };
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int col = (tid + n * tpr) * 8;
    left[n] = (d - col) * SIZE;
    valid[n] = min(max(d - col, 0), 8);
    active[n] = ODD ? col - (int)(threadIdx.x & 31) * 8 < d : col < d;
    p1[n] = param8(a.gate, col, valid[n], 1.f);
    p2[n] = param8(a.pre_gamma, col, valid[n], 1.f);
    const Block8 g = param8(a.post_gamma, col, valid[n], 1.f);
    Block8 q = CENTRED ? param8(a.post_beta, col, valid[n], 0.f) : fill8(0.f);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      if (DROP) p1[n].v[h] = mul2(p1[n].v[h], both(a.factor));
      if (CENTRED) q.v[h] = mul2(q.v[h], p1[n].v[h]);
      p1[n].v[h] = mul2(p1[n].v[h], g.v[h]);
    }
    if (CENTRED) {
      shift1(n).set(q);
      shift2(n).set(param8(a.pre_beta, col, valid[n], 0.f));
    }
  }
  int64_t row = ((int64_t)blockIdx.x * groups + group) * R, ahead = row;
  uint8_t *const mine = dyn + B::place(), *const ring_end = mine + stages * STAGE;
  auto start = [&](const T *p, int64_t ld) {
    return reinterpret_cast<const char *>(p + row * ld + tid * 8);
  };
  const char *b_ahead = start(a.b, c.ldb), *x_ahead = start(a.x, c.ldx);
  char *r_out = const_cast<char *>(start(a.r, c.ldr)), *y_out = const_cast<char *>(start(a.y, c.ldy));
  // block n of row k of a stage: b, then x
  auto at = [&](uint8_t *stage, int k, int n, int t) {
    return stage + ((k * NB + n) * 2 + t) * B::BYTES;
  };
  auto fill = [&](uint8_t *to) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (ahead + k >= c.rows) break;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (!active[n]) continue;
        B::copy(at(to, k, n, 0), b_ahead + k * c.ldb * SIZE + n * apart, left[n]);
        B::copy(at(to, k, n, 1), x_ahead + k * c.ldx * SIZE + n * apart, left[n]);
      }
    }
    copy_commit();
    ahead += by.rows;
    b_ahead += by.b;
    x_ahead += by.x;
  };
  // the rows' sums over their group
  auto sums = [&](float2 (&s)[R]) {
    if constexpr (R == 1) {
      s[0].x = row_sum(s[0].x + s[0].y, buf, turn, warps);
    } else {
      const float2 t = row_sum2(s[0].x + s[0].y, s[R - 1].x + s[R - 1].y, buf, turn, first_warp, warps);
      s[0].x = t.x;
      s[R - 1].x = t.y;
    }
  };
  for (int i = 0; i < stages - 1; ++i) fill(mine + i * STAGE);
  uint8_t *now = mine, *next = mine + (stages - 1) * STAGE;
  for (int64_t r0 = (int64_t)blockIdx.x * groups * R; r0 < c.rows; r0 += by.rows) {
    // (the stage being filled was read in the iteration before, by this thread or its warp)
    if (ODD) __syncwarp();
    if (stages == 1) fill(next);
    copies_wait(stages - 2);
    auto there = [&](int k, int n) { return active[n] && row + k < c.rows; };
    if (ODD) {
      __syncwarp();
      auto head = [&](const T *p, int64_t ld, int k) {
        return (int)((uint32_t)reinterpret_cast<uintptr_t>(p) + (uint32_t)(row + k) * (uint32_t)ld * SIZE) & 15;
      };
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int hb = head(a.b, c.ldb, k), hx = head(a.x, c.ldx, k);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if (!there(k, n)) continue;
          B::realign(at(now, k, n, 0), hb);
          B::realign(at(now, k, n, 1), hx);
        }
      }
    }
    Block8 v[R][NB];
    float mean1[R], rstd1[R], mean2[R], rstd2[R];
    float2 s[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      s[k] = both(0.f);
      mean1[k] = mean2[k] = 0.f;
      rstd1[k] = rstd2[k] = 1.f;
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        v[k][n] = there(k, n) ? B::load(at(now, k, n, 0)) : fill8(0.f);
        if (layer1) {
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = add2(s[k], v[k][n].v[h]);
        }
      }
    }
    // (here, and not before the loads above: the copies' instructions would delay them)
    if (stages > 1) fill(next);
    if (layer1) {
      sums(s);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        mean1[k] = s[k].x * inv_d;
        s[k] = both(0.f);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
          for (int h = 0; h < 4; ++h) v[k][n].v[h] = add2(v[k][n].v[h], both(-mean1[k]));
          mask8(v[k][n], valid[n]);
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
        const Block8 x = B::load(at(now, k, n, 1));
        Block8 q;
        if (CENTRED) q = shift1(n).get();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          z.v[h] = mul2(z.v[h], both(rstd1[k]));
          z.v[h] = CENTRED ? fma2(z.v[h], p1[n].v[h], q.v[h]) : mul2(z.v[h], p1[n].v[h]);
        }
        if (DROP) drop8(z, dropout_bits(st, tid + n * tpr, (uint32_t)(row + k)), cut);
#pragma unroll
        for (int h = 0; h < 4; ++h) z.v[h] = fma2(both(c.scale), x.v[h], z.v[h]);
        B::store(at(now, k, n, 1), r_out + k * c.ldr * SIZE + n * apart, left[n], z);
        if (layer2) {
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = add2(s[k], z.v[h]);
        } else {
#pragma unroll
          for (int h = 0; h < 4; ++h) s[k] = fma2(z.v[h], z.v[h], s[k]);
        }
      }
    }
    if (norm2) {
      sums(s);
      if (layer2) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
          mean2[k] = s[k].x * inv_d;
          s[k] = both(0.f);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if (!there(k, n)) continue;
#pragma unroll
            for (int h = 0; h < 4; ++h) v[k][n].v[h] = add2(v[k][n].v[h], both(-mean2[k]));
            mask8(v[k][n], valid[n]);
#pragma unroll
            for (int h = 0; h < 4; ++h) s[k] = fma2(v[k][n].v[h], v[k][n].v[h], s[k]);
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
          Block8 q;
          if (CENTRED) q = shift2(n).get();
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            z.v[h] = mul2(z.v[h], both(rstd2[k]));
            z.v[h] = CENTRED ? fma2(z.v[h], p2[n].v[h], q.v[h]) : mul2(z.v[h], p2[n].v[h]);
          }
          B::store(at(now, k, n, 0), y_out + k * c.ldy * SIZE + n * apart, left[n], z);
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
    next = now;
    now = now + STAGE == ring_end ? mine : now + STAGE;
    row += by.rows;
    r_out += by.r;
    y_out += by.y;
  }
}

// ------------------------------------------------- rows of any width, in passes
// One CTA per row, which reads it again (from L2) for each pass; a thread takes
// blocks of eight elements, as the generator gives its bits.  For widths that no ring
// holds, and far from HBM: bf16, two RMS norms, gate and dropout, 8192 x 16384 919 us and
// the gradient 2255 (the bytes 158 and 237), 16384 x 12288 1355 and 3345.  The passes bound it:
// single elements 16 bytes apart over a warp, the generator up to three times.

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

template <typename T, int NB, int R, bool DROP, bool CENTRED, bool ODD>
cudaError_t run(const Fwd<T> &a, cudaStream_t s) {
  auto kernel = join_kernel<T, NB, R, DROP, CENTRED, ODD>;
  constexpr int THREADS = fwd_threads(NB);
  const int tpr = threads_of(a.c.d, NB), groups = groups_of(a.c.rows, R, tpr, J_THREADS, num_sms());
  const size_t stage = (size_t)R * NB * 2 * Blocks<T, THREADS, ODD>::BYTES;
  const size_t own = CENTRED ? 2 * NB * Own8<THREADS>::BYTES : 0;
  const int stages = stages_of(stage, own), threads = tpr * groups;
  const size_t smem = stages * stage + own;
  static int8_t resident[THREADS / 32 + 1] = {};   // CTAs per SM by warps per CTA
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
  const int64_t grid = grid_of(a.c.rows, groups * R, (int64_t)num_sms() * ctas);
  const int64_t rows = grid * groups * R, bytes = rows * sizeof(T);
  const FwdSteps by{rows, bytes * a.c.ldb, bytes * a.c.ldx, bytes * a.c.ldr, bytes * a.c.ldy};
  kernel<<<(unsigned)grid, threads, smem, s>>>(a, by, tpr, groups, stages);
  return cudaGetLastError();
}
template <typename T, int NB, int R, bool ODD>
cudaError_t kinds(const Fwd<T> &a, cudaStream_t s) {
  const bool centred = a.c.post == MOE_NORM_LAYER || a.c.pre == MOE_NORM_LAYER;
  if (a.threshold)
    return centred ? run<T, NB, R, true, true, ODD>(a, s) : run<T, NB, R, true, false, ODD>(a, s);
  return centred ? run<T, NB, R, false, true, ODD>(a, s) : run<T, NB, R, false, false, ODD>(a, s);
}
template <typename T, bool ODD>
cudaError_t forward_ring(const Fwd<T> &a, cudaStream_t s) {
  // few rows: as many threads on each as there can be
  constexpr int R = sizeof(T) == 2 ? 2 : 1;
  return a.c.rows <= num_sms() ? kinds<T, 1, 1, ODD>(a, s) : kinds<T, 2, R, ODD>(a, s);
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
  if (c.d <= J_MAX_D)
    return vectors ? forward_ring<T, sizeof(T) == 4>(a, s) : forward_ring<T, true>(a, s);
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
