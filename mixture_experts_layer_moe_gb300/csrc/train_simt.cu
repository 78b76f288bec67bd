// The grouped products of training on CUDA cores (fp32 FMA accumulation).
//
// The path of fp32 layers (tensor cores multiply fp32 operands in fewer
// bits), written for their sizes: a layer of a few hundred rows, whose
// launches cost as much as its products; and of bf16 layers so small that
// setting up the tensor-core kernels is most of their time (32 x 32 tiles).
// A CTA computes a tile of one segment's rows (RowsProduct) or of one expert's
// gradient (GradProduct) with 256 threads: 64 x 64, or 32 x 32 where the larger
// tiles would not give every SM one.  The next step's operands are loaded into
// registers while the current one is multiplied (two steps ahead took the
// registers of resident CTAs: 770 us for 743 at 4096 rows of 16 experts, d 512,
// d_ff 1024), and shared memory is double buffered, so a step waits for memory
// once, not twice (256 rows, d 128, d_ff
// 512, 4 experts, forward: 49 us without any of it, 15.6 with).
// Large layers are bound by reading the operands from shared memory (4096 rows of
// 16 experts, d 512, d_ff 1024: its wavefronts at 82-92 % of their peak, the FMA pipe
// at 45-54 %; 36 TFLOP/s).  8 x 8 outputs per thread read half as often (FMA 51-64
// %) but need the tile's sums joined from groups of threads: 1 to 18 % less
// time there, up to 18 % more for the short reductions of a router.
// The three storage orders of the operands differ in how a tile is staged
// only: in shared memory both operands lie reduction index first, so that a
// thread reads its values of a step as two vectors.
#include <math.h>

#include "common.cuh"
#include "fp32x2.cuh"
#include "launch.h"
#include "train.h"

namespace moe {
namespace {

constexpr int T_THREADS = 256;

// TILE x TILE outputs per CTA, 4 x 4 per thread, TK reduction indexes a step.
// A 32 x 32 tile has threads for four groups, which take a quarter of a step's
// indexes each and are added up at the end (2 x 2 outputs per thread instead
// read shared memory four times as often).
template <int TILE>
struct Geo {
  static constexpr int TX = TILE / 4, GROUPS = T_THREADS / (TX * TX);
  static constexpr int TK = TILE == 64 ? 16 : 64, LD = TILE + 4;
  static constexpr int LOADS = TILE * TK / 4 / T_THREADS;   // vectors of 4 per thread
  using Buf = float[TK][LD];
};

__device__ __forceinline__ float4 load4(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

// This thread's part of a TK x TILE operand tile, as vectors of 4: element
// (kk, i) is src[i * ld + kk] (K_FAST) or src[kk * ld + i]; zero outside i < ni,
// kk < nk.  The contiguous bound and ld are multiples of 4, and src lies on a
// vector's boundary.
template <typename T, bool K_FAST, int TILE>
struct Part {
  using G = Geo<TILE>;
  float4 v[G::LOADS];
  static __device__ __forceinline__ int kk(int l) { return K_FAST ? l % (G::TK / 4) * 4 : l / (TILE / 4); }
  static __device__ __forceinline__ int ii(int l) { return K_FAST ? l / (G::TK / 4) : l % (TILE / 4) * 4; }
  __device__ __forceinline__ void load(const T *src, int64_t ld, int ni, int nk) {
#pragma unroll
    for (int c = 0; c < G::LOADS; ++c) {
      const int l = threadIdx.x + c * T_THREADS, k = kk(l), i = ii(l);
      v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < ni && k < nk) v[c] = load4(src + (K_FAST ? i * ld + k : k * ld + i));
    }
  }
  __device__ __forceinline__ void store(typename G::Buf &dst) const {
#pragma unroll
    for (int c = 0; c < G::LOADS; ++c) {
      const int l = threadIdx.x + c * T_THREADS, k = kk(l), i = ii(l);
      if (K_FAST) {
        dst[k][i] = v[c].x;
        dst[k + 1][i] = v[c].y;
        dst[k + 2][i] = v[c].z;
        dst[k + 3][i] = v[c].w;
      } else {
        *reinterpret_cast<float4 *>(&dst[k][i]) = v[c];
      }
    }
  }
};

template <int TILE>
__device__ __forceinline__ void tile_fma(float2 (&acc)[4][2], const typename Geo<TILE>::Buf &as,
                                         const typename Geo<TILE>::Buf &bs, int tx, int ty, int g) {
#pragma unroll
  for (int kk = 0; kk < Geo<TILE>::TK; kk += Geo<TILE>::GROUPS) {
    const float4 a4 = *reinterpret_cast<const float4 *>(&as[kk + g][ty * 4]);
    const float4 b4 = *reinterpret_cast<const float4 *>(&bs[kk + g][tx * 4]);
    const float a[4] = {a4.x, a4.y, a4.z, a4.w};
    const float2 b[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = fma2(both(a[i]), b[j], acc[i][j]);
  }
}

// Adds the groups' sums in order, through `scratch` (GROUPS x TILE x TILE
// floats of shared memory that nothing else uses any more), so that each
// thread ends with four neighbouring outputs of one row: acc[0].
template <int TILE>
__device__ __forceinline__ void join_groups(float2 (&acc)[4][2], float *scratch, int tx, int ty,
                                            int g) {
  if constexpr (Geo<TILE>::GROUPS > 1) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4 *>(scratch + (g * TILE + ty * 4 + i) * TILE + tx * 4) =
          make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
    __syncthreads();
    float4 sum = *reinterpret_cast<const float4 *>(scratch + threadIdx.x * 4);
#pragma unroll
    for (int h = 1; h < Geo<TILE>::GROUPS; ++h) {
      const float4 v = *reinterpret_cast<const float4 *>(scratch + h * TILE * TILE + threadIdx.x * 4);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    acc[0][0] = make_float2(sum.x, sum.y);
    acc[0][1] = make_float2(sum.z, sum.w);
  }
}

// This thread's place: its 4 x 4 outputs while summing, and the rows x 4
// outputs it ends with.
template <int TILE>
struct Place {
  static constexpr int ROWS = Geo<TILE>::GROUPS > 1 ? 1 : 4;
  int tx, ty, g, row, col;
  __device__ __forceinline__ Place() {
    constexpr int TX = Geo<TILE>::TX;
    g = threadIdx.x / (TX * TX);
    tx = threadIdx.x % TX;
    ty = threadIdx.x / TX % TX;
    row = ROWS == 1 ? threadIdx.x / TX : ty * 4;
    col = tx * 4;
  }
};

template <typename T>
__device__ __forceinline__ void get4(const void *p, int64_t at, float (&v)[4]) {
  const float4 t = load4(static_cast<const T *>(p) + at);
  v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
}
template <typename T>
__device__ __forceinline__ void put4(void *p, int64_t at, const float (&v)[4]) {
  store4(static_cast<T *>(p) + at, v);
}

// Expert and row range of this CTA's tile; false when there is none.  Every warp
// looks for itself, 32 experts at a time.
template <int TM>
__device__ __forceinline__ bool find_tile(const int32_t *offsets, int E, int rows, int tile, int &e,
                                          int &row0, int &end, int *status) {
  if (offsets == nullptr) {
    e = 0;
    row0 = tile * TM;
    end = rows;
    return row0 < end;
  }
  const unsigned all = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int before = 0;   // tiles of the experts before x0
  for (int x0 = 0; x0 < E; x0 += 32) {
    const int x = x0 + lane;
    int a = 0, b = 0;
    if (x < E) {
      a = offsets[x];
      b = offsets[x + 1];
    }
    const bool bad = a < 0 || b < a || b > rows;
    if (__any_sync(all, bad)) {
      if (bad) set_status(status, MOE_ERR_BAD_INDEX, x);
      return false;
    }
    const int own = (b - a + TM - 1) / TM;
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(all, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned hit = __ballot_sync(all, tile < before + upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      e = x0 + l;
      row0 = __shfl_sync(all, a, l) + (tile - before - __shfl_sync(all, upto - own, l)) * TM;
      end = __shfl_sync(all, b, l);
      return true;
    }
    before += __shfl_sync(all, upto, 31);
  }
  return false;
}

// Steps of a product, with the next step's loads in flight: load(step) fills the
// registers, store(buffer) writes them to shared memory, multiply(buffer) takes
// the step.
template <int BUFS, typename Load, typename Store, typename Multiply>
__device__ __forceinline__ void run_steps(int steps, Load &&load, Store &&store,
                                          Multiply &&multiply) {
  if (steps > 0) load(0);
  for (int step = 0; step < steps; ++step) {
    const int buf = BUFS == 2 ? step & 1 : 0;
    if (BUFS == 1 && step > 0) __syncthreads();
    store(buf);
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
    multiply(buf);
  }
}

// T: the layer's type, TA: A's, TO: that of a gradient's outputs.
template <typename T, int EPI, bool B_ROWS, int TILE, typename TA = T, typename TO = T>
__global__ void __launch_bounds__(T_THREADS) rows_simt_kernel(RowsProduct p, int *status) {
  using G = Geo<TILE>;
  constexpr bool DUAL = EPI == kRowsSwiglu;
  // (three operands of deep steps: one buffer and a second barrier)
  constexpr int BUFS = DUAL && TILE == 32 ? 1 : 2;
  __shared__ __align__(16) typename G::Buf pool[(DUAL ? 3 : 2) * BUFS];
  typename G::Buf *as = pool, *bs = pool + BUFS, *b2s = pool + (DUAL ? 2 * BUFS : 0);
  static_assert(sizeof(pool) >= sizeof(float) * G::GROUPS * TILE * TILE || G::GROUPS == 1,
                "join_groups' scratch");
  pdl_wait();
  if (status_failed(status)) return;
  int e, row0, end;
  if (!find_tile<TILE>(p.offsets, p.num_experts, p.rows, blockIdx.x, e, row0, end, status)) return;
  const int n0 = blockIdx.y * TILE, N = p.N, K = p.K;
  const int64_t lda = p.lda ? p.lda : K;
  const Place<TILE> me;
  const int64_t base = (int64_t)e * N * K + (B_ROWS ? (int64_t)n0 : (int64_t)n0 * K);
  float2 acc[4][2] = {}, acc2[4][2] = {};
  // the steps of the one or two operand pairs, one after the other
  const int steps1 = (K + G::TK - 1) / G::TK;
  const int steps = steps1 * (EPI == kRowsPlain && p.A2 ? 2 : 1);
  Part<TA, true, TILE> pa;
  Part<T, true, TILE> pb2;
  Part<T, !B_ROWS, TILE> pb;
  // (a row's padding, lda > K, holds zeros and may be read)
  const int ka = p.lda ? p.lda : K;
  run_steps<BUFS>(
      steps,
      [&](int step) {
        const bool second = step >= steps1;
        const int k0 = (second ? step - steps1 : step) * G::TK;
        const TA *A = static_cast<const TA *>(second ? p.A2 : p.A) + row0 * lda;
        const T *B = static_cast<const T *>(second ? p.B2 : p.B) + base;
        pa.load(A + k0, lda, end - row0, ka - k0);
        pb.load(B_ROWS ? B + (int64_t)k0 * N : B + k0, B_ROWS ? N : K, N - n0, K - k0);
        if constexpr (DUAL)
          pb2.load(static_cast<const T *>(p.B2) + base + k0, K, N - n0, K - k0);
      },
      [&](int buf) {
        pa.store(as[buf]);
        pb.store(bs[buf]);
        if constexpr (DUAL) pb2.store(b2s[buf]);
      },
      [&](int buf) {
        tile_fma<TILE>(acc, as[buf], bs[buf], me.tx, me.ty, me.g);
        if constexpr (DUAL) tile_fma<TILE>(acc2, as[buf], b2s[buf], me.tx, me.ty, me.g);
      });
  // (the next kernel's CTAs, placed from the start, would share these SMs: 25 us
  // for the two products of the tiny layer's forward, 20 launched apart, 15.6 so)
  pdl_launch_dependents();
  join_groups<TILE>(acc, &pool[0][0][0], me.tx, me.ty, me.g);
  if constexpr (DUAL) join_groups<TILE>(acc2, &pool[0][0][0], me.tx, me.ty, me.g);
  const int c = n0 + me.col;   // (N is a multiple of 4)
  if (c >= N) return;
#pragma unroll
  for (int i = 0; i < Place<TILE>::ROWS; ++i) {
    const int r = row0 + me.row + i;
    if (r >= end) continue;
    const int64_t at = (int64_t)r * N + c;
    float v[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
    if constexpr (EPI == kRowsRelu) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = relu(v[j]);
    } else if constexpr (EPI == kRowsSwiglu) {
      const float u[4] = {acc2[i][0].x, acc2[i][0].y, acc2[i][1].x, acc2[i][1].y};
      put4<T>(p.out_g, at, v);
      put4<T>(p.out_u, at, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = v[j] / (1.f + expf(-v[j])) * u[j];
    } else if constexpr (EPI == kRowsReluGrad) {
      float h[4];
      get4<T>(p.h, at, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = h[j] > 0.f ? v[j] : 0.f;
    } else if constexpr (EPI == kRowsSwigluGrad) {
      float g[4], u[4], du[4];
      get4<T>(p.g, at, g);
      get4<T>(p.u, at, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = 1.f / (1.f + expf(-g[j]));
        du[j] = v[j] * g[j] * s;
        v[j] = v[j] * u[j] * s * (1.f + g[j] * (1.f - s));
      }
      put4<TO>(p.out_u, at, du);
    }
    if (EPI == kRowsPlain && p.add) {
      // the sum of this row's add_k other rows
      for (int j = 0; j < p.add_k; ++j) {
        const int q = p.add_inv[(int64_t)r * p.add_k + j];
        if (q < 0 || q >= p.rows * p.add_k) {
          if (c == 0) set_status(status, MOE_ERR_BAD_INDEX, r * p.add_k + j);
          continue;
        }
        float o[4];
        get4<T>(p.add, (int64_t)q * N + c, o);
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) v[i4] += o[i4];
      }
    }
    put4<TO>(p.out, at, v);
  }
}

// Problems over the same segments share a launch: CTA blockIdx.x takes a tile
// of an expert's gradients, blockIdx.y the expert, blockIdx.z a run of the
// segment's rows where these are cut (the outputs are then partial sums, the
// runs' matrices of an expert one after the other).
struct GradSet {
  GradProduct p[kMaxGradProblems];
  int first[kMaxGradProblems + 1];   // an expert's tiles before problem i
};
template <typename T, int TILE>
__global__ void __launch_bounds__(T_THREADS)
grad_simt_kernel(const __grid_constant__ GradSet set, int *status) {
  using G = Geo<TILE>;
  __shared__ __align__(16) typename G::Buf as[2], bs[2];
  static_assert(sizeof(as) >= sizeof(float) * G::GROUPS * TILE * TILE || G::GROUPS == 1,
                "join_groups' scratch");
  pdl_wait();
  if (status_failed(status)) return;
  int which = 0;
  while ((int)blockIdx.x >= set.first[which + 1]) ++which;
  const GradProduct &p = set.p[which];
  const int M = p.M, N = p.N, e = blockIdx.y;
  const int tile = blockIdx.x - set.first[which], across = (N + TILE - 1) / TILE;
  const int m0 = tile / across * TILE, n0 = tile % across * TILE;
  int beg = p.offsets ? p.offsets[e] : 0, end = p.offsets ? p.offsets[e + 1] : p.rows;
  if (beg < 0 || end < beg || end > p.rows) {
    if (threadIdx.x == 0) set_status(status, MOE_ERR_BAD_INDEX, e);
    return;
  }
  if (gridDim.z > 1) {
    const int run = (end - beg + (int)gridDim.z - 1) / (int)gridDim.z;
    beg = min(end, beg + (int)blockIdx.z * run);
    end = min(end, beg + run);
  }
  const int64_t lda = p.lda ? p.lda : M;
  const Place<TILE> me;
  float2 acc[4][2] = {};
  const T *B = static_cast<const T *>(p.B) + n0;
  auto sum = [&](const auto *A, auto &pa) {
    Part<T, false, TILE> pb;
    run_steps<2>(
        (end - beg + G::TK - 1) / G::TK,
        [&](int step) {
          const int q = beg + step * G::TK;
          pa.load(A + m0 + q * lda, lda, (int)lda - m0, end - q);
          pb.load(B + (int64_t)q * N, N, N - n0, end - q);
        },
        [&](int buf) {
          pa.store(as[buf]);
          pb.store(bs[buf]);
        },
        [&](int buf) { tile_fma<TILE>(acc, as[buf], bs[buf], me.tx, me.ty, me.g); });
  };
  if (sizeof(T) == 4 || p.a_f32) {
    Part<float, false, TILE> pa;
    sum(static_cast<const float *>(p.A), pa);
  } else {
    Part<T, false, TILE> pa;
    sum(static_cast<const T *>(p.A), pa);
  }
  pdl_launch_dependents();
  join_groups<TILE>(acc, &as[0][0][0], me.tx, me.ty, me.g);
  const int c = n0 + me.col;   // (N is a multiple of 4)
  if (c >= N) return;
#pragma unroll
  for (int i = 0; i < Place<TILE>::ROWS; ++i) {
    const int m = m0 + me.row + i;
    const float v[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
    if (m >= M) continue;
    const int64_t at = (((int64_t)e * gridDim.z + blockIdx.z) * M + m) * N + c;
    if (gridDim.z > 1) put4<float>(p.out, at, v);   // partial sums
    else put4<T>(p.out, at, v);
  }
}

// out[i] = sum over the runs of part[run][i], in order.
struct GradSum {
  const float *part[kMaxGradProblems];
  void *out[kMaxGradProblems];
  int64_t per_expert[kMaxGradProblems];   // M * N (a multiple of 4)
  int experts, splits;
  int *status;
};
template <typename T>
__global__ void __launch_bounds__(256) simt_sum_kernel(const __grid_constant__ GradSum a) {
  pdl_wait();
  if (status_failed(a.status)) return;
  const int p = blockIdx.y;
  const int64_t per = a.per_expert[p], total = per * a.experts;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < total;
       i += (int64_t)gridDim.x * 1024) {
    const int64_t e = i / per;
    const float *src = a.part[p] + e * a.splits * per + (i - e * per);
    float x[4] = {};
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) {
      const float4 u = load4(src + s * per);
      x[0] += u.x;
      x[1] += u.y;
      x[2] += u.z;
      x[3] += u.w;
    }
    put4<T>(a.out[p], i, x);
  }
}

template <typename T, int TILE>
cudaError_t launch_rows(const RowsProduct &p, int *status, cudaStream_t s) {
  const int mt = (p.rows + TILE - 1) / TILE + (p.offsets ? p.num_experts : 0);
  const dim3 grid(mt, (p.N + TILE - 1) / TILE);
  if constexpr (sizeof(T) == 2) {
    // (fp32 dg, du and dl)
    auto wide = p.a_f32 ? rows_simt_kernel<T, kRowsPlain, true, TILE, float>
                : p.epi == kRowsReluGrad ? rows_simt_kernel<T, kRowsReluGrad, true, TILE, T, float>
                                         : rows_simt_kernel<T, kRowsSwigluGrad, true, TILE, T, float>;
    if (p.a_f32 || p.out_f32) return launch_pdl(wide, grid, dim3(T_THREADS), 0, s, p, status);
  }
  auto with = p.epi == kRowsPlain && p.b_rows ? rows_simt_kernel<T, kRowsPlain, true, TILE>
              : p.epi == kRowsPlain           ? rows_simt_kernel<T, kRowsPlain, false, TILE>
              : p.epi == kRowsRelu            ? rows_simt_kernel<T, kRowsRelu, false, TILE>
              : p.epi == kRowsSwiglu          ? rows_simt_kernel<T, kRowsSwiglu, false, TILE>
              : p.epi == kRowsReluGrad        ? rows_simt_kernel<T, kRowsReluGrad, true, TILE>
                                              : rows_simt_kernel<T, kRowsSwigluGrad, true, TILE>;
  return launch_pdl(with, grid, dim3(T_THREADS), 0, s, p, status);
}

// Whether this many 64 x 64 tiles give each SM one.
bool large_tiles(int64_t tiles) { return tiles >= num_sms(); }

}  // namespace

cudaError_t launch_rows_simt(const RowsProduct &p, int *status, cudaStream_t s) {
  if (p.dtype == MOE_BF16) return launch_rows<__nv_bfloat16, 32>(p, status, s);
  return large_tiles((int64_t)((p.rows + 63) / 64) * ((p.N + 63) / 64))
             ? launch_rows<float, 64>(p, status, s)
             : launch_rows<float, 32>(p, status, s);
}

// bf16 gradients take the pair kernel where it is the faster.  CUDA cores / pair
// kernel, a backward pass in us.  Of a router: 53 rows, d 80, 3 experts 7 / 10;
// 2048 rows, d 256, 32 experts 14 / 16; 16384 rows, d 128, 8 experts 40 / 40.  Of
// expert FFNs: 1024 rows of 8 experts, d = d_ff = 128 23 / 35; at d = d_ff = 64, 2000
// rows of 2 18 / 17, 4000 of one 23 / 20.
bool grads_small(const GradProduct *p, int count) {
  if (count == 0 || p[0].dtype == MOE_F32) return true;
  const int E = p[0].offsets ? p[0].num_experts : 1;
  if (p[0].offsets && p[0].rows / E > 256) return false;
  for (int i = 0; i < count; ++i)
    if ((int64_t)p[i].rows * p[i].M * p[i].N > kSmallProducts ||
        (int64_t)E * p[i].M * p[i].N > 1 << 19)   // (else storing it is the work)
      return false;
  return true;
}

// Tiles that leave most SMs without work have their rows cut into runs of 256
// at least, with partial sums and a launch that adds them in order.  Whole / cut,
// a backward pass in us, fp32: a router of 2048 rows, d 16, 180 experts 34 / 19;
// of 16384 rows, d 128, 8 experts 185 / 38; FFNs with d = d_ff = 64, 4000 rows of
// one expert 50 / 23.  Runs of 128 lost the added launch: 256 rows, d 128, 4
// experts 12.5 / 15.6.
int grad_splits_simt(const GradProduct *p, int count) {
  if (count == 0) return 1;
  const int E = p[0].offsets ? p[0].num_experts : 1;
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i)
    tiles += (int64_t)E * ((p[i].N + 31) / 32) * ((p[i].M + 31) / 32);
  const int64_t most = 152 / tiles, by_rows = p[0].rows / E / 256;
  const int64_t n = most < by_rows ? most : by_rows;
  return n < 2 ? 1 : (int)n;
}

cudaError_t launch_grad_simt(const GradProduct *p, int count, int splits, float *parts, int *status,
                             cudaStream_t s) {
  const int E = p[0].offsets ? p[0].num_experts : 1;
  GradSet set{};
  auto lay = [&](int tile) {
    for (int i = 0; i < kMaxGradProblems; ++i) {
      const int tiles = i < count ? ((p[i].N + tile - 1) / tile) * ((p[i].M + tile - 1) / tile) : 0;
      if (i < count) set.p[i] = p[i];
      set.first[i + 1] = set.first[i] + tiles;
    }
    return set.first[count];
  };
  const bool bf16 = p[0].dtype == MOE_BF16, large = !bf16 && large_tiles((int64_t)lay(64) * E);
  const dim3 grid(lay(large ? 64 : 32), E, splits);
  GradSum sum{};
  int64_t most = 0;
  if (splits > 1) {
    for (int i = 0; i < count; ++i) {
      const int64_t per = (int64_t)p[i].M * p[i].N;
      sum.part[i] = parts;
      sum.out[i] = p[i].out;
      sum.per_expert[i] = per;
      set.p[i].out = parts;
      parts += per * E * splits;
      if (per * E > most) most = per * E;
    }
    sum.experts = E;
    sum.splits = splits;
    sum.status = status;
  }
  auto with = bf16    ? grad_simt_kernel<__nv_bfloat16, 32>
              : large ? grad_simt_kernel<float, 64>
                      : grad_simt_kernel<float, 32>;
  const cudaError_t e = launch_pdl(with, grid, dim3(T_THREADS), 0, s, set, status);
  if (e != cudaSuccess || splits == 1) return e;
  const int64_t blocks = (most / 4 + 255) / 256;
  return launch_pdl(bf16 ? simt_sum_kernel<__nv_bfloat16> : simt_sum_kernel<float>,
                    dim3((unsigned)(blocks < 608 ? blocks : 608), count), dim3(256), 0, s, sum);
}

}  // namespace moe
