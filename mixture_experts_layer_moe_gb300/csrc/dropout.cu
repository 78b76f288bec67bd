// Dropout of rows: y = x / (1 - q) where element (r, c) is kept, else 0.  A stream
// through HBM: the mask is made from the element's place (philox.cuh), eight
// elements per call of the generator, and never stored.
//
// A thread takes blocks of eight elements, a grid's stride apart (their row and
// place move on by a constant: no division per block), and loads U of them
// before it makes the masks of the first.
#include "common.cuh"
#include "fp32x2.cuh"
#include "launch.h"
#include "philox.cuh"
#include "step.h"
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int D_THREADS = 256;
// Rows this wide at least go by pieces (16384 x 1001: 27 us so, 25 by elements).
constexpr int D_PIECES = 2048;

// A block of eight elements as 16-byte vectors.
template <typename T>
struct Block8 {
  static constexpr int N = 8 * sizeof(T) / 16;
  uint4 v[N];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void store(T *p) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<uint4 *>(p)[i] = v[i];
  }
  __device__ __forceinline__ void drop(const uint4 &bits, uint32_t cut, float factor) {
    const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      constexpr int E = Vec16<T>::N;
      float f[E];
      unpack16<T>(v[i], f);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 g = mul2(make_float2(f[e], f[e + 1]), both(factor));
        f[e] = kept_even(w[(i * E + e) / 2], cut) ? g.x : 0.f;
        f[e + 1] = kept_odd(w[(i * E + e) / 2], cut) ? g.y : 0.f;
      }
      v[i] = pack16<T>(f);
    }
  }
};

struct DropArgs {
  moe_dropout_config c;
  const RngState *rng;
  int threshold, blocks;    // blocks of a row
  float factor;
  int64_t step_rows;        // a grid's stride: rows, and blocks of the last one
  int step_blocks;
};

// Rows on vector boundaries (x and y may be the same).
template <typename T, int U>
__global__ void __launch_bounds__(D_THREADS) dropout_kernel(const __grid_constant__ DropArgs a,
                                                            const T *x, T *y) {
  const moe_dropout_config &c = a.c;
  const RngState st = load_state(a.threshold ? a.rng : nullptr);
  const int64_t start = (int64_t)blockIdx.x * D_THREADS + threadIdx.x;
  int64_t r = start / a.blocks;
  int k = (int)(start - r * a.blocks);
  while (r < c.rows) {
    Block8<T> v[U];
    int64_t row[U];
    int at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      row[u] = r;
      at[u] = k;
      if (r < c.rows && k * 8 + 8 <= c.d) v[u].load(x + r * c.ldx + k * 8);
      r += a.step_rows;
      k += a.step_blocks;
      if (k >= a.blocks) {
        k -= a.blocks;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row[u] >= c.rows) break;
      T *to = y + row[u] * c.ldy + at[u] * 8;
      if (at[u] * 8 + 8 <= c.d) {
        v[u].drop(dropout_bits(st, at[u], (uint32_t)row[u]), (uint32_t)a.threshold << 16, a.factor);
        v[u].store(to);
      } else {
        const uint32_t keep = dropout_keep(st, at[u], (uint32_t)row[u], a.threshold);
        const T *from = x + row[u] * c.ldx + at[u] * 8;
        for (int i = 0; i < c.d - at[u] * 8; ++i)
          to[i] = Elem<T>::from_f(keep >> i & 1 ? Elem<T>::load(from + i) * a.factor : 0.f);
      }
    }
  }
}

// bf16 rows anywhere whose elements lie alike in x and y (a row starts h elements into
// an aligned piece of eight in both): by pieces.  Lanes 1-31 of a warp take 31
// neighbouring pieces; a piece's elements are the last h of one block and the first 8
// - h of the next, whose masks the lane and the one before it make.  (16383 x 7167 141 us
// by single elements, 107 so.)
__global__ void __launch_bounds__(D_THREADS)
dropout_pieces_kernel(const __grid_constant__ DropArgs a, const __nv_bfloat16 *x, __nv_bfloat16 *y) {
  using T = __nv_bfloat16;
  const moe_dropout_config &c = a.c;
  const RngState st = load_state(a.threshold ? a.rng : nullptr);
  const int lane = threadIdx.x & 31;
  const int64_t start = (int64_t)blockIdx.x * (D_THREADS / 32) + (threadIdx.x >> 5);
  int64_t r = start / a.blocks;   // (here blocks of 31 pieces, one per warp)
  int k = (int)(start - r * a.blocks);
  constexpr int U = 2;
  while (r < c.rows) {
    uint4 v[U];
    int64_t at[U];
    int piece[U], e0[U], h[U];
    bool whole[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = r;
      const T *row = x + r * c.ldx;
      h[u] = (int)(reinterpret_cast<uintptr_t>(row) & 15) / 2;
      piece[u] = 31 * k + lane - 1;
      e0[u] = piece[u] * 8 - h[u];
      whole[u] = r < c.rows && lane > 0 && e0[u] >= 0 && e0[u] + 8 <= c.d;
      if (whole[u]) v[u] = *reinterpret_cast<const uint4 *>(row + e0[u]);
      r += a.step_rows;
      k += a.step_blocks;
      if (k >= a.blocks) {
        k -= a.blocks;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] >= c.rows) break;
      const uint32_t own = dropout_keep(st, max(piece[u], 0), (uint32_t)at[u], a.threshold);
      const uint32_t before = __shfl_up_sync(0xffffffffu, own, 1);
      const uint32_t keep = (before | own << 8) >> (8 - h[u]);
      T *to = y + at[u] * c.ldy + e0[u];
      if (whole[u]) {
        float f[8];
        unpack16<T>(v[u], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = keep >> i & 1 ? f[i] * a.factor : 0.f;
        *reinterpret_cast<uint4 *>(to) = pack16<T>(f);
      } else if (lane > 0) {
        const T *from = x + at[u] * c.ldx + e0[u];
        for (int i = max(0, -e0[u]); i < min(8, c.d - e0[u]); ++i)
          to[i] = Elem<T>::from_f(keep >> i & 1 ? Elem<T>::load(from + i) * a.factor : 0.f);
      }
    }
  }
}

// Rows anywhere: a warp takes 256 columns of a row, a lane makes the mask of a
// block, and the elements go by lanes.
template <typename T>
__global__ void __launch_bounds__(D_THREADS) dropout_odd_kernel(const __grid_constant__ DropArgs a,
                                                                const T *x, T *y) {
  const moe_dropout_config &c = a.c;
  const RngState st = load_state(a.threshold ? a.rng : nullptr);
  const int lane = threadIdx.x & 31;
  const int64_t start = (int64_t)blockIdx.x * (D_THREADS / 32) + (threadIdx.x >> 5);
  int64_t r = start / a.blocks;   // (here blocks of 256 columns, one per warp)
  int k = (int)(start - r * a.blocks);
  while (r < c.rows) {
    const T *from = x + r * c.ldx;
    T *to = y + r * c.ldy;
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = k * 256 + i * 32 + lane;
      if (col < c.d) v[i] = from[col];
    }
    const uint32_t keep = dropout_keep(st, k * 32 + lane, (uint32_t)r, a.threshold);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = k * 256 + i * 32 + lane;
      const uint32_t mask = __shfl_sync(0xffffffffu, keep, i * 4 + (lane >> 3));
      if (col < c.d)
        to[col] = Elem<T>::from_f(mask >> (lane & 7) & 1 ? Elem<T>::to_f(v[i]) * a.factor : 0.f);
    }
    r += a.step_rows;
    k += a.step_blocks;
    if (k >= a.blocks) {
      k -= a.blocks;
      ++r;
    }
  }
}

template <typename T>
cudaError_t launch(const moe_dropout_config &c, int threshold, const T *x, const RngState *rng,
                   T *y, cudaStream_t s) {
  constexpr int U = 16 / (int)sizeof(T) / 2;   // (bf16 4, fp32 2: 64 bytes a thread)
  constexpr int E = Vec16<T>::N;
  DropArgs a{c, rng, threshold, 0, dropout_factor(threshold), 0, 0};
  const bool vectors = c.rows == 1 || (c.ldx % E == 0 && c.ldy % E == 0);
  const bool pieces =
      !vectors && sizeof(T) == 2 && (c.ldx - c.ldy) % 8 == 0 && c.d >= D_PIECES;
  a.blocks = vectors ? (c.d + 7) / 8 : pieces ? ((c.d + 14) / 8 + 30) / 31 : (c.d + 255) / 256;
  const int per = vectors ? D_THREADS : D_THREADS / 32;
  const int64_t want = (c.rows * a.blocks + per - 1) / per, most = (int64_t)num_sms() * 8;
  const int64_t grid = want < most ? want : most;
  a.step_rows = grid * per / a.blocks;
  a.step_blocks = (int)(grid * per - a.step_rows * a.blocks);
  if (vectors) dropout_kernel<T, U><<<(unsigned)grid, D_THREADS, 0, s>>>(a, x, y);
  else if (pieces)
    dropout_pieces_kernel<<<(unsigned)grid, D_THREADS, 0, s>>>(a, (const __nv_bfloat16 *)x,
                                                               (__nv_bfloat16 *)y);
  else dropout_odd_kernel<T><<<(unsigned)grid, D_THREADS, 0, s>>>(a, x, y);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(const moe_dropout_config &c, int threshold, const void *x,
                           const uint64_t *rng, void *y, cudaStream_t s) {
  const RngState *st = reinterpret_cast<const RngState *>(rng);
  return c.dtype == MOE_F32
             ? launch<float>(c, threshold, (const float *)x, st, (float *)y, s)
             : launch<__nv_bfloat16>(c, threshold, (const __nv_bfloat16 *)x, st, (__nv_bfloat16 *)y, s);
}

}  // namespace moe
