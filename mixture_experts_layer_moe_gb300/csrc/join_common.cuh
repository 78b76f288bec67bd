// What the block joint's two directions share: rows held in a ring in shared memory,
// the dropout of a thread's share of a row, launch shapes.
#pragma once

#include <initializer_list>

#include "common.cuh"
#include "fp32x2.cuh"
#include "launch.h"
#include "philox.cuh"
#include "rows_common.cuh"
#include "step.h"

namespace moe {
namespace join {

constexpr int J_THREADS = 512;       // threads of a CTA at most
constexpr int J_SMEM = 226 * 1024;   // dynamic shared memory of a CTA at most
constexpr int J_WIDE = 512;          // threads of the kernels for rows of any width
constexpr int J_MAX_D = 16 * J_THREADS;   // the widest row that a ring's CTA holds

template <typename T>
__device__ __forceinline__ float at_or(const T *v, int i, float other) {
  return v ? Elem<T>::load(v + i) : other;
}

// Waits until at most `ahead` of this thread's groups of copies are in flight.
__device__ __forceinline__ void copies_wait(int ahead) {
  if (ahead >= 2) copy_wait<2>();
  else if (ahead == 1) copy_wait<1>();
  else copy_wait<0>();
}

// Sums over a group of threads, a warp or several (in a CTA all groups are alike).
__device__ __forceinline__ float row_sum(float a, float2 (*buf)[32], int &turn, int warps) {
  float (*one)[32] = reinterpret_cast<float (*)[32]>(buf);
  return warps == 1 ? group_sum<true>(a, one, turn, 1) : group_sum<false>(a, one, turn, warps);
}
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 (*buf)[32], int &turn,
                                           int first, int warps) {
  return warps == 1 ? group_sum2<true>(a, b, buf, turn, first, 1)
                    : group_sum2<false>(a, b, buf, turn, first, warps);
}

// ---- A thread owns blocks of eight neighbouring columns, which are what one call of
// the generator covers.
struct Block8 {
  float2 v[4];
};
__device__ __forceinline__ Block8 fill8(float a) { return Block8{both(a), both(a), both(a), both(a)}; }

// Zero where the eight elements of a block are dropped.
__device__ __forceinline__ void drop8(Block8 &b, const uint4 &bits, uint32_t cut) {
  const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    b.v[h].x = kept_even(w[h], cut) ? b.v[h].x : 0.f;
    b.v[h].y = kept_odd(w[h], cut) ? b.v[h].y : 0.f;
  }
}
// Zero from element `valid` on.
__device__ __forceinline__ void mask8(Block8 &b, int valid) {
  if (valid >= 8) return;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    if (2 * h >= valid) b.v[h].x = 0.f;
    if (2 * h + 1 >= valid) b.v[h].y = 0.f;
  }
}

// Blocks of rows in shared memory, for a CTA of up to THREADS threads.  A block's Q
// vectors of 16 bytes lie at fixed distances, whatever the CTA's size, so that
// they are offsets in the instructions (with distances that go by the number of
// threads the gradient's kernel spent a fifth of its instructions on them).
//
// ODD: rows that start anywhere.  A warp copies the aligned pieces that cover its 256
// columns (one more than they fill), and realign() moves each thread's elements to
// the place where it then reads them as vectors; store() goes through the thread's
// place too, to write neighbouring elements from neighbouring lanes.  All of it
// stays within the warp.  Copies end with the row: what lies behind it reads as
// zero.  fp32 rows take this way too where they are whole vectors: a thread's two
// vectors copied by itself leave each request half of its sectors (8192 x 7168
// forward 235 us, 180 so).
template <typename T, int THREADS, bool ODD>
struct Blocks {
  static constexpr int Q = 8 * sizeof(T) / 16;
  static constexpr int WIDTH = 8 * sizeof(T);                   // bytes of a block
  static constexpr int WARP = ODD ? (32 * Q + 1) * 16 : 512;    // bytes of a warp (ODD: all vectors)
  static constexpr int STEP = ODD ? 16 : THREADS * 16;          // from a vector to the next
  static constexpr int BYTES = ODD ? THREADS / 32 * WARP : Q * STEP;

  // where this thread's first vector of the first block lies
  static __device__ __forceinline__ int place() {
    return (threadIdx.x >> 5) * WARP + (threadIdx.x & 31) * (ODD ? WIDTH : 16);
  }
  // copies the block at `from`, of whose row `left` bytes follow (vectors: the block is there)
  static __device__ __forceinline__ void copy(uint8_t *at, const char *from, int left) {
    if constexpr (!ODD) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
        copy16_async(reinterpret_cast<uint4 *>(at + q * STEP), from + q * 16);
    } else {
      const int lane = threadIdx.x & 31;
      at -= lane * WIDTH;
      from -= lane * WIDTH;
      const int head = (int)(reinterpret_cast<uintptr_t>(from) & 15);
      from -= head;
      left += lane * WIDTH + head;
#pragma unroll
      for (int q = 0; q <= Q; ++q) {
        if (q == Q && lane != 0) break;
        const int off = (lane + q * 32) * 16, n = min(max(left - off, 0), 16);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(at + off))),
                     "l"(from + (n ? off : 0)), "r"(n)
                     : "memory");
      }
    }
  }
  // ODD: the block of a row that starts `head` bytes into a piece.  (All copies have
  // landed, and the warp has met since.)
  static __device__ __forceinline__ void realign(uint8_t *at, int head) {
    if (head == 0) return;   // (one for the warp)
    constexpr int N = 4 * (Q + 1);
    uint32_t w[N];
#pragma unroll
    for (int q = 0; q <= Q; ++q)
      *reinterpret_cast<uint4 *>(w + 4 * q) = *reinterpret_cast<const uint4 *>(at + q * 16);
    __syncwarp();
    if (head & 8) {
#pragma unroll
      for (int i = 0; i + 2 < N; ++i) w[i] = w[i + 2];
    }
    if (head & 4) {
#pragma unroll
      for (int i = 0; i + 1 < N; ++i) w[i] = w[i + 1];
    }
    if (sizeof(T) == 2 && (head & 2)) {
#pragma unroll
      for (int i = 0; i < 4 * Q; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
      *reinterpret_cast<uint4 *>(at + q * 16) = *reinterpret_cast<const uint4 *>(w + 4 * q);
  }
  static __device__ __forceinline__ Block8 load(const uint8_t *at) {
    Block8 b;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      unpack16<T>(*reinterpret_cast<const uint4 *>(at + q * STEP),
                  reinterpret_cast<float *>(b.v) + q * 8 / Q);
    return b;
  }
  // stores a block to `to`; ODD: through the place `at`, which nothing else needs any
  // more before the warp next meets
  static __device__ __forceinline__ void store(uint8_t *at, char *to, int left, const Block8 &b) {
    uint4 raw[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
      raw[q] = pack16<T>(reinterpret_cast<const float *>(b.v) + q * 8 / Q);
    if constexpr (!ODD) {
#pragma unroll
      for (int q = 0; q < Q; ++q) reinterpret_cast<uint4 *>(to)[q] = raw[q];
    } else {
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int q = 0; q < Q; ++q) *reinterpret_cast<uint4 *>(at + q * 16) = raw[q];
      __syncwarp();
      at -= lane * WIDTH;
      to -= lane * WIDTH;
      left += lane * WIDTH;
      if ((reinterpret_cast<uintptr_t>(to) & 15) == 0 && left % 16 == 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int off = (q * 32 + lane) * 16;
          if (off < left)
            *reinterpret_cast<uint4 *>(to + off) = *reinterpret_cast<const uint4 *>(at + off);
        }
      } else if (sizeof(T) == 4 || (reinterpret_cast<uintptr_t>(to) & 3) == 0) {
#pragma unroll
        for (int i = 0; i < 8 * (int)sizeof(T) / 4; ++i) {
          const int off = (i * 32 + lane) * 4;
          if (off + 4 <= left)
            *reinterpret_cast<uint32_t *>(to + off) = *reinterpret_cast<const uint32_t *>(at + off);
          else if (off < left)   // (one element of two bytes)
            *reinterpret_cast<uint16_t *>(to + off) = *reinterpret_cast<const uint16_t *>(at + off);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int off = (i * 32 + lane) * 2;
          if (off < left)
            *reinterpret_cast<uint16_t *>(to + off) = *reinterpret_cast<const uint16_t *>(at + off);
        }
      }
    }
  }
};

// The first `valid` elements of a vector of parameters from column col on, then zeros;
// `other` where there is no vector.
template <typename T>
__device__ __forceinline__ Block8 param8(const T *v, int col, int valid, float other) {
  Block8 b = fill8(0.f);
  float *f = reinterpret_cast<float *>(b.v);
  if (v == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < valid ? other : 0.f;
  } else if (valid == 8) {
    constexpr int Q = 8 * sizeof(T) / 16;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      unpack16<T>(reinterpret_cast<const uint4 *>(v + col)[q], f + q * 8 / Q);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) f[i] = Elem<T>::load(v + col + i);
  }
  return b;
}

// Eight floats of this thread in shared memory (THREADS * 32 bytes in all).
template <int THREADS>
struct Own8 {
  static constexpr int BYTES = THREADS * 32;
  uint8_t *at;
  __device__ __forceinline__ explicit Own8(uint8_t *base) : at(base + threadIdx.x * 16) {}
  __device__ __forceinline__ Block8 get() const {
    Block8 b;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      reinterpret_cast<float4 *>(b.v)[q] = *reinterpret_cast<const float4 *>(at + q * THREADS * 16);
    return b;
  }
  __device__ __forceinline__ void set(const Block8 &b) const {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<float4 *>(at + q * THREADS * 16) = reinterpret_cast<const float4 *>(b.v)[q];
  }
};

inline int64_t grid_of(int64_t rows, int groups, int64_t most) {
  const int64_t want = (rows + groups - 1) / groups;
  return want < most ? want : most;
}

// Threads of a row of d columns, NB blocks each (whole warps).
inline int threads_of(int d, int NB) { return (d + 256 * NB - 1) / (256 * NB) * 32; }

// Groups of tpr threads in a CTA of up to `threads`, fewer where there are SMs to
// spare; each takes `rows_each` rows at a time.
inline int groups_of(int64_t rows, int rows_each, int tpr, int threads, int sms) {
  int groups = tpr < threads ? threads / tpr : 1;
  while (groups > 1 && rows <= (int64_t)(groups / 2) * rows_each * sms) groups /= 2;
  return groups;
}

// Stages of a ring that fits beside `other` bytes.
__host__ __device__ constexpr int stages_of(size_t stage, size_t other) {
  int stages = 3;
  while (stages > 1 && stages * stage + other > (size_t)J_SMEM) --stages;
  return stages;
}

// Whether rows this far apart start on a vector.
template <typename T>
bool whole_vectors(const moe_join_config &c, std::initializer_list<int64_t> lds) {
  if (c.d % 8 != 0) return false;
  for (int64_t ld : lds)
    if (c.rows > 1 && ld % Vec16<T>::N != 0) return false;
  return true;
}

}  // namespace join
}  // namespace moe
