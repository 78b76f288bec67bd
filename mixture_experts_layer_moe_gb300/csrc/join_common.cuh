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

constexpr int J_THREADS = 512;
constexpr int J_SMEM = 208 * 1024;   // dynamic shared memory of a CTA at most
constexpr int J_WIDE = 512;          // threads of the kernels for rows of any width

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

// ---- rows of whole vectors: a thread owns NB blocks of eight columns, which are
// what one call of the generator covers
struct Block8 {
  float2 v[4];
};
__device__ __forceinline__ Block8 fill8(float a) { return Block8{both(a), both(a), both(a), both(a)}; }

// A thread's vectors lie a fixed distance apart in the ring, whatever the CTA's size (this
// one holds up to 512 threads): the offsets of a stage's vectors are constants then (with distances that go by
// the number of threads the gradient's kernel spent a fifth of its instructions
// on them).
constexpr int V8_PIECE = J_THREADS * 16;
template <typename T>
struct Vec8 {
  static constexpr int Q = 8 * sizeof(T) / 16;   // 16-byte vectors of a block
  static __device__ __forceinline__ Block8 unpack(const uint4 (&raw)[Q]) {
    Block8 b;
#pragma unroll
    for (int q = 0; q < Q; ++q) unpack16<T>(raw[q], reinterpret_cast<float *>(b.v) + q * 8 / Q);
    return b;
  }
  // block number `block` of a stage of the ring, whose first vector of this thread is `at`
  template <int PIECE>
  static __device__ __forceinline__ Block8 ring(const uint8_t *at, int block) {
    uint4 raw[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q)
      raw[q] = *reinterpret_cast<const uint4 *>(at + (block * Q + q) * PIECE);
    return unpack(raw);
  }
  template <int PIECE>
  static __device__ __forceinline__ void copy(uint8_t *at, int block, const char *from) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      copy16_async(reinterpret_cast<uint4 *>(at + (block * Q + q) * PIECE), from + q * 16);
  }
  static __device__ __forceinline__ void store(char *to, const Block8 &b) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      reinterpret_cast<uint4 *>(to)[q] = pack16<T>(reinterpret_cast<const float *>(b.v) + q * 8 / Q);
  }
  // a vector of parameters, or `other` where there is none
  static __device__ __forceinline__ Block8 param(const T *v, int col, float other) {
    if (v == nullptr) return fill8(other);
    uint4 raw[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) raw[q] = reinterpret_cast<const uint4 *>(v + col)[q];
    return unpack(raw);
  }
};

// Zero where the eight elements of a block are dropped.
__device__ __forceinline__ void drop8(Block8 &b, const uint4 &bits, uint32_t cut) {
  const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    b.v[h].x = kept_even(w[h], cut) ? b.v[h].x : 0.f;
    b.v[h].y = kept_odd(w[h], cut) ? b.v[h].y : 0.f;
  }
}

// ---- other rows: [stage][group][tensor] slots of whole rows, a thread's share in
// pairs of elements tpr apart, sixteen elements in all
template <typename T>
struct Ring {
  using C = Chunk<T, 1>;
  static constexpr int NC = 8;
  uint8_t *base;
  int tid, tpr, group, groups, tensors, d, slot;

  __device__ __forceinline__ int col(int i) const { return tid + 2 * i * tpr; }
  __device__ __forceinline__ uint8_t *row(int stage, int t) const {
    return base + (int64_t)((stage * groups + group) * tensors + t) * slot;
  }
  __device__ __forceinline__ void copy(int stage, int t, const T *src, const T *end) const {
    copy_row(row(stage, t), src, d, end, tid, tpr);
  }
  // pair i of tensor t, whose row src was copied
  __device__ __forceinline__ void get(int stage, int i, int t, const T *src, float2 *p) const {
    C::load(reinterpret_cast<const T *>(row(stage, t) + head_of(src)), col(i), tpr, d, p);
  }
};

// A row's dropout mask as bytes in shared memory (read after the group's next
// barrier).
__host__ __device__ constexpr int mask_bytes(int d) { return ((d + 7) / 8 + 15) / 16 * 16; }
template <typename T>
__device__ __forceinline__ void make_masks(const Ring<T> &ring, const RngState &st, uint32_t row,
                                           int threshold, uint8_t *masks) {
  for (int k = ring.tid; k < (ring.d + 7) / 8; k += ring.tpr)
    masks[k] = (uint8_t)dropout_keep(st, k, row, threshold);
}
// Both elements of pair i: kept ones times factor, others 0.
template <typename T>
__device__ __forceinline__ float2 drop_pair(const Ring<T> &ring, const uint8_t *masks, int i,
                                            float2 v, float factor) {
  const int c0 = ring.col(i), c1 = c0 + ring.tpr;
  const bool x = masks[c0 >> 3] >> (c0 & 7) & 1;
  const bool y = c1 < ring.d && (masks[c1 >> 3] >> (c1 & 7) & 1);
  v = mul2(v, both(factor));
  return make_float2(x ? v.x : 0.f, y ? v.y : 0.f);
}

// Pair i of a vector of d parameters, or `other` where there is none.
template <typename T>
__device__ __forceinline__ void params(const Ring<T> &ring, const T *v, int i, float other,
                                       float2 (&p)[1]) {
  p[0] = both(other);
  if (v) Chunk<T, 1>::load(v, ring.col(i), ring.tpr, ring.d, p);
}

inline int64_t grid_of(int64_t rows, int groups, int64_t most) {
  const int64_t want = (rows + groups - 1) / groups;
  return want < most ? want : most;
}

// Threads per row for rows of d elements, `each` per thread (0: wider than a CTA
// holds).
inline int threads_of(int d, int each) {
  const int64_t per_warp = (int64_t)32 * each, warps = (d + per_warp - 1) / per_warp;
  return warps * 32 <= J_THREADS ? (int)warps * 32 : 0;
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
