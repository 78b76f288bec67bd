// What the kernels that walk rows (norms, the block joint) share: how a thread's
// share of a row is cut, asynchronous copies of rows, sums over the threads of a
// row.
#pragma once

#include "common.cuh"
#include "vec16.cuh"

namespace moe {

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

}  // namespace moe
