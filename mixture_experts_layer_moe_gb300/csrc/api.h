// What the C entry points share: argument checks, the layer's workspace layout
// and status conversion (internal; the public ABI is moe.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#define MOE_TRY(expr)                   \
  do {                                  \
    const moe_status _st = (expr);      \
    if (_st != MOE_OK) return _st;      \
  } while (0)

namespace moe {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool ok_ptr(const void *p) { return p != nullptr && aligned(p, 16); }
inline cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }
inline int act_size(const moe_config &c) { return c.act_dtype == MOE_F32 ? 4 : 2; }
inline int h_size(const moe_config &c) { return c.act_dtype == MOE_F32 ? 4 : 2; }
inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

template <typename T>
T *at(void *ws, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(ws) + off);
}

struct Layout {
  size_t status, route_count, sync, logits, topk_idx, topk_gate, counts, offsets, perm, inv_perm,
      x_perm, h, y_perm, y_shared, h_shared, act16, total;
};

moe_status check_config(const moe_config *c);
moe_status check_router_weights(const moe_config &c, const moe_weights *w);
moe_status check_expert_weights(const moe_config &c, const moe_weights *w);
Layout layout_of(const moe_config &c);

}  // namespace moe
