// Host-side launchers of the operators round the layer in a training step
// (internal; the public ABI is moe.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

cudaError_t launch_dropout(const moe_dropout_config &c, int threshold, const void *x,
                           const uint64_t *rng, void *y, cudaStream_t s);

// ------------------------------------------------------------ block joint
struct JoinForward {
  const void *x, *b;
  moe_join_params w;
  const uint64_t *rng;
  void *r, *y;
  float *stats;
};
struct JoinBackward {
  const void *b, *r;
  const float *stats;
  moe_join_params w;
  const uint64_t *rng;
  const void *dr, *dy;
  void *dx, *db;
  moe_join_grads grads;
};
cudaError_t launch_join(const moe_join_config &c, int threshold, const JoinForward &f,
                        cudaStream_t s);
size_t join_backward_scratch(const moe_join_config &c);
cudaError_t launch_join_backward(const moe_join_config &c, int threshold, const JoinBackward &f,
                                 void *scratch, cudaStream_t s);

// ------------------------------------------------------------------- loss
size_t loss_workspace(const moe_loss_config &c);
cudaError_t launch_loss(const moe_loss_config &c, const void *x, const void *W,
                        const int32_t *targets, float *loss, float *lse, void *ws, cudaStream_t s);
cudaError_t launch_loss_backward(const moe_loss_config &c, const void *x, const void *W,
                                 const int32_t *targets, const float *lse, const float *dloss,
                                 void *dx, void *dW, void *ws, cudaStream_t s);

}  // namespace moe
