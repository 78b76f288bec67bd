// The tensor-core products of the cross entropy (loss_pair.cu), for loss.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// Tokens are rows [n][d] of which the first range[1] count (read on the device; all
// without a range);
// `entries` of the vocabulary from v0 on, W their rows [entries][d].
struct LossProduct {
  int n, d, entries, v0;
  const int32_t *range, *target;
  const void *x, *W;
  // sums: (maximum, sum of e^(l - maximum)) per token and half of a tile,
  // [n][chunks], and the target's logit
  float2 *sums;
  int width, chunks;      // entries per tile
  float *at;
  // the logits' gradient divided by *scale, bf16 [n][pitch], columns from `entries` on
  // zero; dx is left divided by it too, dW is not
  const float *lse, *dloss, *scale;
  float z_loss;
  void *dl;
  int pitch;
  // dx in fp32: `splits` ranges of the entries, planes [split][n][d]; added to
  // what they hold, or stored
  float *planes;
  int splits, add;
};

bool loss_pair_supported(const moe_loss_config &c);   // (makes CUDA calls)
// Entries per tile of the forward, and how many partial sums that makes.
int loss_width(int n, int vocab);
inline int loss_chunks(int vocab, int width) { return 2 * ((vocab + width - 1) / width); }
// Ranges of the entries for dx, `most` at most.
int loss_dx_splits(int n, int d, int entries, int most);

cudaError_t launch_loss_sums(const LossProduct &p, int *status, cudaStream_t s);
cudaError_t launch_loss_logit_grad(const LossProduct &p, int *status, cudaStream_t s);
cudaError_t launch_loss_dx(const LossProduct &p, int *status, cudaStream_t s);

// dx (as launch_loss_dx leaves it) and dW [entries][d] (or nullptr) in one pass over W, for
// kLossFewTokens at most; and into how many ranges of the entries dx is cut.
constexpr int kLossFewTokens = 192;
int loss_few_splits(int d, int entries, int most);
cudaError_t launch_loss_few(const LossProduct &p, void *dW, bool want_dx, int *status,
                            cudaStream_t s);

// A few tokens, by streams over W (loss_stream.cu).  The forward's partial sums per token; in
// fp32 the gradient of the logits, dl [entries][pitch], then dx (planes, of `splits` ranges of
// the entries) and dW.
bool loss_stream_supported(const moe_loss_config &c);
int loss_stream_chunks(const moe_loss_config &c);   // CTAs, and partial sums per token
int loss_stream_splits(int d, int entries, int most);
cudaError_t launch_loss_stream_sums(int dtype, const LossProduct &p, int grid, int *status,
                                    cudaStream_t s);
cudaError_t launch_loss_stream_logit_grad(const LossProduct &p, float *dl, int grid, int *status,
                                          cudaStream_t s);
cudaError_t launch_loss_stream_grads(const LossProduct &p, const float *dl, float *dW, bool want_dx,
                                     int *status, cudaStream_t s);

}  // namespace moe
