// Host-side launchers of the training kernels (internal; the public ABI is moe.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// ------------------------------------------------------------- layer norm
cudaError_t launch_norm(const moe_norm_config &c, const void *x, const void *gamma,
                        const void *beta, void *y, float *mean, float *rstd, cudaStream_t s);
size_t norm_backward_scratch(const moe_norm_config &c);
cudaError_t launch_norm_backward(const moe_norm_config &c, const void *x, const void *gamma,
                                 const float *mean, const float *rstd, const void *dy, void *dx,
                                 float *dgamma, float *dbeta, void *scratch, cudaStream_t s);

// a[i] = sum over `count` rows of pa[row][i], i < d, in a fixed order; b from pb
// likewise (each output nullptr: not wanted; b is the second of two).
cudaError_t launch_column_sum(const float *pa, const float *pb, int count, int d, float *a,
                              float *b, const int *status, cudaStream_t s);

// --------------------------------------------------------- combine, router
cudaError_t launch_combine_backward(int dtype, const void *dy, const void *y_perm,
                                    const int32_t *inv_perm, const float *gates, void *dy_perm,
                                    float *dgate, int n, int k, int d, int *status,
                                    cudaStream_t s);

// dl [n][pitch] (dl_f32: fp32, else bf16; columns E .. pitch - 1 zero) and, when dbias is set,
// the column sums, through route_grad_scratch(c) bytes of scratch.
// dl may be nullptr (dbias alone).  inv_perm [n*K], or nullptr: checked here for
// the product that follows, which skips an index outside [0, n*K) and cannot set
// the status itself (CTAs of a pair must not differ on it).
size_t route_grad_scratch(const moe_config &c);
cudaError_t launch_route_grad(const moe_config &c, const float *probs, const int32_t *topk_idx,
                              const float *gates, const float *dgate, const float *f, float aux,
                              const int32_t *inv_perm, void *dl, bool dl_f32, int pitch,
                              float *dbias, float *scratch, int *status, cudaStream_t s);

// dx from the expert rows' gradients and the router's in one pass, where dl has
// entries at the chosen experts alone and these are few.
constexpr int kRouteRowsMaxK = 16;
bool route_rows_supported(const moe_config &c, const float *f);
cudaError_t launch_route_rows(const moe_config &c, const void *Wg, const int32_t *topk_idx,
                              const float *gates, const float *dgate, const int32_t *inv_perm,
                              const void *dx_perm, void *dx, int *status, cudaStream_t s);

// ------------------------------------------------------- grouped products
enum {
  kRowsPlain = 0,       // out = A B (+ A2 B2)
  kRowsRelu = 1,        // out = max(A B, 0)
  kRowsSwiglu = 2,      // out = silu(A B) * (A B2), out_g = A B, out_u = A B2
  kRowsReluGrad = 3,    // out = A B where h > 0
  kRowsSwigluGrad = 4,  // v = A B: out = v u s (1 + g (1 - s)), out_u = v g s
  // on the CUDA cores, A the vocabulary's rows and B the tokens' (LossTerms below)
  kRowsLossSums = 5,    // v = A B: a maximum and a sum of exponentials per token
  kRowsLossGrad = 6,    // out = dloss (e^(v - lse) (1 + 2 z lse) - [target]), fp32
};

// What the cross entropy's epilogues take: per token, and the vocabulary entry of
// row 0.
struct LossTerms {
  const int32_t *target;
  int v0;
  // kRowsLossSums: sums [tokens][chunks], of one tile of entries each; the target's logit
  float2 *sums;
  int chunks;
  float *at;
  // kRowsLossGrad: tokens from range[1] on do not count
  const int32_t *range;
  const float *lse, *dloss;
  float z_loss;
};

// Products that write rows of the segments: for q in segment e,
//   out[q][c] = epi( sum_k A[q][k] B_e(k, c) ),   c < N.
// b_rows: B is stored [E][K][N] (the weights of a gradient), else [E][N][K].
struct RowsProduct {
  int dtype, epi, b_rows;
  const int32_t *offsets;   // nullptr: one segment [0, rows) of expert 0
  int num_experts, rows, K, N;
  int lda;                  // elements from one row of A to the next (0: K)
  const void *A, *A2;       // A2: the second product's rows (kRowsPlain) or nullptr
  const void *B, *B2;
  const void *g, *u, *h;    // kept rows [rows][N] that a gradient's epilogue reads
  void *out, *out_g, *out_u;   // [rows][N]
  // kRowsPlain, one segment: out[q] += sum_j add[add_inv[q * add_k + j]], in fp32
  const void *add;             // [rows * add_k][N] or nullptr
  const int32_t *add_inv;
  int add_k;
  int beside;                  // see launch_gemm_grad
  // For a bf16 layer: A and A2 are fp32 (on the CUDA cores), or out and out_u of a
  // gradient are
  int a_f32, out_f32;
  // kRowsPlain, b_rows, one segment, on the CUDA cores: runs that the reduction is cut into
  // (0: one); out is then fp32 [run][rows][N], for add_runs_simt
  int k_runs;
  // kRowsLossGrad: elements from one row of out to the next, a multiple of 4; columns
  // from N on are written as zeros
  int ldo;
  LossTerms loss;
};
// Entries of a tile of rows (p as launch_rows_simt takes it).
int rows_simt_tile(const RowsProduct &p);
// fp32, and small bf16 products: at most so many multiplications each.
constexpr int64_t kSmallProducts = 1 << 24;
cudaError_t launch_rows_simt(const RowsProduct &p, int *status, cudaStream_t s);
// Runs for such a product whose tiles leave most SMs without work.
int rows_runs_simt(const RowsProduct &p);
// out[i] = sum of parts [run][count], in order (count: a multiple of 4).
cudaError_t add_runs_simt(int dtype, const float *parts, int runs, int64_t count, void *out,
                          int *status, cudaStream_t s);

// The same with the reduction cut into ranges where its tiles are few (bf16), or
// whole with fp32 outputs: how many ranges (1: not cut; by the shape alone), the
// scratch that takes, and the launches; `whole` is the product as the pair
// kernel takes it.
int rows_splits(const RowsProduct &p);
size_t rows_scratch(const RowsProduct &p);
cudaError_t launch_rows_split(const RowsProduct &p, const struct GemmStage &whole, int splits,
                              float *parts, int *status, cudaStream_t s);

// Products over the rows of each segment (a weight's gradient):
//   out_e[m][c] = sum_{q in segment e} A[q][m] B[q][c],   m < M, c < N;
// zero for a segment without rows.
struct GradProduct {
  int dtype;
  const int32_t *offsets;   // nullptr: one segment [0, rows) of expert 0
  int num_experts, rows, M, N;
  int lda;                  // elements from one row of A to the next (0: M)
  const void *A, *B;
  void *out;                // [E][M][N]
  int a_f32;                // on the CUDA cores, for a bf16 layer: A is fp32
  const float *scale;       // on the tensor cores: the sums are multiplied by *scale (nullptr: 1);
                            // the first problem's holds for all of a launch
};
constexpr int kMaxGradProblems = 3;
int grad_splits_simt(const GradProduct *p, int count);
// Up to kMaxGradProblems of them over the same segments in one launch on the CUDA
// cores (where grads_small: fp32, and small bf16 products), with a second that
// adds the runs where the rows are cut into several; splits, parts: as
// grad_splits and grad_scratch (below) say.
bool grads_small(const GradProduct *p, int count);
// add = false: the runs' partial sums stay in parts [problem][expert][run][M][N], also of
// one run.
cudaError_t launch_grad_simt(const GradProduct *p, int count, int splits, float *parts, int *status,
                             cudaStream_t s, bool add = true);
// The same on tensor cores (bf16; SM pairs).
bool gemm_grad_supported(const GradProduct &p);
// Runs that the segments' rows are cut into where the problems are too few to
// fill the SMs (1: not cut), and the scratch that the partial sums take.  Both
// go by the shapes alone.
int grad_splits(const GradProduct *p, int count);
int gemm_grad_splits(const GradProduct *p, int count);   // (whatever their size)
size_t grad_scratch(const GradProduct *p, int count);
// beside: 0, or the SM pairs that it takes so that the next launch, a b_rows
// RowsProduct with `beside` pairs of its own that does not read its results,
// runs at the same time.
cudaError_t launch_gemm_grad(const GradProduct *p, int count, int splits, float *scratch,
                             int beside, int *status, cudaStream_t s);
// A RowsProduct of one segment with a short reduction, on the same kernel.
bool gemm_router_rows_supported(const RowsProduct &p);
cudaError_t launch_gemm_router_rows(const RowsProduct &p, int *status, cudaStream_t s);

}  // namespace moe
