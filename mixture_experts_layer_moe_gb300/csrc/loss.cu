// Softmax cross entropy of a linear layer over a vocabulary, and its gradient
// (moe.h has the formulas), in pieces of the vocabulary.
//
// Only the tokens that count take part in the gradient: a first launch packs their
// rows of x, their targets, lse and dloss, so that nothing a left out row holds, a NaN
// say, meets a sum.  On the tensor cores the products run over the counted tokens alone; on
// the CUDA cores over as many rows as there are tokens, zeros behind the counted ones.
// The forward, where a token's sums are its own, packs where that saves tiles of the
// product (more than 256 tokens on the tensor cores).
//
// Forward: the product reduces its logits as it forms them, to a maximum and a
// sum of exponentials per token and tile, which a second launch joins.  No logits
// are stored.
//
// Gradient, on the tensor cores (loss_pair.cu): a piece's logits are formed again
// and their gradient stored in bf16, dl [n][pitch], which two products then read:
// dW (launch_gemm_grad, rounded once from the whole sum over the tokens) and dx,
// which adds up over the pieces in fp32 and is rounded once at the end.
//
// Gradient, on the CUDA cores (fp32, and small bf16 problems): dl of a piece in
// fp32 with the token contiguous, lT [piece][pitch]: then dx = dl W is a sum over
// lT's rows (GradProduct: cut into runs where the tiles are few) and dW = dl^T x a
// product of its rows (RowsProduct).
//
// A few tokens' forward, and in fp32 their gradient, are streams over W (loss_stream.cu).
#include <math.h>

#include "api.h"
#include "common.cuh"
#include "launch.h"
#include "loss.h"
#include "step.h"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

constexpr int L_UNIT = 256;                            // a piece's entries are a multiple of this
constexpr int64_t L_PIECE_BYTES = (int64_t)256 << 20;  // of a piece's dl, about
constexpr int64_t L_PIECE_MAX = 1 << 22;               // entries of a piece
// Entries of a piece at least: with fewer, dx is read and written again for few products.
// (32000 entries, us without a least / 2048 / 4096 / 8192: 131072 tokens, d 2048 37210 / 33718 /
// 32153 / 31937; 262144, d 1024 50749 / 34778 / 33664 / 33234; f32, 131072 tokens, d 64, 4099
// entries 21264 / 11524 / 8891 / 7112.)
constexpr int64_t L_PIECE_MIN = 8192;
constexpr int L_MAX_SPLITS = 76;

struct LossLayout {
  size_t status, range, scale, list, target, lse, dloss, at, x, sums, logits, dx, acc, parts, total;
  bool pair;    // on the tensor cores
  bool packed;  // the forward packs the tokens that count
  int pitch;    // CUDA cores: tokens, rounded up to whole vectors of fp32
  int piece;    // vocabulary entries of a piece of the gradient at most
  int pieces;
  int width, chunks;   // entries per tile of the forward; partial sums per token
  int planes;          // dx: partial sums of a piece
  bool few;            // dx and dW in one pass (loss_few.cu)
  bool stream, stream_grad;   // the forward, the gradient by streams over W (loss_stream.cu)
};

int elem_size(const moe_loss_config &c) { return c.dtype == MOE_F32 ? 4 : 2; }

// A bf16 problem that is faster without setting up the pair kernels.
bool small_loss(const moe_loss_config &c) {
  return (int64_t)c.n * c.vocab * c.d <= kSmallProducts && c.d <= 256;
}

// dx of a piece on the CUDA cores, dW of one on the tensor cores (operands unset).
GradProduct dx_product(const moe_loss_config &c, const LossLayout &L, int entries) {
  GradProduct p{};
  p.dtype = c.dtype;
  p.num_experts = 1;
  p.rows = entries;
  p.M = c.n;
  p.N = c.d;
  p.lda = L.pitch;
  p.a_f32 = c.dtype == MOE_BF16;
  return p;
}
int dl_pitch(int entries) { return (entries + 7) / 8 * 8; }
GradProduct dw_product(const moe_loss_config &c, int entries) {
  GradProduct p{};
  p.dtype = c.dtype;
  p.offsets = reinterpret_cast<const int32_t *>(16);   // (set by the caller)
  p.num_experts = 1;
  p.rows = c.n;
  p.M = entries;
  p.N = c.d;
  p.lda = dl_pitch(entries);
  return p;
}

// dW of a piece on the CUDA cores (operands unset).
RowsProduct dw_product_simt(const moe_loss_config &c, int entries) {
  RowsProduct p{};
  p.dtype = c.dtype;
  p.epi = kRowsPlain;
  p.b_rows = 1;
  p.num_experts = 1;
  p.rows = entries;
  p.K = c.n;
  p.N = c.d;
  p.a_f32 = c.dtype == MOE_BF16;
  return p;
}

// Entries of a tile of the forward on the CUDA cores.
int sums_tile(const moe_loss_config &c) {
  RowsProduct p{};
  p.dtype = c.dtype;
  p.rows = c.vocab;
  p.N = c.n;
  return rows_simt_tile(p);
}

int dx_splits(const moe_loss_config &c, const LossLayout &L, int entries, int most) {
  return L.few ? loss_few_splits(c.d, entries, most) : loss_dx_splits(c.n, c.d, entries, most);
}

LossLayout loss_layout(const moe_loss_config &c) {
  LossLayout L{};
  const size_t n = c.n, z = elem_size(c);
  L.pair = c.dtype == MOE_BF16 && !small_loss(c);
  L.packed = L.pair && c.n > 256;
  L.few = L.pair && c.n <= kLossFewTokens;
  L.stream = loss_stream_supported(c);
  L.stream_grad = L.stream && c.dtype == MOE_F32;
  L.pitch = (c.n + 3) / 4 * 4;
  // pieces of nearly equal size
  int64_t fit = L_PIECE_BYTES / ((int64_t)(L.pitch > 0 ? L.pitch : 4) * (L.pair ? 2 : 4));
  fit = (fit < L_PIECE_MIN ? L_PIECE_MIN : fit > L_PIECE_MAX ? L_PIECE_MAX : fit) / L_UNIT * L_UNIT;
  L.pieces = (int)((c.vocab + fit - 1) / fit);
  L.piece = (c.vocab + L.pieces - 1) / L.pieces;
  if (L.pieces > 1) L.piece = (L.piece + L_UNIT - 1) / L_UNIT * L_UNIT;
  L.pieces = (c.vocab + L.piece - 1) / L.piece;
  const int last = c.vocab - (L.pieces - 1) * L.piece;
  L.width = L.pair ? loss_width(c.n, c.vocab) : 0;
  if (L.stream) L.chunks = loss_stream_chunks(c);
  else if (L.pair) L.chunks = loss_chunks(c.vocab, L.width);
  else L.chunks = (c.vocab + sums_tile(c) - 1) / sums_tile(c);
  if (L.stream_grad) {
    L.planes = loss_stream_splits(c.d, L.piece, 2 * L_MAX_SPLITS);
  } else if (L.pair) {
    L.planes = dx_splits(c, L, L.piece, L_MAX_SPLITS);
  } else {
    L.planes = 1;
    for (int entries : {L.piece, last}) {
      const GradProduct p = dx_product(c, L, entries);
      const int splits = c.n > 0 ? grad_splits_simt(&p, 1) : 1;
      if (splits > L.planes) L.planes = splits;
    }
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t a = off;
    off += align_up(bytes);
    return a;
  };
  L.status = take(256);
  L.range = take(8);
  L.scale = take(4);
  L.list = take(n * 4);
  L.target = take((size_t)L.pitch * 4);
  L.lse = take((size_t)L.pitch * 4);
  L.dloss = take((size_t)L.pitch * 4);
  L.at = take(n * 4);
  L.x = take(n * c.d * z);
  // what the forward alone and the gradient alone use shares its place
  const size_t both = off;
  L.sums = take(n * L.chunks * sizeof(float2));
  const size_t forward = off;
  off = both;
  L.logits = take(L.pair ? n * dl_pitch(L.piece) * 2 : (size_t)L.piece * L.pitch * 4);
  L.dx = take((size_t)L.planes * n * c.d * 4);
  L.acc = take(!L.pair && L.pieces > 1 ? n * c.d * 4 : 0);
  size_t parts = 0;
  for (int entries : {L.piece, last}) {
    if (L.few || L.stream_grad) break;
    int splits;
    if (L.pair) {
      const GradProduct p = dw_product(c, entries);
      splits = gemm_grad_splits(&p, 1);
    } else {
      splits = rows_runs_simt(dw_product_simt(c, entries));
    }
    const size_t bytes = splits > 1 ? (size_t)splits * entries * c.d * 4 : 0;
    if (bytes > parts) parts = bytes;
  }
  L.parts = take(parts);
  L.total = off > forward ? off : forward;
  return L;
}

// --------------------------------------------------------- tokens that count
// What the first launch reads and packs, in the tokens' order: counted token j
// is token list[j].
struct PackArgs {
  const int32_t *targets;
  const float *lse, *dloss;    // the gradient's, else nullptr
  const uint4 *x;
  int n, vocab, vecs;          // vectors of 16 bytes per row
  int per;                     // tokens per CTA
  int32_t *range;              // {0, tokens that count}
  int32_t *list, *target;
  float *lse_c, *dloss_c;
  float *scale;                // the largest finite |dloss| of those tokens
  uint4 *x_c;                  // rows past the last counted one are zero
  // outputs of the tokens left out
  float *loss_out, *lse_out;
  uint4 *dx_out;
  int *status;
};

constexpr int PACK_THREADS = 256;
// A CTA takes `per` tokens; how many count before them it finds for itself (one launch, and up to
// some 100000 tokens little beside the rows' copies: 131072 tokens, d 64 57 us; but the targets
// read grow with the tokens' square, 1048576 2550 us).
__global__ void __launch_bounds__(PACK_THREADS) loss_pack_kernel(const __grid_constant__ PackArgs a) {
  __shared__ int failed, part[PACK_THREADS / 32];
  __shared__ float largest[PACK_THREADS / 32];
  __shared__ int place[32];   // counted: its position; left out: -1 - the row that it leaves zero
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) failed = status_failed(a.status);
  __syncthreads();
  if (failed) return;
  const int first = blockIdx.x * a.per, count = min(a.per, a.n - first);
  auto counts = [&](int t) { return t >= 0 && t < a.vocab; };
  int c = 0;
  const int4 *four = reinterpret_cast<const int4 *>(a.targets);   // (`first` is not a multiple of 4)
  for (int i = threadIdx.x; i < first / 4; i += PACK_THREADS) {
    const int4 t = four[i];
    c += counts(t.x) + counts(t.y) + counts(t.z) + counts(t.w);
  }
  if ((int)threadIdx.x < first % 4) c += counts(a.targets[first / 4 * 4 + threadIdx.x]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  if (lane == 0) part[warp] = c;
  __syncthreads();
  if (warp == 0) {
    int sum = lane < PACK_THREADS / 32 ? part[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int t = first + lane;
    const bool there = lane < count;
    const int v = there ? a.targets[t] : -1;
    const bool counted = there && counts(v);
    const unsigned mask = __ballot_sync(0xffffffffu, counted);
    const int j = sum + __popc(mask & lanemask_lt());
    if (counted) {
      place[lane] = j;
      a.list[j] = t;
      a.target[j] = v;
      if (a.dloss) {
        a.lse_c[j] = a.lse[t];
        a.dloss_c[j] = a.dloss[t];
      }
    } else if (there) {
      if (v >= a.vocab) set_status(a.status, MOE_ERR_BAD_INDEX, t);
      // (the i-th token left out, i = t - j, makes row n - 1 - i zero)
      place[lane] = -1 - (a.n - 1 - (t - j));
      if (a.loss_out) {
        a.loss_out[t] = 0.f;
        a.lse_out[t] = 0.f;
      }
    }
    if (lane == 0 && blockIdx.x == gridDim.x - 1) {
      a.range[0] = 0;
      a.range[1] = sum + __popc(mask);
    }
  }
  __syncthreads();
  if (a.dloss && blockIdx.x == gridDim.x - 1) {
    // (in the last CTA, which has seen all targets before its own)
    float most = 0.f;
    for (int t = threadIdx.x; t < a.n; t += PACK_THREADS) {
      const float v = fabsf(a.dloss[t]);
      if (counts(a.targets[t]) && isfinite(v)) most = fmaxf(most, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) largest[warp] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < PACK_THREADS / 32; ++w) most = fmaxf(most, largest[w]);
      *a.scale = most;
    }
  }
  // a warp per row, or the whole CTA for its one row
  const int step = a.per == 1 ? PACK_THREADS : 32, who = a.per == 1 ? 0 : warp;
  for (int i = who; i < count; i += PACK_THREADS / 32) {
    const int p = place[i];
    const bool zero = p < 0;
    const uint4 *from = a.x + (int64_t)(first + i) * a.vecs;
    uint4 *to = a.x_c + (int64_t)(zero ? -1 - p : p) * a.vecs;
    uint4 *out = zero && a.dx_out ? a.dx_out + (int64_t)(first + i) * a.vecs : nullptr;
#pragma unroll 4
    for (int v = a.per == 1 ? threadIdx.x : lane; v < a.vecs; v += step) {
      to[v] = zero ? make_uint4(0, 0, 0, 0) : from[v];
      if (out) out[v] = make_uint4(0, 0, 0, 0);
    }
  }
}

cudaError_t launch_pack(const moe_loss_config &c, const LossLayout &L, const void *x,
                        const int32_t *targets, const float *lse, const float *dloss, float *loss_out,
                        float *lse_out, void *dx_out, void *ws, cudaStream_t s) {
  PackArgs a{};
  a.targets = targets;
  a.lse = lse;
  a.dloss = dloss;
  a.x = (const uint4 *)x;
  a.n = c.n;
  a.vocab = c.vocab;
  a.vecs = c.d * elem_size(c) / 16;
  a.per = c.n <= 2048 ? 1 : c.n <= 16384 ? 8 : 32;
  a.range = at<int32_t>(ws, L.range);
  a.list = at<int32_t>(ws, L.list);
  a.target = at<int32_t>(ws, L.target);
  a.lse_c = at<float>(ws, L.lse);
  a.dloss_c = at<float>(ws, L.dloss);
  a.scale = at<float>(ws, L.scale);
  a.x_c = at<uint4>(ws, L.x);
  a.loss_out = loss_out;
  a.lse_out = lse_out;
  a.dx_out = (uint4 *)dx_out;
  a.status = at<int>(ws, L.status);
  return launch_pdl(loss_pack_kernel, dim3((c.n + a.per - 1) / a.per), dim3(PACK_THREADS), 0, s, a);
}

// ------------------------------------------------------------- softmax sums
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

// Joins (maximum, sum) pairs over a warp.
__device__ __forceinline__ float2 join_pairs(float2 v) {
  float top = v.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return make_float2(top, warp_sum_xor(v.y * expf(v.x - shift_of(top))));
}

struct FinishArgs {
  const float2 *sums;          // [token][pitch], `chunks` of them
  int chunks, pitch, n, vocab;
  float z_loss;
  const int32_t *range, *list; // packed tokens, else nullptr
  const int32_t *targets;
  const float *at;
  float *loss, *lse;
  int *status;
};
// A token's chunks are joined by a warp, or (WIDE: few tokens) by a CTA.
template <bool WIDE>
__global__ void __launch_bounds__(256) loss_finish_kernel(const __grid_constant__ FinishArgs a) {
  __shared__ float2 s[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = WIDE ? blockIdx.x : blockIdx.x * 8 + warp;
  constexpr int STEP = WIDE ? 256 : 32;
  pdl_wait();
  // (a packed call's bad targets are reported by the launch before, others here, by
  // CTAs that exchange nothing with others)
  if (a.range && status_failed(a.status)) return;
  const int count = a.range ? a.range[1] : a.n;
  if (j >= count) return;
  const float2 *mine = a.sums + (int64_t)j * a.pitch;
  float2 v = make_float2(-INFINITY, 0.f);
#pragma unroll 4
  for (int i = WIDE ? threadIdx.x : lane; i < a.chunks; i += STEP) {
    const float2 u = mine[i];
    const float up = fmaxf(v.x, u.x), shift = shift_of(up);
    v.y = v.y * expf(v.x - shift) + u.y * expf(u.x - shift);
    v.x = up;
  }
  v = join_pairs(v);
  if (WIDE) {
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = join_pairs(lane < 8 ? s[lane] : make_float2(-INFINITY, 0.f));
  }
  if (WIDE ? threadIdx.x != 0 : lane != 0) return;
  const int t = a.list ? a.list[j] : j, target = a.targets[t];
  // (the target's logit meets the maximum first: from lse, rounded at the logits' size, it would
  // leave a sure token's loss nothing but that rounding.  The sum holds the maximum's 1, so no loss
  // is negative.)
  const float log_sum = logf(v.y);
  float lse = v.x + log_sum, loss = (v.x - a.at[j]) + log_sum + a.z_loss * lse * lse;
  if (target < 0 || target >= a.vocab) {
    if (target >= a.vocab) set_status(a.status, MOE_ERR_BAD_INDEX, t);
    lse = loss = 0.f;
  }
  a.lse[t] = lse;
  a.loss[t] = loss;
}

// dx of the counted tokens from the partial sums [planes][n][d], added in order (times
// *scale, if given); or (acc_out) what a piece adds to the sum of those before, `acc`.
struct DxArgs {
  const float *parts, *acc;
  float *acc_out;
  int planes, n, vecs;
  const float *scale;
  const int32_t *range, *list;
  void *dx;
  const int *status;
};
// Vector i of it, v = the planes' sum.
template <typename T>
__device__ __forceinline__ void put_dx(const DxArgs &a, int64_t i, float4 (&v)[Vec16<T>::N / 4], float k) {
  constexpr int V = Vec16<T>::N / 4;
  const int64_t j = i / a.vecs;
  if (a.acc_out) {
#pragma unroll
    for (int h = 0; h < V; ++h) reinterpret_cast<float4 *>(a.acc_out)[i * V + h] = v[h];
  } else {
#pragma unroll
    for (int h = 0; h < V; ++h) v[h] = make_float4(v[h].x * k, v[h].y * k, v[h].z * k, v[h].w * k);
    reinterpret_cast<uint4 *>(a.dx)[(int64_t)a.list[j] * a.vecs + (i - j * a.vecs)] =
        pack16<T>(reinterpret_cast<const float *>(v));
  }
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
template <typename T>
__global__ void __launch_bounds__(256) loss_dx_kernel(const __grid_constant__ DxArgs a) {
  constexpr int N = Vec16<T>::N, V = N / 4;
  pdl_wait();
  if (status_failed(a.status)) return;
  const int64_t total = (int64_t)a.range[1] * a.vecs, plane = (int64_t)a.n * a.vecs * V;
  const float k = a.scale ? *a.scale : 1.f;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const float4 *from = reinterpret_cast<const float4 *>(a.parts) + i * V;
    float4 v[V];
#pragma unroll
    for (int h = 0; h < V; ++h)
      v[h] = a.acc ? reinterpret_cast<const float4 *>(a.acc)[i * V + h] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = 0; p < a.planes; ++p) {
#pragma unroll
      for (int h = 0; h < V; ++h) v[h] = add4(v[h], from[p * plane + h]);
    }
    put_dx<T>(a, i, v, k);
  }
}
// 16 planes and more: 32 vectors per CTA, whose warps take the planes in turn; their sums
// are added in order.  (One fp32 token, d 512, 8192 entries, 152 planes: 33.3 us for 20.6; from 4
// planes on 300 bf16 tokens, d 7168 took 459 for 441.)
template <typename T>
__global__ void __launch_bounds__(256) loss_dx_wide_kernel(const __grid_constant__ DxArgs a) {
  constexpr int N = Vec16<T>::N, V = N / 4;
  __shared__ float4 s[8][V][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (status_failed(a.status)) return;
  const int64_t total = (int64_t)a.range[1] * a.vecs, plane = (int64_t)a.n * a.vecs * V;
  const float k = a.scale ? *a.scale : 1.f;
  for (int64_t i0 = (int64_t)blockIdx.x * 32; i0 < total; i0 += (int64_t)gridDim.x * 32) {
    const int64_t i = i0 + lane;
    float4 v[V];
#pragma unroll
    for (int h = 0; h < V; ++h) v[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < total) {
      const float4 *from = reinterpret_cast<const float4 *>(a.parts) + i * V;
#pragma unroll 8
      for (int p = warp; p < a.planes; p += 8) {
#pragma unroll
        for (int h = 0; h < V; ++h) v[h] = add4(v[h], from[p * plane + h]);
      }
    }
#pragma unroll
    for (int h = 0; h < V; ++h) s[warp][h][lane] = v[h];
    __syncthreads();
    if (warp == 0 && i < total) {
#pragma unroll
      for (int h = 0; h < V; ++h) {
        v[h] = a.acc ? reinterpret_cast<const float4 *>(a.acc)[i * V + h]
                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) v[h] = add4(v[h], s[w][h][lane]);
      }
      put_dx<T>(a, i, v, k);
    }
    __syncthreads();
  }
}

unsigned blocks_of(int64_t threads) {
  const int64_t b = (threads + 255) / 256, most = (int64_t)num_sms() * 8;
  return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

#define LOSS_TRY(expr)                       \
  do {                                       \
    const cudaError_t _e = (expr);           \
    if (_e != cudaSuccess) return _e;        \
  } while (0)

cudaError_t finish_dx(const moe_loss_config &c, const LossLayout &L, int planes, const float *acc,
                      float *acc_out, void *dx, void *ws, cudaStream_t s) {
  const bool f32 = c.dtype == MOE_F32, wide = planes >= 16;
  const DxArgs a{at<float>(ws, L.dx), acc, acc_out, planes, c.n, c.d * elem_size(c) / 16,
                 L.pair ? at<float>(ws, L.scale) : nullptr, at<int32_t>(ws, L.range),
                 at<int32_t>(ws, L.list), dx, at<int>(ws, L.status)};
  auto kernel = f32 ? (wide ? loss_dx_wide_kernel<float> : loss_dx_kernel<float>)
                    : (wide ? loss_dx_wide_kernel<__nv_bfloat16> : loss_dx_kernel<__nv_bfloat16>);
  return launch_pdl(kernel, dim3(blocks_of((int64_t)c.n * a.vecs * (wide ? 8 : 1))), dim3(256), 0, s, a);
}

// The logits' product on the CUDA cores, over entries v0 .. of the vocabulary.
RowsProduct simt_product(const moe_loss_config &c, int epi, const void *x, const void *W, int v0,
                         int entries) {
  RowsProduct p{};
  p.dtype = c.dtype;
  p.epi = epi;
  p.num_experts = 1;
  p.rows = entries;
  p.K = c.d;
  p.N = c.n;
  p.A = (const char *)W + (size_t)v0 * c.d * elem_size(c);
  p.B = x;
  p.loss.v0 = v0;
  return p;
}

// The operands that the products on the tensor cores and the streams share, over entries
// v0 .. of the vocabulary, whose rows are W.
LossProduct loss_product(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                         int entries, void *ws) {
  LossProduct p{};
  p.n = c.n;
  p.d = c.d;
  p.entries = entries;
  p.v0 = v0;
  p.range = at<int32_t>(ws, L.range);
  p.target = at<int32_t>(ws, L.target);
  p.x = at<void>(ws, L.x);
  p.W = W;
  p.lse = at<float>(ws, L.lse);
  p.dloss = at<float>(ws, L.dloss);
  p.scale = at<float>(ws, L.scale);
  p.z_loss = c.z_loss;
  p.dl = at<void>(ws, L.logits);
  p.pitch = dl_pitch(entries);
  p.planes = at<float>(ws, L.dx);
  return p;
}

cudaError_t piece_gradient_stream(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                                  int entries, int i, void *dx, void *dW, void *ws, cudaStream_t s) {
  int *status = at<int>(ws, L.status);
  const size_t first = (size_t)v0 * c.d;
  LossProduct p = loss_product(c, L, (const float *)W + first, v0, entries, ws);
  p.pitch = L.pitch;
  p.splits = loss_stream_splits(c.d, entries, L.planes);
  float *dl = at<float>(ws, L.logits), *acc = at<float>(ws, L.acc);
  LOSS_TRY(launch_loss_stream_logit_grad(p, dl, loss_stream_chunks(c), status, s));
  LOSS_TRY(launch_loss_stream_grads(p, dl, dW ? (float *)dW + first : nullptr, dx != nullptr, status, s));
  if (!dx) return cudaSuccess;
  return finish_dx(c, L, p.splits, i > 0 ? acc : nullptr, i + 1 < L.pieces ? acc : nullptr, dx, ws, s);
}

cudaError_t piece_gradient_simt(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                                int entries, int i, void *dx, void *dW, void *ws, cudaStream_t s) {
  const size_t row = (size_t)c.d * elem_size(c);
  int *status = at<int>(ws, L.status);
  RowsProduct l = simt_product(c, kRowsLossGrad, at<void>(ws, L.x), W, v0, entries);
  l.out = at<void>(ws, L.logits);
  l.ldo = L.pitch;
  l.loss.target = at<int32_t>(ws, L.target);
  l.loss.range = at<int32_t>(ws, L.range);
  l.loss.lse = at<float>(ws, L.lse);
  l.loss.dloss = at<float>(ws, L.dloss);
  l.loss.z_loss = c.z_loss;
  LOSS_TRY(launch_rows_simt(l, status, s));
  if (dW) {
    RowsProduct p = dw_product_simt(c, entries);
    void *out = (char *)dW + v0 * row;
    float *parts = at<float>(ws, L.parts);
    p.lda = L.pitch;
    p.A = at<void>(ws, L.logits);
    p.B = at<void>(ws, L.x);
    p.k_runs = rows_runs_simt(p);
    p.out = p.k_runs > 1 ? parts : out;
    LOSS_TRY(launch_rows_simt(p, status, s));
    if (p.k_runs > 1)
      LOSS_TRY(add_runs_simt(c.dtype, parts, p.k_runs, (int64_t)entries * c.d, out, status, s));
  }
  if (!dx) return cudaSuccess;
  GradProduct p = dx_product(c, L, entries);
  p.A = at<void>(ws, L.logits);
  p.B = (const char *)W + v0 * row;
  const int splits = grad_splits_simt(&p, 1);
  LOSS_TRY(launch_grad_simt(&p, 1, splits, at<float>(ws, L.dx), status, s, false));
  float *acc = at<float>(ws, L.acc);
  return finish_dx(c, L, splits, i > 0 ? acc : nullptr, i + 1 < L.pieces ? acc : nullptr, dx, ws, s);
}

cudaError_t piece_gradient_pair(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                                int entries, int i, void *dx, void *dW, void *ws, cudaStream_t s) {
  int *status = at<int>(ws, L.status);
  LossProduct p = loss_product(c, L, (const char *)W + (size_t)v0 * c.d * 2, v0, entries, ws);
  void *out = dW ? (char *)dW + (size_t)v0 * c.d * 2 : nullptr;
  // (the last piece may be cut into fewer ranges, and adds to the first planes)
  p.splits = entries == L.piece ? L.planes : dx_splits(c, L, entries, L.planes);
  p.add = i > 0;
  LOSS_TRY(launch_loss_logit_grad(p, status, s));
  if (L.few) {
    LOSS_TRY(launch_loss_few(p, out, dx != nullptr, status, s));
  } else if (dW) {
    GradProduct g = dw_product(c, entries);
    g.offsets = p.range;
    g.A = p.dl;
    g.B = p.x;
    g.out = out;
    g.scale = p.scale;
    if (!gemm_grad_supported(g)) return cudaErrorNotSupported;
    LOSS_TRY(launch_gemm_grad(&g, 1, gemm_grad_splits(&g, 1), at<float>(ws, L.parts), 0, status, s));
  }
  if (!dx) return cudaSuccess;
  if (!L.few) LOSS_TRY(launch_loss_dx(p, status, s));
  return i + 1 < L.pieces ? cudaSuccess : finish_dx(c, L, L.planes, nullptr, nullptr, dx, ws, s);
}

}  // namespace

size_t loss_workspace(const moe_loss_config &c) { return loss_layout(c).total; }

cudaError_t launch_loss(const moe_loss_config &c, const void *x, const void *W,
                        const int32_t *targets, float *loss, float *lse, void *ws, cudaStream_t s) {
  const LossLayout L = loss_layout(c);
  if (L.pair && !loss_pair_supported(c)) return cudaErrorNotSupported;
  FinishArgs f{};
  f.sums = at<float2>(ws, L.sums);
  f.chunks = f.pitch = L.chunks;
  f.n = c.n;
  f.vocab = c.vocab;
  f.z_loss = c.z_loss;
  f.targets = targets;
  f.at = at<float>(ws, L.at);
  f.loss = loss;
  f.lse = lse;
  f.status = at<int>(ws, L.status);
  if (L.packed) {
    LOSS_TRY(launch_pack(c, L, x, targets, nullptr, nullptr, loss, lse, nullptr, ws, s));
    f.range = at<int32_t>(ws, L.range);
    f.list = at<int32_t>(ws, L.list);
  }
  if (L.stream) {
    LossProduct p = loss_product(c, L, W, 0, c.vocab, ws);
    p.target = targets;
    p.x = x;
    p.sums = at<float2>(ws, L.sums);
    p.chunks = L.chunks;
    p.at = at<float>(ws, L.at);
    f.chunks = loss_stream_chunks(c);
    LOSS_TRY(launch_loss_stream_sums(c.dtype, p, f.chunks, f.status, s));
  } else if (L.pair) {
    LossProduct p = loss_product(c, L, W, 0, c.vocab, ws);
    p.sums = at<float2>(ws, L.sums);
    p.width = L.width;
    p.chunks = L.chunks;
    p.at = at<float>(ws, L.at);
    if (!L.packed) {
      p.range = nullptr;
      p.target = targets;
      p.x = x;
    }
    LOSS_TRY(launch_loss_sums(p, f.status, s));
  } else {
    RowsProduct p = simt_product(c, kRowsLossSums, x, W, 0, c.vocab);
    p.loss.target = targets;
    p.loss.sums = at<float2>(ws, L.sums);
    p.loss.chunks = L.chunks;
    p.loss.at = at<float>(ws, L.at);
    LOSS_TRY(launch_rows_simt(p, f.status, s));
  }
  if (c.n <= 8 * num_sms())
    return launch_pdl(loss_finish_kernel<true>, dim3(c.n), dim3(256), 0, s, f);
  return launch_pdl(loss_finish_kernel<false>, dim3((c.n + 7) / 8), dim3(256), 0, s, f);
}

cudaError_t launch_loss_backward(const moe_loss_config &c, const void *x, const void *W,
                                 const int32_t *targets, const float *lse, const float *dloss,
                                 void *dx, void *dW, void *ws, cudaStream_t s) {
  const LossLayout L = loss_layout(c);
  if (L.pair && !loss_pair_supported(c)) return cudaErrorNotSupported;
  LOSS_TRY(launch_pack(c, L, x, targets, lse, dloss, nullptr, nullptr, dx, ws, s));
  auto piece = L.pair ? piece_gradient_pair : L.stream_grad ? piece_gradient_stream : piece_gradient_simt;
  for (int v0 = 0, i = 0; v0 < c.vocab; v0 += L.piece, ++i)
    LOSS_TRY(piece(c, L, W, v0, c.vocab - v0 < L.piece ? c.vocab - v0 : L.piece, i, dx, dW, ws, s));
  return cudaSuccess;
}

}  // namespace moe
