// Softmax cross entropy of a linear layer over a vocabulary, and its gradient
// (moe.h has the formulas), in pieces of the vocabulary.
//
// Only the tokens that count take part: a first launch packs their rows of x,
// their targets and (for the gradient) lse and dloss, so that the products run
// over them alone and nothing a left out row holds, a NaN say, meets a sum.
//
// On the CUDA cores (fp32, and small bf16 problems) a piece's logits lie in the
// workspace in fp32 with the token contiguous, lT [piece][pitch]: then dx = dl W
// is a sum over lT's rows (GradProduct: cut into runs where the tiles are few)
// and dW = dl^T x a product of its rows (RowsProduct).
//
// On the tensor cores (other bf16 problems, loss_pair.cu) the forward reduces the
// logits as it forms them.  The gradient forms a piece's logits again and
// stores their gradient in bf16, dl [n][pitch], which two products then read: dW
// (launch_gemm_grad, rounded once from the whole sum over the tokens) and dx,
// which adds up over the pieces in fp32 and is rounded once at the end.
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

constexpr int L_CHUNK = 256;                           // vocabulary entries of a partial sum
constexpr int64_t L_PIECE_BYTES = (int64_t)256 << 20;  // of a piece's logits, about
constexpr int64_t L_PIECE_MAX = 1 << 22;               // entries of a piece
constexpr int L_MAX_SPLITS = 76;

struct LossLayout {
  size_t status, range, list, target, lse, dloss, at, x, sums, logits, dx, parts, total;
  bool pair;    // on the tensor cores
  int pitch;    // CUDA cores: tokens, rounded up to whole vectors of fp32
  int piece;    // vocabulary entries of a piece at most (a multiple of L_CHUNK where there are several)
  int pieces;
  int width, chunks;   // entries per tile of the forward; partial sums per token
  int planes;          // dx: its partial sums
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

LossLayout loss_layout(const moe_loss_config &c) {
  LossLayout L{};
  const size_t n = c.n, z = elem_size(c);
  L.pair = c.dtype == MOE_BF16 && !small_loss(c);
  L.pitch = (c.n + 3) / 4 * 4;
  int64_t fit = L_PIECE_BYTES / ((int64_t)L.pitch * (L.pair ? 2 : 4) + 1) / L_CHUNK * L_CHUNK;
  if (fit > L_PIECE_MAX) fit = L_PIECE_MAX;
  L.piece = (int)(fit < L_CHUNK ? L_CHUNK : fit < c.vocab ? fit : c.vocab);
  L.pieces = (int)(((int64_t)c.vocab + L.piece - 1) / L.piece);
  L.width = L.pair ? loss_width(c.n, c.vocab) : 0;
  L.chunks = L.pair ? loss_chunks(c.vocab, L.width) : (c.vocab + L_CHUNK - 1) / L_CHUNK;
  L.planes = L.pair ? loss_dx_splits(c.n, c.d, L.piece, L_MAX_SPLITS) : L.pieces;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t a = off;
    off += align_up(bytes);
    return a;
  };
  L.status = take(256);
  L.range = take(8);
  L.list = take(n * 4);
  L.target = take((size_t)L.pitch * 4);
  L.lse = take((size_t)L.pitch * 4);
  L.dloss = take((size_t)L.pitch * 4);
  L.at = take(n * 4);
  L.x = take(n * c.d * z);
  const size_t both = off;
  // what the forward alone and the gradient alone use shares its place
  L.sums = take(n * L.chunks * sizeof(float2));
  if (!L.pair) L.logits = take((size_t)L.piece * L.pitch * 4);
  const size_t forward = off;
  if (L.pair) {
    off = both;
    L.logits = take(n * dl_pitch(L.piece) * 2);
  }
  L.dx = take((size_t)L.planes * n * c.d * (L.pair ? 4 : z));
  size_t parts = 0;
  if (L.pair) {
    for (int entries : {L.piece, c.vocab - (L.pieces - 1) * L.piece}) {
      const GradProduct p = dw_product(c, entries);
      const size_t bytes = grad_scratch(&p, 1);
      if (bytes > parts) parts = bytes;
    }
  } else if (c.n > 0) {
    const GradProduct p = dx_product(c, L, L.piece);
    const int splits = grad_splits_simt(&p, 1);
    if (splits > 1) parts = (size_t)splits * n * c.d * 4;
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
  uint4 *x_c;                  // rows past the last counted one are zero
  // outputs of the tokens left out
  float *loss_out, *lse_out;
  uint4 *dx_out;
  int *status;
};

constexpr int PACK_THREADS = 256;
// A CTA takes `per` tokens; how many count before them it finds for itself.
__global__ void __launch_bounds__(PACK_THREADS) loss_pack_kernel(const __grid_constant__ PackArgs a) {
  __shared__ int failed, before, part[PACK_THREADS / 32];
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
  a.x_c = at<uint4>(ws, L.x);
  a.loss_out = loss_out;
  a.lse_out = lse_out;
  a.dx_out = (uint4 *)dx_out;
  a.status = at<int>(ws, L.status);
  return launch_pdl(loss_pack_kernel, dim3((c.n + a.per - 1) / a.per), dim3(PACK_THREADS), 0, s, a);
}

// ------------------------------------------------------------- softmax sums
// e^(v - m) where m is a maximum of v: 0 terms of an empty maximum stay 0.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

// (maximum, sum of e^(l - maximum)) of one chunk of the vocabulary for 32
// tokens: eight warps of 32 entries each, then joined.
__global__ void __launch_bounds__(256)
loss_chunk_kernel(const float *__restrict__ lt, int pitch, int entries, int v0, int chunks,
                  const int32_t *__restrict__ range, const int32_t *__restrict__ target,
                  float *__restrict__ at, float2 *__restrict__ sums, const int *status) {
  __shared__ float2 s[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 32 + lane, e0 = blockIdx.y * L_CHUNK + warp * 32;
  pdl_launch_dependents();
  pdl_wait();
  if (status_failed(status)) return;
  const bool there = j < range[1];
  float v[32], m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = there && e0 + i < entries ? lt[(int64_t)(e0 + i) * pitch + j] : -INFINITY;
    m = fmaxf(m, v[i]);
  }
  const float shift = shift_of(m);
#pragma unroll
  for (int i = 0; i < 32; ++i) sum += expf(v[i] - shift);
  s[warp][lane] = make_float2(m, sum);
  if (there) {
    const int t = target[j] - v0 - e0;
    if (t >= 0 && t < 32 && e0 + t < entries) at[j] = lt[(int64_t)(e0 + t) * pitch + j];
  }
  __syncthreads();
  if (warp != 0 || !there) return;
  m = -INFINITY;
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, s[w][lane].x);
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += s[w][lane].y * expf(s[w][lane].x - shift_of(m));
  sums[(int64_t)j * chunks + v0 / L_CHUNK + blockIdx.y] = make_float2(m, sum);
}

// A warp per counted token joins its chunks.
__global__ void __launch_bounds__(256)
loss_finish_kernel(const float2 *__restrict__ sums, int chunks, float z_loss,
                   const int32_t *__restrict__ range, const int32_t *__restrict__ list,
                   const float *__restrict__ at, float *__restrict__ loss, float *__restrict__ lse_out,
                   const int *status) {
  const int lane = threadIdx.x & 31;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  if (status_failed(status) || j >= range[1]) return;
  const float2 *mine = sums + (int64_t)j * chunks;
  float m = -INFINITY, sum = 0.f;
  for (int i = lane; i < chunks; i += 32) {
    const float2 v = mine[i];
    const float up = fmaxf(m, v.x), shift = shift_of(up);
    sum = sum * expf(m - shift) + v.y * expf(v.x - shift);
    m = up;
  }
  float top = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  sum = warp_sum_xor(sum * expf(m - shift_of(top)));
  if (lane != 0) return;
  const float lse = top + logf(sum);
  const int t = list[j];
  lse_out[t] = lse;
  loss[t] = lse - at[j] + z_loss * lse * lse;
}

// lT <- dl, four tokens per thread; columns of tokens that do not count are zero.
__global__ void __launch_bounds__(256)
loss_grad_kernel(float4 *__restrict__ lt, int pitch4, int entries, int v0, float z_loss,
                 const int32_t *__restrict__ range, const int4 *__restrict__ target,
                 const float4 *__restrict__ lse, const float4 *__restrict__ dloss,
                 const int *status) {
  pdl_launch_dependents();
  pdl_wait();
  if (status_failed(status)) return;
  const int m = range[1];
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)entries * pitch4;
       i += (int64_t)gridDim.x * 256) {
    const int e = (int)(i / pitch4), q = (int)(i - (int64_t)e * pitch4);
    const float4 l = lt[i], ls = lse[q], dl = dloss[q];
    const int4 t = target[q];
    auto one = [&](int k, float l1, float lse1, float dloss1, int t1) {
      if (4 * q + k >= m) return 0.f;
      const float p = expf(l1 - lse1) * fmaf(2.f * z_loss, lse1, 1.f);
      return dloss1 * (t1 == v0 + e ? p - 1.f : p);
    };
    lt[i] = make_float4(one(0, l.x, ls.x, dl.x, t.x), one(1, l.y, ls.y, dl.y, t.y),
                        one(2, l.z, ls.z, dl.z, t.z), one(3, l.w, ls.w, dl.w, t.w));
  }
}

// dx of the counted tokens: the partial sums [planes][n][d] of type TI, added in
// order.
template <typename T, typename TI>
__global__ void __launch_bounds__(256)
loss_dx_kernel(const TI *__restrict__ parts, int planes, int n, int vecs,
               const int32_t *__restrict__ range, const int32_t *__restrict__ list,
               T *__restrict__ dx, const int *status) {
  constexpr int N = Vec16<T>::N, NI = Vec16<TI>::N;
  pdl_wait();
  if (status_failed(status)) return;
  const int64_t total = (int64_t)range[1] * vecs, plane = (int64_t)n * vecs * (N / NI);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t j = i / vecs;
    const uint4 *from = reinterpret_cast<const uint4 *>(parts) + i * (N / NI);
    float v[N], w[NI];
#pragma unroll
    for (int h = 0; h < N / NI; ++h) unpack16<TI>(from[h], v + h * NI);
#pragma unroll 4
    for (int p = 1; p < planes; ++p) {
#pragma unroll
      for (int h = 0; h < N / NI; ++h) {
        unpack16<TI>(from[p * plane + h], w);
#pragma unroll
        for (int k = 0; k < NI; ++k) v[h * NI + k] += w[k];
      }
    }
    reinterpret_cast<uint4 *>(dx)[(int64_t)list[j] * vecs + (i - j * vecs)] = pack16<T>(v);
  }
}

unsigned blocks_of(int64_t threads) {
  const int64_t b = (threads + 255) / 256, most = (int64_t)num_sms() * 8;
  return (unsigned)(b < 1 ? 1 : b < most ? b : most);
}

// A piece's logits, in the workspace.
cudaError_t piece_logits(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                         int entries, void *ws, cudaStream_t s) {
  RowsProduct p{};
  p.dtype = c.dtype;
  p.epi = kRowsPlain;
  p.num_experts = 1;
  p.rows = entries;
  p.K = c.d;
  p.N = c.n;
  p.A = (const char *)W + (size_t)v0 * c.d * elem_size(c);
  p.B = at<void>(ws, L.x);
  p.out = at<void>(ws, L.logits);
  p.ldo = L.pitch;
  p.out_f32 = c.dtype == MOE_BF16;
  return launch_rows_simt(p, at<int>(ws, L.status), s);
}

template <typename T, typename TI>
cudaError_t finish_dx(const moe_loss_config &c, const LossLayout &L, void *dx, void *ws,
                      cudaStream_t s) {
  const int vecs = c.d / Vec16<T>::N;
  return launch_pdl(loss_dx_kernel<T, TI>, dim3(blocks_of((int64_t)c.n * vecs)), dim3(256), 0, s,
                    at<TI>(ws, L.dx), L.planes, c.n, vecs, at<int32_t>(ws, L.range),
                    at<int32_t>(ws, L.list), (T *)dx, at<int>(ws, L.status));
}

// The operands that a piece's products on the tensor cores share.
LossProduct pair_product(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                         int entries, void *ws) {
  LossProduct p{};
  p.n = c.n;
  p.d = c.d;
  p.entries = entries;
  p.v0 = v0;
  p.range = at<int32_t>(ws, L.range);
  p.target = at<int32_t>(ws, L.target);
  p.x = at<void>(ws, L.x);
  p.W = (const char *)W + (size_t)v0 * c.d * 2;
  p.width = L.width;
  p.chunks = L.chunks;
  p.sums = at<float2>(ws, L.sums);
  p.at = at<float>(ws, L.at);
  p.lse = at<float>(ws, L.lse);
  p.dloss = at<float>(ws, L.dloss);
  p.z_loss = c.z_loss;
  p.dl = at<void>(ws, L.logits);
  p.pitch = dl_pitch(entries);
  p.planes = at<float>(ws, L.dx);
  return p;
}

#define LOSS_TRY(expr)                       \
  do {                                       \
    const cudaError_t _e = (expr);           \
    if (_e != cudaSuccess) return _e;        \
  } while (0)

cudaError_t piece_gradient_simt(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                                int entries, int i, bool dx, void *dW, void *ws, cudaStream_t s) {
  const size_t row = (size_t)c.d * elem_size(c);
  int *status = at<int>(ws, L.status);
  LOSS_TRY(piece_logits(c, L, W, v0, entries, ws, s));
  LOSS_TRY(launch_pdl(loss_grad_kernel, dim3(blocks_of((int64_t)entries * L.pitch / 4)), dim3(256),
                      0, s, at<float4>(ws, L.logits), L.pitch / 4, entries, v0, c.z_loss,
                      at<int32_t>(ws, L.range), at<int4>(ws, L.target), at<float4>(ws, L.lse),
                      at<float4>(ws, L.dloss), status));
  if (dW) {
    RowsProduct p{};
    p.dtype = c.dtype;
    p.epi = kRowsPlain;
    p.b_rows = 1;
    p.num_experts = 1;
    p.rows = entries;
    p.K = c.n;
    p.N = c.d;
    p.lda = L.pitch;
    p.A = at<void>(ws, L.logits);
    p.B = at<void>(ws, L.x);
    p.out = (char *)dW + v0 * row;
    p.a_f32 = c.dtype == MOE_BF16;
    LOSS_TRY(launch_rows_simt(p, status, s));
  }
  if (!dx) return cudaSuccess;
  GradProduct p = dx_product(c, L, entries);
  p.A = at<void>(ws, L.logits);
  p.B = (const char *)W + v0 * row;
  p.out = at<char>(ws, L.dx) + (size_t)i * c.n * row;
  return launch_grad_simt(&p, 1, grad_splits_simt(&p, 1), at<float>(ws, L.parts), status, s);
}

cudaError_t piece_gradient_pair(const moe_loss_config &c, const LossLayout &L, const void *W, int v0,
                                int entries, int i, bool dx, void *dW, void *ws, cudaStream_t s) {
  int *status = at<int>(ws, L.status);
  LossProduct p = pair_product(c, L, W, v0, entries, ws);
  LOSS_TRY(launch_loss_logit_grad(p, status, s));
  if (dW) {
    GradProduct g = dw_product(c, entries);
    g.offsets = p.range;
    g.A = p.dl;
    g.B = p.x;
    g.out = (char *)dW + (size_t)v0 * c.d * 2;
    const int splits = grad_splits(&g, 1);
    float *parts = at<float>(ws, L.parts);
    if (grads_small(&g, 1)) {
      LOSS_TRY(launch_grad_simt(&g, 1, splits, parts, status, s));
    } else {
      if (!gemm_grad_supported(g)) return cudaErrorNotSupported;
      LOSS_TRY(launch_gemm_grad(&g, 1, splits, parts, 0, status, s));
    }
  }
  if (!dx) return cudaSuccess;
  // (the last piece may be cut into fewer ranges, and adds to the first planes)
  p.splits = entries == L.piece ? L.planes : loss_dx_splits(c.n, c.d, entries, L.planes);
  p.add = i > 0;
  return launch_loss_dx(p, status, s);
}

}  // namespace

size_t loss_workspace(const moe_loss_config &c) { return loss_layout(c).total; }

cudaError_t launch_loss(const moe_loss_config &c, const void *x, const void *W,
                        const int32_t *targets, float *loss, float *lse, void *ws, cudaStream_t s) {
  const LossLayout L = loss_layout(c);
  if (L.pair && !loss_pair_supported(c)) return cudaErrorNotSupported;
  int *status = at<int>(ws, L.status);
  LOSS_TRY(launch_pack(c, L, x, targets, nullptr, nullptr, loss, lse, nullptr, ws, s));
  if (L.pair) {
    LOSS_TRY(launch_loss_sums(pair_product(c, L, W, 0, c.vocab, ws), status, s));
  } else {
    for (int v0 = 0; v0 < c.vocab; v0 += L.piece) {
      const int entries = c.vocab - v0 < L.piece ? c.vocab - v0 : L.piece;
      LOSS_TRY(piece_logits(c, L, W, v0, entries, ws, s));
      LOSS_TRY(launch_pdl(loss_chunk_kernel,
                          dim3((c.n + 31) / 32, (entries + L_CHUNK - 1) / L_CHUNK), dim3(256), 0, s,
                          at<float>(ws, L.logits), L.pitch, entries, v0, L.chunks,
                          at<int32_t>(ws, L.range), at<int32_t>(ws, L.target), at<float>(ws, L.at),
                          at<float2>(ws, L.sums), status));
    }
  }
  return launch_pdl(loss_finish_kernel, dim3((c.n + 7) / 8), dim3(256), 0, s,
                    at<float2>(ws, L.sums), L.chunks, c.z_loss, at<int32_t>(ws, L.range),
                    at<int32_t>(ws, L.list), at<float>(ws, L.at), loss, lse, status);
}

cudaError_t launch_loss_backward(const moe_loss_config &c, const void *x, const void *W,
                                 const int32_t *targets, const float *lse, const float *dloss,
                                 void *dx, void *dW, void *ws, cudaStream_t s) {
  const LossLayout L = loss_layout(c);
  if (L.pair && !loss_pair_supported(c)) return cudaErrorNotSupported;
  LOSS_TRY(launch_pack(c, L, x, targets, lse, dloss, nullptr, nullptr, dx, ws, s));
  auto piece = L.pair ? piece_gradient_pair : piece_gradient_simt;
  for (int v0 = 0, i = 0; v0 < c.vocab; v0 += L.piece, ++i) {
    const int entries = c.vocab - v0 < L.piece ? c.vocab - v0 : L.piece;
    LOSS_TRY(piece(c, L, W, v0, entries, i, dx != nullptr, dW, ws, s));
  }
  if (!dx) return cudaSuccess;
  if (c.dtype == MOE_F32) return finish_dx<float, float>(c, L, dx, ws, s);
  return L.pair ? finish_dx<__nv_bfloat16, float>(c, L, dx, ws, s)
                : finish_dx<__nv_bfloat16, __nv_bfloat16>(c, L, dx, ws, s);
}

}  // namespace moe
