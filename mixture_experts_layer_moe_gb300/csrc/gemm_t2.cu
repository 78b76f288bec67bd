// Grouped expert GEMM on a pair of SMs (tcgen05.mma.cta_group::2), weights on
// the MMA's M side and tokens on its N side.
//
// Each expert runs its FFN projection on its own dispatched segment ("How
// Mixture of Experts Scales Model Parameters", sections "Dense models" and
// "The forward pass: dispatch, then combine"):
//   out[q][j] = epi( sum_i A[q][i] * W_e[j][i] )   for q in segment e,
// computed as the transposed tile D[j][q] = sum_i W_e[j][i] * A[q][i]: 256
// weight rows j (MMA M, 128 in each CTA of a two-CTA cluster, one per TMEM
// lane) by up to 256 tokens q of the segment (MMA N: a segment splits into
// blocks of nearly equal size, rounded up to 16, so that a ragged segment
// costs MMAs as wide as its tokens and no tile is a thin remainder).  SwiGLU
// fuses h = silu(A W1^T) * (A W3^T) in the epilogue.
//
// Why a CTA pair: with M = 256 split over two SMs and the token tile split
// along N (each CTA stages half of the token rows, the MMA reads both halves),
// each SM stages 16 KB of weights and 16 KB of tokens per 64-wide k-block for
// a 128 x 256 x 64 share of the product, against 48 KB for the same share on
// one SM with a 128 x 256 tile: a third less shared-memory and L2 traffic per
// MMA cycle.
//
// Roles (persistent, one CTA per SM, clusters of two):
//   warp 0     TMA producer in both CTAs: this CTA's 128 weight rows and its
//              half of the token rows per stage (128-byte swizzle, 6 stages);
//              every copy signals the stage barrier of the pair's first CTA
//              (cp.async.bulk.tensor .cta_group::2), whose producer expects the
//              bytes of both.
//   warp 1     allocates 512 TMEM columns in both CTAs (cta_group::2); in the
//              first CTA one thread issues the MMAs (M 256, N <= 256, K 16) into
//              two accumulators of 256 columns and commits to the barriers of
//              both CTAs at once (multicast arrive).
//   warps 2..  epilogue in both CTAs: each drains its own TMEM lanes, applies
//              the activation, rounds to bf16 and stores the rows masked to the
//              segment, then arrives (remotely, for the second CTA) on the
//              first CTA's accumulator-empty barrier.
// For SwiGLU, a CTA's 128 weight rows are 64 rows of W1 (TMEM lanes 0..63)
// and the same 64 rows of W3 (lanes 64..127), each one 64-row TMA box (eight
// 16-row boxes interleaving them per lane quarter measured 29 % slower: the
// copy engine's cost grows with the number of boxes).  The epilogue warp of
// lane quarter q (W1) and that of quarter q + 2 (W3) then trade half of each
// 32-token chunk through shared memory, so each finishes 16 tokens with the
// gate value and the up value side by side; a tile has 128 output columns (64
// per CTA), otherwise 256 (128 per CTA).
//
// Training runs on the same kernel.  The forward may keep both products beside
// h (EPI 5).  A gradient multiplies by the weights as the forward stores them
// (dh = dy W2 reduces over W2's rows): they enter as an M-major operand (WROWS),
// and dx = dg W1 + du W3 sums both pairs into one accumulator.  dg and du are
// formed in the epilogue of dh (EPI 7; EPI 6 for the ReLU) from the kept rows.
// Measured one launch at a time on 2048 rows of 2 experts, d 4096, d_ff 14336:
// up with kept products 1725 TFLOP/s, down 1630, dg and du 1442, dx 1696
// (tensor pipe 79, 73, 63 and 77 % active).
//
// Tiles are ordered expert-major, then weight block, then token block, so the
// clusters running together share one expert's weight block and segment in
// L2 (token block, then weight block, when a segment outweighs its weights).
// Pair p takes tiles p, p + pairs, ...  (An atomic tile counter, which kept
// the pairs sharing a weight block in step and cut the fine-grained up
// projection's DRAM reads from 22.4 to 18.0 GB, measured 5-7 % slower.)  The
// tile list comes from the segment offsets on the device; empty segments give
// no tiles.
#include "common.cuh"
#include "gate_math.cuh"
#include "launch.h"
#include "pair_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace pair;

constexpr int PM = 128;                         // weight rows per CTA (MMA M = 256 per pair)
constexpr int PN = 256;                         // tokens per tile at most (MMA N)
constexpr int PN_SHORT = 32;                    // token rows of a short box
constexpr int PK = 64;                          // k-block
constexpr int PS = 6;                           // pipeline stages
constexpr int P_B_BYTES = (PN / 2) * PK * 2;    // this CTA's half of the token tile: 16 KB
constexpr int P_A_BYTES = PM * PK * 2;          // this CTA's weight rows: 16 KB
constexpr int P_STAGE = P_B_BYTES + P_A_BYTES;  // 32 KB (tokens first, then weights)
// epilogue warps: one to three per TMEM lane quarter, which take turns of 32
// tokens (16 for a gradient).  A training epilogue moves two to four values per
// product; where the reduction is short it is what bounds the kernel (64
// experts of 512 rows, d = d_ff = 1024: up projection 155 -> 133 us with 8
// warps, dg and du 183 -> 132 with 8 and 120 with 12).
template <int EPI>
constexpr int epi_warps() { return EPI == 6 || EPI == 7 ? 12 : EPI == 5 ? 8 : 4; }
template <int EPI>
constexpr int pair_threads() { return 32 * (2 + epi_warps<EPI>()); }
constexpr uint32_t P_TMEM_COLS = 512;           // two accumulators of PN columns
constexpr int P_MAX_E = 256;
// SwiGLU exchange: two chunk buffers per column half (two warp pairs with one
// buffer each, or one pair with two, alternating), each with 16 values per
// lane going each way; rows of 17 floats avoid bank conflicts
constexpr int P_XROW = 17;
constexpr int P_XBUF = 32 * P_XROW;              // floats of one direction of one chunk
constexpr size_t P_XBYTES = (size_t)2 * 2 * 2 * P_XBUF * 4;   // halves x buffers x directions
constexpr size_t P_DYN_SMEM = 1024 + (size_t)PS * P_STAGE + P_XBYTES;
static_assert(P_STAGE % 1024 == 0, "stage alignment");

struct PShared {
  uint64_t full[PS];    // first CTA: tokens + weights of both CTAs landed
  uint64_t empty[PS];   // both CTAs: the MMAs that read the stage completed
  uint64_t tfull[2];    // both CTAs: the accumulator's MMAs completed
  uint64_t tempty[2];   // first CTA: both CTAs' epilogues drained the accumulator
  uint64_t drain;
  uint32_t tmem_base;
  int abort, failed_on_entry, num_tiles;
  int offs[P_MAX_E + 1];
  int tile_start[P_MAX_E];
};

struct PArgs {
  const int32_t *offsets;  // nullptr: one segment [0, rows) of expert 0
  int num_experts;
  int rows;                // token rows of A (and of out)
  int K;
  int N;                   // output columns (weight rows of W, and of W3 for SwiGLU)
  __nv_bfloat16 *out;      // [rows][N]
  int *status;
  int tok_major;           // 1: token block outer, weight block fastest
  int pairs;               // operand pairs summed (2: out = A W + A2 W2, EPI 0 on row-stored weights)
  // training: what the forward keeps (EPI 5) and what a gradient reads and adds (EPI 6, 7), [rows][N]
  __nv_bfloat16 *out_g, *out_u;
  const uint16_t *g, *u, *h;
  // EPI 8: fp32 partial sums parts[mat][split][rows][N] of `splits` ranges of
  // the reduction, for one or two weight matrices
  float *parts;
  int splits, mats;
  // 1: runs beside the kernel before, whose results it does not read (that
  // kernel lets it start once all before are complete), and ends after it
  int beside;
};

// Tensor maps of the token rows (whole boxes, and the short ones for blocks of
// at most 2 * PN_SHORT tokens), of the second pair's rows, and of the weights.
struct PMaps {
  CUtensorMap X, Xs, X2, X2s, W, W3;
};

struct PTile {
  int e, tok0, ntok, seg_end, wb;
  int mat, split;   // EPI 8
  int kb0, kb1;     // k-blocks
};

// Tokens per block of a segment of c tokens: the segment splits into
// ceil(c / PN) blocks of nearly equal size, rounded up to 16 (the MMA's N
// step), so that no block is a thin remainder.  A tile's weight copies cost
// the same whatever its N, and a thin block's MMAs are too short to hide them.
__device__ __forceinline__ int block_tokens(int c) {
  const int nb = max(1, (c + PN - 1) / PN);
  return ((c + nb - 1) / nb + 15) & ~15;
}
__device__ __forceinline__ int token_blocks(int c) {
  return c > 0 ? (c + block_tokens(c) - 1) / block_tokens(c) : 0;
}

__device__ __forceinline__ PTile p_decode(const PShared &sh, int E, int t, int n_wb,
                                          bool tok_major) {
  int lo = 0, hi = E;   // largest e with tile_start[e] <= t (skips empty experts)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sh.tile_start[mid] <= t) lo = mid; else hi = mid;
  }
  PTile tl;
  tl.e = lo;
  const int beg = sh.offs[lo], end = sh.offs[lo + 1];
  const int bt = block_tokens(end - beg);
  const int m_tiles = token_blocks(end - beg);
  const int local = t - sh.tile_start[lo];
  // weight-major: token blocks fastest, so pairs running side by side share a
  // weight block; token-major (a segment larger than its weights, e.g. the
  // shared expert's 16k tokens): weight blocks fastest, so the weights stay
  // in L2 and each token block comes from DRAM once
  int tb;
  if (tok_major) {
    tb = local / n_wb;
    tl.wb = local - tb * n_wb;
  } else {
    tl.wb = local / m_tiles;
    tb = local - tl.wb * m_tiles;
  }
  tl.tok0 = beg + tb * bt;
  tl.ntok = min(bt, end - tl.tok0);
  tl.seg_end = min(end, tl.tok0 + bt);
  return tl;
}

// Kept rows of a gradient's epilogue: this thread's column of 16 tokens (h for
// the ReLU, g and u for SwiGLU; 0 outside the segment).
constexpr int KEPT = 16;
template <int EPI>
__device__ __forceinline__ void load_kept(const PArgs &args, int tok0, int end, int col, bool col_ok,
                                          uint16_t (&kg)[KEPT], uint16_t (&ku)[KEPT]) {
  const size_t at = (size_t)tok0 * args.N + col;
  const uint16_t *g = (EPI == 6 ? args.h : args.g) + at, *u = args.u + at;
#pragma unroll
  for (int i = 0; i < KEPT; ++i) {
    const bool ok = col_ok && tok0 + i < end;
    kg[i] = ok ? __ldg(g + (size_t)i * args.N) : (uint16_t)0;
    if constexpr (EPI == 7) ku[i] = ok ? __ldg(u + (size_t)i * args.N) : (uint16_t)0;
  }
}

// EPI: 0 plain, 1 relu, 2 swiglu (W = W1 rows, W3 = W3 rows), 5 swiglu that
// also stores both products, 6 relu gradient, 7 swiglu gradient, 8 fp32 partial
// sums of a range of the reduction.
// WROWS: the weights are stored with the output column contiguous ([E][K][N],
// the forward's weights as their gradients read them): the MMA takes them as
// an M-major operand, staged as two boxes of 64 columns x 64 reduction rows
// (128-byte swizzle, the boxes 8 KB apart), and no transposed copy is made.
template <int EPI, bool WROWS>
__global__ void __launch_bounds__(pair_threads<EPI>(), 1)
gemm_t2_kernel(const __grid_constant__ PMaps maps, const PArgs args) {
  constexpr bool GATED = EPI == 2 || EPI == 5;        // two weight matrices side by side
  constexpr int P_EPI = epi_warps<EPI>(), P_THREADS = pair_threads<EPI>(), TURNS = P_EPI / 4;
  static_assert(!WROWS || !GATED, "the gated forward reads weights stored by output column");
  constexpr int OUT_CTA = GATED ? PM / 2 : PM;        // output columns per CTA per tile
  constexpr int OUT_TILE = 2 * OUT_CTA;
  extern __shared__ uint8_t dyn_smem[];
  __shared__ PShared sh;
  uint8_t *smem = dyn_smem + ((1024 - (tc::smem_u32(dyn_smem) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int E = args.offsets ? args.num_experts : 1;
  // weight blocks of a matrix, and all that a token block meets (with EPI 8 a
  // block is its matrix's, then split by ranges of the reduction)
  const int n_wb1 = (args.N + OUT_TILE - 1) / OUT_TILE;
  const int n_wb = EPI == 8 ? n_wb1 * args.mats * args.splits : n_wb1;
  const int KB1 = (args.K + PK - 1) / PK;             // k-blocks of one operand pair
  const int KB = WROWS ? KB1 * args.pairs : KB1;
  const int KBS = EPI == 8 ? (KB + args.splits - 1) / args.splits : KB;   // of one range
  auto decode = [&](int t) {
    PTile tl = p_decode(sh, E, t, n_wb, args.tok_major != 0);
    tl.mat = 0;
    tl.split = 0;
    if constexpr (EPI == 8) {
      tl.split = tl.wb % args.splits;
      tl.wb /= args.splits;
      tl.mat = tl.wb / n_wb1;
      tl.wb -= tl.mat * n_wb1;
    }
    tl.kb0 = tl.split * KBS;
    tl.kb1 = min(KB, tl.kb0 + KBS);
    return tl;
  };

  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&maps.X);
    tc::prefetch_tmap(&maps.Xs);
    tc::prefetch_tmap(&maps.W);
    if (GATED || WROWS || EPI == 8) tc::prefetch_tmap(&maps.W3);
    if (WROWS) {
      tc::prefetch_tmap(&maps.X2);
      tc::prefetch_tmap(&maps.X2s);
    }
  }
  if (warp == 1) tmem_alloc2(&sh.tmem_base, P_TMEM_COLS);
  if (threadIdx.x == 32) {
    for (int s = 0; s < PS; ++s) {
      tc::mbar_init(&sh.full[s], 1);
      tc::mbar_init(&sh.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&sh.tfull[a], 1);
      tc::mbar_init(&sh.tempty[a], 2 * P_EPI);   // one arrival per epilogue warp of each CTA
    }
    tc::mbar_init(&sh.drain, 1);
    tc::fence_mbar_init();
  }
  // (all above ran beside the end of the kernel before; from here on its
  // results are read)
  if (!WROWS || !args.beside) pdl_wait();
  if (threadIdx.x == 0) {
    sh.failed_on_entry = status_failed(args.status) ? 1 : 0;
    sh.abort = sh.failed_on_entry;
  }
  for (int i = threadIdx.x; i <= E; i += P_THREADS)
    sh.offs[i] = args.offsets ? args.offsets[i] : (i == 0 ? 0 : args.rows);
  __syncthreads();
  if (warp == 0) {
    // tile prefix over experts: lane l owns experts 8l .. 8l+7
    int cnt[8];
    int sum = 0, bad = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      cnt[i] = 0;
      if (e < E) {
        const int b = sh.offs[e], en = sh.offs[e + 1];
        if (b < 0 || en < b || en > args.rows) bad = 1;
        else cnt[i] = token_blocks(en - b) * n_wb;
      }
      sum += cnt[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      if (e < E) sh.tile_start[e] = run;
      run += cnt[i];
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      sh.num_tiles = bad ? 0 : total;
      if (bad && rank == 0) set_status(args.status, MOE_ERR_BAD_INDEX, -1);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  // both CTAs' barriers are initialised before either CTA touches the other's
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;
  const int num_tiles = sh.num_tiles;
  volatile int *abort = &sh.abort;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t used = 0, used_phase = 0;   // bit s: stage s was used, in which phase last
      const uint32_t full0 = map_to_rank(tc::smem_u32(&sh.full[0]), 0);
      for (int t = pair; t < num_tiles && !*abort; t += n_pairs) {
        const PTile tl = decode(t);
        const int ntok = tl.ntok;
        const int half = ((ntok + 15) & ~15) >> 1;   // tokens staged by each CTA
        // few tokens take a short box: whole ones would be half of what this
        // SM copies, beside the weights that a block of few tokens waits for
        // (one token, d 4096, d_ff 14336, one expert, forward: 99 -> 78 us)
        const bool few = half <= PN_SHORT;
        const uint32_t bytes = 2u * (P_A_BYTES + (few ? PN_SHORT : PN / 2) * PK * 2);
        const CUtensorMap *x1 = few ? &maps.Xs : &maps.X, *x2 = few ? &maps.X2s : &maps.X2;
        const int brow = tl.tok0 + (int)rank * half;
        const int wrow = tl.wb * OUT_TILE + (int)rank * OUT_CTA;
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!tc::mbar_wait(&sh.empty[stage], phase ^ 1u, abort)) break;
          uint8_t *sb = smem + stage * P_STAGE;
          uint8_t *sa = sb + P_B_BYTES;
          const uint32_t bar = full0 + (uint32_t)stage * 8;
          used |= 1u << stage;
          used_phase = phase ? used_phase | 1u << stage : used_phase & ~(1u << stage);
          if (rank == 0) tc::mbar_arrive_expect_tx(&sh.full[stage], bytes);   // of both CTAs
          if constexpr (WROWS) {
            const bool second = kb >= KB1;
            const int k0 = (second ? kb - KB1 : kb) * PK;
            const CUtensorMap *w = second ? &maps.W3 : &maps.W;
            tma2_load_2d(second ? x2 : x1, bar, sb, k0, brow);
            tma2_load_3d(w, bar, sa, wrow, k0, tl.e);                       // columns 0..63
            tma2_load_3d(w, bar, sa + P_A_BYTES / 2, wrow + 64, k0, tl.e);  // columns 64..127
          } else if constexpr (GATED) {
            tma2_load_2d(x1, bar, sb, kb * PK, brow);
            tma2_load_3d(&maps.W, bar, sa, kb * PK, wrow, tl.e);                    // rows 0..63
            tma2_load_3d(&maps.W3, bar, sa + P_A_BYTES / 2, kb * PK, wrow, tl.e);   // rows 64..127
          } else {
            tma2_load_2d(x1, bar, sb, kb * PK, brow);
            tma2_load_3d(EPI == 8 && tl.mat ? &maps.W3 : &maps.W, bar, sa, kb * PK, wrow, tl.e);
          }
          if (++stage == PS) { stage = 0; phase ^= 1u; }
        }
      }
      if (*abort && rank == 0) {
        // let the copies in flight land before the pair exits (the second
        // CTA's copies count on these barriers too)
        for (int s = 0; s < PS; ++s)
          if ((used >> s) & 1u)
            tc::mbar_wait_drain(&sh.full[s], (used_phase >> s) & 1u, 100000000ull);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (first CTA of the pair)
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      // descriptors of stage 0; an MMA's own differ in the low words, in units
      // of 16 bytes (building them anew for every MMA left the tensor pipe
      // waiting for this thread)
      const uint32_t sb0 = tc::smem_u32(smem);
      const uint64_t b_desc = tc::smem_desc_sw128(sb0);
      const uint64_t a_desc = WROWS ? tc::smem_desc_sw128_mn(sb0 + P_B_BYTES, P_A_BYTES / 2)
                                    : tc::smem_desc_sw128(sb0 + P_B_BYTES);
      const uint32_t a_lo = (uint32_t)a_desc, a_hi = (uint32_t)(a_desc >> 32);
      const uint32_t b_lo = (uint32_t)b_desc, b_hi = (uint32_t)(b_desc >> 32);
      for (int t = pair; t < num_tiles && ok && !*abort; t += n_pairs, ++local) {
        const PTile tl = decode(t);
        const int ntok = tl.ntok;
        const uint32_t idesc =
            tc::idesc_bf16_f32(2 * PM, (ntok + 15) & ~15) | (WROWS ? tc::kIdescAMajorMN : 0u);
        const int acc = local & 1;
        if (!mbar_wait_cluster(&sh.tempty[acc], ((local >> 1) & 1) ^ 1u, abort)) { ok = false; break; }
        tc::tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * PN);
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!tc::mbar_wait(&sh.full[stage], phase, abort)) { ok = false; break; }
          tc::tc_fence_after();
          const uint32_t at = (uint32_t)(stage * (P_STAGE / 16));
#pragma unroll
          for (int k = 0; k < PK / 16; ++k)
            mma2_bf16_lo(d_tmem, a_lo + at + k * (WROWS ? 128 : 2), a_hi, b_lo + at + k * 2, b_hi,
                         idesc, (kb != tl.kb0 || k != 0) ? 1u : 0u);
          mma2_commit_both(&sh.empty[stage]);
          if (++stage == PS) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        mma2_commit_both(&sh.tfull[acc]);
      }
      if (*abort) {
        mma2_commit_self(&sh.drain);
        tc::mbar_wait_drain(&sh.drain, 0, 100000000ull);
      }
    }
  } else {
    // ---------------- epilogue (both CTAs): warp w drains TMEM lanes 32*(w%4) .. +31
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const int pq = quarter & 1;                  // SwiGLU: W1 quarter pq pairs with W3 quarter pq + 2
    const bool w3 = quarter >= 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tempty_first = map_to_rank(tc::smem_u32(&sh.tempty[0]), 0);
    float *xbuf = reinterpret_cast<float *>(smem + (size_t)PS * P_STAGE);
    int local = 0;
    for (int t = pair; t < num_tiles; t += n_pairs, ++local) {
      const PTile tl = decode(t);
      const int ntok = tl.ntok;
      const int acc = local & 1;
      // this thread's output column
      const int col =
          tl.wb * OUT_TILE + (int)rank * OUT_CTA + (GATED ? pq : quarter) * 32 + lane;
      const bool col_ok = col < args.N;
      uint16_t *o = reinterpret_cast<uint16_t *>(args.out) + col;
      float *plane =
          args.parts + (size_t)(tl.mat * args.splits + tl.split) * args.rows * args.N + col;   // EPI 8
      // a gradient's kept rows: the first chunk is in flight during the wait
      uint16_t kg[KEPT], ku[KEPT];
      if constexpr (EPI == 6 || EPI == 7)
        load_kept<EPI>(args, tl.tok0 + part * KEPT, tl.seg_end, col, col_ok, kg, ku);
      const bool ok = tc::mbar_wait(&sh.tfull[acc], (local >> 1) & 1, abort);
      if constexpr (GATED) {
        // the two warps of a pair meet on named barriers below: they agree on
        // going on first (a warp whose wait ran out has raised *abort)
        if (tc::bar_or(1 + pq + 2 * part, 64, !ok)) break;
      } else {
        if (!__all_sync(0xffffffffu, ok)) break;
      }
      tc::tc_fence_after();
      const uint32_t tb = lane_base + (uint32_t)(acc * PN);
      if constexpr (EPI == 6 || EPI == 7) {
        // 16 tokens at a time: the next ones' kept rows are in flight while
        // these are formed and stored
#pragma unroll 1
        for (int c = part; c * KEPT < ntok; c += TURNS) {
          uint32_t a[KEPT];
          tc::tmem_ld16(tb + (uint32_t)(c * KEPT), a);
          tc::tmem_ld_wait();
          const int tok0 = tl.tok0 + c * KEPT;
          uint16_t dg[KEPT], du[KEPT];
#pragma unroll
          for (int i = 0; i < KEPT; ++i) {
            const float v = __uint_as_float(a[i]);
            if constexpr (EPI == 6) {
              dg[i] = bf16_value(kg[i]) > 0.f ? bf16_bits(v) : (uint16_t)0;
            } else {
              float a_g, a_u;
              swiglu_grad(v, bf16_value(kg[i]), bf16_value(ku[i]), a_g, a_u);
              dg[i] = bf16_bits(a_g);
              du[i] = bf16_bits(a_u);
            }
          }
          load_kept<EPI>(args, tok0 + KEPT * TURNS, tl.seg_end, col, col_ok, kg, ku);
          if (col_ok) {
            uint16_t *og = o + (size_t)tok0 * args.N;
            uint16_t *ou = reinterpret_cast<uint16_t *>(args.out_u) + (size_t)tok0 * args.N + col;
#pragma unroll
            for (int i = 0; i < KEPT; ++i) {
              if (tok0 + i < tl.seg_end) {
                og[(size_t)i * args.N] = dg[i];
                if constexpr (EPI == 7) ou[(size_t)i * args.N] = du[i];
              }
            }
          }
        }
      } else {
#pragma unroll 1
        for (int c = part; c * 32 < ntok; c += TURNS) {
          uint32_t a[32];
          tc::tmem_ld32(tb + (uint32_t)(c * 32), a);
          tc::tmem_ld_wait();
          const int tok0 = tl.tok0 + c * 32;
          if constexpr (GATED) {
            // the W1 warp (gate values) finishes tokens 0..15 of the chunk, the
            // W3 warp (up values) tokens 16..31; each hands the other its half
            // (buffer c & 1: alternating for one pair, one for each of two)
            float *to_w3 = xbuf + (size_t)((pq * 2 + (c & 1)) * 2) * P_XBUF;   // gates 16..31
            float *to_w1 = to_w3 + P_XBUF;                                    // ups 0..15
            float *mine = w3 ? to_w1 : to_w3;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              mine[lane * P_XROW + i] = __uint_as_float(w3 ? a[i] : a[16 + i]);
            asm volatile("bar.sync %0, 64;" ::"r"(5 + pq + 2 * part) : "memory");
            const float *theirs = w3 ? to_w3 : to_w1;
            uint16_t hv[16], gv[EPI == 5 ? 16 : 1], uv[EPI == 5 ? 16 : 1];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float other = theirs[lane * P_XROW + i];
              const float g = w3 ? other : __uint_as_float(a[i]);
              const float u = w3 ? __uint_as_float(a[16 + i]) : other;
              hv[i] = bf16_bits(silu_mul(g, u));
              if constexpr (EPI == 5) {
                gv[i] = bf16_bits(g);
                uv[i] = bf16_bits(u);
              }
            }
            const int tsub = w3 ? 16 : 0;
            // a pair with one buffer: both have read it before either writes again
            if (TURNS == 2) asm volatile("bar.sync %0, 64;" ::"r"(9 + pq + 2 * part) : "memory");
            if (col_ok) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int tok = tok0 + tsub + i;
                if (tok < tl.seg_end) {
                  o[(size_t)tok * args.N] = hv[i];
                  if constexpr (EPI == 5) {
                    reinterpret_cast<uint16_t *>(args.out_g)[(size_t)tok * args.N + col] = gv[i];
                    reinterpret_cast<uint16_t *>(args.out_u)[(size_t)tok * args.N + col] = uv[i];
                  }
                }
              }
            }
          } else {
            if (col_ok) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float v = __uint_as_float(a[i]);
                if constexpr (EPI == 1) v = relu(v);
                const int tok = tok0 + i;
                if (tok >= tl.seg_end) continue;
                if constexpr (EPI == 8) plane[(size_t)tok * args.N] = v;
                else o[(size_t)tok * args.N] = bf16_bits(v);
              }
            }
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty_first + (uint32_t)(acc * sizeof(uint64_t)));
    }
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  // neither CTA leaves (or frees its tensor memory) while the other may still
  // read its shared memory, signal its barriers or write its tensor memory
  cluster_sync();
  if (warp == 1) {
    tc::tc_fence_after();
    tmem_dealloc2(tmem_base, P_TMEM_COLS);
  }
  if (threadIdx.x == 0 && sh.abort && !sh.failed_on_entry)
    set_status(args.status, MOE_ERR_TIMEOUT, blockIdx.x);
  if (WROWS && args.beside) pdl_wait();
}

int pairs_resident(const void *kernel, int threads, size_t smem) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (num_sms() / 2));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = num_sms() / 2;
  }
  return n;
}

template <int EPI, bool WROWS>
cudaError_t launch_t2(const GemmStage &g, int *status, cudaStream_t s) {
  constexpr bool GATED = EPI == 2 || EPI == 5;
  static int pairs = 0;
  if (pairs == 0) {
    cudaError_t e = cudaFuncSetAttribute(gemm_t2_kernel<EPI, WROWS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)P_DYN_SMEM);
    if (e != cudaSuccess) return e;
    pairs = pairs_resident(reinterpret_cast<const void *>(gemm_t2_kernel<EPI, WROWS>),
                           pair_threads<EPI>(), P_DYN_SMEM);
  }
  const int E = g.offsets ? g.num_experts : 1;
  PMaps m;
  auto bf16_map = [](CUtensorMap *m, const void *p, int rank, const uint64_t *dims,
                     const uint32_t *box) {
    return make_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, rank, dims, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  };
  const uint64_t dX[2] = {(uint64_t)(g.lda ? g.lda : g.K), (uint64_t)g.rows};
  const uint32_t bX[2] = {PK, PN / 2}, bXs[2] = {PK, PN_SHORT};
  // weights by output column: boxes of 64 reduction elements x 128 (64) rows;
  // by reduction row: boxes of 64 columns x 64 reduction rows
  const uint64_t dW[3] = {(uint64_t)(WROWS ? g.N : g.K), (uint64_t)(WROWS ? g.K : g.N),
                          (uint64_t)E};
  const uint32_t bW[3] = {PK, (uint32_t)(WROWS ? PK : GATED ? PM / 2 : PM), 1};
  if (!bf16_map(&m.X, g.A, 2, dX, bX) || !bf16_map(&m.Xs, g.A, 2, dX, bXs) ||
      !bf16_map(&m.W, g.B, 3, dW, bW))
    return cudaErrorInvalidValue;
  m.W3 = m.W;
  m.X2 = m.X;
  m.X2s = m.Xs;
  if (g.B3 && !bf16_map(&m.W3, g.B3, 3, dW, bW)) return cudaErrorInvalidValue;
  if (g.A2 && (!bf16_map(&m.X2, g.A2, 2, dX, bX) || !bf16_map(&m.X2s, g.A2, 2, dX, bXs)))
    return cudaErrorInvalidValue;
  PArgs a{};
  a.offsets = g.offsets;
  a.num_experts = g.num_experts;
  a.rows = g.rows;
  a.K = g.K;
  a.N = g.N;
  a.out = static_cast<__nv_bfloat16 *>(g.out);
  a.status = status;
  a.pairs = g.A2 ? 2 : 1;
  a.out_g = static_cast<__nv_bfloat16 *>(g.out_g);
  a.out_u = static_cast<__nv_bfloat16 *>(g.out_u);
  a.g = static_cast<const uint16_t *>(g.kept_g);
  a.u = static_cast<const uint16_t *>(g.kept_u);
  a.h = static_cast<const uint16_t *>(g.kept_h);
  a.parts = g.parts;
  a.splits = g.splits;
  a.mats = g.mats;
  a.beside = g.beside;
  // token blocks outer when an average segment holds more rows than the
  // weights it meets (the shared expert's one segment of all n tokens)
  const long seg_rows = (long)g.rows / (E > 0 ? E : 1);
  a.tok_major = seg_rows > (long)g.N * (GATED ? 2 : 1) ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (g.beside ? g.beside : pairs));
  cfg.blockDim = dim3(pair_threads<EPI>());
  cfg.dynamicSmemBytes = P_DYN_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // the forward's products start beside the end of the kernel before (18.1
  // against 22.6 us for 200 tokens, 62.0 against 67.5 for 1024 x 2 of 16
  // experts, d 1024, d_ff 2048); the gradients' measured slower so (150.4
  // against 154.2 us for the latter's backward)
  cfg.numAttrs = WROWS && !g.beside ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, gemm_t2_kernel<EPI, WROWS>, m, a);
}

}  // namespace

bool gemm_t2_supported(const GemmStage &g) {
  const bool epi_ok =
      g.epi == kEpiPartial ||
      (g.w_rows ? g.epi == 0 || g.epi == kEpiReluGrad || g.epi == kEpiSwigluGrad
                : (g.epi >= 0 && g.epi <= 2) || g.epi == kEpiSwigluKeep);
  return g.rows > 0 && tensor_maps_available() && g.a_dtype == MOE_BF16 &&
         g.b_dtype == MOE_BF16 && g.out_dtype == MOE_BF16 && epi_ok && g.num_experts <= P_MAX_E &&
         (g.lda ? g.lda : g.K) % 8 == 0 && g.N % 8 == 0 && num_sms() >= 2;
}

cudaError_t launch_gemm_t2(const GemmStage &g, int *status, cudaStream_t s) {
  if (g.w_rows) {
    switch (g.epi) {
      case kEpiReluGrad: return launch_t2<kEpiReluGrad, true>(g, status, s);
      case kEpiSwigluGrad: return launch_t2<kEpiSwigluGrad, true>(g, status, s);
      case kEpiPartial: return launch_t2<kEpiPartial, true>(g, status, s);
      default: return launch_t2<0, true>(g, status, s);
    }
  }
  switch (g.epi) {
    case 1: return launch_t2<1, false>(g, status, s);
    case 2: return launch_t2<2, false>(g, status, s);
    case kEpiSwigluKeep: return launch_t2<kEpiSwigluKeep, false>(g, status, s);
    case kEpiPartial: return launch_t2<kEpiPartial, false>(g, status, s);
    default: return launch_t2<0, false>(g, status, s);
  }
}

}  // namespace moe
