// Weight gradients of the grouped products on a pair of SMs
// (tcgen05.mma.cta_group::2): for every expert e
//   out_e[m][c] = sum_{q in segment e} A[q][m] * B[q][c],
// zero for a segment without rows.  dW2 = dy^T h, dW1 = dg^T x and
// dW3 = du^T x of an expert (up to three such problems) share one launch, so
// that only the last wave of the whole list is partly filled.
//
// The reduction runs over the segment's rows, which both operands store
// strided: the MMA takes both as M-/N-major operands, staged as boxes of 64
// columns x 64 rows (128-byte swizzle), and no transposed copy is made.  The
// tile is D[m][c]: 256 output rows m on M (one per TMEM lane, 128 per CTA), up
// to 256 output columns c on N, so that a thread of the epilogue holds
// neighbouring elements of one output row: it packs them to 16 bytes, and each
// warp hands 32 rows x 64 columns at a time to a TMA store (clipped at the
// matrix's edge).  With m and c the other way round,
// a thread's elements lie a row apart, and 2-byte stores took 9.5 us a tile:
// 2.70 ms for the gradients of 32 experts (d 7168, d_ff 2048) with 18 rows
// each, against 0.65 so, which is what filling 2.8 GB with one value takes here
// (4.06 TB/s: HBM writes alone run slower than a copy).
//
// A segment ends anywhere: the last k-block of a tile reads into the next
// segment (or past the array, where the copy fills zeros).  Steps of 16 rows
// beyond the end are not issued; the rows between the end and the next
// multiple of 16 are zeroed in shared memory, in both operands (a stray NaN
// times zero would be NaN).  A k-block that needs this lands on a barrier of
// its own in each CTA; a fixer warp per CTA zeroes the rows, makes the writes
// visible to the async proxy, and the first CTA's fixer, once it has heard
// from the second's, completes the stage's barrier that the MMA waits on.
//
// Few tiles (a router's gradient: experts x d) leave SM pairs idle.  Then each
// segment is cut into `splits` runs of rows: the tiles of a run store fp32
// partial sums, and a second launch adds them in order and rounds once.
//
// A_K: the same tile for out[t][c] = sum_k A[t][k] B[k][c] over one segment,
// A's reduction index contiguous (the router's share of its dx: short reductions,
// where the store of the result is the work, and this epilogue's packed stores
// are what that needs).
//
// ADD, with A_K: plus sum_{j < add_k} add[add_inv[t * add_k + j]][c], the
// gradients of the token's expert rows, in the same fp32 sum, rounded once.  The
// gathered rows are the work then, so two pipeline stages feed the MMAs and the
// rest of shared memory is a ring of gathered pieces per epilogue warp, 112 KB
// in flight per SM (GatherRing).  16384 tokens, d 7168, 8 rows each, 256 experts:
// 404 us, 5.3 TB/s; one launch that stores dl Wg and one that sums took 434 and
// rounded dl Wg to bf16 in between.  (Gathering into registers instead, 8 or 16
// epilogue warps: 520 to 770 us.)
//
// Roles (persistent, one CTA per SM, clusters of two): warp 0 TMA producer in
// both CTAs, warp 1 of the first CTA issues the MMAs into two accumulators of
// 256 columns, warps 2-9 drain them (two warps per lane quarter, taking turns
// of 64 columns), warp 10 is the fixer.
#include "common.cuh"
#include "launch.h"
#include "pair_common.cuh"
#include "tc_common.cuh"
#include "train.h"
#include "vec16.cuh"

namespace moe {
namespace {

using namespace pair;

constexpr int GM = 128;                       // output rows per CTA (MMA M = 256 per pair)
constexpr int GN = 256;                       // output columns per tile at most (MMA N)
constexpr int GK = 64;                        // segment rows per k-block
constexpr int GS = 6;                         // pipeline stages
constexpr int g_stages(bool add) { return add ? 2 : GS; }
constexpr int G_BOX = 64 * GK * 2;            // one 64 x 64 box: 8 KB
constexpr int G_STAGE = 4 * G_BOX;            // two boxes of B (N side), two of A (M side)
constexpr int G_EPI = 8;                      // epilogue warps: two per TMEM lane quarter
constexpr int G_THREADS = 32 * (3 + G_EPI);
constexpr uint32_t G_TMEM_COLS = 512;
constexpr int G_MAX_E = 256;
constexpr int G_OUT = 32 * 128;               // one store: 32 rows x 64 columns, 128-byte swizzle
// ADD: a ring of G_RING such pieces per epilogue warp, each 32 gathered rows x 64
// columns
constexpr int G_RING = 4;
constexpr size_t g_dyn_smem(bool add) {
  return 1024 + (size_t)g_stages(add) * G_STAGE + (size_t)G_EPI * G_OUT * (add ? 1 + G_RING : 1);
}

struct GShared {
  uint64_t full[GS];        // first CTA: both CTAs' boxes landed (and were fixed)
  uint64_t empty[GS];       // both CTAs: the MMAs that read the stage completed
  uint64_t tail_full[GS];   // this CTA's boxes of a k-block that needs fixing landed
  uint64_t peer_fixed[GS];  // first CTA: the second CTA's fixer is done
  uint64_t tfull[2], tempty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort, failed_on_entry, bad;
  int offs[G_MAX_E + 1];
};

struct GArgs {
  const int32_t *offsets;
  int num_experts, rows, problems;
  int M[kMaxGradProblems], N[kMaxGradProblems];
  int first[kMaxGradProblems + 1];   // an expert's tiles before problem i
  int width;                         // output columns per tile
  int splits;                        // runs of rows per segment
  int beside;                        // 1: the next kernel runs beside this one
  int *status;
  // ADD: the rows added to the output ([M * add_k][N]).  An index outside them is
  // skipped.
  const uint4 *add;
  const int32_t *add_inv;
  int add_k;
};
struct GMaps {
  CUtensorMap a[kMaxGradProblems], b[kMaxGradProblems], out[kMaxGradProblems];
};

struct GTile {
  int e, prob, m0, c0, nc, beg, len;   // nc columns from c0
  int z;                               // the output matrix
};

template <bool SPLIT>
__device__ __forceinline__ GTile g_decode(const GShared &sh, const GArgs &args, int t) {
  GTile tl;
  const int per = args.first[args.problems];
  const int z = t / per;               // the expert, or expert * splits + run
  tl.e = SPLIT ? z / args.splits : z;
  int r = t - z * per;
  tl.prob = 0;
  while (tl.prob + 1 < args.problems && r >= args.first[tl.prob + 1]) ++tl.prob;
  r -= args.first[tl.prob];
  const int cols = (args.N[tl.prob] + args.width - 1) / args.width;
  const int mb = r / cols;
  tl.m0 = mb * 2 * GM;
  tl.c0 = (r - mb * cols) * args.width;
  tl.nc = min(args.width, args.N[tl.prob] - tl.c0);
  tl.beg = sh.offs[tl.e];
  tl.len = sh.offs[tl.e + 1] - tl.beg;
  tl.z = z;
  if (SPLIT) {
    // runs of whole k-blocks
    const int run = ((tl.len + args.splits - 1) / args.splits + GK - 1) / GK * GK;
    const int from = min(tl.len, (z - tl.e * args.splits) * run);
    tl.beg += from;
    tl.len = min(run, tl.len - from);
  }
  return tl;
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ uint32_t bf16x2_bits(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t *>(&h);
}

// ADD: the rows that one epilogue warp adds, in the order in which it adds them
// (tile, 64 columns, slot), copied asynchronously into its ring G_RING steps
// ahead, across the tiles' borders.  A step is 32 rows x 64 columns, laid out as a
// store's piece: row r's 16-byte vector v at 128 r + 16 (v ^ r % 8).  Eight lanes
// copy a row's 128 bytes; a row or column that is not there is filled with
// zeros.
struct GatherRing {
  const GShared &sh;
  const GArgs &args;
  uint8_t *ring;
  int pair, n_pairs, num_tiles, rank, quarter, part, lane;
  int t, row, col0, nc, c, j;   // the next step to copy: tile, its first row and columns, slot
  int index;                    // this lane's row's, of that step
  int fill, take;

  // the first step of tile t, or of the next tile with one
  __device__ __forceinline__ void seek() {
    for (; t < num_tiles; t += n_pairs) {
      const GTile tl = g_decode<false>(sh, args, t);
      row = tl.m0 + rank * GM + quarter * 32;
      col0 = tl.c0;
      nc = tl.nc;
      c = part * 64;
      if (row < args.M[0] && c < nc) return;
    }
  }
  __device__ __forceinline__ void load_index() {
    index = -1;
    if (t < num_tiles && row + lane < args.M[0])
      index = __ldg(args.add_inv + (int64_t)(row + lane) * args.add_k + j);
    if (index >= args.M[0] * args.add_k) index = -1;
  }
  __device__ __forceinline__ void start() {
    t = pair;
    j = fill = take = 0;
    seek();
    load_index();
    for (int i = 0; i < G_RING; ++i) copy();
  }
  // copies a step (or nothing, past the last) as an asynchronous group
  __device__ __forceinline__ void copy() {
    if (t < num_tiles) {
      const int v = lane & 7, col = col0 + c + v * 8, N = args.N[0];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (lane >> 3) + 4 * i;
        const int from = __shfl_sync(0xffffffffu, index, r);
        const bool there = from >= 0 && col < N;
        const uint4 *src = args.add + (there ? ((int64_t)from * N + col) / 8 : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         tc::smem_u32(ring + fill * G_OUT + r * 128 + ((v ^ (r & 7)) << 4))),
                     "l"(src), "r"(there ? 16 : 0)
                     : "memory");
      }
      if (++j == args.add_k) {
        j = 0;
        c += 128;
        if (c >= nc) {
          t += n_pairs;
          seek();
        }
      }
      load_index();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = (fill + 1) % G_RING;
  }
  // adds the next step, this lane's row of it
  __device__ __forceinline__ void add(uint32_t (&a)[2][32]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(G_RING - 1) : "memory");
    __syncwarp();
    const uint8_t *piece = ring + take * G_OUT + lane * 128;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float f[8];
      unpack16<__nv_bfloat16>(*reinterpret_cast<const uint4 *>(piece + ((q ^ (lane & 7)) << 4)), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t &x = a[q >> 2][(q & 3) * 8 + e];
        x = __float_as_uint(__uint_as_float(x) + f[e]);
      }
    }
    __syncwarp();   // (read by all before it is filled again)
    take = (take + 1) % G_RING;
    copy();
  }
};

template <bool A_K, bool SPLIT, bool ADD>
__global__ void __launch_bounds__(G_THREADS, 1)
gemm_grad_kernel(const __grid_constant__ GMaps maps, const __grid_constant__ GArgs args) {
  constexpr int STAGES = g_stages(ADD);
  extern __shared__ uint8_t dyn_smem[];
  __shared__ GShared sh;
  uint8_t *smem = dyn_smem + ((1024 - (tc::smem_u32(dyn_smem) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int E = args.offsets ? args.num_experts : 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < args.problems; ++i) {
      tc::prefetch_tmap(&maps.a[i]);
      tc::prefetch_tmap(&maps.b[i]);
      tc::prefetch_tmap(&maps.out[i]);
    }
  }
  if (warp == 1) tmem_alloc2(&sh.tmem_base, G_TMEM_COLS);
  if (threadIdx.x == 32) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(&sh.full[s], 1);
      tc::mbar_init(&sh.empty[s], 1);
      tc::mbar_init(&sh.tail_full[s], 1);
      tc::mbar_init(&sh.peer_fixed[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&sh.tfull[a], 1);
      tc::mbar_init(&sh.tempty[a], 2 * G_EPI);
    }
    tc::mbar_init(&sh.drain, 1);
    tc::fence_mbar_init();
  }
  // (all above ran beside the end of the kernel before; from here on its
  // results are read)
  pdl_wait();
  if (args.beside) pdl_launch_dependents();
  if (threadIdx.x == 0) {
    sh.failed_on_entry = status_failed(args.status) ? 1 : 0;
    sh.abort = sh.failed_on_entry;
    sh.bad = 0;
  }
  for (int i = threadIdx.x; i <= E; i += G_THREADS)
    sh.offs[i] = args.offsets ? args.offsets[i] : (i == 0 ? 0 : args.rows);
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += G_THREADS) {
    const int b = sh.offs[i], en = sh.offs[i + 1];
    if (b < 0 || en < b || en > args.rows) sh.bad = 1;   // (same value from every writer)
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;
  const int num_tiles = sh.bad ? 0 : E * args.splits * args.first[args.problems];
  if (sh.bad && rank == 0 && threadIdx.x == 0) set_status(args.status, MOE_ERR_BAD_INDEX, -1);
  volatile int *abort = &sh.abort;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      // (the loop below feeds both SMs' tensor cores from one thread: what it
      // does per k-block is kept short)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t tail_phase = 0;                            // bit s: phase of stage s's next fixed use
      uint32_t used = 0, used_phase = 0, used_tail = 0;   // the last use of each stage
      const uint32_t full0 = map_to_rank(tc::smem_u32(&sh.full[0]), 0);
      const uint32_t tail0 = map_to_rank(tc::smem_u32(&sh.tail_full[0]), rank);
      for (int t = pair; t < num_tiles && !*abort; t += n_pairs) {
        const GTile tl = g_decode<SPLIT>(sh, args, t);
        const int half = ((tl.nc + 15) & ~15) >> 1;       // output columns staged by each CTA
        const bool two = half > 64;                       // one or two boxes of them
        const uint32_t bytes = (uint32_t)(two ? 4 : 3) * G_BOX;
        const CUtensorMap *ma = &maps.a[tl.prob], *mb = &maps.b[tl.prob];
        const int m = tl.m0 + (int)rank * GM, c = tl.c0 + (int)rank * half;
        const int end = tl.beg + tl.len;
        for (int q = tl.beg; q < end; q += GK) {
          if (!tc::mbar_wait(&sh.empty[stage], phase ^ 1u, abort)) break;
          const uint32_t bit = 1u << stage;
          uint32_t bar = full0 + (uint32_t)stage * 8;
          used |= bit;
          used_phase = phase ? used_phase | bit : used_phase & ~bit;
          used_tail &= ~bit;
          if (!A_K && end - q < GK && ((end - q) & 15) != 0) {
            bar = tail0 + (uint32_t)stage * 8;
            tc::mbar_arrive_expect_tx(&sh.tail_full[stage], bytes);
            used_tail |= bit;
            used_phase = tail_phase & bit ? used_phase | bit : used_phase & ~bit;
            tail_phase ^= bit;
          } else if (rank == 0) {
            tc::mbar_arrive_expect_tx(&sh.full[stage], 2 * bytes);
          }
          uint8_t *sb = smem + stage * G_STAGE;
          tma2_load_2d(mb, bar, sb, c, q);
          if constexpr (A_K) {
            tma2_load_2d(ma, bar, sb + 2 * G_BOX, q, m);
          } else {
            tma2_load_2d(ma, bar, sb + 2 * G_BOX, m, q);
            tma2_load_2d(ma, bar, sb + 3 * G_BOX, m + 64, q);
          }
          if (two) tma2_load_2d(mb, bar, sb + G_BOX, c + 64, q);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (*abort) {
        // let the copies in flight land before the pair exits (the second
        // CTA's whole k-blocks count on the first CTA's barriers)
        for (int s = 0; s < STAGES; ++s) {
          if (!((used >> s) & 1u)) continue;
          const uint32_t ph = (used_phase >> s) & 1u;
          if ((used_tail >> s) & 1u) tc::mbar_wait_drain(&sh.tail_full[s], ph, 100000000ull);
          else if (rank == 0) tc::mbar_wait_drain(&sh.full[s], ph, 100000000ull);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (first CTA of the pair)
      int stage = 0;
      uint32_t phase = 0;
      int local = 0;
      bool ok = true;
      const uint32_t sa0 = tc::smem_u32(smem) + 2 * G_BOX;
      const uint64_t b_desc = tc::smem_desc_sw128_mn(tc::smem_u32(smem), G_BOX);
      const uint64_t a_desc = A_K ? tc::smem_desc_sw128(sa0) : tc::smem_desc_sw128_mn(sa0, G_BOX);
      const uint32_t b_lo = (uint32_t)b_desc, b_hi = (uint32_t)(b_desc >> 32);
      const uint32_t a_lo = (uint32_t)a_desc, a_hi = (uint32_t)(a_desc >> 32);
      for (int t = pair; t < num_tiles && ok && !*abort; t += n_pairs) {
        const GTile tl = g_decode<SPLIT>(sh, args, t);
        if (tl.len == 0) continue;
        const uint32_t idesc = tc::idesc_bf16_f32(2 * GM, (tl.nc + 15) & ~15) |
                               (A_K ? 0u : tc::kIdescAMajorMN) | tc::kIdescBMajorMN;
        const int acc = local & 1;
        if (!mbar_wait_cluster(&sh.tempty[acc], ((local >> 1) & 1) ^ 1u, abort)) break;
        tc::tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * GN);
        for (int k = 0; k < tl.len; k += GK) {
          if (!tc::mbar_wait(&sh.full[stage], phase, abort)) { ok = false; break; }
          tc::tc_fence_after();
          // (low descriptor words: 16-byte units; 16 rows are 2048 bytes, 16
          // elements of a contiguous reduction 32)
          constexpr uint32_t A_STEP = A_K ? 2 : 128;
          const uint32_t bl = b_lo + (uint32_t)(stage * (G_STAGE / 16));
          const uint32_t al = a_lo + (uint32_t)(stage * (G_STAGE / 16));
          const int left = tl.len - k;
          mma2_bf16_lo(d_tmem, al, a_hi, bl, b_hi, idesc, k != 0);
          if (left > 48) {
#pragma unroll
            for (int i = 1; i < 4; ++i)
              mma2_bf16_lo(d_tmem, al + i * A_STEP, a_hi, bl + i * 128, b_hi, idesc, 1u);
          } else {
            if (left > 16) mma2_bf16_lo(d_tmem, al + A_STEP, a_hi, bl + 128, b_hi, idesc, 1u);
            if (left > 32) mma2_bf16_lo(d_tmem, al + 2 * A_STEP, a_hi, bl + 256, b_hi, idesc, 1u);
          }
          mma2_commit_both(&sh.empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        mma2_commit_both(&sh.tfull[acc]);
        ++local;
      }
      if (*abort) {
        mma2_commit_self(&sh.drain);
        tc::mbar_wait_drain(&sh.drain, 0, 100000000ull);
      }
    }
  } else if (warp == 2 + G_EPI) {
    // ---------------- fixer (both CTAs; with A_K the copies fill zeros past
    // both operands' ends)
    int stage = 0;
    uint32_t tail_phase = 0;
    for (int t = pair; t < num_tiles; t += n_pairs) {
      const GTile tl = g_decode<SPLIT>(sh, args, t);
      const int kb = (tl.len + GK - 1) / GK;
      if (kb == 0) continue;
      const int at = (stage + kb - 1) % STAGES;
      stage = (stage + kb) % STAGES;
      const int valid = tl.len - (kb - 1) * GK;           // rows of the last k-block
      if (A_K || (valid & 15) == 0) continue;
      const uint32_t ph = (tail_phase >> at) & 1u;
      tail_phase ^= 1u << at;
      const bool ok = tc::mbar_wait(&sh.tail_full[at], ph, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      // rows valid .. next multiple of 16 of every box (a swizzled row is a
      // permutation of its own 128 bytes)
      // (8 lanes per row, 4 rows at a time)
      uint8_t *base = smem + at * G_STAGE + (lane & 7) * 16;
      for (int r = valid + (lane >> 3); r < ((valid + 15) & ~15); r += 4) {
#pragma unroll
        for (int box = 0; box < 4; ++box)
          *reinterpret_cast<uint4 *>(base + box * G_BOX + r * 128) = make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
      __syncwarp();
      if (rank == 1) {
        if (lane == 0) mbar_arrive_cluster(map_to_rank(tc::smem_u32(&sh.peer_fixed[at]), 0));
      } else {
        const bool peer = mbar_wait_cluster(&sh.peer_fixed[at], ph, abort);
        if (!__all_sync(0xffffffffu, peer)) break;
        if (lane == 0) tc::mbar_arrive(&sh.full[at]);
      }
    }
  } else {
    // ---------------- epilogue (both CTAs): warp w drains TMEM lanes 32*(w%4) .. +31
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tempty_first = map_to_rank(tc::smem_u32(&sh.tempty[0]), 0);
    uint8_t *stage_out = smem + STAGES * G_STAGE + (warp - 2) * G_OUT;
    int local = 0;
    GatherRing gather{sh, args, smem + STAGES * G_STAGE + (G_EPI + (warp - 2) * G_RING) * G_OUT,
                      pair, n_pairs, num_tiles, (int)rank, quarter, part, lane};
    if (ADD) gather.start();
    for (int t = pair; t < num_tiles; t += n_pairs) {
      const GTile tl = g_decode<SPLIT>(sh, args, t);
      const int row = tl.m0 + (int)rank * GM + quarter * 32;   // this warp's first row
      const bool rows_ok = row < args.M[tl.prob];
      const int acc = local & 1;
      if (tl.len != 0) {
        const bool ok = tc::mbar_wait(&sh.tfull[acc], (local >> 1) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc::tc_fence_after();
      } else if (__any_sync(0xffffffffu, *abort)) {
        break;
      }
      const uint32_t tb = lane_base + (uint32_t)(acc * GN);
#pragma unroll 1
      for (int c = part * 64; c < tl.nc; c += 128) {
        uint32_t a[2][32];
        if (tl.len != 0) {
          tc::tmem_ld32(tb + (uint32_t)c, a[0]);
          tc::tmem_ld32(tb + (uint32_t)(c + 32), a[1]);
          tc::tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) a[0][i] = a[1][i] = 0;
        }
        if (!rows_ok) continue;
        if (ADD)
          for (int j = 0; j < args.add_k; ++j) gather.add(a);
#pragma unroll
        for (int half = 0; half < (SPLIT ? 2 : 1); ++half) {
          // a 128-byte piece of each row: 64 elements, or 32 partial sums
          const int col = tl.c0 + c + half * 32;
          if (SPLIT && col >= args.N[tl.prob]) break;
          if (lane == 0) tc::bulk_wait_read<0>();   // the store before has read the buffer
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint4 w;
            if constexpr (SPLIT) {
              const uint32_t *v = &a[half][q * 4];
              w = make_uint4(v[0], v[1], v[2], v[3]);
            } else {
              const uint32_t *v = &a[q >> 2][(q & 3) * 8];
              w = make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                             bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
            }
            *reinterpret_cast<uint4 *>(stage_out + lane * 128 + ((q ^ (lane & 7)) << 4)) = w;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) tc::tma_store_3d(&maps.out[tl.prob], stage_out, col, row, tl.z);
        }
      }
      if (tl.len != 0) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_first + (uint32_t)(acc * sizeof(uint64_t)));
        ++local;
      }
    }
    if (lane == 0) tc::bulk_wait_all();
    if (ADD) asm volatile("cp.async.wait_group 0;" ::: "memory");
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
    tmem_dealloc2(tmem_base, G_TMEM_COLS);
  }
  if (threadIdx.x == 0 && sh.abort && !sh.failed_on_entry)
    set_status(args.status, MOE_ERR_TIMEOUT, blockIdx.x);
}

// out[i] = sum over the runs of partial[run][i], in order: the runs' matrices
// of one expert follow one another.
struct SumArgs {
  const float *part[kMaxGradProblems];
  __nv_bfloat16 *out[kMaxGradProblems];
  int64_t per_expert[kMaxGradProblems];   // M * N (a multiple of 8)
  int experts, splits;
  int *status;
};
__global__ void __launch_bounds__(256) grad_sum_kernel(SumArgs a) {
  pdl_wait();
  if (status_failed(a.status)) return;
  const int p = blockIdx.y;
  const int64_t per = a.per_expert[p], total = per * a.experts;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < total;
       i += (int64_t)gridDim.x * 256 * 8) {
    const int64_t e = i / per;
    const float4 *src = reinterpret_cast<const float4 *>(a.part[p] + e * a.splits * per + (i - e * per));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float4 u = src[s * (per / 4)], v = src[s * (per / 4) + 1];
      x.x += u.x; x.y += u.y; x.z += u.z; x.w += u.w;
      y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
    }
    auto pack = [](float l, float h) { return bf16x2_bits(__float_as_uint(l), __float_as_uint(h)); };
    *reinterpret_cast<uint4 *>(a.out[p] + i) =
        make_uint4(pack(x.x, x.y), pack(x.z, x.w), pack(y.x, y.y), pack(y.z, y.w));
  }
}

constexpr int kPairs = 76;   // SM pairs that the plans count on

template <bool A_K, bool SPLIT, bool ADD = false>
cudaError_t launch(const GMaps &maps, const GArgs &a, cudaStream_t s) {
  auto kernel = gemm_grad_kernel<A_K, SPLIT, ADD>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(G_THREADS);
  cfg.dynamicSmemBytes = g_dyn_smem(ADD);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;   // (the occupancy query takes the cluster alone)
  static int pairs = 0;
  if (pairs == 0) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)g_dyn_smem(ADD));
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs < 1) {
      cudaGetLastError();
      pairs = num_sms() / 2;
    }
  }
  cfg.gridDim = dim3(2 * (a.beside ? a.beside : pairs));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

int64_t tiles_of(const GradProduct *p, int count, int width) {
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i)
    tiles += (int64_t)(p[i].offsets ? p[i].num_experts : 1) *
             ((p[i].M + 2 * GM - 1) / (2 * GM)) * ((p[i].N + width - 1) / width);
  return tiles;
}

// Narrower tiles where 256 columns leave SM pairs without a tile.
int width_of(const GradProduct *p, int count, int splits) {
  int width = GN;
  while (width > 64 && tiles_of(p, count, width) * splits < kPairs) width /= 2;
  return width;
}

bool encode(CUtensorMap *m, const void *p, int rank, const uint64_t *dims, const uint32_t *box) {
  return make_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, rank, dims, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

bool gemm_grad_supported(const GradProduct &p) {
  return p.dtype == MOE_BF16 && p.rows > 0 && tensor_maps_available() &&
         p.num_experts <= G_MAX_E && (p.lda ? p.lda : p.M) % 8 == 0 && p.N % 8 == 0 &&
         num_sms() >= 2;
}

// Two tiles per pair at most, and 512 rows of an average segment per run at
// least: a run's tile then costs more than the 512 KB of partial sums that it
// adds to write and read.  (Router gradient of 16384 tokens, 256 experts, d
// 7168: 28 tiles, 155 us at 64 columns each; 64 us in 140 runs of 256
// columns and their sum.)
int grad_splits(const GradProduct *p, int count) {
  if (count == 0) return 1;
  if (grads_small(p, count)) return grad_splits_simt(p, count);
  const int64_t tiles = tiles_of(p, count, GN);
  const int E = p[0].offsets ? p[0].num_experts : 1;
  if (tiles >= kPairs) return 1;
  const int64_t most = 2 * kPairs / tiles, by_rows = p[0].rows / E / 512;
  const int64_t n = most < by_rows ? most : by_rows;
  return n < 2 ? 1 : (int)n;
}

size_t grad_scratch(const GradProduct *p, int count) {
  const int splits = grad_splits(p, count);
  size_t bytes = 0;
  for (int i = 0; splits > 1 && i < count; ++i)
    bytes += (size_t)splits * (p[i].offsets ? p[i].num_experts : 1) * p[i].M * p[i].N * 4;
  return bytes;
}

cudaError_t launch_gemm_grad(const GradProduct *p, int count, int splits, float *scratch,
                             int beside, int *status, cudaStream_t s) {
  GMaps maps{};
  GArgs a{};
  a.offsets = p[0].offsets;
  a.num_experts = p[0].num_experts;
  a.rows = p[0].rows;
  a.problems = count;
  a.status = status;
  a.splits = splits;
  a.beside = beside;
  a.width = width_of(p, count, splits);
  const int E = p[0].offsets ? p[0].num_experts : 1;
  const uint32_t box[2] = {64, GK}, box_out[3] = {splits > 1 ? 32u : 64u, 32, 1};
  SumArgs sum{};
  sum.experts = E;
  sum.splits = splits;
  sum.status = status;
  int64_t most = 0;
  for (int i = 0; i < count; ++i) {
    a.M[i] = p[i].M;
    a.N[i] = p[i].N;
    a.first[i + 1] = a.first[i] + ((p[i].M + 2 * GM - 1) / (2 * GM)) *
                                      ((p[i].N + a.width - 1) / a.width);
    const uint64_t da[2] = {(uint64_t)(p[i].lda ? p[i].lda : p[i].M), (uint64_t)p[i].rows};
    const uint64_t db[2] = {(uint64_t)p[i].N, (uint64_t)p[i].rows};
    const uint64_t dout[3] = {(uint64_t)p[i].N, (uint64_t)p[i].M, (uint64_t)E * splits};
    if (!encode(&maps.a[i], p[i].A, 2, da, box) || !encode(&maps.b[i], p[i].B, 2, db, box))
      return cudaErrorInvalidValue;
    if (splits == 1) {
      if (!encode(&maps.out[i], p[i].out, 3, dout, box_out)) return cudaErrorInvalidValue;
      continue;
    }
    sum.part[i] = scratch;
    sum.out[i] = static_cast<__nv_bfloat16 *>(p[i].out);
    sum.per_expert[i] = (int64_t)p[i].M * p[i].N;
    if (!make_tensor_map(&maps.out[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, scratch, 3, dout, box_out,
                         CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    scratch += (int64_t)splits * E * sum.per_expert[i];
    if (sum.per_expert[i] * E > most) most = sum.per_expert[i] * E;
  }
  if (splits == 1) return launch<false, false>(maps, a, s);
  const cudaError_t e = launch<false, true>(maps, a, s);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (most / 8 + 255) / 256;
  return launch_pdl(grad_sum_kernel, dim3((unsigned)(blocks < 1216 ? blocks : 1216), count),
                    dim3(256), 0, s, sum);
}

bool gemm_router_rows_supported(const RowsProduct &p) {
  return p.dtype == MOE_BF16 && p.epi == kRowsPlain && p.b_rows && p.offsets == nullptr &&
         p.A2 == nullptr && p.rows > 0 && tensor_maps_available() && p.N % 8 == 0 &&
         (p.lda ? p.lda : p.K) % 8 == 0 && num_sms() >= 2;
}

cudaError_t launch_gemm_router_rows(const RowsProduct &p, int *status, cudaStream_t s) {
  GradProduct shape{};
  shape.M = p.rows;
  shape.N = p.N;
  GMaps maps{};
  GArgs a{};
  a.num_experts = 1;
  a.rows = p.K;      // the reduction
  a.problems = 1;
  a.status = status;
  a.splits = 1;
  a.width = width_of(&shape, 1, 1);
  a.M[0] = p.rows;
  a.N[0] = p.N;
  a.first[1] = (int)tiles_of(&shape, 1, a.width);
  const uint64_t da[2] = {(uint64_t)(p.lda ? p.lda : p.K), (uint64_t)p.rows};
  const uint64_t db[2] = {(uint64_t)p.N, (uint64_t)p.K};
  const uint64_t dout[3] = {(uint64_t)p.N, (uint64_t)p.rows, 1};
  const uint32_t box_a[2] = {GK, GM}, box_b[2] = {64, GK}, box_out[3] = {64, 32, 1};
  if (!encode(&maps.a[0], p.A, 2, da, box_a) || !encode(&maps.b[0], p.B, 2, db, box_b) ||
      !encode(&maps.out[0], p.out, 3, dout, box_out))
    return cudaErrorInvalidValue;
  a.add = static_cast<const uint4 *>(p.add);
  a.add_inv = p.add_inv;
  a.add_k = p.add_k;
  return p.add ? launch<true, false, true>(maps, a, s) : launch<true, false>(maps, a, s);
}

}  // namespace moe
