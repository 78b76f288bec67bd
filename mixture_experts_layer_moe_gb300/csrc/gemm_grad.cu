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
// each, against TODO_MEASURED.
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
// Roles (persistent, one CTA per SM, clusters of two): warp 0 TMA producer in
// both CTAs, warp 1 of the first CTA issues the MMAs into two accumulators of
// 256 columns, warps 2-9 drain them (two warps per lane quarter, taking turns
// of 64 columns), warp 10 is the fixer.
#include "common.cuh"
#include "launch.h"
#include "pair_common.cuh"
#include "tc_common.cuh"
#include "train.h"

namespace moe {
namespace {

using namespace pair;

constexpr int GM = 128;                       // output rows per CTA (MMA M = 256 per pair)
constexpr int GN = 256;                       // output columns per tile at most (MMA N)
constexpr int GK = 64;                        // segment rows per k-block
constexpr int GS = 6;                         // pipeline stages
constexpr int G_BOX = 64 * GK * 2;            // one 64 x 64 box: 8 KB
constexpr int G_STAGE = 4 * G_BOX;            // two boxes of B (N side), two of A (M side)
constexpr int G_EPI = 8;                      // epilogue warps: two per TMEM lane quarter
constexpr int G_THREADS = 32 * (3 + G_EPI);
constexpr uint32_t G_TMEM_COLS = 512;
constexpr int G_MAX_E = 256;
constexpr int G_OUT = 32 * 128;               // one store: 32 rows x 64 columns, 128-byte swizzle
constexpr size_t G_DYN_SMEM = 1024 + (size_t)GS * G_STAGE + (size_t)G_EPI * G_OUT;

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
  int *status;
};
struct GMaps {
  CUtensorMap a[kMaxGradProblems], b[kMaxGradProblems], out[kMaxGradProblems];
};

struct GTile {
  int e, prob, m0, c0, nc, beg, len;   // nc columns from c0
};

__device__ __forceinline__ GTile g_decode(const GShared &sh, const GArgs &args, int t) {
  GTile tl;
  const int per = args.first[args.problems];
  tl.e = t / per;
  int r = t - tl.e * per;
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
  return tl;
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ uint32_t bf16x2_bits(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t *>(&h);
}

__global__ void __launch_bounds__(G_THREADS, 1)
gemm_grad_kernel(const __grid_constant__ GMaps maps, const __grid_constant__ GArgs args) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ GShared sh;
  uint8_t *smem = dyn_smem + ((1024 - (tc::smem_u32(dyn_smem) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int E = args.offsets ? args.num_experts : 1;

  if (threadIdx.x == 0) {
    sh.failed_on_entry = status_failed(args.status) ? 1 : 0;
    sh.abort = sh.failed_on_entry;
    sh.bad = 0;
  }
  for (int i = threadIdx.x; i <= E; i += G_THREADS)
    sh.offs[i] = args.offsets ? args.offsets[i] : (i == 0 ? 0 : args.rows);
  if (warp == 1) tmem_alloc2(&sh.tmem_base, G_TMEM_COLS);
  if (threadIdx.x == 32) {
    for (int s = 0; s < GS; ++s) {
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
  const int num_tiles = sh.bad ? 0 : E * args.first[args.problems];
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
        const GTile tl = g_decode(sh, args, t);
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
          if (end - q < GK && ((end - q) & 15) != 0) {
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
          tma2_load_2d(ma, bar, sb + 2 * G_BOX, m, q);
          tma2_load_2d(ma, bar, sb + 3 * G_BOX, m + 64, q);
          if (two) tma2_load_2d(mb, bar, sb + G_BOX, c + 64, q);
          if (++stage == GS) { stage = 0; phase ^= 1u; }
        }
      }
      if (*abort) {
        // let the copies in flight land before the pair exits (the second
        // CTA's whole k-blocks count on the first CTA's barriers)
        for (int s = 0; s < GS; ++s) {
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
      const uint64_t desc = tc::smem_desc_sw128_mn(tc::smem_u32(smem), G_BOX);
      const uint32_t desc_lo = (uint32_t)desc, desc_hi = (uint32_t)(desc >> 32);
      for (int t = pair; t < num_tiles && ok && !*abort; t += n_pairs) {
        const GTile tl = g_decode(sh, args, t);
        if (tl.len == 0) continue;
        const uint32_t idesc = tc::idesc_bf16_f32(2 * GM, (tl.nc + 15) & ~15) |
                               tc::kIdescAMajorMN | tc::kIdescBMajorMN;
        const int acc = local & 1;
        if (!mbar_wait_cluster(&sh.tempty[acc], ((local >> 1) & 1) ^ 1u, abort)) break;
        tc::tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * GN);
        for (int k = 0; k < tl.len; k += GK) {
          if (!tc::mbar_wait(&sh.full[stage], phase, abort)) { ok = false; break; }
          tc::tc_fence_after();
          // (low descriptor words: 16-byte units, 2048 bytes per 16 rows)
          const uint32_t b_lo = desc_lo + (uint32_t)(stage * (G_STAGE / 16));
          const uint32_t a_lo = b_lo + 2 * G_BOX / 16;
          const int left = tl.len - k;
          mma2_bf16_lo(d_tmem, a_lo, desc_hi, b_lo, desc_hi, idesc, k != 0);
          if (left > 48) {
#pragma unroll
            for (int i = 1; i < 4; ++i)
              mma2_bf16_lo(d_tmem, a_lo + i * 128, desc_hi, b_lo + i * 128, desc_hi, idesc, 1u);
          } else {
            if (left > 16) mma2_bf16_lo(d_tmem, a_lo + 128, desc_hi, b_lo + 128, desc_hi, idesc, 1u);
            if (left > 32) mma2_bf16_lo(d_tmem, a_lo + 256, desc_hi, b_lo + 256, desc_hi, idesc, 1u);
          }
          mma2_commit_both(&sh.empty[stage]);
          if (++stage == GS) { stage = 0; phase ^= 1u; }
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
    // ---------------- fixer (both CTAs)
    int stage = 0;
    uint32_t tail_phase = 0;
    for (int t = pair; t < num_tiles; t += n_pairs) {
      const GTile tl = g_decode(sh, args, t);
      const int kb = (tl.len + GK - 1) / GK;
      if (kb == 0) continue;
      const int at = (stage + kb - 1) % GS;
      stage = (stage + kb) % GS;
      const int valid = tl.len - (kb - 1) * GK;           // rows of the last k-block
      if ((valid & 15) == 0) continue;
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
    uint8_t *stage_out = smem + GS * G_STAGE + (warp - 2) * G_OUT;
    int local = 0;
    for (int t = pair; t < num_tiles; t += n_pairs) {
      const GTile tl = g_decode(sh, args, t);
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
        if (lane == 0) tc::bulk_wait_read<0>();   // the store before has read the buffer
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t *v = &a[q >> 2][(q & 3) * 8];
          *reinterpret_cast<uint4 *>(stage_out + lane * 128 + ((q ^ (lane & 7)) << 4)) =
              make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]),
                         bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::tma_store_3d(&maps.out[tl.prob], stage_out, tl.c0 + c, row, tl.e);
      }
      if (tl.len != 0) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_first + (uint32_t)(acc * sizeof(uint64_t)));
        ++local;
      }
    }
    if (lane == 0) tc::bulk_wait_all();
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
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

int pairs_resident() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (num_sms() / 2));
  cfg.blockDim = dim3(G_THREADS);
  cfg.dynamicSmemBytes = G_DYN_SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_grad_kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = num_sms() / 2;
  }
  return n;
}

}  // namespace

bool gemm_grad_supported(const GradProduct &p) {
  return p.dtype == MOE_BF16 && p.rows > 0 && tensor_maps_available() &&
         p.num_experts <= G_MAX_E && (p.lda ? p.lda : p.M) % 8 == 0 && p.N % 8 == 0 &&
         num_sms() >= 2;
}

cudaError_t launch_gemm_grad(const GradProduct *p, int count, int *status, cudaStream_t s) {
  static int pairs = 0;
  if (pairs == 0) {
    const cudaError_t e = cudaFuncSetAttribute(
        gemm_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G_DYN_SMEM);
    if (e != cudaSuccess) return e;
    pairs = pairs_resident();
  }
  GMaps maps{};
  GArgs a{};
  a.offsets = p[0].offsets;
  a.num_experts = p[0].num_experts;
  a.rows = p[0].rows;
  a.problems = count;
  a.status = status;
  const uint32_t box[2] = {64, GK}, box_out[3] = {64, 32, 1};
  const int E = p[0].offsets ? p[0].num_experts : 1;
  // narrower tiles where 256 columns leave SM pairs without a tile
  for (a.width = GN; a.width > 64; a.width /= 2) {
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i)
      tiles += (int64_t)E * ((p[i].M + 2 * GM - 1) / (2 * GM)) * ((p[i].N + a.width - 1) / a.width);
    if (tiles >= pairs) break;
  }
  for (int i = 0; i < count; ++i) {
    a.M[i] = p[i].M;
    a.N[i] = p[i].N;
    a.first[i + 1] = a.first[i] + ((p[i].M + 2 * GM - 1) / (2 * GM)) *
                                      ((p[i].N + a.width - 1) / a.width);
    const uint64_t da[2] = {(uint64_t)(p[i].lda ? p[i].lda : p[i].M), (uint64_t)p[i].rows};
    const uint64_t db[2] = {(uint64_t)p[i].N, (uint64_t)p[i].rows};
    const uint64_t dout[3] = {(uint64_t)p[i].N, (uint64_t)p[i].M, (uint64_t)E};
    if (!make_tensor_map(&maps.a[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p[i].A, 2, da, box,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&maps.b[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p[i].B, 2, db, box,
                         CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_tensor_map(&maps.out[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p[i].out, 3, dout,
                         box_out, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(G_THREADS);
  cfg.dynamicSmemBytes = G_DYN_SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_grad_kernel, maps, a);
}

}  // namespace moe
