// The products of the cross entropy on a pair of SMs (tcgen05.mma.cta_group::2),
// tokens on the MMA's M side (256 per tile, 128 in each CTA, one per TMEM lane)
// and up to 256 columns on its N side:
//   kSums   l[t][v] = sum_k x[t][k] W[v][k], which the epilogue reduces to a
//           maximum and a sum of exponentials per token as it drains the tile;
//   kGrad   the same product, turned into dl = dloss (e^(l - lse) (1 + 2 z lse) -
//           [v = target]) / unit in the epilogue and stored in bf16 (zeros in the rows of the
//           last 32 tokens that do not count);
//   kDx     dx[t][c] = sum_v dl[t][v] W[v][c], W read as it is stored (an N-major
//           operand), in fp32.
// unit is the largest |dloss|: divided by it, the target's entry of a token whose
// probability is small is near -1 and so nearly exact.  (With dloss = 1 / count in
// it, rounding it is off the same way for every token, and so is the whole gradient:
// 4096 tokens, 65536 entries, dx and dW 2.6e-3 of their norms off, 1.9e-3 so, 1.7e-3
// being the result's own rounding.)
// With a token per lane the softmax runs over a thread's own accumulator columns:
// no exchange between lanes, and neither logits nor exponentials leave the SM.
// (With tokens on the N side, as the experts' products have them, every column of
// the vocabulary would be a lane's and each maximum and sum a reduction over the
// warps.)
//
// Roles (persistent, one CTA per SM, clusters of two): warp 0 TMA producer in
// both CTAs (128-byte swizzle, 6 stages of 32 KB), warp 1 of the first CTA issues
// the MMAs into two accumulators of 256 columns, warps 2-9 drain them, two warps
// per lane quarter that take turns of columns.  Rows of x past the counted ones
// are not stored, so what the lanes there hold does not matter.
//
// Tiles go through the vocabulary in bands of 16 token blocks: the pairs running
// together share a few blocks of W and the band's rows of x, which stay in L2,
// and W streams through once per band.
#include <math.h>

#include "common.cuh"
#include "fp32x2.cuh"
#include "launch.h"
#include "loss.h"
#include "pair_common.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace pair;

enum LossMode { kSums, kGrad, kDx };

constexpr int LM = 128;                       // tokens per CTA (MMA M = 256 per pair)
constexpr int LN = 256;                       // columns per tile at most (MMA N)
constexpr int LK = 64;                        // k-block
constexpr int LS = 6;                         // pipeline stages
constexpr int L_B = (LN / 2) * LK * 2;        // this CTA's half of the columns: 16 KB
constexpr int L_A = LM * LK * 2;              // its tokens: 16 KB
constexpr int L_STAGE = L_B + L_A;
constexpr int L_SHORT = 32;                   // rows of a short box of tokens
constexpr int L_EPI = 8;                      // epilogue warps
constexpr int L_THREADS = 32 * (2 + L_EPI);
constexpr int L_OUT = 32 * 128;               // one store: 32 rows of 128 bytes
constexpr size_t L_SMEM = 1024 + (size_t)LS * L_STAGE + (size_t)L_EPI * L_OUT;
constexpr int L_BAND = 16;
constexpr uint32_t L_TMEM_COLS = 512;
constexpr float kLog2e = 1.4426950408889634f;
// kSums: k-blocks that the tensor core adds up by itself.  Its sums are cut off, not
// rounded, at each step, so that their error grows with the number of steps;
// longer reductions are added up in registers, rounded.  (4096 tokens over 131072 entries,
// d 4096: the losses 2.0e-6 of their norm off, 4.8e-7 so; 2494 us without and 2560
// with, 8 k-blocks 2.3e-7 and 2780.)
constexpr int L_UNIT_KB = 16, L_UNIT_FEW_KB = 8;   // (one block of tokens: HBM bounds it)

struct LShared {
  uint64_t full[LS];    // first CTA: both CTAs' boxes landed
  uint64_t empty[LS];   // both CTAs: the MMAs that read the stage completed
  uint64_t tfull[2];    // both CTAs: the accumulator's MMAs completed
  uint64_t tempty[2];   // first CTA: both CTAs' epilogues drained the accumulator
  uint64_t drain;
  uint32_t tmem_base;
  int abort, failed_on_entry, counted;
};

struct LArgs {
  LossProduct p;
  int cols, K, width;   // of the product: columns, reduction, columns per tile
  int *status;
};
struct LMaps {
  CUtensorMap A, As, B, out;
};
struct LTile {
  int row0, col0, col, z, kb0, kb1;
};

__device__ __forceinline__ LTile l_decode(int t, int mt, int nt, int KB, int splits, int width) {
  LTile tl;
  tl.z = t / (mt * nt);
  int r = t - tl.z * mt * nt;
  const int band = r / (L_BAND * nt), first = band * L_BAND, tall = min(L_BAND, mt - first);
  r -= first * nt;
  tl.col = r / tall;
  tl.row0 = (first + r - tl.col * tall) * 2 * LM;
  tl.col0 = tl.col * width;
  const int each = (KB + splits - 1) / splits;
  tl.kb0 = tl.z * each;
  tl.kb1 = min(KB, tl.kb0 + each);
  return tl;
}

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <LossMode MODE>
__global__ void __launch_bounds__(L_THREADS, 1)
loss_pair_kernel(const __grid_constant__ LMaps maps, const __grid_constant__ LArgs args) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ LShared sh;
  uint8_t *smem = dyn_smem + ((1024 - (tc::smem_u32(dyn_smem) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const LossProduct &p = args.p;
  const int width = args.width;

  if (threadIdx.x == 0) {
    tc::prefetch_tmap(&maps.A);
    tc::prefetch_tmap(&maps.As);
    tc::prefetch_tmap(&maps.B);
    if (MODE != kSums) tc::prefetch_tmap(&maps.out);
  }
  if (warp == 1) tmem_alloc2(&sh.tmem_base, L_TMEM_COLS);
  if (threadIdx.x == 32) {
    for (int s = 0; s < LS; ++s) {
      tc::mbar_init(&sh.full[s], 1);
      tc::mbar_init(&sh.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&sh.tfull[a], 1);
      tc::mbar_init(&sh.tempty[a], 2 * L_EPI);
    }
    tc::mbar_init(&sh.drain, 1);
    tc::fence_mbar_init();
  }
  // (all above ran beside the end of the kernel before; from here on its
  // results are read)
  pdl_wait();
  if (threadIdx.x == 0) {
    sh.failed_on_entry = status_failed(args.status) ? 1 : 0;
    sh.abort = sh.failed_on_entry;
    sh.counted = p.range ? min(max(p.range[1], 0), p.n) : p.n;
  }
  tc::tc_fence_before();
  __syncthreads();
  // both CTAs' barriers are initialised before either CTA touches the other's
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;
  const int m = sh.counted, mt = (m + 2 * LM - 1) / (2 * LM), nt = (args.cols + width - 1) / width;
  const int KB = (args.K + LK - 1) / LK, splits = MODE == kDx ? p.splits : 1;
  const int num_tiles = mt * nt * splits;
  const int sum_unit = mt > 1 ? L_UNIT_KB : L_UNIT_FEW_KB;
  volatile int *abort = &sh.abort;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs)
      int stage = 0;
      uint32_t phase = 0;
      uint32_t used = 0, used_phase = 0;   // bit s: stage s was used, in which phase last
      const uint32_t full0 = map_to_rank(tc::smem_u32(&sh.full[0]), 0);
      const int half = width / 2;          // columns staged by each CTA
      // (kDx: one or two boxes of 64 columns)
      const bool two = MODE == kDx && half > 64;
      const uint32_t b_bytes =
          MODE == kDx ? (two ? 2u : 1u) * 64 * LK * 2 : (uint32_t)half * LK * 2;
      // bytes of a CTA's tokens, by how many there are from its first on
      auto a_bytes = [](int rows) {
        return rows <= 0 ? 0u : (uint32_t)(rows <= L_SHORT ? L_SHORT : LM) * LK * 2;
      };
      for (int t = pair; t < num_tiles && !*abort; t += n_pairs) {
        const LTile tl = l_decode(t, mt, nt, KB, splits, width);
        const int row = tl.row0 + (int)rank * LM, c = tl.col0 + (int)rank * half;
        const int rows = m - row;
        const CUtensorMap *a_map = rows <= L_SHORT ? &maps.As : &maps.A;
        const uint32_t bytes = 2 * b_bytes + a_bytes(m - tl.row0) + a_bytes(m - tl.row0 - LM);
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!tc::mbar_wait(&sh.empty[stage], phase ^ 1u, abort)) break;
          uint8_t *sb = smem + stage * L_STAGE;
          const uint32_t bar = full0 + (uint32_t)stage * 8;
          used |= 1u << stage;
          used_phase = phase ? used_phase | 1u << stage : used_phase & ~(1u << stage);
          if (rank == 0) tc::mbar_arrive_expect_tx(&sh.full[stage], bytes);   // of both CTAs
          if constexpr (MODE == kDx) {
            tma2_load_2d(&maps.B, bar, sb, c, kb * LK);
            if (two) tma2_load_2d(&maps.B, bar, sb + L_B / 2, c + 64, kb * LK);
          } else {
            tma2_load_2d(&maps.B, bar, sb, kb * LK, c);
          }
          if (rows > 0) tma2_load_2d(a_map, bar, sb + L_B, kb * LK, row);
          if (++stage == LS) { stage = 0; phase ^= 1u; }
        }
      }
      if (*abort && rank == 0) {
        // let the copies in flight land before the pair exits (the second
        // CTA's copies count on these barriers too)
        for (int s = 0; s < LS; ++s)
          if ((used >> s) & 1u)
            tc::mbar_wait_drain(&sh.full[s], (used_phase >> s) & 1u, 100000000ull);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------- MMA issuer (first CTA of the pair)
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t sb0 = tc::smem_u32(smem);
      const uint64_t b_desc = MODE == kDx ? tc::smem_desc_sw128_mn(sb0, L_B / 2)
                                          : tc::smem_desc_sw128(sb0);
      const uint64_t a_desc = tc::smem_desc_sw128(sb0 + L_B);
      const uint32_t a_lo = (uint32_t)a_desc, a_hi = (uint32_t)(a_desc >> 32);
      const uint32_t b_lo = (uint32_t)b_desc, b_hi = (uint32_t)(b_desc >> 32);
      const uint32_t idesc =
          tc::idesc_bf16_f32(2 * LM, width) | (MODE == kDx ? tc::kIdescBMajorMN : 0u);
      for (int t = pair; t < num_tiles && ok && !*abort; t += n_pairs) {
        const LTile tl = l_decode(t, mt, nt, KB, splits, width);
        // (one loop with a test for a unit's start in it: 5 % slower)
        const int unit = MODE == kSums ? sum_unit : tl.kb1 - tl.kb0;
        for (int ku = tl.kb0; ku < tl.kb1; ku += unit, ++local) {
          const int ke = min(tl.kb1, ku + unit);
          if (!mbar_wait_cluster(&sh.tempty[local & 1], ((local >> 1) & 1) ^ 1u, abort)) ok = false;
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t d_tmem = tmem_base + (uint32_t)((local & 1) * LN);
          for (int kb = ku; kb < ke; ++kb) {
            if (!tc::mbar_wait(&sh.full[stage], phase, abort)) { ok = false; break; }
            tc::tc_fence_after();
            // (low descriptor words: 16-byte units; 16 elements of a contiguous
            // reduction are 32 bytes, 16 rows 2048)
            const uint32_t at = (uint32_t)(stage * (L_STAGE / 16));
#pragma unroll
            for (int k = 0; k < LK / 16; ++k)
              mma2_bf16_lo(d_tmem, a_lo + at + k * 2, a_hi, b_lo + at + k * (MODE == kDx ? 128 : 2),
                           b_hi, idesc, (kb != ku || k != 0) ? 1u : 0u);
            mma2_commit_both(&sh.empty[stage]);
            if (++stage == LS) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          mma2_commit_both(&sh.tfull[local & 1]);
        }
      }
      if (*abort) {
        mma2_commit_self(&sh.drain);
        tc::mbar_wait_drain(&sh.drain, 0, 100000000ull);
      }
    }
  } else {
    // ---------------- epilogue (both CTAs): warp w drains TMEM lanes 32*(w%4) .. +31
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tempty_first = map_to_rank(tc::smem_u32(&sh.tempty[0]), 0);
    uint8_t *stage_out = smem + LS * L_STAGE + (warp - 2) * L_OUT;
    int local = 0;
    bool ok = true;
    for (int t = pair; t < num_tiles; t += n_pairs, ++local) {
      const LTile tl = l_decode(t, mt, nt, KB, splits, width);
      const int row = tl.row0 + (int)rank * LM + quarter * 32;   // this warp's first token
      const int j = row + lane;
      const bool there = j < m;
      // this token's target, from the tile's first column on
      int target = -1;
      float lse = 0.f, scale = 0.f, dloss = 0.f;
      if (MODE != kDx && there) {
        target = p.target[j] - p.v0 - tl.col0;
        if (MODE == kGrad) {
          lse = p.lse[j];
          const float unit = *p.scale;
          // (unit 0: what there is is zero or not finite, and stays so times it)
          dloss = unit > 0.f ? p.dloss[j] / unit : p.dloss[j];
          scale = dloss * fmaf(2.f * p.z_loss, lse, 1.f);
        }
      }
      // kSums: the logits of this warp's turns of 32 columns, unit by unit
      constexpr int TURNS = MODE == kSums ? LN / 64 : 1;
      float sum_of[TURNS][32];
      if constexpr (MODE == kSums) {
        for (int kb = tl.kb0; kb < tl.kb1; kb += sum_unit) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&sh.tfull[local & 1], (local >> 1) & 1, abort));
          if (!ok) break;
          tc::tc_fence_after();
          if (row < m) {
            const uint32_t tb = lane_base + (uint32_t)((local & 1) * LN);
#pragma unroll
            for (int q = 0; q < 2 * TURNS; ++q) {
              const int c = part * 32 + (q >> 1) * 64;
              if (c >= width) continue;
              uint32_t a[16];
              tc::tmem_ld16(tb + (uint32_t)(c + (q & 1) * 16), a);
              tc::tmem_ld_wait();
              float *to = sum_of[q >> 1] + (q & 1) * 16;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                to[i] = __uint_as_float(a[i]) + (kb == tl.kb0 ? 0.f : to[i]);
            }
          }
          if (kb + sum_unit < tl.kb1) {   // (the last unit is released below)
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0)
              mbar_arrive_cluster(tempty_first + (uint32_t)((local & 1) * sizeof(uint64_t)));
            ++local;
          }
        }
      } else {
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sh.tfull[local & 1], (local >> 1) & 1, abort));
        tc::tc_fence_after();
      }
      if (!ok) break;
      const int acc = local & 1;
      const uint32_t tb = lane_base + (uint32_t)(acc * LN);
      if constexpr (MODE == kSums) {
        // the accumulator is drained: the MMAs go on while the sums are formed
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_first + (uint32_t)(acc * sizeof(uint64_t)));
      }
      if (row < m) {
        if constexpr (MODE == kSums) {
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int q = 0; q < TURNS; ++q) {
            const int c = part * 32 + q * 64;
            const int left = args.cols - tl.col0 - c;   // columns that there are
            if (c >= width || left <= 0) continue;
            float (&l)[32] = sum_of[q], up = top;
            if (left < 32) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= left) l[i] = -INFINITY;
            }
            const int here = target - c;
            if (__any_sync(0xffffffffu, here >= 0 && here < 32)) {
              float at = 0.f;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i == here) at = l[i];
              if (here >= 0 && here < 32) p.at[j] = at;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) up = fmaxf(up, l[i]);
            // (the maximum is taken away before the factor: taken away after it, rounded, it would be off
            // by up to half an ulp of itself, and every exponential by that as a factor)
            const float2 shift = both(up == -INFINITY ? 0.f : -up);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 e = mul2(add2(make_float2(l[i], l[i + 1]), shift), both(kLog2e));
              s0 += exp2_fast(e.x);
              s1 += exp2_fast(e.y);
            }
            sum = fmaf(sum, exp2_fast((top + shift.x) * kLog2e), s0 + s1);
            top = up;
          }
          if (there) p.sums[(size_t)j * p.chunks + 2 * tl.col + part] = make_float2(top, sum);
        } else if constexpr (MODE == kGrad) {
#pragma unroll 1
          for (int c = part * 64; c < width; c += 128) {
            const int left = args.cols - tl.col0 - c;
            if (left <= 0) break;
            // (the last turn of an odd number of 32 columns)
            const bool narrow = width - c < 64;
            if (lane == 0) tc::bulk_wait_read<0>();   // the store before has read the buffer
            __syncwarp();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (half == 1 && narrow) break;
              uint32_t a[32];
              tc::tmem_ld32(tb + (uint32_t)(c + 32 * half), a);
              tc::tmem_ld_wait();
              float g[32];
#pragma unroll
              for (int i = 0; i < 32; ++i)
                g[i] = there ? scale * exp2_fast((__uint_as_float(a[i]) - lse) * kLog2e) : 0.f;
              const int here = target - c - 32 * half;
              if (__any_sync(0xffffffffu, here >= 0 && here < 32)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i == here) g[i] -= dloss;
              }
              if (left - 32 * half < 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i >= left - 32 * half) g[i] = 0.f;
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float *v = g + q * 8;
                const uint4 w = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                           pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                const int col = tl.col0 + c + q * 8;
                if (!narrow)
                  *reinterpret_cast<uint4 *>(stage_out + lane * 128 +
                                             (((half * 4 + q) ^ (lane & 7)) << 4)) = w;
                else if (j < p.n && col < p.pitch)   // (pitch: whole vectors)
                  *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.dl) +
                                             (int64_t)j * p.pitch + col) = w;
              }
            }
            if (narrow) break;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc::tma_store_3d(&maps.out, stage_out, tl.col0 + c, row, 0);
          }
        } else {
#pragma unroll 1
          for (int c = part * 32; c < width; c += 64) {
            const int col = tl.col0 + c;
            if (col >= args.cols) break;
            uint32_t a[32];
            tc::tmem_ld32(tb + (uint32_t)c, a);
            tc::tmem_ld_wait();
            if (lane == 0) tc::bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4 *>(stage_out + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                  make_uint4(a[q * 4], a[q * 4 + 1], a[q * 4 + 2], a[q * 4 + 3]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              if (p.add) tc::tma_add_3d(&maps.out, stage_out, col, row, tl.z);
              else tc::tma_store_3d(&maps.out, stage_out, col, row, tl.z);
            }
          }
        }
      }
      if constexpr (MODE != kSums) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_first + (uint32_t)(acc * sizeof(uint64_t)));
      }
    }
    if (MODE != kSums && lane == 0) tc::bulk_wait_all();
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
    tmem_dealloc2(tmem_base, L_TMEM_COLS);
  }
  if (threadIdx.x == 0 && sh.abort && !sh.failed_on_entry)
    set_status(args.status, MOE_ERR_TIMEOUT, blockIdx.x);
}

constexpr int kPairs = 76;   // SM pairs that the plans count on

bool bf16_map(CUtensorMap *m, const void *ptr, int rank, const uint64_t *dims, const uint32_t *box) {
  return make_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, rank, dims, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
}

template <LossMode MODE>
cudaError_t launch(const LMaps &maps, const LArgs &a, cudaStream_t s) {
  auto kernel = loss_pair_kernel<MODE>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(L_THREADS);
  cfg.dynamicSmemBytes = L_SMEM;
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
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L_SMEM);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2 * (num_sms() / 2));
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs < 1) {
      cudaGetLastError();
      pairs = num_sms() / 2;
    }
  }
  cfg.gridDim = dim3(2 * pairs);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

// The operands of the logits: rows of x, and of W in boxes of half a tile.
bool logit_maps(const LossProduct &p, int width, LMaps &m) {
  const uint64_t dx[2] = {(uint64_t)p.d, (uint64_t)p.n};
  const uint64_t dw[2] = {(uint64_t)p.d, (uint64_t)p.entries};
  const uint32_t ba[2] = {LK, LM}, bs[2] = {LK, L_SHORT}, bw[2] = {LK, (uint32_t)(width / 2)};
  return bf16_map(&m.A, p.x, 2, dx, ba) && bf16_map(&m.As, p.x, 2, dx, bs) &&
         bf16_map(&m.B, p.W, 2, dw, bw);
}

// Rounds of tiles of this width (columns) on the SM pairs, with what a tile costs
// beside its columns.
int64_t rounds_cost(int64_t tiles, int width) { return (tiles + kPairs - 1) / kPairs * (width + 32); }

}  // namespace

bool loss_pair_supported(const moe_loss_config &c) {
  return c.dtype == MOE_BF16 && tensor_maps_available() && num_sms() >= 2;
}

int loss_width(int n, int vocab) {
  int best = LN;
  int64_t least = INT64_MAX;
  for (int w = LN; w >= 64; w -= 32) {
    const int64_t tiles = (((int64_t)n + 2 * LM - 1) / (2 * LM)) * ((vocab + w - 1) / w);
    const int64_t cost = rounds_cost(tiles, w);
    if (cost < least) {
      least = cost;
      best = w;
    }
  }
  return best;
}

int loss_dx_splits(int n, int d, int entries, int most) {
  const int64_t tiles = (((int64_t)n + 2 * LM - 1) / (2 * LM)) * ((d + LN - 1) / LN);
  const int KB = (entries + LK - 1) / LK;
  int best = 1;
  double least = 1e30;
  // time in units of a k-block's MMAs: rounds of tiles, each with what storing
  // it costs, and the planes' sum
  for (int s = 1; s <= most && s <= KB; ++s) {
    const int each = (KB + s - 1) / s;
    if ((KB + each - 1) / each != s) continue;   // (a range would be empty)
    if (s > 1 && each < 8) break;
    const double cost = (double)((tiles * s + kPairs - 1) / kPairs) * (each + 12) +
                        (double)s * n * d * 4e-6;
    if (cost < 0.97 * least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

cudaError_t launch_loss_sums(const LossProduct &p, int *status, cudaStream_t s) {
  LArgs a{p, p.entries, p.d, p.width, status};
  LMaps m{};
  if (!logit_maps(p, p.width, m)) return cudaErrorInvalidValue;
  return launch<kSums>(m, a, s);
}

cudaError_t launch_loss_logit_grad(const LossProduct &p, int *status, cudaStream_t s) {
  // (in steps of 64 columns, whole stores: 300 tokens, d 7168, 32003 entries 457 us for 432)
  const int width = loss_width(p.n, p.entries);
  LArgs a{p, p.entries, p.d, width, status};
  LMaps m{};
  const uint64_t dout[3] = {(uint64_t)p.pitch, (uint64_t)p.n, 1};
  const uint32_t box[3] = {64, 32, 1};
  if (!logit_maps(p, width, m) || !bf16_map(&m.out, p.dl, 3, dout, box)) return cudaErrorInvalidValue;
  return launch<kGrad>(m, a, s);
}

cudaError_t launch_loss_dx(const LossProduct &p, int *status, cudaStream_t s) {
  LArgs a{p, p.d, p.entries, LN, status};
  LMaps m{};
  const uint64_t da[2] = {(uint64_t)p.pitch, (uint64_t)p.n};
  const uint64_t dw[2] = {(uint64_t)p.d, (uint64_t)p.entries};
  const uint64_t dout[3] = {(uint64_t)p.d, (uint64_t)p.n, (uint64_t)p.splits};
  const uint32_t ba[2] = {LK, LM}, bs[2] = {LK, L_SHORT}, bw[2] = {64, LK}, box[3] = {32, 32, 1};
  if (!bf16_map(&m.A, p.dl, 2, da, ba) || !bf16_map(&m.As, p.dl, 2, da, bs) ||
      !bf16_map(&m.B, p.W, 2, dw, bw) ||
      !make_tensor_map(&m.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.planes, 3, dout, box,
                       CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return launch<kDx>(m, a, s);
}

}  // namespace moe
