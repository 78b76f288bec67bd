// dx = dl W and dW = dl^T x of the cross entropy for few tokens (kLossFewTokens at
// most), in one pass over W.
//
// With so few tokens both products are bound by HBM: dx reads W, dW is as large
// as W and written.  Each on its own moves data one way (dW at the 4.06 TB/s that
// writes alone reach here); together every SM reads and writes at once.
//   A CTA takes 128 columns c of both and a range of the vocabulary, and walks it in
// blocks of 128 entries v.  A block needs dl[t][v] (from L2: all CTAs of a range
// read the same) and W[v][c]; x[t][c] stays in shared memory.
//   D1[t][c] += sum_v dl[t][v] W[v][c]     t on the MMA's M side, one or two tiles
//                                          of 128; kept in tensor memory to the end
//   D2[v][c]  = sum_t dl[t][v] x[t][c]     v on the M side: the same tile of dl, read
//                                          as an M-major operand; drained block by
//                                          block to bf16 and stored
// The ranges' D1 go to fp32 planes [range][t][c], which a later launch adds in order.
// dl's rows from the last counted token to the next multiple of 16 are zero
// (loss_pair.cu stores them so), and x's rows there too.
//
// Roles: warp 0 TMA producer, warp 1 issues the MMAs, warps 2-5 drain D2 and at the
// end D1.  The ring's cut goes by the tokens that count: boxes of a multiple of 32 of
// them, and as many stages as fit.  (With 64 columns dl's way from L2 weighs
// more: 75 tokens counted, 32003 entries, d 7168: the whole gradient 296 us, 246 so;
// as two launches, side by side, 287.)
#include "common.cuh"
#include "launch.h"
#include "loss.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int F_C = 128;                       // columns of a CTA, in two boxes of 64
constexpr int F_V = 128;                       // entries of a block
constexpr int F_BOX = F_V * 64 * 2;            // one box of W: 16 KB
constexpr int F_W = 2 * F_BOX;
constexpr int F_MAX_STAGES = 5;
constexpr int F_RING = 208 * 1024;             // the ring's stages, then x
constexpr int F_OUT = 32 * 128;                // one store: 32 rows of 128 bytes
constexpr int F_EPI = 4;                       // epilogue warps
constexpr int F_THREADS = 32 * (2 + F_EPI);
constexpr size_t F_SMEM = 1024 + F_RING + (size_t)F_EPI * F_OUT;
constexpr uint32_t F_TMEM_COLS = 512;          // D1: two tiles of 128 columns, D2: two buffers
static_assert(F_EPI * F_OUT >= 12 * 1024,
              "an operand of 128 tokens whose box is shorter reads past it, and past x at most this far");

struct FShared {
  uint64_t full[F_MAX_STAGES], empty[F_MAX_STAGES];
  uint64_t xfull;                 // x landed
  uint64_t d2full[2], d2empty[2];
  uint64_t done;                  // the last MMA completed
  uint32_t tmem_base;
  int abort, failed_on_entry, counted;
};
struct FArgs {
  int n, d, entries, splits;
  int want_dx, want_dw, add;
  const int32_t *range;
  const float *scale;   // dW's sums are multiplied by it
  int *status;
};
struct FMaps {
  CUtensorMap dl[4], x[4];   // boxes of 64 entries, or columns, x 32, 64, 96, 128 tokens
  CUtensorMap W, dW, planes;
};

// How the counted tokens cut the ring: tokens of the one or two tiles' boxes (rows of
// 128 bytes), bytes of a box of x, of a stage, and how many stages.
struct FCut {
  int rows[2], tiles, x_box, stage_bytes, stages;
};
__device__ __forceinline__ FCut cut_of(int m) {
  FCut c;
  const int all = (m + 31) / 32 * 32;
  c.tiles = all > 128 ? 2 : 1;
  c.rows[0] = min(all, 128);
  c.rows[1] = all - c.rows[0];
  c.x_box = all * 128;
  c.stage_bytes = F_W + 2 * all * 128;
  c.stages = min(F_MAX_STAGES, (F_RING - 2 * c.x_box) / c.stage_bytes);
  return c;
}

__global__ void __launch_bounds__(F_THREADS, 1)
loss_few_kernel(const __grid_constant__ FMaps maps, const __grid_constant__ FArgs args) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ FShared sh;
  uint8_t *smem = dyn_smem + ((1024 - (tc::smem_u32(dyn_smem) & 1023)) & 1023);
  uint8_t *out_smem = smem + F_RING;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x * F_C, z = blockIdx.y;
  // this CTA's blocks of the vocabulary
  const int blocks = (args.entries + F_V - 1) / F_V, each = (blocks + args.splits - 1) / args.splits;
  const int vb0 = z * each, vb1 = min(blocks, vb0 + each);

  if (warp == 1) tc::tmem_alloc(&sh.tmem_base, F_TMEM_COLS);
  if (threadIdx.x == 0) {
    for (int s = 0; s < F_MAX_STAGES; ++s) {
      tc::mbar_init(&sh.full[s], 1);
      tc::mbar_init(&sh.empty[s], 1);
    }
    tc::mbar_init(&sh.xfull, 1);
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&sh.d2full[a], 1);
      tc::mbar_init(&sh.d2empty[a], F_EPI);
    }
    tc::mbar_init(&sh.done, 1);
    tc::fence_mbar_init();
    tc::prefetch_tmap(&maps.W);
    tc::prefetch_tmap(&maps.dW);
  }
  // (all above ran beside the end of the kernel before; from here on its
  // results are read)
  pdl_wait();
  if (threadIdx.x == 0) {
    sh.failed_on_entry = status_failed(args.status) ? 1 : 0;
    sh.abort = sh.failed_on_entry;
    sh.counted = min(max(args.range[1], 0), args.n);
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;
  const int m = sh.counted;
  const FCut cut = cut_of(m);
  uint8_t *x_smem = smem + cut.stages * cut.stage_bytes;
  const bool want_dx = args.want_dx && m > 0;
  volatile int *abort = &sh.abort;
  const uint32_t d2_base = tmem_base + 2 * F_C;

  if (warp == 0) {
    // ---------------- TMA producer
    if (lane == 0 && m > 0 && !*abort) {
      int stage = 0;
      uint32_t phase = 0, used = 0, used_phase = 0;
      if (args.want_dw) {
        tc::mbar_arrive_expect_tx(&sh.xfull, 2 * cut.x_box);
        for (int t = 0; t < cut.tiles; ++t)
          for (int h = 0; h < 2; ++h)
            tc::tma_load_2d(&maps.x[cut.rows[t] / 32 - 1], &sh.xfull,
                            x_smem + h * cut.x_box + t * 128 * 128, c0 + h * 64, t * 128);
      }
      const uint32_t bytes = cut.stage_bytes - (want_dx ? 0 : F_W);
      for (int vb = vb0; vb < vb1; ++vb) {
        if (!tc::mbar_wait(&sh.empty[stage], phase ^ 1u, abort)) break;
        uint8_t *at = smem + stage * cut.stage_bytes;
        used |= 1u << stage;
        used_phase = phase ? used_phase | 1u << stage : used_phase & ~(1u << stage);
        tc::mbar_arrive_expect_tx(&sh.full[stage], bytes);
        if (want_dx) {
          tc::tma_load_2d(&maps.W, &sh.full[stage], at, c0, vb * F_V);
          tc::tma_load_2d(&maps.W, &sh.full[stage], at + F_BOX, c0 + 64, vb * F_V);
        }
        at += F_W;
        for (int t = 0; t < cut.tiles; ++t) {
          const CUtensorMap *dl = &maps.dl[cut.rows[t] / 32 - 1];
          for (int h = 0; h < 2; ++h) {
            tc::tma_load_2d(dl, &sh.full[stage], at, vb * F_V + h * 64, t * 128);
            at += cut.rows[t] * 128;
          }
        }
        if (++stage == cut.stages) { stage = 0; phase ^= 1u; }
      }
      if (*abort) {
        // let the copies in flight land before the CTA exits
        if (args.want_dw) tc::mbar_wait_drain(&sh.xfull, 0, 100000000ull);
        for (int s = 0; s < F_MAX_STAGES; ++s)
          if ((used >> s) & 1u)
            tc::mbar_wait_drain(&sh.full[s], (used_phase >> s) & 1u, 100000000ull);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer
    if (lane == 0 && m > 0) {
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = !args.want_dw || tc::mbar_wait(&sh.xfull, 0, abort);
      const uint32_t idesc1 = tc::idesc_bf16_f32(128, F_C) | tc::kIdescBMajorMN;
      const uint32_t idesc2 = idesc1 | tc::kIdescAMajorMN;
      const int steps = (m + 15) / 16;   // of 16 tokens, 8 in a tile
      const int box[2] = {cut.rows[0] * 128, cut.rows[1] * 128};
      for (int vb = vb0; vb < vb1 && ok && !*abort; ++vb, ++local) {
        const int acc = local & 1;
        if (args.want_dw && !tc::mbar_wait(&sh.d2empty[acc], ((local >> 1) & 1) ^ 1u, abort)) break;
        if (!tc::mbar_wait(&sh.full[stage], phase, abort)) break;
        tc::tc_fence_after();
        const uint32_t w = tc::smem_u32(smem + stage * cut.stage_bytes), dl = w + F_W;
        if (args.want_dw) {
          for (int k = 0; k < steps; ++k) {
            const uint32_t a = dl + (k < 8 ? k * 2048 : 2 * box[0] + (k - 8) * 2048);
            const uint32_t b = tc::smem_u32(x_smem) + k * 2048;
            tc::mma_bf16(d2_base + acc * F_C, tc::smem_desc_sw128_mn(a, k < 8 ? box[0] : box[1]),
                         tc::smem_desc_sw128_mn(b, cut.x_box), idesc2, k != 0);
          }
          tc::mma_commit(&sh.d2full[acc]);
        }
        if (want_dx) {
          for (int t = 0; t < cut.tiles; ++t) {
#pragma unroll
            for (int k = 0; k < F_V / 16; ++k) {
              const uint32_t a = dl + t * 2 * box[0] + (k >> 2) * box[t] + (k & 3) * 32;
              tc::mma_bf16(tmem_base + t * F_C, tc::smem_desc_sw128(a),
                           tc::smem_desc_sw128_mn(w + k * 2048, F_BOX), idesc1, vb != vb0 || k != 0);
            }
          }
        }
        tc::mma_commit(&sh.empty[stage]);
        if (++stage == cut.stages) { stage = 0; phase ^= 1u; }
      }
      tc::mma_commit(&sh.done);
      if (*abort) tc::mbar_wait_drain(&sh.done, 0, 100000000ull);
    }
  } else {
    // ---------------- epilogue: warp w drains TMEM lanes 32*(w%4) .. +31
    const int quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    uint8_t *buf = out_smem + (warp - 2) * F_OUT, *mine = buf + lane * 128;
    // this warp's buffer once the store before has read it, and its next store
    auto reuse = [&]() {
      if (lane == 0) tc::bulk_wait_read<0>();
      __syncwarp();
    };
    auto flush = [&](const CUtensorMap *map, int x, int y, int zz, bool add) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        if (add) tc::tma_add_3d(map, buf, x, y, zz);
        else tc::tma_store_3d(map, buf, x, y, zz);
      }
    };
    bool ok = !sh.failed_on_entry;
    const float scale = *args.scale;
    if (args.want_dw) {
      int local = 0;
      for (int vb = vb0; vb < vb1 && ok; ++vb, ++local) {
        const int acc = local & 1, row = vb * F_V + quarter * 32;
        if (m > 0) {
          ok = __all_sync(0xffffffffu, tc::mbar_wait(&sh.d2full[acc], (local >> 1) & 1, abort));
          if (!ok) break;
          tc::tc_fence_after();
        }
        for (int half = 0; half < 2; ++half) {
          uint32_t a[2][32];
          if (m > 0) {
            const uint32_t from = d2_base + lane_base + acc * F_C + half * 64;
            tc::tmem_ld32(from, a[0]);
            tc::tmem_ld32(from + 32, a[1]);
            tc::tmem_ld_wait();
            if (half == 1) {
              tc::tc_fence_before();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&sh.d2empty[acc]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) a[0][i] = a[1][i] = 0;
          }
          if (row >= args.entries || c0 + half * 64 >= args.d) continue;
          reuse();
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t *v = &a[q >> 2][(q & 3) * 8];
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[2 * i]) * scale,
                                                             __uint_as_float(v[2 * i + 1]) * scale);
              w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(mine + ((q ^ (lane & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          flush(&maps.dW, c0 + half * 64, row, 0, false);
        }
      }
    }
    if (ok && want_dx) {
      ok = tc::mbar_wait(&sh.done, 0, abort) && !*abort;
      ok = __all_sync(0xffffffffu, ok);
      tc::tc_fence_after();
      for (int t = 0; t < cut.tiles && ok; ++t) {
        const int row = t * 128 + quarter * 32;
        if (row >= m) break;
        for (int c = 0; c < F_C && c0 + c < args.d; c += 32) {
          uint32_t a[32];
          tc::tmem_ld32(tmem_base + lane_base + t * F_C + c, a);
          tc::tmem_ld_wait();
          reuse();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint4 *>(mine + ((q ^ (lane & 7)) << 4)) =
                make_uint4(a[q * 4], a[q * 4 + 1], a[q * 4 + 2], a[q * 4 + 3]);
          flush(&maps.planes, c0 + c, row, z, args.add);
        }
      }
    }
    if (lane == 0) tc::bulk_wait_all();
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem_base, F_TMEM_COLS);
  }
  if (threadIdx.x == 0 && sh.abort && !sh.failed_on_entry)
    set_status(args.status, MOE_ERR_TIMEOUT, blockIdx.x);
}

}  // namespace

// Ranges of the vocabulary, so that rounds of CTAs on 152 SMs are nearly full; a CTA
// costs some blocks beside its own (set-up, D1's store).
int loss_few_splits(int d, int entries, int most) {
  const int64_t columns = (d + F_C - 1) / F_C;
  const int blocks = (entries + F_V - 1) / F_V;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= most && s <= blocks; ++s) {
    const int each = (blocks + s - 1) / s;
    if ((blocks + each - 1) / each != s) continue;   // (a range would be empty)
    const int64_t cost = (columns * s + 151) / 152 * (each + 8);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

cudaError_t launch_loss_few(const LossProduct &p, void *dW, bool want_dx, int *status,
                            cudaStream_t s) {
  FArgs a{p.n, p.d, p.entries, p.splits, want_dx, dW != nullptr, p.add, p.range, p.scale, status};
  FMaps m{};
  auto bf16_map = [](CUtensorMap *t, const void *ptr, int rank, const uint64_t *dims,
                     const uint32_t *box) {
    return make_tensor_map(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, rank, dims, box,
                           CU_TENSOR_MAP_SWIZZLE_128B);
  };
  const uint64_t ddl[2] = {(uint64_t)p.pitch, (uint64_t)p.n};
  const uint64_t dx[2] = {(uint64_t)p.d, (uint64_t)p.n};
  const uint64_t dw[3] = {(uint64_t)p.d, (uint64_t)p.entries, 1};
  const uint64_t dp[3] = {(uint64_t)p.d, (uint64_t)p.n, (uint64_t)p.splits};
  const uint32_t tile[2] = {64, F_V}, store[3] = {64, 32, 1}, plane[3] = {32, 32, 1};
  for (int i = 0; i < 4; ++i) {
    const uint32_t box[2] = {64, 32u * (i + 1)};
    if (!bf16_map(&m.dl[i], p.dl, 2, ddl, box) || !bf16_map(&m.x[i], p.x, 2, dx, box))
      return cudaErrorInvalidValue;
  }
  if (!bf16_map(&m.W, p.W, 2, dw, tile) ||
      !bf16_map(&m.dW, dW ? dW : p.W, 3, dw, store) ||
      !make_tensor_map(&m.planes, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.planes, 3, dp, plane,
                       CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  static bool set = false;
  if (!set) {
    const cudaError_t e = cudaFuncSetAttribute(
        loss_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)F_SMEM);
    if (e != cudaSuccess) return e;
    set = true;
  }
  return launch_pdl(loss_few_kernel, dim3((p.d + F_C - 1) / F_C, p.splits), dim3(F_THREADS), F_SMEM, s,
                    m, a);
}

}  // namespace moe
