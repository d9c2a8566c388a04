// Weight gradient of a linear on tcgen05:
//   dw[n][k] = sum_m dz[m][n] * x[m][k]     (BF16 x BF16, FP32 sums).
//
// The contraction runs over the tokens, the rows of both operands, so both
// are "MN-major" to the tensor cores: their contiguous dimension is the
// output's. TMA brings boxes of 64 tokens x 64 columns (128 bytes, 128-byte
// swizzle) and the MMA descriptors name that order, so nothing is transposed.
// Tokens past M are zero-filled by TMA in both operands.
//
// What bounds it is the tensor pipe, if the operands arrive: a 128 x 256 tile
// on one SM would load 48 KB per 512 MMA cycles, 96 bytes per clock and SM,
// about what L2 can deliver. So two SMs (a cluster of two CTAs, cta_group::2)
// share a 256 x 256 tile: each loads its 128 rows of dz^T and its 128 columns
// of x (32 KB per 64 tokens, 64 bytes per clock), holds its 128 output rows in
// TMEM, and the pair's MMA (M = 256, N = 256, K = 16) reads the operands of
// both. The accumulator is double-buffered (2 x 256 of the 512 TMEM columns),
// so a tile's stores overlap the next tile's products.
//
// Roles per CTA (12 warps):
//   warp 0   lanes 0, 1: TMA producers of the two 64-column boxes of dz;
//   warp 1   lanes 0, 1: of x. Loads of both CTAs complete on the stage's
//            barrier in the leader (CTA rank 0 of the pair);
//   warp 2   leader: MMA issuer; both: TMEM allocation;
//   warps 4-11  epilogue: warp 4 + 4h + q owns TMEM lane quadrant q and
//            columns [128h, 128h + 128) of its CTA's 128 x 256 accumulator.
// A commit stalls its issuer for a few hundred cycles, so stages are released
// in pairs: one commit per 8 MMAs (1024 cycles of the pair's tensor pipes).
// Every wait is bounded (kWaitLimitCycles) and reports to the error word.
//
// Few tiles and many tokens (a 1024 x 1024 weight is 16 tiles for 74 pairs): given
// a workspace, the tokens are split into runs, each (tile, run) is a unit of
// work that stores its FP32 sums there, and grad_join_kernel adds the runs in
// order.
#include <cuda_bf16.h>

#include <cstring>

#include "internal.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

struct GradCfg {
  static constexpr int BT = 64;                    // tokens per stage
  static constexpr int TILE = 256;                 // output rows and columns of a pair's tile
  static constexpr int BOX_BYTES = BT * 128;       // 64 tokens x 64 BF16
  static constexpr int OP_BYTES = 2 * BOX_BYTES;   // one operand's 128 columns
  static constexpr int STAGE_BYTES = 2 * OP_BYTES; // both operands of this CTA
  static constexpr int ST = 6;                     // stages, released two at a time
  static constexpr int PAIRS = ST / 2;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int OUT_BYTES = 32 * 128;       // per epilogue warp: 32 rows x 128 B
  static constexpr int NBAR = ST + PAIRS + 4;
  static constexpr size_t SMEM_TILES =
      static_cast<size_t>(ST) * STAGE_BYTES + static_cast<size_t>(EPI_WARPS) * OUT_BYTES;
  static constexpr size_t SMEM = 1024 + SMEM_TILES + 8 * NBAR + 16;
  // Both operands MN-major (bits 15 and 16).
  static constexpr uint32_t IDESC = make_idesc(1u, 1u, 256, 256) | (1u << 15) | (1u << 16);
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(ST % 2 == 0, "stages are released in pairs");
};

// ------------------------------------------------------- CTA-pair instructions
// Arrival on a barrier of the pair that says only that this warp's TMEM reads are
// done (ordered by tcgen05.wait and the tcgen05 fences on both sides): no memory
// is handed over, and a release at cluster scope, which waits for the warp's
// stores in flight, cost about 2500 cycles per tile here.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 2-D tile load into this CTA's shared memory, counted on a barrier of the
// pair (own or peer's; an address in the cluster's shared window).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// One arrival on the barrier at this offset in both CTAs of the pair when all
// MMAs issued so far by this thread have completed.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// D[tmem of both] (+)= A * B, A and B in the shared memory of both CTAs.
__device__ __forceinline__ void mma_f16_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Tile store that adds to what is there (FP32).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, const void* src, int32_t c0,
                                           int32_t c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(c0), "r"(c1)
               : "memory");
}

// Descriptor of an MN-major operand tile: boxes of 64 columns (128 bytes,
// 128-byte swizzle) x BT tokens. Eight tokens are one 1024-byte swizzle atom
// (stride byte offset); the next 64 columns are one box further (leading byte
// offset). Sixteen tokens (one MMA's K) advance the start address by 2048.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(GradCfg::BOX_BYTES >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

template <bool FP32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GradCfg::THREADS, 1)
    grad_weight_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                       const __grid_constant__ CUtensorMap tm_w, void* __restrict__ dw, int64_t lddw,
                       int N, int K, int k_tma, int all_steps, int run_steps, int run_rows,
                       int ktiles, int tiles, int gk, int accumulate, unsigned* __restrict__ err) {
  using C = GradCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;                 // ST stages: dz (two boxes), x (two boxes)
  uint8_t* sOut = smem + C::ST * C::STAGE_BYTES;  // EPI_WARPS x 4 KB staging
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::SMEM_TILES);
  uint64_t* full = bars;                // leader: stage landed in both CTAs (4 arrivals + tx)
  uint64_t* empty = full + C::ST;       // stage pair read by the MMAs       (1 commit)
  uint64_t* acc_full = empty + C::PAIRS;  // accumulator complete            (1 commit)
  uint64_t* acc_empty = acc_full + 2;     // leader: accumulator read        (16 epilogue warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = static_cast<int>(blockIdx.x >> 1), npairs = static_cast<int>(gridDim.x >> 1);
  const int ntiles_n = tiles / ktiles;
  // Units of work: (tile, run of run_steps stages); one run unless the tokens
  // are split, and then run r stores at row r * run_rows.
  const int runs = (all_steps + run_steps - 1) / run_steps, units = tiles * runs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) mbar_init(&full[s], 4);
    for (int p = 0; p < C::PAIRS; ++p) mbar_init(&empty[p], 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);
    }
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and TMEM exist
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_launch_dependents();  // the kernel after this one waits for this grid before it reads dw

  if (warp < 2) {
    if (lane < 2) {
      // ------------------------------------------------------- producers
      const CUtensorMap* map = warp == 0 ? &tm_a : &tm_b;
      uint8_t* dst = smem + warp * C::OP_BYTES + lane * C::BOX_BYTES;
      const uint32_t full0 = map_to_rank(full, 0);
      tma_prefetch_map(map);
      int j = 0;
      bool ok = true;
      for (int unit = pair; unit < units && ok; unit += npairs) {
        int kt, nt;
        tile_coords(unit / runs, ktiles, ntiles_n, gk, kt, nt);
        const int s0 = unit % runs * run_steps, s1 = min(s0 + run_steps, all_steps);
        const int col = (warp == 0 ? nt : kt) * C::TILE + static_cast<int>(rank) * 128 + lane * 64;
        for (int s = s0; s < s1; ++s, ++j) {
          const int stage = j % C::ST;
          if ((stage & 1) == 0 && j >= C::ST) {  // the pair's last use has been read
            if (!mbar_wait(&empty[stage >> 1], static_cast<uint32_t>((j / C::ST - 1) & 1), err,
                           kErrWaitLoad)) {
              ok = false;
              break;
            }
          }
          // The leader's barrier counts this box and the peer's.
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::BOX_BYTES);
          tma_load_2d_pair(dst + stage * C::STAGE_BYTES, map, full0 + 8u * stage, col, s * C::BT);
        }
      }
      // Drain: the leader waits until the last stages have landed in both
      // CTAs; the peer is kept alive by the cluster barrier at the end.
      if (rank == 0)
        for (int jj = (j > C::ST ? j - C::ST : 0); jj < j; ++jj)
          mbar_wait(&full[jj % C::ST], static_cast<uint32_t>((jj / C::ST) & 1), err, kErrWaitLoad);
    }
  } else if (warp == 2) {
    if (rank == 0 && lane == 0) {
      // ------------------------------------------------------ MMA issuer
      const uint64_t a0 = sw128_mnmajor_desc(smem_addr(smem));
      const uint64_t b0 = sw128_mnmajor_desc(smem_addr(smem + C::OP_BYTES));
      int j = 0, it = 0;
      bool ok = true;
      for (int unit = pair; unit < units && ok; unit += npairs, ++it) {
        const int buf = it & 1;
        const int s0 = unit % runs * run_steps, steps = min(run_steps, all_steps - s0);
        if (it >= 2) {
          if (!mbar_wait(&acc_empty[buf], static_cast<uint32_t>(((it >> 1) - 1) & 1), err, kErrWaitMma)) break;
          tc_fence_after_sync();
        }
        const uint32_t d = tmem + static_cast<uint32_t>(buf * C::TILE);
        for (int s = 0; s < steps; ++s, ++j) {
          const int stage = j % C::ST;
          if (!mbar_wait(&full[stage], static_cast<uint32_t>((j / C::ST) & 1), err, kErrWaitMma)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t off = static_cast<uint64_t>((stage * C::STAGE_BYTES) >> 4);
#pragma unroll
          for (int q = 0; q < C::BT / 16; ++q)
            mma_f16_ss_pair(d, a0 + off + (2048u >> 4) * q, b0 + off + (2048u >> 4) * q, C::IDESC,
                            s > 0 || q > 0 ? 1u : 0u);
          if (stage & 1) tc_commit_pair(&empty[stage >> 1]);
        }
        if (ok) tc_commit_pair(&acc_full[buf]);
      }
      // Drain: all MMAs complete before TMEM is released and either CTA
      // leaves (the last accumulator's commit is the last one).
      if (it > 0 && ok)
        mbar_wait(&acc_full[(it - 1) & 1], static_cast<uint32_t>(((it - 1) >> 1) & 1), err, kErrWaitMma);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 4, quad = warp & 3, h = ew >> 2;
    uint8_t* stage = sOut + ew * C::OUT_BYTES;
    uint8_t* srow = stage + lane * 128;
    const uint32_t acc_empty0 = map_to_rank(acc_empty, 0);
    constexpr int CW = FP32 ? 32 : 64;       // columns of a 128-byte staging row
    constexpr int EPC = FP32 ? 4 : 8;        // elements of a 16-byte chunk
    int it = 0;
    for (int unit = pair; unit < units; unit += npairs, ++it) {
      int kt, nt;
      tile_coords(unit / runs, ktiles, ntiles_n, gk, kt, nt);
      const int row_off = unit % runs * run_rows;
      const int buf = it & 1;
      if (!mbar_wait_warp(&acc_full[buf], static_cast<uint32_t>((it >> 1) & 1), err, kErrWaitEpilogue)) break;
      tc_fence_after_sync();
      const uint32_t t = tmem + (static_cast<uint32_t>(quad * 32) << 16) +
                         static_cast<uint32_t>(buf * C::TILE + 128 * h);
      const int r0 = nt * C::TILE + static_cast<int>(rank) * 128 + quad * 32;  // first output row
      const int n = r0 + lane;
      // All 128 columns into registers at once: one load's latency instead of
      // four (about 450 cycles each here), and the accumulator is released
      // before the stores.
      uint32_t p[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32x32_issue(t + 32u * i, p[i]);
      tmem_ld_wait(p[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) reg_fence(p[i]);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8u * buf);
#pragma unroll
      for (int i = 0; i < 128 / CW; ++i) {
        const int base = kt * C::TILE + 128 * h + CW * i;  // first output column
        uint4 o[8];
        if constexpr (FP32) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            o[c] = make_uint4(p[i][4 * c], p[i][4 * c + 1], p[i][4 * c + 2], p[i][4 * c + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t* f = &p[2 * i + c / 4][8 * (c % 4)];
            auto w = [&](int e) { return cvt_bf16x2(__uint_as_float(f[e + 1]), __uint_as_float(f[e])); };
            o[c] = make_uint4(w(0), w(2), w(4), w(6));
          }
        }
        if (lane == 0) tma_store_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(srow + ((c ^ (lane & 7)) << 4)) = o[c];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && r0 < N && base < k_tma) {
          if (FP32 && accumulate)
            tma_add_2d(&tm_w, stage, base, row_off + r0);
          else
            tma_store_2d(&tm_w, stage, base, row_off + r0);
          tma_store_commit();
        }
        // The columns of a ragged K past the last whole 16 bytes.
        if (k_tma < K && k_tma >= base && k_tma < base + CW && n < N) {
          const uint8_t* src = srow + ((((k_tma - base) / EPC) ^ (lane & 7)) << 4);
          const int64_t at = static_cast<int64_t>(n) * lddw + k_tma;
          for (int e = 0; e < K - k_tma; ++e) {
            if constexpr (FP32) {
              float* w = static_cast<float*>(dw) + at + e;
              const float v = reinterpret_cast<const float*>(src)[e];
              *w = accumulate ? *w + v : v;
            } else {
              static_cast<uint16_t*>(dw)[at + e] = reinterpret_cast<const uint16_t*>(src)[e];
            }
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_all();
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may still signal it or read it
  if (warp == 2) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, 512);
  }
}

// dw (+)= the sum of the runs, in order; parts is [runs][rows][ld] FP32, four
// columns per thread, ld a multiple of 4 that covers K.
template <bool FP32>
__global__ void __launch_bounds__(256)
    grad_join_kernel(const float* __restrict__ parts, int runs, int64_t rows, int64_t ld, void* dw,
                     int64_t lddw, int64_t N, int64_t K, int accumulate) {
  pdl_wait();
  const int64_t per = ld / 4, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = i / per, k = i % per * 4;
  if (n >= N) return;
  const float* p = parts + n * ld + k;
  float4 a = *reinterpret_cast<const float4*>(p);
#pragma unroll 4
  for (int r = 1; r < runs; ++r) {
    const float4 b = *reinterpret_cast<const float4*>(p + r * rows * ld);
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
  }
  const float v[4] = {a.x, a.y, a.z, a.w};
  if constexpr (FP32) {
    float* w = static_cast<float*>(dw) + n * lddw + k;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k + e < K) w[e] = accumulate ? w[e] + v[e] : v[e];
  } else {
    uint16_t* w = static_cast<uint16_t*>(dw) + n * lddw + k;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k + e < K) w[e] = static_cast<uint16_t>(cvt_bf16x2(0.0f, v[e]));
  }
}

// How the tokens are split: runs of whole stages, chosen from the sizes alone (for
// the 74 CTA pairs of a B200; the sums do not depend on how many there are). Runs
// are at least kMinRunSteps stages (512 tokens) long, and all units run at once.
// Measured, whole -> split, FP32 out: 1024 x 1024 weights, 1024 tokens 11.5 -> 12.2 us,
// 2048 16.4 -> 14.3, 4096 26.4 -> 17.0; 256 x 256, 1024 tokens 11.0 -> 10.0, 4096 25.4 ->
// 11.5. With runs of 256 tokens, 512 tokens of 1024 x 1024 went 8.9 -> 10.8, 1024 -> 12.6.
constexpr int64_t kGradPairs = 74, kMinRunSteps = 8;
struct TokenSplit {
  int64_t run_steps, runs;
};
TokenSplit token_split(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = cdiv(N, GradCfg::TILE) * cdiv(K, GradCfg::TILE), steps = cdiv(M, GradCfg::BT);
  int64_t runs = kGradPairs / tiles;
  if (runs > steps / kMinRunSteps) runs = steps / kMinRunSteps;
  if (runs < 2) return {steps, 1};
  const int64_t run_steps = cdiv(steps, runs);
  return {run_steps, cdiv(steps, run_steps)};
}

// Pairs that can be resident at once (queried once per device and form).
template <bool FP32>
cudaError_t resident_pairs(int num_sms, int* pairs) {
  static int known[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms / 2 * 2));
    cfg.blockDim = dim3(GradCfg::THREADS);
    cfg.dynamicSmemBytes = GradCfg::SMEM;
    e = cudaOccupancyMaxActiveClusters(&n, grad_weight_kernel<FP32>, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (n > num_sms / 2) n = num_sms / 2;
    __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  }
  *pairs = n;
  return cudaSuccess;
}

// Output columns (x) whose operand columns a raster group may keep in L2.
constexpr int64_t kRasterBytesGrad = 48ll << 20;

// The product of N x K sums into [N][ldw] at w (FP32 or BF16), or, split into
// runs, into [runs][run_rows][ldw] FP32.
template <bool FP32>
cudaError_t launch_grad(const Launch& L, const uint16_t* dz, int64_t lddz, const uint16_t* x,
                        int64_t ldx, void* w, int64_t ldw, bool accumulate, int64_t M, int64_t N,
                        int64_t K, const TokenSplit& split, int64_t run_rows) {
  using C = GradCfg;
  CUtensorMap ta, tb, tw;
  if (!make_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dz, N, M, 2 * lddz, 64, C::BT) ||
      !make_tmap_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, K, M, 2 * ldx, 64, C::BT))
    return cudaErrorInvalidValue;
  constexpr int kEsz = FP32 ? 4 : 2;
  // A run's rows and columns are padded to what the stores write.
  const int64_t k_out = split.runs > 1 ? ldw : K;
  const int64_t rows_out = split.runs > 1 ? split.runs * run_rows : N;
  const int64_t k_tma = k_out & ~int64_t{16 / kEsz - 1};  // whole 16-byte chunks
  if (k_tma > 0) {
    if (!make_tmap_2d(&tw, FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      w, k_tma, rows_out, kEsz * ldw, 128 / kEsz, 32))
      return cudaErrorInvalidValue;
  } else {
    memset(&tw, 0, sizeof(tw));
  }
  auto kern = grad_weight_kernel<FP32>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = resident_pairs<FP32>(L.num_sms, &pairs);
  if (e != cudaSuccess) return e;
  const int64_t ktiles = cdiv(K, C::TILE), tiles = ktiles * cdiv(N, C::TILE), steps = cdiv(M, C::BT);
  const int64_t units = tiles * split.runs;
  if (tiles * steps > 0x7FFFFFFFLL || rows_out > 0x7FFFFFFFLL) return cudaErrorInvalidValue;  // 32-bit counters
  if (units < pairs) pairs = static_cast<int>(units);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = L.stream;
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, tw, w, ldw, static_cast<int>(N),
                            static_cast<int>(k_out), static_cast<int>(k_tma), static_cast<int>(steps),
                            static_cast<int>(split.run_steps), static_cast<int>(run_rows),
                            static_cast<int>(ktiles), static_cast<int>(tiles),
                            raster_group(ktiles, C::TILE * M * 2, kRasterBytesGrad),
                            accumulate ? 1 : 0, L.err);
}

int64_t run_rows_of(int64_t N) { return round_up(N, GradCfg::TILE); }

cudaError_t launch_split_grad(const Launch& L, const uint16_t* dz, int64_t lddz, const uint16_t* x,
                              int64_t ldx, void* dw, int64_t lddw, bool fp32, bool accumulate,
                              int64_t M, int64_t N, int64_t K, const TokenSplit& split, float* ws) {
  const int64_t rows = run_rows_of(N), ld = round_up(K, 4);
  cudaError_t e = launch_grad<true>(L, dz, lddz, x, ldx, ws, ld, false, M, N, K, split, rows);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(N * (ld / 4), 256)));
  cfg.blockDim = dim3(256);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp32 ? grad_join_kernel<true> : grad_join_kernel<false>,
                            static_cast<const float*>(ws), static_cast<int>(split.runs), rows, ld, dw,
                            lddw, N, K, accumulate ? 1 : 0);
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" {

size_t fp8blk_linear_grad_weight_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const TokenSplit s = token_split(M, N, K);
  return s.runs < 2 ? 0
                    : static_cast<size_t>(s.runs) * static_cast<size_t>(run_rows_of(N)) *
                          static_cast<size_t>(round_up(K, 4)) * sizeof(float);
}

fp8blk_status fp8blk_linear_grad_weight(const void* dz, int64_t lddz, const void* x, int64_t ldx,
                                        void* dw, int64_t lddw, int32_t dw_fp32, int32_t accumulate,
                                        int64_t M, int64_t N, int64_t K, void* workspace,
                                        size_t workspace_bytes, fp8blk_stream stream) {
  if (M < 0 || N < 0 || K < 0) return FP8BLK_ERR_INVALID_ARG;
  if ((dw_fp32 != 0 && dw_fp32 != 1) || (accumulate != 0 && accumulate != 1) ||
      (accumulate && !dw_fp32))
    return FP8BLK_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return FP8BLK_OK;
  if (!dw || lddw < K || M > kInt32Max || N > kInt32Max || K > kInt32Max) return FP8BLK_ERR_INVALID_ARG;
  if (lddw % (dw_fp32 ? 4 : 8) || !aligned(dw, 16)) return FP8BLK_ERR_ALIGNMENT;
  if (M > 0) {
    if (!dz || !x || lddz < N || ldx < K) return FP8BLK_ERR_INVALID_ARG;
    if (lddz % 8 || ldx % 8 || !aligned(dz, 16) || !aligned(x, 16)) return FP8BLK_ERR_ALIGNMENT;
    if (one_of(dw, dz, x)) return FP8BLK_ERR_INVALID_ARG;
  } else if (accumulate) {
    return FP8BLK_OK;
  }
  Launch L;
  fp8blk_status st = current_launch(stream, &L);
  if (st != FP8BLK_OK) return st;
  if (M == 0) {  // an empty sum
    const size_t esz = dw_fp32 ? 4 : 2;
    return cuda_status(cudaMemset2DAsync(dw, static_cast<size_t>(lddw) * esz, 0,
                                         static_cast<size_t>(K) * esz, static_cast<size_t>(N), L.stream));
  }
  const uint16_t* a = static_cast<const uint16_t*>(dz);
  const uint16_t* b = static_cast<const uint16_t*>(x);
  TokenSplit split = token_split(M, N, K);
  const size_t need = fp8blk_linear_grad_weight_workspace_size(M, N, K);
  if (need && workspace && workspace_bytes >= need && aligned(workspace, 256))
    return cuda_status(launch_split_grad(L, a, lddz, b, ldx, dw, lddw, dw_fp32 != 0, accumulate != 0,
                                         M, N, K, split, static_cast<float*>(workspace)));
  split = {cdiv(M, GradCfg::BT), 1};
  return cuda_status(
      dw_fp32 ? launch_grad<true>(L, a, lddz, b, ldx, dw, lddw, accumulate != 0, M, N, K, split, 0)
              : launch_grad<false>(L, a, lddz, b, ldx, dw, lddw, false, M, N, K, split, 0));
}

}  // extern "C"
