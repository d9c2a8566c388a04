// Block-scaled FP8 x FP8 linear (W8A8) on tcgen05:
//   y[m][n] = BF16( sum_kb sx[kb][m] * s[n/128][kb] * P_kb[m][n] ),
//   P_kb = (128-wide K slab of qx) . (same slab of q)^T, E4M3 x E4M3 -> FP32.
// FastVideo PR #1829, "Purpose": the linear is x times the dequantized weight,
// computed the way the Blackwell groupwise GEMM does it (scales applied per
// 128-wide K group). The scales are arbitrary floats, not powers of two, and
// the weight blocks are 128 x 128, so they are applied in software to each
// slab's FP32 partial ("promotion") rather than by the MMA.
//
// Persistent kernel: one CTA per SM walks output tiles of 128 tokens by 256
// weight rows (two weight blocks) in raster groups (tile_coords): the token
// tiles of one weight tile are neighbours and share it through L2, and a
// group of token tiles (at most 24 MB of activation codes) meets every
// weight tile before the next group starts.
// Every ring runs on across tiles, so the next tile's loads and MMAs overlap
// this tile's stores.
//
// The single-thread control loops set the pace on this part: a commit stalls
// its issuer's MMA stream for a few hundred cycles and every barrier or TMA
// operation costs on the order of a hundred cycles of that thread's time. So
// the work per control operation is made large (one N=256 MMA covers a whole
// 128 x 256 x 32 step; one stage barrier covers a whole slab), the control
// work is spread over four threads, and ring positions are powers of two.
//   warp 0     TMA producer of the activation slab [128 x 128 B] per stage;
//   warp 1     TMA producer of the weight slab [256 x 128 B] per stage;
//   warp 2, 3  MMA issuers: issuer e takes the slabs j with j % 2 == e, each
//              4 x (M=128, N=256, K=32) into its own 256-column TMEM partial,
//              then one commit to the slab's "done" barrier. While one issuer
//              waits or commits, the other's MMAs keep the tensor pipe busy.
//              (warp 2 also allocates TMEM.)
//   warps 4-11 promotion/epilogue: warp 4 + 4h + q owns TMEM lane quadrant q
//              (32 token rows) and partial columns [128h, 128h + 128), i.e.
//              weight block n0/128 + h, so each thread's scale per slab is
//              c = sx[kb][m] * s[n0/128 + h][kb]: acc += P * c with packed
//              FP32x2 FMAs. At the end of a tile the warp writes its 32 x 128
//              BF16 block, 64 columns at a time, into a 128B-swizzled staging
//              buffer and TMA-stores it. The store clips rows at M and columns
//              at N rounded down to 8 (the bulk copy moves whole 16-byte
//              chunks); the last < 8 columns of a ragged N are written from
//              the staging buffer with plain stores.
// Every wait is bounded (kWaitLimitCycles) and reports to the error word.
//
// EPI chooses what follows the sums (epilogue.cuh). kEpiFused adds the bias,
// applies the activation, adds the residual and rounds once; a thread holds
// one token row and 128 columns, finished 64 at a time by one copy of the code;
// the residual of a half comes by TMA into the staging buffer that then takes
// the output, the first half's during the tile's products (and the second's
// into L2), and the sums start from the bias.
// kEpiGated runs two weights as one: a tile's 256 weight rows are 128 gate
// rows and the 128 up rows of the same outputs (two 128-row boxes per slab, one
// issued by each of two lanes of warp 1), and an epilogue warp takes 64 gate
// columns and the same 64 up columns of the partial, so g and u of an output
// meet in one thread and act(g) * u is stored from the staging buffer as a
// plain y is: the pre-activations never leave the SM unless the caller keeps
// them. The multiply work per slab is unchanged.
//
// SPLIT > 1 (with an epilogue only): when there are far fewer tiles than SMs (a
// narrow layer and few tokens), a cluster of SPLIT CTAs shares one tile, each
// taking a run of its K slabs; at the end the CTAs trade FP32 sums through
// distributed shared memory, so that each has the whole sum, added in a fixed
// order, of 1 / SPLIT of the tile's columns, and finishes those.
#include <cuda_bf16.h>

#include <cstring>

#include "epilogue.cuh"
#include "internal.cuh"
#include "ptx.cuh"
#include "schedule.cuh"

namespace fp8blk {
namespace {

struct W8A8Cfg {
  static constexpr int BM = 128;                          // tokens per tile (MMA M)
  static constexpr int BN = 256;                          // weight rows per tile (MMA N)
  static constexpr int A_BYTES = BM * 128;                // activation slab
  static constexpr int B_BYTES = BN * 128;                // weight slab
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;   // one K slab of both operands
  static constexpr int ST = 4;                            // stages (power of two)
  static constexpr int RD = 8;                            // "slab done" ring (power of two)
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 128 + 32 * EPI_WARPS;
  static constexpr int OUT_BYTES = 32 * 128;              // per epilogue warp: 32 rows x 64 BF16
  static constexpr int NBAR = ST + RD + 2 + EPI_WARPS;
  static constexpr size_t SMEM_TILES =
      static_cast<size_t>(ST) * STAGE_BYTES + static_cast<size_t>(EPI_WARPS) * OUT_BYTES;
  static constexpr size_t SMEM = 1024 + SMEM_TILES + 8 * NBAR + 16;
  static constexpr uint32_t IDESC = make_idesc(0u, 0u, BM, BN);  // E4M3 x E4M3 -> F32
  // The launch gives 384 threads x 168 registers; the control warpgroup keeps
  // 56 and the two epilogue warpgroups take 224 each (128 x (56 + 2 x 224)).
  static constexpr int REG_CTRL = 56, REG_EPI = 224, REG_LAUNCH = 168;
  static_assert(128 * (REG_CTRL + 2 * REG_EPI) <= THREADS * REG_LAUNCH, "register split");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert((ST & (ST - 1)) == 0 && (RD & (RD - 1)) == 0, "power-of-two rings");
  // Slab j's "done" barrier is reused by slab j + RD, which must not complete
  // before every waiter on slab j has passed: the producers wait on slab j
  // before loading slab j + ST (RD >= ST keeps slab j + RD's loads behind
  // that wait), and the promotion warps wait on slab j before releasing the
  // partial of slab j, which slab j + 2 (same issuer, same TMEM slot) waits
  // for (RD >= 2).
  static_assert(RD >= ST && RD >= 2 && RD % 2 == 0, "done ring depth");
};

// Bounded wait on `bar` for the phase parity of its use `use` (0, 1, 2, ...).
__device__ __forceinline__ bool wait_use(uint64_t* bar, int use, unsigned* err, unsigned flag) {
  return mbar_wait(bar, static_cast<uint32_t>(use & 1), err, flag);
}

// 64 columns of one row per lane, from 32 column pairs, into the swizzled
// staging buffer: 16-byte chunk c of row r sits at chunk position c ^ (r % 8).
__device__ __forceinline__ void stage_row(uint8_t* srow, int lane, const uint64_t* v) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint4 o;
    o.x = cvt_bf16x2_pair(v[4 * c + 0]);
    o.y = cvt_bf16x2_pair(v[4 * c + 1]);
    o.z = cvt_bf16x2_pair(v[4 * c + 2]);
    o.w = cvt_bf16x2_pair(v[4 * c + 3]);
    *reinterpret_cast<uint4*>(srow + ((c ^ (lane & 7)) << 4)) = o;
  }
}

__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

// Adds two BF16 values to a pair of FP32 ones.
__device__ __forceinline__ void add_bf16x2(uint64_t& v, uint32_t b) {
  float lo, hi;
  unpack2(v, lo, hi);
  v = pack_f32x2(lo + bf16_lo_to_f32(b), hi + bf16_hi_to_f32(b));
}

// p[n] and p[n + 1] of the N values of p (n even), missing ones 0.
__device__ __forceinline__ uint32_t load_bf16x2(const uint16_t* p, int n, int N) {
  if (n + 1 < N) return __ldg(reinterpret_cast<const uint32_t*>(p + n));
  return n < N ? __ldg(p + n) : 0u;
}

// Stores the staged 32 x 64 block at (row r0, column base): by TMA up to
// column n_tma, the last < 8 columns of a ragged N by plain stores.
__device__ __forceinline__ void store_staged(const CUtensorMap* map, const uint8_t* stage,
                                             const uint8_t* srow, uint16_t* dst_row, int lane,
                                             int base, int r0, int m, int M, int N, int n_tma) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && r0 < M && base < n_tma) {
    tma_store_2d(map, stage, base, r0);
    tma_store_commit();
  }
  if (n_tma < N && n_tma >= base && n_tma < base + 64 && m < M) {
    const int cl = n_tma - base;  // first tail column within these 64
    const uint16_t* src =
        reinterpret_cast<const uint16_t*>(srow + (((cl >> 3) ^ (lane & 7)) << 4));
    for (int e = 0; e < N - n_tma; ++e) dst_row[n_tma + e] = src[e];
  }
}

__device__ __forceinline__ const CUtensorMap* residual_map(const EpiParams<kEpiFused>& ep) {
  return &ep.tm_res;
}
template <int EPI>
__device__ __forceinline__ const CUtensorMap* residual_map(const EpiParams<EPI>&) {
  return nullptr;
}

// (In PTX, so that choosing among array elements stays a choice of registers and
// does not become an index into memory.)
__device__ __forceinline__ uint64_t select64(bool c, uint64_t a, uint64_t b) {
  uint64_t r;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tselp.b64 %0, %1, %2, p;\n\t}"
      : "=l"(r)
      : "l"(a), "l"(b), "r"(static_cast<int>(c)));
  return r;
}

// 16 columns of a row, of which the first `left` exist; p is 16-byte aligned.
__device__ __forceinline__ void store_row16(uint16_t* p, const float (&f)[16], int left) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = cvt_bf16x2(f[2 * i + 1], f[2 * i]);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (left >= 8 * g + 8) {
      reinterpret_cast<uint4*>(p)[g] = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
    } else {
#pragma unroll
      for (int i = 8 * g; i < 8 * g + 8; ++i)
        if (i < left) p[i] = static_cast<uint16_t>(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
  }
}
__device__ __forceinline__ void add_row16(const uint16_t* p, float (&f)[16], int left) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (left >= 8 * g + 8) {
      const uint4 r = reinterpret_cast<const uint4*>(p)[g];
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[8 * g + 2 * i] += bf16_lo_to_f32(w[i]);
        f[8 * g + 2 * i + 1] += bf16_hi_to_f32(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 8 * g; i < 8 * g + 8; ++i)
        if (i < left) f[i] += bf16_bits_to_f32(p[i]);
    }
  }
}

// The end of a tile shared by a cluster of S CTAs. A part is 1 / S of the tile:
// 128 / S column pairs (gated: half of them gate, half up, of the same outputs);
// warp (quad, h) holds 32 rows of the S / 2 parts h S / 2 .., and CTA q finishes
// part q. The other CTAs' sums of a part arrive in the stage ring (free once
// every CTA has finished its slabs), one slot per CTA, [quad][pair][lane].
// Every thread of the cluster passes both barriers, whatever happened before.
template <int EPI, int S>
__device__ __forceinline__ void finish_split(uint64_t (&acc)[64], bool ok, uint8_t* ring, int rank,
                                             int quad, int h, int lane, int nt, int r0, int M,
                                             int N, uint16_t* y, int64_t ldy,
                                             const EpiParams<EPI>& ep) {
  constexpr int PP = 128 / S, PL = S / 2, SLOT = PP * 1024;
  constexpr bool GATED = EPI == kEpiGated;
  auto at = [](int pl, int i) {  // index in acc of pair i of the warp's part pl
    if (!GATED) return pl * PP + i;
    return i < PP / 2 ? pl * (PP / 2) + i : 32 + pl * (PP / 2) + i - PP / 2;
  };
  const bool rows = r0 < M;  // the warp has rows
  cluster_sync();
  if (ok && rows) {
#pragma unroll
    for (int pl = 0; pl < PL; ++pl) {
      const int q = h * PL + pl;
      if (q != rank) {
        const int slot = rank < q ? rank : rank - 1;
        const uint32_t a = map_to_rank(ring, q) + slot * SLOT + quad * (PP * 256) + lane * 8;
#pragma unroll
        for (int i = 0; i < PP; ++i) st_cluster_u64(a + 256u * i, acc[at(pl, i)]);
      }
    }
  }
  cluster_sync();
  if (!ok || !rows || h != rank / PL) return;
  uint64_t v[PP];
#pragma unroll
  for (int i = 0; i < PP; ++i) {
    v[i] = acc[at(0, i)];
#pragma unroll
    for (int pl = 1; pl < PL; ++pl) v[i] = select64(pl == rank % PL, acc[at(pl, i)], v[i]);
  }
  const uint8_t* in = ring + quad * (PP * 256) + lane * 8;
#pragma unroll 1
  for (int s = 0; s < S - 1; ++s) {
#pragma unroll
    for (int i = 0; i < PP; ++i)
      fadd2(v[i], *reinterpret_cast<const uint64_t*>(in + s * SLOT + 256 * i));
  }
  const int m = r0 + lane;
  if (m >= M) return;
  constexpr int COLS = GATED ? PP : 2 * PP;  // output columns of a part
  const int col0 = (nt * S + rank) * COLS;
  const int64_t row = m;
#pragma unroll
  for (int c = 0; c < COLS / 16; ++c) {
    const int base = col0 + 16 * c, left = N - base;
    if (left <= 0) break;
    float f[16];
#pragma unroll
    for (int p = 0; p < 8; ++p) unpack2(v[8 * c + p], f[2 * p], f[2 * p + 1]);
    if constexpr (GATED) {
      float u[16];
#pragma unroll
      for (int p = 0; p < 8; ++p) unpack2(v[PP / 2 + 8 * c + p], u[2 * p], u[2 * p + 1]);
      if (ep.e.g) {
        store_row16(ep.e.g + row * ep.e.ldgu + base, f, left);
        store_row16(ep.e.u + row * ep.e.ldgu + base, u, left);
      }
      act_apply(ep.e.act, f);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] *= u[i];
    } else {
      if (ep.e.bias) add_row16(ep.e.bias + base, f, left);
      if (ep.e.preact) store_row16(ep.e.preact + row * ep.e.ldp + base, f, left);
      act_apply(ep.e.act, f);
      if (ep.e.residual) add_row16(ep.e.residual + row * ep.e.ldr + base, f, left);
    }
    store_row16(y + row * ldy + base, f, left);
  }
}

template <int EPI, int SPLIT>
__global__ void __launch_bounds__(W8A8Cfg::THREADS, 1)
    w8a8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_y, const float* __restrict__ sx,
                     int64_t ldsx, const float* __restrict__ sw, uint16_t* __restrict__ y,
                     int64_t ldy, int M, int N, int n_tma, int KB, int mtiles, int ntiles_total,
                     int gm, int a_bytes, unsigned* __restrict__ err,
                     const __grid_constant__ EpiParams<EPI> ep) {
  using C = W8A8Cfg;
  constexpr bool GATED = EPI == kEpiGated;
  constexpr int TILE_N = GATED ? C::BN / 2 : C::BN;  // output columns of a tile
  static_assert(SPLIT == 1 || EPI != kEpiPlain, "only with an epilogue");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;                            // ST stages: A then B
  uint8_t* sOut = smem + C::ST * C::STAGE_BYTES;             // EPI_WARPS x 4 KB staging
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::SMEM_TILES);
  uint64_t* full = bars;               // stage landed       (2 or 3 producers + tx)
  uint64_t* done = full + C::ST;       // slab's MMAs done   (1 commit)
  uint64_t* pempty = done + C::RD;     // partial consumed   (8 epilogue warps), one per issuer
  uint64_t* rfull = pempty + 2;        // residual landed    (1 + tx), one per epilogue warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rfull + C::EPI_WARPS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ntiles_n = ntiles_total / mtiles;
  const int my_tiles =
      static_cast<int>(blockIdx.x) < ntiles_total ? (ntiles_total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
  // This CTA's run of a tile's slabs, and its tiles.
  const int rank = SPLIT > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int kb0 = SPLIT > 1 ? KB * rank / SPLIT : 0, kb1 = SPLIT > 1 ? KB * (rank + 1) / SPLIT : KB;
  const int first_tile = static_cast<int>(blockIdx.x) / SPLIT;
  const int total_slabs = SPLIT > 1 ? kb1 - kb0 : my_tiles * KB;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) mbar_init(&full[s], GATED ? 3 : 2);
    for (int b = 0; b < C::RD; ++b) mbar_init(&done[b], 1);
    for (int b = 0; b < 2; ++b) mbar_init(&pempty[b], C::EPI_WARPS);
    for (int b = 0; b < C::EPI_WARPS; ++b) mbar_init(&rfull[b], 1);
    mbar_init_fence();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // The next kernel in the stream may be scheduled now; it reads y after its
  // own griddepcontrol.wait.
  pdl_launch_dependents();

  // Each warpgroup sets its register budget at the top of its role.
  if (warp < 4) {
    setmaxnreg_dec<C::REG_CTRL>();
    if (warp < 2 && (lane == 0 || (GATED && warp == 1 && lane == 1))) {
      // ------------------------------------------------- producers (A, B)
      const bool is_a = warp == 0;
      const CUtensorMap* map = is_a ? &tm_a : &tm_b;
      uint32_t bytes = is_a ? static_cast<uint32_t>(a_bytes) : C::B_BYTES;
      uint8_t* dst0 = smem + (is_a ? 0 : C::A_BYTES);
      if constexpr (GATED) {  // gate rows, then up rows
        if (!is_a) {
          bytes = C::B_BYTES / 2;
          if (lane == 1) {
            map = &ep.tm_up;
            dst0 += C::B_BYTES / 2;
          }
        }
      }
      tma_prefetch_map(map);
      // Launched as a programmatic dependent of the activation quantizer:
      // the weights may stream at once, the activation codes only once that
      // kernel has completed (a no-op for an ordinary launch).
      if (is_a) pdl_wait();
      int j = 0;  // slab counter (across tiles)
      bool ok = true;
      for (int tile = first_tile; tile < ntiles_total && ok; tile += gridDim.x) {
        int mt, nt;
        tile_coords(tile, mtiles, ntiles_n, gm, mt, nt);
        const int row0 = is_a ? mt * C::BM : nt * TILE_N;
        for (int kb = kb0; kb < kb1; ++kb, ++j) {
          const int stage = j & (C::ST - 1);
          if (j >= C::ST) {  // the slab that last used this stage has finished
            const int jo = j - C::ST;
            if (!wait_use(&done[jo & (C::RD - 1)], jo / C::RD, err, kErrWaitLoad)) {
              ok = false;
              break;
            }
          }
          mbar_arrive_expect_tx(&full[stage], bytes);
          tma_load_2d(dst0 + stage * C::STAGE_BYTES, map, &full[stage], kb * 128, row0);
        }
      }
      // Drain: the loads of the last stages have landed before the CTA may
      // exit (on a time-out the other producer's half may be missing; the
      // waits are bounded).
      for (int jj = (j > C::ST ? j - C::ST : 0); jj < j; ++jj)
        wait_use(&full[jj & (C::ST - 1)], jj / C::ST, err, kErrWaitLoad);
    } else if (warp >= 2 && lane == 0) {
      // ----------------------------------------------------- MMA issuers
      const int e = warp - 2;
      const uint64_t adesc0 = sw128_kmajor_desc(smem_addr(smem));
      const uint64_t bdesc0 = sw128_kmajor_desc(smem_addr(smem + C::A_BYTES));
      const uint32_t d = tmem + static_cast<uint32_t>(e * C::BN);
      int last = -1;
      for (int j = e; j < total_slabs; j += 2) {
        if (!wait_use(&full[j & (C::ST - 1)], j / C::ST, err, kErrWaitMma)) break;
        const int u = j >> 1;  // use of this issuer's partial
        if (u >= 1 && !wait_use(&pempty[e], u - 1, err, kErrWaitMma)) break;
        tc_fence_after_sync();
        const uint64_t soff = static_cast<uint64_t>(((j & (C::ST - 1)) * C::STAGE_BYTES) >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8f6f4_ss(d, adesc0 + soff + 2u * k, bdesc0 + soff + 2u * k, C::IDESC, k > 0 ? 1u : 0u);
        tc_commit(&done[j & (C::RD - 1)]);
        last = j;
      }
      // Drain: this issuer's MMAs have completed before TMEM is released.
      if (last >= 0) wait_use(&done[last & (C::RD - 1)], last / C::RD, err, kErrWaitMma);
    }
    if constexpr (SPLIT > 1) {  // the barriers of finish_split
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    setmaxnreg_inc<C::REG_EPI>();
    // -------------------------------------------------- promotion/epilogue
    pdl_wait();  // the activation scales come from the kernel before
    const int ew = warp - 4;
    const int quad = warp & 3;  // TMEM lanes this warp may access
    const int h = ew >> 2;      // partial columns [128h, 128h + 128); gated: 64h.. of each half
    const int row = quad * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16) +
                            static_cast<uint32_t>(h * (TILE_N / 2));
    uint8_t* stage = sOut + ew * C::OUT_BYTES;
    uint8_t* srow = stage + lane * 128;
    int j = 0;
    bool ok = true;
    // Loads the residual of the 32 x 64 block at (r0, base) into the staging
    // buffer once that buffer's last store has been read out. Two loads per
    // tile that has rows for this warp, whether or not the columns exist (what
    // does not is filled with zeros), so the barrier's phase is the half's number.
    auto load_residual = [&](int base, int r0) {
      __syncwarp();
      if (lane == 0) {
        tma_store_wait_read<0>();
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(&rfull[ew], C::OUT_BYTES);
        tma_load_2d(stage, residual_map(ep), &rfull[ew], base, r0);
      }
    };
    for (int tile = first_tile; tile < ntiles_total && ok; tile += gridDim.x) {
      int mt, nt;
      tile_coords(tile, mtiles, ntiles_n, gm, mt, nt);
      const int m0 = mt * C::BM;
      const int col0 = nt * TILE_N + (TILE_N / 2) * h;  // first output column of this warp
      const bool has_cols = col0 < N;
      const int m = m0 + row;
      // sx is group-major with ldsx covering whole 128-row tiles, so rows
      // past M read padding (their results are never stored).
      const float* sx_col = sx + (m < M ? m : 0);
      const float* sw_row = sw + static_cast<int64_t>(has_cols ? (col0 >> 7) : 0) * KB;
      const float* sw_up = nullptr;
      if constexpr (GATED) sw_up = ep.e.s_up + static_cast<int64_t>(has_cols ? (col0 >> 7) : 0) * KB;
      uint64_t acc[64];  // column pairs (gated: 32 of the gate, then 32 of up)
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      if constexpr (EPI == kEpiFused && SPLIT == 1) {
        if (ep.e.residual && m0 + quad * 32 < M) {
          // (The staging buffer serves z first where that is kept.)
          if (!ep.e.preact) load_residual(col0, m0 + quad * 32);
          if (lane == 0) tma_prefetch_2d(&ep.tm_res, col0 + 64, m0 + quad * 32);
        }
        if (ep.e.bias) {  // the sums start from the bias
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t mine = load_bf16x2(ep.e.bias, col0 + 64 * hh + 2 * lane, N);
#pragma unroll
            for (int p = 0; p < 32; ++p) {
              const uint32_t b = __shfl_sync(0xFFFFFFFFu, mine, p);
              acc[32 * hh + p] = pack_f32x2(bf16_lo_to_f32(b), bf16_hi_to_f32(b));
            }
          }
        }
      }
      // The two scale factors of a slab are loaded one slab ahead and only
      // multiplied when used, so the product does not wait on the loads.
      float fx = has_cols ? __ldg(sx_col + kb0 * ldsx) : 0.0f, fw = has_cols ? __ldg(sw_row + kb0) : 0.0f;
      float fu = GATED && has_cols ? __ldg(sw_up + kb0) : 0.0f;
      for (int kb = kb0; kb < kb1; ++kb, ++j) {
        const float c = fx * fw;
        const float cu = GATED ? fx * fu : 0.0f;
        if (has_cols && kb + 1 < kb1) {
          fx = __ldg(sx_col + (kb + 1) * ldsx);
          fw = __ldg(sw_row + kb + 1);
          if constexpr (GATED) fu = __ldg(sw_up + kb + 1);
        }
        if (!mbar_wait_warp(&done[j & (C::RD - 1)], static_cast<uint32_t>((j / C::RD) & 1), err,
                            kErrWaitEpilogue)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t tp = t_lane + static_cast<uint32_t>((j & 1) * C::BN);
        // With an epilogue, 16 columns per load: its own registers and two
        // 32-column loads exceed the budget, and the spills and reloads that
        // follow land in this loop (512 x 5120 x 51200 without activation:
        // 225 us against 162). The plain kernel keeps the wider loads (139
        // against 143).
        if constexpr (GATED) {
          tmem_axpy2_narrow<2>(tp, c, acc);
          tmem_axpy2_narrow<2>(tp + 128u, cu, acc + 32);
        } else if constexpr (EPI == kEpiFused) {
          tmem_axpy2_narrow<4>(tp, c, acc);
        } else {
          tmem_axpy2<4>(tp, c, acc);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pempty[j & 1]);
      }
      if constexpr (SPLIT > 1) {
        finish_split<EPI, SPLIT>(acc, ok, smem, rank, quad, h, lane, nt, m0 + quad * 32, M, N, y, ldy, ep);
        break;
      }
      if (!ok) break;
      // Output, 64 columns at a time: the staging buffer's previous store has
      // been read out before it is written again.
      const int r0 = m0 + quad * 32;
      if (EPI != kEpiPlain && r0 >= M) continue;  // no rows for this warp
      uint16_t* yrow = y + static_cast<int64_t>(m) * ldy;
      if constexpr (GATED) {
        if (ep.e.g) {  // kept pre-activations
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
          stage_row(srow, lane, acc);
          store_staged(&ep.tm_g, stage, srow, ep.e.g + static_cast<int64_t>(m) * ep.e.ldgu, lane,
                       col0, r0, m, M, N, n_tma);
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
          stage_row(srow, lane, acc + 32);
          store_staged(&ep.tm_u, stage, srow, ep.e.u + static_cast<int64_t>(m) * ep.e.ldgu, lane,
                       col0, r0, m, M, N, n_tma);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[16];
#pragma unroll
          for (int p = 0; p < 8; ++p) unpack2(acc[8 * c + p], v[2 * p], v[2 * p + 1]);
          act_apply(ep.e.act, v);
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            float u0, u1;
            unpack2(acc[32 + 8 * c + p], u0, u1);
            acc[8 * c + p] = pack_f32x2(v[2 * p] * u0, v[2 * p + 1] * u1);
          }
        }
        if (lane == 0) tma_store_wait_read<0>();
        __syncwarp();
        stage_row(srow, lane, acc);
        store_staged(&tm_y, stage, srow, yrow, lane, col0, r0, m, M, N, n_tma);
      } else if constexpr (EPI == kEpiFused) {
        const FusedEpi& e = ep.e;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int base = col0 + 64 * hh;
          uint64_t* v = acc + 32 * hh;
          if (e.preact) {
            if (lane == 0) tma_store_wait_read<0>();
            __syncwarp();
            stage_row(srow, lane, v);
            store_staged(&ep.tm_pre, stage, srow, e.preact + static_cast<int64_t>(m) * e.ldp, lane,
                         base, r0, m, M, N, n_tma);
            if (e.residual) load_residual(base, r0);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float f[16];
#pragma unroll
            for (int p = 0; p < 8; ++p) unpack2(v[8 * c + p], f[2 * p], f[2 * p + 1]);
            act_apply(e.act, f);
#pragma unroll
            for (int p = 0; p < 8; ++p) v[8 * c + p] = pack_f32x2(f[2 * p], f[2 * p + 1]);
          }
          if (e.residual) {
            if (!mbar_wait_warp(&rfull[ew], static_cast<uint32_t>(hh), err, kErrWaitEpilogue)) {
              ok = false;
              break;
            }
            // A lane adds its own row's residual, then its output takes the place.
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint4 r = *reinterpret_cast<const uint4*>(srow + ((c ^ (lane & 7)) << 4));
              add_bf16x2(v[4 * c + 0], r.x);
              add_bf16x2(v[4 * c + 1], r.y);
              add_bf16x2(v[4 * c + 2], r.z);
              add_bf16x2(v[4 * c + 3], r.w);
            }
          } else {
            if (lane == 0) tma_store_wait_read<0>();
            __syncwarp();
          }
          stage_row(srow, lane, v);
          store_staged(&tm_y, stage, srow, yrow, lane, base, r0, m, M, N, n_tma);
          if (hh == 0 && e.residual && !e.preact) load_residual(base + 64, r0);
        }
        if (!ok) break;
      } else {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int base = col0 + 64 * hh;
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
          stage_row(srow, lane, acc + 32 * hh);
          store_staged(&tm_y, stage, srow, yrow, lane, base, r0, m, M, N, n_tma);
        }
      }
    }
    if (lane == 0) tma_store_wait_all();
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// A map of 32 x 64 blocks over the first n_tma columns of a BF16 matrix: stores
// take N rounded down to 8 (none if N < 8), loads all of N.
bool block_map(CUtensorMap* map, const uint16_t* p, int64_t n_tma, int64_t M, int64_t ld) {
  if (n_tma > 0 && p) return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, n_tma, M, 2 * ld, 64, 32);
  memset(map, 0, sizeof(*map));
  return true;
}

template <int EPI, int SPLIT = 1>
cudaError_t launch_epi(const Launch& L, const uint8_t* qx, int64_t ldqx, const float* sx,
                       int64_t ldsx, const uint8_t* q, int64_t ldq, const float* sw, uint16_t* y,
                       int64_t ldy, int64_t M, int64_t N, int64_t K, bool after_act_quant,
                       EpiParams<EPI>& ep) {
  using C = W8A8Cfg;
  CUtensorMap ta, tb, ty;
  // Fewer than BM tokens: load only the first round_up(M, 8) activation rows
  // of a slab. The MMA still reads BM rows; the rows past those only reach
  // output rows >= M, which are never stored.
  const int64_t a_rows = M < C::BM ? round_up(M, 8) : C::BM;
  if (!make_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, qx, K, M, ldqx, 128,
                    static_cast<uint32_t>(a_rows)))
    return cudaErrorInvalidValue;
  constexpr int kTileN = EPI == kEpiGated ? C::BN / 2 : C::BN;
  if (!make_tmap_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, N, ldq, 128, kTileN))
    return cudaErrorInvalidValue;
  const int64_t n_tma = N & ~int64_t{7};
  if (!block_map(&ty, y, n_tma, M, ldy)) return cudaErrorInvalidValue;
  if constexpr (EPI == kEpiFused) {
    if (!block_map(&ep.tm_pre, ep.e.preact, n_tma, M, ep.e.ldp) ||
        !block_map(&ep.tm_res, ep.e.residual, N, M, ep.e.ldr))
      return cudaErrorInvalidValue;
  } else if constexpr (EPI == kEpiGated) {
    if (!make_tmap_2d(&ep.tm_up, CU_TENSOR_MAP_DATA_TYPE_UINT8, ep.e.q_up, K, N, ldq, 128, kTileN) ||
        !block_map(&ep.tm_g, ep.e.g, n_tma, M, ep.e.ldgu) ||
        !block_map(&ep.tm_u, ep.e.u, n_tma, M, ep.e.ldgu))
      return cudaErrorInvalidValue;
  }
  auto kern = w8a8_gemm_kernel<EPI, SPLIT>;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  {
    // The register split needs the launch allocation it was sized for
    // (checked once).
    static const cudaError_t regs = [&] {
      cudaFuncAttributes fa;
      cudaError_t r = cudaFuncGetAttributes(&fa, reinterpret_cast<const void*>(kern));
      if (r != cudaSuccess) return r;
      return fa.numRegs < C::REG_LAUNCH ? cudaErrorInvalidConfiguration : cudaSuccess;
    }();
    if (regs != cudaSuccess) return regs;
  }
  const int64_t mtiles = cdiv(M, C::BM), tiles = mtiles * cdiv(N, kTileN);
  // Slab counters are 32-bit per CTA.
  if (tiles * cdiv(K, 128) > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  const int grid = SPLIT > 1 ? static_cast<int>(tiles * SPLIT)
                             : static_cast<int>(tiles < L.num_sms ? tiles : L.num_sms);
  // After the activation quantizer: a programmatic dependent launch, so the
  // GEMM's set-up and weight loads overlap that kernel.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  int nattr = 0;
  if (after_act_quant) {
    attr[nattr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[nattr++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (SPLIT > 1) {
    attr[nattr].id = cudaLaunchAttributeClusterDimension;
    attr[nattr].val.clusterDim.x = SPLIT;
    attr[nattr].val.clusterDim.y = 1;
    attr[nattr++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = nattr;
  return cudaLaunchKernelEx(&cfg, kern, ta, tb, ty, sx, ldsx, sw, y, ldy, static_cast<int>(M),
                            static_cast<int>(N), static_cast<int>(n_tma),
                            static_cast<int>(cdiv(K, 128)), static_cast<int>(mtiles),
                            static_cast<int>(tiles), raster_group(mtiles, C::BM * K, kRasterBytesW8A8),
                            static_cast<int>(a_rows * 128), L.err, ep);
}

// Clusters of S CTAs that can be resident at once (0 on an error; queried once per
// device and form): a cluster lies within one group of SMs, so it is fewer than
// num_sms / S.
template <int EPI, int S>
int64_t resident_clusters() {
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (n == 0) {
    auto kern = w8a8_gemm_kernel<EPI, S>;
    if (ensure_smem_limit(reinterpret_cast<const void*>(kern), W8A8Cfg::SMEM) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(W8A8Cfg::THREADS);
    cfg.dynamicSmemBytes = W8A8Cfg::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) return 0;
    __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  }
  return n;
}

template <int EPI>
cudaError_t launch_split(const Launch& L, const uint8_t* qx, int64_t ldqx, const float* sx,
                         int64_t ldsx, const uint8_t* q, int64_t ldq, const float* sw, uint16_t* y,
                         int64_t ldy, int64_t M, int64_t N, int64_t K, EpiParams<EPI>& ep) {
  using C = W8A8Cfg;
  const int64_t tiles = cdiv(M, C::BM) * cdiv(N, EPI == kEpiGated ? C::BN / 2 : C::BN);
  const int split = ctas_per_tile(tiles, cdiv(K, 128), L.num_sms, [](int s) {
    return s == 2 ? resident_clusters<EPI, 2>() : s == 4 ? resident_clusters<EPI, 4>() : resident_clusters<EPI, 8>();
  });
  switch (split) {
    case 8: return launch_epi<EPI, 8>(L, qx, ldqx, sx, ldsx, q, ldq, sw, y, ldy, M, N, K, true, ep);
    case 4: return launch_epi<EPI, 4>(L, qx, ldqx, sx, ldsx, q, ldq, sw, y, ldy, M, N, K, true, ep);
    case 2: return launch_epi<EPI, 2>(L, qx, ldqx, sx, ldsx, q, ldq, sw, y, ldy, M, N, K, true, ep);
  }
  return launch_epi<EPI>(L, qx, ldqx, sx, ldsx, q, ldq, sw, y, ldy, M, N, K, true, ep);
}

}  // namespace

cudaError_t launch_w8a8_gemm(const Launch& L, const uint8_t* qx, int64_t ldqx, const float* sx,
                             int64_t ldsx, const uint8_t* q, int64_t ldq, const float* sw,
                             uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                             bool after_act_quant) {
  EpiParams<kEpiPlain> ep;
  return launch_epi<kEpiPlain>(L, qx, ldqx, sx, ldsx, q, ldq, sw, y, ldy, M, N, K, after_act_quant, ep);
}

cudaError_t launch_w8a8_fused(const Launch& L, const uint8_t* qx, int64_t ldqx, const float* sx,
                              int64_t ldsx, const uint8_t* q, int64_t ldq, const float* sw,
                              uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                              const FusedEpi& e) {
  EpiParams<kEpiFused> ep;
  ep.e = e;
  return launch_split<kEpiFused>(L, qx, ldqx, sx, ldsx, q, ldq, sw, y, ldy, M, N, K, ep);
}

cudaError_t launch_w8a8_gated(const Launch& L, const uint8_t* qx, int64_t ldqx, const float* sx,
                              int64_t ldsx, const uint8_t* q, int64_t ldq, const float* sw,
                              uint16_t* h, int64_t ldh, int64_t M, int64_t N, int64_t K,
                              const GatedEpi& e) {
  EpiParams<kEpiGated> ep;
  ep.e = e;
  return launch_split<kEpiGated>(L, qx, ldqx, sx, ldsx, q, ldq, sw, h, ldh, M, N, K, ep);
}

}  // namespace fp8blk
