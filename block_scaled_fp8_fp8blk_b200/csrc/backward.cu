// The memory-bound kernels of the backward passes: the gated product's and
// the epilogue's derivative, and the transposed weight that turns dx = dz . W
// into an ordinary linear.
//
// Each touches every byte once: 16-byte loads and stores along the rows,
// enough of them in flight per SM to cover the latency of HBM, and nothing
// kept between kernels but the column sums of the bias gradient.
//
// dg, du and dz leave FP32 here, rounded to BF16 once: they are the operands of the
// tensor cores' products that follow, whose kind takes BF16 on both sides, and the
// traffic of these kernels (FP32 copies would take half as much time again, and
// a second BF16 term to carry the rest would double the products). What is
// computed from them carries that rounding: a relative norm of 1.7e-3 in dx and dw
// before their own. The bias gradient is summed before it.
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = bf16_lo_to_f32(w.x), v[1] = bf16_hi_to_f32(w.x);
  v[2] = bf16_lo_to_f32(w.y), v[3] = bf16_hi_to_f32(w.y);
  v[4] = bf16_lo_to_f32(w.z), v[5] = bf16_hi_to_f32(w.z);
  v[6] = bf16_lo_to_f32(w.w), v[7] = bf16_hi_to_f32(w.w);
}

// Eight BF16 values of a row from column c on: one 16-byte load where all
// eight exist, else the existing ones and zeros.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t c, int64_t n) {
  if (c + 8 <= n) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < n) w[i / 2] |= static_cast<uint32_t>(row[c + i]) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(cvt_bf16x2(v[1], v[0]), cvt_bf16x2(v[3], v[2]), cvt_bf16x2(v[5], v[4]),
                    cvt_bf16x2(v[7], v[6]));
}

// dg = dh u act'(g), du = dh act(g) of eight columns. The slope, at most 1.13 in
// magnitude, comes into the product first: dh u alone may overflow where dg does
// not (and infinity times a slope of 0 would be NaN).
template <int KIND>
__device__ __forceinline__ void gated_slopes(ActParams act, const uint4& d, const uint4& g,
                                             const uint4& u, uint4& dg, uint4& du) {
  act.kind = KIND;
  const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v0, v1;
    const float s0 = act_slope(act, bf16_lo_to_f32(gw[i]), v0);
    const float s1 = act_slope(act, bf16_hi_to_f32(gw[i]), v1);
    const float d0 = bf16_lo_to_f32(dw[i]), d1 = bf16_hi_to_f32(dw[i]);
    a[i] = cvt_bf16x2(d1 * s1 * bf16_hi_to_f32(uw[i]), d0 * s0 * bf16_lo_to_f32(uw[i]));
    b[i] = cvt_bf16x2(d1 * v1, d0 * v0);
  }
  dg = make_uint4(a[0], a[1], a[2], a[3]);
  du = make_uint4(b[0], b[1], b[2], b[3]);
}

// Eight columns per thread, rows in steps of the grid. The columns between N and
// Np = round_up(N, 128) get zeros (the loads give dh = 0 there). Bound by HBM, so the
// loads in flight count: one branch on the activation per eight columns and operands
// unpacked as they are used take 35 registers, seven blocks an SM. Unpacked in
// advance with the branch in each element, 57 and four: 84 us against 78 at 2048 x
// 25600 with silu (cleared L2), 166 against 160 at 4096 with gelu.
__global__ void __launch_bounds__(256)
    gated_backward_kernel(const uint16_t* __restrict__ dh, int64_t lddh,
                          const uint16_t* __restrict__ g, const uint16_t* __restrict__ u,
                          int64_t ldgu, ActParams act, uint16_t* __restrict__ dgu, int64_t lddgu,
                          int64_t M, int64_t N, int64_t Np) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= Np) return;
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const uint4 d = load8(dh + m * lddh, c, N), gv = load8(g + m * ldgu, c, N),
                uv = load8(u + m * ldgu, c, N);
    uint4 dg, du;
    if (act.kind == kActLogistic) {
      gated_slopes<kActLogistic>(act, d, gv, uv, dg, du);
    } else if (act.kind == kActNormal) {
      gated_slopes<kActNormal>(act, d, gv, uv, dg, du);
    } else {
      gated_slopes<kActMax>(act, d, gv, uv, dg, du);
    }
    uint16_t* out = dgu + m * lddgu + c;
    *reinterpret_cast<uint4*>(out) = dg;
    *reinterpret_cast<uint4*>(out + Np) = du;
  }
}

// dz = dy act'(z) and, with SUM, the column sums of the unrounded products. A
// block takes 256 columns (32 lanes x 8) and a run of rows, eight at a time, two
// steps in flight; each thread sums its rows, the block adds its eight warps in
// order, and the blocks of one column strip are added in order by
// column_sum_kernel. So the order of the sum depends on the sizes alone. Four
// blocks fit an SM (64 registers a thread). dz may be dy or z: a thread writes
// only what it has read.
constexpr int kStripCols = 256, kRowsPerStep = 8;

// One row's eight columns: d *= act'(z), stored, summed.
template <bool SUM>
__device__ __forceinline__ void epilogue_backward_row(float (&d)[8], const float (&v)[8], bool has_z,
                                                      const ActParams& act, uint16_t* out, int64_t c,
                                                      int64_t N, float (&sum)[8]) {
  if (has_z) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a;
      d[i] *= act_slope(act, v[i], a);
    }
  }
  if (out) {
    if (c + 8 <= N) {
      *reinterpret_cast<uint4*>(out + c) = pack8(d);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < N) out[c + i] = static_cast<uint16_t>(cvt_bf16x2(0.0f, d[i]));
    }
  }
  if constexpr (SUM) {
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += d[i];
  }
}

template <bool SUM>
__global__ void __launch_bounds__(256, 4)
    epilogue_backward_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* z, int64_t ldz,
                             ActParams act, uint16_t* dz, int64_t lddz, float* sums, int64_t M,
                             int64_t N, int64_t rows) {
  if constexpr (SUM) pdl_launch_dependents();  // column_sum_kernel, which waits for this grid
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kStripCols + lane * 8;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * rows;
  const int64_t m1 = m0 + rows < M ? m0 + rows : M;
  float sum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
  auto row_out = [&](int64_t m) { return dz ? dz + m * lddz : nullptr; };
  int64_t m = m0 + warp;
  if (c + 8 <= N) {
    for (; m + kRowsPerStep < m1; m += 2 * kRowsPerStep) {  // two rows: all loads first
      const int64_t mb = m + kRowsPerStep;
      const uint4 da = *reinterpret_cast<const uint4*>(dy + m * lddy + c);
      const uint4 db = *reinterpret_cast<const uint4*>(dy + mb * lddy + c);
      uint4 za = make_uint4(0u, 0u, 0u, 0u), zb = za;
      if (z) {
        za = *reinterpret_cast<const uint4*>(z + m * ldz + c);
        zb = *reinterpret_cast<const uint4*>(z + mb * ldz + c);
      }
      float d[8], v[8];
      unpack8(da, d);
      unpack8(za, v);
      epilogue_backward_row<SUM>(d, v, z != nullptr, act, row_out(m), c, N, sum);
      unpack8(db, d);
      unpack8(zb, v);
      epilogue_backward_row<SUM>(d, v, z != nullptr, act, row_out(mb), c, N, sum);
    }
  }
  if (c < N) {
#pragma unroll 1
    for (; m < m1; m += kRowsPerStep) {
      float d[8], v[8];
      unpack8(load8(dy + m * lddy, c, N), d);
      if (z) unpack8(load8(z + m * ldz, c, N), v);
      epilogue_backward_row<SUM>(d, v, z != nullptr, act, row_out(m), c, N, sum);
    }
  }
  if constexpr (SUM) {
    __shared__ float s[8][kStripCols];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[warp][lane * 8 + i] = sum[i];
    __syncthreads();
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kStripCols + threadIdx.x;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += s[w][threadIdx.x];
    if (n < N) sums[static_cast<int64_t>(blockIdx.y) * N + n] = t;
  }
}

__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ parts,
                                                         int64_t splits, int64_t N,
                                                         float* __restrict__ out) {
  pdl_wait();
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n >= N) return;
  float t = 0.0f;
#pragma unroll 4
  for (int64_t i = 0; i < splits; ++i) t += parts[i * N + n];
  out[n] = t;
}

// Row runs of epilogue_backward_kernel, whole steps of eight rows: about 2368
// blocks in all, four times what a B200 holds at once (4 x 148), so that the last
// wave weighs little. (600 blocks, 8 more than fit, took 162 us at 4096 x 25600.)
struct RowSplit {
  int64_t rows, splits;
};
RowSplit row_split(int64_t M, int64_t N) {
  // Few rows: one run, which needs no second kernel.
  if (M <= 128) return {round_up(M, kRowsPerStep), 1};
  const int64_t strips = cdiv(N, kStripCols), want = cdiv(2368, strips);
  const int64_t rows = round_up(cdiv(M, want), kRowsPerStep);
  return {rows, cdiv(M, rows)};
}

// qt[k][n] = q[n][k] for one 128 x 128 block of codes per thread block. A
// thread takes 4 rows x 16 codes (four 16-byte loads, a warp four whole 128-byte
// lines at a time), transposes 4 x 4 codes in registers, and the words cross
// through shared memory: word (k, n / 4) sits in 16-byte chunk (n / 16) ^ (k / 16)
// of row k, so that the writes (8 values of k / 16, 4 of n / 4) touch 32 different
// banks and the reads are whole rows, 16 bytes a lane. The second weight of a
// gated pair (blockIdx.z = 1) goes n_end columns further right.
__global__ void __launch_bounds__(256)
    transpose_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s,
                     const uint8_t* __restrict__ q2, const float* __restrict__ s2, int64_t ldq,
                     int64_t N, int64_t K, uint8_t* __restrict__ qt, int64_t ldqt,
                     float* __restrict__ st, int64_t ldst, int64_t n_end) {
  if (blockIdx.z) q = q2, s = s2, qt += n_end, st += gridDim.y;
  __shared__ __align__(16) uint32_t t[128 * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t kb = blockIdx.x, nb = blockIdx.y;
  const int64_t k0 = kb * 128, n0 = nb * 128;
  {
    const int r = lane & 3, k16 = lane >> 2;
    const int64_t k = k0 + 16 * k16, n = n0 + 16 * warp + 4 * r;
    uint32_t w[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (n + i < N && k < K) {
        const uint8_t* p = q + (n + i) * ldq + k;
        if (k + 16 <= K) {
          v = *reinterpret_cast<const uint4*>(p);
        } else {
          uint64_t lo = 0, hi = 0;
#pragma unroll 1
          for (int e = 0; k + e < K; ++e) {
            const uint64_t b = static_cast<uint64_t>(p[e]) << (8 * (e & 7));
            if (e < 8) lo |= b; else hi |= b;
          }
          v = make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                         static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32));
        }
      }
      w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
    }
    const int col = 4 * (warp ^ k16) + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // Byte e of the four rows' words: pairs of rows interleaved, then halves.
      const uint32_t a = __byte_perm(w[0][j], w[1][j], 0x5140), c = __byte_perm(w[2][j], w[3][j], 0x5140);
      const uint32_t d = __byte_perm(w[0][j], w[1][j], 0x7362), f = __byte_perm(w[2][j], w[3][j], 0x7362);
      uint32_t* o = t + (16 * k16 + 4 * j) * 32 + col;
      o[0] = __byte_perm(a, c, 0x5410);
      o[32] = __byte_perm(a, c, 0x7632);
      o[64] = __byte_perm(d, f, 0x5410);
      o[96] = __byte_perm(d, f, 0x7632);
    }
  }
  __syncthreads();
  const int64_t n = n0 + 16 * (lane & 7);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kk = 4 * warp + (lane >> 3) + 32 * i;
    if (k0 + kk >= K) break;
    const uint4 v = reinterpret_cast<const uint4*>(t)[kk * 8 + ((lane & 7) ^ (kk >> 4))];
    uint8_t* p = qt + (k0 + kk) * ldqt + n;
    if (n + 16 <= n_end) {
      *reinterpret_cast<uint4*>(p) = v;
    } else {
      uint64_t lo = v.x | static_cast<uint64_t>(v.y) << 32, hi = v.z | static_cast<uint64_t>(v.w) << 32;
#pragma unroll 1
      for (int e = 0; e < 16 && n + e < n_end; ++e)
        p[e] = static_cast<uint8_t>((e < 8 ? lo : hi) >> (8 * (e & 7)));
    }
  }
  if (threadIdx.x == 0) st[kb * ldst + nb] = s[nb * gridDim.x + kb];
}

// `count` weights side by side, n_end columns each.
fp8blk_status transpose(const uint8_t* q, const float* s, const uint8_t* q2, const float* s2,
                        int count, int64_t ldq, int64_t N, int64_t K, uint8_t* qt, int64_t ldqt,
                        float* st, int64_t ldst, int64_t n_end, fp8blk_stream stream) {
  if (N < 0 || K < 0) return FP8BLK_ERR_INVALID_ARG;
  if (N == 0 || K == 0) return FP8BLK_OK;
  if (!q || !s || !q2 || !s2 || !qt || !st || ldq < K || ldqt < count * n_end ||
      ldst < count * cdiv(N, 128))
    return FP8BLK_ERR_INVALID_ARG;
  // Grid limits: blocks of K along x, of N along y.
  if (cdiv(K, 128) > kInt32Max || cdiv(N, 128) > 65535) return FP8BLK_ERR_INVALID_ARG;
  if (ldq % 16 || ldqt % 16 || !aligned(q, 16) || !aligned(q2, 16) || !aligned(qt, 16) ||
      !aligned(s, 4) || !aligned(s2, 4) || !aligned(st, 4))
    return FP8BLK_ERR_ALIGNMENT;
  if (one_of(qt, q, q2) || one_of(st, s, s2)) return FP8BLK_ERR_INVALID_ARG;
  Launch L;
  const fp8blk_status status = current_launch(stream, &L);
  if (status != FP8BLK_OK) return status;
  const dim3 grid(static_cast<unsigned>(cdiv(K, 128)), static_cast<unsigned>(cdiv(N, 128)),
                  static_cast<unsigned>(count));
  transpose_kernel<<<grid, 256, 0, L.stream>>>(q, s, q2, s2, ldq, N, K, qt, ldqt, st, ldst, n_end);
  return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" {

fp8blk_status fp8blk_gated_backward(const void* dh, int64_t lddh, const void* g, const void* u,
                                    int64_t ldgu, int32_t activation, void* dgu, int64_t lddgu,
                                    int64_t M, int64_t N, fp8blk_stream stream) {
  if (!valid_activation(activation) || M < 0 || N < 0) return FP8BLK_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return FP8BLK_OK;
  if (M > kInt32Max || N > kInt32Max) return FP8BLK_ERR_INVALID_ARG;
  const int64_t Np = round_up(N, 128);
  if (!dh || !g || !u || !dgu || lddh < N || ldgu < N || lddgu < 2 * Np) return FP8BLK_ERR_INVALID_ARG;
  if (lddh % 8 || ldgu % 8 || lddgu % 8 || !aligned(dh, 16) || !aligned(g, 16) || !aligned(u, 16) ||
      !aligned(dgu, 16))
    return FP8BLK_ERR_ALIGNMENT;
  if (one_of(dgu, dh, g, u)) return FP8BLK_ERR_INVALID_ARG;
  Launch L;
  fp8blk_status st = current_launch(stream, &L);
  if (st != FP8BLK_OK) return st;
  const int64_t gx = cdiv(Np, 8 * 256);
  // Rows in steps of gridDim.y: at most 16 blocks per SM in all.
  const int64_t gy_max = cdiv(16 * L.num_sms, gx);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(M < gy_max ? M : gy_max));
  gated_backward_kernel<<<grid, 256, 0, L.stream>>>(
      static_cast<const uint16_t*>(dh), lddh, static_cast<const uint16_t*>(g),
      static_cast<const uint16_t*>(u), ldgu, act_params(activation), static_cast<uint16_t*>(dgu),
      lddgu, M, N, Np);
  return cuda_status(cudaGetLastError());
}

size_t fp8blk_epilogue_backward_workspace_size(int64_t M, int64_t N) {
  if (M <= 0 || N <= 0) return 0;
  const RowSplit r = row_split(M, N);
  return r.splits > 1 ? static_cast<size_t>(r.splits) * static_cast<size_t>(N) * sizeof(float) : 0;
}

fp8blk_status fp8blk_epilogue_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz,
                                       int32_t activation, void* dz, int64_t lddz, float* dbias,
                                       int64_t M, int64_t N, void* workspace,
                                       size_t workspace_bytes, fp8blk_stream stream) {
  if (!valid_activation(activation) || M < 0 || N < 0) return FP8BLK_ERR_INVALID_ARG;
  if (M > kInt32Max || N > kInt32Max) return FP8BLK_ERR_INVALID_ARG;
  if (N == 0 || (M == 0 && !dbias)) return FP8BLK_OK;
  if (!aligned(dbias, 4)) return FP8BLK_ERR_ALIGNMENT;
  const bool identity = activation == FP8BLK_ACT_NONE;
  if (M > 0) {
    if (!dy || lddy < N || (!identity && !z)) return FP8BLK_ERR_INVALID_ARG;
    if (lddy % 8 || !aligned(dy, 16)) return FP8BLK_ERR_ALIGNMENT;
    if (!identity) {
      if (ldz < N) return FP8BLK_ERR_INVALID_ARG;
      if (ldz % 8 || !aligned(z, 16)) return FP8BLK_ERR_ALIGNMENT;
    }
    if (dz) {
      if (lddz < N || (dz == dy && lddz != lddy) || (dz == z && !identity && lddz != ldz))
        return FP8BLK_ERR_INVALID_ARG;
      if (lddz % 8 || !aligned(dz, 16)) return FP8BLK_ERR_ALIGNMENT;
    }
    if (dbias) {
      const size_t need = fp8blk_epilogue_backward_workspace_size(M, N);
      if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return FP8BLK_ERR_WORKSPACE;
    }
  }
  if (M > 0 && one_of(dbias, dy, z, dz)) return FP8BLK_ERR_INVALID_ARG;
  if (identity && dz == dy) dz = nullptr;  // already there
  if (M > 0 && !dz && !dbias) return FP8BLK_OK;
  Launch L;
  fp8blk_status st = current_launch(stream, &L);
  if (st != FP8BLK_OK) return st;
  if (M == 0)
    return cuda_status(cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * sizeof(float), L.stream));
  const RowSplit r = row_split(M, N);
  const dim3 grid(static_cast<unsigned>(cdiv(N, kStripCols)), static_cast<unsigned>(r.splits));
  const uint16_t* dyp = static_cast<const uint16_t*>(dy);
  const uint16_t* zp = identity ? nullptr : static_cast<const uint16_t*>(z);
  uint16_t* dzp = static_cast<uint16_t*>(dz);
  const ActParams act = act_params(activation);
  if (!dbias) {
    epilogue_backward_kernel<false><<<grid, 256, 0, L.stream>>>(dyp, lddy, zp, ldz, act, dzp, lddz,
                                                                nullptr, M, N, r.rows);
    return cuda_status(cudaGetLastError());
  }
  float* sums = r.splits > 1 ? static_cast<float*>(workspace) : dbias;
  epilogue_backward_kernel<true><<<grid, 256, 0, L.stream>>>(dyp, lddy, zp, ldz, act, dzp, lddz,
                                                             sums, M, N, r.rows);
  if (cudaGetLastError() != cudaSuccess) return FP8BLK_ERR_CUDA;
  if (r.splits == 1) return FP8BLK_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cdiv(N, 256)));
  cfg.blockDim = dim3(256);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, column_sum_kernel, static_cast<const float*>(sums),
                                        r.splits, N, dbias));
}

fp8blk_status fp8blk_transpose_weight(const uint8_t* q, int64_t ldq, const float* scale_inv,
                                      int64_t N, int64_t K, uint8_t* qt, int64_t ldqt, float* st,
                                      int64_t ldst, int32_t zero_pad, fp8blk_stream stream) {
  if (zero_pad != 0 && zero_pad != 1) return FP8BLK_ERR_INVALID_ARG;
  return transpose(q, scale_inv, q, scale_inv, 1, ldq, N, K, qt, ldqt, st, ldst,
                   zero_pad ? round_up(N, 128) : N, stream);
}

fp8blk_status fp8blk_transpose_gated_weights(const uint8_t* q_gate, const float* s_gate,
                                             const uint8_t* q_up, const float* s_up, int64_t ldq,
                                             int64_t N, int64_t K, uint8_t* qt, int64_t ldqt,
                                             float* st, fp8blk_stream stream) {
  return transpose(q_gate, s_gate, q_up, s_up, 2, ldq, N, K, qt, ldqt, st, 2 * cdiv(N, 128),
                   round_up(N, 128), stream);
}

}  // extern "C"
