// Entry points of the linears with an epilogue and of the gated linear
// (include/fp8blk.h): argument checks, then the launches of gemm_w8a16.cu and
// gemm_w8a8.cu. The empty product (K = 0) has a kernel of its own here.
#include <cuda_runtime.h>

#include "epilogue.cuh"
#include "internal.cuh"
#include "ptx.cuh"

namespace fp8blk {
namespace {

// K = 0: z = bias, y = act(bias) + residual; one thread per element, rows in
// steps of the grid.
__global__ void __launch_bounds__(256) empty_product_kernel(FusedEpi e, uint16_t* y, int64_t ldy,
                                                            int64_t M, int64_t N) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (n >= N) return;
  const float z = e.bias ? bf16_bits_to_f32(e.bias[n]) : 0.0f;
  const float a = act_value(e.act, z);
  const uint16_t zb = static_cast<uint16_t>(cvt_bf16x2(0.0f, z));
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const float r = e.residual ? bf16_bits_to_f32(e.residual[m * e.ldr + n]) : 0.0f;
    if (e.preact) e.preact[m * e.ldp + n] = zb;
    y[m * ldy + n] = static_cast<uint16_t>(cvt_bf16x2(0.0f, a + r));
  }
}

// A BF16 matrix operand with a leading dimension (not null).
fp8blk_status check_matrix(const void* p, int64_t ld, int64_t cols) {
  if (ld < cols) return FP8BLK_ERR_INVALID_ARG;
  if (ld % 8 || !aligned(p, 16)) return FP8BLK_ERR_ALIGNMENT;
  return FP8BLK_OK;
}

fp8blk_status linear_epilogue(int mode, const void* x, int64_t ldx, const uint8_t* q, int64_t ldq,
                              const float* scale_inv, void* y, int64_t ldy, int64_t M, int64_t N,
                              int64_t K, const fp8blk_epilogue* ep, void* ws, size_t ws_bytes,
                              fp8blk_stream stream) {
  if (!ep || !valid_activation(ep->activation)) return FP8BLK_ERR_INVALID_ARG;
  fp8blk_status st = validate_linear(x, ldx, q, ldq, scale_inv, y, ldy, M, N, K, ws, ws_bytes,
                                     required_workspace(mode, M, N, K));
  if (st != FP8BLK_OK) return st;
  if (M == 0 || N == 0) return FP8BLK_OK;
  if (!aligned(ep->bias, 16)) return FP8BLK_ERR_ALIGNMENT;
  if (ep->residual && (st = check_matrix(ep->residual, ep->ldr, N)) != FP8BLK_OK) return st;
  if (ep->residual == y && ep->ldr != ldy) return FP8BLK_ERR_INVALID_ARG;
  if (ep->preact && (st = check_matrix(ep->preact, ep->ldp, N)) != FP8BLK_OK) return st;
  if (ep->preact && (ep->preact == y || ep->preact == ep->residual)) return FP8BLK_ERR_INVALID_ARG;
  // An output over an input would be written while other tiles still read it.
  for (const void* out : {static_cast<const void*>(y), static_cast<const void*>(ep->preact)})
    if (one_of(out, ep->bias) || (K > 0 && one_of(out, x, q, scale_inv))) return FP8BLK_ERR_INVALID_ARG;
  Launch L;
  st = current_launch(stream, &L);
  if (st != FP8BLK_OK) return st;
  const FusedEpi e = {static_cast<const uint16_t*>(ep->bias),
                      static_cast<const uint16_t*>(ep->residual),
                      ep->ldr,
                      static_cast<uint16_t*>(ep->preact),
                      ep->ldp,
                      act_params(ep->activation)};
  uint16_t* yo = static_cast<uint16_t*>(y);
  if (K == 0) {
    const dim3 grid(static_cast<unsigned>(cdiv(N, 256)), static_cast<unsigned>(M < 1024 ? M : 1024));
    empty_product_kernel<<<grid, 256, 0, L.stream>>>(e, yo, ldy, M, N);
    return cuda_status(cudaGetLastError());
  }
  const uint16_t* xi = static_cast<const uint16_t*>(x);
  if (mode == 0)
    return cuda_status(launch_w8a16_fused(L, xi, ldx, q, ldq, scale_inv, yo, ldy, M, N, K, ws, ws_bytes, e));
  uint8_t* qx = static_cast<uint8_t*>(ws);
  float* sx = reinterpret_cast<float*>(qx + w8a8_sx_offset(M, K));
  const int64_t ldqx = w8a8_ldqx(K), ldsx = w8a8_ldsx(M);
  if (launch_quantize_act(L, xi, M, K, ldx, qx, ldqx, sx, ldsx) != cudaSuccess) return FP8BLK_ERR_CUDA;
  return cuda_status(launch_w8a8_fused(L, qx, ldqx, sx, ldsx, q, ldq, scale_inv, yo, ldy, M, N, K, e));
}

fp8blk_status gated_linear(int mode, const void* x, int64_t ldx, const uint8_t* q_gate,
                           const float* s_gate, const uint8_t* q_up, const float* s_up, int64_t ldq,
                           int32_t activation, void* h, int64_t ldh, void* g, void* u, int64_t ldgu,
                           int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                           fp8blk_stream stream) {
  if (!valid_activation(activation)) return FP8BLK_ERR_INVALID_ARG;
  if (N > kInt32Max / 2) return FP8BLK_ERR_INVALID_ARG;
  fp8blk_status st = validate_linear(x, ldx, q_gate, ldq, s_gate, h, ldh, M, N, K, ws, ws_bytes,
                                     required_workspace(mode, M, 2 * N, K));
  if (st != FP8BLK_OK) return st;
  if (M == 0 || N == 0) return FP8BLK_OK;
  if (K > 0) {
    if (!q_up || !s_up) return FP8BLK_ERR_INVALID_ARG;
    if (!aligned(q_up, 16) || !aligned(s_up, 4)) return FP8BLK_ERR_ALIGNMENT;
  }
  if ((g == nullptr) != (u == nullptr)) return FP8BLK_ERR_INVALID_ARG;
  if (g) {
    if ((st = check_matrix(g, ldgu, N)) != FP8BLK_OK) return st;
    if ((st = check_matrix(u, ldgu, N)) != FP8BLK_OK) return st;
    if (g == u || g == h || u == h) return FP8BLK_ERR_INVALID_ARG;
  }
  for (const void* out : {h, g, u})
    if (K > 0 && one_of(out, x, q_gate, s_gate, q_up, s_up)) return FP8BLK_ERR_INVALID_ARG;
  Launch L;
  st = current_launch(stream, &L);
  if (st != FP8BLK_OK) return st;
  if (K == 0) {  // g = u = 0, so h = 0
    const size_t w = static_cast<size_t>(N) * 2, rows = static_cast<size_t>(M);
    cudaError_t e = cudaMemset2DAsync(h, static_cast<size_t>(ldh) * 2, 0, w, rows, L.stream);
    if (e == cudaSuccess && g) {
      e = cudaMemset2DAsync(g, static_cast<size_t>(ldgu) * 2, 0, w, rows, L.stream);
      if (e == cudaSuccess) e = cudaMemset2DAsync(u, static_cast<size_t>(ldgu) * 2, 0, w, rows, L.stream);
    }
    return cuda_status(e);
  }
  const GatedEpi e = {q_up, s_up, static_cast<uint16_t*>(g), static_cast<uint16_t*>(u), ldgu,
                      act_params(activation)};
  const uint16_t* xi = static_cast<const uint16_t*>(x);
  uint16_t* ho = static_cast<uint16_t*>(h);
  if (mode == 0)
    return cuda_status(
        launch_w8a16_gated(L, xi, ldx, q_gate, ldq, s_gate, ho, ldh, M, N, K, ws, ws_bytes, e));
  uint8_t* qx = static_cast<uint8_t*>(ws);
  float* sx = reinterpret_cast<float*>(qx + w8a8_sx_offset(M, K));
  const int64_t ldqx = w8a8_ldqx(K), ldsx = w8a8_ldsx(M);
  if (launch_quantize_act(L, xi, M, K, ldx, qx, ldqx, sx, ldsx) != cudaSuccess) return FP8BLK_ERR_CUDA;
  return cuda_status(
      launch_w8a8_gated(L, qx, ldqx, sx, ldsx, q_gate, ldq, s_gate, ho, ldh, M, N, K, e));
}

}  // namespace
}  // namespace fp8blk

using namespace fp8blk;

extern "C" {

fp8blk_status fp8blk_linear_w8a16_epilogue(const void* x, int64_t ldx, const uint8_t* q,
                                           int64_t ldq, const float* scale_inv, void* y,
                                           int64_t ldy, int64_t M, int64_t N, int64_t K,
                                           const fp8blk_epilogue* epilogue, void* workspace,
                                           size_t workspace_bytes, fp8blk_stream stream) {
  return linear_epilogue(0, x, ldx, q, ldq, scale_inv, y, ldy, M, N, K, epilogue, workspace,
                         workspace_bytes, stream);
}

fp8blk_status fp8blk_linear_w8a8_epilogue(const void* x, int64_t ldx, const uint8_t* q, int64_t ldq,
                                          const float* scale_inv, void* y, int64_t ldy, int64_t M,
                                          int64_t N, int64_t K, const fp8blk_epilogue* epilogue,
                                          void* workspace, size_t workspace_bytes,
                                          fp8blk_stream stream) {
  return linear_epilogue(1, x, ldx, q, ldq, scale_inv, y, ldy, M, N, K, epilogue, workspace,
                         workspace_bytes, stream);
}

fp8blk_status fp8blk_gated_linear_w8a16(const void* x, int64_t ldx, const uint8_t* q_gate,
                                        const float* s_gate, const uint8_t* q_up,
                                        const float* s_up, int64_t ldq, int32_t activation, void* h,
                                        int64_t ldh, void* g, void* u, int64_t ldgu, int64_t M,
                                        int64_t N, int64_t K, void* workspace,
                                        size_t workspace_bytes, fp8blk_stream stream) {
  return gated_linear(0, x, ldx, q_gate, s_gate, q_up, s_up, ldq, activation, h, ldh, g, u, ldgu, M,
                      N, K, workspace, workspace_bytes, stream);
}

fp8blk_status fp8blk_gated_linear_w8a8(const void* x, int64_t ldx, const uint8_t* q_gate,
                                       const float* s_gate, const uint8_t* q_up, const float* s_up,
                                       int64_t ldq, int32_t activation, void* h, int64_t ldh,
                                       void* g, void* u, int64_t ldgu, int64_t M, int64_t N,
                                       int64_t K, void* workspace, size_t workspace_bytes,
                                       fp8blk_stream stream) {
  return gated_linear(1, x, ldx, q_gate, s_gate, q_up, s_up, ldq, activation, h, ldh, g, u, ldgu, M,
                      N, K, workspace, workspace_bytes, stream);
}

}  // extern "C"
