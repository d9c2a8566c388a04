/*
 * fp8blk -- the block-FP8 linear layer on NVIDIA B200 (sm_100a).
 *
 * Format (FastVideo PR #1829, "MiniMax H3: block-FP8 text encoder on Hopper,
 * its converter, and a 4xH100 FastH3 profile", section "Changes", converter
 * bullet): a linear's weight W[N][K] (nn.Linear order: N outputs, K inputs)
 * is stored as E4M3 codes q[N][K] plus one float weight_scale_inv per
 * 128 x 128 block, s[ceil(N/128)][ceil(K/128)]. Element (n, k) belongs to
 * block (n/128, k/128) and stands for E4M3(q[n][k]) * s[n/128][k/128]
 * (section "Purpose" and the tests bullet of "Changes": the dequantizer is
 * the code times its block's scale, broadcast over the block).
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers on the current CUDA device.
 *    The caller owns every buffer; the library allocates nothing (the linear
 *    calls take a caller-provided workspace) and never synchronizes.
 *  - Matrices are row-major with an explicit leading dimension ("ld"),
 *    counted in elements. Scale grids are dense row-major.
 *  - Calls are asynchronous and ordered on `stream` (a cudaStream_t; NULL is
 *    the legacy default stream). Argument errors are reported synchronously,
 *    before anything is launched; a failed launch returns FP8BLK_ERR_CUDA; a
 *    fault inside a kernel shows up at the caller's next synchronization.
 *  - The device must have compute capability 10.x (B200 class); otherwise
 *    FP8BLK_ERR_UNSUPPORTED_DEVICE. There is no fallback path.
 *  - Every tensor pointer must be 16-byte aligned (scale pointers: 4-byte).
 *  - A size of 0 is valid: nothing is read and (except the K = 0 linear, which
 *    writes y = 0) nothing is written.
 *  - Inputs must be finite; NaN and infinity are outside the contract.
 *  - Calls are reentrant; concurrent calls on different streams are safe as
 *    long as they do not share output or workspace buffers.
 */
#ifndef FP8BLK_H
#define FP8BLK_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FP8BLK_EXPORT __attribute__((visibility("default")))
#else
#define FP8BLK_EXPORT
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fp8blk_status {
  FP8BLK_OK = 0,
  FP8BLK_ERR_INVALID_ARG = 1,        /* negative size, ld too small, NULL pointer  */
  FP8BLK_ERR_ALIGNMENT = 2,          /* pointer or leading dimension misaligned    */
  FP8BLK_ERR_UNSUPPORTED_DEVICE = 3, /* current device is not compute capability 10.x */
  FP8BLK_ERR_WORKSPACE = 4,          /* workspace NULL or smaller than required    */
  FP8BLK_ERR_CUDA = 5,               /* a CUDA runtime call or launch failed       */
  FP8BLK_ERR_TIMEOUT = 6             /* a kernel gave up waiting (device error word set) */
} fp8blk_status;

/* A cudaStream_t, passed as an opaque pointer so this header needs no CUDA headers. */
typedef void* fp8blk_stream;

/* ---------------------------------------------------------------------------
 * (1) Converter: BF16 weight -> E4M3 codes + weight_scale_inv.
 * FastVideo PR #1829, section "Changes", converter bullet (E4M3 codes with a
 * float weight_scale_inv grid of shape [N/128, K/128]). For each 128 x 128 block:
 *   amax = max |W| over the block's in-bounds elements (ragged edge blocks
 *          are not padded with anything but zeros),
 *   s    = amax / 448            (float division, round to nearest even),
 *   q    = E4M3(W / s)           (float division, then round to nearest even
 *                                 with saturation to +-448);
 * a block whose elements are all +-0 gets s = 0 and codes 0x00 / 0x80 that
 * keep each element's sign.
 *   w         : BF16 [N][ldw], ldw >= K, ldw % 8 == 0           (input)
 *   q         : uint8 [N][ldq], ldq >= K, ldq % 16 == 0         (output; columns
 *               K..ldq-1 are not written)
 *   scale_inv : float [ceil(N/128)][ceil(K/128)], dense          (output)
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_quantize_weight(const void* w, int64_t N, int64_t K, int64_t ldw,
                                     uint8_t* q, int64_t ldq, float* scale_inv,
                                     fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * (2) Dequantizer: E4M3 codes + scales -> BF16 weight.
 * FastVideo PR #1829, section "Purpose" (the Hopper route materializes the
 * BF16 weight) and the tests bullet of "Changes" (bit-exact against the
 * scale broadcast over each block):
 *   w[n][k] = BF16( float(E4M3(q[n][k])) * s[n/128][k/128] )
 * with one float multiply and one round-to-nearest-even to BF16.
 *   q         : uint8 [N][ldq], ldq >= K, ldq % 16 == 0          (input)
 *   scale_inv : float [ceil(N/128)][ceil(K/128)]                  (input)
 *   w         : BF16 [N][ldw], ldw >= K, ldw % 8 == 0            (output)
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_dequantize(const uint8_t* q, int64_t ldq, const float* scale_inv,
                                int64_t N, int64_t K, void* w, int64_t ldw,
                                fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Activation quantizer (the first stage of fp8blk_linear_w8a8, exposed so its
 * output can be checked and reused). The Blackwell route of FastVideo PR
 * #1829 quantizes activations before its groupwise GEMM (section "Changes",
 * loader bullet); groups are 1 x 128 along K with the converter's recipe:
 *   sx[g][m] = max_{k in group g} |x[m][k]| / 448,  qx[m][k] = E4M3(x[m][k] / sx[g][m])
 *   x   : BF16 [M][ldx], ldx >= K, ldx % 8 == 0                   (input)
 *   qx  : uint8 [M][ldqx], ldqx >= K, ldqx % 16 == 0              (output)
 *   sx  : float [ceil(K/128)][ldsx], ldsx >= M, ldsx % 4 == 0     (output; note the
 *         group-major layout: the M scales of one K-group are contiguous)
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_quantize_act(const void* x, int64_t M, int64_t K, int64_t ldx,
                                  uint8_t* qx, int64_t ldqx, float* sx, int64_t ldsx,
                                  fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * (3) Linear, BF16 activations x block-FP8 weight ("W8A16"):
 *   y[m][n] = BF16( sum_kb s[n/128][kb] * P_kb[m][n] ),
 *   P_kb[m][n] = sum_{k in slab kb} x[m][k] * E4M3(q[n][k])   (FP32)
 * i.e. y = x . dequant(W)^T (FastVideo PR #1829, "Purpose": the same
 * computation as the Blackwell groupwise GEMM), with the block scale applied to
 * the FP32 partial of each 128-wide K slab and FP32 accumulation across
 * slabs. Tensor cores see the exact BF16 image of each E4M3 code.
 *   x : BF16 [M][ldx], ldx >= K, ldx % 8 == 0                        (input)
 *   q : uint8 [N][ldq], ldq >= K, ldq % 16 == 0; scale_inv as above  (input)
 *   y : BF16 [M][ldy], ldy >= N, ldy % 8 == 0; must not alias the inputs (output)
 *   workspace : 256-byte aligned; its contents on entry do not matter and
 *               are scratch on return.
 *     - M <= 128: fp8blk_workspace_size(0, M, N, K) bytes are required. The
 *       slabs are split evenly over the SMs (stream-K) and the workspace
 *       holds the FP32 partials of tiles split between SMs (at most
 *       160 x 2 x BT x 128 x 4 bytes, BT the token tile: 16, 32, 64 or 128).
 *     - M > 128: optional. Tiles of 256 tokens run whole, one per SM at a
 *       time; when the last wave of tiles would leave at least 15% of the SM
 *       time idle and the workspace holds fp8blk_workspace_size(0, M, N, K)
 *       bytes, that wave's slabs are split evenly over the SMs instead
 *       (partials of [256][128] floats, two per SM). NULL or a smaller
 *       workspace runs every tile whole.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_linear_w8a16(const void* x, int64_t ldx, const uint8_t* q, int64_t ldq,
                                  const float* scale_inv, void* y, int64_t ldy,
                                  int64_t M, int64_t N, int64_t K,
                                  void* workspace, size_t workspace_bytes,
                                  fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * (4) Linear with FP8 activations ("W8A8"): x is first quantized per 1 x 128
 * K-group (see fp8blk_quantize_act) into the workspace, then
 *   y[m][n] = BF16( sum_kb sx[kb][m] * s[n/128][kb] * P_kb[m][n] ),
 *   P_kb[m][n] = sum_{k in slab kb} E4M3(qx[m][k]) * E4M3(q[n][k])  (FP32)
 * on E4M3 x E4M3 tensor cores. Arguments as for fp8blk_linear_w8a16, with
 * workspace >= fp8blk_workspace_size(1, M, N, K). Workspace layout (so the
 * quantized activations can be inspected): qx uint8 [M][round_up(K, 16)] at
 * offset 0, then sx float [ceil(K/128)][round_up(M, 128)] at the next
 * 256-byte boundary.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_linear_w8a8(const void* x, int64_t ldx, const uint8_t* q, int64_t ldq,
                                 const float* scale_inv, void* y, int64_t ldy,
                                 int64_t M, int64_t N, int64_t K,
                                 void* workspace, size_t workspace_bytes,
                                 fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * W8A8 linear without a workspace argument. (The pages have no counterpart:
 * this is a calling convenience of this library.) For callers that cannot
 * allocate device memory -- e.g. a runtime that plans every buffer before it
 * starts serving and forbids allocation afterwards, or host code that must
 * not call cudaMalloc because it can synchronize the device and stall other
 * streams. Computes exactly what fp8blk_linear_w8a8 computes, with the same
 * arguments minus the workspace; its scratch is a fixed array of
 * FP8BLK_NOALLOC_SCRATCH_BYTES built into the library, present on every GPU
 * that loads it until the process exits. The call itself allocates nothing.
 *  - Limit: the problem must satisfy fp8blk_workspace_size(1, M, N, K) <=
 *    FP8BLK_NOALLOC_SCRATCH_BYTES (M * round_up(K, 16) bytes of codes plus the
 *    scales; e.g. M = 2048 at K = 5120); larger problems return
 *    FP8BLK_ERR_WORKSPACE before anything is launched.
 *  - The first call on a device (with that device current) looks up the
 *    array's device address once; make that first call before any stream
 *    capture (a first call on a capturing stream returns INVALID_ARG).
 *  - All calls share the one array: calls that can overlap on the GPU (on
 *    different streams, or from different threads) race on it and must be
 *    ordered by the caller.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, WORKSPACE (too large), CUDA.
 * ------------------------------------------------------------------------- */
#define FP8BLK_NOALLOC_SCRATCH_BYTES (16 * 1024 * 1024)
FP8BLK_EXPORT fp8blk_status fp8blk_linear_w8a8_noalloc(const void* x, int64_t ldx, const uint8_t* q,
                                                       int64_t ldq, const float* scale_inv, void* y,
                                                       int64_t ldy, int64_t M, int64_t N, int64_t K,
                                                       fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * W8A8 linear on activations already quantized by fp8blk_quantize_act, so
 * that sibling linears reading the same x (Q, K and V; gate and up) quantize
 * it once (FastVideo PR #1829, "Changes": the Blackwell route quantizes the
 * activations before the groupwise GEMM). Computes
 *   y[m][n] = BF16( sum_kb sx[kb][m] * s[n/128][kb] * P_kb[m][n] )
 * exactly as fp8blk_linear_w8a8 does after its own quantization step.
 *   qx : uint8 [M][ldqx], ldqx >= K, ldqx % 16 == 0, 16-byte aligned (input)
 *   sx : float [ceil(K/128)][ldsx], ldsx >= M, 4-byte aligned          (input)
 *   q, scale_inv, y, M, N, K : as for fp8blk_linear_w8a8.
 * No workspace. Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_linear_w8a8_quantized(const uint8_t* qx, int64_t ldqx,
                                                         const float* sx, int64_t ldsx,
                                                         const uint8_t* q, int64_t ldq,
                                                         const float* scale_inv, void* y,
                                                         int64_t ldy, int64_t M, int64_t N,
                                                         int64_t K, fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * A sequence of linears on device weights, launched back to back so that each
 * GEMM starts streaming its weights while the kernels before it finish
 * (programmatic dependent launch). This is the decode-time case: the weight
 * stream is the whole cost, and the linears of a layer follow one another.
 * Each job computes exactly what fp8blk_linear_w8a16 (mode 0) or
 * fp8blk_linear_w8a8 (mode 1) computes from the same arguments, in job order;
 * a job's x may be an earlier job's y, and a job's y may overwrite an
 * earlier job's x. The caller promises that no job writes another job's
 * weights (q, scale_inv): weights are read before the previous job has
 * finished. The first job waits for all earlier work on `stream`.
 *   jobs      : njobs job descriptions (host memory), each as for the linear
 *               calls (device pointers)
 *   workspace : DEVICE, at least the largest fp8blk_workspace_size(mode, M,
 *               N, K) over the jobs (the jobs use it one after another)
 * Every job is checked before anything is launched.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
typedef struct fp8blk_linear_args {
  int32_t mode;              /* 0 = W8A16, 1 = W8A8 */
  const void* x;             /* BF16 [M][ldx] */
  int64_t ldx;
  const uint8_t* q;          /* E4M3 codes [N][ldq] */
  int64_t ldq;
  const float* scale_inv;    /* [ceil(N/128)][ceil(K/128)] */
  void* y;                   /* BF16 [M][ldy] */
  int64_t ldy;
  int64_t M, N, K;
} fp8blk_linear_args;

FP8BLK_EXPORT fp8blk_status fp8blk_linear_sequence(const fp8blk_linear_args* jobs, int64_t njobs,
                                                   void* workspace, size_t workspace_bytes,
                                                   fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Layerwise FP8 weight streaming (FastVideo PR #1829, "Purpose": the FP8
 * checkpoint is what keeps the encoder resident, and what an offloaded
 * encoder moves instead of BF16 weights; the page reports both the memory
 * and the offload time of the two forms). Runs a sequence of linears whose
 * codes and scales live in HOST memory through a ring of `nslots` device
 * weight slots: job i's weights are copied into slot i % nslots on `copy`
 * while earlier jobs run on `compute`; job i's linear runs on `compute` once
 * its copy has landed, and a slot is refilled only after the linear that
 * read it has finished. Each job computes exactly what fp8blk_linear_w8a16
 * (mode 0) or fp8blk_linear_w8a8 (mode 1) computes from the same weights on
 * the device.
 *   jobs[i].q_host     : uint8 [N][ldq] in HOST memory (pinned, or the
 *                        copies are not asynchronous), ldq >= K, ldq % 16 == 0
 *   jobs[i].scale_host : float [ceil(N/128)][ceil(K/128)] in HOST memory
 *   jobs[i].x, ldx, y, ldy, M, N, K : DEVICE activations and output, as for
 *                        the linear calls (x read, y written on `compute`)
 *   slots      : DEVICE, nslots consecutive slots of slot_bytes each;
 *                256-byte aligned, slot_bytes % 256 == 0 and
 *                slot_bytes >= fp8blk_stream_slot_bytes(N, K, ldq) of every
 *                job (codes at the start of a slot, scales after them)
 *   workspace  : DEVICE, as for the linear calls, at least the largest
 *                fp8blk_workspace_size(mode, M, N, K) over the jobs
 *   compute, copy : streams (the same stream twice is valid: no overlap)
 *   events     : 2 * nslots cudaEvent_t created by the caller (timing
 *                disabled is best); the library only records and waits on them
 * The copies of a call start after the work already enqueued on `compute`,
 * so consecutive calls may share slots and events.
 * Everything is enqueued asynchronously: on return nothing need have run.
 * Every job is checked before anything is enqueued; a CUDA error while
 * enqueuing returns FP8BLK_ERR_CUDA with the jobs before it enqueued.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
typedef struct fp8blk_linear_job {
  int32_t mode;              /* 0 = W8A16, 1 = W8A8 */
  const uint8_t* q_host;     /* host codes [N][ldq] */
  const float* scale_host;   /* host scales [ceil(N/128)][ceil(K/128)] */
  int64_t ldq;
  const void* x;             /* device BF16 activations [M][ldx] */
  int64_t ldx;
  void* y;                   /* device BF16 output [M][ldy] */
  int64_t ldy;
  int64_t M, N, K;
} fp8blk_linear_job;

/* A cudaEvent_t, passed as an opaque pointer. */
typedef void* fp8blk_event;

/* Bytes of one weight slot for an N x K linear with code pitch ldq: the
 * codes rounded up to 256 bytes, then the scales, rounded up to 256. Pure
 * host function; 0 for negative sizes or ldq < K. */
FP8BLK_EXPORT size_t fp8blk_stream_slot_bytes(int64_t N, int64_t K, int64_t ldq);

FP8BLK_EXPORT fp8blk_status fp8blk_streamed_linears(const fp8blk_linear_job* jobs, int64_t njobs,
                                                    void* slots, size_t slot_bytes, int32_t nslots,
                                                    void* workspace, size_t workspace_bytes,
                                                    fp8blk_stream compute, fp8blk_stream copy,
                                                    fp8blk_event* events);

/* ---------------------------------------------------------------------------
 * The feed-forward operators: what a layer does around its linears, in the
 * kernels of the linears. Weights are in the block-FP8 form of this header;
 * the backward calls return gradients with respect to the activations and the
 * dequantized weights (E4M3 code times scale). Activation functions:
 *   NONE       z
 *   RELU       max(z, 0)                    (derivative 0 at z = 0)
 *   GELU       z Phi(z), Phi the normal distribution function
 *   GELU_TANH  z / 2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
 *   SILU       z / (1 + exp(-z))
 * All of them are computed in FP32 from FP32 sums; BF16 results are rounded
 * once, to nearest even. That includes dg, du and dz below, so input and weight
 * gradients made from them (an FP32 weight gradient too) are FP32 sums of rounded
 * terms: 1.7e-3 in relative norm from those of unrounded ones, the size of one BF16
 * rounding. Outputs must not overlap inputs or one another, except where a call says
 * so; the same pointer for both is refused with INVALID_ARG.
 * ------------------------------------------------------------------------- */
typedef enum fp8blk_activation {
  FP8BLK_ACT_NONE = 0,
  FP8BLK_ACT_RELU = 1,
  FP8BLK_ACT_GELU = 2,
  FP8BLK_ACT_GELU_TANH = 3,
  FP8BLK_ACT_SILU = 4
} fp8blk_activation;

/* What follows a linear's product: z = x . dequant(W)^T + bias,
 * y = act(z) + residual. Null pointers leave a part out. */
typedef struct fp8blk_epilogue {
  const void* bias;       /* BF16 [N] or NULL */
  int32_t activation;     /* an fp8blk_activation */
  const void* residual;   /* BF16 [M][ldr] or NULL; ldr >= N, ldr % 8 == 0; may be y
                             itself (same pointer, ldr == ldy), must not overlap it otherwise */
  int64_t ldr;
  void* preact;           /* BF16 [M][ldp] or NULL: receives z, rounded to BF16, for the
                             backward pass; ldp >= N, ldp % 8 == 0 */
  int64_t ldp;
} fp8blk_epilogue;

/* ---------------------------------------------------------------------------
 * fp8blk_linear_w8a16 / fp8blk_linear_w8a8 with an epilogue. Arguments,
 * workspace and ordering as for those calls; K = 0 gives y = act(bias) +
 * residual. The FP32 sum is never rounded before the epilogue. The order of a sum
 * depends on the sizes and the GPU alone (repeated calls agree bit for bit), but
 * it may differ from that of the linear without epilogue.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_linear_w8a16_epilogue(
    const void* x, int64_t ldx, const uint8_t* q, int64_t ldq, const float* scale_inv, void* y,
    int64_t ldy, int64_t M, int64_t N, int64_t K, const fp8blk_epilogue* epilogue, void* workspace,
    size_t workspace_bytes, fp8blk_stream stream);
FP8BLK_EXPORT fp8blk_status fp8blk_linear_w8a8_epilogue(
    const void* x, int64_t ldx, const uint8_t* q, int64_t ldq, const float* scale_inv, void* y,
    int64_t ldy, int64_t M, int64_t N, int64_t K, const fp8blk_epilogue* epilogue, void* workspace,
    size_t workspace_bytes, fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Gated linear, the first half of a gated feed-forward block: both
 * projections, the activation and the product in one kernel,
 *   g = x . dequant(Wg)^T, u = x . dequant(Wu)^T, h[m][n] = BF16(act(g) * u),
 * with BF16 activations (w8a16) or activations quantized per 1 x 128 K-group
 * (w8a8), as in the linear calls.
 *   q_gate, q_up : uint8 [N][ldq], one ldq for both; ldq >= K, ldq % 16 == 0
 *   s_gate, s_up : float [ceil(N/128)][ceil(K/128)]
 *                  (a fused [2N][K] weight with N % 128 == 0 is passed as its
 *                  two halves)
 *   h    : BF16 [M][ldh], ldh >= N, ldh % 8 == 0                     (output)
 *   g, u : BF16 [M][ldgu] or both NULL: the pre-activations, rounded to BF16,
 *          for fp8blk_gated_backward (h itself is computed from the unrounded
 *          sums); ldgu >= N, ldgu % 8 == 0                            (output)
 *   workspace : as for the linear calls, for 2 N outputs: fp8blk_workspace_size(
 *          mode, M, 2 * N, K) bytes, required and optional as there.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_gated_linear_w8a16(
    const void* x, int64_t ldx, const uint8_t* q_gate, const float* s_gate, const uint8_t* q_up,
    const float* s_up, int64_t ldq, int32_t activation, void* h, int64_t ldh, void* g, void* u,
    int64_t ldgu, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
    fp8blk_stream stream);
FP8BLK_EXPORT fp8blk_status fp8blk_gated_linear_w8a8(
    const void* x, int64_t ldx, const uint8_t* q_gate, const float* s_gate, const uint8_t* q_up,
    const float* s_up, int64_t ldq, int32_t activation, void* h, int64_t ldh, void* g, void* u,
    int64_t ldgu, int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
    fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Backward pass of the gated product: from dh and the kept g, u,
 *   dg = BF16(dh * u * act'(g)),  du = BF16(dh * act(g)).
 *   dh   : BF16 [M][lddh]; g, u : BF16 [M][ldgu]                     (input)
 *   dgu  : BF16 [M][lddgu], lddgu >= 2 * round_up(N, 128): dg in columns
 *          [0, N), du in [Np, Np + N) with Np = round_up(N, 128); columns
 *          [N, Np) and [Np + N, 2 Np) are set to 0                    (output)
 * All leading dimensions % 8 == 0. That layout is the activation operand of
 * the linears against the two transposed weights side by side (see
 * fp8blk_transpose_gated_weights): dx = dg . Wg + du . Wu in one product.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_gated_backward(const void* dh, int64_t lddh, const void* g,
                                                  const void* u, int64_t ldgu, int32_t activation,
                                                  void* dgu, int64_t lddgu, int64_t M, int64_t N,
                                                  fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Backward pass of an epilogue: from dy and the kept z,
 *   dz = BF16(dy * act'(z)),  dbias[n] = sum_m dy[m][n] * act'(z[m][n])
 * (the residual's gradient is dy itself). dbias is summed in FP32 from the
 * unrounded products, in an order that depends on M and N alone.
 *   dy : BF16 [M][lddy]; z : BF16 [M][ldz], may be NULL with NONE    (input)
 *   dz    : BF16 [M][lddz] or NULL; may be dy or z itself             (output)
 *   dbias : float [N] or NULL, 4-byte aligned                         (output)
 *   workspace : fp8blk_epilogue_backward_workspace_size(M, N) bytes, 256-byte
 *           aligned, needed when dbias is given (its contents are scratch)
 * All leading dimensions % 8 == 0. M = 0 sets dbias to 0.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, WORKSPACE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_epilogue_backward(const void* dy, int64_t lddy, const void* z,
                                                     int64_t ldz, int32_t activation, void* dz,
                                                     int64_t lddz, float* dbias, int64_t M,
                                                     int64_t N, void* workspace,
                                                     size_t workspace_bytes, fp8blk_stream stream);

/* Workspace bytes of fp8blk_epilogue_backward with dbias. Pure host function;
 * 0 for negative sizes, and where no workspace is needed. */
FP8BLK_EXPORT size_t fp8blk_epilogue_backward_workspace_size(int64_t M, int64_t N);

/* ---------------------------------------------------------------------------
 * Transposed weight: qt[k][n] = q[n][k], st[k/128][n/128] = s[n/128][k/128].
 * The blocks are square, so the transpose of a block-FP8 weight is one, code
 * for code, and dx = dz . dequant(W) is a linear call on (qt, st):
 * fp8blk_linear_w8a16(dz, qt, st) with N and K exchanged.
 *   q  : uint8 [N][ldq], ldq >= K, ldq % 16 == 0; scale_inv as above (input)
 *   qt : uint8 [K][ldqt], ldqt >= round_up(N, 128) if zero_pad, else N;
 *        ldqt % 16 == 0; columns [N, round_up(N, 128)) are set to 0 if
 *        zero_pad, else not written                                   (output)
 *   st : float [ceil(K/128)][ldst], ldst >= ceil(N/128)               (output)
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_transpose_weight(const uint8_t* q, int64_t ldq,
                                                    const float* scale_inv, int64_t N, int64_t K,
                                                    uint8_t* qt, int64_t ldqt, float* st,
                                                    int64_t ldst, int32_t zero_pad,
                                                    fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Both weights of a gated linear transposed side by side, the layout that
 * fp8blk_gated_backward's output multiplies (Np = round_up(N, 128)): the gate
 * weight in columns [0, N), the up weight in [Np, Np + N), zero codes between.
 *   q_gate, q_up : uint8 [N][ldq]; s_gate, s_up : as above            (input)
 *   qt : uint8 [K][ldqt], ldqt >= 2 Np, ldqt % 16 == 0                (output)
 *   st : float [ceil(K/128)][2 Np / 128], dense                       (output)
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_transpose_gated_weights(
    const uint8_t* q_gate, const float* s_gate, const uint8_t* q_up, const float* s_up, int64_t ldq,
    int64_t N, int64_t K, uint8_t* qt, int64_t ldqt, float* st, fp8blk_stream stream);

/* ---------------------------------------------------------------------------
 * Weight gradient of a linear: dw[n][k] = sum_m dz[m][n] * x[m][k], BF16
 * operands, FP32 sums in an order that depends on the sizes (and on whether a
 * workspace was given) alone. The sums are of dz as it is given: where that is an
 * output of the calls above, of its rounded values.
 *   dz : BF16 [M][lddz], lddz >= N; x : BF16 [M][ldx], ldx >= K      (input)
 *   dw : float (dw_fp32 = 1) or BF16 (dw_fp32 = 0) [N][lddw], lddw >= K (output)
 *   accumulate : 1 adds the sums to dw (FP32 only), 0 overwrites it
 *   workspace : optional, 256-byte aligned, scratch: with
 *          fp8blk_linear_grad_weight_workspace_size(M, N, K) bytes (0 where it
 *          would not help) a weight of few tiles has its tokens split over the
 *          GPU. NULL or a smaller one runs every tile whole.
 * lddz, ldx % 8 == 0; lddw % 4 == 0 (FP32) or % 8 == 0 (BF16). M = 0 sets dw
 * to 0, or leaves it with accumulate.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_linear_grad_weight(const void* dz, int64_t lddz, const void* x,
                                                      int64_t ldx, void* dw, int64_t lddw,
                                                      int32_t dw_fp32, int32_t accumulate,
                                                      int64_t M, int64_t N, int64_t K,
                                                      void* workspace, size_t workspace_bytes,
                                                      fp8blk_stream stream);

/* Workspace bytes of fp8blk_linear_grad_weight. Pure host function; 0 for
 * negative sizes, and where no workspace is used. */
FP8BLK_EXPORT size_t fp8blk_linear_grad_weight_workspace_size(int64_t M, int64_t N, int64_t K);

/* Workspace bytes for a linear: mode 0 = W8A16, 1 = W8A8. Pure host function;
 * returns 0 for an invalid mode or negative sizes. */
FP8BLK_EXPORT size_t fp8blk_workspace_size(int mode, int64_t M, int64_t N, int64_t K);

/* ---------------------------------------------------------------------------
 * Element codec of the converter, exposed for verification: codes[i] =
 * E4M3(v[i]) with round-to-nearest-even and saturation to +-448 (NaN -> 0x7F),
 * the same device routine the converter and the activation quantizer use.
 *   v : float [n] (device, 16-byte aligned); codes : uint8 [n] (device, 16-byte aligned)
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED_DEVICE, CUDA.
 * ------------------------------------------------------------------------- */
FP8BLK_EXPORT fp8blk_status fp8blk_encode_e4m3(const float* v, int64_t n, uint8_t* codes, fp8blk_stream stream);

/* Self-test of the failure-detection path: launches one warp that waits, with
 * the kernels' own bounded wait, on an mbarrier phase that nothing completes.
 * After limit_cycles SM cycles (1000 <= limit_cycles <= 4e9; a few million is
 * about a millisecond) the wait gives up, sets flag 16 in the error word and
 * the kernel returns, leaving the context usable: fp8blk_read_device_error
 * then reports FP8BLK_ERR_TIMEOUT with word 16. No fault, trap or hang.
 * Errors: INVALID_ARG, UNSUPPORTED_DEVICE, CUDA. */
FP8BLK_EXPORT fp8blk_status fp8blk_selftest_wait_timeout(int64_t limit_cycles, fp8blk_stream stream);

/* Reads and clears the current device's error word (bit flags set by a kernel
 * whose bounded wait ran out: 1 load, 2 MMA, 4 epilogue, 8 weight expansion,
 * 16 the self-test above).
 * Synchronizes the device. *word receives the flags; returns FP8BLK_ERR_TIMEOUT
 * when any flag was set, FP8BLK_OK when none, FP8BLK_ERR_CUDA on a CUDA error. */
FP8BLK_EXPORT fp8blk_status fp8blk_read_device_error(uint32_t* word);

/* Human-readable name of a status code (static storage). */
FP8BLK_EXPORT const char* fp8blk_status_string(fp8blk_status status);

/* Library version: major * 10000 + minor * 100 + patch. */
FP8BLK_EXPORT int fp8blk_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8BLK_H */
