// The element-wise functions that follow a linear's product (bias,
// activation, residual; the gate of a feed-forward block) and the parameters
// that carry them into the GEMM epilogues.
//
// Activations. silu(z) = z s(z) and gelu_tanh(z) = z s(2 sqrt(2/pi) (z +
// 0.044715 z^3)) with the logistic s are one form, z s(c1 z + c3 z^3); relu
// and the identity are max(z, lo) with lo = 0 and -infinity; gelu(z) = z
// Phi(z) with the normal distribution function Phi. So three cases cover the
// five names, chosen by a branch that is uniform over the grid. All of it is
// computed in FP32 from the FP32 product; 2^x and 1/x are the approximate
// instructions, whose error (a few units of 2^-23, growing with the exponent's
// magnitude) is far below half a BF16 step. Their subnormal results count as 0,
// which would lose the far tails (silu is still a normal number at z = -92, where
// its logistic is not), so the exponents are shifted by kTailBits and the result is
// scaled back by a multiplication, which underflows gradually.
//
// What bounds this code inside a GEMM is instruction fetch: a thread holds 64
// to 128 sums in registers, so the code is unrolled that many times and run
// once per tile. With the branch inside act_value per element and the library's
// erfcf inlined, the W8A16 linear of 512 x 5120 x 51200 took 485 us with no
// activation at all against 256 us plain; so a group of values takes one
// branch (act_apply), and Phi is a short formula of its own.
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "fp8blk.h"

namespace fp8blk {

enum ActKind : int { kActMax = 0, kActLogistic = 1, kActNormal = 2 };

struct ActParams {
  int kind;
  float c1, c3;  // kActLogistic: z s(c1 z + c3 z^3), both times -log2(e)
  float lo;      // kActMax: max(z, lo)
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTailBits = 24.0f, kTailScale = 5.9604644775390625e-8f;  // 2^-24

inline bool valid_activation(int a) { return a >= FP8BLK_ACT_NONE && a <= FP8BLK_ACT_SILU; }

inline ActParams act_params(int a) {
  switch (a) {
    case FP8BLK_ACT_RELU: return {kActMax, 0.0f, 0.0f, 0.0f};
    case FP8BLK_ACT_GELU: return {kActNormal, 0.0f, 0.0f, 0.0f};
    case FP8BLK_ACT_GELU_TANH:  // 2 sqrt(2/pi), and 0.044715 of it
      return {kActLogistic, -kLog2e * 1.5957691216057308f, -kLog2e * 0.07135481282673f, 0.0f};
    case FP8BLK_ACT_SILU: return {kActLogistic, -kLog2e, 0.0f, 0.0f};
  }
  return {kActMax, 0.0f, 0.0f, -INFINITY};
}

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The larger of two; NaN if either is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Phi(z) = 1 - Phi(-z), and for x = |z| / sqrt 2 the tail Phi(-|z|) = erfc(x) / 2
// = erfcx(x) exp(-x^2) / 2, which keeps its relative accuracy where 1 + erf
// would cancel. erfcx(x) is a polynomial in t = 1 / (1 + 0.6 x), fitted to it for
// 0 <= x <= 10 with equal relative error (3.1e-7; 6e-7 in FP32); beyond 10.2,
// exp(-x^2) is 0 in FP32. gauss is exp(-z^2/2).
__device__ __forceinline__ float act_normal(float z, float& gauss) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = fast_rcp(fmaf(0.6f, x, 1.0f));
  gauss = kTailScale * fast_exp2(fmaf(-kLog2e * x, x, kTailBits));
  // (half the fitted coefficients)
  float p = 0.5f * -0.09208156913518906f;
  p = fmaf(p, t, 0.5f * 0.4119424819946289f);
  p = fmaf(p, t, 0.5f * -0.6444502472877502f);
  p = fmaf(p, t, 0.5f * 0.2837655544281006f);
  p = fmaf(p, t, 0.5f * 0.07341350615024567f);
  p = fmaf(p, t, 0.5f * 0.29160067439079285f);
  p = fmaf(p, t, 0.5f * 0.33724918961524963f);
  p = fmaf(p, t, 0.5f * 0.3385600745677948f);
  const float tail = t * p * gauss;
  return z < 0.0f ? tail : 1.0f - tail;
}

// The logistic, 1 / (1 + 2^(c1 z + c3 z^3)), both terms of the sum times 2^-24.
// At |z| = kLogisticMax it is exactly 0 or 1 in FP32 (the power is infinite or 0), so
// z is clamped there and z^3 stays finite; from z = -104 on it is 0, and z times it
// would be less than a thousandth of the least BF16 number.
constexpr float kLogisticMax = 110.0f;
__device__ __forceinline__ float act_logistic(const ActParams& a, float zc) {
  return kTailScale * fast_rcp(kTailScale + fast_exp2(fmaf(zc, fmaf(a.c3, zc * zc, a.c1), -kTailBits)));
}

__device__ __forceinline__ float act_value(const ActParams& a, float z) {
  if (a.kind == kActLogistic) return z * act_logistic(a, fminf(fmaxf(z, -kLogisticMax), kLogisticMax));
  if (a.kind == kActNormal) {
    float gauss;
    return z * act_normal(z, gauss);
  }
  return max_nan(z, a.lo);
}

// act of a group of values, with one branch.
template <int N>
__device__ __forceinline__ void act_apply(const ActParams& a, float (&v)[N]) {
  if (a.kind == kActLogistic) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= act_logistic(a, fminf(fmaxf(v[i], -kLogisticMax), kLogisticMax));
  } else if (a.kind == kActNormal) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float gauss;
      v[i] *= act_normal(v[i], gauss);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = max_nan(v[i], a.lo);
  }
}

// act(z) and its derivative; relu's is 0 at 0. A NaN stays one in both (relu's
// derivative of it is 1).
__device__ __forceinline__ float act_slope(const ActParams& a, float z, float& value) {
  if (a.kind == kActLogistic) {
    const float zc = -max_nan(-max_nan(z, -kLogisticMax), -kLogisticMax);
    const float s = act_logistic(a, zc);
    value = z * s;
    return fmaf(zc * s * (1.0f - s), (-1.0f / kLog2e) * fmaf(3.0f * a.c3, zc * zc, a.c1), s);
  }
  if (a.kind == kActNormal) {
    float gauss;
    const float cdf = act_normal(z, gauss);
    value = z * cdf;
    return fmaf(z * 0.39894228040143268f, gauss, cdf);
  }
  value = max_nan(z, a.lo);
  return a.lo == 0.0f && z <= 0.0f ? 0.0f : 1.0f;
}

// What a GEMM does with its FP32 sums.
enum Epi : int {
  kEpiPlain = 0,  // y = BF16(sum)
  kEpiFused = 1,  // z = sum + bias; y = BF16(act(z) + residual); z kept if asked
  kEpiGated = 2,  // two weights: h = BF16(act(g) * u); g and u kept if asked
};

// Host-side description of kEpiFused (any pointer may be null).
struct FusedEpi {
  const uint16_t* bias;      // [N], 16-byte aligned
  const uint16_t* residual;  // [M][ldr]; may be y itself
  int64_t ldr;
  uint16_t* preact;  // [M][ldp]
  int64_t ldp;
  ActParams act;
};

// Host-side description of kEpiGated: the up weight beside the gate weight
// that the GEMM takes as its own, and where g and u go (both or neither).
struct GatedEpi {
  const uint8_t* q_up;
  const float* s_up;
  uint16_t* g;
  uint16_t* u;
  int64_t ldgu;
  ActParams act;
};

// Kernel-side parameters.
template <int EPI>
struct EpiParams {};

template <>
struct EpiParams<kEpiFused> {
  // Where the kernel moves rows by TMA: the store map of z and the load map of
  // the residual.
  CUtensorMap tm_pre, tm_res;
  FusedEpi e;
};

template <>
struct EpiParams<kEpiGated> {
  CUtensorMap tm_up;   // codes of the up weight
  CUtensorMap tm_g, tm_u;  // store maps of g and u (as tm_pre)
  GatedEpi e;
};

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}

}  // namespace fp8blk
