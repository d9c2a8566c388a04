// The element-wise functions that follow a linear's product (bias,
// activation, residual; the gate of a feed-forward block) and the parameters
// that carry them into the GEMM epilogues.
//
// Activations. silu(z) = z s(z) and gelu_tanh(z) = z s(2 sqrt(2/pi) (z +
// 0.044715 z^3)) with the logistic s are one form, z s(c1 z + c3 z^3); relu
// and the identity are max(z, lo) with lo = 0 and -infinity; gelu(z) = z
// Phi(z) with the normal distribution function Phi(z) = erfc(-z/sqrt 2) / 2,
// whose tail keeps its relative accuracy (1 + erf would cancel). So three
// cases cover the five names, chosen by a branch that is uniform over the
// grid. All of it is computed in FP32 from the FP32 product; exp and the
// division use the fast forms, whose error (a few units of 2^-23, growing with
// |z| through the exponent) is far below the BF16 half step 2^-9.
#pragma once

#include <cuda.h>
#include <math.h>
#include <stdint.h>

#include "fp8blk.h"

namespace fp8blk {

enum ActKind : int { kActMax = 0, kActLogistic = 1, kActNormal = 2 };

struct ActParams {
  int kind;
  float c1, c3;  // kActLogistic: z s(c1 z + c3 z^3)
  float lo;      // kActMax: max(z, lo)
};

inline bool valid_activation(int a) { return a >= FP8BLK_ACT_NONE && a <= FP8BLK_ACT_SILU; }

inline ActParams act_params(int a) {
  switch (a) {
    case FP8BLK_ACT_RELU: return {kActMax, 0.0f, 0.0f, 0.0f};
    case FP8BLK_ACT_GELU: return {kActNormal, 0.0f, 0.0f, 0.0f};
    case FP8BLK_ACT_GELU_TANH:  // 2 sqrt(2/pi), and 0.044715 of it
      return {kActLogistic, 1.5957691216057308f, 0.07135481282673f, 0.0f};
    case FP8BLK_ACT_SILU: return {kActLogistic, 1.0f, 0.0f, 0.0f};
  }
  return {kActMax, 0.0f, 0.0f, -INFINITY};
}

// s(c1 z + c3 z^3). Beyond |z| = 100 the logistic is exactly 0 or 1 in FP32
// (exp(100) overflows to infinity), so z is clamped there: z^3 stays finite.
__device__ __forceinline__ float act_logistic(const ActParams& a, float zc) {
  return __fdividef(1.0f, 1.0f + __expf(-zc * fmaf(a.c3, zc * zc, a.c1)));
}

__device__ __forceinline__ float act_value(const ActParams& a, float z) {
  if (a.kind == kActLogistic) return z * act_logistic(a, fminf(fmaxf(z, -100.0f), 100.0f));
  if (a.kind == kActNormal) return 0.5f * z * erfcf(z * -0.70710678118654752f);
  return fmaxf(z, a.lo);
}

// act(z) and its derivative; relu's is 0 at 0.
__device__ __forceinline__ float act_slope(const ActParams& a, float z, float& value) {
  if (a.kind == kActLogistic) {
    const float zc = fminf(fmaxf(z, -100.0f), 100.0f);
    const float s = act_logistic(a, zc);
    value = z * s;
    return fmaf(zc * s * (1.0f - s), fmaf(3.0f * a.c3, zc * zc, a.c1), s);
  }
  if (a.kind == kActNormal) {
    const float cdf = 0.5f * erfcf(z * -0.70710678118654752f);
    value = z * cdf;
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), cdf);
  }
  value = fmaxf(z, a.lo);
  return z > a.lo ? 1.0f : 0.0f;
}

// What a GEMM does with its FP32 sums.
enum Epi : int {
  kEpiPlain = 0,  // y = BF16(sum)
  kEpiFused = 1,  // z = sum + bias; y = BF16(act(z) + residual); z kept if asked
  kEpiGated = 2,  // two weights: h = BF16(act(g) * u); g and u kept if asked
};

// Host-side description of kEpiFused (any pointer may be null).
struct FusedEpi {
  const uint16_t* bias;      // [N]
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
  CUtensorMap tm_pre;  // store map of z (only where the kernel stores by TMA)
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
