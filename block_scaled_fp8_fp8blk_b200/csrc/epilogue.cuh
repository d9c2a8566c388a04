// The element-wise functions that follow a linear's product (bias,
// activation, residual; the gate of a feed-forward block) and the parameters
// that carry them into the GEMM epilogues.
//
// Activations. silu(z) = z s(z) and gelu_tanh(z) = z s(2 sqrt(2/pi) (z +
// 0.044715 z^3)) with the logistic s are one form, z s(c1 z + c3 z^3); relu
// and the identity are max(z, lo) with lo = 0 and -infinity; gelu(z) = z
// Phi(z) with the normal distribution function Phi. So three cases cover the
// five names, chosen by a branch that is uniform over the grid. All of it is
// computed in FP32 from the FP32 product; exp and the division use the fast
// forms, whose error (a few units of 2^-23, growing with |z| through the
// exponent) is far below half a BF16 step.
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

// Phi(z) = 1 - Phi(-z), and for x = |z| / sqrt 2 the tail Phi(-|z|) = erfc(x) / 2
// = erfcx(x) exp(-x^2) / 2, which keeps its relative accuracy where 1 + erf
// would cancel. erfcx(x) is a polynomial in t = 1 / (1 + 0.6 x), fitted to it for
// 0 <= x <= 10 with equal relative error (3.1e-7; 6e-7 in FP32); beyond, exp(-x^2)
// is 0 in FP32.
__device__ __forceinline__ float act_normal(float z) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __fdividef(1.0f, fmaf(0.6f, x, 1.0f));
  float p = -0.09208156913518906f;
  p = fmaf(p, t, 0.4119424819946289f);
  p = fmaf(p, t, -0.6444502472877502f);
  p = fmaf(p, t, 0.2837655544281006f);
  p = fmaf(p, t, 0.07341350615024567f);
  p = fmaf(p, t, 0.29160067439079285f);
  p = fmaf(p, t, 0.33724918961524963f);
  p = fmaf(p, t, 0.3385600745677948f);
  const float tail = 0.5f * t * p * __expf(-x * x);
  return z < 0.0f ? tail : 1.0f - tail;
}

// s(c1 z + c3 z^3). Beyond |z| = 100 the logistic is exactly 0 or 1 in FP32
// (exp(100) overflows to infinity), so z is clamped there: z^3 stays finite.
__device__ __forceinline__ float act_logistic(const ActParams& a, float zc) {
  return __fdividef(1.0f, 1.0f + __expf(-zc * fmaf(a.c3, zc * zc, a.c1)));
}

__device__ __forceinline__ float act_value(const ActParams& a, float z) {
  if (a.kind == kActLogistic) return z * act_logistic(a, fminf(fmaxf(z, -100.0f), 100.0f));
  if (a.kind == kActNormal) return z * act_normal(z);
  return fmaxf(z, a.lo);
}

// act of a group of values, with one branch.
template <int N>
__device__ __forceinline__ void act_apply(const ActParams& a, float (&v)[N]) {
  if (a.kind == kActLogistic) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= act_logistic(a, fminf(fmaxf(v[i], -100.0f), 100.0f));
  } else if (a.kind == kActNormal) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= act_normal(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = fmaxf(v[i], a.lo);
  }
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
    const float cdf = act_normal(z);
    value = z * cdf;
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), cdf);
  }
  value = fmaxf(z, a.lo);
  return z > a.lo ? 1.0f : 0.0f;
}

// Eight BF16 values p[0..8) of a row of which n (possibly <= 0, possibly more
// than 8) exist, as four words; missing ones are 0. p is 16-byte aligned.
__device__ __forceinline__ uint4 load_bf16x8(const uint16_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const uint4*>(p);
  uint64_t lo = 0, hi = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const uint64_t v = static_cast<uint64_t>(p[i]) << (16 * (i & 3));
    if (i < 4) lo |= v; else hi |= v;
  }
  return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                    static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32));
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
