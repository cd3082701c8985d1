// sq_activation.hpp -- the SiLU and GELU whose outputs the layer quantises
// [P1 DualScale motivation; P2 section 3], shared by the kernels that produce
// the layer's input (act_kernels.hip, norm_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>

namespace sq {

// GELU in its exact form z/2 (1 + erf(z / sqrt 2)), evaluated as
// z/2 erfc(-z / sqrt 2): the same function, but 1 + erf cancels to nothing in
// fp32 for z below about -4 while erfc keeps its relative precision.
// erfc(x), x = |z| / sqrt 2 >= 0, in the form of Numerical Recipes (Press et
// al., "Numerical Recipes in C", 2nd ed., section 6.2): t exp(-x^2 + P(t)),
// t = 1 / (1 + x/2), P a degree-9 Chebyshev fit, relative error below 1.2e-7
// for every x >= 0.  Branch free: erfc(-x) = 2 - erfc(x) gives z >= 0.
// Rounding x itself would cost about 2 x^2 ulps in the tail, so x enters
// only t; -x^2 = -z^2/2 is carried as an exact pair (one product and its FMA
// error), and its product with log2 e is split so that exp2 of the large
// part sees none of the small part's rounding.  With one-ulp reciprocal and
// exp2 the result is within 2^-20 of the true value, relative, over the
// whole bf16 input range (swept on the CPU with those errors injected).
// Large parts below -120 are evaluated 64 binades up and scaled back
// exactly, so results in the subnormal range are not flushed.
__device__ __forceinline__ float gelu_f32(float z) {
  const float kLog2e = 1.44269504f;             // log2 e, rounded to fp32
  const float kLog2eLo = 1.92596303e-08f;       // log2 e - kLog2e
  const float a = fminf(fabsf(z), 20.0f);  // erfc(20 / sqrt 2) underflows: the same result
  const float x = a * 0.70710678f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, x, 1.0f));
  float P = __builtin_fmaf(t, 0.17087277f, -0.82215223f);
  P = __builtin_fmaf(t, P, 1.48851587f);
  P = __builtin_fmaf(t, P, -1.13520398f);
  P = __builtin_fmaf(t, P, 0.27886807f);
  P = __builtin_fmaf(t, P, -0.18628806f);
  P = __builtin_fmaf(t, P, 0.09678418f);
  P = __builtin_fmaf(t, P, 0.37409196f);
  P = __builtin_fmaf(t, P, 1.00002368f);
  P = __builtin_fmaf(t, P, -1.26551223f);
  const float p = a * a, e = __builtin_fmaf(a, a, -p);  // z^2 = p + e exactly
  const float q = -0.5f * p, qe = -0.5f * e;           // -x^2 = q + qe exactly
  const float hi = q * kLog2e;
  float lo = __builtin_fmaf(q, kLog2e, -hi);
  lo = __builtin_fmaf(q, kLog2eLo, lo);
  lo = __builtin_fmaf(qe + P, kLog2e, lo);
  const bool deep = hi < -120.0f;
  const float eh = __builtin_amdgcn_exp2f(deep ? hi + 64.0f : hi) * (deep ? 0x1p-64f : 1.0f);
  const float E = t * eh * __builtin_amdgcn_exp2f(lo);
  return 0.5f * z * (z < 0.0f ? E : 2.0f - E);
}

// SiLU z / (1 + e^-z) as z sigmoid(z), the sigmoid from e^-|z| (library
// expf): e^-z itself overflows for z below about -88.7, where z / (1 + e^-z)
// would give 0 while the true value is still a normal float.
__device__ __forceinline__ float silu_f32(float z) {
  const float ez = expf(-fabsf(z));
  const float r = 1.0f / (1.0f + ez);
  return z * (z >= 0.0f ? r : ez * r);
}

// SiLU z / (1 + e^-z) for a kernel that also normalises, from the hardware's
// one-ulp exp2 and reciprocal: eleven issue slots, where the library expf and
// an IEEE divide would make that kernel compute-bound.  Rounding the product
// z log2 e costs 0.7 |z| 2^-24 of e^-z, so the result is within 2^-18 of the
// true value, relative, down to z = -60 and within 2^-17 to z = -87 (bf16
// rounds at 2^-8); below -88.7, where e^-z overflows, it is -0 for a true
// value smaller than 2^-121.
__device__ __forceinline__ float silu_hw(float z) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// GELU for the same kernels: erfc(x) = t exp(-x^2 + P(t)), t = 1 / (1 + x/2),
// as gelu_f32, but with P of degree 5 (a Chebyshev fit of ln(erfc(x) e^{x^2} /
// t) over 1/7 <= t <= 1, off by 9e-6) and one exp2.  Rounding its argument
// costs up to |z|^2 2^-24 of the result, so it is within 2^-15 of the true
// value, relative, to |z| = 13, where it leaves the normal range.  A third of
// gelu_f32's instructions less: group norm of 64.6 M elements 88 against
// 118 us.
__device__ __forceinline__ float gelu_hw(float z) {
  const float a = fminf(fabsf(z), 16.0f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35355339f, 1.0f));
  float P = __builtin_fmaf(t, 0.227630612f, -0.705695652f);
  P = __builtin_fmaf(t, P, 0.470517736f);
  P = __builtin_fmaf(t, P, 0.256549538f);
  P = __builtin_fmaf(t, P, 1.01750154f);
  P = __builtin_fmaf(t, P, -1.26649683f);
  const float E = t * __builtin_amdgcn_exp2f(__builtin_fmaf(a * -0.5f, a, P) * 1.44269504f);
  return 0.5f * z * (z < 0.0f ? E : 2.0f - E);
}

}  // namespace sq
