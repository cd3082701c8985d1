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
// z log2 e costs up to 2^-18.5 of e^-z, so the result is within 2^-17 of the
// true value, relative, over the whole fp32 range (swept on the CPU with those
// errors injected).  Below z = -64, where e^-z would soon overflow and its
// reciprocal be flushed, it is taken 32 binades down and the result scaled
// back, exactly but for a result in the subnormal range: that is DEEP, which
// gives the same bits for every other z.  Eight values take four slots to look
// whether one of them needs it; DEEP for each costs four an element (group norm
// of 1024x1024x128 to codes: 157 against 150 us).
template <bool DEEP>
__device__ __forceinline__ float silu_hw(float z) {
  const bool deep = DEEP && z < -64.0f;
  const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(z, -1.44269504f, deep ? -32.0f : 0.0f));
  return z * __builtin_amdgcn_rcpf(1.0f + e) * (deep ? 0x1p-32f : 1.0f);
}

__device__ __forceinline__ void silu8_hw(float v[8]) {
  float lowest = v[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) lowest = fminf(lowest, v[j]);
  if (__builtin_expect(__any(lowest < -64.0f), 0)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_hw<true>(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_hw<false>(v[j]);
  }
}

// GELU for the same kernels: erfc(x) = t exp(-x^2 + P(t)), t = 1 / (1 + x/2),
// as gelu_f32, but as one exp2, of -x^2 log2 e + Q(t), Q of degree 7 (fitted to
// log2(erfc(x) e^{x^2} / t) over 0.15 <= t <= 1 for the least largest error,
// off by 1e-6).  x^2 log2 e = z^2 / (2 ln 2) is up to 122 where the result is
// still normal, so its product is carried as a pair and rounded once, with Q:
// 2^-18.5 of the result, which is within 2^-17 of the true value, relative,
// down to 2^-125 (swept on the CPU with the hardware's errors injected).
__device__ __forceinline__ float gelu_hw(float z) {
  const float a = fminf(fabsf(z), 16.0f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.35355339f, 1.0f));
  float Q = __builtin_fmaf(t, -0.26787168f, 1.0716369f);
  Q = __builtin_fmaf(t, Q, -1.4226438f);
  Q = __builtin_fmaf(t, Q, 0.48533854f);
  Q = __builtin_fmaf(t, Q, -0.047347467f);
  Q = __builtin_fmaf(t, Q, 0.5655435f);
  Q = __builtin_fmaf(t, Q, 1.441063f);
  Q = __builtin_fmaf(t, Q, -1.82572f);
  const float p = a * 0.7213475f, r = __builtin_fmaf(a, 0.7213475f, -p);
  const float E = t * __builtin_amdgcn_exp2f(__builtin_fmaf(-p, a, __builtin_fmaf(-r, a, Q)));
  return 0.5f * z * (z < 0.0f ? E : 2.0f - E);
}

}  // namespace sq
