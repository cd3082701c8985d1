/* Accuracy of the GELU that MXFP4 quantisation applies to bf16 values, on the CPU.
 *
 * Mirrors gelu_bf16 of segmented_dual_scale_amd/csrc/sq_activation.hpp operation
 * by operation in fp32, with the hardware reciprocal and exp2 each off by -1, 0
 * or +1 ulp in every combination, and their results below fp32's normal range
 * flushed.  Every finite bf16 input is checked against the fp64 definition:
 *   |f32 result - fp64 value| <= 2^-17 |fp64 value| + 2^-125.
 * Exit status 0 when every input is within the bound and infinities and NaN give
 * NaN; prints the largest relative error.
 * Build: cc -O2 -ffp-contract=off mx_activation_sweep.c -lm
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static int d_rcp, d_exp;

static float from_bits(uint32_t u) {
  float x;
  memcpy(&x, &u, 4);
  return x;
}

static float hw(float x, int d) { /* a hardware result: x moved by d ulps, flushed */
  uint32_t u;
  memcpy(&u, &x, 4);
  if (x != 0.0f && isfinite(x)) u += (uint32_t)d;
  x = from_bits(u);
  return fabsf(x) < 0x1p-126f ? 0.0f : x;
}

static float gelu32(float z) {
  const float t = hw(1.0f / fmaf(fabsf(z), 0.35355339f, 1.0f), d_rcp);
  float Q = fmaf(t, -0.26787168f, 1.0716369f);
  Q = fmaf(t, Q, -1.4226438f);
  Q = fmaf(t, Q, 0.48533854f);
  Q = fmaf(t, Q, -0.047347467f);
  Q = fmaf(t, Q, 0.5655435f);
  Q = fmaf(t, Q, 1.441063f);
  Q = fmaf(t, Q, -2.82572f);
  const float s = z * z;
  Q = fmaf(s, -9.629815e-9f, Q);
  const float E = t * hw(exp2f(fmaf(s, -0x1.715476p-1f, Q)), d_exp);
  return fmaf(-fabsf(z), E, fmaxf(z, 0.0f));
}

int main(void) {
  for (d_rcp = -1; d_rcp <= 1; ++d_rcp)
    for (d_exp = -1; d_exp <= 1; ++d_exp) {
      double worst = 0.0, worst_z = 0.0;
      for (uint32_t bits = 0; bits < 65536u; ++bits) {
        const float z = from_bits(bits << 16), y = gelu32(z);
        if (!isfinite(z)) {
          if (!isnan(y)) return 1;
          continue;
        }
        const double v = 0.5 * (double)z * erfc(-(double)z / sqrt(2.0)), err = fabs((double)y - v);
        if (!(err <= ldexp(fabs(v), -17) + 0x1p-125)) {
          printf("z=%.9g value %.9g, fp64 %.9g, outside the bound\n", z, y, v);
          return 1;
        }
        if (fabs(v) > 1e-36 && err / fabs(v) > worst) worst = err / fabs(v), worst_z = z;
      }
      printf("gelu (rcp %+d, exp2 %+d): max relative error 2^%.2f at z=%g\n", d_rcp, d_exp,
             log2(worst), worst_z);
    }
  return 0;
}
