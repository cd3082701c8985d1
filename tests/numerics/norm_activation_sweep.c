/* Accuracy of the activations of the group norm kernel, on the CPU.
 *
 * Mirrors silu_hw of segmented_dual_scale_amd/csrc/sq_activation.hpp operation
 * by operation in fp32, with the hardware reciprocal and exp2 each off by -1, 0
 * or +1 ulp in every combination, and their results below fp32's normal range
 * flushed.  Every finite bf16 input and 2^20 fp32 inputs in -128 .. 128 are
 * checked against the fp64 definition:
 *   |f32 result - fp64 value| <= 2^-17 |fp64 value| + 2^-140.
 * Exit status 0 when every input is within the bound; prints the largest
 * relative error.  Build: cc -O2 -ffp-contract=off norm_activation_sweep.c -lm
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

static float silu32(float z) {
  const int deep = z < -64.0f;
  const float e = hw(exp2f(fmaf(z, -1.44269504f, deep ? -32.0f : 0.0f)), d_exp);
  return z * hw(1.0f / (1.0f + e), d_rcp) * (deep ? 0x1p-32f : 1.0f);
}

static double silu64(double z) { return z / (1.0 + exp(-z)); }

static double worst, worst_z;

static int check(const char *name, float (*f)(float), double (*ref)(double), double tiny, float z) {
  const double v = ref((double)z), err = fabs((double)f(z) - v);
  if (!(err <= ldexp(fabs(v), -17) + tiny)) {
    printf("%s: z=%.9g value %.9g, fp64 %.9g, outside the bound\n", name, z, f(z), v);
    return 1;
  }
  if (fabs(v) > 1e-36 && err / fabs(v) > worst) {
    worst = err / fabs(v);
    worst_z = z;
  }
  return 0;
}

static int sweep(const char *name, float (*f)(float), double (*ref)(double), double tiny) {
  worst = 0.0;
  for (uint32_t bits = 0; bits < 65536u; ++bits) {
    const float z = from_bits(bits << 16);
    if (isfinite(z) && check(name, f, ref, tiny, z)) return 1;
  }
  for (int i = -(1 << 19); i < 1 << 19; ++i)
    if (check(name, f, ref, tiny, (float)i * 0x1p-12f + (float)(i % 61) * 0x1p-18f)) return 1;
  printf("%s (rcp %+d, exp2 %+d): max relative error 2^%.2f at z=%g\n", name, d_rcp, d_exp,
         log2(worst), worst_z);
  return 0;
}

int main(void) {
  for (d_rcp = -1; d_rcp <= 1; ++d_rcp)
    for (d_exp = -1; d_exp <= 1; ++d_exp)
      if (sweep("silu", silu32, silu64, 0x1p-140)) return 1;
  return 0;
}
