/* Accuracy of the activations of the group norm kernel, on the CPU.
 *
 * Mirrors silu_hw and gelu_hw of segmented_dual_scale_amd/csrc/sq_activation.hpp
 * operation by operation in fp32, with the hardware reciprocal and exp2 each off
 * by -1, 0 or +1 ulp in every combination, and their results below fp32's normal
 * range flushed.  Every finite bf16 input and 2^20 fp32 inputs, in -128 .. 128
 * for SiLU and -16 .. 16 for GELU, are checked against the fp64 definitions:
 *   |f32 result - fp64 value| <= 2^-17 |fp64 value| + 2^-140 (GELU: 2^-125).
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

static float gelu32(float z) {
  const float a = fminf(fabsf(z), 16.0f);
  const float t = hw(1.0f / fmaf(a, 0.35355339f, 1.0f), d_rcp);
  float Q = fmaf(t, -0.26787168f, 1.0716369f);
  Q = fmaf(t, Q, -1.4226438f);
  Q = fmaf(t, Q, 0.48533854f);
  Q = fmaf(t, Q, -0.047347467f);
  Q = fmaf(t, Q, 0.5655435f);
  Q = fmaf(t, Q, 1.441063f);
  Q = fmaf(t, Q, -1.82572f);
  const float p = a * 0.7213475f, r = fmaf(a, 0.7213475f, -p);
  const float E = t * hw(exp2f(fmaf(-p, a, fmaf(-r, a, Q))), d_exp);
  return 0.5f * z * (z < 0.0f ? E : 2.0f - E);
}

static double silu64(double z) { return z / (1.0 + exp(-z)); }
static double gelu64(double z) { return 0.5 * z * erfc(-z / sqrt(2.0)); }

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

static int sweep(const char *name, float (*f)(float), double (*ref)(double), double top,
                 double tiny) {
  worst = 0.0;
  for (uint32_t bits = 0; bits < 65536u; ++bits) {
    const float z = from_bits(bits << 16);
    if (isfinite(z) && check(name, f, ref, tiny, z)) return 1;
  }
  for (int i = -(1 << 19); i < 1 << 19; ++i)
    if (check(name, f, ref, tiny, (float)(top * ((double)i / (1 << 19) + (i % 61) * 0x1p-25)))) return 1;
  printf("%s (rcp %+d, exp2 %+d): max relative error 2^%.2f at z=%g\n", name, d_rcp, d_exp,
         log2(worst), worst_z);
  return 0;
}

int main(void) {
  for (d_rcp = -1; d_rcp <= 1; ++d_rcp)
    for (d_exp = -1; d_exp <= 1; ++d_exp)
      if (sweep("silu", silu32, silu64, 128.0, 0x1p-140) ||
          sweep("gelu", gelu32, gelu64, 16.0, 0x1p-125))
        return 1;
  return 0;
}
