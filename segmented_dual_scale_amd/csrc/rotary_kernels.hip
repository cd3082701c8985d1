// rotary_kernels.hip -- what stands between a QKV projection and attention: the
// root-mean-square norm of every head of q and k, then rotary positions of one
// or several axes (text; height and width; time, height and width).
//   t = x gamma / sqrt(mean x^2 + eps)                       (over a head's D)
//   pair i turns by the angle position[axis(i)] * freq[i]:
//   a' = a cos - b sin,  b' = b cos + a sin
//
// Bound by memory: q and k read once and written once.  A wave takes the heads
// of one token, so the token's angles are worked out once, one pair to a lane,
// and shared through LDS.  The angle is reduced in fp64 pairs (the product of
// a position and a frequency, in turns, less its nearest quarter), so positions
// up to 2^31 lose nothing; sine and cosine of what is left, at most pi/4, are
// their Taylor polynomials to x^9 and x^8, off by less than 2^-25.
#include "sq_pieces.hpp"

namespace sq {

namespace {

// cos and sin of position * freq.  The angle in radians and then in turns are
// each kept as a rounded product and what the rounding left.
__device__ __forceinline__ float2 turn(int position, double freq) {
  constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLo = -0x1.6b01ec5417056p-57;  // 1 / (2 pi)
  const double u = (double)position * freq, u_lo = __builtin_fma((double)position, freq, -u);
  const double t = u * kTurn;
  const double t_lo = __builtin_fma(u, kTurn, -t) + __builtin_fma(u, kTurnLo, u_lo * kTurn);
  const double quarter = __builtin_rint(4.0 * t);
  const float x = (float)((t - 0.25 * quarter) + t_lo) * 6.28318530717958647692f;
  const int q = (int)(quarter - 4.0 * __builtin_floor(0.25 * quarter));  // 0..3
  const float z = x * x;
  float s = __builtin_fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
  s = __builtin_fmaf(z, s, 8.3333333e-3f);
  s = __builtin_fmaf(z, s, -1.6666667e-1f);
  s = __builtin_fmaf(z * x, s, x);
  float c = __builtin_fmaf(z, 2.4801587e-5f, -1.3888889e-3f);  // 1/8!, -1/6!
  c = __builtin_fmaf(z, c, 4.1666667e-2f);
  c = __builtin_fmaf(z, c, -0.5f);
  c = __builtin_fmaf(z, c, 1.0f);
  const float cc = q & 1 ? s : c, ss = q & 1 ? c : s;
  return make_float2((q + 1) & 2 ? -cc : cc, q & 2 ? -ss : ss);
}

// LPH lanes share a head, a unit of two 8-element pieces (eight pairs) each:
// neighbouring pieces where pairs are neighbours, else the pieces half a turned
// part apart; behind the R turned elements, neighbouring pieces again.  A wave
// takes U times 64 / LPH heads of its token.
template <int LPH, int U, bool HALVES>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryProblem a) {
  __shared__ float2 angles[4][8 * LPH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kHeads = 64 / LPH;
  const int64_t item = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + wave;
  const int64_t token = item / a.chunks;
  if (token >= a.B * a.L) return;  // whole waves; no barrier follows
  const int chunk = (int)(item - token * a.chunks);
  const int64_t b = token / a.L, l = token - b * a.L;
  const int u = lane % LPH, sub = lane / LPH;
  const int turned = a.R / 16;  // units that turn
  const int lo = u < turned && HALVES ? 8 * u : 16 * u;
  const int hi = u < turned && HALVES ? lo + a.R / 2 : lo + 8;
  const bool has_lo = lo < a.D, has_hi = hi < a.D;
  v4u x[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = (chunk * U + i) * kHeads + sub;
    const RotaryTensor &t = h < a.q.heads ? a.q : a.k;
    const int hh = h < a.q.heads ? h : h - a.q.heads;
    const uint16_t *p = t.in + b * t.in_stride[0] + l * t.in_stride[1] + hh * t.in_stride[2];
    x[i][0] = x[i][1] = v4u{0u, 0u, 0u, 0u};
    if (hh < t.heads && has_lo) x[i][0] = *reinterpret_cast<const v4u *>(p + lo);
    if (hh < t.heads && has_hi) x[i][1] = *reinterpret_cast<const v4u *>(p + hi);
  }
  for (int i = lane; i < a.R / 2; i += 64) {
    int axis = 0;
    while (axis + 1 < a.n_axes && i >= a.axis_end[axis]) ++axis;
    angles[wave][i] = turn(a.positions[b * a.pos_batch + l * a.n_axes + axis], a.freq[i]);
  }
  __builtin_amdgcn_wave_barrier();  // the wave's own LDS accesses keep their order
  float2 cs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    cs[j] = u < turned ? angles[wave][8 * u + j] : make_float2(1.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = (chunk * U + i) * kHeads + sub;
    const RotaryTensor &t = h < a.q.heads ? a.q : a.k;
    const int hh = h < a.q.heads ? h : h - a.q.heads;
    float f[16];
    unpack8(x[i][0], f);
    unpack8(x[i][1], f + 8);
    if (a.norm) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) s = __builtin_fmaf(f[j], f[j], s);
      const float rstd = __builtin_amdgcn_rsqf(part_sum(s, LPH) / (float)a.D + a.eps);
      float g[16];
      load8f<false>(t.gamma ? t.gamma + lo : nullptr, has_lo ? 8 : 0, 1.0f, g);
      load8f<false>(t.gamma ? t.gamma + hi : nullptr, has_hi ? 8 : 0, 1.0f, g + 8);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = f[j] * rstd * g[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float &p = HALVES && u < turned ? f[j] : f[2 * j];
      float &r = HALVES && u < turned ? f[8 + j] : f[2 * j + 1];
      const float pa = p, pb = r;
      p = pa * cs[j].x - pb * cs[j].y;
      r = pb * cs[j].x + pa * cs[j].y;
    }
    if (hh >= t.heads) continue;
    uint16_t *o = t.out + b * t.out_stride[0] + l * t.out_stride[1] + hh * t.out_stride[2];
    if (has_lo) *reinterpret_cast<v4u *>(o + lo) = pack8(f);
    if (has_hi) *reinterpret_cast<v4u *>(o + hi) = pack8(f + 8);
  }
}

template <int LPH, int U>
void launch_rotary_u(const RotaryProblem &p, hipStream_t s) {
  RotaryProblem a = p;
  const int heads = a.q.heads + a.k.heads, per = U * (64 / LPH);
  a.chunks = (heads + per - 1) / per;
  // a grid dimension holds 2^32 threads
  const int64_t blocks = (a.B * a.L * a.chunks + 3) / 4, rows = (blocks + (1 << 20) - 1) >> 20;
  const dim3 grid((unsigned)((blocks + rows - 1) / rows), (unsigned)rows);
  if (a.halves) hipLaunchKernelGGL((rotary_kernel<LPH, U, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((rotary_kernel<LPH, U, false>), grid, dim3(256), 0, s, a);
}

template <int LPH>
void launch_rotary_lph(const RotaryProblem &a, hipStream_t s) {
  const int64_t steps = (a.q.heads + a.k.heads + 64 / LPH - 1) / (64 / LPH);
  // few tokens: more waves rather than more heads a wave
  const int64_t waves = a.B * a.L * steps;
  if (waves <= 4096 || steps == 1) launch_rotary_u<LPH, 1>(a, s);
  else if (steps % 3 == 0) launch_rotary_u<LPH, 3>(a, s);
  else if (steps == 2) launch_rotary_u<LPH, 2>(a, s);
  else launch_rotary_u<LPH, 4>(a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryProblem &a, hipStream_t s) {
  const int units = (a.D + 15) / 16;
  if (units <= 1) launch_rotary_lph<1>(a, s);
  else if (units <= 2) launch_rotary_lph<2>(a, s);
  else if (units <= 4) launch_rotary_lph<4>(a, s);
  else if (units <= 8) launch_rotary_lph<8>(a, s);
  else if (units <= 16) launch_rotary_lph<16>(a, s);
  else launch_rotary_lph<32>(a, s);
  return hipGetLastError();
}

}  // namespace sq
