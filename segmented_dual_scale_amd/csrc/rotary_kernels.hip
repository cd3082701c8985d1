// rotary_kernels.hip -- what stands between a QKV projection and attention: the
// root-mean-square norm of every head of q and k, then rotary positions of one
// or several axes (text; height and width; time, height and width).
//   t = x gamma / sqrt(mean x^2 + eps)                       (over a head's D)
//   pair i turns by the angle position[axis(i)] * freq[i]:
//   a' = a cos - b sin,  b' = b cos + a sin
//
// Bound by memory: q and k read once and written once.  A wave takes heads of one
// token, so the token's angles are worked out once, one pair to a lane, and
// shared through LDS.  The angle is reduced in fp64 pairs (the product of
// a position and a frequency, in turns, less its nearest quarter), so positions
// up to 2^31 lose nothing; sine and cosine of what is left, at most pi/4, are
// their Taylor polynomials to x^9 and x^8, off by less than 2^-25.  32760 tokens,
// 12 + 12 heads of 128: 72 to 76 us, 5.3 to 5.6 TB/s; 4429 tokens, 24 + 24 heads of
// 64: 11 to 13 us, 4.3 to 4.9 TB/s.
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
  double quarter = __builtin_rint(4.0 * t);
  double rest = (t - 0.25 * quarter) + t_lo;
  // past 2^40 turns or so what the rounding left is whole quarters itself
  const double more = __builtin_rint(4.0 * rest);
  rest -= 0.25 * more;
  quarter = (quarter - 4.0 * __builtin_floor(0.25 * quarter)) + more;
  const float x = (float)rest * 6.28318530717958647692f;
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
// takes up to U times 64 / LPH heads of q or of k of one token: what depends on the
// token alone (addresses, angles) is uniform or shared, and the weights of the norm
// are multiplied into sine and cosine, four factors a pair, ahead of the heads.
// WHOLE: the units are all there and all turn (R = D = 16 LPH).
template <int LPH, int U, bool HALVES, bool WHOLE>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryProblem a) {
  __shared__ float2 angles[4][8 * LPH];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kHeads = 64 / LPH;
  // uniform, below 2^32
  const uint32_t item = (blockIdx.y * gridDim.x + blockIdx.x) * 4 + wave;
  const uint32_t token = item / (uint32_t)a.chunks;
  if (token >= (uint32_t)(a.B * a.L)) return;  // whole waves; no barrier follows
  const int chunk = (int)(item - token * (uint32_t)a.chunks);
  const uint32_t b = token / (uint32_t)a.L, l = token - b * (uint32_t)a.L;
  const RotaryTensor &t = chunk < a.q_chunks ? a.q : a.k;
  const int h0 = (chunk < a.q_chunks ? chunk : chunk - a.q_chunks) * U * kHeads + lane / LPH;
  const uint16_t *in = t.in + b * t.in_stride[0] + l * t.in_stride[1];
  uint16_t *out = t.out + b * t.out_stride[0] + l * t.out_stride[1];
  const int u = lane % LPH;
  const int R = WHOLE ? 16 * LPH : a.R;
  const bool turns = WHOLE || u < R / 16;
  const int lo = turns && HALVES ? 8 * u : 16 * u, hi = turns && HALVES ? lo + R / 2 : lo + 8;
  const bool has_lo = WHOLE || lo < a.D, has_hi = WHOLE || hi < a.D;
  v4u x[U][2];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = min(h0 + i * kHeads, t.heads - 1);  // past the last head that one again
    const uint16_t *p = in + h * t.in_stride[2];
    if (!WHOLE) x[i][0] = x[i][1] = v4u{0u, 0u, 0u, 0u};
    if (has_lo) x[i][0] = *reinterpret_cast<const v4u *>(p + lo);
    if (has_hi) x[i][1] = *reinterpret_cast<const v4u *>(p + hi);
  }
  float g[16];
  load8f<false>(t.gamma ? t.gamma + lo : nullptr, has_lo ? 8 : 0, 1.0f, g);
  load8f<false>(t.gamma ? t.gamma + hi : nullptr, has_hi ? 8 : 0, 1.0f, g + 8);
  const int32_t *pos = a.positions + b * a.pos_batch + (int64_t)l * a.n_axes;
  for (int i = lane; i < R / 2; i += 64) {
    int axis = 0;
    while (axis + 1 < a.n_axes && i >= a.axis_end[axis]) ++axis;
    angles[wave][i] = turn(pos[axis], a.freq[i]);
  }
  __builtin_amdgcn_wave_barrier();  // the wave's own LDS accesses keep their order
  // element e of the unit turns with its partner: HALVES j and 8 + j, else 2 j and 2 j + 1
  constexpr int A = HALVES ? 1 : 2, B = HALVES ? 8 : 1;
  float ca[8], sb[8], cb[8], sa[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 cs = turns ? angles[wave][8 * u + j] : make_float2(1.0f, 0.0f);
    ca[j] = cs.x * g[A * j];
    sa[j] = cs.y * g[A * j];
    cb[j] = cs.x * g[A * j + B];
    sb[j] = cs.y * g[A * j + B];
  }
  const float inv_d = 1.0f / (float)a.D;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int h = h0 + i * kHeads;
    float f[16];
    unpack8(x[i][0], f);
    unpack8(x[i][1], f + 8);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) s = __builtin_fmaf(f[j], f[j], s);
    const float mean = part_sum(s, LPH) * inv_d + a.eps;
    float rstd = a.norm ? __builtin_amdgcn_rsqf(mean) : 1.0f;
    const bool large = a.norm && mean == INFINITY;
    if (__builtin_expect(__any(large), 0)) {
      s = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float v = f[j] * kSmall;
        s = __builtin_fmaf(v, v, s);
      }
      s = small_rsq(part_sum(s, LPH) * inv_d, a.eps);
      rstd = large ? s : rstd;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] *= rstd;
    float o[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = f[A * j], r = f[A * j + B];
      o[A * j] = __builtin_fmaf(p, ca[j], -(r * sb[j]));
      o[A * j + B] = __builtin_fmaf(r, cb[j], p * sa[j]);
    }
    if (!WHOLE && !turns) {  // not through 0 times a partner that may be infinite
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[A * j] = f[A * j] * ca[j];
        o[A * j + B] = f[A * j + B] * cb[j];
      }
    }
    if (h >= t.heads) continue;
    uint16_t *p = out + h * t.out_stride[2];
    if (has_lo) *reinterpret_cast<v4u *>(p + lo) = pack8(o);
    if (has_hi) *reinterpret_cast<v4u *>(p + hi) = pack8(o + 8);
  }
}

template <int LPH, int U>
void launch_rotary_u(const RotaryProblem &p, hipStream_t s) {
  RotaryProblem a = p;
  constexpr int per = U * (64 / LPH);
  a.q_chunks = (a.q.heads + per - 1) / per;
  a.chunks = a.q_chunks + (a.k.heads + per - 1) / per;
  // a grid dimension holds 2^32 threads
  const int64_t blocks = (a.B * a.L * a.chunks + 3) / 4, rows = (blocks + (1 << 20) - 1) >> 20;
  const dim3 grid((unsigned)((blocks + rows - 1) / rows), (unsigned)rows);
  const bool whole = a.R == a.D && a.D == 16 * LPH;
#define SQ_ROTARY(HALVES, WHOLE) \
  hipLaunchKernelGGL((rotary_kernel<LPH, U, HALVES, WHOLE>), grid, dim3(256), 0, s, a)
  if (a.halves && whole) SQ_ROTARY(true, true);
  else if (a.halves) SQ_ROTARY(true, false);
  else if (whole) SQ_ROTARY(false, true);
  else SQ_ROTARY(false, false);
#undef SQ_ROTARY
}

template <int LPH>
void launch_rotary_lph(const RotaryProblem &a, hipStream_t s) {
  constexpr int per = 64 / LPH;
  const int steps = ((a.q.heads > a.k.heads ? a.q.heads : a.k.heads) + per - 1) / per;
  // few tokens: more waves rather than more heads a wave
  if (steps == 1 || a.B * a.L * steps <= 2048) launch_rotary_u<LPH, 1>(a, s);
  else if (steps % 3 == 0) launch_rotary_u<LPH, 3>(a, s);
  else launch_rotary_u<LPH, 2>(a, s);
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
