// norm_kernels.hip -- the normalisations in front of a quantised linear layer,
// fused with the activation, the modulation and the DualScale quantisation:
//   * channels-last group norm with SiLU / GELU (image UNets), and
//   * layer norm modulated by a request's shift and scale, with the gated
//     residual update before it: the AdaNorm block whose conditioning layer
//     emits shift, scale and gate [P2 section 1; P1 "SegLinear", the AdaNorm
//     chunking].
// Both emit the layer's input as bf16 X, as its int8 codes, or both, so the
// normalised X need not return from memory to be quantised.
//
// [P1] "SegQuant: A Semantics-Aware and Generalizable Quantization Framework
//      for Diffusion Models" (papernotes.org notes).
// [P2] "SegQuant" (hliangzhao.me).
//
// Statistics are fp32 and never E[x^2] - E[x]^2: the mean is known, or taken
// over a few values in registers, before squares are summed, and pieces are
// joined as (count, mean, sum of squared deviations).
#include "sq_activation.hpp"
#include "sq_pieces.hpp"

namespace sq {

namespace {

// ------------------------------------------------- modulated layer norm --
// One row per TPR threads (a wave, or a workgroup of four), NCH 16-byte
// pieces per thread held in registers: read once, mean and squared deviations
// from the registers, written once.  A row group walks rows_per consecutive
// rows and keeps the request's shift, scale and gate in registers between
// them.

template <int TPR, int NCH, bool TAIL>
__global__ __launch_bounds__(256) void adanorm_kernel(AdaNormProblem a) {
  __shared__ float lds[4];
  const int t = threadIdx.x % TPR;
  const int64_t first =
      ((int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR) * a.rows_per;
  const int64_t last = min(first + a.rows_per, a.M);
  const float inv_k = 1.0f / (float)a.K;
  // NCH is the piece count of thread 0: only the last piece can be short
  const int n_last = min(8, max(0, (int)a.K - 8 * (t + (NCH - 1) * TPR)));
#define SQ_N(c) ((c) < NCH - 1 ? 8 : n_last)
  float ip[NCH], in[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    ip[c] = in[c] = 0.0f;
    if (a.out.q && SQ_N(c) > 0) seg_scales(a.out, 8 * (t + c * TPR), ip[c], in[c]);
  }
  v4u sc[NCH], sh[NCH], ga[NCH];
  // a row's h and branch are loaded while the row before it is worked on, the
  // first row's while its request is looked up
  v4u h[NCH], y[NCH], next_h[NCH], next_y[NCH];
  auto load_row = [&](int64_t r) {
    const bool last_row = r == a.M - 1;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      next_h[c] = load8<TAIL>(a.h + r * a.ld_h + 8 * (t + c * TPR), SQ_N(c), last_row);
      if (a.branch)
        next_y[c] = load8<TAIL>(a.branch + r * a.ld_b + 8 * (t + c * TPR), SQ_N(c), last_row);
    }
  };
  constexpr bool kAhead = NCH <= 4;  // beyond, the registers cost more waves than this gains
  if (kAhead && first < last) load_row(first);
  int64_t until = first;  // sc, sh and ga hold for the rows before this one
  for (int64_t r = first; r < last; ++r) {
    if (!kAhead) load_row(r);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      h[c] = next_h[c];
      y[c] = next_y[c];
    }
    if (kAhead && r + 1 < last) load_row(r + 1);
    if (r >= until) {
      int64_t req;
      if (a.row_offset) {
        const RowRequest f = find_request(a.row_offset, a.n_req, r);
        if (f.req >= a.n_req) break;  // behind the last request: left as it is
        if (f.req < 0) continue;      // before the first one
        req = f.req;
        until = f.end;
      } else {
        req = r / a.rows_per_req;
        until = (req + 1) * a.rows_per_req;
      }
      const bool last_row = req == a.n_req - 1;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int64_t at = req * a.ld_mod + 8 * (t + c * TPR);
        sc[c] = sh[c] = ga[c] = v4u{0u, 0u, 0u, 0u};
        if (a.scale) sc[c] = load8<TAIL>(a.scale + at, SQ_N(c), last_row);
        if (a.shift) sh[c] = load8<TAIL>(a.shift + at, SQ_N(c), last_row);
        if (a.gate) ga[c] = load8<TAIL>(a.gate + at, SQ_N(c), last_row);
      }
    }
    if (a.branch) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float f[8], g[8], b[8];
        unpack8(h[c], f);
        unpack8(ga[c], g);
        unpack8(y[c], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] + (a.gate ? g[j] * b[j] : b[j]);
        h[c] = pack8(f);  // the norm reads the residual stream as it is stored
        if (a.h_out)
          store8<TAIL>(a.h_out + r * a.ld_ho + 8 * (t + c * TPR), h[c], SQ_N(c),
                       a.out.stream);
      }
    }
    h[NCH - 1] = keep8<TAIL>(h[NCH - 1], n_last);
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float f[8];
      unpack8(h[c], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
    }
    const float mean = row_sum<TPR>(s, lds) * inv_k;
    float s2 = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float f[8];
      unpack8(h[c], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float d = f[j] - mean;
        if (c == NCH - 1 && j >= n_last) d = 0.0f;
        s2 = __builtin_fmaf(d, d, s2);
      }
    }
    const float rstd = __builtin_amdgcn_rsqf(row_sum<TPR>(s2, lds) * inv_k + a.eps);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if (c == NCH - 1 && n_last == 0) continue;
      const int k = 8 * (t + c * TPR);
      float f[8], m[8], b[8];
      unpack8(h[c], f);
      if (a.gamma || a.beta) {
        load8f<TAIL>(a.gamma ? a.gamma + k : nullptr, SQ_N(c), 1.0f, m);
        load8f<TAIL>(a.beta ? a.beta + k : nullptr, SQ_N(c), 0.0f, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf((f[j] - mean) * rstd, m[j], b[j]);
        unpack8(sc[c], m);
        unpack8(sh[c], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(f[j], m[j], f[j]) + b[j];
      } else {
        unpack8(sc[c], m);
        unpack8(sh[c], b);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          f[j] = __builtin_fmaf(f[j] - mean, __builtin_fmaf(m[j], rstd, rstd), b[j]);
      }
      emit8<TAIL>(a.out, r, k, SQ_N(c), pack8(f), ip[c], in[c]);
    }
  }
#undef SQ_N
}

// Rows longer than the registers take: one workgroup per row, the row read
// three times (the second and third from the cache).
__global__ __launch_bounds__(256) void adanorm_long_kernel(AdaNormProblem a) {
  __shared__ float lds[4];
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    int64_t req;
    if (a.row_offset) {
      const RowRequest f = find_request(a.row_offset, a.n_req, r);
      if (f.req < 0 || f.req >= a.n_req) continue;
      req = f.req;
    } else {
      req = r / a.rows_per_req;
    }
    const uint16_t *h = a.h + r * a.ld_h;
    const uint16_t *ga = a.gate ? a.gate + req * a.ld_mod : nullptr;
    // h' of piece k, recomputed in each pass
    auto piece = [&](int64_t k, int n, float f[8]) -> v4u {
      v4u v = load8<true>(h + k, n, r == a.M - 1);
      if (a.branch) {
        float g[8], b[8];
        unpack8(v, f);
        unpack8(load8<true>(a.branch + r * a.ld_b + k, n, r == a.M - 1), b);
        if (ga) unpack8(load8<true>(ga + k, n, req == a.n_req - 1), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] + (ga ? g[j] * b[j] : b[j]);
        v = pack8(f);
      }
      v = keep8<true>(v, n);
      unpack8(v, f);
      return v;
    };
    float s = 0.0f, s2 = 0.0f, f[8];
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < a.K; k += 8 * 256) {
      piece(k, (int)min((int64_t)8, a.K - k), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
    }
    const float mean = row_sum<256>(s, lds) / (float)a.K;
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < a.K; k += 8 * 256) {
      const int n = (int)min((int64_t)8, a.K - k);
      piece(k, n, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = j < n ? f[j] - mean : 0.0f;
        s2 = __builtin_fmaf(d, d, s2);
      }
    }
    const float rstd = __builtin_amdgcn_rsqf(row_sum<256>(s2, lds) / (float)a.K + a.eps);
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < a.K; k += 8 * 256) {
      const int n = (int)min((int64_t)8, a.K - k);
      float m[8], b[8], ip = 0.0f, in = 0.0f;
      // each thread reads its piece of h before it writes the same piece of
      // h_out, and no later pass reads either: h_out may be h itself
      const v4u v = piece(k, n, f);
      if (a.branch && a.h_out) store8<true>(a.h_out + r * a.ld_ho + k, v, n, a.out.stream);
      load8f<true>(a.gamma ? a.gamma + k : nullptr, n, 1.0f, m);
      load8f<true>(a.beta ? a.beta + k : nullptr, n, 0.0f, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf((f[j] - mean) * rstd, m[j], b[j]);
      v4u sc = {0u, 0u, 0u, 0u}, sh = sc;
      if (a.scale) sc = load8<true>(a.scale + req * a.ld_mod + k, n, req == a.n_req - 1);
      if (a.shift) sh = load8<true>(a.shift + req * a.ld_mod + k, n, req == a.n_req - 1);
      unpack8(sc, m);
      unpack8(sh, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(f[j], m[j], f[j]) + b[j];
      if (a.out.q) seg_scales(a.out, k, ip, in);
      emit8<true>(a.out, r, k, n, pack8(f), ip, in);
    }
  }
}

// ---------------------------------------------------------- group norm ----
// Channels last: row p of a sample holds its C channels; a group is D = C/G
// neighbouring channels of every row.  A workgroup covers `cb` 16-byte
// columns (8 channels each) of a range of rows; thread t keeps column t % cb
// and walks rows t / cb, + rs, ... so its per-channel values stay in
// registers and consecutive threads read consecutive bytes.
struct GnTile {
  int cb, col, rsub, rs;  // columns; this thread's column, first row; rows per step
  bool active;
  int c0, c1;  // channels of the workgroup's columns
  int g0, ng;  // groups they touch
  int c, nv;   // this thread's first channel and how many of its 8 exist
};

template <int T, bool TAIL>
__device__ __forceinline__ GnTile gn_tile(const GroupNormProblem &a, int c0, int c1) {
  GnTile t;
  t.c0 = c0;
  t.c1 = c1;
  t.cb = (c1 - c0 + 7) / 8;
  t.rs = div24(T, t.cb);
  t.rsub = div24(threadIdx.x, t.cb);
  t.col = threadIdx.x - t.rsub * t.cb;
  t.active = t.rsub < t.rs;
  t.g0 = div24(c0, a.D);
  t.ng = div24(c1 - 1, a.D) - t.g0 + 1;
  t.c = c0 + 8 * t.col;
  t.nv = TAIL ? min(8, c1 - t.c) : 8;
  return t;
}

// How the threads of a workgroup share out the groups of its columns: n
// neighbouring threads (a power of two) per group, as many as there are, so
// each looks at about eight of the workgroup's 8T per-channel values.
template <int T>
struct GroupShare {
  int n, log2n;  // threads per group
  int first;     // this thread's place among them
  int step;      // groups handled at a time
  __device__ explicit GroupShare(int ng) {
    log2n = 0;
    while ((ng << (log2n + 1)) <= T) ++log2n;
    n = 1 << log2n;
    first = threadIdx.x & (n - 1);
    step = T >> log2n;
  }
  // Sum over the n threads, in each of them.  Above a wave (then there is one
  // step) every thread of the workgroup has to call it.
  __device__ __forceinline__ float total(float v, float *waves) const {
    if (n <= 64) return part_sum(v, n);
    v = part_sum(v, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
    const int w0 = (threadIdx.x & ~(n - 1)) >> 6;
    for (int w = 0; w < n / 64; ++w) v += waves[w0 + w];
    return v;
  }
};

// Calls f(row step, LDS index) for this thread's share of a group's values,
// which stand at row step r and channel c of [rs][8 cb].
template <int T, class F>
__device__ __forceinline__ void each_value(const GnTile &t, const GroupShare<T> &sh, int g, int D,
                                           F f) {
  const int lo = max((t.g0 + g) * D, t.c0) - t.c0;
  const int d = min((t.g0 + g + 1) * D, t.c1) - t.c0 - lo;
  const int dr = div24(sh.n, d), dc = sh.n - dr * d;
  int r = div24(sh.first, d), c = sh.first - r * d;
  while (r < t.rs) {
    f(r, r * 8 * t.cb + lo + c);
    r += dr;
    c += dc;
    if (c >= d) {
      c -= d;
      ++r;
    }
  }
}

// Group (less t.g0) of each of this thread's 8 channels; past the last
// channel, the last group.
__device__ __forceinline__ void gn_groups(const GnTile &t, int D, int g[8]) {
  int at = div24(t.c, D), left = (at + 1) * D - t.c;
  at -= t.g0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] = min(at, t.ng - 1);
    if (--left == 0) {
      ++at;
      left = D;
    }
  }
}

// Sums of v over every group of the workgroup's columns, in a fixed order, to
// gs[group - g0].  buf: 8T floats, waves: T/64.
template <int T>
__device__ __forceinline__ void group_sum(const float v[8], const GnTile &t, float *buf,
                                          float *waves, float *gs, int D) {
  if (t.active) {
    v4f *p = reinterpret_cast<v4f *>(buf + threadIdx.x * 8);
    p[0] = v4f{v[0], v[1], v[2], v[3]};
    p[1] = v4f{v[4], v[5], v[6], v[7]};
  }
  __syncthreads();
  const GroupShare<T> sh(t.ng);
  for (int g0 = 0; g0 < t.ng; g0 += sh.step) {
    const int g = g0 + (threadIdx.x >> sh.log2n);
    float s = 0.0f;
    if (g < t.ng) each_value<T>(t, sh, g, D, [&](int, int at) { s += buf[at]; });
    s = sh.total(s, waves);
    if (g < t.ng && sh.first == 0) gs[g] = s;
  }
  __syncthreads();
}

// This thread's per-channel normalisation t = (z - mu) a + b.  a starts as the
// weight and b as the bias, the sample's modulation folded into both: loaded
// while the statistics are on their way, a then gets 1/sqrt(var + eps).
struct GnAffine {
  float mu[8], a[8], b[8];

  template <bool TAIL>
  __device__ __forceinline__ void load(const GroupNormProblem &p, const GnTile &t,
                                       int64_t sample) {
    float m[8];
    load8f<TAIL>(p.gamma ? p.gamma + t.c : nullptr, t.nv, 1.0f, a);
    load8f<TAIL>(p.beta ? p.beta + t.c : nullptr, t.nv, 0.0f, b);
    if (p.scale) {
      unpack8(load8<TAIL>(p.scale + sample * p.ld_mod + t.c, t.nv, sample == p.B - 1), m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = __builtin_fmaf(a[j], m[j], a[j]);
        b[j] = __builtin_fmaf(b[j], m[j], b[j]);
      }
    }
    if (p.shift) {
      unpack8(load8<TAIL>(p.shift + sample * p.ld_mod + t.c, t.nv, sample == p.B - 1), m);
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] += m[j];
    }
  }
};

template <int ACT>
__device__ __forceinline__ v4u gn_apply8(v4u z, const GnAffine &f) {
  float v[8];
  unpack8(z, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = __builtin_fmaf(v[j] - f.mu[j], f.a[j], f.b[j]);
    if (ACT == 2) v[j] = gelu_hw(v[j]);
  }
  if (ACT == 1) silu8_hw(v);
  return pack8(v);
}

// A group's whole slice of a sample in one workgroup's registers (U pieces
// per thread): one launch, one read, one write.
template <int T, int U, int ACT, bool TAIL>
__global__ __launch_bounds__(T) void groupnorm_one_kernel(GroupNormProblem a) {
  extern __shared__ float smem[];
  const int64_t sample = blockIdx.y;
  const int c0 = blockIdx.x * a.groups_per_block * a.D;
  const GnTile t = gn_tile<T, TAIL>(a, c0, min(c0 + a.groups_per_block * a.D, a.C));
  float *buf = smem, *waves = buf + 8 * T, *gs = waves + T / 64;
  const int64_t row0 = sample * a.P;
  v4u z[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = t.rsub + u * t.rs;
    z[u] = v4u{0u, 0u, 0u, 0u};
    if (t.active && p < a.P)
      z[u] = load8<TAIL>(a.z + (row0 + p) * a.ld_z + t.c, t.nv, row0 + p == a.B * a.P - 1);
  }
  GnAffine af;
  if (t.active) af.load<TAIL>(a, t, sample);
  float s[8], f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    unpack8(z[u], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += f[j];
  }
  const float inv_n = 1.0f / ((float)a.P * (float)a.D);
  int g[8];
  gn_groups(t, a.D, g);
  group_sum<T>(s, t, buf, waves, gs, a.D);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    af.mu[j] = gs[g[j]] * inv_n;
    s[j] = 0.0f;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool in = t.active && t.rsub + u * t.rs < a.P;
    unpack8(z[u], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = in && j < t.nv ? f[j] - af.mu[j] : 0.0f;
      s[j] = __builtin_fmaf(d, d, s[j]);
    }
  }
  group_sum<T>(s, t, buf, waves, gs, a.D);
  if (!t.active) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) af.a[j] *= __builtin_amdgcn_rsqf(gs[g[j]] * inv_n + a.eps);
  float ip = 0.0f, in = 0.0f;
  if (a.out.q) seg_scales(a.out, t.c, ip, in);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int p = t.rsub + u * t.rs;
    if (p < a.P) emit8<TAIL>(a.out, row0 + p, t.c, t.nv, gn_apply8<ACT>(z[u], af), ip, in);
  }
}

// Pieces of one workgroup's statistics: rows of block i of a sample, and the
// channels of group g in its columns.
__device__ __forceinline__ int gn_rows(const GroupNormProblem &a, int blk) {
  return (int)min((int64_t)a.rows_per_block, a.P - (int64_t)blk * a.rows_per_block);
}

__device__ __forceinline__ int gn_chans(const GroupNormProblem &a, int g, int colblk) {
  const int lo = max(g * a.D, colblk * a.cols_per_block);
  const int hi = min((g + 1) * a.D, min((colblk + 1) * a.cols_per_block, a.C));
  return max(0, hi - lo);
}

// nb <= U more values of 8 channels to the running mean and squared
// deviations of cnt values: their own mean and deviations from registers,
// then the pairs joined (Chan, Golub, LeVeque 1979).
template <int U>
__device__ __forceinline__ void add_rows(const v4u v[U], int nb, float mean[8], float m2[8],
                                         float &cnt) {
  const float n = (float)nb, inv = 1.0f / n, w = n / (cnt + n), cw = cnt * w;
  float s[8], f[8], q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = q[j] = 0.0f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= nb) break;
    unpack8(v[u], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] += f[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] *= inv;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= nb) break;
    unpack8(v[u], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = f[j] - s[j];
      q[j] = __builtin_fmaf(d, d, q[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = s[j] - mean[j];
    mean[j] = __builtin_fmaf(d, w, mean[j]);
    m2[j] += __builtin_fmaf(d * d, cw, q[j]);
  }
  cnt += n;
}

// Launch 1 of 2: mean and squared deviations of every group over one block of
// rows (and columns), to a.part[sample][column block][row block][group].
template <int T, bool TAIL>
__global__ __launch_bounds__(T) void groupnorm_stats_kernel(GroupNormProblem a) {
  constexpr int U = 8;
  extern __shared__ float smem[];
  const int blk = blockIdx.x, colblk = blockIdx.y;
  const int64_t sample = blockIdx.z;
  const int c0 = colblk * a.cols_per_block;
  const GnTile t = gn_tile<T, TAIL>(a, c0, min(c0 + a.cols_per_block, a.C));
  float2 *buf = reinterpret_cast<float2 *>(smem);  // [T][8] mean, squared deviations
  float *waves = smem + 16 * T, *counts = waves + T / 64;  // [rs]: rows of a row step
  const int64_t p0 = (int64_t)blk * a.rows_per_block;
  const int rows = gn_rows(a, blk);
  const int64_t row0 = sample * a.P + p0;
  auto load_z = [&](int p) {  // past the block: its last row again
    p = min(p, rows - 1);
    return load8<TAIL>(a.z + (row0 + p) * a.ld_z + t.c, t.nv, row0 + p == a.B * a.P - 1);
  };
  float mean[8], m2[8], cnt = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) mean[j] = m2[j] = 0.0f;
  if (t.active) {
    v4u next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = load_z(t.rsub + u * t.rs);
    int p = t.rsub;
    for (; p + (U - 1) * t.rs < rows; p += U * t.rs) {
      v4u v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = next[u];
        if (p + U * t.rs < rows) next[u] = load_z(p + (U + u) * t.rs);
      }
      add_rows<U>(v, U, mean, m2, cnt);
    }
    if (p < rows) add_rows<U>(next, (rows - p + t.rs - 1) / t.rs, mean, m2, cnt);
  }
  if (t.active) {
    v4f *p = reinterpret_cast<v4f *>(buf + threadIdx.x * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      p[j] = v4f{mean[2 * j], m2[2 * j], mean[2 * j + 1], m2[2 * j + 1]};
    if (t.col == 0) counts[t.rsub] = cnt;
  }
  __syncthreads();
  float2 *part = reinterpret_cast<float2 *>(a.part) +
                 ((sample * gridDim.y + colblk) * a.n_row_blocks + blk) * a.G + t.g0;
  const GroupShare<T> sh(t.ng);
  for (int g0 = 0; g0 < t.ng; g0 += sh.step) {
    const int g = g0 + (threadIdx.x >> sh.log2n);
    float s = 0.0f;
    if (g < t.ng)
      each_value<T>(t, sh, g, a.D, [&](int r, int at) { s = __builtin_fmaf(counts[r], buf[at].x, s); });
    const float mu = sh.total(s, waves) / ((float)rows * (float)gn_chans(a, t.g0 + g, colblk));
    s = 0.0f;
    if (g < t.ng)
      each_value<T>(t, sh, g, a.D, [&](int r, int at) {
        const float2 v = buf[at];
        const float d = v.x - mu;
        s += __builtin_fmaf(d * d, counts[r], v.y);
      });
    s = sh.total(s, waves);
    if (g < t.ng && sh.first == 0) part[g] = make_float2(mu, s);
  }
}

// Launch 2 of 2: join the blocks' statistics, normalise, activate, store.
// The blocks are joined around one block's mean p: with n_i values of mean
// m_i, S1 = sum n_i (m_i - p) and S2 = sum M2_i + n_i (m_i - p)^2 give mean p +
// S1/N and variance S2/N - (S1/N)^2.  That block, of n_0 values, is part of the
// whole, so (mean - p)^2 <= (N/n_0) variance and the subtraction loses at most
// log2 (N/n_0) bits of fp32.  It is a full one: the first rows, and of the
// group's first two column blocks the one with more of its channels (the first
// may hold a single one), so with 256 blocks a sample N/n_0 <= 2^9.
template <int T, int ACT, bool TAIL>
__global__ __launch_bounds__(T) void groupnorm_apply_kernel(GroupNormProblem a) {
  constexpr int U = 4;
  extern __shared__ float smem[];
  // part `part` of the rows of statistics block blk, the last parts first:
  // they were read last and the cache may still hold them
  const int part_no = a.parts - 1 - (int)(blockIdx.x / a.n_row_blocks);
  const int blk = blockIdx.x - (a.parts - 1 - part_no) * a.n_row_blocks;
  const int colblk = blockIdx.y, ncb = gridDim.y;
  const int64_t sample = blockIdx.z;
  const int c0 = colblk * a.cols_per_block;
  const GnTile t = gn_tile<T, TAIL>(a, c0, min(c0 + a.cols_per_block, a.C));
  const int in_block = part_no * a.rows_per_part;
  const int rows = min(a.rows_per_part, gn_rows(a, blk) - in_block);
  if (rows <= 0) return;
  const int64_t p0 = sample * a.P + (int64_t)blk * a.rows_per_block + in_block;
  auto load_z = [&](int p) {  // past the block: its last row again
    p = min(p, rows - 1);
    return load8<TAIL>(a.z + (p0 + p) * a.ld_z + t.c, t.nv, p0 + p == a.B * a.P - 1);
  };
  v4u z[U];  // the first rows are on their way while the statistics are joined
#pragma unroll
  for (int u = 0; u < U; ++u) z[u] = load_z(t.rsub + u * t.rs);
  GnAffine af;
  if (t.active) af.load<TAIL>(a, t, sample);

  const int width = max(T, 8 * t.cb);  // at most as many groups
  float2 *sums = reinterpret_cast<float2 *>(smem);
  float *mean = smem + 2 * width, *rstd = mean + width;
  const float2 *part =
      reinterpret_cast<const float2 *>(a.part) + sample * ncb * a.n_row_blocks * a.G;
  const float inv_n = 1.0f / ((float)a.P * (float)a.D);
  const int last = a.n_row_blocks - 1;
  const int slices = max(1, div24(T, t.ng));  // threads that share a group, ng apart
  for (int i = threadIdx.x; i < slices * t.ng; i += T) {
    const int slice = div24(i, t.ng), g = i - slice * t.ng + t.g0;
    int cb0 = 0, cb1 = 0;
    if (ncb > 1) {
      cb0 = g * a.D / a.cols_per_block;
      cb1 = ((g + 1) * a.D - 1) / a.cols_per_block;
    }
    const int pb = cb0 + (cb1 > cb0 && gn_chans(a, g, cb0) < gn_chans(a, g, cb0 + 1));
    const float pivot = part[(int64_t)pb * a.n_row_blocks * a.G + g].x;
    float s1 = 0.0f, s2 = 0.0f;
    for (int cb = cb0; cb <= cb1; ++cb) {
      const float chans = (float)gn_chans(a, g, cb);
      const float full = chans * (float)a.rows_per_block, rest = chans * (float)gn_rows(a, last);
      const float2 *q = part + (int64_t)cb * a.n_row_blocks * a.G + g;
#pragma unroll 8
      for (int e = slice; e < a.n_row_blocks; e += slices) {
        const float2 v = q[(int64_t)e * a.G];
        const float cnt = e < last ? full : rest, d = v.x - pivot;
        s1 = __builtin_fmaf(cnt, d, s1);
        s2 += __builtin_fmaf(cnt * d, d, v.y);
      }
    }
    sums[i] = make_float2(s1, s2);
    if (slice == 0) mean[i] = pivot;
  }
  __syncthreads();
  int log2n = 0;  // now n neighbouring threads per group
  while (log2n < 6 && (2 << log2n) <= slices) ++log2n;
  const int n = 1 << log2n, first = threadIdx.x & (n - 1);
  for (int i = threadIdx.x >> log2n; i < t.ng; i += T >> log2n) {
    float s1 = 0.0f, s2 = 0.0f;
    for (int k = first; k < slices; k += n) {
      const float2 v = sums[k * t.ng + i];
      s1 += v.x;
      s2 += v.y;
    }
    s1 = part_sum(s1, n) * inv_n;
    s2 = part_sum(s2, n) * inv_n;
    if (first == 0) {
      mean[i] += s1;
      rstd[i] = __builtin_amdgcn_rsqf(fmaxf(s2 - s1 * s1, 0.0f) + a.eps);
    }
  }
  __syncthreads();
  if (!t.active) return;
  int g[8];
  gn_groups(t, a.D, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    af.mu[j] = mean[g[j]];
    af.a[j] *= rstd[g[j]];
  }
  float ip = 0.0f, in = 0.0f;
  if (a.out.q) seg_scales(a.out, t.c, ip, in);
  for (int p = t.rsub; p < rows; p += U * t.rs) {
    v4u now[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      now[u] = z[u];
      if (p + U * t.rs < rows) z[u] = load_z(p + (U + u) * t.rs);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p + u * t.rs < rows)
        emit8<TAIL>(a.out, p0 + p + u * t.rs, t.c, t.nv, gn_apply8<ACT>(now[u], af), ip, in);
  }
}

}  // namespace

// ------------------------------------------------------------- launches ----
namespace {

template <int TPR, int NCH>
void launch_adanorm_n(const AdaNormProblem &a, hipStream_t s) {
  const int64_t per = a.rows_per * (256 / TPR);
  const dim3 grid((unsigned)((a.M + per - 1) / per));
  if (a.K % 8)
    hipLaunchKernelGGL((adanorm_kernel<TPR, NCH, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((adanorm_kernel<TPR, NCH, false>), grid, dim3(256), 0, s, a);
}

template <int TPR>
void launch_adanorm_t(const AdaNormProblem &a, hipStream_t s) {
  switch (((a.K + 7) / 8 + TPR - 1) / TPR) {
    case 1: return launch_adanorm_n<TPR, 1>(a, s);
    case 2: return launch_adanorm_n<TPR, 2>(a, s);
    case 3: return launch_adanorm_n<TPR, 3>(a, s);
    case 4: return launch_adanorm_n<TPR, 4>(a, s);
    case 5: return launch_adanorm_n<TPR, 5>(a, s);
    case 6: return launch_adanorm_n<TPR, 6>(a, s);
    case 7: return launch_adanorm_n<TPR, 7>(a, s);
    default: return launch_adanorm_n<TPR, 8>(a, s);
  }
}

}  // namespace

// A wave per row up to 4096 columns (8 pieces per lane), a workgroup per row
// up to 16384; a workgroup too where the rows alone would leave most of the
// 256 CUs without work.
hipError_t launch_adanorm(const AdaNormProblem &p, hipStream_t s) {
  AdaNormProblem a = p;
  const int64_t chunks = (a.K + 7) / 8;
  a.out.stream = 2 * a.M * a.K * ((a.out.x != nullptr) + (a.h_out != nullptr)) > kStreamBytes;
  // rows per row group: 8192 waves where that is at most 16 rows; beyond, a
  // grid of at most 2^20 workgroups
  a.rows_per = (a.M + (1 << 20) - 1) >> 20;
  if (a.M > 256 && chunks <= 64 * 8) {
    const int64_t rows = (a.M + 8191) / 8192;
    if (a.rows_per < rows) a.rows_per = rows < 16 ? rows : 16;
    launch_adanorm_t<64>(a, s);
  } else if (chunks <= 256 * 8) {
    launch_adanorm_t<256>(a, s);
  } else {
    hipLaunchKernelGGL(adanorm_long_kernel, dim3((unsigned)(a.M < 65536 ? a.M : 65536)), dim3(256),
                       0, s, a);
  }
  return hipGetLastError();
}

namespace {

constexpr int kGnT = 512;        // threads of the two launches
constexpr int kGnMaxCols = 256;  // 16-byte columns of a workgroup

// Smallest count of neighbouring groups whose channels start on a 16-byte
// column wherever the block stands.
int gn_groups_per_block(int G, int D) {
  int g = 1;
  while (g < G && (g * D) % 8) ++g;
  return g < G ? g : G;
}

// Threads and pieces per thread of the one-launch kernel; u == 0 where a group
// block does not fit its registers.
struct GnOne {
  int t, u;
};

GnOne gn_one(const GroupNormProblem &a, int gpb) {
  const int64_t cb = ((int64_t)gpb * a.D + 7) / 8;
  for (int t = 256; t <= 512; t *= 2) {
    const int64_t most = t == 256 ? 8 : 16;
    if (cb > t) continue;
    const int64_t rs = t / cb, u = (a.P + rs - 1) / rs;
    if (u <= most) return {t, (int)u};
  }
  return {0, 0};
}

void gn_plan(GroupNormProblem &a) {
  a.groups_per_block = gn_groups_per_block(a.G, a.D);
  if (gn_one(a, a.groups_per_block).u) {
    a.n_row_blocks = 0;
    return;
  }
  const int64_t chunks = ((int64_t)a.C + 7) / 8, ncb = (chunks + kGnMaxCols - 1) / kGnMaxCols;
  a.cols_per_block = (int)(8 * ((chunks + ncb - 1) / ncb));
  // statistics: about one workgroup per CU (every workgroup of the second
  // launch reads all blocks of its sample), four rows or more per thread
  const int64_t rs = kGnT / (a.cols_per_block / 8);
  int64_t want = 256 / (a.B * ncb);
  if (want < 1) want = 1;
  int64_t rows = (a.P + want - 1) / want;
  if (rows < 4 * rs) rows = 4 * rs;
  a.rows_per_block = (int)(rows < (1 << 20) ? rows : 1 << 20);
  a.n_row_blocks = (int)((a.P + a.rows_per_block - 1) / a.rows_per_block);
  // apply: 2048 workgroups where that leaves eight rows per thread
  const int64_t rs2 = kGnT / (a.cols_per_block / 8);
  a.parts = 8;
  while (a.parts > 1 && a.rows_per_block < a.parts * 8 * rs2) a.parts /= 2;
  a.rows_per_part = (a.rows_per_block + a.parts - 1) / a.parts;
}

}  // namespace

size_t groupnorm_workspace_bytes(const GroupNormProblem &p) {
  GroupNormProblem a = p;
  gn_plan(a);
  if (!a.n_row_blocks) return 0;
  const int64_t ncb = (a.C + a.cols_per_block - 1) / a.cols_per_block;
  return sizeof(float) * 2 * (size_t)a.B * (size_t)a.n_row_blocks * (size_t)ncb * (size_t)a.G;
}

template <int T, int U, int ACT, bool TAIL>
static void launch_groupnorm_one(const GroupNormProblem &a, hipStream_t s) {
  const int gpb = a.groups_per_block;
  const dim3 grid((unsigned)((a.G + gpb - 1) / gpb), (unsigned)a.B);
  const size_t lds = sizeof(float) * (8 * T + T / 64 + 8 * (size_t)((gpb * a.D + 7) / 8));
  hipLaunchKernelGGL((groupnorm_one_kernel<T, U, ACT, TAIL>), grid, dim3(T), lds, s, a);
}

template <int ACT, bool TAIL>
static void launch_groupnorm_act(const GroupNormProblem &a, hipStream_t s) {
  if (!a.n_row_blocks) {
    const GnOne o = gn_one(a, a.groups_per_block);
    if (o.t == 256 && o.u <= 2) return launch_groupnorm_one<256, 2, ACT, TAIL>(a, s);
    if (o.t == 256 && o.u <= 4) return launch_groupnorm_one<256, 4, ACT, TAIL>(a, s);
    if (o.t == 256) return launch_groupnorm_one<256, 8, ACT, TAIL>(a, s);
    if (o.u <= 8) return launch_groupnorm_one<512, 8, ACT, TAIL>(a, s);
    return launch_groupnorm_one<512, 16, ACT, TAIL>(a, s);
  }
  const unsigned ncb = (unsigned)((a.C + a.cols_per_block - 1) / a.cols_per_block);
  const int width = a.cols_per_block > kGnT ? a.cols_per_block : kGnT;
  hipLaunchKernelGGL((groupnorm_stats_kernel<kGnT, TAIL>),
                     dim3((unsigned)a.n_row_blocks, ncb, (unsigned)a.B), dim3(kGnT),
                     sizeof(float) * (17 * kGnT + kGnT / 64), s, a);
  hipLaunchKernelGGL((groupnorm_apply_kernel<kGnT, ACT, TAIL>),
                     dim3((unsigned)(a.n_row_blocks * a.parts), ncb, (unsigned)a.B),
                     dim3(kGnT), sizeof(float) * 4 * width, s, a);
}

hipError_t launch_groupnorm(const GroupNormProblem &p, hipStream_t s) {
  GroupNormProblem a = p;
  gn_plan(a);
  a.out.stream = 2 * a.B * a.P * a.C > kStreamBytes;
  const bool tail = a.C % 8 != 0;
#define SQ_GN(ACT) tail ? launch_groupnorm_act<ACT, true>(a, s) : launch_groupnorm_act<ACT, false>(a, s)
  if (a.act == 1) SQ_GN(1);
  else if (a.act == 2) SQ_GN(2);
  else SQ_GN(0);
#undef SQ_GN
  return hipGetLastError();
}

}  // namespace sq
