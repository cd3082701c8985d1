// rmsnorm_kernels.hip -- the residual update and root-mean-square norm in front
// of a quantised linear layer, fused with the quantisation:
//   h' = bf16(h + branch),  x = bf16(h' gamma / sqrt(mean h'^2 + eps))
// and x as bf16, as DualScale int8 codes [P2 section 3], as MXFP4, or any of
// them together.
//
// [P2] "SegQuant" (hliangzhao.me).
//
// One row per TPR threads (a wave, or a workgroup of four), NCH 16-byte pieces
// per thread held in registers: read once, squares summed in fp32 from the
// registers, written once.  Bound by memory: two reads and up to three writes
// of a row.  36864x1536 with the residual, to h' and x: 91 us, 5.0 TB/s;
// 4429x1536 with the residual, to h' and MXFP4: 12 us, 3.7 TB/s, a row a wave with
// nothing under its chain of loads, sum and stores.
#include "sq_mx.hpp"
#include "sq_pieces.hpp"

namespace sq {

namespace {

// x of a piece of h', to the outputs.  The lanes of a quad hold a block of
// MXFP4: K is a multiple of 64 there, so they have pieces or have none
// together.
template <bool TAIL>
__device__ __forceinline__ void rms_emit(const RmsNormProblem &a, int64_t r, int64_t k, int n,
                                         v4u h, const float gamma[8], float rstd, float ip,
                                         float in) {
  float f[8];
  unpack8(h, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * gamma[j];
  const v4u x = pack8(f);
  emit8<TAIL>(a.out, r, k, n, x, ip, in);
  if (a.mx.codes) mx_emit8(a.mx, r, (int)k, x);
}

// The last 64 columns of a row's last MXFP4 tile where K ends before them: zeros.
__device__ __forceinline__ void rms_pad(const RmsNormProblem &a, int64_t r, int t) {
  if (!a.mx.codes || a.K % kMxTileK == 0 || t >= 2) return;
  const int kb = (int)(a.K >> 5) + t;
  *reinterpret_cast<v4u *>(a.mx.codes + mx_code_at(a.mx, r, kb)) = v4u{0u, 0u, 0u, 0u};
  a.mx.scales[mx_scale_at(a.mx, r, kb)] = 0;
}

// s and the squares of a piece.  SMALL: of its values times 2^-80.
template <bool SMALL>
__device__ __forceinline__ float add_squares(v4u h, float s) {
  float f[8];
  unpack8(h, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (SMALL) f[j] *= kSmall;
    s = __builtin_fmaf(f[j], f[j], s);
  }
  return s;
}

template <int TPR, int NCH, bool TAIL>
__global__ __launch_bounds__(256) void rmsnorm_kernel(RmsNormProblem a) {
  __shared__ float lds[4];
  const int t = threadIdx.x % TPR;
  const int64_t first = ((int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR) * a.rows_per;
  const int64_t last = min(first + a.rows_per, a.M);
  const float inv_k = 1.0f / (float)a.K;
  // NCH is the piece count of thread 0: only the last piece can be short
  const int n_last = min(8, max(0, (int)a.K - 8 * (t + (NCH - 1) * TPR)));
#define SQ_N(c) ((c) < NCH - 1 ? 8 : n_last)
  constexpr bool kAhead = NCH <= 4;  // beyond, the registers cost more waves than this gains
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
  if (kAhead && first < last) load_row(first);
  float ip[NCH], in[NCH], gamma[kAhead ? NCH : 1][8];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    ip[c] = in[c] = 0.0f;
    if (a.out.q && SQ_N(c) > 0) seg_scales(a.out, 8 * (t + c * TPR), ip[c], in[c]);
    if (kAhead)
      load8f<TAIL>(a.gamma ? a.gamma + 8 * (t + c * TPR) : nullptr, SQ_N(c), 1.0f, gamma[c]);
  }
  for (int64_t r = first; r < last; ++r) {
    if (!kAhead) load_row(r);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      h[c] = next_h[c];
      y[c] = next_y[c];
    }
    if (kAhead && r + 1 < last) load_row(r + 1);
    if (a.branch) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float f[8], b[8];
        unpack8(h[c], f);
        unpack8(y[c], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += b[j];
        h[c] = pack8(f);  // the norm reads the residual stream as it is stored
        if (a.h_out)
          store8<TAIL>(a.h_out + r * a.ld_ho + 8 * (t + c * TPR), h[c], SQ_N(c), a.out.stream);
      }
    }
    if (TAIL) h[NCH - 1] = keep8<TAIL>(h[NCH - 1], n_last);
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) s = add_squares<false>(h[c], s);
    const float mean = row_sum<TPR>(s, lds) * inv_k + a.eps;
    float rstd = __builtin_amdgcn_rsqf(mean);
    if (__builtin_expect(mean == INFINITY, 0)) {  // the same in all threads of the row
      s = 0.0f;
#pragma unroll
      for (int c = 0; c < NCH; ++c) s = add_squares<true>(h[c], s);
      rstd = small_rsq(row_sum<TPR>(s, lds) * inv_k, a.eps);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if (c == NCH - 1 && n_last == 0) continue;
      const int k = 8 * (t + c * TPR);
      if (kAhead) {
        rms_emit<TAIL>(a, r, k, SQ_N(c), h[c], gamma[kAhead ? c : 0], rstd, ip[c], in[c]);
      } else {
        float g[8];
        load8f<TAIL>(a.gamma ? a.gamma + k : nullptr, SQ_N(c), 1.0f, g);
        rms_emit<TAIL>(a, r, k, SQ_N(c), h[c], g, rstd, ip[c], in[c]);
      }
    }
    rms_pad(a, r, t);
  }
#undef SQ_N
}

// Rows longer than the registers take: one workgroup per row, the row read
// twice (the second time from the cache), h' computed in both.
__global__ __launch_bounds__(256) void rmsnorm_long_kernel(RmsNormProblem a) {
  __shared__ float lds[4];
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const uint16_t *h = a.h + r * a.ld_h, *b = a.branch ? a.branch + r * a.ld_b : nullptr;
    auto piece = [&](int64_t k, int n) {
      v4u v = load8<true>(h + k, n, r == a.M - 1);
      if (b) {
        float f[8], y[8];
        unpack8(v, f);
        unpack8(load8<true>(b + k, n, r == a.M - 1), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += y[j];
        v = pack8(f);
      }
      return keep8<true>(v, n);
    };
    float s = 0.0f;
    for (int64_t k = 8 * threadIdx.x; k < a.K; k += 8 * 256)
      s = add_squares<false>(piece(k, (int)min((int64_t)8, a.K - k)), s);
    const float mean = row_sum<256>(s, lds) / (float)a.K + a.eps;
    float rstd = __builtin_amdgcn_rsqf(mean);
    if (mean == INFINITY) {
      s = 0.0f;
      for (int64_t k = 8 * threadIdx.x; k < a.K; k += 8 * 256)
        s = add_squares<true>(piece(k, (int)min((int64_t)8, a.K - k)), s);
      rstd = small_rsq(row_sum<256>(s, lds) / (float)a.K, a.eps);
    }
    for (int64_t k = 8 * threadIdx.x; k < a.K; k += 8 * 256) {
      const int n = (int)min((int64_t)8, a.K - k);
      const v4u v = piece(k, n);  // before h' is stored, which may be where h or branch is
      if (a.h_out) store8<true>(a.h_out + r * a.ld_ho + k, v, n, a.out.stream);
      float ip = 0.0f, in = 0.0f, g[8];
      if (a.out.q) seg_scales(a.out, k, ip, in);
      load8f<true>(a.gamma ? a.gamma + k : nullptr, n, 1.0f, g);
      rms_emit<true>(a, r, k, n, v, g, rstd, ip, in);
    }
    rms_pad(a, r, threadIdx.x);
  }
}

template <int TPR, int NCH>
void launch_rmsnorm_n(const RmsNormProblem &a, hipStream_t s) {
  const int64_t per = a.rows_per * (256 / TPR);
  const dim3 grid((unsigned)((a.M + per - 1) / per));
  if (a.K % 8)
    hipLaunchKernelGGL((rmsnorm_kernel<TPR, NCH, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((rmsnorm_kernel<TPR, NCH, false>), grid, dim3(256), 0, s, a);
}

template <int TPR>
void launch_rmsnorm_t(const RmsNormProblem &a, hipStream_t s) {
  switch (((a.K + 7) / 8 + TPR - 1) / TPR) {
    case 1: return launch_rmsnorm_n<TPR, 1>(a, s);
    case 2: return launch_rmsnorm_n<TPR, 2>(a, s);
    case 3: return launch_rmsnorm_n<TPR, 3>(a, s);
    case 4: return launch_rmsnorm_n<TPR, 4>(a, s);
    case 5: return launch_rmsnorm_n<TPR, 5>(a, s);
    case 6: return launch_rmsnorm_n<TPR, 6>(a, s);
    case 7: return launch_rmsnorm_n<TPR, 7>(a, s);
    default: return launch_rmsnorm_n<TPR, 8>(a, s);
  }
}

}  // namespace

// A wave per row up to 4096 columns (8 pieces per lane), a workgroup per row
// up to 16384; a workgroup too where the rows alone would leave most of the
// 256 CUs without work.
hipError_t launch_rmsnorm(const RmsNormProblem &p, hipStream_t s) {
  RmsNormProblem a = p;
  const int64_t chunks = (a.K + 7) / 8;
  a.out.stream = 2 * a.M * a.K * ((a.out.x != nullptr) + (a.h_out != nullptr)) > kStreamBytes;
  // rows per row group: 8192 waves where that is at most 16 rows; beyond, a
  // grid of at most 2^20 workgroups
  a.rows_per = (a.M + (1 << 20) - 1) >> 20;
  if (a.M > 256 && chunks <= 64 * 8) {
    const int64_t rows = (a.M + 8191) / 8192;
    if (a.rows_per < rows) a.rows_per = rows < 16 ? rows : 16;
    launch_rmsnorm_t<64>(a, s);
  } else if (chunks <= 256 * 8) {
    launch_rmsnorm_t<256>(a, s);
  } else {
    hipLaunchKernelGGL(rmsnorm_long_kernel, dim3((unsigned)(a.M < 65536 ? a.M : 65536)), dim3(256),
                       0, s, a);
  }
  return hipGetLastError();
}

}  // namespace sq
