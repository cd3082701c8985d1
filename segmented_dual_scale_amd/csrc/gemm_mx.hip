// gemm_mx.hip -- the product of two MXFP4 matrices (sq_mx.hpp):
//   y[m][n] = bf16( sum_b 2^(ex[m][b] + ew[n][b]) sum_{k in b} cx[m][k] cw[n][k] )
// with the scaled 16x16x128 matrix-core instruction, which multiplies four
// blocks of 32 by their two powers of two and adds in fp32.
#include <type_traits>

#include "sq_mx.hpp"
#include "sq_rows.hpp"

namespace sq {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

// The weight is the first operand, so that a lane's four results are
// neighbouring columns of y: lane 16 g + j holds columns 4 g .. 4 g + 3 of row j.
template <int STEP>
__device__ __forceinline__ v4f mx_mfma(v4u w, uint32_t sw, v4u x, uint32_t sx, v4f c) {
  const v8i a = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  const v8i b = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, STEP, (int)sw, STEP,
                                                          (int)sx);
}

struct MxGemmArgs {
  MxGemmProblem p;
  int32_t kt, ks;          // tiles along K of the codes, of the scales
  int32_t mt, nt;          // row tiles of x, of w
  int32_t tiles_m, tiles_n;  // workgroup tiles
};

// Each wave computes (16 RM) x (16 RN) of y, its operands straight from memory.
template <int RM, int RN>
__global__ __launch_bounds__(256) void mx_gemm_kernel(MxGemmArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tm = blockIdx.x % a.tiles_m, tn = blockIdx.x / a.tiles_m;
  const int m0 = (tm * 2 + (wave & 1)) * RM, n0 = (tn * 2 + (wave >> 1)) * RN;
  const uint8_t *xp[RM], *wp[RN], *xs[RM], *ws[RN];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int64_t t = min(m0 + i, a.mt - 1);
    xp[i] = a.p.x + ((t * a.kt) << 10) + 16 * lane;
    xs[i] = a.p.x_scale + ((t * a.ks) << 8) + 4 * lane;
  }
#pragma unroll
  for (int i = 0; i < RN; ++i) {
    const int64_t t = min(n0 + i, a.nt - 1);
    wp[i] = a.p.w + ((t * a.kt) << 10) + 16 * lane;
    ws[i] = a.p.w_scale + ((t * a.ks) << 8) + 4 * lane;
  }
  v4f acc[RM][RN];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < a.ks; ++s) {
    uint32_t sx[RM], sw[RN];
#pragma unroll
    for (int i = 0; i < RM; ++i) sx[i] = *reinterpret_cast<const uint32_t *>(xs[i] + ((int64_t)s << 8));
#pragma unroll
    for (int i = 0; i < RN; ++i) sw[i] = *reinterpret_cast<const uint32_t *>(ws[i] + ((int64_t)s << 8));
    const int steps = min(4, a.kt - 4 * s);
    auto step = [&](auto c) {
      constexpr int STEP = decltype(c)::value;
      if (STEP >= steps) return;
      const int64_t at = (int64_t)(4 * s + STEP) << 10;
      v4u x[RM], w[RN];
#pragma unroll
      for (int i = 0; i < RM; ++i) x[i] = *reinterpret_cast<const v4u *>(xp[i] + at);
#pragma unroll
      for (int i = 0; i < RN; ++i) w[i] = *reinterpret_cast<const v4u *>(wp[i] + at);
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < RN; ++j) acc[i][j] = mx_mfma<STEP>(w[j], sw[j], x[i], sx[i], acc[i][j]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 3>{});
  }
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int64_t m = (int64_t)(m0 + i) * 16 + (lane & 15);
#pragma unroll
    for (int j = 0; j < RN; ++j) {
      const int n = (n0 + j) * 16 + 4 * (lane >> 4);
      if (m < a.p.M && n < a.p.N)
        *reinterpret_cast<v2u *>(a.p.y + m * a.p.ld_y + n) =
            v2u{cvt_bf16x2(acc[i][j][0], acc[i][j][1]), cvt_bf16x2(acc[i][j][2], acc[i][j][3])};
    }
  }
}

}  // namespace

hipError_t launch_gemm_mx(const MxGemmProblem &p, hipStream_t s) {
  MxGemmArgs a{p, (int32_t)mx_tiles_k(p.K), (int32_t)mx_scale_tiles_k(p.K),
               (int32_t)mx_row_tiles(p.M), (int32_t)mx_row_tiles(p.N), 0, 0};
  a.tiles_m = (a.mt + 7) / 8;
  a.tiles_n = (a.nt + 7) / 8;
  hipLaunchKernelGGL((mx_gemm_kernel<4, 4>), dim3((unsigned)(a.tiles_m * (int64_t)a.tiles_n)),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace sq
