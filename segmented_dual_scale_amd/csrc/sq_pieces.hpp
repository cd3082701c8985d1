// sq_pieces.hpp -- device helpers of the kernels that walk rows of bf16 in
// pieces of 8 elements (16 bytes): norm_kernels.hip, rmsnorm_kernels.hip,
// rotary_kernels.hip, mx_kernels.hip and gemm_mx.hip.
#pragma once

#include <cmath>

#include "sq_rows.hpp"

namespace sq {

// Bf16 outputs above this many bytes are stored past the caches: the 256 MB
// last-level cache could not hold them for their reader, and their lines
// would be written back during the next pass instead.  Group norm
// 1024x1024x128 (268 MB out): 51 + 84 us for the two launches, against 73 +
// 87 us with cached stores, whose write-back the next call's statistics pass
// then waits for.
constexpr int64_t kStreamBytes = 128 << 20;

__device__ __forceinline__ void unpack8(v4u v, float f[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(v[j]);
    f[2 * j + 1] = bf16_hi(v[j]);
  }
}

__device__ __forceinline__ v4u pack8(const float f[8]) {
  v4u v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = cvt_bf16x2(f[2 * j], f[2 * j + 1]);
  return v;
}

// A row's pieces.  TAIL: rows end inside a piece, whose n elements count (the
// code for it is half of a kernel's registers, so it is built apart); without
// TAIL n is 8, or 0 for no piece.  Rows stand a multiple of 8 elements apart,
// so a whole piece may be read in every row but the array's last, which may
// end with the allocation; what the padding holds is not used.
template <bool TAIL>
__device__ __forceinline__ v4u load8(const uint16_t *p, int n, bool last_row) {
  v4u v = {0u, 0u, 0u, 0u};
  if (n >= 8 || (TAIL && n > 0 && !last_row)) return *reinterpret_cast<const v4u *>(p);
  if (!TAIL) return v;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) v[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  return v;
}

// v with the elements from n on zeroed.
template <bool TAIL>
__device__ __forceinline__ v4u keep8(v4u v, int n) {
  if (TAIL) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 2 * j + 1 < n ? v[j] : 2 * j < n ? v[j] & 0xffffu : 0u;
  }
  return v;
}

// The padding is not written: a short piece goes out as 4, 2 and 1 elements.
// stream: past the caches (see kStreamBytes).
template <bool TAIL>
__device__ __forceinline__ void store8(uint16_t *p, v4u v, int n, bool stream) {
  if (n >= 8) {
    if (stream) {
      asm volatile("" ::: "memory");  // between them, or the compiler makes the
      __builtin_nontemporal_store(v, reinterpret_cast<v4u *>(p));  // two stores one
      asm volatile("" ::: "memory");
    } else {
      *reinterpret_cast<v4u *>(p) = v;
    }
  }
  if (!TAIL || n >= 8) return;
  const uint32_t a = n & 4 ? v[2] : v[0], b = n & 4 ? v[3] : v[1];
  if (n & 4) *reinterpret_cast<v2u *>(p) = v2u{v[0], v[1]};
  if (n & 2) *reinterpret_cast<uint32_t *>(p + (n & 4)) = a;
  if (n & 1) p[n & 6] = (uint16_t)(n & 2 ? b : a);
}

template <bool TAIL>
__device__ __forceinline__ void store8(int8_t *p, v2u v, int n) {
  if (n >= 8) *reinterpret_cast<v2u *>(p) = v;
  if (!TAIL || n >= 8) return;
  const uint32_t a = n & 4 ? v[1] : v[0];
  if (n & 4) *reinterpret_cast<uint32_t *>(p) = v[0];
  if (n & 2) *reinterpret_cast<uint16_t *>(p + (n & 4)) = (uint16_t)a;
  if (n & 1) p[n & 6] = (int8_t)(n & 2 ? a >> 16 : a);
}

// 8 fp32 parameters at p (16-byte aligned), dflt where there are none.
template <bool TAIL>
__device__ __forceinline__ void load8f(const float *p, int n, float dflt, float f[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = dflt;
  if (!p) return;
  if (n >= 8) {
    const v4f lo = *reinterpret_cast<const v4f *>(p), hi = *reinterpret_cast<const v4f *>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = lo[j], f[4 + j] = hi[j];
  } else if (TAIL) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) f[j] = p[j];
  }
}

// A row of finite values whose squares overflow is summed once more, its values
// times kSmall: the largest square is then 2^96, and what the sum of those that
// vanish could add is below 2^-63 of it.  1 / sqrt(mean + eps) from the mean of such
// squares; below 2^-126, where the values are near the largest of all, its last bit
// is 2^-21 of it.
constexpr float kSmall = 0x1p-80f;

__device__ __forceinline__ float small_rsq(float mean, float eps) {
  return __builtin_amdgcn_rsqf(mean + eps * kSmall * kSmall) * kSmall;
}

// Inverse scales of the K-segment that holds column k (every boundary is a
// multiple of 64, so an 8-element piece lies in one segment).
__device__ __forceinline__ void seg_scales(const NormOut &o, int64_t k, float &ip, float &in) {
  int seg = 0;
  while (seg + 1 < o.ks.n && k >= 64 * (int64_t)o.ks.end64[seg]) ++seg;
  ip = o.act[2 * o.ks.n + seg];
  in = o.act[3 * o.ks.n + seg];
}

// Bf16 piece x of row `row`, columns k .. k+n-1 -> the outputs asked for.
template <bool TAIL>
__device__ __forceinline__ void emit8(const NormOut &o, int64_t row, int64_t k, int n, v4u x,
                                      float ip, float in) {
  if (o.x) store8<TAIL>(o.x + row * o.ld_x + k, x, n, o.stream);
  if (o.q) {
    int8_t *q = o.q + row * o.ld_q + k;
    if (o.plane_stride) {
      v2u p, m;
      quant8_planes(x, ip, in, p, m);
      store8<TAIL>(q, p, n);
      store8<TAIL>(q + o.plane_stride, m, n);
    } else {
      store8<TAIL>(q, quant8_signed(x, ip, in), n);
    }
  }
}

// Sum over n neighbouring lanes (a power of two up to 64), in each of them.
// Within 16 lanes by data-parallel moves: once the lanes of a quad (of half a
// row) agree, mirroring the half row (the row) pairs a lane with the other.
__device__ __forceinline__ float part_sum(float v, int n) {
#define SQ_DPP(ctrl) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, false))
  if (n > 1) SQ_DPP(0xB1);   // quad_perm [1,0,3,2]
  if (n > 2) SQ_DPP(0x4E);   // quad_perm [2,3,0,1]
  if (n > 4) SQ_DPP(0x141);  // row_half_mirror
  if (n > 8) SQ_DPP(0x140);  // row_mirror
#undef SQ_DPP
  if (n > 16) v += __shfl_xor(v, 16, 64);
  if (n > 32) v += __shfl_xor(v, 32, 64);
  return v;
}

__device__ __forceinline__ float wave_sum(float v) { return part_sum(v, 64); }

// Sum over the TPR threads of a row.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *lds) {
  v = wave_sum(v);
  if (TPR > 64) {
    __syncthreads();  // the last sum's readers are done with lds
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += lds[w];
  }
  return v;
}

}  // namespace sq
