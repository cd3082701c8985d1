// mx_kernels.hip -- the microscaled 4-bit format (sq_mx.hpp): quantisation of
// bf16 activations, with the SiLU or GELU before it, quantisation of fp32
// weights, and the values back.
//
// A block's scale is a power of two, so an element times its inverse is exact
// and the only rounding is the conversion's, to nearest even: the codes follow
// from the bf16 values bit for bit.
#include "sq_activation.hpp"
#include "sq_mx.hpp"
#include "sq_pieces.hpp"

namespace sq {

namespace {

struct MxQuantArgs {
  const uint16_t *x;
  int64_t M, ld_x;
  int32_t K;
  MxOut out;
};

// gelu_bf16's E of every bf16 magnitude from 2^-11 to below 16, in LDS.  Below, where
// GELU rounds to z / 2, E of 0 gives that too, and above, E is 0: the result of every
// bf16 value is gelu_bf16's, bit for bit.
constexpr int kGeluFirst = 0x3a00, kGeluCount = 0x4180 - kGeluFirst;

template <int THREADS>
__device__ __forceinline__ void gelu_table(float *table) {
  for (int i = threadIdx.x; i < kGeluCount; i += THREADS)
    table[i] = gelu_bf16_e(i ? __uint_as_float((uint32_t)(kGeluFirst + i) << 16) : 0.0f);
}

// Two values; their places in the table (in bytes) are found in both halves at once.
__device__ __forceinline__ uint32_t gelu_pair(uint32_t z, const float *table) {
  typedef unsigned short v2s __attribute__((ext_vector_type(2)));
  v2s at = __builtin_bit_cast(v2s, z & 0x7fff7fffu);
  at = __builtin_elementwise_sub_sat(at, v2s{kGeluFirst, kGeluFirst});
  at = __builtin_elementwise_min(at, v2s{kGeluCount - 1, kGeluCount - 1}) << 2;
  const uint32_t both = __builtin_bit_cast(uint32_t, at);
  const char *t = reinterpret_cast<const char *>(table);
  const float lo = *reinterpret_cast<const float *>(t + (both & 0xffffu));
  const float hi = *reinterpret_cast<const float *>(t + (both >> 16));
  return cvt_bf16x2(gelu_bf16_of(bf16_lo(z), lo), gelu_bf16_of(bf16_hi(z), hi));
}

// A scale tile, 16 rows x 512 k, to 256 threads: 16 lanes a row, so that a load
// takes 256 neighbouring bytes of each of four rows and the tile's code tiles and its
// 256 bytes of scales are written whole.  4429x1536 5.3 us (3.2 TB/s).  GELU (ACT 2) by
// the table, which two tiles share: computed it took 24 issue slots a value and was
// bound by them, 9216x12288 68 us and 4096x6144 19.7 in a graph; by the table 47
// (6.2 TB/s) and 13.3 (one or four tiles 47 and 49, 14.0 and 14.2).  The smallest
// sizes pay 0.2 us for it.
constexpr int kGeluTiles = 2;

template <int ACT>
__global__ __launch_bounds__(ACT == 2 ? 256 * kGeluTiles : 256) void mx_quantize_kernel(
    MxQuantArgs a) {
  constexpr int TILES = ACT == 2 ? kGeluTiles : 1;
  __shared__ float table[ACT == 2 ? kGeluCount : 1];
  const int lane = threadIdx.x & 255, j = lane >> 4, col = lane & 15, g = col >> 2, q = col & 3;
  const int64_t tile = (int64_t)blockIdx.y * TILES + (threadIdx.x >> 8), row = tile * 16 + j;
  const int k0 = blockIdx.x * kMxScaleK;
  v4u x[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = k0 + s * kMxTileK + 8 * col;
    x[s] = v4u{0u, 0u, 0u, 0u};
    if (row < a.M && k < a.K) x[s] = *reinterpret_cast<const v4u *>(a.x + row * a.ld_x + k);
  }
  if (ACT == 2) {  // under the loads
    gelu_table<256 * TILES>(table);
    __syncthreads();
    if (tile * 16 >= a.M) return;  // whole waves; no barrier follows
  }
  uint32_t scales = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (k0 + s * kMxTileK >= a.K) break;
    if (ACT == 1) {
      float f[8];
      unpack8(x[s], f);
      silu8_hw(f);
      x[s] = pack8(f);
    }
    if (ACT == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[s][i] = gelu_pair(x[s][i], table);
    }
    uint32_t byte;
    const uint32_t c = mx_piece(x[s], byte);
    uint8_t *t = a.out.codes + ((tile * a.out.kt + (k0 >> 7) + s) << 10);
    *reinterpret_cast<uint32_t *>(t + ((g << 4 | j) << 4) + 4 * q) = c;
    scales |= byte << (8 * s);
  }
  if (q == 0)
    *reinterpret_cast<uint32_t *>(a.out.scales + ((tile * a.out.ks + blockIdx.x) << 8) +
                                  ((g << 4 | j) << 2)) = scales;
}

struct MxWeightArgs {
  const float *w;
  int64_t ld_w;
  int32_t K, N;
  MxOut out;
};

// One thread per block of 32 k of a column; a wave reads 64 columns of a row.
// Columns of W are the rows of the format.  Blocks past K are zeros.
__global__ __launch_bounds__(256) void mx_weight_kernel(MxWeightArgs a) {
  const int n = blockIdx.x * 64 + (threadIdx.x & 63);
  const int kb = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  float f[32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    f[i] = 32 * kb < a.K ? a.w[(int64_t)(32 * kb + i) * a.ld_w + n] : 0.0f;
    top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  }
  const uint32_t byte = mx_scale_byte(top >> 23);
  const float inv = mx_inverse(byte);
  v4u c;
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] *= inv;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = mx_codes8(f + 8 * i);
  if (kb < 4 * a.out.kt) *reinterpret_cast<v4u *>(a.out.codes + mx_code_at(a.out, n, kb)) = c;
  a.out.scales[mx_scale_at(a.out, n, kb)] = (uint8_t)byte;
}

__global__ __launch_bounds__(256) void mx_unpack_kernel(MxOut in, int64_t R, int32_t K, float *x,
                                                        int64_t ld_x) {
  const int64_t blocks = K / 32;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < R * blocks;
       i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / blocks;
    const int kb = (int)(i - row * blocks);
    const v4u c = *reinterpret_cast<const v4u *>(in.codes + mx_code_at(in, row, kb));
    const int byte = in.scales[mx_scale_at(in, row, kb)];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const uint32_t code = c[e >> 3] >> (4 * (e & 7)) & 15u;
      const uint32_t m = code & 7u;
      // 0, 0.5, then 1 + mantissa / 2 times 2^(exponent - 1)
      float v = m < 2 ? 0.5f * (float)m
                      : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
      v = byte == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(v, byte - 127);
      x[row * ld_x + 32 * kb + e] = code & 8u ? -v : v;
    }
  }
}

}  // namespace

hipError_t launch_quantize_mx(const uint16_t *x, int64_t M, int64_t K, int64_t ld_x, int32_t act,
                              uint8_t *codes, uint8_t *scales, hipStream_t s) {
  const MxQuantArgs a{x, M, ld_x, (int32_t)K, {codes, scales, mx_tiles_k(K), mx_scale_tiles_k(K)}};
  // grid.y holds 65535 row tiles; more rows go in further launches
  constexpr int64_t kMost = 65534;
  for (int64_t r = 0; r < M; r += kMost * kMxTileRows) {
    MxQuantArgs p = a;
    const int64_t tiles = mx_row_tiles(M - r) < kMost ? mx_row_tiles(M - r) : kMost;
    p.x += r * ld_x;
    p.M -= r;
    p.out.codes += (r / kMxTileRows * a.out.kt) << 10;
    p.out.scales += (r / kMxTileRows * a.out.ks) << 8;
    const unsigned ks = (unsigned)a.out.ks, all = (unsigned)tiles;
    if (act == 1)
      hipLaunchKernelGGL(mx_quantize_kernel<1>, dim3(ks, all), dim3(256), 0, s, p);
    else if (act == 2)
      hipLaunchKernelGGL(mx_quantize_kernel<2>, dim3(ks, (all + kGeluTiles - 1) / kGeluTiles),
                         dim3(256 * kGeluTiles), 0, s, p);
    else
      hipLaunchKernelGGL(mx_quantize_kernel<0>, dim3(ks, all), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_weight_mx(const float *w, int64_t K, int64_t N, int64_t ld_w,
                                     uint8_t *codes, uint8_t *scales, hipStream_t s) {
  const MxWeightArgs a{w, ld_w, (int32_t)K, (int32_t)N,
                       {codes, scales, mx_tiles_k(K), mx_scale_tiles_k(K)}};
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)(4 * a.out.ks));
  hipLaunchKernelGGL(mx_weight_kernel, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_unpack_mx(const uint8_t *codes, const uint8_t *scales, int64_t R, int64_t K,
                            float *x, int64_t ld_x, hipStream_t s) {
  MxOut in{const_cast<uint8_t *>(codes), const_cast<uint8_t *>(scales), mx_tiles_k(K),
           mx_scale_tiles_k(K)};
  const int64_t groups = (R * (K / 32) + 255) / 256;
  if (groups)
    hipLaunchKernelGGL(mx_unpack_kernel, dim3((unsigned)(groups < 65536 ? groups : 65536)),
                       dim3(256), 0, s, in, R, (int32_t)K, x, ld_x);
  return hipGetLastError();
}

}  // namespace sq
