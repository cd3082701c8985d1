// gemm_mx.hip -- the product of two MXFP4 matrices (sq_mx.hpp):
//   y[m][n] = bf16( sum_b 2^(ex[m][b] + ew[n][b]) sum_{k in b} cx[m][k] cw[n][k] )
// with the scaled 16x16x128 matrix-core instruction, which multiplies four
// blocks of 32 by their two powers of two and adds in fp32.
//
// On random operands a loop of that instruction alone reaches 6.25 PFLOP/s, its
// power holding the clock down.  The product in a captured graph, by card:
//   8192^3 222 to 230 us (4.9 PFLOP/s), 9216x4608x12288 208 to 220 (4.9), 4096x1536x6144
//   22.3 to 23.5 (3.4), 4429x4608x1536 23.7 to 24.8 (2.6), 4429x1536x1536 10.7 to 11.1 (1.9)
// and one launch at a time in a kernel trace 221, 25.2, 25.0 and 11.7 for the last four.
// The smaller ones are launch, first loads and last stores, about 6 us, and parts of
// a round of workgroups.  On operands of zeros, which leave the clock alone, the
// first two take 170 and 157 us.
#include <cmath>
#include <type_traits>

#include "sq_activation.hpp"
#include "sq_mx.hpp"
#include "sq_pieces.hpp"

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
  int32_t kt, ks;            // tiles along K of the codes, of the scales
  int32_t mt, nt;            // row tiles of x, of w
  int32_t tiles_m, tiles_n;  // workgroup tiles
};

// Workgroup -> tile.  Workgroups go to the 8 XCDs in turn, so each XCD gets a
// contiguous range of tiles, in groups of 8 row tiles, that share x and w in
// its L2.
__device__ __forceinline__ void tile_of(const MxGemmArgs &a, int &tm, int &tn) {
  const int total = a.tiles_m * a.tiles_n, each = total >> 3, rest = total & 7;
  const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
  const int id = xcd * each + min(xcd, rest) + at;
  const int span = 8 * a.tiles_n, first = id / span * 8, rows = min(8, a.tiles_m - first);
  const int in = id - first * a.tiles_n;
  tn = in / rows;
  tm = first + in - tn * rows;
}

// ------------------------------------------------------------- up to 16 rows --
struct MxRowsArgs {
  MxGemmProblem p;
  const uint16_t *z;  // bf16 input (FUSED)
  int64_t ld_z;
  int32_t kt, ks;
  uint32_t per_row;  // e * per_row >> 32 = e / (K / 8) for the e of FUSED, below 2^16
};

// MT tiles of x rows and NT tiles of w columns to a workgroup, whose waves take
// the steps of 128 k in turn and add up through LDS: bound by the weight's bytes
// and, below some megabytes of them, by latency, so a wave has P steps of weights
// in flight before it waits for x.  FUSED (ACT as in mx_kernels.hip): each
// workgroup quantises its rows of z itself, to LDS.  2x9216x1536 behind SiLU 4.4
// us, 1.7 TB/s; 77x4608x1536 7 us, from its codes 4.5.
template <int WAVES, int MT, int NT, bool FUSED, int ACT>
__global__ __launch_bounds__(64 * WAVES) void mx_rows_kernel(MxRowsArgs a) {
  constexpr int P = FUSED && MT > 1 ? 2 : MT == 1 ? 4 : 3;
  extern __shared__ uint8_t smem[];
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int M = (int)a.p.M, K = (int)a.p.K, nt = (int)(a.p.N >> 4), n0 = blockIdx.x * NT;
  const int mt = (M + 15) >> 4, m0 = blockIdx.y * MT;
  const uint8_t *w[NT], *sw[NT], *x[MT], *sx[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = min(n0 + j, nt - 1);
    w[j] = a.p.w + ((t * a.kt) << 10) + 16 * lane;
    sw[j] = a.p.w_scale + ((t * a.ks) << 8) + 4 * lane;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t t = min(m0 + i, mt - 1);
    x[i] = a.p.x + ((t * a.kt) << 10) + 16 * lane;
    sx[i] = a.p.x_scale + ((t * a.ks) << 8) + 4 * lane;
  }
  v4u wt[P][NT], xt[P][MT];
  uint32_t ws[P][NT], xs[P][MT];
  // steps u0, u0 + WAVES, ...; past the last one that again
  auto load = [&](int u0) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int u = min(u0 + p * WAVES, a.kt - 1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        wt[p][j] = *reinterpret_cast<const v4u *>(w[j] + ((int64_t)u << 10));
        ws[p][j] = *reinterpret_cast<const uint32_t *>(sw[j] + ((u >> 2) << 8));
      }
      if (!FUSED) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          xt[p][i] = *reinterpret_cast<const v4u *>(x[i] + ((int64_t)u << 10));
          xs[p][i] = *reinterpret_cast<const uint32_t *>(sx[i] + ((u >> 2) << 8));
        }
      }
    }
  };
  // block kb of the m-th of these rows at 16 (kb rows + m), its scale behind all of them
  const int rows = min(16 * MT, M - 16 * m0);
  uint8_t *const codes = smem, *const scales = smem + (K >> 5) * rows * 16;
  if (FUSED) {
    // 8 values at a time; all of a thread's, up to Z, are asked for before any is waited
    // for, and before the weights: loads come back in order
    constexpr int Z = 4, kThreads = 64 * WAVES;
    const uint32_t per = (uint32_t)K >> 3, all = rows * per;
    const uint16_t *const z = a.z + 16 * m0 * a.ld_z;
    v4u v[Z];
    auto ask = [&](uint32_t first) {
#pragma unroll
      for (int i = 0; i < Z; ++i) {
        const uint32_t e = min(first + i * kThreads, all - 1), m = __umulhi(e, a.per_row);
        v[i] = *reinterpret_cast<const v4u *>(z + m * a.ld_z + 8 * (e - m * per));
      }
    };
    ask(threadIdx.x);
    load(wave);
    for (uint32_t first = threadIdx.x; first < all; first += Z * kThreads) {
      if (first != threadIdx.x) ask(first);
#pragma unroll
      for (int i = 0; i < Z; ++i) {
        const uint32_t e = first + i * kThreads, m = __umulhi(e, a.per_row), k8 = e - m * per;
        if (e >= all) break;
        if (ACT) {
          float f[8];
          unpack8(v[i], f);
          if (ACT == 1) silu8_hw(f);
          if (ACT == 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = gelu_bf16(f[j]);
          }
          v[i] = pack8(f);
        }
        uint32_t byte;
        const uint32_t c = mx_piece(v[i], byte);
        const int at = (k8 >> 2) * rows + m, q = k8 & 3;
        *reinterpret_cast<uint32_t *>(codes + 16 * at + 4 * q) = c;
        if (q == 0) scales[at] = (uint8_t)byte;
      }
    }
    __syncthreads();
  } else {
    load(wave);
  }
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int u0 = wave; u0 < a.kt; u0 += P * WAVES) {
    if (u0 != wave) load(u0);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int u = u0 + p * WAVES;
      if (u >= a.kt) break;
      const int shift = 8 * (u & 3);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        v4u c = xt[p][i];
        uint32_t s = xs[p][i] >> shift;
        if (FUSED) {
          const int kb = 4 * u + g, at = kb * rows + 16 * i + r;
          c = v4u{0u, 0u, 0u, 0u};
          s = 0;
          if (16 * i + r < rows && 32 * kb < K) {
            c = *reinterpret_cast<const v4u *>(codes + 16 * at);
            s = scales[at];
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = mx_mfma<0>(wt[p][j], ws[p][j] >> shift, c, s, acc[i][j]);
      }
    }
  }
  __syncthreads();  // all have read x
  v4f *sums = reinterpret_cast<v4f *>(smem);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[((wave * MT + i) * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int t = wave; t < MT * NT; t += WAVES) {
    v4f y = sums[t * 64 + lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) y += sums[(i * MT * NT + t) * 64 + lane];
    const int64_t m = (int64_t)(m0 + t / NT) * 16 + r;
    const int n = (n0 + t % NT) * 16 + 4 * g;
    if (m < M && n < a.p.N)
      *reinterpret_cast<v2u *>(a.p.y + m * a.p.ld_y + n) =
          v2u{cvt_bf16x2(y[0], y[1]), cvt_bf16x2(y[2], y[3])};
  }
}

// ------------------------------------------------ both operands through LDS --
typedef __attribute__((address_space(3))) void lds_void;

// s_waitcnt: at most N vector-memory operations left (gfx9 encoding: vmcnt in
// bits 3:0 and 15:14).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// 16 bytes a lane, to lds (uniform) + 16 lane
__device__ __forceinline__ void copy16(const uint8_t *p, uint8_t *lds) {
  __builtin_amdgcn_global_load_lds(p, (lds_void *)lds, 16, 0, 0);
}

// 4 bytes a lane, to lds (uniform) + 4 lane
__device__ __forceinline__ void copy4(const uint8_t *p, uint8_t *lds) {
  __builtin_amdgcn_global_load_lds(p, (lds_void *)lds, 4, 0, 0);
}

// No memory access moves across.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void keep_uniform(const uint8_t *&p) { asm("" : "+s"(p)); }

template <int V>
using lc = std::integral_constant<int, V>;

// A workgroup of WM x WN waves owns 16 (WM RM) rows x 16 (WN RN) columns of y, a
// wave RM x RN tiles of it.  K goes in stages of 128 through four LDS buffers,
// filled by 16-byte global->LDS copies; the scales of four stages through SCALES
// more.  While a wave multiplies stage u it reads the operands of stage u + 1, one
// x tile into the registers its last products have just released and one w tile
// into a second set, and copies its part of stage u + 3 into the buffer of stage
// u - 1.  The one barrier of a stage says that stage u + 1 has arrived and that
// all waves have multiplied stage u - 1, and so read it: reads in flight need
// not end before it.
//
// At 9216x4608x12288 the matrix cores are busy in 65 % of the clocks (counters) and the
// clock is held to 1.8 GHz; the LDS's reads take 30 %.  What reads less of it is
// slower: four waves of twice the tile each (8192^3: 268 us against 227), one to a
// SIMD; half of w straight to registers, which both waves of a column then load
// (229 us against 216).
//
// Of two neighbouring w tiles, instruction q takes rows 4 q .. 4 q + 3 and 8 + 4 q
// .. 11 + 4 q of each, so that its results in a lane, with those of the other, are
// 8 neighbouring columns of y.
// The copies bring them into that order: every operand is read from LDS at 16
// bytes a lane.
//
// Scales may stand at any 4 bytes (a slice of a larger buffer).  WIDE: both arrays
// stand at 16, and go in copies of 16 bytes a lane; else in copies of 4 (8192^3 240 us
// against 230, 4429x4608x1536 26.0 against 24.8, 4096x1536x6144 24.7 against 23.2).
template <int RM, int RN, int WM, int WN, int SCALES, bool WIDE>
__global__ __launch_bounds__(64 * WM * WN) void mx_gemm_lds_kernel(MxGemmArgs a) {
  constexpr int kWaves = WM * WN, kXT = WM * RM, kWT = WN * RN, kTiles = kXT + kWT;
  constexpr int kStage = kTiles * 1024, kCopies = (kTiles + kWaves - 1) / kWaves;
  constexpr int kXS = (kXT + 3) / 4, kScaleGroups = kXS + kWT / 4;
  static_assert(RN % 4 == 0 && kXT % 2 == 0, "tiles");
  extern __shared__ uint8_t smem[];
  uint8_t *const scale_lds = smem + 4 * kStage;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wn = wave / WM;
  int tm, tn;
  tile_of(a, tm, tn);
  const int kt = a.kt;

  // this wave's copies: KiB wave, wave + kWaves, ... of a stage, x tiles first; past
  // the last of them that one again (waves that copy less would wait for less).
  // Lane (g, r) of w's KiB 2 t + q brings block g of the row that is row r of
  // instruction q: 8 (r / 4 % 2) + 4 q + r % 4 of tile 2 t + r / 8.
  const uint8_t *src[kCopies];
  uint32_t piece[kCopies];
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int t = min(c * kWaves + wave, kTiles - 1), wt = tn * kWT + ((t - kXT) & ~1);
    if (t < kXT) {
      src[c] = a.p.x + ((int64_t)min(tm * kXT + t, a.mt - 1) * kt << 10);
      piece[c] = lane * 16;
    } else {
      const int first = min(wt, a.nt - 1), mine = min(wt + (r >> 3), a.nt - 1);
      src[c] = a.p.w + ((int64_t)first * kt << 10);
      piece[c] = ((uint32_t)((mine - first) * kt) << 10) +
                 (g * 16 + 2 * (r & 4) + 4 * ((t - kXT) & 1) + (r & 3)) * 16;
    }
  }
  // copy c of the next stage; a uniform pointer moves on, the lane's part stays
  // apart (the empty statement keeps the compiler from adding the two ahead of the
  // loop, into two registers of every lane for each of them)
  auto copy = [&](int c, int buf) {
    const int t = min(c * kWaves + wave, kTiles - 1);
    copy16(src[c] + piece[c], smem + buf * kStage + t * 1024);
    src[c] += 1024;
    keep_uniform(src[c]);
  };
  // scales: 1 KiB of four tiles a copy, in the same orders: its 16 bytes 16 g + r
  auto scale_src = [&](int s, int q, int g, int r) {
    if (q < kXS)
      return a.p.x_scale + (((int64_t)min(tm * kXT + q * 4 + g, a.mt - 1) * a.ks + s) << 8) +
             16 * r;
    return a.p.w_scale +
           (((int64_t)min(tn * kWT + (q - kXS) * 4 + (g & 2) + (r >> 1 & 1), a.nt - 1) * a.ks + s)
            << 8) +
           (r >> 2) * 64 + (r & 1) * 32 + (g & 1) * 16;
  };
  auto copy_scales = [&](int s) {
#pragma unroll
    for (int c = 0; c < (kScaleGroups + kWaves - 1) / kWaves; ++c) {
      const int q = c * kWaves + wave;
      if (q >= kScaleGroups) break;
      uint8_t *const to = scale_lds + (s % SCALES) * kScaleGroups * 1024 + q * 1024;
      if (WIDE) {
        copy16(scale_src(s, q, g, r), to);
      } else {
        // (the empty statement: addresses are worked out anew for each block, or four of
        // them would stay in every lane's registers through the loop)
        int sb = s, qb = q;
        asm("" : "+s"(sb), "+s"(qb));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          copy4(scale_src(sb, qb, i, lane >> 2) + 4 * (lane & 3), to + 256 * i);
      }
    }
  };
  auto x_tile = [&](int buf, int i) {
    return *reinterpret_cast<const v4u *>(smem + buf * kStage + (wm * RM + i) * 1024 + lane * 16);
  };
  auto w_tile = [&](int buf, int j) {
    return *reinterpret_cast<const v4u *>(smem + buf * kStage + (kXT + wn * RN + j) * 1024 +
                                          lane * 16);
  };
  auto x_scale = [&](int s, int i) {
    return *reinterpret_cast<const uint32_t *>(scale_lds + (s % SCALES) * kScaleGroups * 1024 +
                                               (wm * RM + i) * 256 + lane * 4);
  };
  auto w_scale = [&](int s, int j) {
    return *reinterpret_cast<const uint32_t *>(scale_lds + (s % SCALES) * kScaleGroups * 1024 +
                                               (4 * kXS + wn * RN + j) * 256 + lane * 4);
  };

  v4f acc[RM][RN];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v4u x[RM], w[2][RN];
  uint32_t sx[RM], sw[RN];

  copy_scales(0);
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (u < kt) {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy(c, u);
    }
  if (kt >= 3) wait_vm<2 * kCopies>();
  else wait_vm<0>();
  stage_barrier();
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    x[i] = x_tile(0, i);
    sx[i] = x_scale(0, i);
  }
#pragma unroll
  for (int j = 0; j < RN; ++j) {
    w[0][j] = w_tile(0, j);
    sw[j] = w_scale(0, j);
  }

  // stage u = 4 s + T.  WHOLE: stages u + 1 .. u + 3 exist.  At the
  // end of K the operands read for a stage that does not exist are what its buffer
  // holds, and no product takes them.
  auto step = [&](int s, auto t_, auto whole_) {
    constexpr int T = decltype(t_)::value;
    constexpr bool WHOLE = decltype(whole_)::value != 0;
    constexpr int NEXT = (T + 1) & 3, FREE = (T + 3) & 3;
    const int u = 4 * s + T;
    // stage u + 1 has arrived when at most the copies of u + 2 are left
    if (WHOLE || u + 2 < kt) wait_vm<kCopies>();
    else wait_vm<0>();
    stage_barrier();
    // the next block's scales, needed behind the barrier of T = 3, when only the
    // copies of T = 2 may be left.  Into the buffer of this block's they go once all
    // waves have used stage T = 0, and so read them
    if (T == 2 - SCALES && (WHOLE || 4 * s + 4 < kt)) copy_scales(s + 1);
    if (!WHOLE && u + 3 < kt) {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy(c, FREE);
    }
    __builtin_amdgcn_sched_barrier(0);
    uint32_t nw[RN];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
#pragma unroll
      for (int j = 0; j < RN; ++j)
        acc[i][j] = mx_mfma<T>(w[T & 1][j], sw[j], x[i], sx[i], acc[i][j]);
      x[i] = x_tile(NEXT, i);
#pragma unroll
      for (int j = i * RN / RM; j < (i + 1) * RN / RM; ++j) w[(T + 1) & 1][j] = w_tile(NEXT, j);
      if (T == 3) {
        sx[i] = x_scale(s + 1, i);
#pragma unroll
        for (int j = i * RN / RM; j < (i + 1) * RN / RM; ++j) nw[j] = w_scale(s + 1, j);
      }
      if (WHOLE) {
#pragma unroll
        for (int c = i * kCopies / RM; c < (i + 1) * kCopies / RM; ++c) copy(c, FREE);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (T == 3) {
#pragma unroll
      for (int j = 0; j < RN; ++j) sw[j] = nw[j];
    }
  };
  int s = 0;
  for (; 4 * s + 8 <= kt; ++s) {
    step(s, lc<0>{}, lc<1>{});
    step(s, lc<1>{}, lc<1>{});
    step(s, lc<2>{}, lc<1>{});
    step(s, lc<3>{}, lc<1>{});
  }
  for (; 4 * s < kt; ++s) {
    step(s, lc<0>{}, lc<0>{});
    if (4 * s + 1 < kt) step(s, lc<1>{}, lc<0>{});
    if (4 * s + 2 < kt) step(s, lc<2>{}, lc<0>{});
    if (4 * s + 3 < kt) step(s, lc<3>{}, lc<0>{});
  }
  // Lane (g, j) of x tile i has columns 8 g .. 8 g + 7 of every 32 of row j.  Through
  // LDS, a wave's part to itself, eight lanes take a row's 128 bytes, so that stores
  // fill whole cache lines.  Piece c of a row stands at c ^ (row % 8): neither side
  // meets in a bank more than twice.
  static_assert(RN == 4 && 16 * RM * 128 * kWaves <= 4 * kStage, "the results' rows");
  stage_barrier();  // all waves have read the last stage
  uint8_t *const rows = smem + wave * (16 * RM * 128);
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; j += 2) {
      const v4f &lo = acc[i][j], &hi = acc[i][j + 1];
      *reinterpret_cast<v4u *>(rows + (16 * i + r) * 128 + ((2 * j + g) ^ (r & 7)) * 16) =
          v4u{cvt_bf16x2(lo[0], lo[1]), cvt_bf16x2(lo[2], lo[3]), cvt_bf16x2(hi[0], hi[1]),
              cvt_bf16x2(hi[2], hi[3])};
    }
  const int row = lane >> 3, n = (tn * kWT + wn * RN) * 16 + 8 * (lane & 7);
  const int64_t m0 = (int64_t)(tm * kXT + wm * RM) * 16 + row;
  uint16_t *const y = a.p.y + m0 * a.p.ld_y + n;
#pragma unroll
  for (int i = 0; i < 2 * RM; ++i) {
    const v4u v = *reinterpret_cast<const v4u *>(rows + (8 * i + row) * 128 +
                                                 ((lane & 7) ^ (row & 7)) * 16);
    if (m0 + 8 * i < a.p.M && n < a.p.N) *reinterpret_cast<v4u *>(y + 8 * i * a.p.ld_y) = v;
  }
}

}  // namespace

template <int RM, int RN, int WM, int WN, int SCALES>
static hipError_t launch_mx_lds(MxGemmArgs a, hipStream_t s) {
  const bool wide = !((reinterpret_cast<uintptr_t>(a.p.x_scale) |
                       reinterpret_cast<uintptr_t>(a.p.w_scale)) & 15);
  constexpr int kXT = WM * RM, kWT = WN * RN;
  constexpr int kLds = 4096 * (kXT + kWT) + 1024 * SCALES * ((kXT + 3) / 4 + kWT / 4);
  a.tiles_m = (a.mt + kXT - 1) / kXT;
  a.tiles_n = (a.nt + kWT - 1) / kWT;
  const dim3 grid((unsigned)(a.tiles_m * (int64_t)a.tiles_n)), block(64 * WM * WN);
  if (wide)
    hipLaunchKernelGGL((mx_gemm_lds_kernel<RM, RN, WM, WN, SCALES, true>), grid, block, kLds, s, a);
  else
    hipLaunchKernelGGL((mx_gemm_lds_kernel<RM, RN, WM, WN, SCALES, false>), grid, block, kLds, s,
                       a);
  return hipGetLastError();
}

// Time of a product in us by tiles of some shape: workgroups beyond what fits the
// chip at once go in further rounds, each of kt steps and what its start and end
// cost.  step and fixed are fits to measured times from K = 128 to 12288.  A tile
// that is alone on its CU goes in whole rounds; those that share one overlap each
// other's ends, so half of a part counts, and steps are shorter while CUs are free.
struct MxTile {
  int rows, cols;  // in tiles of 16
  int per_cu;
  float step, fixed;
};

static float mx_cost(const MxTile &t, const MxGemmArgs &a) {
  const float tiles = (float)((a.mt + t.rows - 1) / t.rows) * (float)((a.nt + t.cols - 1) / t.cols);
  const float kt = (float)a.kt;
  float rounds = tiles / (256.0f * (float)t.per_cu);
  if (t.per_cu == 1) return ceilf(rounds) * (kt * t.step + t.fixed);
  if (rounds < 1.0f) return kt * t.step * (0.5f + 0.5f * rounds) + t.fixed;
  return 0.5f * (rounds + ceilf(rounds)) * (kt * t.step + t.fixed);
}

// The same by workgroups of 32 x 32 that split K over their waves: 4 KiB a step
// and workgroup from the L2 at 22 TB/s, and a chain of loads for each of a wave's
// steps.
static float mx_rows_cost(const MxGemmArgs &a) {
  const float groups = (float)((a.mt + 1) / 2) * (float)((a.nt + 1) / 2), kt = (float)a.kt;
  return 2.0f + groups * kt * (4096.0f / 22e6f) + 0.25f * kt / (a.kt >= 16 ? 8.0f : 4.0f);
}

// Measured, the chosen one against the next best (us): 9216x4608x12288 224x256 220,
// 256x256 228, 192x256 242; 8192^3 256x256 232, 224x256 244; 4429x4608x1536 128x128
// 24.8, 192x256 25.9; 3000x3200x2560 192x256 18.8, 224x256 20.0; 4096x1536x6144
// 128x256 23.5, 128x128 24.4; 1024x1536x1536 64x128 5.2, split K 5.8, 128x128 6.5;
// 256x1536x6144 split K 6.2, 64x128 10.4.  160x256 was left out: 3000x3200x2560 16.4
// against 17.3 and 2048x4608x1536 12.1 against 12.7 with operands in the caches, but with
// operands from memory, behind the norm and before the rotary positions, the three
// kernels at 4429x4608x1536 took 55.6 us against 51.6 (one card, in turn, six times).
constexpr MxTile kMxTiles[] = {
    {16, 16, 1, 0.78f, 5.5f}, {14, 16, 1, 0.69f, 6.5f}, {12, 16, 1, 0.59f, 5.6f},
    {8, 16, 1, 0.41f, 3.6f},  {8, 8, 2, 0.49f, 3.3f},   {4, 8, 3, 0.47f, 2.6f},
};

template <int WAVES, int MT, int NT>
static hipError_t launch_rows(const MxGemmProblem &p, hipStream_t s) {
  const MxRowsArgs a{p, nullptr, 0, (int32_t)mx_tiles_k(p.K), (int32_t)mx_scale_tiles_k(p.K), 0};
  const int64_t nt = p.N / 16, mt = mx_row_tiles(p.M);
  hipLaunchKernelGGL((mx_rows_kernel<WAVES, MT, NT, false, 0>),
                     dim3((unsigned)((nt + NT - 1) / NT), (unsigned)((mt + MT - 1) / MT)),
                     dim3(64 * WAVES), sizeof(float) * 4 * 64 * MT * NT * WAVES, s, a);
  return hipGetLastError();
}

// Up to 16 rows.  Two column tiles a workgroup where that leaves a workgroup per
// CU; as many waves as leave each two steps of K and the chip about 4096.  The same for
// rows of bf16 and of codes, which so have the same sums: 4x1536x6144 on 16 waves 4.7
// and 3.7 us, on 8 5.4 and 4.3; 1x4096x4096 4.2 and 3.8, 4.2 and 3.8.
static int one_row_tile_waves(const MxGemmProblem &p) {
  const int64_t nt = p.N / 16, kt = mx_tiles_k(p.K);
  return kt >= 32 && nt <= 256 ? 16 : kt >= 16 ? 8 : 4;
}

static hipError_t launch_one_row_tile(const MxGemmProblem &p, hipStream_t s) {
  const int waves = one_row_tile_waves(p);
  if (p.N / 16 >= 512) return waves == 8 ? launch_rows<8, 1, 2>(p, s) : launch_rows<4, 1, 2>(p, s);
  if (waves == 16) return launch_rows<16, 1, 1>(p, s);
  return waves == 8 ? launch_rows<8, 1, 1>(p, s) : launch_rows<4, 1, 1>(p, s);
}

template <int WAVES, int MT, int NT>
static hipError_t launch_fused(const MxRowsArgs &a, int32_t act, hipStream_t s) {
  const int64_t mt = mx_row_tiles(a.p.M), rows = a.p.M < 16 * MT ? a.p.M : 16 * MT;
  const dim3 grid((unsigned)((a.p.N / 16 + NT - 1) / NT), (unsigned)((mt + MT - 1) / MT));
  const dim3 block(64 * WAVES);
  const size_t codes = (size_t)(rows * (a.p.K / 32) * 17);
  size_t lds = sizeof(float) * 4 * 64 * MT * NT * WAVES;
  if (lds < codes) lds = codes;
#define SQ_ROWS(ACT) \
  hipLaunchKernelGGL((mx_rows_kernel<WAVES, MT, NT, true, ACT>), grid, block, lds, s, a)
  if constexpr (MT == 1) {
    if (act == 1) SQ_ROWS(1);
    else if (act == 2) SQ_ROWS(2);
    else SQ_ROWS(0);
  } else {
    SQ_ROWS(0);
  }
#undef SQ_ROWS
  return hipGetLastError();
}

// Workgroups of two row tiles and NT column tiles.
static int64_t mx_groups(int64_t M, int64_t N, int nt) {
  return ((N / 16 + nt - 1) / nt) * ((mx_row_tiles(M) + 1) / 2);
}

// More than 16 rows of bf16 without an activation: each workgroup quantises its 32 rows,
// up to 96 values a thread (K 1536), where one workgroup a CU or fewer do that.  In a
// captured graph against two launches, us, by K:
//                                      512        1024       1536       2048       2560
//   77 rows, N 1536,  72 workgroups  3.7 / 5.1  4.7 / 5.3  5.6 / 5.8  6.5 / 5.9  7.7 / 6.4
//   300,     N 1536, 240             4.5 / 5.3  5.4 / 5.9  6.4 / 6.5  7.9 / 6.9  9.7 / 7.5
//   77,      N 4608, 216             4.4 / 5.2  5.4 / 5.7  6.5 / 6.2  7.8 / 6.5  9.0 / 7.0
//   160,     N 4608, 360             5.8 / 5.6  7.5 / 6.3  9.4 / 7.0  11.5 / 7.3  13.8 / 8.3
// The one cell inside the limit that loses, by 0.2 to 0.3 us, gains 2.5 us from the host, as
// every other does (7.5 against 10.1).  An activation on top costs more than a launch: SiLU
// 77x1536x1536 8.7 against 6.9.
static bool mx_few_rows(int64_t M, int64_t N, int64_t K) {
  return 32 * K <= 96 * 512 && mx_groups(M, N, 4) <= 256;
}

// Up to 16 rows: every workgroup quantises all of z, up to 48 values a thread of 8 waves
// (of 4 up to K = 1920).  In a captured graph, where a second launch costs least, with no
// activation / SiLU / GELU: 4 x 1536 (24 values) 3.8 / 4.6 / 5.3 us against 5.3 / 5.8 /
// 6.3 in two launches, 8 x 1536 (48) 4.6 / 6.1 / 7.6 against 5.4 / 6.2 / 6.2, 16 x 1536
// (96) 5.8 / 8.8 / 11.8 against 5.6 / 6.2 / 6.3 (N = 9216); from the host the
// second launch costs 3 us more.
bool mx_quantises_inside(int64_t M, int64_t K) {
  return M <= 16 && M * K <= 48 * 64 * (mx_tiles_k(K) >= 16 ? 8 : 4);
}

// Two column tiles a workgroup where that leaves a workgroup per CU.
hipError_t launch_gemm_mx_bf16(const MxGemmProblem &p, const uint16_t *z, int64_t ld_z, int32_t act,
                               hipStream_t s) {
  const MxRowsArgs a{p, z, ld_z, (int32_t)mx_tiles_k(p.K), (int32_t)mx_scale_tiles_k(p.K),
                     (uint32_t)((1ll << 32) / (p.K / 8) + 1)};
  if (p.M > 16)
    return mx_groups(p.M, p.N, 2) <= 256 ? launch_fused<8, 2, 2>(a, act, s)
                                         : launch_fused<8, 2, 4>(a, act, s);
  const int waves = one_row_tile_waves(p);
  if (p.N / 16 >= 512)
    return waves == 8 ? launch_fused<8, 1, 2>(a, act, s) : launch_fused<4, 1, 2>(a, act, s);
  if (waves == 16) return launch_fused<16, 1, 1>(a, act, s);
  return waves == 8 ? launch_fused<8, 1, 1>(a, act, s) : launch_fused<4, 1, 1>(a, act, s);
}

static MxGemmArgs mx_args(const MxGemmProblem &p) {
  return {p, (int32_t)mx_tiles_k(p.K), (int32_t)mx_scale_tiles_k(p.K), (int32_t)mx_row_tiles(p.M),
          (int32_t)mx_row_tiles(p.N), 0, 0};
}

int mx_choice(int64_t M, int64_t N, int64_t K) {
  MxGemmProblem p{};
  p.M = M;
  p.N = N;
  p.K = K;
  const MxGemmArgs a = mx_args(p);
  int best = 0;
  for (int i = 1; i < (int)(sizeof kMxTiles / sizeof kMxTiles[0]); ++i)
    if (mx_cost(kMxTiles[i], a) < mx_cost(kMxTiles[best], a)) best = i;
  return mx_rows_cost(a) < mx_cost(kMxTiles[best], a) && a.mt <= 65535 ? -1 : best;
}

bool mx_rows_inside(int64_t M, int64_t N, int64_t K) {
  return M > 16 && mx_few_rows(M, N, K) && mx_choice(M, N, K) < 0;
}

hipError_t launch_gemm_mx(const MxGemmProblem &p, hipStream_t s) {
  if (p.M <= 16) return launch_one_row_tile(p, s);
  const MxGemmArgs a = mx_args(p);
  const int best = mx_choice(p.M, p.N, p.K);
  // eight waves where the product of bf16 input has them, so that both give the same
  // bits (of up to four steps the order is the same); otherwise by time
  if (best < 0)
    return a.kt >= 16 || (a.kt > 4 && mx_few_rows(p.M, p.N, p.K)) ? launch_rows<8, 2, 2>(p, s)
                                                                  : launch_rows<4, 2, 2>(p, s);
  switch (best) {
    case 0: return launch_mx_lds<8, 4, 2, 4, 2>(a, s);
    case 1: return launch_mx_lds<7, 4, 2, 4, 2>(a, s);
    case 2: return launch_mx_lds<6, 4, 2, 4, 2>(a, s);
    case 3: return launch_mx_lds<4, 4, 2, 4, 2>(a, s);
    case 4: return launch_mx_lds<4, 4, 2, 2, 2>(a, s);
    default: return launch_mx_lds<2, 4, 2, 2, 1>(a, s);  // three workgroups' LDS fit a CU
  }
}

}  // namespace sq
