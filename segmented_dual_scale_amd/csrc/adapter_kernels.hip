// adapter_kernels.hip -- low-rank adapters of many requests beside a shared
// linear layer: for row m of a request whose adapter is a, and column n in
// N-segment j (an output-segmented layer [P1 "SegLinear", pattern one] has a
// pair of factors per segment),
//   t[m][j][r] = alpha_a * sum_k x[m][k] A_a[j*rank + r][k]       (shrink)
//   y[m][n]    = bf16( base[m][n] + sum_r t[m][j][r] B_a[n][r] )  (expand)
//
// [P1] "SegQuant: A Semantics-Aware and Generalizable Quantization Framework
//      for Diffusion Models" (papernotes.org notes).
//
// Two launches: every output column needs t over the whole of K, so a grid
// has to end in between.  Rows are cut into tiles inside each request, on the
// device from the requests' row offsets, so a tile has one adapter and the
// calls need no host copy of the batch layout.
//
// Both products run on the bf16 16x16x32 matrix-core instruction: lane l gives
// row l%16 of either operand, 8 contracted values (chunk l/16 of 32); lane l
// gets rows 4(l/16) .. +3 of the first operand against row l%16 of the second.
// Neighbouring lanes thus hold different rows, and a load or store in that
// order is a cache access per lane (measured: 64 per instruction, which bound
// both kernels).  So operands come through LDS, copied there in 1 KiB pieces
// of whole rows, 16-byte chunks permuted so that the operand reads hit
// different banks, and results leave through LDS row by row.
//
// t stands between the launches as fp32 blocks of 16 ranks, [part of K][block]
// [row][16]: a tile's rows of a block are contiguous.
#include "sq_device.hpp"
#include "sq_launch.hpp"

namespace sq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Tile `tile` of a batch cut into tiles of at most BM rows of one request, and
// that request's adapter (-1: none, or an index outside the table).  Offsets
// outside [0, M] are clamped, so no row outside the batch is named whatever
// they hold; rows == 0: no such tile.  One wave asks; the adapter indices are
// loaded beside the offsets, since a kernel of a few microseconds is a chain
// of dependent loads before its first useful one.
struct RowTile {
  int32_t rows, adapter;
  int64_t row0;
};

template <int BM>
__device__ __forceinline__ RowTile find_tile(const AdapterProblem &p, int tile) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < p.n_req; i0 += 64) {
    const int i = min(i0 + lane, p.n_req - 1);
    const int id = p.adapter[i];
    const int lo = (int)min(max((int64_t)p.row_offset[i], (int64_t)0), p.M);
    const int hi = (int)min(max((int64_t)p.row_offset[i + 1], (int64_t)0), p.M);
    const int mine = i0 + lane < p.n_req && hi > lo ? (hi - lo + BM - 1) / BM : 0;
    int upto = mine;  // tiles of the requests i0 .. i0 + lane
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      upto += lane >= o ? v : 0;
    }
    const uint64_t holds = __ballot(tile < upto);
    if (holds) {
      const int l = __ffsll((unsigned long long)holds) - 1;
      const int at = (tile - (__builtin_amdgcn_readlane(upto, l) -
                              __builtin_amdgcn_readlane(mine, l))) * BM;
      const int a = __builtin_amdgcn_readlane(id, l);
      RowTile t;
      t.row0 = (int64_t)__builtin_amdgcn_readlane(lo, l) + at;
      t.rows = min(BM, __builtin_amdgcn_readlane(hi, l) - __builtin_amdgcn_readlane(lo, l) - at);
      t.adapter = a >= 0 && a < p.n_adapters ? a : -1;
      return t;
    }
    tile -= __builtin_amdgcn_readlane(upto, 63);
  }
  return {0, -1, 0};
}

__device__ __forceinline__ int rank_of(const AdapterProblem &p, int a) {
  if (!p.rank_of) return p.rank;
  return min(max(__builtin_amdgcn_readfirstlane(p.rank_of[a]), 0), p.rank);
}

// Block of 16 ranks of t: rows of 16 values.
__device__ __forceinline__ float *t_block(const AdapterProblem &p, int part, int block) {
  return p.t + ((int64_t)part * (p.ns.n * p.rank / 16) + block) * p.M * 16;
}

typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from global memory to 1 KiB of LDS, in lane order.
__device__ __forceinline__ void copy_lds16(const void *g, void *l) {
  __builtin_amdgcn_global_load_lds(g, (lds_void *)l, 16, 0, 0);
}

// Wait until at most N vector-memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_copies() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N & 48) << 10) | 0x0f70);
  __builtin_amdgcn_sched_barrier(0);
}

// ------------------------------------------------------------- shrink ----
// Grid: (row tile, block of 16 NT factor rows, part of K).  WV waves take every
// WV-th 64-wide step of K, each with its own rotating pair of LDS buffers and
// no barrier; their sums meet in LDS.  A copy is 8 rows x 128 bytes, whole
// cache lines: copies of 64 bytes a row asked for each line twice, and the
// second request waited on the first's (8192x6144, rank 64: 33 against NN us).
// Lane l copies chunk (l%8) ^ ((row/2)%8) of its row, so operand row r finds
// chunk c at place c ^ ((r/2)%8) and 16 lanes read 16 different groups of four
// banks.
template <int MT, int NT, int WV>
__global__ __launch_bounds__(64 * WV) void adapter_shrink_kernel(AdapterProblem p) {
  constexpr int kStep = (MT + NT) * 2048;  // bytes of a wave's step
  constexpr int kSums = WV * MT * NT * 1024;
  constexpr int kBytes = 2 * WV * kStep > kSums ? 2 * WV * kStep : kSums;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kBytes];
  const RowTile t = find_tile<16 * MT>(p, blockIdx.x);
  const int a = t.adapter;
  if (t.rows == 0 || a < 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rt = p.ns.n * p.rank, c0 = blockIdx.y * 16 * NT;
  const int64_t k0 = (int64_t)blockIdx.z * p.k_per_split;
  const int64_t k1 = min(k0 + p.k_per_split, p.K);
  const int pieces = k1 > k0 ? (int)((k1 - k0) / 64) : 0;
  const int steps = wave < pieces ? (pieces - wave + WV - 1) / WV : 0;

  const uint16_t *xp[2 * MT], *ap[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int row = 8 * i + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
    xp[i] = p.x + (t.row0 + min(row, t.rows - 1)) * p.ld_x + k0 + 64 * wave + 8 * chunk;
  }
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const int row = 8 * i + (lane >> 3), chunk = (lane & 7) ^ ((row >> 1) & 7);
    ap[i] = p.a + ((int64_t)a * rt + min(c0 + row, rt - 1)) * p.K + k0 + 64 * wave + 8 * chunk;
  }
  uint8_t *mine = smem + wave * 2 * kStep;
  auto copy = [&](int step) {
    uint8_t *to = mine + (step & 1) * kStep;
    const int64_t k = 64 * WV * (int64_t)step;
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) copy_lds16(xp[i] + k, to + 1024 * i);
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j) copy_lds16(ap[j] + k, to + 1024 * (2 * MT + j));
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  // this lane's 16 bytes of an operand block, for either half of the 64
  const int r = lane & 15, g = lane >> 4, f = (r >> 1) & 7;
  const int at[2] = {128 * r + 16 * (g ^ f), 128 * r + 16 * ((4 + g) ^ f)};
  if (steps > 0) copy(0);
  for (int s = 0; s < steps; ++s) {
    if (s + 1 < steps) {
      copy(s + 1);
      wait_copies<2 * (MT + NT)>();
    } else {
      wait_copies<0>();
    }
    const uint8_t *from = mine + (s & 1) * kStep;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4u x[MT], w[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) x[i] = *reinterpret_cast<const v4u *>(from + 2048 * i + at[h]);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        w[j] = *reinterpret_cast<const v4u *>(from + 2048 * (MT + j) + at[h]);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma(w[j], x[i], acc[i][j]);
    }
  }

  const float alpha = p.alpha ? p.alpha[a] : 1.0f;
  const int rank = rank_of(p, a);
  __syncthreads();  // the buffers become the sums
  v4f(*sums)[MT * NT][64] = reinterpret_cast<v4f(*)[MT * NT][64]>(smem);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // stored row by row: lane l has row l/4, ranks 4 (l%4) .. +3 of a block
  const int from = 16 * (lane & 3) + (lane >> 2);
  for (int u = wave; u < MT * NT; u += WV) {
    const int m = 16 * (u / NT) + (lane >> 2), c = c0 + 16 * (u % NT);
    v4f v = sums[0][u][from];
#pragma unroll
    for (int w = 1; w < WV; ++w) v += sums[w][u][from];
    const int q = c - div24(c, p.rank) * p.rank + 4 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = q + i < rank ? v[i] * alpha : 0.0f;
    if (m < t.rows && c < rt)
      *reinterpret_cast<v4f *>(t_block(p, blockIdx.z, c / 16) + (t.row0 + m) * 16 +
                               4 * (lane & 3)) = v;
  }
}

// ------------------------------------------------------------- expand ----
// Four fp32 values as bf16: the upper halves of the fp32 words (hi), and what
// they leave (lo).  x = hi + lo to 2^-15, so t enters the second product with
// 16 bits of mantissa at the cost of a second matrix-core operand.
__device__ __forceinline__ void split4(v4f f, v2u &hi, v2u &lo) {
  float h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0xffff0000u;
    h[i] = __uint_as_float(b);
    // an infinite t is all in hi: inf - inf would turn it into NaN
    l[i] = (b & 0x7f800000u) == 0x7f800000u ? 0.0f : f[i] - h[i];
  }
  hi = v2u{cvt_bf16x2(h[0], h[1]), cvt_bf16x2(h[2], h[3])};
  lo = v2u{cvt_bf16x2(l[0], l[1]), cvt_bf16x2(l[2], l[3])};
}

// Run `run` of column blocks: at most per_run blocks of 64 columns of one
// segment, runs numbered through the segments; seg == ns.n: past the last.
struct ColRun {
  int seg, n0, end;  // first column, end of the run
};

__device__ __forceinline__ ColRun find_run(const NSegEnds &ns, int run, int per_run) {
  ColRun c{0, 0, 0};
  const int width = 64 * per_run;
  for (int off = 0, end; c.seg < ns.n; ++c.seg, off = end) {
    end = 16 * (int)ns.end16[c.seg];
    const int runs = (end - off + width - 1) / width;
    if (run < runs) {
      c.n0 = off + width * run;
      c.end = min(c.n0 + width, end);
      break;
    }
    run -= runs;
  }
  return c;
}

// Grid: (row tile, run of column blocks of one segment).  A workgroup keeps
// its rows' t in LDS as matrix-core operands, made once by its four waves; the
// waves take the run's blocks of 64 columns in turn.  16 ranks fill one
// instruction: its 32 contracted values are t's hi then lo halves against the
// 16 values of B twice.  A block's B (RC blocks of 16 ranks) is 2 RC KiB of
// contiguous memory, copied to LDS with chunk c of column n at place c ^
// f(n), and held in registers for all rows, so the next block's copy runs
// under this one's products; its base is loaded a block ahead too.
template <int MT, int RC>
struct ExpandLds {
  v4u t[MT * RC][64];
  uint8_t b[4][2048 * RC];
  float out[4][16][68];  // a row of 64 columns, padded
};

template <int RC>
__device__ __forceinline__ int b_place(int chunk, int col) {
  return RC == 4 ? chunk ^ ((col >> 1) & 7) : RC == 2 ? chunk ^ ((col >> 2) & 3)
       : RC == 1 ? chunk ^ ((col >> 3) & 1) : chunk;  // its own inverse
}

template <int MT, int RC>
__global__ __launch_bounds__(256) void adapter_expand_kernel(AdapterProblem p) {
  __shared__ __attribute__((aligned(1024))) ExpandLds<MT, RC> lds;
  const ColRun run = find_run(p.ns, blockIdx.y, p.run_tiles);
  const RowTile t = find_tile<16 * MT>(p, blockIdx.x);
  const int a = t.adapter;
  if (t.rows == 0 || run.seg == p.ns.n || (a < 0 && p.base == p.y)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int orow = lane >> 3, ocol = 8 * (lane & 7);  // this lane's place in a row of the output
  v4u base[MT][2], b[RC][4];

  auto load_base = [&](int i, int n0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = 16 * i + 8 * h + orow;
      base[i][h] = v4u{0u, 0u, 0u, 0u};
      if (p.base && m < t.rows && n0 + ocol < run.end)
        base[i][h] = *reinterpret_cast<const v4u *>(p.base + (t.row0 + m) * p.ld_base + n0 + ocol);
    }
  };
  auto copy_b = [&](int n0) {
#pragma unroll
    for (int q = 0; q < 2 * RC; ++q) {
      const int flat = 64 * q + lane, n = flat / (2 * RC), place = flat % (2 * RC);
      copy_lds16(p.b + ((int64_t)a * p.N + min(n0 + n, run.end - 1)) * p.rank +
                     8 * b_place<RC>(place, n),
                 lds.b[wave] + 1024 * q);
    }
  };

  int n0 = run.n0 + 64 * wave;
  if (n0 < run.end) {
    if (a >= 0) copy_b(n0);
#pragma unroll
    for (int i = 0; i < MT; ++i) load_base(i, n0);
  }
  int rank = 0;
  if (a >= 0) {
    rank = rank_of(p, a);
    for (int f = wave; f < MT * RC; f += 4) {
      // lane l: row l/4, ranks 4 (l%4) .. +3 of the block
      const int m = min(16 * (f / RC) + (lane >> 2), t.rows - 1);
      const int block = (run.seg * p.rank) / 16 + f % RC;
      v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int s0 = 0; s0 < p.splits; s0 += 4) {  // the parts of K that the shrink left
        v4f u[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          u[s] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
          if (s0 + s < p.splits)
            u[s] = *reinterpret_cast<const v4f *>(t_block(p, s0 + s, block) + (t.row0 + m) * 16 +
                                                  4 * (lane & 3));
        }
        sum += (u[0] + u[1]) + (u[2] + u[3]);
      }
      v2u hi, lo;
      split4(sum, hi, lo);
      // operand lane 16 c + row holds ranks 8c .. +7 (lo: 32 lanes on)
      v2u *to = reinterpret_cast<v2u *>(lds.t[f]) +
                2 * (16 * ((lane & 3) >> 1) + (lane >> 2)) + (lane & 1);
      to[0] = hi;
      to[64] = lo;
    }
  }
  __syncthreads();
  for (; n0 < run.end; n0 += 256) {
    const bool more = n0 + 256 < run.end;
    if (a >= 0) {
      wait_copies<0>();
#pragma unroll
      for (int e = 0; e < RC; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 16 * j + r;
          b[e][j] = *reinterpret_cast<const v4u *>(
              lds.b[wave] + 32 * RC * n + 16 * b_place<RC>(2 * e + (g & 1), n));
        }
      __builtin_amdgcn_s_waitcnt(0xc07f);  // the reads are done: the buffer is free
      __builtin_amdgcn_sched_barrier(0);
      if (more) copy_b(n0 + 256);
#pragma unroll
      for (int e = 0; e < RC; ++e) {
        if (16 * e + 16 > rank) {  // what is stored past an adapter's rank is not used
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int at = 16 * e + 8 * (g & 1) + 2 * q;
              b[e][j][q] = at + 1 < rank ? b[e][j][q] : at < rank ? b[e][j][q] & 0xffffu : 0u;
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      v4u y[2] = {base[i][0], base[i][1]};
      if (more) load_base(i, n0 + 256);
      if (a >= 0) {
        v4f acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < RC; ++e) {
          const v4u tf = lds.t[i * RC + e][lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = mfma(b[e][j], tf, acc[j]);
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<v4f *>(&lds.out[wave][r][16 * j + 4 * g]) = acc[j];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4f *d = reinterpret_cast<const v4f *>(&lds.out[wave][8 * h + orow][ocol]);
          const v4f u = d[0], v = d[1];
          y[h][0] = cvt_bf16x2(bf16_lo(y[h][0]) + u[0], bf16_hi(y[h][0]) + u[1]);
          y[h][1] = cvt_bf16x2(bf16_lo(y[h][1]) + u[2], bf16_hi(y[h][1]) + u[3]);
          y[h][2] = cvt_bf16x2(bf16_lo(y[h][2]) + v[0], bf16_hi(y[h][2]) + v[1]);
          y[h][3] = cvt_bf16x2(bf16_lo(y[h][3]) + v[2], bf16_hi(y[h][3]) + v[3]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = 16 * i + 8 * h + orow;
        if (m < t.rows && n0 + ocol < run.end)
          *reinterpret_cast<v4u *>(p.y + (t.row0 + m) * p.ld_y + n0 + ocol) = y[h];
      }
    }
  }
}

// The same for ranks above 64: t and B pass through the registers 16 ranks at
// a time, straight from memory.  Column 32 (j/2) + 8q + 4 (j%2) + i is row 4q +
// i of instruction j, so a lane ends with 8 neighbouring columns twice.
template <int MT>
__global__ __launch_bounds__(256) void adapter_expand_wide_kernel(AdapterProblem p) {
  const ColRun ct =
      find_run(p.ns, blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), 1);
  const RowTile t = find_tile<16 * MT>(p, blockIdx.x);
  const int a = t.adapter;
  if (t.rows == 0 || ct.seg == p.ns.n || (a < 0 && p.base == p.y)) return;
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4, k = 8 * (g & 1);
  v4f acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (a >= 0) {
    const int rank = rank_of(p, a);
    const uint16_t *bp[4];
    int64_t tp[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      bp[j] = p.b + ((int64_t)a * p.N +
                     min(ct.n0 + 8 * (r >> 2) + (r & 3) + 4 * (j & 1) + 32 * (j >> 1), ct.end - 1)) *
                        p.rank + k;
#pragma unroll
    for (int i = 0; i < MT; ++i)
      tp[i] = (t.row0 + min(16 * i + r, t.rows - 1)) * 16 + k;
    for (int c = 0; c < rank; c += 16) {
      v4u b[4], tv[MT];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const v4u *>(bp[j] + c);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        v4f u = {0.0f, 0.0f, 0.0f, 0.0f}, v = u;
        for (int s = 0; s < p.splits; ++s) {
          const float *q = t_block(p, s, (ct.seg * p.rank + c) / 16) + tp[i];
          u += *reinterpret_cast<const v4f *>(q);
          v += *reinterpret_cast<const v4f *>(q + 4);
        }
        v2u h0, h1, l0, l1;
        split4(u, h0, l0);
        split4(v, h1, l1);
        tv[i] = g >= 2 ? v4u{l0[0], l0[1], l1[0], l1[1]} : v4u{h0[0], h0[1], h1[0], h1[1]};
      }
      if (c + 16 > rank) {  // what is stored past an adapter's rank is not used
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = c + k + 2 * e;
            b[j][e] = at + 1 < rank ? b[j][e] : at < rank ? b[j][e] & 0xffffu : 0u;
          }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma(b[j], tv[i], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = t.row0 + 16 * i + r;
    if (16 * i + r >= t.rows) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = ct.n0 + 8 * g + 32 * h;
      if (n >= ct.end) continue;
      v4u y = {0u, 0u, 0u, 0u};
      if (p.base) y = *reinterpret_cast<const v4u *>(p.base + m * p.ld_base + n);
      if (a >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const v4f v = acc[i][2 * h + (e >> 1)];
          y[e] = cvt_bf16x2(bf16_lo(y[e]) + v[2 * (e & 1)], bf16_hi(y[e]) + v[2 * (e & 1) + 1]);
        }
      }
      *reinterpret_cast<v4u *>(p.y + m * p.ld_y + n) = y;
    }
  }
}

// Launch shape from the sizes the host knows.
struct AdapterPlan {
  int mt, nt, splits;  // shrink
  int64_t k_per_split;
  int expand_mt;
};

// Tiles of at most bm rows: every request that has rows adds at most one
// that is not full.
int64_t tile_bound(const AdapterProblem &p, int bm) {
  const int64_t n = p.M / bm + p.n_req;
  return n < p.M ? n : p.M;
}

AdapterPlan adapter_plan(const AdapterProblem &p) {
  AdapterPlan l;
  const int64_t rt = (int64_t)p.ns.n * p.rank;
  const bool few = p.M <= 16 * (int64_t)p.n_req;  // at most 16 rows per request
  // shrink: a tile of BM rows reads BM K values of x and, from L2, rt K of a
  l.mt = few || rt <= 16 ? 1 : rt <= 32 ? 2 : 4;
  l.nt = rt <= 16 ? 1 : rt <= 32 ? 2 : 4;
  auto groups = [&] {
    return tile_bound(p, 16 * l.mt) * ((rt + 16 * l.nt - 1) / (16 * l.nt));
  };
  while (few && l.nt > 1 && groups() < 256) l.nt /= 2;
  // parts of K: while the workgroups do not fill the chip (two to a CU at the
  // largest LDS footprint) and each keeps four steps.  8192x6144, rank 64,
  // 136 tiles: 40, 32, 28, 35, 32 us with 2, 3, 4, 6, 8 parts
  const int64_t steps = (p.K + 255) / 256;
  l.splits = 1;
  while (l.splits < 4 && groups() * l.splits < 512 && steps >= 2 * (l.splits + 1)) ++l.splits;
  l.k_per_split = 256 * ((steps + l.splits - 1) / l.splits);
  l.expand_mt = few ? 1 : 4;
  return l;
}

}  // namespace

size_t adapter_workspace_bytes(const AdapterProblem &p) {
  return sizeof(float) * (size_t)adapter_plan(p).splits * (size_t)p.M * (size_t)p.ns.n *
         (size_t)p.rank;
}

namespace {

template <int MT>
void launch_expand(const AdapterProblem &q, hipStream_t s) {
  AdapterProblem p = q;
  const int64_t rows = tile_bound(p, 16 * MT);
  auto runs = [&](int per_run) {
    int64_t n = 0;
    for (int i = 0, off = 0, end; i < p.ns.n; ++i, off = end) {
      end = 16 * (int)p.ns.end16[i];
      n += (end - off + 64 * per_run - 1) / (64 * per_run);
    }
    return n;
  };
  if (p.rank > 64) {
    hipLaunchKernelGGL((adapter_expand_wide_kernel<MT>),
                       dim3((unsigned)rows, (unsigned)((runs(1) + 3) / 4)), dim3(256), 0, s, p);
    return;
  }
  // column blocks per workgroup: one per wave, and more until the workgroups
  // all fit the chip at once
  p.run_tiles = 4;
  while (p.run_tiles < 64 && rows * runs(p.run_tiles) > (MT == 1 ? 1024 : 768)) p.run_tiles += 4;
  const dim3 grid((unsigned)rows, (unsigned)runs(p.run_tiles));
#define SQ_EXPAND(RC) \
  hipLaunchKernelGGL((adapter_expand_kernel<MT, RC>), grid, dim3(256), 0, s, p)
  if (p.rank == 16) SQ_EXPAND(1);
  else if (p.rank == 32) SQ_EXPAND(2);
  else if (p.rank == 48) SQ_EXPAND(3);
  else SQ_EXPAND(4);
#undef SQ_EXPAND
}

}  // namespace

hipError_t launch_adapter(const AdapterProblem &q, hipStream_t s) {
  AdapterProblem p = q;
  const AdapterPlan l = adapter_plan(p);
  p.splits = l.splits;
  p.k_per_split = l.k_per_split;
  const int64_t rt = (int64_t)p.ns.n * p.rank;
  const dim3 shrink((unsigned)tile_bound(p, 16 * l.mt),
                    (unsigned)((rt + 16 * l.nt - 1) / (16 * l.nt)), (unsigned)l.splits);
#define SQ_SHRINK(MT, NT) \
  hipLaunchKernelGGL((adapter_shrink_kernel<MT, NT, (MT + NT > 5 ? 2 : 4)>), shrink, \
                     dim3(MT + NT > 5 ? 128 : 256), 0, s, p)
#define SQ_SHRINK_NT(MT)            \
  if (l.nt == 1) SQ_SHRINK(MT, 1);  \
  else if (l.nt == 2) SQ_SHRINK(MT, 2); \
  else SQ_SHRINK(MT, 4);
  if (l.mt == 1) {
    SQ_SHRINK_NT(1)
  } else if (l.mt == 2) {
    SQ_SHRINK_NT(2)
  } else {
    SQ_SHRINK_NT(4)
  }
#undef SQ_SHRINK_NT
#undef SQ_SHRINK
  if (l.expand_mt == 1) launch_expand<1>(p, s);
  else launch_expand<4>(p, s);
  return hipGetLastError();
}

}  // namespace sq
