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
#include "sq_rows.hpp"

namespace sq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// The batch in tiles of at most BM rows of one request: request r has the tile
// numbers from off[r]/BM + r up to the next request's, which is at least as
// many as it needs (a last one may be empty), so a tile's request is found by a
// search over the offsets alone and M/BM + n_req tiles are enough.  Where M
// numbers are fewer (a row or so per request: by_row), a tile's number is its
// first row's, and the numbers between a request's tiles are empty.  adapter is
// the request's (-1: none, or an index outside the table); rows == 0: no such
// tile.  Offsets outside [0, M] are clamped, so no row outside the batch is
// named whatever they hold.  One wave asks; up to 64 requests take one step,
// with the adapter indices loaded beside the offsets, since a kernel of a few
// microseconds is a chain of dependent loads before its first useful one.
struct RowTile {
  int32_t rows, adapter;
  int64_t row0;
};

template <int BM>
__device__ __forceinline__ RowTile find_tile(const AdapterProblem &p, int tile) {
  const int lane = threadIdx.x & 63, n = p.n_req;
  auto offset = [&](int i) { return (int)min(max((int64_t)p.row_offset[i], (int64_t)0), p.M); };
  auto first_of = [&](int off, int r) { return p.by_row ? off : off / BM + r; };
  int r, lo, hi, id;  // the last request whose first tile is not past this one
  if (n <= 64) {
    const int i = min(lane, n - 1);
    const int mine = offset(i), next = offset(i + 1), a = p.adapter[i];
    r = __popcll(__ballot(lane < n && first_of(mine, i) <= tile)) - 1;
    if (r < 0) return {0, -1, 0};
    r = __builtin_amdgcn_readfirstlane(r);
    lo = __builtin_amdgcn_readlane(mine, r);
    hi = __builtin_amdgcn_readlane(next, r);
    id = __builtin_amdgcn_readlane(a, r);
  } else {
    int base = 0, width = n, count;  // the request is one of base .. base + width - 1
    for (;;) {  // every step'th of them, then those from the last that fits
      const int step = (width + 63) / 64, i = base + min(lane * step, width - 1);
      count = __popcll(__ballot(lane * step < width && first_of(offset(i), i) <= tile));
      count = __builtin_amdgcn_readfirstlane(count);
      if (count == 0) break;
      base += (count - 1) * step;
      width = min(step, width - (count - 1) * step);
      if (step == 1) break;
    }
    if (base == 0 && count == 0) return {0, -1, 0};
    r = base;
    lo = offset(r);
    hi = offset(r + 1);
    id = p.adapter[r];
  }
  RowTile t;
  const int past = tile - first_of(lo, r);  // tiles (by_row: rows) into the request
  const int64_t first = lo + (int64_t)past * (p.by_row ? 1 : BM);
  // past < 0: offsets that decrease, where the count above is no search
  t.rows = past < 0 || (p.by_row && past % BM) ? 0
           : (int)min((int64_t)BM, max((int64_t)0, hi - first));
  t.row0 = first;
  t.adapter = __builtin_amdgcn_readfirstlane(id >= 0 && id < p.n_adapters ? id : -1);
  return t;
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
// second request waited on the first's (8192x6144, rank 64: 33 against 28 us).
// Lane l copies chunk (l%8) ^ ((row/2)%8) of its row, so operand row r finds
// chunk c at place c ^ ((r/2)%8) and 16 lanes read 16 different groups of four
// banks.
template <int MT, int NT, int WV>
struct Shrink {
  static constexpr int kStep = (MT + NT) * 2048;  // bytes of a wave's step
  static constexpr int kSums = WV * MT * NT * 1024;
  static constexpr int kBytes = 2 * WV * kStep > kSums ? 2 * WV * kStep : kSums;

  // Sums of the tile's rows against factor rows c0 .. over k0 <= k < k1, a
  // wave's share in acc.
  static __device__ __forceinline__ void products(const AdapterProblem &p, const RowTile &t,
                                                  int c0, int64_t k0, int64_t k1, uint8_t *smem,
                                                  v4f acc[MT][NT]) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rt = p.ns.n * p.rank;
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
      ap[i] = p.a + ((int64_t)t.adapter * rt + min(c0 + row, rt - 1)) * p.K + k0 + 64 * wave +
              8 * chunk;
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
  }

  // The waves' shares to LDS (the copies' buffers, once every wave is done).
  static __device__ __forceinline__ void gather(const v4f acc[MT][NT], uint8_t *smem) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < MT * NT; ++u)
      reinterpret_cast<v4f *>(smem)[(wave * MT * NT + u) * 64 + lane] = acc[u / NT][u % NT];
    __syncthreads();
  }

  // Block u = NT * (block of rows) + (block of ranks) of the sum, row by row:
  // lane l has row l/4, ranks 4 (l%4) .. +3; q0 is the block's first rank.
  static __device__ __forceinline__ v4f block(const uint8_t *smem, int u, int q0, int rank,
                                              float alpha) {
    const int lane = threadIdx.x & 63, from = 16 * (lane & 3) + (lane >> 2);
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < WV; ++w)
      v += reinterpret_cast<const v4f *>(smem)[(w * MT * NT + u) * 64 + from];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = q0 + 4 * (lane & 3) + i < rank ? v[i] * alpha : 0.0f;
    return v;
  }
};

template <int MT, int NT, int WV>
__global__ __launch_bounds__(64 * WV) void adapter_shrink_kernel(AdapterProblem p) {
  using Sh = Shrink<MT, NT, WV>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Sh::kBytes];
  const RowTile t = find_tile<16 * MT>(p, blockIdx.x);
  if (t.rows == 0 || t.adapter < 0) return;
  const int rt = p.ns.n * p.rank, c0 = blockIdx.y * 16 * NT;
  const int64_t k0 = (int64_t)blockIdx.z * p.k_per_split;
  v4f acc[MT][NT];
  Sh::products(p, t, c0, k0, min(k0 + p.k_per_split, p.K), smem, acc);
  const float alpha = p.alpha ? p.alpha[t.adapter] : 1.0f;
  const int rank = rank_of(p, t.adapter);
  Sh::gather(acc, smem);
  const int lane = threadIdx.x & 63;
  for (int u = threadIdx.x >> 6; u < MT * NT; u += WV) {
    const int m = 16 * (u / NT) + (lane >> 2), c = c0 + 16 * (u % NT);
    const v4f v = Sh::block(smem, u, c - div24(c, p.rank) * p.rank, rank, alpha);
    if (m < t.rows && c < rt)
      *reinterpret_cast<v4f *>(t_block(p, blockIdx.z, c / 16) + (t.row0 + m) * 16 +
                               4 * (lane & 3)) = v;
  }
}

// ------------------------------------------------------------- expand ----
// Four fp32 values as bf16 parts whose sum they are: hi, the next value below in
// magnitude with a bf16's bits, mid, the next below what hi leaves, and lo, the
// eight bits that remain, so t enters the second product as it is, at the cost
// of matrix-core operands.  "Below" also where x itself is a bf16: no part of a
// nonzero x is 0 then and all have its sign, so an infinite factor gives x's
// infinity and not inf + 0 inf = NaN (from |x| = 2^-110 up, where lo stays in
// bf16's range).  An infinite x becomes two largest bf16 and infinity.
__device__ __forceinline__ void split4(v4f f, v2u &hi, v2u &mid, v2u &lo) {
  auto below = [](float x) {
    const uint32_t b = __float_as_uint(x);
    return __uint_as_float((b << 1 ? b - 1 : b) & 0xffff0000u);
  };
  float h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = below(f[i]);
    m[i] = below(f[i] - h[i]);
    l[i] = f[i] - h[i] - m[i];
  }
  hi = v2u{cvt_bf16x2(h[0], h[1]), cvt_bf16x2(h[2], h[3])};
  mid = v2u{cvt_bf16x2(m[0], m[1]), cvt_bf16x2(m[2], m[3])};
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

// A row block's t in LDS as matrix-core operands, RC blocks of 16 ranks: two
// blocks make an operand each of hi, mid and lo parts, a block left alone one of
// hi and mid and one of lo parts and zeros.
template <int RC>
struct TOperands {
  static constexpr int kPairs = RC / 2, kB = (RC + 1) / 2;  // operands of B
  static constexpr bool kAlone = RC % 2;
  static constexpr int kAll = 3 * kPairs + 2 * kAlone;

  // Four ranks of a row (lane l of a wave: row l/4, ranks 4 (l%4) .. +3) of
  // block e: lane 16 c + row of an operand holds the contracted values 8c .. +7.
  static __device__ __forceinline__ void store(v4u *op, int e, v4f v) {
    const int lane = threadIdx.x & 63;
    v2u hi, mid, lo;
    split4(v, hi, mid, lo);
    v2u *to = reinterpret_cast<v2u *>(op + 64 * 3 * (e / 2)) +
              2 * (16 * ((lane & 3) >> 1) + (lane >> 2)) + (lane & 1);
    if (kAlone && e == RC - 1) {
      to[0] = hi;
      to[64] = mid;
      to[128] = lo;
      to[192] = v2u{0u, 0u};
    } else {
      to += 64 * (e & 1);
      to[0] = hi;
      to[128] = mid;
      to[256] = lo;
    }
  }
};

// The second product for a workgroup's rows and a run of columns.  t stands in
// LDS as matrix-core operands; the four waves take the run's blocks of 64
// columns in turn.  32 ranks take three instructions, one for each part of t
// against the same operand of B, and 16 ranks alone two: hi and mid parts
// against the 16 values of B twice, lo parts against them and zeros.  (Both
// launches, 8192 x 1536, rank 64, K 6144: 48.4 us; t in two parts, which holds 16
// bits of it, 47.6; an operand of B for every 16 ranks 56.4.)  A block's B (RC
// blocks of 16 ranks) is 2 RC KiB of contiguous memory, copied to LDS with
// chunk c of column n at place c ^ f(n), and held in registers for all rows,
// so the next block's copy runs under this one's products; its base is loaded
// a block ahead too.
template <int RC>
__device__ __forceinline__ int b_place(int chunk, int col) {
  return RC == 4 ? chunk ^ ((col >> 1) & 7) : RC == 2 ? chunk ^ ((col >> 2) & 3)
       : RC == 1 ? chunk ^ ((col >> 3) & 1) : chunk;  // its own inverse
}

template <int MT, int RC>
struct Expand {
  using Ops = TOperands<RC>;
  static constexpr int kB = 2048 * RC;        // bytes of a block's B, per wave
  static constexpr int kOut = 16 * 68 * 4;    // 16 rows of 64 columns, padded, per wave
  static constexpr int kBytes = 4 * (kB + kOut);

  const AdapterProblem &p;
  const RowTile &t;
  const ColRun &run;
  uint8_t *b_lds;
  float (*out)[68];
  int n0;  // this wave's next block of columns
  v4u base[MT][2];

  __device__ __forceinline__ Expand(const AdapterProblem &p, const RowTile &t, const ColRun &run,
                                    uint8_t *lds)
      : p(p), t(t), run(run) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    b_lds = lds + wave * kB;
    out = reinterpret_cast<float(*)[68]>(lds + 4 * kB + wave * kOut);
    n0 = run.n0 + 64 * wave;
  }

  // FULL: every row and column of the tile's blocks is there
  template <bool FULL = false>
  __device__ __forceinline__ void load_base(int i, int n) {
    const int lane = threadIdx.x & 63;
    const int64_t col = n + 8 * (lane & 7);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = 16 * i + 8 * h + (lane >> 3);
      base[i][h] = v4u{0u, 0u, 0u, 0u};
      if (p.base && (FULL || (m < t.rows && col < run.end)))
        base[i][h] = *reinterpret_cast<const v4u *>(p.base + (t.row0 + m) * p.ld_base + col);
    }
  }

  __device__ __forceinline__ void first_base() {
    if (n0 < run.end) {
#pragma unroll
      for (int i = 0; i < MT; ++i) load_base(i, n0);
    }
  }

  __device__ __forceinline__ void copy_b(int n) {
    if (t.adapter < 0 || n >= run.end) return;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int q = 0; q < 2 * RC; ++q) {
      const int flat = 64 * q + lane, col = flat / (2 * RC), place = flat % (2 * RC);
      copy_lds16(p.b + ((int64_t)t.adapter * p.N + min(n + col, run.end - 1)) * p.rank +
                     8 * b_place<RC>(place, col),
                 b_lds + 1024 * q);
    }
  }

  __device__ __forceinline__ void columns(const v4u *tv, int rank) {
    if (t.rows == 16 * MT && (run.end - run.n0) % 64 == 0)
      columns_of<true>(tv, rank);
    else
      columns_of<false>(tv, rank);
  }

  template <bool FULL>
  __device__ __forceinline__ void columns_of(const v4u *tv, int rank) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int orow = lane >> 3, ocol = 8 * (lane & 7);  // this lane's place in a row of y
    const uint32_t lower = g < 2 ? ~0u : 0u;  // not against the zeros
    for (; n0 < run.end; n0 += 256) {
      const bool more = n0 + 256 < run.end;
      v4u b[Ops::kB][4];
      // this lane's first rank of operand q of B
      auto rank_at = [&](int q) { return 32 * q + 8 * (q < Ops::kPairs ? g : g & 1); };
      if (t.adapter >= 0) {
        wait_copies<0>();
#pragma unroll
        for (int q = 0; q < Ops::kB; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int n = 16 * j + r;
            b[q][j] = *reinterpret_cast<const v4u *>(b_lds + 32 * RC * n +
                                                     16 * b_place<RC>(rank_at(q) / 8, n));
          }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // the reads are done: the buffer is free
        __builtin_amdgcn_sched_barrier(0);
        copy_b(n0 + 256);
#pragma unroll
        for (int q = 0; q < Ops::kB; ++q) {
          if (32 * q + (q < Ops::kPairs ? 32 : 16) > rank) {
            // what is stored past an adapter's rank is not used
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int at = rank_at(q) + 2 * w;
                b[q][j][w] = at + 1 < rank ? b[q][j][w] : at < rank ? b[q][j][w] & 0xffffu : 0u;
              }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        v4u y[2] = {base[i][0], base[i][1]};
        if (more) load_base<FULL>(i, n0 + 256);
        if (t.adapter >= 0) {
          v4f acc[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < Ops::kB; ++q) {
            const v4u *tq = tv + (i * Ops::kAll + 3 * q) * 64 + lane;
#pragma unroll
            for (int part = q < Ops::kPairs ? 2 : 1; part >= 0; --part) {
              const v4u tf = tq[64 * part];
              const bool half = q == Ops::kPairs && part == 1;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                acc[j] = mfma(half ? b[q][j] & lower : b[q][j], tf, acc[j]);
            }
          }
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<v4f *>(&out[r][16 * j + 4 * g]) = acc[j];
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4f *d = reinterpret_cast<const v4f *>(&out[8 * h + orow][ocol]);
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
          if (FULL || (m < t.rows && n0 + ocol < run.end))
            *reinterpret_cast<v4u *>(p.y + (t.row0 + m) * p.ld_y + n0 + ocol) = y[h];
        }
      }
    }
  }
};

// Grid: (row tile, run of column blocks of one segment).
template <int MT, int RC>
__global__ __launch_bounds__(256) void adapter_expand_kernel(AdapterProblem p) {
  using Ex = Expand<MT, RC>;
  using Ops = TOperands<RC>;
  constexpr int kOps = MT * Ops::kAll * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kOps + Ex::kBytes];
  const ColRun run = find_run(p.ns, blockIdx.y, p.run_tiles);
  const RowTile t = find_tile<16 * MT>(p, blockIdx.x);
  if (t.rows == 0 || run.seg == p.ns.n || (t.adapter < 0 && p.base == p.y)) return;
  v4u *tv = reinterpret_cast<v4u *>(smem);
  Ex ex(p, t, run, smem + kOps);
  int rank = 0;
  if (t.adapter >= 0) {
    // t first and all of it at once, then what is needed after it: loads come
    // back in the order of their issue
    constexpr int F = (MT * RC + 3) / 4;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    v4f u[F][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {  // the parts of K that the shrink left
#pragma unroll
      for (int i = 0; i < F; ++i) u[i][s] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      if (s < p.splits) {
#pragma unroll
        for (int i = 0; i < F; ++i) {
          const int f = min(wave + 4 * i, MT * RC - 1);
          const int64_t row = t.row0 + min(16 * (f / RC) + (lane >> 2), t.rows - 1);
          u[i][s] = *reinterpret_cast<const v4f *>(
              t_block(p, s, (run.seg * p.rank) / 16 + f % RC) + row * 16 + 4 * (lane & 3));
        }
      }
    }
    ex.copy_b(ex.n0);
    ex.first_base();
    rank = rank_of(p, t.adapter);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      const int f = wave + 4 * i;
      if (f < MT * RC)
        Ops::store(tv + 64 * Ops::kAll * (f / RC), f % RC,
                   (u[i][0] + u[i][1]) + (u[i][2] + u[i][3]));
    }
  } else {
    ex.first_base();
  }
  __syncthreads();
  ex.columns(tv, rank);
}

// ------------------------------------------------------- in one launch ----
// Grid: (row tile, run of column blocks of one segment), each workgroup making
// its rows' t for that segment over the whole of K and then its columns.  The
// factor a is read by every row tile and x by every run, from the caches, in
// return for a launch and t's way through memory.
template <int MT, int RC>
__global__ __launch_bounds__(256) void adapter_one_kernel(AdapterProblem p) {
  using Sh = Shrink<MT, RC, 4>;
  using Ex = Expand<MT, RC>;
  using Ops = TOperands<RC>;
  // the copies' buffers become the sums, B and the output rows, the operands
  constexpr int kOperands = Sh::kSums + Ex::kBytes, kAfter = kOperands + MT * Ops::kAll * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t
      smem[Sh::kBytes > kAfter ? Sh::kBytes : kAfter];
  const ColRun run = find_run(p.ns, blockIdx.y, p.run_tiles);
  const RowTile t = find_tile<16 * MT>(p, blockIdx.x);
  if (t.rows == 0 || run.seg == p.ns.n || (t.adapter < 0 && p.base == p.y)) return;
  v4u *tv = reinterpret_cast<v4u *>(smem + kOperands);
  Ex ex(p, t, run, smem + Sh::kSums);
  ex.first_base();
  int rank = 0;
  if (t.adapter >= 0) {
    v4f acc[MT][RC];
    Sh::products(p, t, run.seg * p.rank, 0, p.K, smem, acc);
    const float alpha = p.alpha ? p.alpha[t.adapter] : 1.0f;
    rank = rank_of(p, t.adapter);
    Sh::gather(acc, smem);
    ex.copy_b(ex.n0);  // behind the sums, under the making of the operands
    for (int f = threadIdx.x >> 6; f < MT * RC; f += 4)
      Ops::store(tv + 64 * Ops::kAll * (f / RC), f % RC,
                 Sh::block(smem, f, 16 * (f % RC), rank, alpha));
    __syncthreads();
  }
  ex.columns(tv, rank);
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
      v4u b[4], tv[MT], tl[MT];
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
        v2u h0, h1, m0, m1, l0, l1;
        split4(u, h0, m0, l0);
        split4(v, h1, m1, l1);
        tv[i] = g >= 2 ? v4u{m0[0], m0[1], m1[0], m1[1]} : v4u{h0[0], h0[1], h1[0], h1[1]};
        tl[i] = g >= 2 ? v4u{0u, 0u, 0u, 0u} : v4u{l0[0], l0[1], l1[0], l1[1]};
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
        for (int j = 0; j < 4; ++j) {
          // the lo parts fill half an instruction: zeros against the other half
          acc[i][j] = mfma(b[j] & (g < 2 ? ~0u : 0u), tl[i], acc[i][j]);
          acc[i][j] = mfma(b[j], tv[i], acc[i][j]);
        }
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

// Tile numbers of the batch (find_tile).
int64_t tile_bound(const AdapterProblem &p, int bm) {
  return p.by_row ? p.M : p.M / bm + p.n_req;
}

// Column blocks of 64 in runs of at most per_run, no run across a segment.
int64_t column_runs(const AdapterProblem &p, int per_run) {
  int64_t n = 0;
  for (int i = 0, off = 0, end; i < p.ns.n; ++i, off = end) {
    end = 16 * (int)p.ns.end16[i];
    n += (end - off + 64 * per_run - 1) / (64 * per_run);
  }
  return n;
}

// Column blocks of a run in the second of two launches: one per wave, and more
// until the workgroups of all row tiles fit the chip at once.
int run_tiles_for(const AdapterProblem &p, int64_t rows, int64_t at_once) {
  int n = 4;
  while (n < 64 && rows * column_runs(p, n) > at_once) n += 4;
  return n;
}

// Whether the form in one launch is taken.  It saves a launch and t's way
// through memory, and pays with one workgroup walking the whole of K and with
// reading x and a once per run of columns.  One launch | two (us, MI355X, rank
// 16, 32, 64; 1024 and 4096 rows in four requests, 8192 in eight; x from the
// last-level cache):
//   N 1536               K 1536                  K 3584                  K 6144
//   64 requests of a row  6.5  7.6  8.6           8.1  8.1 10.7           8.7  9.9 14.5
//                       | 7.8  8.2  8.7         | 8.1  8.9  9.7         | 8.4  9.4 10.9
//   1024 rows             6.8  7.9  9.4           8.2 10.5 13.9          12.5 13.8 19.5
//                       | 9.7 10.4 15.2        | 10.7 11.9 17.7        | 11.8 13.0 20.4
//   4096 rows            14.0 15.5 17.0          19.9 20.1 26.8          21.3 26.4 35.6
//                      | 14.2 16.4 20.8        | 18.6 19.9 26.1        | 22.5 22.8 31.6
//   N 4608, 3 segments
//   4096 rows            21.6 22.5 36.1          31.8 31.5 44.5          42.9 43.7 58.5
//                      | 28.3 28.7 43.6        | 33.5 35.2 51.9        | 38.2 47.0 66.9
//   8192 rows            38.9 41.2 57.9          55.7 58.8 78.9          72.4 83.6 108.9
//                      | 40.2 47.5 57.7        | 47.1 58.4 71.7        | 61.4 79.2  97.6
// So: K up to 4096, less for few rows of high rank, and x no more than the
// caches hold: above, x comes from memory, which many short copies per
// workgroup use less well (8192 rows, K 6144, N 1536, rank 64, x from memory:
// 58 against 47 us, though 41 against 49 with x in the last-level cache).
// A few rows per request fill a sixteenth of a tile or little more in either
// form, and the table goes on, rank 16 (MB of x):
//   rows, requests        4096, 512     16384, 1024    65536, 4096   65536, 65536
//   N 1536, K 1536     13.9 | 16.5 (12)  38 |  43 (48) 189 | 200 (192)  866 |  901
//           K 4096     18.5 | 21.5 (32)  68 |  70 (128) 277 | 295 (512) 1176 | 1195
//   N 4608, 3 segments
//           K 1536     30.5 | 33.5      135 | 139      561 | 521      2642 | 2518
//           K 4096     42.7 | 41.9      198 | 176      807 | 665      3562 | 3221
// There what counts is x read again by every segment after the first, as far as
// it passes the 256 MB of the last-level cache.  Cells with the slower form: N
// 1536, 4096 rows, K 3584 (1 to 7 %), 64 rows, K 3584, rank 32 (10 %), 1024 rows,
// K 6144, rank 64 (5 %); N 4608, 4096 rows, K 6144, ranks 32 and 64 (8 and 14 %);
// K 4096 with 3 segments up to 16384 rows of few to a request (2 to 13 %).
bool in_one_launch(const AdapterProblem &p, bool few) {
  if (p.rank > 64) return false;
  const int64_t x_bytes = 2 * p.M * p.K;
  if (few)
    return p.K <= (p.rank > 16 ? 2048 : 4096) && x_bytes * (p.ns.n - 1) <= (256 << 20);
  return p.K <= 4096 && x_bytes <= (48 << 20);
}

// Column blocks of a run in one launch: a longer run walks K fewer times, a
// shorter one spreads better.  Estimated in us: a workgroup's start, steps of K
// and blocks of a wave, two or three of them side by side on a CU at hardly
// more than the time of one, or what all read of x and a from the caches at 13
// TB/s, whichever is more.  64 requests, K 1536, six segments of 24 blocks,
// rank 32: 13.6 us with runs of 12 (3 workgroups a CU), 13.9 with runs of 24;
// 4096 rows of a request, K 3584, N 1536, rank 64: 24.9 with runs of 12, 20.2
// with one of 24.
int one_run_tiles(const AdapterProblem &p) {
  // about as many as are not empty (by_row: about a row each).  64 requests of 8
  // rows, K and N 1536, rank 16: 6.7 us; taken for 512 tiles, which leaves 64
  // workgroups, 9.4
  const int64_t tiles = p.by_row ? p.M : tile_bound(p, 16) - p.n_req / 2;
  const double start = 3.0 + (p.K / 256.0) * (0.1 + 0.004 * p.rank);
  double best = 0.0;
  int take = 4;
  for (int n = 4; n <= 64; n += n < 16 ? 4 : 8) {
    const int64_t groups = tiles * column_runs(p, n);
    const double per_cu = (double)((groups + 255) / 256);
    const double walk = (per_cu > 2.5 ? 0.4 * per_cu : 1.0) * (start + 0.8 * ((n + 3) / 4));
    const double bytes = 2.0 * groups * p.K * (16 + p.rank) / 13e6;
    const double cost = walk > bytes ? walk : bytes;
    if (n == 4 || cost < best) {
      best = cost;
      take = n;
    }
  }
  return take;
}

}  // namespace

size_t adapter_plan(AdapterProblem &p) {
  const int64_t rt = (int64_t)p.ns.n * p.rank;
  const bool few = p.M <= 16 * (int64_t)p.n_req;  // at most 16 rows per request
  p.by_row = p.M <= p.M / 16 + p.n_req;           // implies few: all tiles have 16 rows
  // shrink: a tile of BM rows reads BM K values of x and, from L2, rt K of a
  p.mt = few || rt <= 16 ? 1 : rt <= 32 ? 2 : 4;
  p.nt = rt <= 16 ? 1 : rt <= 32 ? 2 : 4;
  auto groups = [&] {
    return tile_bound(p, 16 * p.mt) * ((rt + 16 * p.nt - 1) / (16 * p.nt));
  };
  while (few && p.nt > 1 && groups() < 256) p.nt /= 2;
  // parts of K: while the workgroups do not fill the chip (two to a CU at the
  // largest LDS footprint) and each keeps two steps of 256.  8192x6144, rank
  // 64, 136 tiles: 40, 32, 28, 35, 32 us with 2, 3, 4, 6, 8 parts
  const int64_t steps = (p.K + 255) / 256;
  p.splits = 1;
  while (p.splits < 4 && groups() * p.splits < 512 && steps >= 2 * (p.splits + 1)) ++p.splits;
  p.k_per_split = 256 * ((steps + p.splits - 1) / p.splits);
  p.expand_mt = few ? 1 : 4;
  p.one = in_one_launch(p, few);
  p.run_tiles = p.one ? one_run_tiles(p)
                      : run_tiles_for(p, tile_bound(p, 16 * p.expand_mt), few ? 1024 : 768);
  return p.one ? 0 : sizeof(float) * (size_t)p.splits * (size_t)p.M * (size_t)rt;
}

namespace {

template <int MT>
void launch_expand(const AdapterProblem &p, hipStream_t s) {
  const unsigned rows = (unsigned)tile_bound(p, 16 * MT);
  if (p.rank > 64) {
    hipLaunchKernelGGL((adapter_expand_wide_kernel<MT>),
                       dim3(rows, (unsigned)((column_runs(p, 1) + 3) / 4)), dim3(256), 0, s, p);
    return;
  }
  const dim3 grid(rows, (unsigned)column_runs(p, p.run_tiles));
#define SQ_EXPAND(RC) \
  hipLaunchKernelGGL((adapter_expand_kernel<MT, RC>), grid, dim3(256), 0, s, p)
  if (p.rank == 16) SQ_EXPAND(1);
  else if (p.rank == 32) SQ_EXPAND(2);
  else if (p.rank == 48) SQ_EXPAND(3);
  else SQ_EXPAND(4);
#undef SQ_EXPAND
}

}  // namespace

hipError_t launch_adapter(const AdapterProblem &p, hipStream_t s) {
  if (p.one) {
    const dim3 grid((unsigned)tile_bound(p, 16), (unsigned)column_runs(p, p.run_tiles));
#define SQ_ONE(RC) hipLaunchKernelGGL((adapter_one_kernel<1, RC>), grid, dim3(256), 0, s, p)
    if (p.rank == 16) SQ_ONE(1);
    else if (p.rank == 32) SQ_ONE(2);
    else if (p.rank == 48) SQ_ONE(3);
    else SQ_ONE(4);
#undef SQ_ONE
    return hipGetLastError();
  }
  const int64_t rt = (int64_t)p.ns.n * p.rank;
  const dim3 shrink((unsigned)tile_bound(p, 16 * p.mt),
                    (unsigned)((rt + 16 * p.nt - 1) / (16 * p.nt)), (unsigned)p.splits);
#define SQ_SHRINK(MT, NT)                                                            \
  hipLaunchKernelGGL((adapter_shrink_kernel<MT, NT, (MT + NT > 5 ? 2 : 4)>), shrink, \
                     dim3(MT + NT > 5 ? 128 : 256), 0, s, p)
#define SQ_SHRINK_NT(MT)                \
  if (p.nt == 1) SQ_SHRINK(MT, 1);      \
  else if (p.nt == 2) SQ_SHRINK(MT, 2); \
  else SQ_SHRINK(MT, 4);
  if (p.mt == 1) {
    SQ_SHRINK_NT(1)
  } else if (p.mt == 2) {
    SQ_SHRINK(2, 2);
  } else {
    SQ_SHRINK(4, 4);
  }
#undef SQ_SHRINK_NT
#undef SQ_SHRINK
  if (p.expand_mt == 1) launch_expand<1>(p, s);
  else launch_expand<4>(p, s);
  return hipGetLastError();
}

}  // namespace sq
