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
// Both products run on the bf16 16x16x32 matrix-core instruction with the
// adapter as its first operand, so that a lane ends up with neighbouring
// ranks (shrink) or columns (expand) of one row and stores them in one piece.
// Instruction operands: lane l gives row l%16 of either operand, 8 values of
// the contracted index; results: lane l holds rows 4(l/16) .. +3 of the first
// operand against row l%16 of the second.
#include "sq_device.hpp"
#include "sq_launch.hpp"

namespace sq {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v4f mfma(v4u a, v4u b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                 __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Tile `tile` of a batch cut into tiles of at most BM rows of one request.
// Offsets outside [0, M] are clamped, so no row outside the batch is named
// whatever they hold; rows == 0: no such tile.
struct RowTile {
  int32_t req, rows;
  int64_t row0;
};

template <int BM>
__device__ __forceinline__ RowTile find_tile(const int32_t *off, int32_t n, int64_t M, int tile) {
  const int lane = threadIdx.x & 63;
  for (int i0 = 0; i0 < n; i0 += 64) {
    const int i = min(i0 + lane, n - 1);
    const int lo = (int)min(max((int64_t)off[i], (int64_t)0), M);
    const int hi = (int)min(max((int64_t)off[i + 1], (int64_t)0), M);
    const int mine = i0 + lane < n && hi > lo ? (hi - lo + BM - 1) / BM : 0;
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
      RowTile t;
      t.req = i0 + l;
      t.row0 = (int64_t)__builtin_amdgcn_readlane(lo, l) + at;
      t.rows = min(BM, __builtin_amdgcn_readlane(hi, l) - __builtin_amdgcn_readlane(lo, l) - at);
      return t;
    }
    tile -= __builtin_amdgcn_readlane(upto, 63);
  }
  return {0, 0, 0};
}

// A request's adapter (-1: none, or an index outside the table) and its rank.
__device__ __forceinline__ int adapter_of(const AdapterProblem &p, int req) {
  const int a = __builtin_amdgcn_readfirstlane(p.adapter[req]);
  return a >= 0 && a < p.n_adapters ? a : -1;
}

__device__ __forceinline__ int rank_of(const AdapterProblem &p, int a) {
  if (!p.rank_of) return p.rank;
  return min(max(__builtin_amdgcn_readfirstlane(p.rank_of[a]), 0), p.rank);
}

// ------------------------------------------------------------- shrink ----
// Grid: (row tile, block of 16 NT factor rows, part of K); four waves take
// every fourth 64-wide step of K and their sums meet in LDS.  A lane reads 16
// consecutive elements of its row, so four lanes cover a 128-byte line; both
// operands use the same order of k, so it does not matter which.
template <int MT, int NT>
__global__ __launch_bounds__(256) void adapter_shrink_kernel(AdapterProblem p) {
  __shared__ v4f sums[4][MT * NT][64];
  const RowTile t = find_tile<16 * MT>(p.row_offset, p.n_req, p.M, blockIdx.x);
  if (t.rows == 0) return;
  const int a = adapter_of(p, t.req);
  if (a < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int rt = p.ns.n * p.rank, c0 = blockIdx.y * 16 * NT;
  const uint16_t *xp[MT], *ap[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    xp[i] = p.x + (t.row0 + min(16 * i + r, t.rows - 1)) * p.ld_x + 16 * g;
#pragma unroll
  for (int i = 0; i < NT; ++i)
    ap[i] = p.a + ((int64_t)a * rt + min(c0 + 16 * i + r, rt - 1)) * p.K + 16 * g;
  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t k0 = (int64_t)blockIdx.z * p.k_per_split;
  const int64_t k1 = min(k0 + p.k_per_split, p.K);
#pragma clang loop unroll(disable)
  for (int64_t k = k0 + 64 * wave; k < k1; k += 256) {
    v4u x[MT][2], w[NT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      x[i][0] = *reinterpret_cast<const v4u *>(xp[i] + k);
      x[i][1] = *reinterpret_cast<const v4u *>(xp[i] + k + 8);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      w[j][0] = *reinterpret_cast<const v4u *>(ap[j] + k);
      w[j][1] = *reinterpret_cast<const v4u *>(ap[j] + k + 8);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma(w[j][h], x[i][h], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) sums[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  const float alpha = p.alpha ? p.alpha[a] : 1.0f;
  const int rank = rank_of(p, a);
  float *out = p.t + (int64_t)blockIdx.z * p.M * rt;
  for (int u = wave; u < MT * NT; u += 4) {
    const int m = 16 * (u / NT) + r, c = c0 + 16 * (u % NT) + 4 * g;
    v4f v = sums[0][u][lane] + sums[1][u][lane] + sums[2][u][lane] + sums[3][u][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = c % p.rank + i < rank ? v[i] * alpha : 0.0f;
    if (m < t.rows && c < rt) *reinterpret_cast<v4f *>(out + (t.row0 + m) * rt + c) = v;
  }
}

// ------------------------------------------------------------- expand ----
// Eight fp32 values as bf16, the upper halves of the fp32 words (hi), or what
// they leave (lo): x = hi + lo to 2^-17, so t enters the second product with
// 16 bits of mantissa at the cost of a second matrix-core operand.
__device__ __forceinline__ v4u split8(v4f u, v4f v, bool lo) {
  float f[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(f[i]) & 0xffff0000u;
    // an infinite t is all in hi: inf - inf would turn it into NaN
    const float rest = (b & 0x7f800000u) == 0x7f800000u ? 0.0f : f[i] - __uint_as_float(b);
    f[i] = lo ? rest : __uint_as_float(b);
  }
  v4u o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return o;
}

// Grid: (row tile, four blocks of 64 columns); each wave has its own 64
// columns of one N-segment and all the tile's rows.  16 ranks fill one
// instruction: its 32 contracted values are t's hi then lo halves against
// the 16 values of B twice.  First-operand row 4q + i of instruction j is
// column 16q + 4j + i, so lane group q holds 16 neighbouring columns after
// the four instructions.
template <int MT>
__global__ __launch_bounds__(256) void adapter_expand_kernel(AdapterProblem p) {
  const RowTile t = find_tile<16 * MT>(p.row_offset, p.n_req, p.M, blockIdx.x);
  if (t.rows == 0) return;
  int tile = blockIdx.y * 4 + (threadIdx.x >> 6), seg = 0;
  for (;; ++seg) {  // which 64 columns of which segment
    if (seg == p.ns.n) return;
    const int tiles = (p.ns.end[seg] - p.ns.off[seg] + 63) / 64;
    if (tile < tiles) break;
    tile -= tiles;
  }
  const int n0 = p.ns.off[seg] + 64 * tile;
  const int cols = min(64, p.ns.end[seg] - n0);
  const int a = adapter_of(p, t.req);
  if (a < 0 && p.base == p.y) return;
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  v4f acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  if (a >= 0) {
    const int rank = rank_of(p, a), rt = p.ns.n * p.rank, k = 8 * (g & 1);
    const uint16_t *bp[4];
    const float *tp[MT];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + min(16 * (r >> 2) + 4 * j + (r & 3), cols - 1);
      bp[j] = p.b + ((int64_t)a * p.N + n) * p.rank + k;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
      tp[i] = p.t + (t.row0 + min(16 * i + r, t.rows - 1)) * rt + seg * p.rank + k;
    for (int c = 0; c < rank; c += 16) {
      v4u b[4], tv[MT];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const v4u *>(bp[j] + c);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        v4f u = *reinterpret_cast<const v4f *>(tp[i] + c);
        v4f v = *reinterpret_cast<const v4f *>(tp[i] + c + 4);
        for (int s = 1; s < p.splits; ++s) {
          u += *reinterpret_cast<const v4f *>(tp[i] + s * p.M * rt + c);
          v += *reinterpret_cast<const v4f *>(tp[i] + s * p.M * rt + c + 4);
        }
        tv[i] = split8(u, v, g >= 2);
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
  if (16 * g >= cols) return;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + r;
    if (m >= t.rows) continue;
    v4u lo = {0u, 0u, 0u, 0u}, hi = lo;
    if (p.base) {
      const uint16_t *q = p.base + (t.row0 + m) * p.ld_base + n0 + 16 * g;
      lo = *reinterpret_cast<const v4u *>(q);
      hi = *reinterpret_cast<const v4u *>(q + 8);
    }
    if (a >= 0) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = pack_bf16x2(bf16_lo(lo[e]) + acc[i][e >> 1][2 * (e & 1)],
                            bf16_hi(lo[e]) + acc[i][e >> 1][2 * (e & 1) + 1]);
        hi[e] = pack_bf16x2(bf16_lo(hi[e]) + acc[i][2 + (e >> 1)][2 * (e & 1)],
                            bf16_hi(hi[e]) + acc[i][2 + (e >> 1)][2 * (e & 1) + 1]);
      }
    }
    uint16_t *q = p.y + (t.row0 + m) * p.ld_y + n0 + 16 * g;
    *reinterpret_cast<v4u *>(q) = lo;
    *reinterpret_cast<v4u *>(q + 8) = hi;
  }
}

// Launch shape from the sizes the host knows.
struct AdapterPlan {
  int mt, nt, splits;
  int64_t k_per_split;
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
  l.mt = p.M <= 16 * (int64_t)p.n_req ? 1 : 2;
  l.nt = rt <= 16 ? 1 : rt <= 32 ? 2 : 4;
  int64_t groups = tile_bound(p, 16 * l.mt) * ((rt + 16 * l.nt - 1) / (16 * l.nt));
  while (l.nt > 1 && groups < 256) {
    l.nt /= 2;
    groups = tile_bound(p, 16 * l.mt) * ((rt + 16 * l.nt - 1) / (16 * l.nt));
  }
  const int64_t steps = (p.K + 255) / 256;
  l.splits = 1;
  while (l.splits < 4 && groups * l.splits < 256 && steps >= 4 * l.splits) l.splits *= 2;
  l.k_per_split = 256 * ((steps + l.splits - 1) / l.splits);
  l.splits = (int)((p.K + l.k_per_split - 1) / l.k_per_split);
  return l;
}

}  // namespace

size_t adapter_workspace_bytes(const AdapterProblem &p) {
  return sizeof(float) * (size_t)adapter_plan(p).splits * (size_t)p.M * (size_t)p.ns.n *
         (size_t)p.rank;
}

hipError_t launch_adapter(const AdapterProblem &q, hipStream_t s) {
  AdapterProblem p = q;
  const AdapterPlan l = adapter_plan(p);
  p.splits = l.splits;
  p.k_per_split = l.k_per_split;
  const int64_t rt = (int64_t)p.ns.n * p.rank;
  const dim3 shrink((unsigned)tile_bound(p, 16 * l.mt),
                    (unsigned)((rt + 16 * l.nt - 1) / (16 * l.nt)), (unsigned)l.splits);
#define SQ_SHRINK(MT, NT) \
  hipLaunchKernelGGL((adapter_shrink_kernel<MT, NT>), shrink, dim3(256), 0, s, p)
  if (l.mt == 1) {
    if (l.nt == 1) SQ_SHRINK(1, 1);
    else if (l.nt == 2) SQ_SHRINK(1, 2);
    else SQ_SHRINK(1, 4);
  } else {
    if (l.nt == 1) SQ_SHRINK(2, 1);
    else if (l.nt == 2) SQ_SHRINK(2, 2);
    else SQ_SHRINK(2, 4);
  }
#undef SQ_SHRINK
  int64_t tiles = 0;
  for (int i = 0; i < p.ns.n; ++i) tiles += (p.ns.end[i] - p.ns.off[i] + 63) / 64;
  if (l.mt == 1)
    hipLaunchKernelGGL((adapter_expand_kernel<1>),
                       dim3((unsigned)tile_bound(p, 16), (unsigned)((tiles + 3) / 4)), dim3(256),
                       0, s, p);
  else
    hipLaunchKernelGGL((adapter_expand_kernel<4>),
                       dim3((unsigned)tile_bound(p, 64), (unsigned)((tiles + 3) / 4)), dim3(256),
                       0, s, p);
  return hipGetLastError();
}

}  // namespace sq
