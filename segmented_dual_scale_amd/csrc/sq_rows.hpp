// sq_rows.hpp -- what the kernels around the layer share: norm_kernels.hip and
// rmsnorm_kernels.hip (the normalisations that feed it), rotary_kernels.hip (q
// and k behind it) and adapter_kernels.hip (the low-rank adapters beside it).
// First the host-side launch interface of the C-ABI front end (api.cpp), whose
// arguments are already validated; then device helpers.
#pragma once

#include "sq_device.hpp"
#include "sq_launch.hpp"

namespace sq {

// Segment lists of the calls below, small enough to be cheap as kernel
// arguments (a launch with 1.2 KB of them costs the host about 1 us more):
// the ends of the K-segments before the last in steps of 64 columns, of all
// N-segments in steps of 16.
struct KSegEnds {
  int32_t n;
  uint16_t end64[kMaxKSeg];
};

struct NSegEnds {
  int32_t n;
  uint16_t end16[kMaxNSeg];
};

// Where a producer of the layer's input puts it: bf16 x, int8 codes q, or
// both.
struct NormOut {
  uint16_t *x;
  int64_t ld_x;
  int8_t *q;
  int64_t ld_q;
  int64_t plane_stride;  // elements between the + and - planes (0: signed)
  const float *act;      // [4][n_kseg]
  KSegEnds ks;
  bool stream;  // store x past the caches, filled in by the launch
};

struct GroupNormProblem {
  const uint16_t *z;  // [B * P][ld_z]
  int64_t B, P, ld_z;
  int32_t C, G, D;  // channels, groups, channels per group
  float eps;
  const float *gamma, *beta;       // [C], optional
  const uint16_t *scale, *shift;   // [B][ld_mod], optional
  int64_t ld_mod;
  int32_t act;  // 0 none, 1 SiLU, 2 GELU
  NormOut out;
  float *part;  // workspace of the two-launch form
  // launch shape, filled in by the launch
  int32_t groups_per_block, rows_per_block, n_row_blocks, cols_per_block, parts, rows_per_part;
};

hipError_t launch_groupnorm(const GroupNormProblem &p, hipStream_t s);
// Bytes of `part` the launch needs (B, P, C, G and D of the problem decide).
size_t groupnorm_workspace_bytes(const GroupNormProblem &p);

struct AdaNormProblem {
  const uint16_t *h;
  int64_t M, K, ld_h;
  const uint16_t *branch, *gate;  // optional: h' = h + gate * branch
  int64_t ld_b;
  uint16_t *h_out;
  int64_t ld_ho;
  float eps;
  const float *gamma, *beta;      // [K], optional
  const uint16_t *scale, *shift;  // [n_req][ld_mod], as gate; optional
  int64_t ld_mod;
  const int32_t *row_offset;  // device [n_req + 1], or null: equal requests
  int32_t n_req;
  int64_t rows_per_req;
  NormOut out;
  int64_t rows_per;  // rows a row group walks, filled in by the launch
};

hipError_t launch_adanorm(const AdaNormProblem &p, hipStream_t s);

// MXFP4 rows (sq_mx.hpp); codes null: none.
struct MxOut {
  uint8_t *codes, *scales;
  int64_t kt, ks;  // tiles along K of the codes, of the scales
};

struct RmsNormProblem {
  const uint16_t *h;
  int64_t M, K, ld_h;
  const uint16_t *branch;  // optional: h' = h + branch
  int64_t ld_b;
  uint16_t *h_out;
  int64_t ld_ho;
  float eps;
  const float *gamma;  // [K], optional
  NormOut out;
  MxOut mx;
  int64_t rows_per;  // rows a row group walks, filled in by the launch
};

hipError_t launch_rmsnorm(const RmsNormProblem &p, hipStream_t s);

// q or k: elements between samples, tokens and heads
struct RotaryTensor {
  const uint16_t *in;
  uint16_t *out;
  int64_t in_stride[3], out_stride[3];
  const float *gamma;  // [D], optional
  int32_t heads;
};

constexpr int kMaxAxes = 8;

struct RotaryProblem {
  int64_t B, L;
  int32_t D, R;  // head width, its first R elements turn
  RotaryTensor q, k;
  bool norm, halves;
  float eps;
  const int32_t *positions;  // [L][n_axes], or one such table per sample
  int64_t pos_batch;         // elements between samples, 0: shared
  const double *freq;        // [R / 2]
  int32_t n_axes;
  int32_t axis_end[kMaxAxes];  // in pairs
  int32_t q_chunks, chunks;  // waves per token for q, for both; filled in by the launch
};

hipError_t launch_rotary(const RotaryProblem &p, hipStream_t s);

struct AdapterProblem {
  int64_t M, N, K;
  const uint16_t *x;
  int64_t ld_x;
  const int32_t *row_offset;  // device [n_req + 1]
  const int32_t *adapter;     // device [n_req]
  int32_t n_req, n_adapters, rank;
  const int32_t *rank_of;  // device [n_adapters], optional
  const uint16_t *a;       // [n_adapters][ns.n * rank][K]
  const uint16_t *b;       // [n_adapters][N][rank]
  const float *alpha;      // device [n_adapters], optional
  NSegEnds ns;
  const uint16_t *base;  // optional; may be y
  int64_t ld_base;
  uint16_t *y;
  int64_t ld_y;
  float *t;  // workspace [splits][ns.n * rank / 16][M][16]
  // launch shape, filled in by adapter_plan
  bool one;                // one launch, no t in memory
  bool by_row;             // tiles numbered by their first rows
  int32_t mt, nt, splits;  // shrink: blocks of 16 rows, of 16 ranks, parts of K
  int64_t k_per_split;
  int32_t expand_mt, run_tiles;  // second product: blocks of 16 rows, of 64 columns
};

// Choose the launch shape from the sizes (M, N, K, n_req, rank and the
// segments) and return the bytes of `t` it needs.
size_t adapter_plan(AdapterProblem &p);
// Launch a planned problem.
hipError_t launch_adapter(const AdapterProblem &p, hipStream_t s);

// The same rounding by the hardware's packed conversion (RNE; NaN stays NaN).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  typedef float v2f __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2bf));
}

// x / d for 0 <= x < 2^24 and d >= 1, from the reciprocal with a correction:
// a quarter of the instructions of an integer division.
__device__ __forceinline__ int div24(int x, int d) {
  int q = (int)((float)x * __builtin_amdgcn_rcpf((float)d));
  const int r = x - q * d;
  q -= r < 0 ? 1 : 0;
  q += r >= d ? 1 : 0;
  return q;
}

// Request of a row in a packed batch: off[0..n] are row offsets, request i
// holds rows off[i] .. off[i+1]-1.  req is the number of off[1..n] that are
// <= row: -1 for a row before off[0], n behind off[n]; end is the first row
// after the request.  One wave asks about one row, 64 offsets a step, each step
// leaving a 64th.  Whatever off holds, only off[0..n] is read.
struct RowRequest {
  int32_t req;
  int64_t end;
};

__device__ __forceinline__ RowRequest find_request(const int32_t *off, int32_t n, int64_t row) {
  const int lane = threadIdx.x & 63;
  int base = 0, limit = n;  // off[1..base] <= row; off beyond limit > row
  while (limit - base > 64) {
    const int step = (limit - base + 63) / 64, at = base + (lane + 1) * step;
    const int32_t v = off[min(at, limit)];
    base += __popcll(__ballot(at <= limit && v <= row)) * step;
    limit = min(base + step, limit);
  }
  const int at = base + 1 + lane;
  const int32_t v = off[min(at, limit)];
  int req = base + __popcll(__ballot(at <= limit && v <= row));
  req = __builtin_amdgcn_readfirstlane(req);
  RowRequest r;
  r.end = off[min(req + 1, n)];
  r.req = off[0] <= row ? req : -1;
  return r;
}

}  // namespace sq
