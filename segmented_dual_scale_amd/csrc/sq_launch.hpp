// sq_launch.hpp -- host-side launch interface between the C-ABI front end
// (api.cpp) and the kernels.  Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sq {

constexpr int kMaxKSeg = 128;
constexpr int kMaxNSeg = 128;

// A segmented dimension in the form the kernels read from their arguments.
struct SegTable {
  int32_t n;
  int32_t off[kMaxKSeg];
  int32_t end[kMaxKSeg];  // exclusive
};

struct NSegTable {
  int32_t n;
  int32_t off[kMaxNSeg];
  int32_t end[kMaxNSeg];
};

// single: one symmetric scale per segment, written into both halves
hipError_t launch_calibrate(const uint16_t *x, int64_t M, int64_t K, int64_t ld_x,
                            const SegTable &ks, float *act, bool single, hipStream_t s);

// single: both signs quantised with the + half's inverse
hipError_t launch_quantize(const uint16_t *x, int64_t M, int64_t K, int64_t ld_x,
                           const SegTable &ks, const float *act, int8_t *q, int64_t ld_q,
                           int32_t layout, bool single, hipStream_t s);

// act: 1 SiLU, 2 GELU.  q (codes, with scales) and x_out (bf16 activation)
// are each optional; at least one is given.
hipError_t launch_act_quantize(const uint16_t *z, int64_t M, int64_t K, int64_t ld_z, int32_t act,
                               const SegTable &ks, const float *scales, int8_t *q, int64_t ld_q,
                               int32_t layout, uint16_t *x_out, int64_t ld_xo, hipStream_t s);

// w4: 4-bit codes in the nibble layout (K*N/2 bytes) instead of int8
hipError_t launch_quantize_weight(const float *w, int64_t K, int64_t N, int64_t ld_w,
                                  const SegTable &ks, const NSegTable &ns, bool per_column,
                                  int8_t *w_packed, float *w_scale, bool w4, hipStream_t s);

hipError_t launch_unpack_weight(const int8_t *w_packed, int64_t K, int64_t N, int8_t *w_kn,
                                int64_t ld_w, bool w4, hipStream_t s);

// 4-bit packed tiles -> int8 packed tiles (K*N bytes)
hipError_t launch_widen_w4(const int8_t *w4, int64_t K, int64_t N, int8_t *w8, hipStream_t s);

struct GemmProblem {
  int64_t M, N, K;
  const uint16_t *x;
  int64_t ld_x;
  const int8_t *xq;
  int64_t ld_q;
  int32_t q_layout;
  const int8_t *w_packed;
  const float *w_scale;
  const float *act;
  SegTable ks;
  uint16_t *y;
  int64_t ld_y;
  int32_t *acc_debug;
  bool single_scale;  // one product on the signed code, + half's scales only
  bool w4;            // w_packed holds 4-bit codes (small-M streaming kernel only)
};

hipError_t launch_gemm_tile(const GemmProblem &p, hipStream_t s);
hipError_t launch_gemm_smallm(const GemmProblem &p, hipStream_t s);
// the large-M kernel with both operands staged through LDS
hipError_t launch_gemm_lds(const GemmProblem &p, hipStream_t s);

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

constexpr int kSmallMMax = 16;

// Whether the streaming small-M kernel takes this shape (and so reads
// 4-bit weight tiles directly).
bool smallm_reads_w4(int64_t M, int64_t K, int n_kseg, bool bf16_input);

// Output columns per workgroup of the tile kernel for these K-segments.
int tile_columns(const SegTable &ks);
// Whether the tile kernel should run from int8 codes quantised beforehand
// (one extra launch) rather than quantise bf16 input itself.
bool tile_quantize_first(int64_t M, int64_t N, const SegTable &ks);

}  // namespace sq
