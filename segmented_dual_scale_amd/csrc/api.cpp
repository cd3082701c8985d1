// api.cpp -- the C ABI of libsegquant (declared in include/segquant.h):
// argument validation, segment tables, kernel choice and launch.
//
// Every check runs before the first HIP call, so an invalid call enqueues
// nothing, touches no buffer and behaves the same on a machine without a
// GPU.  Errors are returned as status codes with a thread-local detail text;
// nothing is thrown across the ABI.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/segquant.h"
#include "sq_api.hpp"
#include "sq_launch.hpp"
#include "sq_rows.hpp"

namespace {

thread_local std::string g_err;

int vfail(int status, const char *fmt, va_list ap) {
  char buf[512];
  vsnprintf(buf, sizeof buf, fmt, ap);
  g_err = buf;
  return status;
}

int fail(int status, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  const int r = vfail(status, fmt, ap);
  va_end(ap);
  return r;
}

int ok() {
  g_err.clear();
  return SEGQ_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kI32Max = 0x7fffffff;

// K-segment list -> kernel table.  require64: every boundary but the end of
// K is a multiple of 64; max_width: 0 for no limit.
int read_kseg(int32_t n, const int32_t *off, const int32_t *wid, int64_t K, int64_t max_width,
              sq::SegTable &t) {
  if (n < 1) return fail(SEGQ_ERR_SEGMENTS, "K-segment count %d < 1", n);
  if (n > SEGQ_MAX_KSEG)
    return fail(SEGQ_ERR_UNSUPPORTED, "K-segment count %d > %d", n, SEGQ_MAX_KSEG);
  if (!off || !wid) return fail(SEGQ_ERR_NULL, "K-segment offset/width array is NULL");
  int64_t at = 0;
  t.n = n;
  for (int32_t i = 0; i < n; ++i) {
    if (off[i] != at)
      return fail(SEGQ_ERR_SEGMENTS, "K-segment %d starts at %d, expected %lld", i, off[i],
                  (long long)at);
    if (wid[i] <= 0) return fail(SEGQ_ERR_SEGMENTS, "K-segment %d has width %d", i, wid[i]);
    if (max_width > 0 && wid[i] > max_width)
      return fail(SEGQ_ERR_UNSUPPORTED, "K-segment %d width %d exceeds %lld (int32 bound)", i,
                  wid[i], (long long)max_width);
    at += wid[i];
    if (at < K && at % 64 != 0)
      return fail(SEGQ_ERR_ALIGN, "K-segment boundary %lld is not a multiple of 64",
                  (long long)at);
    t.off[i] = off[i];
    t.end[i] = (int32_t)at;
  }
  if (at != K)
    return fail(SEGQ_ERR_SEGMENTS, "K-segments cover %lld columns, K is %lld", (long long)at,
                (long long)K);
  return SEGQ_OK;
}

int read_nseg(int32_t n, const int32_t *off, const int32_t *wid, int64_t N, sq::NSegTable &t) {
  if (n < 1) return fail(SEGQ_ERR_SEGMENTS, "N-segment count %d < 1", n);
  if (n > sq::kMaxNSeg) return fail(SEGQ_ERR_UNSUPPORTED, "N-segment count %d > %d", n, sq::kMaxNSeg);
  if (!off || !wid) return fail(SEGQ_ERR_NULL, "N-segment offset/width array is NULL");
  int64_t at = 0;
  t.n = n;
  for (int32_t i = 0; i < n; ++i) {
    if (off[i] != at)
      return fail(SEGQ_ERR_SEGMENTS, "N-segment %d starts at %d, expected %lld", i, off[i],
                  (long long)at);
    if (wid[i] <= 0) return fail(SEGQ_ERR_SEGMENTS, "N-segment %d has width %d", i, wid[i]);
    at += wid[i];
    t.off[i] = off[i];
    t.end[i] = (int32_t)at;
  }
  if (at != N)
    return fail(SEGQ_ERR_SEGMENTS, "N-segments cover %lld columns, N is %lld", (long long)at,
                (long long)N);
  return SEGQ_OK;
}

int check_x(const uint16_t *x, int64_t M, int64_t K, int64_t ld_x) {
  if (M < 0 || K < 1 || M > kI32Max || K > kI32Max)
    return fail(SEGQ_ERR_SHAPE, "bad shape M=%lld K=%lld", (long long)M, (long long)K);
  if (ld_x < K) return fail(SEGQ_ERR_SHAPE, "ld_x %lld < K %lld", (long long)ld_x, (long long)K);
  if (M > 0 && !x) return fail(SEGQ_ERR_NULL, "x_bf16 is NULL");
  if (ld_x % 8 != 0) return fail(SEGQ_ERR_ALIGN, "ld_x %lld is not a multiple of 8", (long long)ld_x);
  if (x && !aligned16(x)) return fail(SEGQ_ERR_ALIGN, "x_bf16 is not 16-byte aligned");
  return SEGQ_OK;
}

int hip_status(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(SEGQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

// ------------------------------------------- operands that share memory --
typedef __int128 I128;  // leading dimensions have no upper limit

I128 floor_div(I128 a, I128 b) {  // b > 0
  return a / b - (a % b < 0 ? 1 : 0);
}

// Sum of floor((a i + b) / m) over 0 <= i < n, for a, b >= 0 and m > 0: whole
// multiples of m taken out, then the same count seen along the other axis, as
// in Euclid's algorithm.  Modulo 2^128.
unsigned __int128 floor_sum(unsigned __int128 n, unsigned __int128 m, unsigned __int128 a,
                                   unsigned __int128 b) {
  unsigned __int128 sum = 0;
  while (n > 0) {
    sum += (n % 2 ? (n - 1) / 2 * n : n / 2 * (n - 1)) * (a / m) + n * (b / m);
    const unsigned __int128 top = a % m * n + b % m;
    n = top / m;
    b = top % m;
    const unsigned __int128 t = m;
    m = a % m;
    a = t;
    if (!m) break;
  }
  return sum;
}

// Rows of `width` bytes, `ld` bytes apart.
struct Rows {
  const void *at;
  I128 ld, width;
  int64_t n;
  bool empty() const { return !at || width < 1 || n < 1; }
};

Rows bf16_rows(const uint16_t *p, int64_t ld, int64_t width, int64_t n) {
  return {p, 2 * (I128)ld, 2 * (I128)width, n};
}

Rows one_run(const void *p, I128 bytes) { return {p, bytes, bytes, 1}; }

// Whether two matrices share bytes; they may stand side by side in one buffer.
// Rows i and j share some where 0 < i ld_p - d + w_p - j ld_q < w_p + w_q.  The
// number of steps grows as the logarithm of the leading dimensions.
bool rows_meet(const Rows &p, const Rows &q) {
  if (p.empty() || q.empty()) return false;
  const I128 d = (I128)reinterpret_cast<uintptr_t>(q.at) - (I128)reinterpret_cast<uintptr_t>(p.at);
  const I128 q_end = d + (q.n - 1) * q.ld;  // q's last row
  if (d >= (p.n - 1) * p.ld + p.width || q_end + q.width <= 0) return false;
  // the rows of p that meet a row of q at `at`
  auto met = [&](I128 at) {
    I128 first = floor_div(at - p.width, p.ld) + 1, last = floor_div(at + q.width - 1, p.ld);
    if (first < 0) first = 0;
    if (last > p.n - 1) last = p.n - 1;
    return first <= last;
  };
  if (met(d) || met(q_end)) return true;
  // any other meeting is with rows of p between these two, where the rows j of
  // q that row i meets are counted without a look at q's ends
  I128 first = floor_div(d + q.width - 1, p.ld) + 1, last = floor_div(q_end - p.width, p.ld);
  if (first < 0) first = 0;
  if (last > p.n - 1) last = p.n - 1;
  if (first > last) return false;
  const I128 start = first * p.ld - d, a = p.ld % q.ld;
  return floor_sum(last - first + 1, q.ld, a, start + p.width - 1) !=
         floor_sum(last - first + 1, q.ld, a, start - q.width);
}

// An operand of a call.  For an input, the outputs (bit i: the i'th) that may be
// the input itself, where every element is read before it is written.
struct Operand {
  const char *name;
  Rows rows;
  unsigned in_place;
};

// Refuse a call whose outputs share bytes with each other or with an input.
template <size_t NOut, size_t NIn>
int check_apart(const Operand (&outs)[NOut], const Operand (&ins)[NIn]) {
  const Operand *all[NOut + NIn];
  I128 at[NOut + NIn], end[NOut + NIn];
  for (size_t i = 0; i < NOut + NIn; ++i) {
    all[i] = i < NOut ? &outs[i] : &ins[i - NOut];
    const Rows &r = all[i]->rows;
    at[i] = (I128)reinterpret_cast<uintptr_t>(r.at);
    end[i] = r.empty() ? at[i] : at[i] + (r.n - 1) * r.ld + r.width;
  }
  for (size_t i = 0; i < NOut; ++i)
    for (size_t j = i + 1; j < NOut + NIn; ++j) {
      if (end[i] <= at[j] || end[j] <= at[i]) continue;
      const Rows &out = all[i]->rows, &in = all[j]->rows;
      if (j >= NOut && (all[j]->in_place >> i & 1) && out.at == in.at && out.ld == in.ld) continue;
      if (rows_meet(out, in))
        return fail(SEGQ_ERR_SHAPE, "%s overlaps %s", all[i]->name, all[j]->name);
    }
  return SEGQ_OK;
}

// The codes a call writes, and the scales it reads for them.
Rows code_rows(const sq::NormOut &o, int64_t M, int64_t K) {
  return {o.q, o.ld_q, K, o.plane_stride ? 2 * M : M};
}

Rows scale_rows(const sq::NormOut &o) {
  return one_run(o.q ? o.act : nullptr, 4 * (I128)sizeof(float) * o.ks.n);
}

}  // namespace

namespace sq {

int api_fail(int status, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  const int r = vfail(status, fmt, ap);
  va_end(ap);
  return r;
}

int api_hip_status(hipError_t e, const char *what) { return hip_status(e, what); }

static int gemm_check_shape(int64_t M, int64_t N, int64_t K, uint32_t flags);

int gemm_validate(const GemmCall &c, SegTable &ks) {
  int st = gemm_check_shape(c.M, c.N, c.K, c.flags);
  if (st) return st;
  if (c.M > 0) {
    if ((c.x != nullptr) == (c.xq != nullptr))
      return fail(SEGQ_ERR_NULL, "exactly one of x_bf16 and xq must be given");
    if (c.x) {
      if ((st = check_x(c.x, c.M, c.K, c.ld_x))) return st;
    } else {
      if (c.q_layout != SEGQ_Q_SIGNED && c.q_layout != SEGQ_Q_PLANES)
        return fail(SEGQ_ERR_SHAPE, "unknown q_layout %d", c.q_layout);
      if (c.q_layout == SEGQ_Q_PLANES && (c.flags & SEGQ_GEMM_SINGLE_SCALE))
        return fail(SEGQ_ERR_UNSUPPORTED, "the single-scale product takes bf16 or signed-code input");
      if (c.ld_q < c.K)
        return fail(SEGQ_ERR_SHAPE, "ld_q %lld < K %lld", (long long)c.ld_q, (long long)c.K);
      if (c.ld_q % 16 != 0)
        return fail(SEGQ_ERR_ALIGN, "ld_q %lld is not a multiple of 16", (long long)c.ld_q);
      if (!aligned16(c.xq)) return fail(SEGQ_ERR_ALIGN, "xq is not 16-byte aligned");
    }
    if (!c.w_packed || !c.w_scale || !c.act || !c.y)
      return fail(SEGQ_ERR_NULL, "w_packed, w_scale, act_scales or y_bf16 is NULL");
    if (!aligned16(c.w_packed)) return fail(SEGQ_ERR_ALIGN, "w_packed is not 16-byte aligned");
    if (c.ld_y < c.N)
      return fail(SEGQ_ERR_SHAPE, "ld_y %lld < N %lld", (long long)c.ld_y, (long long)c.N);
    if ((reinterpret_cast<uintptr_t>(c.y) & 1u) ||
        (c.acc && (reinterpret_cast<uintptr_t>(c.acc) & 3u)))
      return fail(SEGQ_ERR_ALIGN, "y_bf16 or acc_debug is misaligned");
  }
  if ((st = read_kseg(c.n_kseg, c.kseg_offset, c.kseg_width, c.K, SEGQ_MAX_KSEG_WIDTH, ks)))
    return st;
  return ok();
}

static bool quantize_first(int kernel, int64_t M, int64_t N, const sq::SegTable &ks,
                           uint32_t flags);
static size_t w4_widen_bytes(int kernel, int64_t M, int64_t N, int64_t K, const sq::SegTable &ks,
                             uint32_t flags, bool bf16_input);

size_t gemm_workspace_need(const GemmCall &c, const SegTable &ks, uint32_t flags) {
  const int kernel = segquant_gemm_kernel_for(c.M, c.N, c.K, flags);
  return w4_widen_bytes(kernel, c.M, c.N, c.K, ks, flags, c.x != nullptr) +
         (c.x && quantize_first(kernel, c.M, c.N, ks, flags) ? (size_t)(c.M * c.K) : 0);
}

int gemm_enqueue(const GemmCall &c, const SegTable &ks, void *workspace, size_t workspace_bytes) {
  if (c.M == 0) return ok();
  const int64_t M = c.M, N = c.N, K = c.K;
  const uint32_t flags = c.flags;
  sq::GemmProblem p{};
  p.M = M; p.N = N; p.K = K;
  p.x = c.x; p.ld_x = c.ld_x;
  p.xq = c.xq; p.ld_q = c.ld_q; p.q_layout = c.q_layout;
  p.w_packed = c.w_packed; p.w_scale = c.w_scale; p.act = c.act;
  p.ks = ks;
  p.y = c.y; p.ld_y = c.ld_y; p.acc_debug = c.acc;
  p.single_scale = (flags & SEGQ_GEMM_SINGLE_SCALE) != 0;
  hipStream_t stream = (hipStream_t)c.stream;
  const int kernel = segquant_gemm_kernel_for(M, N, K, flags);
  // 4-bit weights: the streaming small-M kernel reads them as they are;
  // every other path first widens them to int8 tiles in the workspace
  const size_t widen = w4_widen_bytes(kernel, M, N, K, ks, flags, c.x != nullptr);
  if (widen && (!workspace || workspace_bytes < widen))
    return fail(SEGQ_ERR_UNSUPPORTED,
                "4-bit weights on this shape need a workspace of at least %zu bytes "
                "(segquant_gemm_workspace_bytes)", widen);
  p.w4 = (flags & SEGQ_GEMM_W4) && !widen;
  if (widen) {
    int8_t *w8 = static_cast<int8_t *>(workspace);
    hipError_t e = sq::launch_widen_w4(c.w_packed, K, N, w8, stream);
    if (e != hipSuccess) return hip_status(e, "widen launch");
    p.w_packed = w8;
  }
  uint8_t *ws_rest = workspace ? static_cast<uint8_t *>(workspace) + widen : nullptr;
  const size_t ws_rest_bytes = workspace ? workspace_bytes - widen : 0;
  if (c.x && ws_rest && quantize_first(kernel, M, N, ks, flags) &&
      ws_rest_bytes >= (size_t)(M * K)) {
    // quantise once into the workspace, then the GEMM from the signed codes
    int8_t *codes = reinterpret_cast<int8_t *>(ws_rest);
    hipError_t e = sq::launch_quantize(c.x, M, K, c.ld_x, ks, c.act, codes, K, SEGQ_Q_SIGNED,
                                       p.single_scale, stream);
    if (e != hipSuccess) return hip_status(e, "quantize launch");
    p.x = nullptr;
    p.ld_x = 0;
    p.xq = codes;
    p.ld_q = K;
    p.q_layout = SEGQ_Q_SIGNED;
  }
  hipError_t e = kernel == SEGQ_KERNEL_SMALLM ? sq::launch_gemm_smallm(p, stream)
                                              : sq::launch_gemm_tile(p, stream);
  return hip_status(e, "gemm launch");
}

}  // namespace sq

extern "C" {

const char *segquant_status_string(int status) {
  switch (status) {
    case SEGQ_OK: return "ok";
    case SEGQ_ERR_NULL: return "null pointer";
    case SEGQ_ERR_SHAPE: return "invalid shape";
    case SEGQ_ERR_SEGMENTS: return "invalid segment list";
    case SEGQ_ERR_ALIGN: return "misaligned size, boundary or pointer";
    case SEGQ_ERR_UNSUPPORTED: return "unsupported (beyond library limits)";
    case SEGQ_ERR_HIP: return "HIP runtime error";
    default: return "unknown status";
  }
}

const char *segquant_last_error(void) { return g_err.c_str(); }

int segquant_version(void) { return 110; }

size_t segquant_weight_packed_bytes_w4(int64_t K, int64_t N) {
  return segquant_weight_packed_bytes(K, N) / 2;
}

size_t segquant_weight_packed_bytes(int64_t K, int64_t N) {
  if (K < 64 || N < 16 || K % 64 || N % 16 || K > kI32Max || N > kI32Max) return 0;
  return (size_t)K * (size_t)N;
}

static int calibrate(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x, int32_t n_kseg,
                     const int32_t *kseg_offset, const int32_t *kseg_width, float *act_scales,
                     bool single, void *stream) {
  int st = check_x(x_bf16, M, K, ld_x);
  if (st) return st;
  if (!act_scales) return fail(SEGQ_ERR_NULL, "act_scales is NULL");
  sq::SegTable ks{};
  if ((st = read_kseg(n_kseg, kseg_offset, kseg_width, K, 0, ks))) return st;
  return hip_status(
      sq::launch_calibrate(x_bf16, M, K, ld_x, ks, act_scales, single, (hipStream_t)stream),
      "calibrate launch");
}

int segquant_calibrate_amax(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x,
                            int32_t n_kseg, const int32_t *kseg_offset,
                            const int32_t *kseg_width, float *act_scales, void *stream) {
  return calibrate(x_bf16, M, K, ld_x, n_kseg, kseg_offset, kseg_width, act_scales, false, stream);
}

int segquant_calibrate_amax_single(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x,
                                   int32_t n_kseg, const int32_t *kseg_offset,
                                   const int32_t *kseg_width, float *act_scales, void *stream) {
  return calibrate(x_bf16, M, K, ld_x, n_kseg, kseg_offset, kseg_width, act_scales, true, stream);
}

int segquant_quantize_dualscale(const uint16_t *x_bf16, int64_t M, int64_t K, int64_t ld_x,
                                int32_t n_kseg, const int32_t *kseg_offset,
                                const int32_t *kseg_width, const float *act_scales,
                                int8_t *q_out, int64_t ld_q, int32_t q_layout, void *stream) {
  int st = check_x(x_bf16, M, K, ld_x);
  if (st) return st;
  if (!act_scales) return fail(SEGQ_ERR_NULL, "act_scales is NULL");
  if (M > 0 && !q_out) return fail(SEGQ_ERR_NULL, "q_out is NULL");
  if (q_layout != SEGQ_Q_SIGNED && q_layout != SEGQ_Q_PLANES)
    return fail(SEGQ_ERR_SHAPE, "unknown q_layout %d", q_layout);
  if (ld_q < K) return fail(SEGQ_ERR_SHAPE, "ld_q %lld < K %lld", (long long)ld_q, (long long)K);
  if (ld_q % 16 != 0) return fail(SEGQ_ERR_ALIGN, "ld_q %lld is not a multiple of 16", (long long)ld_q);
  if (q_out && !aligned16(q_out)) return fail(SEGQ_ERR_ALIGN, "q_out is not 16-byte aligned");
  sq::SegTable ks{};
  if ((st = read_kseg(n_kseg, kseg_offset, kseg_width, K, 0, ks))) return st;
  return hip_status(sq::launch_quantize(x_bf16, M, K, ld_x, ks, act_scales, q_out, ld_q, q_layout,
                                        false, (hipStream_t)stream),
                    "quantize launch");
}

int segquant_activate_quantize(const uint16_t *z_bf16, int64_t M, int64_t K, int64_t ld_z,
                               int32_t act_kind, int32_t n_kseg, const int32_t *kseg_offset,
                               const int32_t *kseg_width, const float *act_scales,
                               int8_t *q_out, int64_t ld_q, int32_t q_layout, uint16_t *x_out,
                               int64_t ld_xo, void *stream) {
  int st = check_x(z_bf16, M, K, ld_z);
  if (st) return st;
  if (act_kind != SEGQ_ACT_SILU && act_kind != SEGQ_ACT_GELU)
    return fail(SEGQ_ERR_SHAPE, "unknown act_kind %d", act_kind);
  if (!q_out && !x_out) return fail(SEGQ_ERR_NULL, "neither q_out nor x_out is given");
  if (q_out) {
    if (!act_scales) return fail(SEGQ_ERR_NULL, "act_scales is NULL");
    if (q_layout != SEGQ_Q_SIGNED && q_layout != SEGQ_Q_PLANES)
      return fail(SEGQ_ERR_SHAPE, "unknown q_layout %d", q_layout);
    if (ld_q < K) return fail(SEGQ_ERR_SHAPE, "ld_q %lld < K %lld", (long long)ld_q, (long long)K);
    if (ld_q % 16 != 0)
      return fail(SEGQ_ERR_ALIGN, "ld_q %lld is not a multiple of 16", (long long)ld_q);
    if (!aligned16(q_out)) return fail(SEGQ_ERR_ALIGN, "q_out is not 16-byte aligned");
  }
  if (x_out) {
    if (ld_xo < K) return fail(SEGQ_ERR_SHAPE, "ld_xo %lld < K %lld", (long long)ld_xo, (long long)K);
    if (ld_xo % 8 != 0 || !aligned16(x_out))
      return fail(SEGQ_ERR_ALIGN, "x_out must be 16-byte aligned with ld_xo a multiple of 8");
  }
  sq::SegTable ks{};
  if ((st = read_kseg(n_kseg, kseg_offset, kseg_width, K, 0, ks))) return st;
  return hip_status(sq::launch_act_quantize(z_bf16, M, K, ld_z, act_kind, ks, act_scales, q_out,
                                            ld_q, q_layout, x_out, ld_xo, (hipStream_t)stream),
                    "activate-quantize launch");
}

// The outputs shared by the calls that produce a layer's input: int8 codes
// (with their scales), bf16 x, or both, of M rows of K columns.
static int check_norm_out(int64_t M, int64_t K, int32_t n_kseg, const int32_t *kseg_offset,
                          const int32_t *kseg_width, const float *act_scales, int8_t *q_out,
                          int64_t ld_q, int32_t q_layout, uint16_t *x_out, int64_t ld_xo,
                          sq::NormOut &o) {
  if (q_out) {
    if (!act_scales) return fail(SEGQ_ERR_NULL, "act_scales is NULL");
    if (q_layout != SEGQ_Q_SIGNED && q_layout != SEGQ_Q_PLANES)
      return fail(SEGQ_ERR_SHAPE, "unknown q_layout %d", q_layout);
    if (ld_q < K) return fail(SEGQ_ERR_SHAPE, "ld_q %lld < K %lld", (long long)ld_q, (long long)K);
    if (ld_q % 16 != 0)
      return fail(SEGQ_ERR_ALIGN, "ld_q %lld is not a multiple of 16", (long long)ld_q);
    if (!aligned16(q_out)) return fail(SEGQ_ERR_ALIGN, "q_out is not 16-byte aligned");
  }
  if (x_out) {
    if (ld_xo < K) return fail(SEGQ_ERR_SHAPE, "ld_xo %lld < K %lld", (long long)ld_xo, (long long)K);
    if (ld_xo % 8 != 0 || !aligned16(x_out))
      return fail(SEGQ_ERR_ALIGN, "x_out must be 16-byte aligned with ld_xo a multiple of 8");
  }
  o.x = x_out;
  o.ld_x = ld_xo;
  o.q = q_out;
  o.ld_q = ld_q;
  o.plane_stride = q_layout == SEGQ_Q_PLANES ? M * ld_q : 0;
  o.act = act_scales;
  sq::SegTable ks{};
  const int st = read_kseg(n_kseg, kseg_offset, kseg_width, K, 0, ks);
  if (st) return st;
  o.ks.n = ks.n;
  for (int32_t i = 0; i + 1 < ks.n; ++i) {
    if (ks.end[i] / 64 > 0xffff)
      return fail(SEGQ_ERR_UNSUPPORTED, "K-segment boundary %d is beyond %d", ks.end[i],
                  64 * 0xffff);
    o.ks.end64[i] = (uint16_t)(ks.end[i] / 64);
  }
  return SEGQ_OK;
}

// An optional bf16 matrix: pointer, leading dimension, row length.
static int check_rows(const uint16_t *p, int64_t ld, int64_t len, const char *what) {
  if (!p) return SEGQ_OK;
  if (ld < len)
    return fail(SEGQ_ERR_SHAPE, "%s: leading dimension %lld < %lld", what, (long long)ld,
                (long long)len);
  if (ld % 8 != 0 || !aligned16(p))
    return fail(SEGQ_ERR_ALIGN, "%s must be 16-byte aligned with a leading dimension that is a "
                "multiple of 8", what);
  return SEGQ_OK;
}

static int check_norm_params(const float *gamma, const float *beta, float eps) {
  if (!(eps >= 1.17549435e-38f) || eps > 3.0e38f)
    return fail(SEGQ_ERR_SHAPE, "eps must be positive, finite and at least 2^-126");
  if (!aligned16(gamma) || !aligned16(beta))
    return fail(SEGQ_ERR_ALIGN, "gamma or beta is not 16-byte aligned");
  return SEGQ_OK;
}

static int groupnorm_sizes(int64_t B, int64_t P, int64_t C, int32_t groups,
                           sq::GroupNormProblem &p) {
  if (B < 0 || P < 0 || C < 1 || B > kI32Max || P > kI32Max || C > kI32Max ||
      (P > 0 && B > kI32Max / P))
    return fail(SEGQ_ERR_SHAPE, "bad shape B=%lld P=%lld C=%lld", (long long)B, (long long)P,
                (long long)C);
  if (groups < 1 || C % groups != 0)
    return fail(SEGQ_ERR_SHAPE, "%d groups do not divide %lld channels", groups, (long long)C);
  if (C > (1 << 20) || B > 65535)
    return fail(SEGQ_ERR_UNSUPPORTED, "C %lld > 2^20 or B %lld > 65535", (long long)C,
                (long long)B);
  p.B = B;
  p.P = P;
  p.C = (int32_t)C;
  p.G = groups;
  p.D = (int32_t)(C / groups);
  return SEGQ_OK;
}

size_t segquant_groupnorm_workspace_bytes(int64_t B, int64_t P, int64_t C, int32_t groups) {
  sq::GroupNormProblem p{};
  if (groupnorm_sizes(B, P, C, groups, p)) return 0;
  ok();
  return B && P ? sq::groupnorm_workspace_bytes(p) : 0;
}

int segquant_groupnorm_quantize(const uint16_t *z_bf16, int64_t B, int64_t P, int64_t C,
                                int64_t ld_z, int32_t groups, float eps, const float *gamma,
                                const float *beta, const uint16_t *scale, const uint16_t *shift,
                                int64_t ld_mod, int32_t act_kind, int32_t n_kseg,
                                const int32_t *kseg_offset, const int32_t *kseg_width,
                                const float *act_scales, int8_t *q_out, int64_t ld_q,
                                int32_t q_layout, uint16_t *x_out, int64_t ld_xo, void *workspace,
                                size_t workspace_bytes, void *stream) {
  sq::GroupNormProblem p{};
  int st = groupnorm_sizes(B, P, C, groups, p);
  if (st) return st;
  const int64_t M = B * P;
  if ((st = check_x(z_bf16, M, C, ld_z))) return st;
  if ((st = check_norm_params(gamma, beta, eps))) return st;
  if ((st = check_rows(scale, ld_mod, C, "scale"))) return st;
  if ((st = check_rows(shift, ld_mod, C, "shift"))) return st;
  if (act_kind != SEGQ_ACT_NONE && act_kind != SEGQ_ACT_SILU && act_kind != SEGQ_ACT_GELU)
    return fail(SEGQ_ERR_SHAPE, "unknown act_kind %d", act_kind);
  if (M > 0 && !q_out && !x_out) return fail(SEGQ_ERR_NULL, "neither q_out nor x_out is given");
  if ((st = check_norm_out(M, C, n_kseg, kseg_offset, kseg_width, act_scales, q_out, ld_q, q_layout,
                           x_out, ld_xo, p.out)))
    return st;
  if (x_out && x_out == z_bf16 && ld_xo != ld_z)
    return fail(SEGQ_ERR_SHAPE, "x_out on z_bf16 needs ld_xo = ld_z");
  if (M == 0) return ok();
  const size_t need = sq::groupnorm_workspace_bytes(p);
  if (need && (!workspace || workspace_bytes < need))
    return fail(SEGQ_ERR_UNSUPPORTED,
                "this shape needs a workspace of at least %zu bytes "
                "(segquant_groupnorm_workspace_bytes)", need);
  if (workspace && !aligned16(workspace))
    return fail(SEGQ_ERR_ALIGN, "workspace is not 16-byte aligned");
  const Operand outs[] = {{"x_out", bf16_rows(x_out, ld_xo, C, M)},
                          {"q_out", code_rows(p.out, M, C)},
                          {"workspace", one_run(workspace, need)}};
  const Operand ins[] = {{"z_bf16", bf16_rows(z_bf16, ld_z, C, M), 1},
                         {"gamma", one_run(gamma, sizeof(float) * (I128)C)},
                         {"beta", one_run(beta, sizeof(float) * (I128)C)},
                         {"scale", bf16_rows(scale, ld_mod, C, B)},
                         {"shift", bf16_rows(shift, ld_mod, C, B)},
                         {"act_scales", scale_rows(p.out)}};
  if ((st = check_apart(outs, ins))) return st;
  p.z = z_bf16;
  p.ld_z = ld_z;
  p.eps = eps;
  p.gamma = gamma;
  p.beta = beta;
  p.scale = scale;
  p.shift = shift;
  p.ld_mod = ld_mod;
  p.act = act_kind;
  p.part = static_cast<float *>(workspace);
  return hip_status(sq::launch_groupnorm(p, (hipStream_t)stream), "groupnorm launch");
}

int segquant_adanorm_quantize(const uint16_t *h_bf16, int64_t M, int64_t K, int64_t ld_h,
                              const uint16_t *branch, int64_t ld_b, const uint16_t *gate,
                              uint16_t *h_out, int64_t ld_ho, float eps, const float *gamma,
                              const float *beta, const uint16_t *scale, const uint16_t *shift,
                              int64_t ld_mod, int32_t n_req, const int32_t *row_offset,
                              int32_t n_kseg, const int32_t *kseg_offset,
                              const int32_t *kseg_width, const float *act_scales, int8_t *q_out,
                              int64_t ld_q, int32_t q_layout, uint16_t *x_out, int64_t ld_xo,
                              void *stream) {
  sq::AdaNormProblem p{};
  int st = check_x(h_bf16, M, K, ld_h);
  if (st) return st;
  if (n_req < 1) return fail(SEGQ_ERR_SHAPE, "n_req %d < 1", n_req);
  if (!row_offset && M % n_req != 0)
    return fail(SEGQ_ERR_SHAPE, "%d equal requests do not divide %lld rows", n_req, (long long)M);
  if (reinterpret_cast<uintptr_t>(row_offset) & 3u)
    return fail(SEGQ_ERR_ALIGN, "row_offset is not 4-byte aligned");
  if (!branch && (gate || h_out)) return fail(SEGQ_ERR_NULL, "gate or h_out without branch");
  if ((st = check_norm_params(gamma, beta, eps))) return st;
  if ((st = check_rows(branch, ld_b, K, "branch"))) return st;
  if ((st = check_rows(h_out, ld_ho, K, "h_out"))) return st;
  if ((st = check_rows(gate, ld_mod, K, "gate"))) return st;
  if ((st = check_rows(scale, ld_mod, K, "scale"))) return st;
  if ((st = check_rows(shift, ld_mod, K, "shift"))) return st;
  if (h_out && h_out == h_bf16 && ld_ho != ld_h)
    return fail(SEGQ_ERR_SHAPE, "h_out on h_bf16 needs ld_ho = ld_h");
  if (M > 0 && !q_out && !x_out && !h_out)
    return fail(SEGQ_ERR_NULL, "none of q_out, x_out and h_out is given");
  if ((st = check_norm_out(M, K, n_kseg, kseg_offset, kseg_width, act_scales, q_out, ld_q, q_layout,
                           x_out, ld_xo, p.out)))
    return st;
  if (M == 0) return ok();
  const Operand outs[] = {{"h_out", bf16_rows(h_out, ld_ho, K, M)},
                          {"x_out", bf16_rows(x_out, ld_xo, K, M)},
                          {"q_out", code_rows(p.out, M, K)}};
  const Operand ins[] = {{"h_bf16", bf16_rows(h_bf16, ld_h, K, M), 1},
                         {"branch", bf16_rows(branch, ld_b, K, M), 1},
                         {"gate", bf16_rows(gate, ld_mod, K, n_req)},
                         {"scale", bf16_rows(scale, ld_mod, K, n_req)},
                         {"shift", bf16_rows(shift, ld_mod, K, n_req)},
                         {"gamma", one_run(gamma, sizeof(float) * (I128)K)},
                         {"beta", one_run(beta, sizeof(float) * (I128)K)},
                         {"row_offset", one_run(row_offset, sizeof(int32_t) * ((I128)n_req + 1))},
                         {"act_scales", scale_rows(p.out)}};
  if ((st = check_apart(outs, ins))) return st;
  p.h = h_bf16;
  p.M = M;
  p.K = K;
  p.ld_h = ld_h;
  p.branch = branch;
  p.gate = gate;
  p.ld_b = ld_b;
  p.h_out = h_out;
  p.ld_ho = ld_ho;
  p.eps = eps;
  p.gamma = gamma;
  p.beta = beta;
  p.scale = scale;
  p.shift = shift;
  p.ld_mod = ld_mod;
  p.row_offset = row_offset;
  p.n_req = n_req;
  p.rows_per_req = M / n_req;
  return hip_status(sq::launch_adanorm(p, (hipStream_t)stream), "adanorm launch");
}

static int adapter_sizes(int64_t M, int64_t N, int64_t K, int32_t n_req, int32_t rank,
                         int32_t n_nseg, sq::AdapterProblem &p) {
  if (M < 0 || N < 1 || K < 1 || M > kI32Max || N > kI32Max || K > kI32Max)
    return fail(SEGQ_ERR_SHAPE, "bad shape M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                (long long)K);
  if (K % 64 || N % 16)
    return fail(SEGQ_ERR_ALIGN, "adapters need K %% 64 == 0 and N %% 16 == 0 (K=%lld N=%lld)",
                (long long)K, (long long)N);
  if (M > (1 << 27) || n_req > (1 << 22) || N > 16 * 0xffff)
    return fail(SEGQ_ERR_UNSUPPORTED, "M %lld > 2^27, n_req %d > 2^22 or N %lld > %d", (long long)M,
                n_req, (long long)N, 16 * 0xffff);
  if (n_req < 1) return fail(SEGQ_ERR_SHAPE, "n_req %d < 1", n_req);
  if (rank < 1 || rank % SEGQ_ADAPTER_RANK_STEP)
    return fail(SEGQ_ERR_ALIGN, "rank %d is not a multiple of %d", rank, SEGQ_ADAPTER_RANK_STEP);
  if (rank > SEGQ_ADAPTER_RANK_MAX)
    return fail(SEGQ_ERR_UNSUPPORTED, "rank %d > %d", rank, SEGQ_ADAPTER_RANK_MAX);
  if (n_nseg < 1) return fail(SEGQ_ERR_SEGMENTS, "N-segment count %d < 1", n_nseg);
  if (n_nseg > sq::kMaxNSeg)
    return fail(SEGQ_ERR_UNSUPPORTED, "N-segment count %d > %d", n_nseg, sq::kMaxNSeg);
  p.M = M;
  p.N = N;
  p.K = K;
  p.n_req = n_req;
  p.rank = rank;
  p.ns.n = n_nseg;
  return SEGQ_OK;
}

static int adapter_segments(int32_t n_nseg, const int32_t *nseg_offset, const int32_t *nseg_width,
                            int64_t N, sq::AdapterProblem &p) {
  sq::NSegTable ns{};
  const int st = read_nseg(n_nseg, nseg_offset, nseg_width, N, ns);
  if (st) return st;
  for (int32_t i = 0; i < ns.n; ++i) {
    if (ns.off[i] % 16)
      return fail(SEGQ_ERR_ALIGN, "N-segment boundary %d is not a multiple of 16", ns.off[i]);
    p.ns.end16[i] = (uint16_t)(ns.end[i] / 16);
  }
  return SEGQ_OK;
}

size_t segquant_adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t n_req,
                                        int32_t rank, int32_t n_nseg, const int32_t *nseg_offset,
                                        const int32_t *nseg_width) {
  sq::AdapterProblem p{};
  if (adapter_sizes(M, N, K, n_req, rank, n_nseg, p) ||
      adapter_segments(n_nseg, nseg_offset, nseg_width, N, p))
    return 0;
  ok();
  return M ? sq::adapter_plan(p) : 0;
}

int segquant_adapter_add(int64_t M, int64_t N, int64_t K, const uint16_t *x_bf16, int64_t ld_x,
                         int32_t n_req, const int32_t *row_offset, const int32_t *adapter,
                         int32_t n_adapters, int32_t rank, const int32_t *rank_of,
                         const uint16_t *a, const uint16_t *b, const float *alpha, int32_t n_nseg,
                         const int32_t *nseg_offset, const int32_t *nseg_width,
                         const uint16_t *base_bf16, int64_t ld_base, uint16_t *y_bf16,
                         int64_t ld_y, void *workspace, size_t workspace_bytes, void *stream) {
  sq::AdapterProblem p{};
  int st = adapter_sizes(M, N, K, n_req, rank, n_nseg, p);
  if (st) return st;
  if (n_adapters < 1) return fail(SEGQ_ERR_SHAPE, "n_adapters %d < 1", n_adapters);
  if ((st = check_x(x_bf16, M, K, ld_x))) return st;
  if ((st = adapter_segments(n_nseg, nseg_offset, nseg_width, N, p))) return st;
  if (M == 0) return ok();
  if (!row_offset || !adapter || !a || !b || !y_bf16)
    return fail(SEGQ_ERR_NULL, "row_offset, adapter, a, b or y_bf16 is NULL");
  if (!aligned16(a) || !aligned16(b)) return fail(SEGQ_ERR_ALIGN, "a or b is not 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(row_offset) | reinterpret_cast<uintptr_t>(adapter) |
       reinterpret_cast<uintptr_t>(rank_of) | reinterpret_cast<uintptr_t>(alpha)) & 3u)
    return fail(SEGQ_ERR_ALIGN, "row_offset, adapter, rank_of or alpha is not 4-byte aligned");
  if ((st = check_rows(base_bf16, ld_base, N, "base_bf16"))) return st;
  if ((st = check_rows(y_bf16, ld_y, N, "y_bf16"))) return st;
  if (base_bf16 == y_bf16 && ld_base != ld_y)
    return fail(SEGQ_ERR_SHAPE, "base_bf16 on y_bf16 needs ld_base = ld_y");
  const size_t need = sq::adapter_plan(p);
  if (need && (!workspace || workspace_bytes < need))
    return fail(SEGQ_ERR_UNSUPPORTED,
                "adapters of this shape need a workspace of at least %zu bytes "
                "(segquant_adapter_workspace_bytes)", need);
  if (!aligned16(workspace)) return fail(SEGQ_ERR_ALIGN, "workspace is not 16-byte aligned");
  const I128 factors = 2 * (I128)n_adapters * rank;  // bytes of a per column of it, of b per row
  const Operand outs[] = {{"y_bf16", bf16_rows(y_bf16, ld_y, N, M)},
                          {"workspace", one_run(workspace, need)}};
  const Operand ins[] = {{"base_bf16", bf16_rows(base_bf16, ld_base, N, M), 1},
                         {"x_bf16", bf16_rows(x_bf16, ld_x, K, M)},
                         {"a", one_run(a, factors * n_nseg * K)},
                         {"b", one_run(b, factors * N)},
                         {"row_offset", one_run(row_offset, sizeof(int32_t) * ((I128)n_req + 1))},
                         {"adapter", one_run(adapter, sizeof(int32_t) * (I128)n_req)},
                         {"rank_of", one_run(rank_of, sizeof(int32_t) * (I128)n_adapters)},
                         {"alpha", one_run(alpha, sizeof(float) * (I128)n_adapters)}};
  if ((st = check_apart(outs, ins))) return st;
  p.x = x_bf16;
  p.ld_x = ld_x;
  p.row_offset = row_offset;
  p.adapter = adapter;
  p.n_adapters = n_adapters;
  p.rank_of = rank_of;
  p.a = a;
  p.b = b;
  p.alpha = alpha;
  p.base = base_bf16;
  p.ld_base = ld_base;
  p.y = y_bf16;
  p.ld_y = ld_y;
  p.t = static_cast<float *>(workspace);
  return hip_status(sq::launch_adapter(p, (hipStream_t)stream), "adapter launch");
}

static int quantize_weight(const float *w, int64_t K, int64_t N, int64_t ld_w, int32_t n_kseg,
                           const int32_t *kseg_offset, const int32_t *kseg_width, int32_t n_nseg,
                           const int32_t *nseg_offset, const int32_t *nseg_width,
                           int32_t per_column, int8_t *w_packed, float *w_scale, bool w4,
                           void *stream) {
  if (K < 1 || N < 1 || K > kI32Max || N > kI32Max)
    return fail(SEGQ_ERR_SHAPE, "bad shape K=%lld N=%lld", (long long)K, (long long)N);
  if (ld_w < N) return fail(SEGQ_ERR_SHAPE, "ld_w %lld < N %lld", (long long)ld_w, (long long)N);
  if (!w || !w_packed || !w_scale) return fail(SEGQ_ERR_NULL, "w, w_packed or w_scale is NULL");
  if (K % 64 || N % 16)
    return fail(SEGQ_ERR_ALIGN, "weight needs K %% 64 == 0 and N %% 16 == 0 (K=%lld N=%lld)",
                (long long)K, (long long)N);
  if (!aligned16(w_packed) || (reinterpret_cast<uintptr_t>(w) & 3u))
    return fail(SEGQ_ERR_ALIGN, "w_packed must be 16-byte and w 4-byte aligned");
  sq::SegTable ks{};
  int st = read_kseg(n_kseg, kseg_offset, kseg_width, K, 0, ks);
  if (st) return st;
  sq::NSegTable ns{};
  ns.n = 1;
  ns.off[0] = 0;
  ns.end[0] = (int32_t)N;
  if (!per_column && (st = read_nseg(n_nseg, nseg_offset, nseg_width, N, ns))) return st;
  return hip_status(sq::launch_quantize_weight(w, K, N, ld_w, ks, ns, per_column != 0, w_packed,
                                               w_scale, w4, (hipStream_t)stream),
                    "quantize_weight launch");
}

int segquant_quantize_weight(const float *w, int64_t K, int64_t N, int64_t ld_w,
                             int32_t n_kseg, const int32_t *kseg_offset,
                             const int32_t *kseg_width, int32_t n_nseg,
                             const int32_t *nseg_offset, const int32_t *nseg_width,
                             int32_t per_column, int8_t *w_packed, float *w_scale,
                             void *stream) {
  return quantize_weight(w, K, N, ld_w, n_kseg, kseg_offset, kseg_width, n_nseg, nseg_offset,
                         nseg_width, per_column, w_packed, w_scale, false, stream);
}

int segquant_quantize_weight_w4(const float *w, int64_t K, int64_t N, int64_t ld_w,
                                int32_t n_kseg, const int32_t *kseg_offset,
                                const int32_t *kseg_width, int32_t n_nseg,
                                const int32_t *nseg_offset, const int32_t *nseg_width,
                                int32_t per_column, int8_t *w_packed, float *w_scale,
                                void *stream) {
  return quantize_weight(w, K, N, ld_w, n_kseg, kseg_offset, kseg_width, n_nseg, nseg_offset,
                         nseg_width, per_column, w_packed, w_scale, true, stream);
}

static int unpack_weight(const int8_t *w_packed, int64_t K, int64_t N, int8_t *w_kn,
                         int64_t ld_w, bool w4, void *stream) {
  if (segquant_weight_packed_bytes(K, N) == 0)
    return fail(SEGQ_ERR_ALIGN, "weight needs K %% 64 == 0 and N %% 16 == 0 (K=%lld N=%lld)",
                (long long)K, (long long)N);
  if (ld_w < N) return fail(SEGQ_ERR_SHAPE, "ld_w %lld < N %lld", (long long)ld_w, (long long)N);
  if (!w_packed || !w_kn) return fail(SEGQ_ERR_NULL, "w_packed or w_kn is NULL");
  if (!aligned16(w_packed)) return fail(SEGQ_ERR_ALIGN, "w_packed is not 16-byte aligned");
  return hip_status(sq::launch_unpack_weight(w_packed, K, N, w_kn, ld_w, w4, (hipStream_t)stream),
                    "unpack launch");
}

int segquant_unpack_weight(const int8_t *w_packed, int64_t K, int64_t N, int8_t *w_kn,
                           int64_t ld_w, void *stream) {
  return unpack_weight(w_packed, K, N, w_kn, ld_w, false, stream);
}

int segquant_unpack_weight_w4(const int8_t *w_packed, int64_t K, int64_t N, int8_t *w_kn,
                              int64_t ld_w, void *stream) {
  return unpack_weight(w_packed, K, N, w_kn, ld_w, true, stream);
}

}  // extern "C"

namespace sq {
static int gemm_check_shape(int64_t M, int64_t N, int64_t K, uint32_t flags) {
  if (M < 0 || N < 1 || K < 1 || M > kI32Max || N > kI32Max || K > kI32Max)
    return fail(SEGQ_ERR_SHAPE, "bad shape M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                (long long)K);
  if (K % 64 || N % 16)
    return fail(SEGQ_ERR_ALIGN, "GEMM needs K %% 64 == 0 and N %% 16 == 0 (K=%lld N=%lld)",
                (long long)K, (long long)N);
  if (flags & ~(SEGQ_GEMM_FORCE_TILE | SEGQ_GEMM_FORCE_SMALLM | SEGQ_GEMM_FUSED_QUANT |
                SEGQ_GEMM_SINGLE_SCALE | SEGQ_GEMM_W4))
    return fail(SEGQ_ERR_SHAPE, "unknown flags 0x%x", flags);
  if ((flags & SEGQ_GEMM_FORCE_TILE) && (flags & SEGQ_GEMM_FORCE_SMALLM))
    return fail(SEGQ_ERR_SHAPE, "both kernels forced");
  if ((flags & SEGQ_GEMM_FORCE_SMALLM) && M > sq::kSmallMMax)
    return fail(SEGQ_ERR_UNSUPPORTED, "the small-M kernel takes M <= %d (M=%lld)", sq::kSmallMMax,
                (long long)M);
  return SEGQ_OK;
}
}  // namespace sq

extern "C" {

int segquant_gemm_kernel_for(int64_t M, int64_t N, int64_t K, uint32_t flags) {
  int st = sq::gemm_check_shape(M, N, K, flags);
  if (st) return st;
  if (flags & SEGQ_GEMM_FORCE_TILE) return SEGQ_KERNEL_TILE;
  if (flags & SEGQ_GEMM_FORCE_SMALLM) return SEGQ_KERNEL_SMALLM;
  return M <= sq::kSmallMMax ? SEGQ_KERNEL_SMALLM : SEGQ_KERNEL_TILE;
}

int segquant_gemm_halves(const float *act_scales_host, int32_t n_kseg) {
  if (!act_scales_host) return fail(SEGQ_ERR_NULL, "act_scales_host is NULL");
  if (n_kseg < 1 || n_kseg > SEGQ_MAX_KSEG)
    return fail(SEGQ_ERR_SEGMENTS, "K-segment count %d outside [1, %d]", n_kseg, SEGQ_MAX_KSEG);
  for (int32_t i = 0; i < n_kseg; ++i) {
    const float s_neg = act_scales_host[n_kseg + i], inv_neg = act_scales_host[3 * n_kseg + i];
    if (s_neg != 0.0f || inv_neg != 0.0f) return 0;  // the - half carries values: both halves
  }
  return (int)SEGQ_GEMM_SINGLE_SCALE;
}

}  // extern "C"

namespace sq {
static bool quantize_first(int kernel, int64_t M, int64_t N, const sq::SegTable &ks,
                           uint32_t flags) {
  return kernel == SEGQ_KERNEL_TILE && !(flags & SEGQ_GEMM_FUSED_QUANT) &&
         sq::tile_quantize_first(M, N, ks);
}

// Bytes of the widened int8 weight a W4 call needs in its workspace (0 when
// the small-M streaming kernel reads the 4-bit tiles itself).
static size_t w4_widen_bytes(int kernel, int64_t M, int64_t N, int64_t K, const sq::SegTable &ks,
                             uint32_t flags, bool bf16_input) {
  if (!(flags & SEGQ_GEMM_W4)) return 0;
  if (kernel == SEGQ_KERNEL_SMALLM && sq::smallm_reads_w4(M, K, ks.n, bf16_input)) return 0;
  return (size_t)K * (size_t)N;
}
}  // namespace sq

extern "C" {

size_t segquant_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t n_kseg,
                                     const int32_t *kseg_offset, const int32_t *kseg_width,
                                     uint32_t flags) {
  if (sq::gemm_check_shape(M, N, K, flags)) return 0;
  sq::SegTable ks{};
  if (read_kseg(n_kseg, kseg_offset, kseg_width, K, SEGQ_MAX_KSEG_WIDTH, ks)) return 0;
  ok();
  const int kernel = segquant_gemm_kernel_for(M, N, K, flags);
  return sq::w4_widen_bytes(kernel, M, N, K, ks, flags, true) +
         (sq::quantize_first(kernel, M, N, ks, flags) ? (size_t)(M * K) : 0);
}

int segquant_gemm_w8a8_seg(int64_t M, int64_t N, int64_t K,
                           const uint16_t *x_bf16, int64_t ld_x,
                           const int8_t *xq, int64_t ld_q, int32_t q_layout,
                           const int8_t *w_packed, const float *w_scale,
                           int32_t n_kseg, const int32_t *kseg_offset,
                           const int32_t *kseg_width, const float *act_scales,
                           uint16_t *y_bf16, int64_t ld_y, int32_t *acc_debug,
                           void *workspace, size_t workspace_bytes,
                           uint32_t flags, void *stream) {
  const sq::GemmCall c{M,       N,          K,        x_bf16,      ld_x,        xq,
                       ld_q,    q_layout,   w_packed, w_scale,     n_kseg,      kseg_offset,
                       kseg_width, act_scales, y_bf16, ld_y,     acc_debug,   flags,
                       stream};
  if (workspace && !aligned16(workspace))
    return fail(SEGQ_ERR_ALIGN, "workspace is not 16-byte aligned");
  sq::SegTable ks{};
  int st = sq::gemm_validate(c, ks);
  if (st) return st;
  return sq::gemm_enqueue(c, ks, workspace, workspace ? workspace_bytes : 0);
}

}  // extern "C"
