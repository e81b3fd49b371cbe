// diff.cuh -- what the differential attentions share: arguments of the output
// and the host-side checks.
//
// A head's result over a set of keys is kept per map m as (m_m, l_m, O_m):
// reference maximum and sum in base 2, and the unnormalised O_m of 2 D values.
// Partials over disjoint keys join per map as in any split softmax,
//   w_ms = 2^(m_ms - M_m) / L_m,  L_m = sum_s l_ms 2^(m_ms - M_m),
// and the head's output is (sum_s w_1s O_1s) - lambda (sum_s w_2s O_2s), normed.
#pragma once

#include <cmath>

#include "device.cuh"
#include "internal.h"

namespace nk {

constexpr float kDiffLog2e = 1.4426950408889634f;
constexpr float kDiffLn2 = 0.6931471805599453f;

// f16 weights without a factor per key are stored times 2^this: they are at most 2^8 (the lazy
// reference's lag), and what lies below 2^-14 of f16's range is held to a fixed step only.
constexpr int kDiffWeightLift = 7;

struct DiffOut {
  const float* lambda;
  int64_t lambda_stride;
  const __nv_bfloat16* w;  // nullptr: no norm
  float eps, out_scale;
  __nv_bfloat16* out;  // [tokens][Hq / 2][2 D]
  float* lse;          // [tokens][Hq] or nullptr
};

// Four values of a head's output: o times the norm's factor (and scale), times
// the weight; one rounding.
__device__ __forceinline__ uint2 diff_finish(const float (&o)[4], float f, const __nv_bfloat16* w, int d) {
  float x[4];
  if (w) {
    const uint2 v = *reinterpret_cast<const uint2*>(w + d);
    const float ww[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                         __uint_as_float(v.y & 0xFFFF0000u)};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = o[i] * f * ww[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = o[i] * f;
  }
  return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// At most this many splits of a decoded row: bounds the join's work and its shared memory.
constexpr int kDiffMaxSplits = 128;

// Valid length of row b as the decode kernels take it (0: refused, no keys).
__device__ __forceinline__ int diff_length(const int32_t* frontiers, const int32_t* table_rows, int b, int L, int C,
                                           int* row_out, int* report) {
  const int F = __ldcg(frontiers + b), row = __ldcg(table_rows + b);
  const bool ok = F >= 0 && F <= L * 64 && row >= 0 && row < C;
  if (!ok && report) set_status(report, NK_STATUS_FRONTIER);
  *row_out = ok ? row : 0;
  return ok ? F : 0;
}

// The split plan of a decode, a lane per row (B <= 8): `chunk` pages to a split,
// the smallest count (at least ceil(longest / kDiffMaxSplits)) whose splits,
// max(1, ceil(pages / chunk)) for every row, add up to at most `ctas`.  32
// candidates are tried at once: every CTA computes the plan before its first
// copy, and a bisection over the rows cost it 1.5 us.
struct DiffRows {
  int F, row, pages;  // of row `lane`
  int chunk;
  int ns, end;  // its splits; splits up to and with it
};

__device__ __forceinline__ DiffRows diff_rows(const int32_t* frontiers, const int32_t* table_rows, int B, int L, int C,
                                              int ctas, int* report) {
  const int lane = threadIdx.x & 31;
  DiffRows r;
  r.F = r.row = 0;
  if (lane < B) r.F = diff_length(frontiers, table_rows, lane, L, C, &r.row, report);
  r.pages = (r.F + 63) >> 6;
  const int total = __reduce_add_sync(0xffffffffu, r.pages), most = __reduce_max_sync(0xffffffffu, r.pages);
  const int least = max(1, (most + kDiffMaxSplits - 1) / kDiffMaxSplits);
  const int room = max(ctas - B, 1);
  int hi = max((total + room - 1) / room, least);  // always fits: sum ceil(N_b / c) <= total / c + B
  int lo = min(max(least, (total + ctas - 1) / ctas), hi);
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, c = lo + lane * step;
    int n = 0;
    for (int b = 0; b < B; ++b) n += max(1, (__shfl_sync(0xffffffffu, r.pages, b) + c - 1) / c);
    const int k = __ffs(__ballot_sync(0xffffffffu, c >= hi || n <= ctas)) - 1;  // the first that fits
    if (k > 0) hi = min(hi, lo + k * step);
    lo = k < 0 ? lo + 31 * step + 1 : k == 0 ? hi = lo : lo + (k - 1) * step + 1;
  }
  r.chunk = hi;
  r.ns = lane < B ? max(1, (r.pages + hi - 1) / hi) : 0;
  r.end = r.ns;
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, r.end, off);
    if (lane >= off) r.end += x;
  }
  return r;
}

// What split `cta` of the plan works on; b < 0: nothing.
struct DiffSplit {
  int b, row, F, p0, n;  // pages [p0, p0 + n) of the row; n = 0 only for a row without keys
};

__device__ __forceinline__ DiffSplit diff_split(const DiffRows& r, int B, int cta) {
  const unsigned own = __ballot_sync(0xffffffffu, (threadIdx.x & 31) < B && cta < r.end);
  DiffSplit s;
  s.b = __ffs(own) - 1;
  const int from = max(s.b, 0);
  s.row = __shfl_sync(0xffffffffu, r.row, from);
  s.F = __shfl_sync(0xffffffffu, r.F, from);
  s.p0 = (cta - __shfl_sync(0xffffffffu, r.end - r.ns, from)) * r.chunk;
  s.n = min(r.chunk, __shfl_sync(0xffffffffu, r.pages, from) - s.p0);
  return s;
}

// Checks that decode and prefill share; fills `o`.
int check_diff(const char* what, const void* q, int32_t Hq, const nk_pool* pool, int32_t layer, const int32_t* tables,
               const int32_t* table_rows, const int32_t* lengths, int32_t B, int32_t T, float scale, const nk_diff* diff,
               void* out, float* lse, DiffOut* o);

// Shape alone (for the workspace queries): pairs of KV heads, head_dim, B, T.
int check_diff_shape(const nk_pool* pool, int32_t B, int32_t T, int32_t Hq);

}  // namespace nk
