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

// Pages per split of a decode: the smallest count (at least ceil(maxp /
// max_splits)) whose splits, max(1, ceil(N_b / c)) for every row, add up to at
// most `ctas`.
__device__ __forceinline__ int diff_chunk(const int* F, int B, int ctas, int max_splits) {
  int total = 0, maxp = 0;
  for (int b = 0; b < B; ++b) {
    const int n = (F[b] + 63) >> 6;
    total += n;
    maxp = max(maxp, n);
  }
  const int least = max(1, (maxp + max_splits - 1) / max_splits);
  const int room = max(ctas - B, 1);
  int hi = max((total + room - 1) / room, least);  // always fits: sum ceil(N_b / c) <= total / c + B
  int lo = min(max(least, (total + ctas - 1) / ctas), hi);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    int n = 0;
    for (int b = 0; b < B; ++b) n += max(1, (((F[b] + 63) >> 6) + mid - 1) / mid);
    if (n <= ctas) hi = mid;
    else lo = mid + 1;
  }
  return hi;
}

// Valid length of row b as the decode kernels take it (0: refused, no keys).
__device__ __forceinline__ int diff_length(const int32_t* frontiers, const int32_t* table_rows, int b, int L, int C,
                                           int* row_out, int* report) {
  const int F = frontiers[b], row = table_rows[b];
  const bool ok = F >= 0 && F <= L * 64 && row >= 0 && row < C;
  if (!ok && report) set_status(report, NK_STATUS_FRONTIER);
  *row_out = ok ? row : 0;
  return ok ? F : 0;
}

// At most this many splits of a decoded row: bounds the join's work.
constexpr int kDiffMaxSplits = 128;

// Checks that decode and prefill share; fills `o`.
int check_diff(const char* what, const void* q, int32_t Hq, const nk_pool* pool, int32_t layer, const int32_t* tables,
               const int32_t* table_rows, const int32_t* lengths, int32_t B, int32_t T, float scale, const nk_diff* diff,
               void* out, float* lse, DiffOut* o);

// Shape alone (for the workspace queries): pairs of KV heads, head_dim, B, T.
int check_diff_shape(const nk_pool* pool, int32_t B, int32_t T, int32_t Hq);

}  // namespace nk
