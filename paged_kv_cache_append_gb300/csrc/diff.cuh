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

// Checks that decode and prefill share; fills `o`.
int check_diff(const char* what, const void* q, int32_t Hq, const nk_pool* pool, int32_t layer, const int32_t* tables,
               const int32_t* table_rows, const int32_t* lengths, int32_t B, int32_t T, float scale, const nk_diff* diff,
               void* out, float* lse, DiffOut* o);

// Shape alone (for the workspace queries): pairs of KV heads, head_dim, B, T.
int check_diff_shape(const nk_pool* pool, int32_t B, int32_t T, int32_t Hq);

}  // namespace nk
