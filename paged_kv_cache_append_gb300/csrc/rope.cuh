// rope.cuh -- one head row in registers: RMS norm over the head, rotation of
// its leading dims by the position's angles, and the KV codecs from fp32.
//
// A row of D elements is held by LPR = D / 8 consecutive lanes, 8 elements
// (one 16-byte bf16 load) each; a warp holds 32 / LPR rows.  With x the row,
//   y_d = x_d * rsqrt(mean(x^2) + eps) * (w_d + offset)       (norm, optional)
//   (a, b) -> (a cos - b sin, b cos + a sin)                  (rotation)
// over the pairs (i, i + rd/2) (halves) or (2i, 2i + 1) (pairs), i < rd/2;
// dims >= rd pass.  rd is a multiple of 16, so in the halves layout a lane's 8
// dims have their partners in one other lane (rd / 16 lanes away) and share
// its angles.  Everything is fp32 from the bf16 input to the last rounding:
// the result is rounded once, to bf16 or to the codes of the page.
#pragma once

#include "device.cuh"
#include "encode.cuh"
#include "internal.h"

namespace nk {

// Rows of one operand: element (token n, head h, dim d) at
// ptr[n * token_stride + h * head_stride + d].
struct RowsIn {
  const __nv_bfloat16* ptr;
  int64_t token_stride, head_stride;
};

struct RopeArgs {
  const float* cos_sin;  // [positions][rd]: rd/2 cosines, rd/2 sines
  int positions, rd, pairs;
  float eps, offset;
};

// The angles of one lane's 8 dims at one position.  Halves: cos[k], sin[k] of
// dim 8 l + k, the sine negated where the lane holds the first half (its
// partner term is subtracted).  Pairs: cos / sin of pair k in [k], k < 4.
struct Angles {
  float c[8], s[8];
  bool on;  // the lane's dims are rotated
};

__device__ __forceinline__ void load_angles(const RopeArgs& rp, int pos, int l, Angles& a) {
  const int e0 = 8 * l, half = rp.rd >> 1;
  a.on = e0 < rp.rd;
  if (!a.on) return;
  const float* row = rp.cos_sin + static_cast<int64_t>(pos) * rp.rd;
  if (rp.pairs) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + (e0 >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + (e0 >> 1)));
    a.c[0] = c.x, a.c[1] = c.y, a.c[2] = c.z, a.c[3] = c.w;
    a.s[0] = s.x, a.s[1] = s.y, a.s[2] = s.z, a.s[3] = s.w;
    return;
  }
  const bool lo = e0 < half;
  const int i = lo ? e0 : e0 - half;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + i + 4 * u));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i + 4 * u));
    a.c[4 * u] = c.x, a.c[4 * u + 1] = c.y, a.c[4 * u + 2] = c.z, a.c[4 * u + 3] = c.w;
    a.s[4 * u] = s.x, a.s[4 * u + 1] = s.y, a.s[4 * u + 2] = s.z, a.s[4 * u + 3] = s.w;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) a.s[k] = lo ? -a.s[k] : a.s[k];
}

// The lane holding the rotation partners of lane `lane` (row position l).
__device__ __forceinline__ int partner_lane(const RopeArgs& rp, int lane, int l) {
  const int hop = rp.rd >> 4;
  if (rp.pairs || 8 * l >= rp.rd) return lane;
  return l < hop ? lane + hop : lane - hop;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Norm weights of a lane: its own 8 and, in the halves layout, its partner's.
struct Weights {
  float own[8], other[8];
  bool on;
};

__device__ __forceinline__ void load_weights(const RopeArgs& rp, const __nv_bfloat16* w, int lane, int l, int src,
                                             Weights& o) {
  o.on = w != nullptr;
  if (!o.on) return;
  unpack8(*reinterpret_cast<const uint4*>(w + 8 * l), o.own);
  unpack8(*reinterpret_cast<const uint4*>(w + 8 * (l + src - lane)), o.other);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    o.own[k] += rp.offset;
    o.other[k] += rp.offset;
  }
}

// The row's 8 values of this lane, normed and rotated.  All 32 lanes of the
// warp call it together (`src`: partner_lane).
template <int LPR>
__device__ __forceinline__ void norm_rotate(const uint4& raw, const RopeArgs& rp, const Angles& a, const Weights& w,
                                            int src, float (&y)[8]) {
  float x[8];
  unpack8(raw, x);
  float r = 1.f;
  if (w.on) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    r = rsqrtf(fmaf(ss, 1.f / (8 * LPR), rp.eps));
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = x[k] * r * w.own[k];
  }
  if (rp.pairs) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float p = x[2 * k], q = x[2 * k + 1];
      y[2 * k] = a.on ? fmaf(p, a.c[k], -q * a.s[k]) : p;
      y[2 * k + 1] = a.on ? fmaf(q, a.c[k], p * a.s[k]) : q;
    }
    return;
  }
  // the partner's bf16 values (four packed words), normed here as there
  uint4 other;
  other.x = __shfl_sync(0xffffffffu, raw.x, src);
  other.y = __shfl_sync(0xffffffffu, raw.y, src);
  other.z = __shfl_sync(0xffffffffu, raw.z, src);
  other.w = __shfl_sync(0xffffffffu, raw.w, src);
  float o[8];
  unpack8(other, o);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (w.on) o[k] = o[k] * r * w.other[k];
    y[k] = a.on ? fmaf(x[k], a.c[k], o[k] * a.s[k]) : x[k];
  }
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&y)[8]) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// Encodes the lane's 8 values of a row into the page's code and scale rows
// with the codec rules of encode.cuh (quotients by the stored scale, rounded
// once).  `live` lanes store; all 32 lanes of the warp call it together.
template <int KIND, int D>
__device__ __forceinline__ void encode8(const float (&y)[8], uint8_t* code_row, uint8_t* scale_row, int l, bool live) {
  constexpr int LPR = D / 8;
  if constexpr (KIND == KIND_BF16) {
    if (live) *reinterpret_cast<uint4*>(code_row + 16 * l) = pack8_bf16(y);
  } else {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(y[k]));
    if constexpr (KIND == KIND_NVFP4) {
      m = group_max<2>(m);
      const uint32_t s8 = f32x2_to_e4m3x2(__fdiv_rn(m, 6.f), 0.f) & 0xFFu;
      const float sv = e4m3_to_f32(s8);
      uint32_t c = 0;
      if (sv != 0.f) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          c |= f32x2_to_e2m1x2(__fdiv_rn(y[2 * k], sv), __fdiv_rn(y[2 * k + 1], sv)) << (8 * k);
      }
      if (live) {
        *reinterpret_cast<uint32_t*>(code_row + 4 * l) = c;
        if ((l & 1) == 0) scale_row[l >> 1] = static_cast<uint8_t>(s8);
      }
    } else {
      constexpr int GL = KIND == KIND_INT8 ? 8 : LPR;  // lanes that share a scale
      m = group_max<GL>(m);
      const __half s = __float2half_rn(fminf(__fdiv_rn(m, KIND == KIND_INT8 ? 127.f : 448.f), 65504.f));
      const float sf = __half2float(s);
      uint32_t c[2] = {0u, 0u};
      if (sf != 0.f) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float u = __fdiv_rn(y[k], sf), v = __fdiv_rn(y[k + 1], sf);
          uint32_t two;
          if constexpr (KIND == KIND_INT8) {
            two = (static_cast<uint32_t>(max(-127, min(127, __float2int_rn(u)))) & 0xFFu) |
                  ((static_cast<uint32_t>(max(-127, min(127, __float2int_rn(v)))) & 0xFFu) << 8);
          } else {
            two = f32x2_to_e4m3x2(u, v);
          }
          c[k >> 2] |= two << (8 * (k & 2));
        }
      }
      if (live) {
        *reinterpret_cast<uint2*>(code_row + 8 * l) = make_uint2(c[0], c[1]);
        if (l % GL == 0) *reinterpret_cast<__half*>(scale_row + 2 * (l / GL)) = s;
      }
    }
  }
}

}  // namespace nk
