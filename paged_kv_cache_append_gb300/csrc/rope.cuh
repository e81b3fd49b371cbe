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
#include "packed.cuh"

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

// Eight bf16 values as four fp32 pairs.
__device__ __forceinline__ void unpack8(const uint4& v, F2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}

// What norm and rotation of a lane's 8 dims at one position come to, once the
// row's 1 / rms r is known: y = r (x c + o s), with x the lane's values, o
// their partners', c = cos * weight and s = +-sin * (the partner's weight).
// It is the same for every head of the token, so a lane computes it once per
// unit and spends three packed operations per two elements and head.  Dims
// that do not turn have o = 0 and s = -0 (so that -0 stays -0).
struct Turn {
  F2 c[4], s[4];
  int src;    // lane of the partners (halves)
  bool on;    // the lane's dims are rotated
  bool norm;
};

template <int LPR>
__device__ __forceinline__ void load_turn(const RopeArgs& rp, const __nv_bfloat16* weight, int pos, int lane, int l,
                                          Turn& t) {
  const int e0 = 8 * l, half = rp.rd >> 1, hop = rp.rd >> 4;
  t.on = e0 < rp.rd;
  t.norm = weight != nullptr;
  t.src = rp.pairs || !t.on ? lane : l < hop ? lane + hop : lane - hop;
  const float* row = rp.cos_sin + static_cast<int64_t>(pos) * rp.rd;
  if (!t.on) {
#pragma unroll
    for (int k = 0; k < 4; ++k) t.c[k] = pack2(1.f, 1.f), t.s[k] = pack2(-0.f, -0.f);
  } else if (rp.pairs) {  // four angles, (cos, cos) and (-sin, sin)
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + (e0 >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + (e0 >> 1)));
    t.c[0] = pack2(c.x, c.x), t.c[1] = pack2(c.y, c.y), t.c[2] = pack2(c.z, c.z), t.c[3] = pack2(c.w, c.w);
    t.s[0] = pack2(-s.x, s.x), t.s[1] = pack2(-s.y, s.y), t.s[2] = pack2(-s.z, s.z), t.s[3] = pack2(-s.w, s.w);
  } else {  // eight angles, the sines negated in the first half
    const bool lo = e0 < half;
    const int i = lo ? e0 : e0 - half;
    const F2 sign = lo ? pack2(-1.f, -1.f) : pack2(1.f, 1.f);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + i + 4 * u));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i + 4 * u));
      t.c[2 * u] = pack2(c.x, c.y), t.c[2 * u + 1] = pack2(c.z, c.w);
      t.s[2 * u] = mul2(pack2(s.x, s.y), sign), t.s[2 * u + 1] = mul2(pack2(s.z, s.w), sign);
    }
  }
  if (t.norm) {
    F2 own[4], other[4];
    unpack8(*reinterpret_cast<const uint4*>(weight + 8 * l), own);
    unpack8(*reinterpret_cast<const uint4*>(weight + 8 * (l + t.src - lane)), other);
    const F2 one = pack2(1.f, 1.f), off = pack2(rp.offset, rp.offset);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (rp.pairs) other[k] = swap2(other[k]);
      t.c[k] = mul2(t.c[k], fma2(own[k], one, off));
      if (t.on) t.s[k] = mul2(t.s[k], fma2(other[k], one, off));
    }
  }
}

// The row's 8 values of this lane, normed and rotated.  All 32 lanes of the
// warp call it together.
template <int LPR>
__device__ __forceinline__ void norm_rotate(const uint4& raw, const RopeArgs& rp, const Turn& t, F2 (&y)[4]) {
  F2 x[4], o[4];
  unpack8(raw, x);
  if (rp.pairs) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = t.on ? swap2(x[k]) : 0ull;
  } else {
    uint4 other;  // the partner's bf16 values, four packed words
    other.x = __shfl_sync(0xffffffffu, raw.x, t.src);
    other.y = __shfl_sync(0xffffffffu, raw.y, t.src);
    other.z = __shfl_sync(0xffffffffu, raw.z, t.src);
    other.w = __shfl_sync(0xffffffffu, raw.w, t.src);
    if (!t.on) other = make_uint4(0u, 0u, 0u, 0u);
    unpack8(other, o);
  }
  if (t.norm) {
    F2 q = mul2(x[0], x[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) q = fma2(x[k], x[k], q);
    float ss, hi;
    unpack2(q, ss, hi);
    ss += hi;
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(fmaf(ss, 1.f / (8 * LPR), rp.eps));
    const F2 r2 = pack2(r, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = mul2(fma2(x[k], t.c[k], mul2(o[k], t.s[k])), r2);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = fma2(x[k], t.c[k], mul2(o[k], t.s[k]));
  }
}

__device__ __forceinline__ uint32_t bf16x2_of(F2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 pack8_bf16(const F2 (&y)[4]) {
  return make_uint4(bf16x2_of(y[0]), bf16x2_of(y[1]), bf16x2_of(y[2]), bf16x2_of(y[3]));
}

// x / s rounded once, from inv = 1 / s rounded once: the quotient's error is
// taken off with one exact remainder, which leaves the rounded quotient (a
// quotient that fp32 holds, such as a tie between two codes, comes out exactly:
// the remainder then is its error times s).  The sign is x's, also of a zero.
// For finite x and s in binary16's or E4M3's range.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv;
  const float r = fmaf(fmaf(-q, s, x), inv, q);
  return __uint_as_float((__float_as_uint(r) & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));
}

// Encodes the lane's 8 values of a row into the page's code and scale rows
// with the codec rules of encode.cuh (quotients by the stored scale, rounded
// once).  `live` lanes store; all 32 lanes of the warp call it together.
template <int KIND, int D>
__device__ __forceinline__ void encode8(const F2 (&y2)[4], uint8_t* code_row, uint8_t* scale_row, int l, bool live) {
  constexpr int LPR = D / 8;
  if constexpr (KIND == KIND_BF16) {
    if (live) *reinterpret_cast<uint4*>(code_row + 16 * l) = pack8_bf16(y2);
  } else {
    float y[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack2(y2[k], y[2 * k], y[2 * k + 1]);
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(y[k]));
    constexpr int GL = KIND == KIND_NVFP4 ? 2 : KIND == KIND_INT8 ? 8 : LPR;  // lanes that share a scale
    m = group_max<GL>(m);
    uint32_t s_bits;  // the stored scale and its value
    float s;
    if constexpr (KIND == KIND_NVFP4) {
      s_bits = f32x2_to_e4m3x2(__fdiv_rn(m, 6.f), 0.f) & 0xFFu;
      s = e4m3_to_f32(s_bits);
    } else {
      const __half h = __float2half_rn(fminf(__fdiv_rn(m, KIND == KIND_INT8 ? 127.f : 448.f), 65504.f));
      s_bits = __half_as_ushort(h);
      s = __half2float(h);
    }
    float v[8];
    const float inv = s != 0.f ? __frcp_rn(s) : 0.f;
    if (m <= 3.402823466e38f) {  // no infinity in the group (a NaN is not in m: it stays one)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = quotient(y[k], s, inv);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __fdiv_rn(y[k], s);
    }
    uint32_t c[2] = {0u, 0u};
    if (s != 0.f) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        if constexpr (KIND == KIND_NVFP4) {
          c[0] |= f32x2_to_e2m1x2(v[k], v[k + 1]) << (4 * k);
        } else {
          uint32_t two;
          if constexpr (KIND == KIND_INT8)
            two = (static_cast<uint32_t>(max(-127, min(127, __float2int_rn(v[k])))) & 0xFFu) |
                  ((static_cast<uint32_t>(max(-127, min(127, __float2int_rn(v[k + 1])))) & 0xFFu) << 8);
          else
            two = f32x2_to_e4m3x2(v[k], v[k + 1]);
          c[k >> 2] |= two << (8 * (k & 2));
        }
      }
    }
    if (live) {
      if constexpr (KIND == KIND_NVFP4) {
        *reinterpret_cast<uint32_t*>(code_row + 4 * l) = c[0];
        if ((l & 1) == 0) scale_row[l >> 1] = static_cast<uint8_t>(s_bits);
      } else {
        *reinterpret_cast<uint2*>(code_row + 8 * l) = make_uint2(c[0], c[1]);
        if (l % GL == 0) *reinterpret_cast<uint16_t*>(scale_row + 2 * (l / GL)) = static_cast<uint16_t>(s_bits);
      }
    }
  }
}

}  // namespace nk
