// rope.cuh -- one head row in registers: RMS norm over the head, rotation of
// its leading dims by the position's angles, and the KV codecs from fp32.
//
// A row of D elements is held by LPR = D / 16 consecutive lanes as two chunks
// of 8 dims (16-byte bf16 loads), so a warp holds 32 / LPR rows.  With x the row,
//   y_d = x_d * rsqrt(mean(x^2) + eps) * (w_d + offset)       (norm, optional)
//   (a, b) -> (a cos - b sin, b cos + a sin)                  (rotation)
// over the pairs (i, i + rd/2) (halves) or (2i, 2i + 1) (pairs), i < rd/2;
// dims >= rd pass.  rd is a multiple of 16: the first rd / 16 lanes of a row
// hold the chunks 8 l and 8 l + rd / 2, which are each other's partners in the
// halves layout, so a rotation needs no other lane; the rest hold two chunks
// in a row of the dims that pass.  (One chunk a lane, its partners fetched by
// shuffles, took 1.6 to 2.1 times the instructions.)  Everything is fp32 from
// the bf16 input to the last rounding: the result is rounded once, to bf16 or
// to the codes of the page.
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
__device__ __forceinline__ void unpack8(const uint4& v, F2* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
}

// First dims of the two chunks of lane l of a row.
struct Chunks {
  int a, b;
  bool turned;  // they are rotated
};

__device__ __forceinline__ Chunks chunks_of(const RopeArgs& rp, int l) {
  const int half = rp.rd >> 1, e = 8 * l;
  if (e < half) return Chunks{e, e + half, true};
  const int at = rp.rd + 2 * (e - half);
  return Chunks{at, at + 8, false};
}

// A lane's 16 values as fp32 pairs, chunk a in [0, 4), chunk b in [4, 8).
using Row16 = F2[8];

// What norm and rotation of a lane's chunks at one position come to, once the
// row's 1 / rms r is known: y = r (x c + o s), with x the lane's values, o
// their partners', c = cos * weight and s = +-sin * (the partner's weight).
// It is the same for every head of the token, so a lane computes it once per
// unit and spends three packed operations per two elements and head.  Dims
// that do not turn have o = 0 and s = -0 (so that -0 stays -0).
struct Turn {
  Row16 c, s;
  bool norm;
};

__device__ __forceinline__ void load_turn(const RopeArgs& rp, const __nv_bfloat16* weight, int pos, const Chunks& ch,
                                          Turn& t) {
  const int half = rp.rd >> 1;
  const float* row = rp.cos_sin + static_cast<int64_t>(pos) * rp.rd;
  t.norm = weight != nullptr;
  if (!ch.turned) {
#pragma unroll
    for (int k = 0; k < 8; ++k) t.c[k] = pack2(1.f, 1.f), t.s[k] = pack2(-0.f, -0.f);
  } else if (rp.pairs) {  // four angles a chunk, (cos, cos) and (-sin, sin)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = (u ? ch.b : ch.a) >> 1;
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + i));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i));
      const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) t.c[4 * u + k] = pack2(cv[k], cv[k]), t.s[4 * u + k] = pack2(-sv[k], sv[k]);
    }
  } else {  // eight angles, the chunks' own: (cos, -sin) for a, (cos, sin) for b
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + ch.a + 4 * u));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + ch.a + 4 * u));
      t.c[2 * u] = t.c[4 + 2 * u] = pack2(c.x, c.y);
      t.c[2 * u + 1] = t.c[5 + 2 * u] = pack2(c.z, c.w);
      t.s[2 * u] = pack2(-s.x, -s.y), t.s[4 + 2 * u] = pack2(s.x, s.y);
      t.s[2 * u + 1] = pack2(-s.z, -s.w), t.s[5 + 2 * u] = pack2(s.z, s.w);
    }
  }
  if (t.norm) {
    F2 w[8];
    unpack8(*reinterpret_cast<const uint4*>(weight + ch.a), w);
    unpack8(*reinterpret_cast<const uint4*>(weight + ch.b), w + 4);
    const F2 one = pack2(1.f, 1.f), off = pack2(rp.offset, rp.offset);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = fma2(w[k], one, off);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      t.c[k] = mul2(t.c[k], w[k]);
      if (ch.turned) t.s[k] = mul2(t.s[k], rp.pairs ? swap2(w[k]) : w[k ^ 4]);
    }
  }
}

// The lane's 16 values of a row, normed and rotated.  All 32 lanes of the
// warp call it together.
template <int LPR>
__device__ __forceinline__ void norm_rotate(const uint4 (&raw)[2], const RopeArgs& rp, const Chunks& ch, const Turn& t,
                                            Row16& y) {
  Row16 x;
  unpack8(raw[0], x);
  unpack8(raw[1], x + 4);
  F2 r2 = pack2(1.f, 1.f);
  if (t.norm) {
    F2 q = mul2(x[0], x[0]), p = mul2(x[1], x[1]);
#pragma unroll
    for (int k = 2; k < 8; k += 2) {
      q = fma2(x[k], x[k], q);
      p = fma2(x[k + 1], x[k + 1], p);
    }
    float ss, hi;
    unpack2(add2(q, p), ss, hi);
    ss += hi;
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(fmaf(ss, 1.f / (16 * LPR), rp.eps));
    r2 = pack2(r, r);
  }
  const bool all = rp.rd == 16 * LPR;  // every lane's dims turn
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    F2 o = rp.pairs ? swap2(x[k]) : x[k ^ 4];
    if (!all && !ch.turned) o = 0ull;
    y[k] = fma2(x[k], t.c[k], mul2(o, t.s[k]));
    if (t.norm) y[k] = mul2(y[k], r2);
  }
}

__device__ __forceinline__ uint32_t bf16x2_of(F2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 pack8_bf16(const F2* y) {
  return make_uint4(bf16x2_of(y[0]), bf16x2_of(y[1]), bf16x2_of(y[2]), bf16x2_of(y[3]));
}

// x / s rounded once, from inv = 1 / s rounded once: the quotient's error is
// taken off with one exact remainder (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990), which leaves the
// rounded quotient (a
// quotient that fp32 holds, such as a tie between two codes, comes out exactly:
// the remainder then is its error times s).  The sign is x's, also of a zero.
// For finite x and s in binary16's or E4M3's range.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv;
  const float r = fmaf(fmaf(-q, s, x), inv, q);
  return __uint_as_float((__float_as_uint(r) & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));
}

// The eight codes of one chunk for the stored scale s and inv = 1 / s (0 for
// s = 0): bytes in c, for NVFP4 eight nibbles in c[0].  `finite`: no infinity
// in the group (a NaN counts for nothing in the maximum and stays one).
template <int KIND>
__device__ __forceinline__ void codes8(const F2* y2, float s, float inv, bool finite, uint32_t (&c)[2]) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) unpack2(y2[k], v[2 * k], v[2 * k + 1]);
  c[0] = c[1] = 0u;
  if (s == 0.f) return;
  if (finite) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = quotient(v[k], s, inv);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fdiv_rn(v[k], s);
  }
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

// The stored scale of a group with the largest magnitude m: its bits and value.
template <int KIND>
__device__ __forceinline__ float scale_of(float m, uint32_t& bits) {
  if constexpr (KIND == KIND_NVFP4) {
    bits = f32x2_to_e4m3x2(__fdiv_rn(m, 6.f), 0.f) & 0xFFu;
    return e4m3_to_f32(bits);
  } else {
    const __half h = __float2half_rn(fminf(__fdiv_rn(m, KIND == KIND_INT8 ? 127.f : 448.f), 65504.f));
    bits = __half_as_ushort(h);
    return __half2float(h);
  }
}

__device__ __forceinline__ float max_of8(const F2* y2) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b;
    unpack2(y2[k], a, b);
    m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
  }
  return m;
}

// Encodes the lane's two chunks of a row into the page's code and scale rows
// with the codec rules of encode.cuh (quotients by the stored scale, rounded
// once).  `live` lanes store; all 32 lanes of the warp call it together.
// maxima: the row's D / 8 chunk maxima in shared memory, private to its lanes
// (the groups of INT8-G64 and NVFP4-G16 are 8 and 2 chunks in a row, which
// different lanes hold).
template <int KIND, int D>
__device__ __forceinline__ void encode16(const Row16& y, uint8_t* code_row, uint8_t* scale_row, const Chunks& ch, int l,
                                         bool live, float* maxima) {
  if constexpr (KIND == KIND_BF16) {
    if (live) {
      *reinterpret_cast<uint4*>(code_row + 2 * ch.a) = pack8_bf16(y);
      *reinterpret_cast<uint4*>(code_row + 2 * ch.b) = pack8_bf16(y + 4);
    }
  } else if constexpr (KIND == KIND_FP8) {
    const float m = group_max<D / 16>(fmaxf(max_of8(y), max_of8(y + 4)));
    uint32_t bits, c[2];
    const float s = scale_of<KIND>(m, bits), inv = s != 0.f ? __frcp_rn(s) : 0.f;
    const bool finite = m <= 3.402823466e38f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      codes8<KIND>(y + 4 * u, s, inv, finite, c);
      if (live) *reinterpret_cast<uint2*>(code_row + (u ? ch.b : ch.a)) = make_uint2(c[0], c[1]);
    }
    if (live && l == 0) *reinterpret_cast<uint16_t*>(scale_row) = static_cast<uint16_t>(bits);
  } else {
    constexpr int GC = KIND == KIND_INT8 ? 8 : 2;  // chunks of a group
    __syncwarp();
    maxima[ch.a >> 3] = max_of8(y);
    maxima[ch.b >> 3] = max_of8(y + 4);
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int d = u ? ch.b : ch.a, g = d / (8 * GC);
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < GC; k += 2) {
        const float2 two = *reinterpret_cast<const float2*>(maxima + g * GC + k);
        m = fmaxf(m, fmaxf(two.x, two.y));
      }
      uint32_t bits, c[2];
      const float s = scale_of<KIND>(m, bits), inv = s != 0.f ? __frcp_rn(s) : 0.f;
      codes8<KIND>(y + 4 * u, s, inv, m <= 3.402823466e38f, c);
      if (!live) continue;
      if constexpr (KIND == KIND_INT8) {
        *reinterpret_cast<uint2*>(code_row + d) = make_uint2(c[0], c[1]);
        if (d % 64 == 0) *reinterpret_cast<uint16_t*>(scale_row + 2 * g) = static_cast<uint16_t>(bits);
      } else {
        *reinterpret_cast<uint32_t*>(code_row + d / 2) = c[0];
        if (d % 16 == 0) scale_row[g] = static_cast<uint8_t>(bits);
      }
    }
  }
}

}  // namespace nk
