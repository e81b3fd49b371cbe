// qtile.cuh -- quantized page tiles in shared memory: the ring geometry of the
// tensor-core kernels that read quantized pages in place (qprefill.cu,
// prefix.cu) and the conversion of a raw tile to the f16 tile their MMAs read.
// The formats and what is exact in them are described in qprefill.cu.
#pragma once

#include "encode.cuh"
#include "tcgen05.cuh"

namespace nk {

// INT8-G64 keys: the power of two e (0..7) with 127 * max_g s_g * 2^-e < 2^15
// (or the largest, 7, when binary16's range forbids it).  The scales are
// finite and >= 0, so 127 * max_g s_g is 0 or a normal fp32 x, and
// x < 2^ex for ex = (biased exponent of x) - 126.
template <int D>
__device__ __forceinline__ int int8_row_shift(const uint8_t* scale_row) {
  float smax = 0.f;
#pragma unroll
  for (int g = 0; g < D / 64; ++g)
    smax = fmaxf(smax, fabsf(__half2float(*reinterpret_cast<const __half*>(scale_row + 2 * g))));
  const int ex = static_cast<int>((__float_as_uint(127.f * smax) >> 23) & 0xFFu) - 126;
  return min(max(ex - 15, 0), 7);
}

// 2^-e for e in [0, 7] (a normal fp32).
__device__ __forceinline__ float pow2_neg(int e) { return __uint_as_float(static_cast<uint32_t>(127 - e) << 23); }

// Rescale threshold of the online softmax, in log2 units: the running maximum
// moves only when a score passes it by more than this, so p <= 2^8.
constexpr float kLazyThr = 8.f;

template <int KK, int KV, int D>
struct QCfg {
  // converter warps (6 .. 5 + NCONV), 8 for every profile: the conversion
  // work sets the pace where only V is converted (raw FP8 keys go to the
  // tensor cores) as well as where both are
  static constexpr int NCONV = 8;
  static constexpr int THREADS = 192 + 32 * NCONV;  // warps 0-3 softmax, 4 producer, 5 MMA
  static constexpr int KCB = code_row_bytes<KK>(D), VCB = code_row_bytes<KV>(D);
  static constexpr int KSB = scale_row_bytes<KK>(D), VSB = scale_row_bytes<KV>(D);
  static constexpr int K_RB = KCB < 128 ? KCB : 128, V_RB = VCB < 128 ? VCB : 128;
  static constexpr int F16 = 64 * D * 2;                           // one f16 page tile
  // INT8-G64 keys are held as two f16 tiles whose sum is exact (K_SPLIT)
  static constexpr bool K_SPLIT = KK == KIND_INT8;
  static constexpr int K_STAGE = K_SPLIT ? 2 * F16 : F16;
  static constexpr int V_STAGE = F16;
  static constexpr int NF = 4;                                     // factor ring (512 B per page)
  static constexpr int RK_CODES = (64 * KCB + 1023) / 1024 * 1024;  // raw K code tile (1024-aligned)
  static constexpr int RV_CODES = (64 * VCB + 1023) / 1024 * 1024;
  static constexpr int RK_STAGE = (RK_CODES + 64 * KSB + 1023) / 1024 * 1024;
  static constexpr int RV_STAGE = (RV_CODES + 64 * VSB + 1023) / 1024 * 1024;
  // FP8-row keys with 128-byte code rows (head_dim >= 128, the swizzle of the
  // f16 tiles) go to the tensor cores as raw E4M3 codes (kind::f8f6f4), with
  // q split exactly into two E4M3 terms: no K conversion, no f16 K tile.
  static constexpr bool K8MMA = (KK == KIND_FP8) && D >= 128;
  static constexpr int NK = K8MMA ? 0 : K_SPLIT ? (D == 256 ? 1 : D == 128 ? 3 : 6)
                                              : D == 256 ? 2 : D == 128 ? 4 : 6;  // f16 K ring
  static constexpr int NV = K8MMA ? (D == 256 ? 3 : 4) : K_SPLIT ? (D == 256 ? 2 : D == 128 ? 3 : 6) : NK;  // f16 V ring
  static constexpr int NRK = K8MMA ? (D == 256 ? 3 : 6) : D == 256 ? (RK_STAGE <= 10240 ? 3 : 2) : 4;  // raw rings
  static constexpr int NRV = D == 256 ? (RV_STAGE <= 10240 || K8MMA ? 3 : 2) : 4;
  static constexpr int NKF = K8MMA ? 0 : NK;  // f16 K ready barriers (the raw FP8 keys need none)
  static constexpr int OFF_V = NK * K_STAGE;
  static constexpr int OFF_RK = OFF_V + NV * V_STAGE;
  static constexpr int OFF_RV = OFF_RK + NRK * RK_STAGE;
  static constexpr int OFF_F = OFF_RV + NRV * RV_STAGE;
  static constexpr int OFF_BAR = OFF_F + NF * 512;
  static constexpr int NBAR = 2 * NKF + 2 * NV + 2 * NRK + 2 * NRV + 2 * NF + 2 + 4;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_S = 0, COL_Q = 128, COL_O = 256;
  static constexpr uint32_t ID_S = K8MMA ? tc::idesc_e4m3(128, 64) : tc::idesc_f16(128, 64, false, false);
  static constexpr uint32_t ID_O = tc::idesc_f16(128, D, false, true);
  static constexpr int UNITS = 64 * (D / 16);  // (key, 16-dim group) units of a tile
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ void q_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Byte address (offset in the raw tile) of byte `col` of key row r in a tile
// staged as blocks of 64 rows x RB bytes with the matching TMA swizzle.
template <int RB>
__device__ __forceinline__ uint32_t raw_off(int r, int col) {
  return static_cast<uint32_t>((col / RB) * (64 * RB)) + swz<RB>(r, col % RB);
}

// Offset of f16 element (key r, dim d) in an f16 tile: 64-dim blocks of
// 64 rows x 128 bytes, 128-byte swizzle (d a multiple of 8: a 16-byte chunk).
__device__ __forceinline__ uint32_t f16_off(int r, int d) {
  return static_cast<uint32_t>((d >> 6) * 8192) + swz<128>(r, (d & 63) * 2);
}

// 16 dims [16 g, 16 g + 16) of key r of an FP8-row or NVFP4-G16 tile: raw
// codes and scales (shared memory) -> 16 exact f16 values (two 16-byte
// chunks).  INT8-G64 tiles are converted in convert_tile.
template <int KIND, int D, int RB>
__device__ __forceinline__ void convert16(const uint8_t* codes, const uint8_t* scales, int r, int g, uint4& lo,
                                          uint4& hi) {
  static_assert(KIND == KIND_FP8 || KIND == KIND_NVFP4, "FP8-row and NVFP4-G16 tiles");
  constexpr int SB = scale_row_bytes<KIND>(D);
  if constexpr (KIND == KIND_FP8) {
    const uint4 w = *reinterpret_cast<const uint4*>(codes + raw_off<RB>(r, 16 * g));
    lo = make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(w.x & 0xFFFFu)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w.x >> 16)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w.y & 0xFFFFu)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w.y >> 16)));
    hi = make_uint4(e4m3x2_to_f16x2(static_cast<uint16_t>(w.z & 0xFFFFu)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w.z >> 16)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w.w & 0xFFFFu)),
                    e4m3x2_to_f16x2(static_cast<uint16_t>(w.w >> 16)));
  } else {  // NVFP4: 8 bytes of codes times the group's E4M3 scale
    const uint2 w = *reinterpret_cast<const uint2*>(codes + raw_off<RB>(r, 8 * g));
    const uint32_t s16 = e4m3x2_to_f16x2(static_cast<uint16_t>(scales[r * SB + g])) & 0xFFFFu;
    const uint32_t s2 = s16 | (s16 << 16);
    lo = make_uint4(hmul2_u32(e2m1x2_byte_to_f16x2<0>(w.x), s2), hmul2_u32(e2m1x2_byte_to_f16x2<1>(w.x), s2),
                    hmul2_u32(e2m1x2_byte_to_f16x2<2>(w.x), s2), hmul2_u32(e2m1x2_byte_to_f16x2<3>(w.x), s2));
    hi = make_uint4(hmul2_u32(e2m1x2_byte_to_f16x2<0>(w.y), s2), hmul2_u32(e2m1x2_byte_to_f16x2<1>(w.y), s2),
                    hmul2_u32(e2m1x2_byte_to_f16x2<2>(w.y), s2), hmul2_u32(e2m1x2_byte_to_f16x2<3>(w.y), s2));
  }
}

// Factor of key r of a raw tile: FP8-row its row scale, INT8-G64 its 2^e,
// NVFP4 1 (the scales are inside the f16 values).
template <int KIND, int D>
__device__ __forceinline__ float key_factor(const uint8_t* scales, int r) {
  constexpr int SB = scale_row_bytes<KIND>(D);
  if constexpr (KIND == KIND_FP8) return __half2float(*reinterpret_cast<const __half*>(scales + r * SB));
  else if constexpr (KIND == KIND_INT8) return __uint_as_float(static_cast<uint32_t>(127 + int8_row_shift<D>(scales + r * SB)) << 23);
  else return 1.f;
}

// One converter thread's share of a page tile, in units of (key r, 16-dim
// group g): key r = (ct & 7) + 8 ((ct >> 3) & 7) and the UPT groups
// UPT (ct >> 6) + [0, UPT), so every unit of a thread shares its key (the
// INT8 key shift is computed once).  Eight consecutive threads take eight
// consecutive keys of one group, so the swizzled 16-byte loads and stores are
// free of bank conflicts; the next eight threads take their groups one step
// ahead, which keeps the 8-byte NVFP4 loads (16 threads per access) apart.
// NCT, the number of converter threads, is a multiple of 64; keys at or past
// `kvalid` become zeros.
//
// SPLIT (INT8-G64 only): the tile is written twice, as k1 = f16(c s') and, at
// f16 + 64 D 2, as the negated remainder k2' = k1 - c s', with s' = s_g 2^-e
// the binary16 scale.  c s' is a multiple of 2^-24 with at most 7 + 11
// significant bits, so the remainder (at most 7 bits, the same multiple) is an
// f16 value and k1 - k2' = c s' exactly: one f16 FMA per pair, fma(c, -s', k1),
// gives it, and the MMA that reads k2' negates its B operand.
template <int KIND, int D, int RB, int NCT, bool SPLIT = false>
__device__ __forceinline__ void convert_tile(const uint8_t* raw, int raw_codes, uint8_t* f16, int ct, int kvalid) {
  constexpr int GPR = D / 16;            // 16-dim groups per key
  constexpr int UPT = (64 * GPR) / NCT;  // units per thread
  static_assert(UPT * NCT == 64 * GPR && UPT >= 1, "converter units");
  static_assert(!SPLIT || KIND == KIND_INT8, "split tiles are for INT8-G64 keys");
  // a thread's UPT groups start at a multiple of UPT, so with 16 UPT dividing
  // 64 they share one INT8-G64 scale group
  static_assert(KIND != KIND_INT8 || 64 % (16 * UPT) == 0, "one scale group per thread");
  constexpr int SB = scale_row_bytes<KIND>(D);
  const uint8_t* scales = raw + raw_codes;
  const int r = (ct & 7) + 8 * ((ct >> 3) & 7);  // the thread's key
  int gg[UPT];
#pragma unroll
  for (int k = 0; k < UPT; ++k) gg[k] = UPT * (ct >> 6) + (k + ((ct >> 3) & 1)) % UPT;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (r >= kvalid) {  // a key at or past the frontier: zeros in every tile
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      const uint32_t o0 = f16_off(r, 16 * gg[k]), o1 = f16_off(r, 16 * gg[k] + 8);
      *reinterpret_cast<uint4*>(f16 + o0) = zero;
      *reinterpret_cast<uint4*>(f16 + o1) = zero;
      if constexpr (SPLIT) {
        *reinterpret_cast<uint4*>(f16 + 128 * D + o0) = zero;
        *reinterpret_cast<uint4*>(f16 + 128 * D + o1) = zero;
      }
    }
    return;
  }
  if constexpr (KIND == KIND_INT8) {
    // code times the key's shifted binary16 scale s' = s_g 2^-e (once per
    // thread; exact unless the shift takes it below binary16's normal range),
    // the product rounded once (k1); SPLIT also stores the remainder k2
    const float shift = pow2_neg(int8_row_shift<D>(scales + r * SB));
    const __half s16 =
        __float2half_rn(__half2float(*reinterpret_cast<const __half*>(scales + r * SB + 2 * ((16 * gg[0]) / 64))) * shift);
    const uint32_t s2 = pack_h2(s16, s16), s2n = s2 ^ 0x80008000u;  // s', -s'
    // every raw load of the thread before any store (the stores could alias)
    uint4 w[UPT];
#pragma unroll
    for (int k = 0; k < UPT; ++k) w[k] = *reinterpret_cast<const uint4*>(raw + raw_off<RB>(r, 16 * gg[k]));
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      const uint32_t wv[4] = {w[k].x ^ 0x80808080u, w[k].y ^ 0x80808080u, w[k].z ^ 0x80808080u,
                              w[k].w ^ 0x80808080u};
      uint32_t k1[8], k2[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t c0 = s8pair_flipped_to_f16x2<0>(wv[q]);
        const uint32_t c1 = s8pair_flipped_to_f16x2<1>(wv[q]);
        k1[2 * q] = hmul2_u32(c0, s2);
        k1[2 * q + 1] = hmul2_u32(c1, s2);
        if constexpr (SPLIT) {
          k2[2 * q] = hfma2_u32(c0, s2n, k1[2 * q]);
          k2[2 * q + 1] = hfma2_u32(c1, s2n, k1[2 * q + 1]);
        }
      }
      const uint32_t o0 = f16_off(r, 16 * gg[k]), o1 = f16_off(r, 16 * gg[k] + 8);
      *reinterpret_cast<uint4*>(f16 + o0) = make_uint4(k1[0], k1[1], k1[2], k1[3]);
      *reinterpret_cast<uint4*>(f16 + o1) = make_uint4(k1[4], k1[5], k1[6], k1[7]);
      if constexpr (SPLIT) {
        *reinterpret_cast<uint4*>(f16 + 128 * D + o0) = make_uint4(k2[0], k2[1], k2[2], k2[3]);
        *reinterpret_cast<uint4*>(f16 + 128 * D + o1) = make_uint4(k2[4], k2[5], k2[6], k2[7]);
      }
    }
  } else {
    uint4 lo[UPT], hi[UPT];
    // every raw load of the thread before any store (the stores could alias)
#pragma unroll
    for (int k = 0; k < UPT; ++k) convert16<KIND, D, RB>(raw, scales, r, gg[k], lo[k], hi[k]);
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      *reinterpret_cast<uint4*>(f16 + f16_off(r, 16 * gg[k])) = lo[k];
      *reinterpret_cast<uint4*>(f16 + f16_off(r, 16 * gg[k] + 8)) = hi[k];
    }
  }
}

}  // namespace nk
