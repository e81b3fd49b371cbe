// diff_decode.cuh -- differential attention of decode / verify tokens over the
// typed KV pool (kernel template; instantiated per profile in
// diff_decode_*.cu): split-K over pages, each page read once for both maps.
//
// For KV heads 2j, 2j + 1 (keys K1, K2; values V = [V1 V2]) and the query rows
// of the heads that share them, o = softmax(Q1 K1^T) V - lambda softmax(Q2 K2^T) V.
// Up to 8 query rows a map (more go to diff_tile.cuh).  A CTA owns one (row b, pair
// j, page range) and stages the four code tiles of a page together.  Its eight
// consumer warps are four slabs of 16 keys times two sides: the warp of side m
//   * computes S_m = K_m Q_m^T of its slab and the softmax of map m (its own
//     running maximum, moved lazily as in decode.cuh),
//   * hands P_m (and the rescale factors) to the other side's warp through
//     shared memory: one exchange of a few registers per lane and page,
//   * multiplies V_m's half of the dims by both maps' weights:
//     O_1[:, m half] += V_m^T P_1^T, O_2[:, m half] += V_m^T P_2^T.
// So every code is converted once, S is computed once, and only P V is done for
// both maps.  Up to 4 query rows (PACK) the two maps' weights fill one 8-column
// operand: map 1 in columns 0-3, map 2 in columns 4-7, half the MMAs and
// accumulators.
//
// Partials of (map, query row) go to the workspace, for the join (diff_decode.cu).
#pragma once

#include "diff.cuh"

namespace nk {

struct DiffDecodeArgs {
  const __nv_bfloat16* q;  // [B][T][Hq][D]
  const int32_t* tables;
  const int32_t* table_rows;
  const int32_t* frontiers;
  const uint8_t* ks;  // scale planes of the layer (nullptr for BF16)
  const uint8_t* vs;
  float2* ws_ml;  // [pair][ctas][2][RB] (m, l)
  float* ws_o;    // [pair][ctas][2][RB][2 D]
  int* status;
  float softmax_scale;
  int B, T, Hq, H, G, L, M, C;
  int ctas;  // CTAs (= partial slots) per pair
  int head_major;
};

constexpr int diff_align(int x, int a) { return (x + a - 1) / a * a; }

template <int KIND>
constexpr int diff_code_bytes(int D) {
  return KIND == KIND_BF16 ? 2 * D : KIND == KIND_NVFP4 ? D / 2 : D;
}
template <int KIND>
constexpr int diff_scale_bytes(int D) {
  return KIND == KIND_BF16 ? 0 : KIND == KIND_INT8 ? 2 * (D / 64) : KIND == KIND_FP8 ? 2 : D / 16;
}

template <int KK, int KV, int D, bool PACK>
struct DiffCfg {
  static constexpr int NW = 8, NCONS = 32 * NW, THREADS = NCONS + 32;
  static constexpr int R = 8;             // columns of one map's S
  static constexpr int RB = PACK ? 4 : R; // query rows of a partial
  static constexpr int NT = PACK ? 1 : 2; // column tiles of P V
  static constexpr int KCB = diff_code_bytes<KK>(D), VCB = diff_code_bytes<KV>(D);
  static constexpr int KSB = diff_scale_bytes<KK>(D), VSB = diff_scale_bytes<KV>(D);
  static constexpr int K_RB = KCB < 128 ? KCB : 128, V_RB = VCB < 128 ? VCB : 128;
  static constexpr int K_TILE = 64 * KCB, V_TILE = 64 * VCB, KS_TILE = 64 * KSB, VS_TILE = 64 * VSB;
  static constexpr int OFF_V = 2 * K_TILE, OFF_KS = OFF_V + 2 * V_TILE, OFF_VS = OFF_KS + 2 * KS_TILE;
  static constexpr int STAGE = diff_align(OFF_VS + 2 * VS_TILE, 1024);
  static_assert(K_TILE % 1024 == 0 && V_TILE % 1024 == 0, "tiles keep the swizzle's alignment");
  static constexpr int TX_BYTES = 2 * (K_TILE + V_TILE + KS_TILE + VS_TILE);
  static constexpr bool MMA_BF16 = KK == KIND_BF16;
  static constexpr int PARTS = MMA_BF16 ? 2 : 1;  // bf16 weights as hi + lo
  static constexpr int OREGS = D / 16 * NT * 4;
  // CTAs per SM: the accumulators and the tiles of a page decide
  static constexpr int MINB = OREGS > 64 || STAGE > 48 * 1024 ? 1 : 2;
  static constexpr int Q_PITCH = D * 2 + 32;
  static constexpr int XW = PARTS * 2 + 3;  // words a lane hands over
  static constexpr int VW_BYTES = KV == KIND_BF16 ? 0 : 16 * D * 2;  // a warp's 16 keys of V as f16
  static constexpr int O_PITCH = 2 * D + 4;  // floats: rows of the combine in different banks
  static constexpr int COMB = 4 * 2 * RB * O_PITCH * 4;
  static constexpr int REST = 2 * R * Q_PITCH + 2 * NW * 32 * XW * 4 + 20 * R * 4 + 1024 + 512;
  static constexpr int BUDGET = (MINB == 1 ? 226 : 113) * 1024 - REST - NW * VW_BYTES;
  static constexpr int NSTAGE = BUDGET / STAGE < 2 ? 2 : BUDGET / STAGE > 8 ? 8 : BUDGET / STAGE;
  // V slabs lie behind the ring; both are free for the combine at the end
  static constexpr int OFF_VW = NSTAGE * STAGE;
  static constexpr int FREE = OFF_VW + NW * VW_BYTES;
  static constexpr int OFF_Q = diff_align(FREE > COMB ? FREE : COMB, 128);
  static constexpr int OFF_X = OFF_Q + 2 * R * Q_PITCH;
  static constexpr int OFF_RED = OFF_X + 2 * NW * 32 * XW * 4;  // m, l [4][2][R] each, M, L [2][R]
  static constexpr int OFF_BAR = diff_align(OFF_RED + 20 * R * 4, 16);
  static constexpr int SMEM = OFF_BAR + 2 * NSTAGE * 8 + 32 * 4 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

template <int KIND>
__device__ __forceinline__ int diff_q_dim(int s, int i, int c) {
  if constexpr (KIND == KIND_BF16) return 16 * s + 2 * c + (i & 1) + (i >> 1) * 8;
  else if constexpr (KIND == KIND_NVFP4) return 32 * (s >> 1) + 8 * c + 4 * (s & 1) + i;
  else return 16 * s + 4 * c + i;
}

template <int KIND, bool HI>
__device__ __forceinline__ uint32_t diff_cvt_pair(uint32_t w) {
  if constexpr (KIND == KIND_INT8) return s8pair_to_f16x2(__byte_perm(w, 0, HI ? 0x3322 : 0x1100));
  else return e4m3x2_to_f16x2(static_cast<uint16_t>(HI ? (w >> 16) : (w & 0xFFFFu)));
}

__device__ __forceinline__ uint32_t diff_movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void diff_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float f16_at(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }

// S (16 keys of slab `slab` x 8 rows) = K Q^T over a staged K tile of one head,
// its scales applied: INT8 group and FP8 row scales multiply fp32 sums, NVFP4
// scales the f16 operand (an exact product).  q: the operands of the k-steps.
template <int KK, int D>
__device__ __forceinline__ void diff_scores(const uint8_t* tile, const uint8_t* scales, int slab, int lane,
                                            const uint32_t (&q)[D / 16][2], float (&S)[4]) {
  constexpr int KCB = diff_code_bytes<KK>(D), KSB = diff_scale_bytes<KK>(D), RB = KCB < 128 ? KCB : 128;
  const int r = lane >> 2, c = lane & 3;
  const int ld = 16 * slab + (lane & 7) + ((lane >> 3) & 1) * 8;  // ldmatrix row of this lane
  const int k0 = 16 * slab + r, k1 = k0 + 8;                      // keys of this lane's S rows
  const uint32_t base = smem_u32(tile);
  S[0] = S[1] = S[2] = S[3] = 0.f;
  if constexpr (KK == KIND_BF16) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const int col = (2 * s + (lane >> 4)) * 16;
      uint32_t A[4];
      ldsm_x4(base + (col / 128) * (64 * 128) + swz<128>(ld, col % 128), A[0], A[1], A[2], A[3]);
      mma16816<true>(S, A, q[s][0], q[s][1]);
    }
  } else if constexpr (KK == KIND_NVFP4) {
#pragma unroll
    for (int cw = 0; cw < KCB / 16; cw += 2) {  // two 16-byte chunks of 32 dims
      const int col = (cw + (lane >> 4)) * 16;
      uint32_t d[4];
      ldsm_x4(base + (col / RB) * (64 * RB) + swz<RB>(ld, col % RB), d[0], d[1], d[2], d[3]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int blk = 2 * (cw + u) + (c >> 1);
        const uint32_t s0 = e4m3x2_to_f16x2(scales[k0 * KSB + blk]) & 0xFFFFu;
        const uint32_t s1 = e4m3x2_to_f16x2(scales[k1 * KSB + blk]) & 0xFFFFu;
        const uint32_t f0 = s0 | (s0 << 16), f1 = s1 | (s1 << 16);
        const uint32_t w0 = d[2 * u], w1 = d[2 * u + 1];
        const uint32_t A0[4] = {hmul2_u32(e2m1x2_byte_to_f16x2<0>(w0), f0), hmul2_u32(e2m1x2_byte_to_f16x2<0>(w1), f1),
                                hmul2_u32(e2m1x2_byte_to_f16x2<1>(w0), f0), hmul2_u32(e2m1x2_byte_to_f16x2<1>(w1), f1)};
        const uint32_t A1[4] = {hmul2_u32(e2m1x2_byte_to_f16x2<2>(w0), f0), hmul2_u32(e2m1x2_byte_to_f16x2<2>(w1), f1),
                                hmul2_u32(e2m1x2_byte_to_f16x2<3>(w0), f0), hmul2_u32(e2m1x2_byte_to_f16x2<3>(w1), f1)};
        const int s = 2 * (cw + u);
        mma16816<false>(S, A0, q[s][0], q[s][1]);
        mma16816<false>(S, A1, q[s + 1][0], q[s + 1][1]);
      }
    }
  } else {  // 8-bit codes: 16 dims per 16-byte chunk
    float Sg[4];
#pragma unroll
    for (int cw = 0; cw < KCB / 16; cw += 2) {
      if constexpr (KK == KIND_INT8) {
        if ((cw & 3) == 0) Sg[0] = Sg[1] = Sg[2] = Sg[3] = 0.f;
      }
      const int col = (cw + (lane >> 4)) * 16;
      uint32_t d[4];
      ldsm_x4(base + (col / RB) * (64 * RB) + swz<RB>(ld, col % RB), d[0], d[1], d[2], d[3]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t A[4] = {diff_cvt_pair<KK, false>(d[2 * u]), diff_cvt_pair<KK, false>(d[2 * u + 1]),
                               diff_cvt_pair<KK, true>(d[2 * u]), diff_cvt_pair<KK, true>(d[2 * u + 1])};
        mma16816<false>(KK == KIND_INT8 ? Sg : S, A, q[cw + u][0], q[cw + u][1]);
      }
      if constexpr (KK == KIND_INT8) {
        if ((cw & 3) == 2) {  // end of a 64-dim group
          const float g0 = f16_at(scales + k0 * KSB + 2 * (cw >> 2)), g1 = f16_at(scales + k1 * KSB + 2 * (cw >> 2));
          S[0] = fmaf(Sg[0], g0, S[0]);
          S[1] = fmaf(Sg[1], g0, S[1]);
          S[2] = fmaf(Sg[2], g1, S[2]);
          S[3] = fmaf(Sg[3], g1, S[3]);
        }
      }
    }
    if constexpr (KK == KIND_FP8) {
      const float g0 = f16_at(scales + k0 * KSB), g1 = f16_at(scales + k1 * KSB);
      S[0] *= g0, S[1] *= g0, S[2] *= g1, S[3] *= g1;
    }
  }
}

// The slab's 16 keys x D dims of a staged quantized V tile as f16 in `vw`
// (64-dim blocks of 16 rows x 128 bytes, 128-byte swizzle), scales applied, keys
// past the frontier zero (`live`: of this lane's key).  Lane: key lane & 15, dims
// [32 dh, +32) of every block, dh = lane >> 4.
template <int KV, int D>
__device__ __forceinline__ void diff_values(const uint8_t* tile, const uint8_t* scales, uint8_t* vw, int slab, int lane,
                                            bool live, uint32_t lift2) {
  constexpr int VCB = diff_code_bytes<KV>(D), VSB = diff_scale_bytes<KV>(D), RB = VCB < 128 ? VCB : 128;
  const int kr = lane & 15, dh = lane >> 4, key = 16 * slab + kr;
#pragma unroll
  for (int q = 0; q < D / 64; ++q) {
    uint8_t* blk = vw + q * (16 * 128);
    const int d0 = 64 * q + 32 * dh;
    if constexpr (KV == KIND_NVFP4) {
      const int col = d0 / 2;
      const uint4 w = *reinterpret_cast<const uint4*>(tile + (col / RB) * (64 * RB) + swz<RB>(key, col % RB));
      // finite codes: a zero scale zeroes a key past the frontier
      const uint32_t s2 = live ? e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(scales + key * VSB + d0 / 16)) : 0u;
      const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {  // 16 dims, one scale group
        const uint32_t sq = __byte_perm(s2, 0, sub ? 0x3232 : 0x1010);
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          h[4 * k + 0] = hmul2_u32(e2m1x2_byte_to_f16x2<0>(wv[2 * sub + k]), sq);
          h[4 * k + 1] = hmul2_u32(e2m1x2_byte_to_f16x2<1>(wv[2 * sub + k]), sq);
          h[4 * k + 2] = hmul2_u32(e2m1x2_byte_to_f16x2<2>(wv[2 * sub + k]), sq);
          h[4 * k + 3] = hmul2_u32(e2m1x2_byte_to_f16x2<3>(wv[2 * sub + k]), sq);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(blk + swz<128>(kr, 64 * dh + 32 * sub + 16 * k)) =
              make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
      }
    } else {
      const uint16_t* sp = reinterpret_cast<const uint16_t*>(scales + key * VSB);
      const uint32_t s1 = KV == KIND_INT8 ? sp[d0 / 64] : sp[0];
      // INT8 codes are finite; FP8 codes may encode NaN and are selected away
      const uint32_t s2 = KV == KIND_INT8 && !live ? 0u : hmul2_u32(s1 | (s1 << 16), lift2);
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const int dd = d0 + 16 * sub;
        const uint4 w = *reinterpret_cast<const uint4*>(tile + (dd / RB) * (64 * RB) + swz<RB>(key, dd % RB));
        const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[2 * k] = hmul2_u32(diff_cvt_pair<KV, false>(wv[k]), s2);
          h[2 * k + 1] = hmul2_u32(diff_cvt_pair<KV, true>(wv[k]), s2);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(blk + swz<128>(kr, 64 * dh + 32 * sub + 16 * k)) =
              KV == KIND_INT8 || live ? make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3])
                                      : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
}

template <int KK, int KV, int D, bool PACK>
__global__ void __launch_bounds__((DiffCfg<KK, KV, D, PACK>::THREADS), (DiffCfg<KK, KV, D, PACK>::MINB))
    diff_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       DiffDecodeArgs a) {
  using Cfg = DiffCfg<KK, KV, D, PACK>;
  constexpr int R = Cfg::R, RB = Cfg::RB, NT = Cfg::NT, NSTAGE = Cfg::NSTAGE, NW = Cfg::NW, NCONS = Cfg::NCONS;
  constexpr int PARTS = Cfg::PARTS, MT = D / 16, XW = Cfg::XW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem + Cfg::OFF_Q;                                 // [2][R][Q_PITCH]
  uint32_t* sx = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_X);   // [2][NW][XW][32]
  float* red_m = reinterpret_cast<float*>(smem + Cfg::OFF_RED);    // [4][2][R]
  float* red_l = red_m + 8 * R;
  float* row_M = red_l + 8 * R;                                    // [2][R]
  float* row_L = row_M + 2 * R;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* empty = full + NSTAGE;
  int* s_flags = reinterpret_cast<int*>(empty + NSTAGE);  // [0] abort
  int* s_F = s_flags + 4;                                 // [8]
  int* s_row = s_flags + 12;                              // [8]
  float* s_qmax = reinterpret_cast<float*>(s_flags + 20); // [8]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int slab = warp >> 1, side = warp & 1;  // consumers: keys [16 slab, +16), map and V half
  const int cta = blockIdx.x, pair = blockIdx.y;

  if (tid == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], NW);
    }
    s_flags[0] = 0;
    fence_barrier_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  griddep_wait();  // pages, lengths and q may come from the kernel ahead
  griddep_launch_dependents();
  if (tid < a.B)
    s_F[tid] = diff_length(a.frontiers, a.table_rows, tid, a.L, a.C, &s_row[tid],
                           cta == 0 && pair == 0 ? a.status : nullptr);
  __syncthreads();

  // ---- which (row, split) this CTA owns ----------------------------------------
  const int chunk = diff_chunk(s_F, a.B, a.ctas, kDiffMaxSplits);
  int b = -1, split = 0, npages = 0;
  for (int i = 0, at = 0; i < a.B; ++i) {
    const int np = (s_F[i] + 63) >> 6, ns = max(1, (np + chunk - 1) / chunk);
    if (cta < at + ns) {
      b = i, split = cta - at, npages = np;
      break;
    }
    at += ns;
  }
  if (b < 0) return;
  const int F = s_F[b], p0 = split * chunk;
  const int n = min(chunk, npages - p0);  // 0 only for a row without keys
  const int rows = a.T * a.G;  // query rows of a map

  // ---- producer warp --------------------------------------------------------------
  if (warp == NW) {
    const int32_t* table = a.tables + static_cast<int64_t>(s_row[b]) * a.L + p0;
    int gnext = 0;
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0) gnext = (i + lane < n) ? table[i + lane] : 0;
      int g = __shfl_sync(0xffffffffu, gnext, i & 31);
      int stop = 0;
      if (lane == 0) {
        const int s = i % NSTAGE;
        if (i >= NSTAGE && !mbar_wait_bounded(&empty[s], ((i / NSTAGE) - 1) & 1, a.status)) {
          s_flags[0] = 1;
          stop = 1;
        } else {
          if (g < 0 || g >= a.M) {  // never copy from outside the pool
            set_status(a.status, NK_STATUS_PAGE_RANGE);
            g = 0;
          }
          uint8_t* st = smem + s * Cfg::STAGE;
          mbar_arrive_expect_tx(&full[s], Cfg::TX_BYTES);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int y = static_cast<int>(tile_row(g, 2 * pair + m, a.H, a.M, a.head_major));
#pragma unroll
            for (int j = 0; j < Cfg::KCB / Cfg::K_RB; ++j)
              tma_load_2d(st + m * Cfg::K_TILE + j * 64 * Cfg::K_RB, &tmk, j * Cfg::K_RB, y, &full[s]);
#pragma unroll
            for (int j = 0; j < Cfg::VCB / Cfg::V_RB; ++j)
              tma_load_2d(st + Cfg::OFF_V + m * Cfg::V_TILE + j * 64 * Cfg::V_RB, &tmv, j * Cfg::V_RB, y, &full[s]);
            if constexpr (Cfg::KS_TILE > 0) {
              bulk_load(st + Cfg::OFF_KS + m * Cfg::KS_TILE, a.ks + static_cast<int64_t>(y) * Cfg::KSB, Cfg::KS_TILE,
                        &full[s]);
              bulk_load(st + Cfg::OFF_VS + m * Cfg::VS_TILE, a.vs + static_cast<int64_t>(y) * Cfg::VSB, Cfg::VS_TILE,
                        &full[s]);
            }
          }
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) break;
    }
    return;  // the copies land in the shared memory of the still-running CTA
  }

  // ---- q rows of both maps to shared memory, f16 with a power-of-two prescale --------
  // Row t G + g of map m is q[b][t][2 (pair G + g) + m][:].  Quantized pages run
  // f16 MMAs: q is scaled by 2^e with max|q| 2^e in [2^14, 2^15) over the map's rows
  // (exact for every element above max|q| 2^-31) and the scores divide it out.
  // PACK: map 2's rows sit in columns 4-7.
  {
    const int st = tid & 127, m = tid >> 7;  // warps 0-3: map 0, 4-7: map 1
    float mx = 0.f;
    for (int i = st; i < R * (D / 8); i += 128) {
      const int col = i / (D / 8), d8 = i % (D / 8);
      const int qr = PACK ? col - 4 * m : col;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (qr >= 0 && qr < rows) {
        const int t = qr / a.G, g = qr % a.G;
        v = *reinterpret_cast<const uint4*>(
            a.q + ((static_cast<int64_t>(b) * a.T + t) * a.Hq + 2 * (pair * a.G + g) + m) * D + d8 * 8);
      }
      *reinterpret_cast<uint4*>(qs + (m * R + col) * Cfg::Q_PITCH + d8 * 16) = v;
      const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&v);
#pragma unroll
      for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(__bfloat162float(e[k])));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (lane == 0) s_qmax[warp] = mx;
  }
  asm volatile("bar.sync 1, %0;" ::"n"(NCONS) : "memory");
  const auto q_exponent = [&](int m) {
    float mx = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = fmaxf(mx, s_qmax[4 * m + w]);
    int ex = 0;
    if (mx > 0.f) frexpf(mx, &ex);
    return mx > 0.f ? min(15 - ex, 100) : 0;
  };
  float sc = a.softmax_scale * kDiffLog2e;
  if constexpr (!Cfg::MMA_BF16) {
    const float mul = ldexpf(1.f, q_exponent(tid >> 7));
    for (int i = tid & 127; i < R * D / 2; i += 128) {
      uint32_t* p = reinterpret_cast<uint32_t*>(qs + ((tid >> 7) * R + i / (D / 2)) * Cfg::Q_PITCH + (i % (D / 2)) * 4);
      const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(p);
      *p = pack_f16x2(__low2float(v) * mul, __high2float(v) * mul);
    }
    sc *= exp2f(-static_cast<float>(q_exponent(side)));
    asm volatile("bar.sync 1, %0;" ::"n"(NCONS) : "memory");
  }
  uint32_t q[D / 16][2];  // operands of this side's map
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const uint8_t* p = qs + (side * R + r) * Cfg::Q_PITCH;
    q[s][0] = *reinterpret_cast<const uint32_t*>(p + 2 * diff_q_dim<KK>(s, 0, c));
    q[s][1] = *reinterpret_cast<const uint32_t*>(p + 2 * diff_q_dim<KK>(s, 2, c));
  }

  // ---- running state: map `side` for the softmax, both maps for this half of V --------
  float nm[2] = {0.f, 0.f}, l_part[2] = {0.f, 0.f};  // minus the reference maximum; sum
  float o[MT][NT][4];                                // tiles: own map, the other's (PACK: one for both)
  int k_run = 0;  // O carries 2^k_run (INT8 / FP8 values near the f16 limit, v_lift)
  int lim[2];     // last key that a column's query sees
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int col = 2 * c + u, qr = PACK ? max(0, col - 4 * side) : col;
    lim[u] = min(F - a.T + qr / a.G, F - 1);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < NT; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
  // PACK: whether this lane's row r (of P^T) and columns 2c, 2c + 1 (of O) are the own map's
  const bool own_r = (r < 4) == (side == 0), own_c = (c < 2) == (side == 0);
  const int kr0 = 16 * slab + r, kr1 = kr0 + 8;

  // A wait that ran out makes the rest of the loop run on whatever the stages
  // hold, without waiting, so that the warps' barriers stay matched; the CTA
  // leaves without results.
  bool aborted = false;
  for (int i = 0; i < n; ++i) {
    const int s = i % NSTAGE;
    const uint8_t* st = smem + s * Cfg::STAGE;
    if (!aborted && !mbar_wait_bounded(&full[s], (i / NSTAGE) & 1, a.status)) aborted = true;
    const int key0 = (p0 + i) * 64;
    const uint8_t* vs_tile = st + Cfg::OFF_VS + side * Cfg::VS_TILE;

    int knew = k_run;
    if constexpr (KV == KIND_INT8 || KV == KIND_FP8) {  // the slab's largest value scale below the frontier
      const int vk = 16 * slab + (lane & 15);
      float smax = 0.f;
      if (key0 + vk < F) {
        if constexpr (KV == KIND_INT8) {
#pragma unroll
          for (int gi = lane >> 4; gi < D / 64; gi += 2) smax = fmaxf(smax, f16_at(vs_tile + vk * Cfg::VSB + 2 * gi));
        } else {
          smax = f16_at(vs_tile + vk * Cfg::VSB);
        }
      }
      knew = v_lift(__reduce_max_sync(0xffffffffu, __float_as_uint(smax)), k_run);
    }

    float S[4];
    diff_scores<KK, D>(st + side * Cfg::K_TILE, st + Cfg::OFF_KS + side * Cfg::KS_TILE, slab, lane, q, S);

    // ---- softmax of this side's map over the slab's keys (lazy reference, base 2) ------
    const int kg0 = key0 + kr0, kg1 = key0 + kr1;
    const bool first = i == 0;
    float alpha[2] = {1.f, 1.f}, top[2];
    S[0] = kg0 <= lim[0] ? fmaf(S[0], sc, nm[0]) : -INFINITY;
    S[1] = kg0 <= lim[1] ? fmaf(S[1], sc, nm[1]) : -INFINITY;
    S[2] = kg1 <= lim[0] ? fmaf(S[2], sc, nm[0]) : -INFINITY;
    S[3] = kg1 <= lim[1] ? fmaf(S[3], sc, nm[1]) : -INFINITY;
    top[0] = fmaxf(S[0], S[2]);
    top[1] = fmaxf(S[1], S[3]);
    bool rescale = false;
    if (__any_sync(0xffffffffu, first || top[0] > 8.f || top[1] > 8.f)) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float v = top[u];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        // the first page takes the exact maximum (a query's keys are a prefix:
        // one that sees none here sees none later), later ones the excess
        const float shift = first ? (v == -INFINITY ? 0.f : v) : fmaxf(v, 0.f);
        alpha[u] = first ? 0.f : ex2(-shift);
        rescale |= shift > 0.f;
        nm[u] -= shift;
        S[u] -= shift;
        S[2 + u] -= shift;
        l_part[u] *= alpha[u];
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      S[u] = ex2(S[u]);
      S[2 + u] = ex2(S[2 + u]);
      l_part[u] += S[u] + S[2 + u];
    }
    rescale = __any_sync(0xffffffffu, rescale) && !first;  // O is 0 before the first page

    // ---- P^T as B operands, and the exchange with the other side's warp -----------------
    uint32_t pb[PARTS][NT][2];
    float al[NT][2];
    {
      uint32_t mine[XW];
      if constexpr (Cfg::MMA_BF16) {  // bf16 weights as hi + lo (about 16 significant bits)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __nv_bfloat162 hi = __floats2bfloat162_rn(S[2 * h], S[2 * h + 1]);
          const __nv_bfloat162 lo = __floats2bfloat162_rn(S[2 * h] - __low2float(hi), S[2 * h + 1] - __high2float(hi));
          mine[h] = diff_movm(*reinterpret_cast<const uint32_t*>(&hi));
          mine[2 * (PARTS - 1) + h] = diff_movm(*reinterpret_cast<const uint32_t*>(&lo));
        }
      } else {
        mine[0] = diff_movm(pack_f16x2(S[0], S[1]));
        mine[1] = diff_movm(pack_f16x2(S[2], S[3]));
      }
      mine[2 * PARTS] = __float_as_uint(alpha[0]);
      mine[2 * PARTS + 1] = __float_as_uint(alpha[1]);
      mine[XW - 1] = rescale;
      uint32_t* to = sx + ((i & 1) * NW + warp) * (XW * 32) + lane;
      const uint32_t* from = sx + ((i & 1) * NW + (warp ^ 1)) * (XW * 32) + lane;
#pragma unroll
      for (int x = 0; x < XW; ++x) to[x * 32] = mine[x];
      asm volatile("bar.sync %0, 64;" ::"r"(2 + slab) : "memory");
      uint32_t other[XW];
#pragma unroll
      for (int x = 0; x < XW; ++x) other[x] = from[x * 32];
      rescale |= other[XW - 1] != 0u;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          const int x = 2 * part + h;
          if constexpr (PACK) {
            pb[part][0][h] = own_r ? mine[x] : other[x];
          } else {
            pb[part][0][h] = mine[x];
            pb[part][NT - 1][h] = other[x];
          }
        }
        const int x = 2 * PARTS + h;
        if constexpr (PACK) {
          al[0][h] = __uint_as_float(own_c ? mine[x] : other[x]);
        } else {
          al[0][h] = __uint_as_float(mine[x]);
          al[NT - 1][h] = __uint_as_float(other[x]);
        }
      }
    }
    if (rescale || knew != k_run) {
      const float kf = pow2i(knew - k_run);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[mt][j][0] *= al[j][0] * kf;
          o[mt][j][1] *= al[j][1] * kf;
          o[mt][j][2] *= al[j][0] * kf;
          o[mt][j][3] *= al[j][1] * kf;
        }
    }
    k_run = knew;

    // ---- O^T (D dims of half `side` x columns) += V^T P^T -----------------------------------
    const uint8_t* vtile = st + Cfg::OFF_V + side * Cfg::V_TILE;
    if constexpr (KV == KIND_BF16) {
      const int kvalid = F - key0, kk0 = 16 * slab + 2 * c;
      uint32_t mlo = 0xFFFFFFFFu, mhi = 0xFFFFFFFFu;  // stale values past the frontier become zero
      if (kvalid < 64) {
        mlo = (kk0 < kvalid ? 0x0000FFFFu : 0u) | (kk0 + 1 < kvalid ? 0xFFFF0000u : 0u);
        mhi = (kk0 + 8 < kvalid ? 0x0000FFFFu : 0u) | (kk0 + 9 < kvalid ? 0xFFFF0000u : 0u);
      }
      const int key = 16 * slab + (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int col = (16 * mt + 8 * ((lane >> 3) & 1)) * 2;
        uint32_t A[4];
        ldsm_x4_t(smem_u32(vtile) + (col / 128) * (64 * 128) + swz<128>(key, col % 128), A[0], A[1], A[2], A[3]);
        A[0] &= mlo, A[1] &= mlo, A[2] &= mhi, A[3] &= mhi;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int part = 0; part < PARTS; ++part) mma16816<true>(o[mt][j], A, pb[part][j][0], pb[part][j][1]);
      }
    } else {
      uint8_t* vw = smem + Cfg::OFF_VW + warp * Cfg::VW_BYTES;
      const uint32_t lift2 = static_cast<uint32_t>(k_run + 15) * 0x04000400u;  // f16x2 of 2^k_run
      // (the previous page's fragments were read before the barrier above)
      diff_values<KV, D>(vtile, vs_tile, vw, slab, lane, key0 + 16 * slab + (lane & 15) < F, lift2);
      __syncwarp();
      const int key = (lane & 7) + ((lane >> 4) & 1) * 8;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int col = (16 * (mt & 3) + 8 * ((lane >> 3) & 1)) * 2;
        uint32_t A[4];
        ldsm_x4_t(smem_u32(vw + (mt >> 2) * (16 * 128)) + swz<128>(key, col), A[0], A[1], A[2], A[3]);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816<false>(o[mt][j], A, pb[0][j][0], pb[0][j][1]);
      }
    }
    __syncwarp();
    if (lane == 0) diff_arrive(&empty[s]);
  }

  // ---- the slabs' results into one partial ----------------------------------------------
  // Sums of a column over the lanes that hold its keys; the reference maximum is
  // -inf for a query that saw no key (one that saw a key has l >= 1; NaN stays).
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float v = l_part[u];
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    v += __shfl_xor_sync(0xffffffffu, v, 16);
    if (r == 0) {
      red_m[(slab * 2 + side) * R + 2 * c + u] = v == 0.f ? -INFINITY : -nm[u];
      red_l[(slab * 2 + side) * R + 2 * c + u] = v;
    }
  }
  if (aborted && lane == 0) s_flags[0] = 1;
  asm volatile("bar.sync 1, %0;" ::"n"(NCONS) : "memory");
  if (s_flags[0]) {  // copies in flight land before the CTA leaves
    if (tid == 0)
      for (int k = max(0, n - NSTAGE); k < n; ++k)
        mbar_wait_bounded(&full[k % NSTAGE], (k / NSTAGE) & 1, a.status, 100000000ull);
    return;
  }
  if (tid < 2 * R) {
    float M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, red_m[w * 2 * R + tid]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float l = red_l[w * 2 * R + tid];
      if (l != 0.f) Ls += l * ex2(red_m[w * 2 * R + tid] - M);
    }
    row_M[tid] = M;
    row_L[tid] = Ls;
  }
  asm volatile("bar.sync 1, %0;" ::"n"(NCONS) : "memory");
  float* comb = reinterpret_cast<float*>(smem);  // [4 slabs][2 maps][RB][O_PITCH], over the ring
  {
    const float unlift = pow2i(-k_run);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int col = 2 * c + u, map = PACK ? c >> 1 : side ^ j;
        const int qr = PACK ? col & 3 : col;
        const float m = red_m[(slab * 2 + map) * R + col];
        const float f = m == -INFINITY ? 0.f : ex2(m - row_M[map * R + col]) * unlift;
        float* dst = comb + ((slab * 2 + map) * RB + qr) * Cfg::O_PITCH + side * D + r;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          dst[16 * mt] = o[mt][j][u] * f;
          dst[16 * mt + 8] = o[mt][j][2 + u] * f;
        }
      }
  }
  asm volatile("bar.sync 1, %0;" ::"n"(NCONS) : "memory");
  const int64_t slot = static_cast<int64_t>(pair) * a.ctas + cta;
  for (int idx = tid; idx < 2 * rows * (D / 2); idx += NCONS) {
    const int d = (idx % (D / 2)) * 4, map = idx / (D / 2) / rows, qr = idx / (D / 2) % rows;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(comb + ((w * 2 + map) * RB + qr) * Cfg::O_PITCH + d);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    *reinterpret_cast<float4*>(a.ws_o + ((slot * 2 + map) * RB + qr) * (2 * D) + d) = v;
  }
  if (tid < 2 * rows) {
    const int map = tid / rows, qr = tid % rows, col = PACK ? qr + 4 * map : qr;
    a.ws_ml[(slot * 2 + map) * RB + qr] = make_float2(row_M[map * R + col], row_L[map * R + col]);
  }
}

template <int KK, int KV, int D, bool PACK>
cudaError_t launch_diff_decode(const nk_pool* p, int layer, const DiffDecodeArgs& a, cudaStream_t s) {
  using Cfg = DiffCfg<KK, KV, D, PACK>;
  auto k = diff_decode_kernel<KK, KV, D, PACK>;
  static std::atomic<uint64_t> granted{0};
  const cudaError_t e = grant_smem(granted, k, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(a.ctas, a.H / 2), dim3(Cfg::THREADS), Cfg::SMEM, s, p->tmap[layer * 2 + 0],
                    p->tmap[layer * 2 + 1], a);
}

template <int KK, int KV, int D, bool PACK>
int diff_ctas_per_sm() {
  using Cfg = DiffCfg<KK, KV, D, PACK>;
  static std::atomic<uint64_t> granted{0};
  static std::atomic<int> cached[64];
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return 1;
  int n = device < 64 ? cached[device].load(std::memory_order_relaxed) : 0;
  if (n) return n;
  auto k = diff_decode_kernel<KK, KV, D, PACK>;
  if (grant_smem(granted, k, Cfg::SMEM) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, Cfg::THREADS, Cfg::SMEM) != cudaSuccess || n < 1)
    n = 1;
  if (device < 64) cached[device].store(n, std::memory_order_relaxed);
  return n;
}

// Per-profile entries (diff_decode_*.cu).  pack: up to 4 query rows.  a ==
// nullptr: only the CTAs per SM are asked, in *per_sm.
using DiffDecodeFn = cudaError_t (*)(const nk_pool*, int layer, const DiffDecodeArgs* a, bool pack, int* per_sm,
                                     cudaStream_t);

template <int KK, int KV, int D, bool PACK>
cudaError_t diff_decode_one(const nk_pool* p, int layer, const DiffDecodeArgs* a, int* per_sm, cudaStream_t s) {
  if (a) return launch_diff_decode<KK, KV, D, PACK>(p, layer, *a, s);
  *per_sm = diff_ctas_per_sm<KK, KV, D, PACK>();
  return cudaSuccess;
}

template <int KK, int KV>
cudaError_t diff_decode_dispatch(const nk_pool* p, int layer, const DiffDecodeArgs* a, bool pack, int* per_sm,
                                 cudaStream_t s) {
  if (p->desc.head_dim == 64)
    return pack ? diff_decode_one<KK, KV, 64, true>(p, layer, a, per_sm, s)
                : diff_decode_one<KK, KV, 64, false>(p, layer, a, per_sm, s);
  return pack ? diff_decode_one<KK, KV, 128, true>(p, layer, a, per_sm, s)
              : diff_decode_one<KK, KV, 128, false>(p, layer, a, per_sm, s);
}

cudaError_t diff_decode_bf16(const nk_pool*, int, const DiffDecodeArgs*, bool, int*, cudaStream_t);
cudaError_t diff_decode_int8(const nk_pool*, int, const DiffDecodeArgs*, bool, int*, cudaStream_t);
cudaError_t diff_decode_fp8(const nk_pool*, int, const DiffDecodeArgs*, bool, int*, cudaStream_t);
cudaError_t diff_decode_nvfp4(const nk_pool*, int, const DiffDecodeArgs*, bool, int*, cudaStream_t);
cudaError_t diff_decode_k8v4(const nk_pool*, int, const DiffDecodeArgs*, bool, int*, cudaStream_t);

}  // namespace nk
