// diff_decode.cuh -- differential attention of decode / verify tokens over the
// typed KV pool (kernel template; instantiated per profile in
// diff_decode_*.cu): split-K over pages, each page read once for both maps.
//
// For KV heads 2j, 2j + 1 (keys K1, K2; values V = [V1 V2]) and the query rows
// of the heads that share them, o = softmax(Q1 K1^T) V - lambda softmax(Q2 K2^T) V.
// Up to 8 query rows a map (the rest goes to diff_tile.cuh).  A CTA, one per SM, owns one
// (row b, pair j, page range) and NG groups of four warps, each with a ring of SG stages of
// its own and every NG-th page; each warp owns 16 keys of a page, for both maps and both
// value heads, so that every code is converted once and no warp waits for another's
// results, and copies one of the group's four tiles (no producer: its warp would cost the
// others registers):
//   QK   mma.m16n8k16, keys as M.  Up to 4 query rows (PACK) both maps fill the 8
//        columns (map 1 in 0-3, map 2 in 4-7): S1 = K1 [Q1 Q2]^T, S2 = K2 [Q1 Q2]^T,
//        of which a lane keeps the one of its columns' map; 8 rows take a tile a map.
//   softmax, base 2, per column over the warp's keys, with a lazy reference.
//   PV   O^T += V^T P^T, dims as M, 64 dims at a time: the warp converts its 16 keys
//        to f16 in 2 KB of its own and reads them back transposed.  FP8-row and
//        INT8-G64 scales multiply the weights instead of the values (32 a lane and
//        head), in fp32 and rounded once, lifted by a power of two per head (v_lift)
//        that O carries; weights over NVFP4 values carry 2^7 (kDiffWeightLift).
// Pages that all queries see whole (all but a row's last) run without masks; in the
// last one the warp zeroes its stale value rows in place.
//
// Two heads to a warp halved the instructions of a page against one head to each of
// two warps that exchange their weights (FP8-row, head_dim 128: 3800 warp instructions a
// page, whose issue bound that form at 46% of the copy rate).
//
// Measured (with the join, L2 cold): 8 requests of 25500 tokens, 16 heads over 4, FP8-row: 45
// us, 69% of the copy rate.  From 65536 to 131072 tokens a request, each further page at this
// share of the copy rate, with up to 4 query rows and with 5 to 8 (head_dim 128: two groups of
// warps instead of three, for the registers): BF16 more than 100% and the same, FP8-row 106%
// and 88%, K8V4 99% and 79%, INT8-G64 92% and 74%, NVFP4 65% and 50% (conversion and
// products bound the shares below 90%).  Beside the pages, the start (plan, first copies) and
// the join take 15 us of every call.
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
  static constexpr int RB = PACK ? 4 : 8;  // query rows of a map
  static constexpr int NT = PACK ? 1 : 2;  // column tiles: both maps, or one each
  static constexpr int KCB = diff_code_bytes<KK>(D), VCB = diff_code_bytes<KV>(D);
  static constexpr int KSB = diff_scale_bytes<KK>(D), VSB = diff_scale_bytes<KV>(D);
  static constexpr int K_RB = KCB < 128 ? KCB : 128, V_RB = VCB < 128 ? VCB : 128;
  static constexpr int K_TILE = 64 * KCB, V_TILE = 64 * VCB, KS_TILE = 64 * KSB, VS_TILE = 64 * VSB;
  static constexpr int OFF_V = 2 * K_TILE, OFF_KS = OFF_V + 2 * V_TILE, OFF_VS = OFF_KS + 2 * KS_TILE;
  static constexpr int STAGE = diff_align(OFF_VS + 2 * VS_TILE, 1024);
  static_assert(K_TILE % 1024 == 0 && V_TILE % 1024 == 0, "tiles keep the swizzle's alignment");
  static constexpr bool MMA_BF16 = KK == KIND_BF16;
  static constexpr bool VAL_FAC = KV == KIND_INT8 || KV == KIND_FP8;
  static constexpr int PARTS = MMA_BF16 ? 2 : 1;  // bf16 weights as hi + lo
  static constexpr int OREGS = 2 * D / 16 * NT * 4;
  static constexpr int Q_PITCH = D * 2 + 32;
  static constexpr int VW_BYTES = KV == KIND_BF16 ? 0 : 16 * 64 * 2;  // a warp's 16 keys x 64 dims of V as f16
  static constexpr int O_PITCH = 2 * D + 4;  // floats: rows of the combine in different banks
  // Stages that fit beside the rest of g groups
  static constexpr int stages(int g) {
    return (227 * 1024 - 1024 - 8 * NT * Q_PITCH - (8 * g + 2) * 2 * RB * 4 - 768 - 4 * g * VW_BYTES) / STAGE;
  }
  // Groups of four warps: as many as the accumulators' registers (128, 168 or 255 a
  // thread) and two stages for each allow
  static constexpr int NG_REGS = OREGS > 64 ? 2 : OREGS > 32 ? 3 : 4;
  static constexpr int groups(int g) { return g > 1 && stages(g) < 2 * g ? groups(g - 1) : g; }
  static constexpr int NG = groups(NG_REGS);
  static constexpr int SG = stages(NG) / NG < 8 ? stages(NG) / NG : 8;  // stages of a group
  static_assert(SG >= 2, "a stage is refilled while the next one is read");
  static constexpr int NW = 4 * NG, THREADS = 32 * NW, NSTAGE = SG * NG;
  static constexpr int COMB = NW * 2 * RB * O_PITCH * 4;
  // V blocks lie behind the ring; both are free for the combine at the end
  static constexpr int OFF_VW = NSTAGE * STAGE;
  static constexpr int FREE = OFF_VW + NW * VW_BYTES;
  static constexpr int OFF_Q = diff_align(FREE > COMB ? FREE : COMB, 128);
  static constexpr int OFF_RED = OFF_Q + 8 * NT * Q_PITCH;  // m, l [NW][2 RB] each, M, L [2 RB]
  static constexpr int OFF_BAR = diff_align(OFF_RED + (2 * NW + 2) * 2 * RB * 4, 16);
  static constexpr int SMEM = OFF_BAR + 2 * NSTAGE * 8 + 64 * 4 + 1024;
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

// The warp's 16 keys x 64 dims (block q) of a staged quantized V tile as f16 in
// `blk` (16 rows x 128 bytes, 128-byte swizzle): NVFP4 values with their scales (an
// exact product), INT8 and FP8 codes alone.  Lane: key lane & 15, dims [32 dh, +32) of
// the block, dh = lane >> 4.
template <int KV, int D>
__device__ __forceinline__ void diff_values(const uint8_t* tile, const uint8_t* scales, uint8_t* blk, int q, int slab,
                                            int lane) {
  constexpr int VCB = diff_code_bytes<KV>(D), VSB = diff_scale_bytes<KV>(D), RB = VCB < 128 ? VCB : 128;
  const int kr = lane & 15, dh = lane >> 4, key = 16 * slab + kr;
  const int d0 = 64 * q + 32 * dh;
  uint32_t w[8], h[16];
  if constexpr (KV == KIND_NVFP4) {
    const int col = d0 / 2;
    const uint4 x = *reinterpret_cast<const uint4*>(tile + (col / RB) * (64 * RB) + swz<RB>(key, col % RB));
    const uint32_t s2 = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(scales + key * VSB + d0 / 16));
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 8 dims; two words to a scale group
      const uint32_t sq = __byte_perm(s2, 0, k >> 1 ? 0x3232 : 0x1010);
      h[4 * k + 0] = hmul2_u32(e2m1x2_byte_to_f16x2<0>(w[k]), sq);
      h[4 * k + 1] = hmul2_u32(e2m1x2_byte_to_f16x2<1>(w[k]), sq);
      h[4 * k + 2] = hmul2_u32(e2m1x2_byte_to_f16x2<2>(w[k]), sq);
      h[4 * k + 3] = hmul2_u32(e2m1x2_byte_to_f16x2<3>(w[k]), sq);
    }
  } else {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const int dd = d0 + 16 * sub;
      const uint4 x = *reinterpret_cast<const uint4*>(tile + (dd / RB) * (64 * RB) + swz<RB>(key, dd % RB));
      w[4 * sub] = x.x, w[4 * sub + 1] = x.y, w[4 * sub + 2] = x.z, w[4 * sub + 3] = x.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[2 * k] = diff_cvt_pair<KV, false>(w[k]);
      h[2 * k + 1] = diff_cvt_pair<KV, true>(w[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint4*>(blk + swz<128>(kr, 64 * dh + 16 * k)) =
        make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
}

template <int KK, int KV, int D, bool PACK>
__global__ void __launch_bounds__((DiffCfg<KK, KV, D, PACK>::THREADS), 1)
    diff_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                       DiffDecodeArgs a) {
  using Cfg = DiffCfg<KK, KV, D, PACK>;
  constexpr int RB = Cfg::RB, NT = Cfg::NT, NSTAGE = Cfg::NSTAGE, NW = Cfg::NW, NG = Cfg::NG, SG = Cfg::SG;
  constexpr int PARTS = Cfg::PARTS, MT = D / 16;
  // How far the largest weight of a warp's first keys lies above 1, in base 2: f16 weights that
  // take no factor are stored as high as they may be (kDiffWeightLift)
  constexpr float TOP = Cfg::MMA_BF16 || Cfg::VAL_FAC ? 0.f : static_cast<float>(kDiffWeightLift);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem + Cfg::OFF_Q;                               // [8 NT columns][Q_PITCH]
  float* red_m = reinterpret_cast<float*>(smem + Cfg::OFF_RED);  // [NW][2][RB]
  float* red_l = red_m + 2 * NW * RB;
  float* row_M = red_l + 2 * NW * RB;                                 // [2][RB]
  float* row_L = row_M + 2 * RB;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* empty = full + NSTAGE;
  int* s_flags = reinterpret_cast<int*>(empty + NSTAGE);  // [0] abort
  float* s_qmax = reinterpret_cast<float*>(s_flags + 4);  // [2][NW]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int grp = warp >> 2, slab = warp & 3;  // keys [16 slab, +16) of pages grp, grp + NG, ..
  const int cta = blockIdx.x, pair = blockIdx.y;

  if (tid == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&full[s], 4);
      mbar_init(&empty[s], 4);
    }
    s_flags[0] = 0;
    fence_barrier_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  __syncthreads();
  griddep_wait();  // pages, lengths and q may come from the kernel ahead
  griddep_launch_dependents();
  const DiffSplit own = diff_split(diff_rows(a.frontiers, a.table_rows, a.B, a.L, a.C, a.ctas,
                                             cta == 0 && pair == 0 && warp == 0 ? a.status : nullptr),
                                   a.B, cta);
  if (own.b < 0) return;
  const int b = own.b, F = own.F, p0 = own.p0, n = own.n;
  const int rows = a.T * a.G;  // query rows of a map

  // ---- copies: a group's ring of SG stages, one of the four tiles from each warp ------
  const int ng = n > grp ? (n - grp + NG - 1) / NG : 0;  // pages of this group
  const int32_t* table = a.tables + static_cast<int64_t>(own.row) * a.L + p0 + grp;
  const int tm = slab & 1;  // warps 0, 1: the pair's keys; 2, 3: its values
  int gnext = 0;
  auto load = [&](int i) {  // page i of the group; called in order, by the whole warp
    if ((i & 31) == 0) gnext = (i + lane < ng) ? table[(i + lane) * NG] : 0;
    int g = __shfl_sync(0xffffffffu, gnext, i & 31);
    if (lane == 0) {
      if (g < 0 || g >= a.M) {  // never copy from outside the pool
        set_status(a.status, NK_STATUS_PAGE_RANGE);
        g = 0;
      }
      const int s = grp * SG + i % SG;
      uint8_t* st = smem + s * Cfg::STAGE;
      const int y = static_cast<int>(tile_row(g, 2 * pair + tm, a.H, a.M, a.head_major));
      if (slab < 2) {
        mbar_arrive_expect_tx(&full[s], Cfg::K_TILE + Cfg::KS_TILE);
#pragma unroll
        for (int j = 0; j < Cfg::KCB / Cfg::K_RB; ++j)
          tma_load_2d(st + tm * Cfg::K_TILE + j * 64 * Cfg::K_RB, &tmk, j * Cfg::K_RB, y, &full[s]);
        if constexpr (Cfg::KS_TILE > 0)
          bulk_load(st + Cfg::OFF_KS + tm * Cfg::KS_TILE, a.ks + static_cast<int64_t>(y) * Cfg::KSB, Cfg::KS_TILE,
                    &full[s]);
      } else {
        mbar_arrive_expect_tx(&full[s], Cfg::V_TILE + Cfg::VS_TILE);
#pragma unroll
        for (int j = 0; j < Cfg::VCB / Cfg::V_RB; ++j)
          tma_load_2d(st + Cfg::OFF_V + tm * Cfg::V_TILE + j * 64 * Cfg::V_RB, &tmv, j * Cfg::V_RB, y, &full[s]);
        if constexpr (Cfg::VS_TILE > 0)
          bulk_load(st + Cfg::OFF_VS + tm * Cfg::VS_TILE, a.vs + static_cast<int64_t>(y) * Cfg::VSB, Cfg::VS_TILE,
                    &full[s]);
      }
    }
    __syncwarp();
  };
  int issued = 0;
  for (; issued < min(SG, ng); ++issued) load(issued);

  // ---- q rows of both maps to shared memory, f16 with a power-of-two prescale --------
  // Column c of the 8 NT: map c / RB, row t G + g = c % RB, q[b][t][2 (pair G + g) + map].
  // Quantized pages run f16 MMAs: a map's q is scaled by 2^e with max|q| 2^e in [2^14,
  // 2^15) over its rows (exact for every element above max|q| 2^-31), and the scores
  // divide it out.
  float mx[2] = {0.f, 0.f};
  for (int i = tid; i < 8 * NT * (D / 8); i += 32 * NW) {
    const int col = i / (D / 8), d8 = i % (D / 8), m = col / RB, qr = col % RB;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (qr < rows) {
      const int t = qr / a.G, g = qr % a.G;
      v = *reinterpret_cast<const uint4*>(
          a.q + ((static_cast<int64_t>(b) * a.T + t) * a.Hq + 2 * (pair * a.G + g) + m) * D + d8 * 8);
    }
    *reinterpret_cast<uint4*>(qs + col * Cfg::Q_PITCH + d8 * 16) = v;
    const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&v);
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) most = fmaxf(most, fabsf(__bfloat162float(e[k])));
    mx[0] = fmaxf(mx[0], m ? 0.f : most);
    mx[1] = fmaxf(mx[1], m ? most : 0.f);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx[m] = fmaxf(mx[m], __shfl_xor_sync(0xffffffffu, mx[m], off));
    if (lane == 0) s_qmax[NW * m + warp] = mx[m];
  }
  __syncthreads();
  float sc[NT];       // scores to base 2: of the columns' map
  float qmul[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) most = fmaxf(most, s_qmax[NW * m + k]);
    int ex = 0;
    if (most > 0.f) frexpf(most, &ex);
    const int e = Cfg::MMA_BF16 || !(most > 0.f) ? 0 : min(15 - ex, 100);
    qmul[m] = ldexpf(1.f, e);
    const float f = a.softmax_scale * kDiffLog2e * exp2f(-static_cast<float>(e));
    if (PACK ? (c >> 1) == m : true) sc[PACK ? 0 : m] = f;
  }
  uint32_t q[NT][D / 16][2];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint8_t* p = qs + (8 * j + r) * Cfg::Q_PITCH;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p + 2 * diff_q_dim<KK>(k, 2 * h, c));
        if constexpr (Cfg::MMA_BF16) {
          q[j][k][h] = x;
        } else {
          const float f = qmul[PACK ? r >> 2 : j];
          q[j][k][h] = pack_f16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
        }
      }
    }

  // ---- running state ------------------------------------------------------------------
  float nm[NT][2], l_part[NT][2];  // per column: minus the reference maximum; sum
  float o[2][MT][NT][4];           // per value head
  // FP8-row / INT8-G64 values: the weights of head v carry 2^lift[v], and so does its O;
  // it falls when a scale's bits reach lift_at[v]
  int lift[2] = {kVLiftInit, kVLiftInit};
  int lim[NT][2];  // last key that a column's query sees
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      nm[j][u] = l_part[j][u] = 0.f;
      lim[j][u] = min(F - a.T + ((8 * j + 2 * c + u) % RB) / a.G, F - 1);
    }
#pragma unroll
  for (int v = 0; v < 2; ++v)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < NT; ++j) o[v][mt][j][0] = o[v][mt][j][1] = o[v][mt][j][2] = o[v][mt][j][3] = 0.f;
  uint8_t* vw = smem + Cfg::OFF_VW + warp * Cfg::VW_BYTES;
  const int ld_row = (lane & 7) + ((lane >> 4) & 1) * 8, ld_col = 16 * ((lane >> 3) & 1);  // transposed reads

  bool aborted = false;
  for (int i = 0; i < ng; ++i) {
    const int s = grp * SG + i % SG;
    uint8_t* st = smem + s * Cfg::STAGE;
    bool ok = mbar_wait_bounded(&full[s], (i / SG) & 1, a.status);  // (one answer for the warp: below)
    const int key0 = (p0 + grp + i * NG) * 64 + 16 * slab;  // this warp's first key
    const uint8_t* vst[2] = {st + Cfg::OFF_VS, st + Cfg::OFF_VS + Cfg::VS_TILE};

    if (key0 + 16 > F) {  // stale value rows become zero, codes and scales
      const int kz = max(0, F - key0);
      for (int x = lane; x < (16 - kz) * 2 * (Cfg::VCB / 16); x += 32) {
        const int v = x / ((16 - kz) * (Cfg::VCB / 16)), y = x % ((16 - kz) * (Cfg::VCB / 16));
        const int key = 16 * slab + kz + y / (Cfg::VCB / 16), col = y % (Cfg::VCB / 16) * 16;
        *reinterpret_cast<uint4*>(st + Cfg::OFF_V + v * Cfg::V_TILE + (col / Cfg::V_RB) * (64 * Cfg::V_RB) +
                                  key * Cfg::V_RB + col % Cfg::V_RB) = make_uint4(0u, 0u, 0u, 0u);
      }
      if constexpr (Cfg::VSB > 0)
        for (int x = lane; x < (16 - kz) * 2 * Cfg::VSB; x += 32) {
          const int v = x / ((16 - kz) * Cfg::VSB), y = x % ((16 - kz) * Cfg::VSB);
          st[Cfg::OFF_VS + v * Cfg::VS_TILE + (16 * slab + kz) * Cfg::VSB + y] = 0;
        }
      __syncwarp();
    }

    float S[NT][4];
    if constexpr (PACK) {  // both heads' scores of all columns; a lane's are those of its map's head
      float S2[4];
      diff_scores<KK, D>(st, st + Cfg::OFF_KS, slab, lane, q[0], S[0]);
      diff_scores<KK, D>(st + Cfg::K_TILE, st + Cfg::OFF_KS + Cfg::KS_TILE, slab, lane, q[0], S2);
#pragma unroll
      for (int e = 0; e < 4; ++e) S[0][e] = c >> 1 ? S2[e] : S[0][e];
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        diff_scores<KK, D>(st + j * Cfg::K_TILE, st + Cfg::OFF_KS + j * Cfg::KS_TILE, slab, lane, q[j], S[j]);
    }

    // ---- the stage of the page before, for the page SG further on ------------------------
    // (here the group's other warps have long left it)
    const bool refill = i > 0 && issued < ng;
    if (refill) {
      const int e = i - 1;
      ok = ok && mbar_wait_bounded(&empty[grp * SG + e % SG], (e / SG) & 1, a.status);
    }
    // Lanes measure the time of a wait each for itself: the warp stops as one, or lanes that left alone would be
    // missed at its next collective instruction (8 rows over 8 x 32768 INT8-G64 tokens: 75 us without the vote, 76 with).
    if (!__all_sync(0xffffffffu, ok)) {
      aborted = true;
      break;
    }
    if (refill) load(issued++);

    // ---- softmax over the warp's keys (lazy reference, base 2) --------------------------
    const bool first = i == 0;
    float alpha[NT][2];
    bool need = first, rescale = false;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] = fmaf(S[j][e], sc[j], nm[j][e & 1]);
      alpha[j][0] = alpha[j][1] = 1.f;
    }
    if (key0 + 15 > F - a.T) {  // not seen whole by every query
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + r + 8 * (e >> 1) > lim[j][e & 1]) S[j][e] = -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) need = need || fmaxf(fmaxf(S[j][0], S[j][1]), fmaxf(S[j][2], S[j][3])) > 8.f + TOP;
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float v = fmaxf(S[j][u], S[j][2 + u]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
          // the first page takes the exact maximum (a query's keys are a prefix:
          // one that sees none here sees none later), later ones the excess
          const float shift = first ? (v == -INFINITY ? 0.f : v - TOP) : fmaxf(v - TOP, 0.f);
          alpha[j][u] = first ? 0.f : ex2(-shift);
          rescale |= shift > 0.f;
          nm[j][u] -= shift;
          S[j][u] -= shift;
          S[j][2 + u] -= shift;
          l_part[j][u] *= alpha[j][u];
        }
      rescale = __any_sync(0xffffffffu, rescale) && !first;  // O is 0 before the first page
    }
    uint32_t pb[PARTS][NT][2];  // P^T as B operands (with a factor per key: below, by head)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[j][e] = ex2(S[j][e]);
      l_part[j][0] += S[j][0] + S[j][2];
      l_part[j][1] += S[j][1] + S[j][3];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (Cfg::MMA_BF16) {  // bf16 weights as hi + lo (about 16 significant bits)
          const __nv_bfloat162 hi = __floats2bfloat162_rn(S[j][2 * h], S[j][2 * h + 1]);
          const __nv_bfloat162 lo =
              __floats2bfloat162_rn(S[j][2 * h] - __low2float(hi), S[j][2 * h + 1] - __high2float(hi));
          pb[0][j][h] = diff_movm(*reinterpret_cast<const uint32_t*>(&hi));
          pb[PARTS - 1][j][h] = diff_movm(*reinterpret_cast<const uint32_t*>(&lo));
        } else if constexpr (!Cfg::VAL_FAC) {
          pb[0][j][h] = diff_movm(pack_f16x2(S[j][2 * h], S[j][2 * h + 1]));
        }
      }
    }

    // ---- O^T (dims x columns) += V^T P^T, head by head ----------------------------------
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float kf = 1.f;
      bool fall = false;
      if constexpr (Cfg::VAL_FAC) {  // does a scale take the lifted weights past 2^15?
        constexpr int GR = KV == KIND_INT8 ? D / 64 : 1;  // scales of a key
        uint32_t most = 0u;
#pragma unroll
        for (int g = 0; g < GR; ++g)
          most = max(most, static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(
                               vst[v] + (16 * slab + (lane & 15)) * Cfg::VSB + 2 * g)));
        // s 2^lift >= 2^7, for the binary16 bits of s (lift <= 30: subnormal scales too)
        const float sm = __half2float(__ushort_as_half(static_cast<uint16_t>(most)));
        fall = __any_sync(0xffffffffu, sm * pow2i(lift[v]) >= 128.f);
        if (fall) {
          const int k = v_lift(__reduce_max_sync(0xffffffffu, __float_as_uint(sm)), lift[v]);
          kf = pow2i(k - lift[v]);
          lift[v] = k;
        }
      }
      if (rescale || fall) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[v][mt][j][e] *= alpha[j][e & 1] * kf;
      }
      const uint8_t* vtile = st + Cfg::OFF_V + v * Cfg::V_TILE;
      if constexpr (KV == KIND_BF16) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int col = 32 * mt + ld_col;
          uint32_t A[4];
          ldsm_x4_t(smem_u32(vtile) + (col / 128) * (64 * 128) + swz<128>(16 * slab + ld_row, col % 128), A[0], A[1],
                    A[2], A[3]);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int part = 0; part < PARTS; ++part) mma16816<true>(o[v][mt][j], A, pb[part][j][0], pb[part][j][1]);
        }
      } else {
        uint32_t ps[NT][2];  // the weights of this head's (and group's) scales
#pragma unroll
        for (int q64 = 0; q64 < D / 64; ++q64) {
          __syncwarp();  // the block before has been read
          diff_values<KV, D>(vtile, vst[v], vw, q64, slab, lane);
          if constexpr (Cfg::VAL_FAC) {
            if (q64 == 0 || KV == KIND_INT8) {
              // weights of keys r (h = 0) and r + 8 with their lifted scales, rounded once
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float f = f16_at(vst[v] + (16 * slab + r + 8 * h) * Cfg::VSB + (KV == KIND_INT8 ? 2 * q64 : 0)) * pow2i(lift[v]);
#pragma unroll
                for (int j = 0; j < NT; ++j) ps[j][h] = diff_movm(pack_f16x2(S[j][2 * h] * f, S[j][2 * h + 1] * f));
              }
            }
          } else if (q64 == 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j) ps[j][0] = pb[0][j][0], ps[j][1] = pb[0][j][1];
          }
          __syncwarp();
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            uint32_t A[4];
            ldsm_x4_t(smem_u32(vw) + swz<128>(ld_row, 32 * mt + ld_col), A[0], A[1], A[2], A[3]);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816<false>(o[v][4 * q64 + mt][j], A, ps[j][0], ps[j][1]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) diff_arrive(&empty[s]);
  }

  // ---- the warps' results into one partial ----------------------------------------------
  // Sums of a column over the lanes that hold its keys; the reference maximum is
  // -inf for a query that saw no key (one that saw a key has l >= 1; NaN stays).
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float v = l_part[j][u];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (r == 0) {
        red_m[warp * 2 * RB + 8 * j + 2 * c + u] = v == 0.f ? -INFINITY : -nm[j][u];
        red_l[warp * 2 * RB + 8 * j + 2 * c + u] = v;
      }
    }
  if (aborted && lane == 0) s_flags[0] = 1;
  __syncthreads();
  if (s_flags[0]) {  // copies in flight land before the CTA leaves
    for (int k = max(0, issued - SG); k < issued; ++k)
      mbar_wait_bounded(&full[grp * SG + k % SG], (k / SG) & 1, a.status, 100000000ull);
    return;
  }
  if (tid < 2 * RB) {
    float M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, red_m[w * 2 * RB + tid]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float l = red_l[w * 2 * RB + tid];
      if (l != 0.f) Ls += l * ex2(red_m[w * 2 * RB + tid] - M);
    }
    row_M[tid] = M;
    row_L[tid] = Ls;
  }
  __syncthreads();
  float* comb = reinterpret_cast<float*>(smem);  // [NW][2 maps][RB][O_PITCH], over the ring
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int col = 8 * j + 2 * c + u;  // = map RB + row
      const float m = red_m[warp * 2 * RB + col];
      const float f = m == -INFINITY ? 0.f : ex2(m - row_M[col]);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float fv = Cfg::VAL_FAC ? f * pow2i(-lift[v]) : f;
        float* dst = comb + (warp * 2 * RB + col) * Cfg::O_PITCH + v * D + r;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          dst[16 * mt] = o[v][mt][j][u] * fv;
          dst[16 * mt + 8] = o[v][mt][j][2 + u] * fv;
        }
      }
    }
  __syncthreads();
  const int64_t slot = static_cast<int64_t>(pair) * a.ctas + cta;
  for (int idx = tid; idx < 2 * rows * (D / 2); idx += 32 * NW) {
    const int d = (idx % (D / 2)) * 4, map = idx / (D / 2) / rows, qr = idx / (D / 2) % rows;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(comb + ((w * 2 + map) * RB + qr) * Cfg::O_PITCH + d);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    *reinterpret_cast<float4*>(a.ws_o + ((slot * 2 + map) * RB + qr) * (2 * D) + d) = v;
  }
  if (tid < 2 * rows) {
    const int map = tid / rows, qr = tid % rows;
    a.ws_ml[(slot * 2 + map) * RB + qr] = make_float2(row_M[map * RB + qr], row_L[map * RB + qr]);
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

// Per-profile entries (diff_decode_*.cu).  pack: up to 4 query rows.
using DiffDecodeFn = cudaError_t (*)(const nk_pool*, int layer, const DiffDecodeArgs&, bool pack, cudaStream_t);

template <int KK, int KV>
cudaError_t diff_decode_dispatch(const nk_pool* p, int layer, const DiffDecodeArgs& a, bool pack, cudaStream_t s) {
  if (p->desc.head_dim == 128)
    return pack ? launch_diff_decode<KK, KV, 128, true>(p, layer, a, s)
                : launch_diff_decode<KK, KV, 128, false>(p, layer, a, s);
  return pack ? launch_diff_decode<KK, KV, 64, true>(p, layer, a, s)
              : launch_diff_decode<KK, KV, 64, false>(p, layer, a, s);
}

cudaError_t diff_decode_bf16(const nk_pool*, int, const DiffDecodeArgs&, bool, cudaStream_t);
cudaError_t diff_decode_int8(const nk_pool*, int, const DiffDecodeArgs&, bool, cudaStream_t);
cudaError_t diff_decode_fp8(const nk_pool*, int, const DiffDecodeArgs&, bool, cudaStream_t);
cudaError_t diff_decode_nvfp4(const nk_pool*, int, const DiffDecodeArgs&, bool, cudaStream_t);
cudaError_t diff_decode_k8v4(const nk_pool*, int, const DiffDecodeArgs&, bool, cudaStream_t);

}  // namespace nk
