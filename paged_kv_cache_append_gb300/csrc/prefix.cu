// prefix.cu -- the prefix pass of the shared-prefix attention (shared.cu): the
// R = B T G query rows of a batch that read one KV head, at most 256, against
// the pages that all of them share, on the 5th-generation tensor cores.
//
// A CTA takes one KV head and one range of the shared pages and leaves one
// partial (m, l, O) for its query rows; the ranges cover all SMs or those that
// share_split leaves to the pass.  A pipeline is 128 query rows,
//   S = Q K^T   tcgen05.mma M 128 x N 64 x K D, the K page in shared memory, S
//               in one of two TMEM buffers
//   O += P V    tcgen05.mma M 128 x N D x K 64, P over its S (TMEM)
// with a softmax warpgroup of its own.  One issuing thread is what bounds the
// prefill kernels (prefill.cu, qprefill.cu): N = 64 products and the waits
// around them keep it busy.  Here two threads issue.
//   head_dim 64, 128: two pipelines, an issuer each, all rows in one CTA.
//     R > 128   the pipelines hold the two halves of the rows and read every
//               page, which is loaded and dequantized once for both;
//     R <= 128  they hold the same rows and take the even and the odd pages;
//               their partials are merged before they leave the CTA.
//   head_dim 256: O takes half of the tensor memory, so one pipeline of 128
//     rows a CTA, one thread issuing the scores and one the values.
//
// Operands and their exactness are those of qprefill.cu (dequantization in
// shared memory, FP8 keys raw from head_dim 128 on, INT8 keys as two tiles, per-key
// factors, the lift of FP8-row values) and of prefill.cu for BF16, except that
// BF16 softmax weights enter as two bf16 terms (hi + lo, 16 bits): the tensor
// time of the second product hides behind HBM there.  No mask: every row sees
// every page whole.
//
// The softmax reads each score once on most pages: it computes the weights
// against the reference maximum that it has, and only where their sum passes
// 2^8 (so that none is above it) does it take the page's maximum and compute
// them again (the scores are intact until P is stored).  32 columns (16 where
// registers are short) are worked on while the next ones load, and two scores
// share an instruction where fp32 has packed forms.  Each of the two steps
// stands in the code once: a second copy of them on the rare path cost 6%.
//
// Warps: 4 softmax and output warps a pipeline, then the TMA producer, two MMA
// issuers and the converters (quantized pools).  All waits are bounded.
#include "internal.h"
#include "packed.cuh"
#include "qtile.cuh"
#include "shared.cuh"
#include "tcgen05.cuh"

namespace nk {

__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct PrefixArgs {
  const __nv_bfloat16* q;  // [B][T][Hq][D]
  const int32_t* tables;
  const int32_t* table_rows;
  const uint8_t* ks;  // scale planes of the layer
  const uint8_t* vs;
  float2* ml;  // [H][tiles][nsplit][128]
  float* o;    // [H][tiles][nsplit][128][D]
  int* status;
  float scale_log2;
  int rows;  // R
  int tiles;  // of 128 rows
  int nsplit, Hq, H, G, L, M, C, head_major;
  SharedPrefix sh;
};

template <int KK, int KV, int D>
struct PrefixCfg {
  static constexpr bool RAW = KK != KIND_BF16;  // quantized: raw rings and converters
  using Q = QCfg<RAW ? KK : KIND_FP8, RAW ? KV : KIND_FP8, D>;  // (their geometry)
  static constexpr int NP = D == 256 ? 1 : 2;  // pipelines
  // converter warps: 8 where tiles of keys and values are both converted or
  // are large, else 4; threads have 128 registers (96 with 19 warps)
  static constexpr int NCONV = !RAW ? 0 : D == 256 || (D == 128 && KK != KIND_FP8) ? 8 : 4;
  static constexpr int W_TMA = 4 * NP, W_MMA = W_TMA + 1, W_CONV = W_MMA + 2;
  static constexpr int THREADS = 32 * (W_CONV + NCONV);
  static constexpr int CH = THREADS > 512 ? 16 : 32;  // score columns in registers while the next ones load
  static constexpr int F16 = 64 * D * 2;
  // Rings: those of qprefill.cu; smaller at head_dim 128 where 64 KB of Q lie
  // next to them.
  static constexpr bool QW = D == 128;
  static constexpr int NK = !RAW ? (D == 256 ? 3 : QW ? 4 : 6) : Q::NK == 0 ? 0 : !QW ? Q::NK : KK == KIND_INT8 ? 2 : 3;
  static constexpr int NV = !RAW ? NK : Q::NK == 0 ? Q::NV : !QW ? Q::NV : 3;
  static constexpr int NRK = !RAW ? 0 : QW && KK == KIND_INT8 ? 2 : Q::NRK;
  static constexpr int NRV = !RAW ? 0 : QW && KK == KIND_INT8 ? 3 : Q::NRV;
  static constexpr int NF = RAW ? Q::NF : 0;
  static constexpr int NKF = NK;
  static constexpr int K_STAGE = RAW ? Q::K_STAGE : F16;
  static constexpr int OFF_V = NK * K_STAGE;
  static constexpr int OFF_RK = OFF_V + NV * F16;
  static constexpr int OFF_RV = OFF_RK + NRK * (RAW ? Q::RK_STAGE : 0);
  static constexpr int OFF_Q = OFF_RV + NRV * (RAW ? Q::RV_STAGE : 0);
  // Q of a pipeline: blocks of 128 rows x 128 bytes (64 bf16 / f16 dims; the
  // hi, then the lo E4M3 terms of 128 dims), 128-byte swizzle; at head_dim 256
  // in tensor memory instead, which S and O leave 128 columns of
  static constexpr bool Q_TMEM = D == 256;
  static constexpr int Q_BYTES = Q_TMEM ? 0 : 128 * D * 2;
  static constexpr int OFF_F = OFF_Q + NP * Q_BYTES;
  // [256] floats: the rows' query scales; then [128] float2: pipeline 1's (m, l)
  static constexpr int OFF_ML = OFF_F + NF * 512;
  static constexpr int OFF_BAR = OFF_ML + 1024;
  static constexpr int NBAR = 2 * NKF + 2 * NV + 2 * NRK + 2 * NRV + 2 * NF + 12;
  // at least half of the SM's shared memory: one CTA per SM owns all 512 TMEM columns
  static constexpr int USED = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr int SMEM = USED > 116 * 1024 ? USED : 116 * 1024;
  // output rows on their way to global memory, over the rings and Q
  static constexpr int PITCH = D + 4;
  static_assert(128 * NP * PITCH * 4 <= OFF_F, "staged output rows");
  static constexpr uint32_t COL_S = 0, COL_Q = 128, COL_O = 256;  // S + 128 w + 64 (buffer), O + 128 w
  static constexpr bool K8MMA = RAW && Q::K8MMA;
  static constexpr bool K_SPLIT = RAW && Q::K_SPLIT;
  static constexpr uint32_t ID_S = !RAW    ? tc::idesc_bf16(128, 64, false, false)
                                   : K8MMA ? tc::idesc_e4m3(128, 64)
                                           : tc::idesc_f16(128, 64, false, false);
  static constexpr uint32_t ID_O = RAW ? tc::idesc_f16(128, D, false, true) : tc::idesc_bf16(128, D, false, true);
  static_assert(!Q_TMEM || NV * F16 >= 128 * 2 * D, "queries on their way to tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// Query rows [first, first + n) of the head whose first query row is at `q`, by
// warp `pw` of the PW that share them, in the form the MMAs read: row m of the
// 128-row blocks at `sq` (blocks of head_dim 256 are rows of 2 D bytes on their
// way to tensor memory), and 2^-e of its power-of-two scale to s_rs[m].  A warp
// reads whole rows, 16 bytes a lane.  Rows past the last are left as they are:
// whatever is in them stays in their own scores and outputs, which nobody
// reads.  (The softmax threads alone, a row each, took 5.3 us for 64 rows of
// FP8 pages at head_dim 256, most of it converting.)
constexpr int kQBatch = 4;  // loads of a lane in flight

template <int D>
__device__ __forceinline__ void load_queries(const __nv_bfloat16* q, int first, int n, int G, int Hq, int g0, int PW,
                                             int lane, uint4 (&x)[kQBatch]) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes a row, rows a load
#pragma unroll
  for (int k = 0; k < kQBatch; ++k) {
    const int m = (g0 + k * PW) * RPI + lane / LPR, flat = first + m;
    x[k] = m < n ? *reinterpret_cast<const uint4*>(q + (static_cast<int64_t>(flat / G) * Hq + flat % G) * D +
                                                   8 * (lane % LPR))
                 : make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int KK, int KV, int D>
__device__ __forceinline__ void prefix_queries(const __nv_bfloat16* q, int first, int n, int G, int Hq, uint8_t* sq,
                                               float* s_rs, int pw, int PW, int lane, uint4 (&x)[kQBatch]) {
  using Cfg = PrefixCfg<KK, KV, D>;
  constexpr int LPR = D / 8, RPI = 32 / LPR, BATCH = kQBatch;
  const int sub = lane / LPR, c = lane % LPR;
#pragma unroll 1
  for (int g0 = pw; g0 * RPI < n; g0 += BATCH * PW) {
    if (g0 != pw) load_queries<D>(q, first, n, G, Hq, g0, PW, lane, x);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int m = (g0 + k * PW) * RPI + sub;
      if ((g0 + k * PW) * RPI >= n) break;  // the same for the warp
      const bool live = m < n;
      // 16-byte chunk j of the row
      auto at = [&](int j) {
        if constexpr (Cfg::Q_TMEM) return sq + m * (2 * D) + ((j ^ m) & (2 * D / 16 - 1)) * 16;
        else return sq + (m >> 7) * Cfg::Q_BYTES + (j >> 3) * 16384 + swz<128>(m & 127, (j & 7) * 16);
      };
      if constexpr (!Cfg::RAW) {
        if (live) *reinterpret_cast<uint4*>(at(c)) = x[k];
      } else {
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        float v[8], mx = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[2 * u] = __uint_as_float(w[u] << 16);
          v[2 * u + 1] = __uint_as_float(w[u] & 0xFFFF0000u);
          mx = fmaxf(mx, fmaxf(fabsf(v[2 * u]), fabsf(v[2 * u + 1])));
        }
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        // f16 q: max|q| 2^e in [2^14, 2^15); E4M3 q: in [2^7, 2^8), as hi + lo
        // (see qprefill.cu); max|q| = f 2^ex, f in [1/2, 1)
        const int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 126;
        const int e = mx > 0.f ? min((Cfg::K8MMA ? 8 : 15) - ex, 100) : 0;
        const float qf = pow2i(e);
        if (live && c == 0) s_rs[m] = pow2i(-e);
        if constexpr (Cfg::K8MMA) {
          uint32_t hv[2], lv[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t hp[2], lp[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float x0 = v[4 * u + 2 * p] * qf, x1 = v[4 * u + 2 * p + 1] * qf;
              const uint16_t h2 = f32x2_to_e4m3x2(x0, x1);
              const uint32_t hb32 = e4m3x2_to_f16x2(h2);
              const __half2 hb = *reinterpret_cast<const __half2*>(&hb32);
              hp[p] = h2;
              lp[p] = f32x2_to_e4m3x2(x0 - __low2float(hb), x1 - __high2float(hb));
            }
            hv[u] = hp[0] | (hp[1] << 16);
            lv[u] = lp[0] | (lp[1] << 16);
          }
          if (live) {
            *reinterpret_cast<uint2*>(at(c >> 1) + 8 * (c & 1)) = make_uint2(hv[0], hv[1]);
            *reinterpret_cast<uint2*>(at(D / 16 + (c >> 1)) + 8 * (c & 1)) = make_uint2(lv[0], lv[1]);
          }
        } else {
          uint32_t h[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) h[u] = pack_f16x2(v[2 * u] * qf, v[2 * u + 1] * qf);
          if (live) *reinterpret_cast<uint4*>(at(c)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
  }
}

template <int KK, int KV, int D>
__global__ void __launch_bounds__((PrefixCfg<KK, KV, D>::THREADS), 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                  const __grid_constant__ PrefixArgs a) {
  using Cfg = PrefixCfg<KK, KV, D>;
  using QC = typename Cfg::Q;
  constexpr int NK = Cfg::NK, NV = Cfg::NV, NRK = Cfg::NRK, NRV = Cfg::NRV, NF = Cfg::NF;
  constexpr int NCONV = Cfg::NCONV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + Cfg::OFF_V;
  uint8_t* sRK = smem + Cfg::OFF_RK;
  uint8_t* sRV = smem + Cfg::OFF_RV;
  uint8_t* sQ = smem + Cfg::OFF_Q;
  float* sF = reinterpret_cast<float*>(smem + Cfg::OFF_F);  // [NF][128]: 64 K factors, 64 V factors
  float2* sML = reinterpret_cast<float2*>(smem + Cfg::OFF_ML);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* k_full = bars;               // K tile ready for the MMA
  uint64_t* k_empty = k_full + Cfg::NKF;  // read by its last S
  uint64_t* v_full = k_empty + Cfg::NKF;
  uint64_t* v_empty = v_full + NV;
  uint64_t* rk_full = v_empty + NV;  // raw tiles landed / consumed
  uint64_t* rk_empty = rk_full + NRK;
  uint64_t* rv_full = rk_empty + NRK;
  uint64_t* rv_empty = rv_full + NRV;
  uint64_t* f_full = rv_empty + NRV;  // per-key factors of a page
  uint64_t* f_empty = f_full + NF;
  uint64_t* s_full = f_empty + NF;  // [2][2] scores of pipeline w in buffer i & 1
  uint64_t* p_full = s_full + 4;    // [2] its weights stored
  uint64_t* o_done = p_full + 2;    // [2] its P V accumulated
  uint64_t* s_empty = o_done + 2;   // [2] one pipeline: P V from the buffer done
  uint64_t* q_ready = s_empty + 2;
  uint64_t* drain = q_ready + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NP = Cfg::NP;
  const int split = blockIdx.x, h = blockIdx.y % a.H, tile = blockIdx.y / a.H;  // tile: one pipeline a CTA
  const bool two = NP == 2 && a.rows > 128;  // the pipelines hold different rows
  const int readers = two ? 2 : 1;  // pipelines that read a page
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();

  // the first of the queries that this warp prepares (below), on their way with the plan's reads
  const int q_first = NP == 1 ? tile * 128 : 0, q_rows = min(a.rows - q_first, 128 * NP);
  const int q_warp = warp < Cfg::W_TMA ? warp : warp - Cfg::W_CONV + Cfg::W_TMA;
  constexpr int QWARPS = Cfg::W_TMA + NCONV;
  const __nv_bfloat16* q_head = a.q + static_cast<int64_t>(h) * a.G * D;
  uint4 q_x[kQBatch];
  const bool q_mine = warp < Cfg::W_TMA || warp >= Cfg::W_CONV;
  if (q_mine) load_queries<D>(q_head, q_first, q_rows, a.G, a.Hq, q_warp, QWARPS, lane, q_x);

  // ---- this CTA's pages [p_lo, p_lo + n) -----------------------------------------
  const int pages = *a.sh.pages;
  int own;
  const int row = prefix_row(a.sh, a.table_rows, pages, a.L, a.C, own);
  const int all = row < 0 ? 0 : pages;
  const int nsplit = share_split(a.sh.shape, all, own).nsplit;
  const int per = (all + nsplit - 1) / nsplit;
  const int p_lo = min(split * per, all);
  const int n = min(p_lo + per, all) - p_lo;
  if (n == 0) return;  // the merge reads no partial of this range
  const int32_t* table = a.tables + static_cast<int64_t>(max(row, 0)) * a.L + p_lo;
  if (tid == 0) {
    for (int i = 0; i < Cfg::NKF; ++i) {
      mbar_init(&k_full[i], Cfg::RAW ? NCONV : 1);
      mbar_init(&k_empty[i], readers);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], Cfg::RAW ? NCONV : 1);
      mbar_init(&v_empty[i], readers);
    }
    for (int i = 0; i < NRK; ++i) {
      mbar_init(&rk_full[i], 1);
      mbar_init(&rk_empty[i], Cfg::K8MMA ? readers + NCONV : NCONV);
    }
    for (int i = 0; i < NRV; ++i) {
      mbar_init(&rv_full[i], 1);
      mbar_init(&rv_empty[i], NCONV);
    }
    for (int i = 0; i < NF; ++i) {
      mbar_init(&f_full[i], NCONV);
      mbar_init(&f_empty[i], 4 * readers);
    }
    for (int w = 0; w < NP; ++w) {
      mbar_init(&s_full[2 * w], 1);
      mbar_init(&s_full[2 * w + 1], 1);
      mbar_init(&p_full[w], 4);
      mbar_init(&o_done[w], 1);
    }
    mbar_init(&s_empty[0], 1);
    mbar_init(&s_empty[1], 1);
    mbar_init(q_ready, 4 * NP);
    mbar_init(drain, 2);
    *s_abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  if (warp == 0) {
    tc::alloc(tslot, 512);
    tc::relinquish();
  }
  // page i of pipeline w, and how many it takes
  const int step = NP == 1 || two ? 1 : 2;
  auto page_of = [&](int w, int i) { return step == 1 ? i : 2 * i + w; };
  auto count_of = [&](int w) { return step == 1 ? n : (n - w + 1) / 2; };
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;
  // partial slot of query row r: [h][tile][split][row]
  auto slot = [&](int r) { return ((static_cast<int64_t>(h) * a.tiles + r / 128) * a.nsplit + split) * 128 + r % 128; };

  // the queries, by the softmax and the converter warps
  if (q_mine) {
    prefix_queries<KK, KV, D>(q_head, q_first, q_rows, a.G, a.Hq, Cfg::Q_TMEM ? sV : sQ, reinterpret_cast<float*>(sML),
                              q_warp, QWARPS, lane, q_x);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    asm volatile("bar.sync 2, %0;" ::"n"(32 * QWARPS) : "memory");
  }

  int k_sent = 0, v_sent = 0;  // tiles whose copies were issued (by the producer's lane 0)
  if (warp == Cfg::W_TMA) {
    // ------------------------------ TMA producer ---------------------------------
    int gnext = 0;
    for (int j = 0; j < n; ++j) {
      if ((j & 31) == 0) gnext = (j + lane < n) ? table[j + lane] : 0;
      int g = __shfl_sync(0xffffffffu, gnext, j & 31);
      int stop = 0;
      if (lane == 0) {
        if (g < 0 || g >= a.M) {  // never copy from outside the pool
          set_status(a.status, NK_STATUS_PAGE_RANGE);
          g = 0;
        }
        const int y = static_cast<int>(tile_row(g, h, a.H, a.M, a.head_major));
        if constexpr (Cfg::RAW) {
          const int rk = j % NRK, rv = j % NRV;
          if (j >= NRK && !mbar_wait_bounded(&rk_empty[rk], ((j / NRK) - 1) & 1, a.status)) stop = 1;
          if (!stop) {
            uint8_t* st = sRK + rk * QC::RK_STAGE;
            mbar_arrive_expect_tx(&rk_full[rk], 64 * QC::KCB + 64 * QC::KSB);
#pragma unroll
            for (int c = 0; c < QC::KCB / QC::K_RB; ++c)
              tma_load_2d(st + c * 64 * QC::K_RB, &tmk, c * QC::K_RB, y, &rk_full[rk]);
            bulk_load(st + QC::RK_CODES, a.ks + static_cast<int64_t>(y) * QC::KSB, 64 * QC::KSB, &rk_full[rk]);
            ++k_sent;
          }
          if (!stop && j >= NRV && !mbar_wait_bounded(&rv_empty[rv], ((j / NRV) - 1) & 1, a.status)) stop = 1;
          if (!stop) {
            uint8_t* st = sRV + rv * QC::RV_STAGE;
            mbar_arrive_expect_tx(&rv_full[rv], 64 * QC::VCB + 64 * QC::VSB);
#pragma unroll
            for (int c = 0; c < QC::VCB / QC::V_RB; ++c)
              tma_load_2d(st + c * 64 * QC::V_RB, &tmv, c * QC::V_RB, y, &rv_full[rv]);
            bulk_load(st + QC::RV_CODES, a.vs + static_cast<int64_t>(y) * QC::VSB, 64 * QC::VSB, &rv_full[rv]);
            ++v_sent;
          }
        } else {
          const int ks = j % NK, vs = j % NV;
          if (j >= NK && !mbar_wait_bounded(&k_empty[ks], ((j / NK) - 1) & 1, a.status)) stop = 1;
          if (!stop) {
            mbar_arrive_expect_tx(&k_full[ks], Cfg::F16);
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_2d(sK + ks * Cfg::F16 + kb * 8192, &tmk, kb * 128, y, &k_full[ks]);
            ++k_sent;
          }
          // the V ring holds the queries on their way to tensor memory at first
          if (Cfg::Q_TMEM && !stop && j == 0 && !mbar_wait_bounded(q_ready, 0, a.status)) stop = 1;
          if (!stop && j >= NV && !mbar_wait_bounded(&v_empty[vs], ((j / NV) - 1) & 1, a.status)) stop = 1;
          if (!stop) {
            mbar_arrive_expect_tx(&v_full[vs], Cfg::F16);
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_2d(sV + vs * Cfg::F16 + kb * 8192, &tmv, kb * 128, y, &v_full[vs]);
            ++v_sent;
          }
        }
        if (stop) *s_abort = 1;
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) break;
    }
  } else if (warp >= Cfg::W_CONV) {
    // ------------- converters: K(0), K(1), V(0), K(2), V(1), ... -------------------
    if constexpr (Cfg::RAW) {
      const int ct = tid - 32 * Cfg::W_CONV;
      bool ok = true;
      for (int i = 0; ok && i <= n; ++i) {
        if (i < n) {  // K(i) and the factors of page i
          const int rk = i % NRK, rv = i % NRV, fs = i % NF;
          ok = mbar_wait_bounded(&rk_full[rk], (i / NRK) & 1, a.status) && !*s_abort;
          if (!ok) break;
          const uint8_t* raw = sRK + rk * QC::RK_STAGE;
          const float kf = ct < 64 ? key_factor<KK, D>(raw + QC::RK_CODES, ct) * a.scale_log2 : 0.f;
          if constexpr (!Cfg::K8MMA) {
            const int ks = i % NK;
            if (i >= NK) ok = mbar_wait_bounded(&k_empty[ks], ((i / NK) - 1) & 1, a.status) && !*s_abort;
            if (!ok) break;
            convert_tile<KK, D, QC::K_RB, 32 * (NCONV > 0 ? NCONV : 8), Cfg::K_SPLIT>(raw, QC::RK_CODES, sK + ks * Cfg::K_STAGE, ct, 64);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
              arrive(&rk_empty[rk]);
              arrive(&k_full[ks]);
            }
          }
          ok = mbar_wait_bounded(&rv_full[rv], (i / NRV) & 1, a.status) && !*s_abort;
          if (ok && i >= NF) ok = mbar_wait_bounded(&f_empty[fs], ((i / NF) - 1) & 1, a.status) && !*s_abort;
          if (!ok) break;
          if (ct < 64) {
            float* fac = sF + fs * 128;
            fac[ct] = kf;
            fac[64 + ct] = key_factor<KV, D>(sRV + rv * QC::RV_STAGE + QC::RV_CODES, ct);
          }
          __syncwarp();
          if (lane == 0) {
            arrive(&f_full[fs]);
            if constexpr (Cfg::K8MMA) arrive(&rk_empty[rk]);  // with the commits of the page's S
          }
        }
        if (i >= 1) {  // V(i - 1)
          const int jj = i - 1, rv = jj % NRV, vs = jj % NV;
          ok = mbar_wait_bounded(&rv_full[rv], (jj / NRV) & 1, a.status) && !*s_abort;
          if (Cfg::Q_TMEM && ok && jj == 0) ok = mbar_wait_bounded(q_ready, 0, a.status);  // (queries in the V ring)
          if (ok && jj >= NV) ok = mbar_wait_bounded(&v_empty[vs], ((jj / NV) - 1) & 1, a.status) && !*s_abort;
          if (!ok) break;
          convert_tile<KV, D, QC::V_RB, 32 * (NCONV > 0 ? NCONV : 8)>(sRV + rv * QC::RV_STAGE, QC::RV_CODES, sV + vs * Cfg::F16, ct, 64);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            arrive(&rv_empty[rv]);
            arrive(&v_full[vs]);
          }
        }
      }
      if (!ok) *s_abort = 1;
    }
  } else if (warp >= Cfg::W_MMA) {
    // ----------------------------- MMA issuers --------------------------------
    // Two pipelines: issuer w does all of pipeline w,
    //   S(0), S(1), P(0) V, S(2), P(1) V, ...
    // and the MMAs of one thread run in issue order, so S(i + 1) cannot
    // overwrite the P(i - 1) in its buffer early.  One pipeline: issuer 0 does
    // the scores, after P(i - 2) V has completed, and issuer 1 the values.
    if (lane == 0) {
      const int me = warp - Cfg::W_MMA, w = NP == 2 ? me : 0, count = count_of(w);
      const uint32_t tS = tmem + Cfg::COL_S + 128 * w, tO = tmem + Cfg::COL_O + 128 * w;
      const uint64_t qd = Cfg::Q_TMEM ? 0 : tc::smem_desc(smem_u32(sQ + (two ? w * Cfg::Q_BYTES : 0)), 16, 1024);
      constexpr int RK = Cfg::K8MMA ? NRK : NK, KS = Cfg::K8MMA ? QC::RK_STAGE : Cfg::K_STAGE;
      const uint64_t kd0 = tc::smem_desc(smem_u32(Cfg::K8MMA ? sRK : sK), 16, 1024);
      const uint64_t vd0 = tc::smem_desc(smem_u32(sV), 8192, 1024);
      uint64_t* kfull = Cfg::K8MMA ? rk_full : k_full;
      uint64_t* kempty = Cfg::K8MMA ? rk_empty : k_empty;
      int ks = step == 1 ? 0 : w, kph = 0, vs = ks, vph = 0;  // ring slots and parities of the next K and V page
      auto scores = [&](int i) {
        if (!mbar_wait_bounded(&kfull[ks], kph, a.status)) return false;
        tc::fence_after();
        const uint32_t d = tS + 64 * (i & 1);
        const uint64_t kd = kd0 + static_cast<uint64_t>((ks * KS) >> 4);
        // 32 bytes of K per product: 16 f16 or 32 E4M3 dims, 8 TMEM columns of Q
        auto product = [&](int part, int kk, uint64_t k, uint32_t id) {
          const uint32_t acc = part > 0 || kk > 0;
          if constexpr (Cfg::Q_TMEM) {
            const uint32_t q = tmem + Cfg::COL_Q + (Cfg::K8MMA ? part * (D / 4) : 0) + kk * 8;
            if constexpr (Cfg::K8MMA) tc::mma_ts_f8(d, q, k, id, acc);
            else tc::mma_ts(d, q, k, id, acc);
          } else {
            const int at = Cfg::K8MMA ? part * 16384 + kk * 32 : (kk >> 2) * 16384 + (kk & 3) * 32;
            const uint64_t q = qd + static_cast<uint64_t>(at >> 4);
            if constexpr (Cfg::K8MMA) tc::mma_ss_f8(d, q, k, id, acc);
            else tc::mma_ss(d, q, k, id, acc);
          }
        };
        constexpr int KPARTS = Cfg::K8MMA || Cfg::K_SPLIT ? 2 : 1;
#pragma unroll
        for (int part = 0; part < KPARTS; ++part)
#pragma unroll
          for (int kk = 0; kk < (Cfg::K8MMA ? D / 32 : D / 16); ++kk)
            product(part, kk,
                    kd + static_cast<uint64_t>(((Cfg::K_SPLIT ? part * Cfg::F16 : 0) + (kk >> 2) * 8192 + (kk & 3) * 32) >> 4),
                    Cfg::K_SPLIT && part > 0 ? tc::idesc_negate_b(Cfg::ID_S) : Cfg::ID_S);
        tc::commit(&s_full[2 * w + (i & 1)]);
        tc::commit(&kempty[ks]);
        if ((ks += step) >= RK) ks -= RK, kph ^= 1;
        return true;
      };
      auto values = [&](int i) {
        bool ok = mbar_wait_bounded(&v_full[vs], vph, a.status);
        if (ok) ok = mbar_wait_bounded(&p_full[w], i & 1, a.status) && !*s_abort;
        if (!ok) return false;
        tc::fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>((vs * Cfg::F16) >> 4);
#pragma unroll
        for (int part = 0; part < (Cfg::RAW ? 1 : 2); ++part)  // BF16: the hi and the lo weights
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_ts(tO, tS + 64 * (i & 1) + 32 * part + kk * 8, vd + static_cast<uint64_t>((kk * 2048) >> 4),
                       Cfg::ID_O, i > 0 || part > 0 || kk > 0);
        tc::commit(&o_done[w]);
        tc::commit(&v_empty[vs]);
        if constexpr (NP == 1) tc::commit(&s_empty[i & 1]);
        if ((vs += step) >= NV) vs -= NV, vph ^= 1;
        return true;
      };
      bool ok = true;
      if (NP == 2 || me == 0) {
        ok = mbar_wait_bounded(q_ready, 0, a.status);
        tc::fence_after();
      }
      if constexpr (NP == 2) {
        if (ok && count > 0) ok = scores(0);
        for (int i = 0; ok && i < count; ++i) {
          if (i + 1 < count) ok = scores(i + 1);
          if (ok) ok = values(i);
        }
      } else if (me == 0) {
        for (int i = 0; ok && i < count; ++i) {
          if (i >= 2) ok = mbar_wait_bounded(&s_empty[i & 1], ((i >> 1) - 1) & 1, a.status) && !*s_abort;
          if (ok) ok = scores(i);
        }
      } else {
        for (int i = 0; ok && i < count; ++i) ok = values(i);
      }
      if (!ok) *s_abort = 1;
      tc::commit(drain);  // arrives once every MMA issued above has completed
    }
  } else {
    // --------------------- softmax warps of pipeline w ---------------------------
    const int w = warp >> 2, m = tid & 127;
    const int flat = 128 * (NP == 1 ? tile : two ? w : 0) + m;
    const bool row_valid = flat < a.rows;
    const bool live = __any_sync(0xffffffffu, row_valid);  // warps without rows only hand on
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lane_base + Cfg::COL_O + 128 * w;
    float rs = 1.f;
    if constexpr (Cfg::RAW) rs = reinterpret_cast<const float*>(sML)[NP == 1 ? m : flat];
    if constexpr (Cfg::Q_TMEM) {  // the lane's row: 2 D bytes, a 32-bit column each
#pragma unroll 1
      for (int j0 = 0; j0 < 2 * D / 16; j0 += 8) {
        uint32_t v[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 y = *reinterpret_cast<const uint4*>(sV + m * (2 * D) + (((j0 + u) ^ m) & (2 * D / 16 - 1)) * 16);
          v[4 * u] = y.x, v[4 * u + 1] = y.y, v[4 * u + 2] = y.z, v[4 * u + 3] = y.w;
        }
        tc::st32(tmem + lane_base + Cfg::COL_Q + 4 * j0, v);
      }
      tc::wait_st();
      tc::fence_before();
    }
    __syncwarp();
    if (lane == 0) arrive(q_ready);

    constexpr bool KEY_FAC = Cfg::RAW && KK != KIND_NVFP4;  // per-key score factors
    constexpr bool VAL_FAC = Cfg::RAW && KV != KIND_NVFP4;  // per-key weight factors
    constexpr int CH = Cfg::CH;
    constexpr int PK = Cfg::RAW ? 32 : 64;                  // columns of P
    // exponents are z rs - m; without key factors z is the raw score and the
    // softmax scale is in rs, with its sign in the direction of the maximum
    const bool up = a.scale_log2 >= 0.f;
    if constexpr (!KEY_FAC) rs *= a.scale_log2;
    const float zmul = KEY_FAC ? rs : fabsf(rs);
    float m_used = -INFINITY, l = 0.f;
    int k_run = KV == KIND_FP8 ? kVLiftInit : 0;  // FP8-row V: the weights, l and O carry 2^k_run (v_lift)
    bool ok = true;
    const int count = count_of(w);
    for (int i = 0; i < count; ++i) {
      const int j = page_of(w, i), fs = Cfg::RAW ? j % (NF > 0 ? NF : 1) : 0;
      const uint32_t tS = tmem + lane_base + Cfg::COL_S + 128 * w + 64 * (i & 1);
      ok = mbar_wait_bounded(&s_full[2 * w + (i & 1)], (i >> 1) & 1, a.status) && !*s_abort;
      if constexpr (Cfg::RAW)
        if (ok) ok = mbar_wait_bounded(&f_full[fs], (j / NF) & 1, a.status) && !*s_abort;
      if (!ok) break;
      tc::fence_after();
      if (live) {
        const float* ksc = sF + fs * 128;
        const float* vsc = ksc + 64;
        // The page's scores times their factors, CH columns at a time, to
        // body(c0, z[CH / 2 pairs]); the next ones load while the body runs.
        auto each = [&](auto body) {
          uint32_t v[2][CH];
          tc::ldn(tS, v[0]);
#pragma unroll
          for (int k = 0; k < 64 / CH; ++k) {
            uint32_t(&u)[CH] = v[k & 1];
            tc::wait_ldn(u);
            if (k + 1 < 64 / CH) tc::ldn(tS + CH * (k + 1), v[(k + 1) & 1]);
            F2 z[CH / 2];
#pragma unroll
            for (int c = 0; c < CH / 2; ++c) z[c] = pack2(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1]));
            if constexpr (KEY_FAC) {
#pragma unroll
              for (int c = 0; c < CH / 4; ++c) {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(ksc + CH * k + 4 * c);
                z[2 * c] = mul2(z[2 * c], f.x);
                z[2 * c + 1] = mul2(z[2 * c + 1], f.y);
              }
            }
            body(CH * k, z);
          }
        };
        // the larger of m and the pairs, of -z for a negative uniform scale
        auto max_of = [&](float m, const F2 (&z)[CH / 2]) {
          float t[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < CH / 2; ++c) {
            float x, y;
            unpack2(z[c], x, y);
            if (KEY_FAC || up) t[c & 3] = max3(t[c & 3], x, y);
            else t[c & 3] = max3(t[c & 3], -x, -y);
          }
          return max3(fmaxf(t[0], t[1]), t[2], t[3]);
        };
        int knew = k_run;
        if constexpr (KV == KIND_FP8) {
          const float2 s2 = *reinterpret_cast<const float2*>(vsc + 2 * lane);
          knew = v_lift(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(s2.x, s2.y))), k_run);
        }
        // the page's largest score, of the rows that ask for it
        auto top = [&] {
          float mx = -INFINITY;
          each([&](int, const F2 (&z)[CH / 2]) { mx = max_of(mx, z); });
          return mx == -INFINITY ? -INFINITY : mx * zmul;
        };
        float mnew = m_used;
        uint32_t pk[PK];
        float sum = 0.f;
        // p = 2^(z rs - mnew + knew)
        auto weights = [&]() {
          const float mu = (mnew == -INFINITY ? 0.f : mnew) - static_cast<float>(knew);
          const F2 rs2 = pack2(rs, rs), nmu2 = pack2(-mu, -mu);
          F2 s0 = 0ull, s1 = 0ull;
          each([&](int c0, const F2 (&z)[CH / 2]) {
#pragma unroll
            for (int c = 0; c < CH / 2; c += 2) {
              float p0, p1, p2, p3;
              unpack2(fma2(z[c], rs2, nmu2), p0, p1);
              unpack2(fma2(z[c + 1], rs2, nmu2), p2, p3);
              p0 = ex2(p0), p1 = ex2(p1), p2 = ex2(p2), p3 = ex2(p3);
              F2 pa = pack2(p0, p1), pb = pack2(p2, p3);
              s0 = add2(s0, pa);
              s1 = add2(s1, pb);
              if constexpr (VAL_FAC) {
                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(vsc + c0 + 2 * c);
                unpack2(mul2(pa, f.x), p0, p1);
                unpack2(mul2(pb, f.y), p2, p3);
              }
              const int k = c0 / 2 + c;
              if constexpr (Cfg::RAW) {
                pk[k] = pack_f16x2(p0, p1);
                pk[k + 1] = pack_f16x2(p2, p3);
              } else {
                pk[k] = pack_bf16x2(p0, p1);
                pk[k + 1] = pack_bf16x2(p2, p3);
                pk[32 + k] = pack_bf16x2(p0 - __uint_as_float(pk[k] << 16), p1 - __uint_as_float(pk[k] & 0xFFFF0000u));
                pk[33 + k] = pack_bf16x2(p2 - __uint_as_float(pk[k + 1] << 16),
                                         p3 - __uint_as_float(pk[k + 1] & 0xFFFF0000u));
              }
            }
          });
          float a0, a1, b0, b1;
          unpack2(s0, a0, a1);
          unpack2(s1, b0, b1);
          sum = (a0 + a1) + (b0 + b1);
        };
        // the first page takes its maximum first, a page with too large a weight afterwards, and then again
        bool ask = m_used == -INFINITY;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          if (__any_sync(0xffffffffu, ask)) {
            const float mx = top();
            if (ask) mnew = mx;
          } else if (pass > 0) {
            break;
          }
          weights();
          ask = sum > ex2(kLazyThr + static_cast<float>(knew));
        }
        const bool resc = mnew != m_used || knew != k_run;
        const float factor = m_used == -INFINITY ? 0.f
                             : resc              ? ex2((m_used - mnew) + static_cast<float>(knew - k_run))
                                                 : 1.f;
        l = l * factor + sum;
        m_used = mnew;
        k_run = knew;
        __syncwarp();
        if constexpr (Cfg::RAW)
          if (lane == 0) arrive(&f_empty[fs]);
        // PV(i - 1) is consumed on every page: a parity wait is sound one phase at a time
        if (i >= 1) {
          ok = mbar_wait_bounded(&o_done[w], (i - 1) & 1, a.status) && !*s_abort;
          if (!ok) break;
          tc::fence_after();
          if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t ov[32];
              tc::ld32(tO + c0, ov);
              tc::wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * factor);
              tc::st32(tO + c0, ov);
            }
          }
        }
#pragma unroll
        for (int c0 = 0; c0 < PK; c0 += 32) tc::st32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(&pk[c0]));
        tc::wait_st();
      } else {  // a warp without rows hands on, in step: it must not arrive for P(i) before P(i - 1) is used
        if constexpr (Cfg::RAW)
          if (lane == 0) arrive(&f_empty[fs]);
        if (i >= 1) ok = mbar_wait_bounded(&o_done[w], (i - 1) & 1, a.status) && !*s_abort;
        if (!ok) break;
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) arrive(&p_full[w]);
    }

    // ---- the CTA's partial: rows by way of shared memory, whole lines out ---------
    ok = mbar_wait_bounded(drain, 0, a.status) && ok && !*s_abort;  // every MMA done: the rings are free
    tc::fence_after();
    const float m_eff = m_used == -INFINITY ? -INFINITY : m_used - static_cast<float>(k_run);
    float* stage = reinterpret_cast<float*>(smem);
    float* mine = stage + (NP == 1 ? m : flat) * Cfg::PITCH;
    // pipeline w's output times f, plus f1 times what the row holds already
    auto put = [&](float f, bool add, float f1) {
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t ov[32];
        tc::ld32(tO + c0, ov);
        tc::wait_ld();
        if (!row_valid) continue;
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          float4* at = reinterpret_cast<float4*>(mine + c0 + c);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (add) {
            v = *at;
            v.x *= f1, v.y *= f1, v.z *= f1, v.w *= f1;
          }
          v.x = fmaf(__uint_as_float(ov[c]), f, v.x);
          v.y = fmaf(__uint_as_float(ov[c + 1]), f, v.y);
          v.z = fmaf(__uint_as_float(ov[c + 2]), f, v.z);
          v.w = fmaf(__uint_as_float(ov[c + 3]), f, v.w);
          *at = v;
        }
      }
    };
    float M = m_eff, L = l;
    if (NP == 1 || two) {
      if (ok && live) put(1.f, false, 0.f);
    } else {
      if (w == 1) {
        sML[m] = make_float2(m_eff, l);
        if (ok && live && count > 0) put(1.f, false, 0.f);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(128 * NP) : "memory");
      if (w == 0 && count_of(1) > 0) {
        const float2 o = sML[m];
        M = fmaxf(m_eff, o.x);
        const float f0 = m_eff == -INFINITY ? 0.f : ex2(m_eff - M), f1 = o.x == -INFINITY ? 0.f : ex2(o.x - M);
        L = l * f0 + o.y * f1;
        if (ok && live) put(f0, true, f1);
      } else if (w == 0) {
        if (ok && live) put(1.f, false, 0.f);
      }
    }
    if (!ok) *s_abort = 1;
    else if (row_valid && (NP == 1 || two || w == 0)) a.ml[slot(flat)] = make_float2(M, L);
  }

  // ---- rows out, and the teardown: every issued MMA has completed ----------------
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (!*s_abort) {
    const int r0 = NP == 1 ? tile * 128 : 0, rows = NP == 1 ? min(a.rows - r0, 128) : a.rows;
    const float* stage = reinterpret_cast<const float*>(smem);
#pragma unroll 4
    for (int idx = tid; idx < rows * (D / 4); idx += Cfg::THREADS) {
      const int r = idx / (D / 4), c = (idx % (D / 4)) * 4;
      *reinterpret_cast<float4*>(a.o + slot(r0 + r) * D + c) =
          *reinterpret_cast<const float4*>(stage + r * Cfg::PITCH + c);
    }
  } else if (warp == Cfg::W_TMA && lane == 0) {  // after an abort, the copies still in flight land before the CTA exits
    constexpr int RK = Cfg::RAW ? NRK : NK, RV = Cfg::RAW ? NRV : NV;
    uint64_t *kf = Cfg::RAW ? rk_full : k_full, *vf = Cfg::RAW ? rv_full : v_full;
    for (int j = max(0, k_sent - RK); j < k_sent; ++j) mbar_wait_bounded(&kf[j % RK], (j / RK) & 1, a.status, 100000000ull);
    for (int j = max(0, v_sent - RV); j < v_sent; ++j) mbar_wait_bounded(&vf[j % RV], (j / RV) & 1, a.status, 100000000ull);
  }
  if (warp == 0) tc::dealloc(tmem, 512);
}

template <int KK, int KV, int D>
static cudaError_t launch_prefix(const nk_pool* p, int layer, const PrefixArgs& a, cudaStream_t s) {
  using Cfg = PrefixCfg<KK, KV, D>;
  auto k = prefix_kernel<KK, KV, D>;
  static std::atomic<uint64_t> granted{0};
  cudaError_t e = grant_smem(granted, k, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  // In clusters of two, which lie on one TPC (two SMs), so that the SMs left to
  // the own pages (share_split) are whole TPCs: where the two kernels shared
  // TPCs, the own-pages CTAs took up to 160 us instead of 99.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.nsplit, a.H * (Cfg::NP == 1 ? a.tiles : 1));
  cfg.blockDim = dim3(Cfg::THREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.y = cfg.gridDim.y % 2 ? 1 : 2;
  at[1].val.clusterDim.x = cfg.gridDim.y % 2 && cfg.gridDim.x % 2 == 0 ? 2 : 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, p->tmap[layer * 2 + 0], p->tmap[layer * 2 + 1], a);
}

template <int KK, int KV>
static cudaError_t launch_prefix_d(int D, const nk_pool* p, int layer, const PrefixArgs& a, cudaStream_t s) {
  return D == 256   ? launch_prefix<KK, KV, 256>(p, layer, a, s)
         : D == 128 ? launch_prefix<KK, KV, 128>(p, layer, a, s)
                    : launch_prefix<KK, KV, 64>(p, layer, a, s);
}

// At most 256 query rows per KV head.
cudaError_t prefix_pass(const nk_pool* p, int layer, const void* q, const int32_t* tables, const int32_t* table_rows,
                        int Hq, float scale_log2, const PrefixParts& parts, const SharedPrefix& sh, cudaStream_t s) {
  const int np = p->n_planes;
  PrefixArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tables = tables;
  a.table_rows = table_rows;
  a.ks = np == 4 ? static_cast<const uint8_t*>(p->ptrs[layer * np + 2]) : nullptr;
  a.vs = np == 4 ? static_cast<const uint8_t*>(p->ptrs[layer * np + 3]) : nullptr;
  a.ml = parts.ml;
  a.o = parts.o;
  a.status = p->status;
  a.scale_log2 = scale_log2;
  a.tiles = parts.tiles;
  a.nsplit = parts.nsplit;
  a.Hq = Hq;
  a.H = p->desc.num_kv_heads;
  a.G = Hq / a.H;
  a.rows = sh.B * sh.T * a.G;
  a.L = p->L;
  a.M = p->M;
  a.C = p->desc.max_concurrency;
  a.head_major = p->desc.order == NK_HEAD_MAJOR;
  a.sh = sh;
  const int D = p->desc.head_dim;
  switch (p->desc.profile) {
    case NK_BF16: return launch_prefix_d<KIND_BF16, KIND_BF16>(D, p, layer, a, s);
    case NK_INT8_G64: return launch_prefix_d<KIND_INT8, KIND_INT8>(D, p, layer, a, s);
    case NK_FP8_E4M3_ROW: return launch_prefix_d<KIND_FP8, KIND_FP8>(D, p, layer, a, s);
    case NK_NVFP4_G16: return launch_prefix_d<KIND_NVFP4, KIND_NVFP4>(D, p, layer, a, s);
    default: return launch_prefix_d<KIND_FP8, KIND_NVFP4>(D, p, layer, a, s);
  }
}

}  // namespace nk
