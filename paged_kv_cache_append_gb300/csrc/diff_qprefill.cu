// diff_qprefill.cu -- differential attention of prompt chunks over quantized
// pages on the 5th-generation tensor cores: INT8-G64, FP8-E4M3FN-row256,
// NVFP4-G16 and K8V4 pools.
//
// The tile, the maps and the partials are those of diff_prefill.cu; the pages are
// dequantized tile by tile in shared memory with the conversions of qprefill.cu
// (exact keys and values but for INT8-G64 values, rounded once to f16):
//   warp 4      TMA producer: the map's raw K tile, and the raw V tiles of both
//               heads with their scales;
//   warps 6-13  converters: raw tiles to f16 tiles, K one page ahead of V, and the
//               per-key factors (one for the scores, one per head for the weights);
//   warp 5      MMA issuer;  warps 0-3 softmax and the partial's store.
// The two heads of a wide value have scales of their own.  NVFP4 values carry
// them, so one P serves both heads: O += P [V1 V2], N = 2 D.  FP8-row and INT8-G64
// values leave a factor per key to the weights, so each head has its own P
// (columns [0, 32) and [32, 64) of the S buffer): O_v += P_v V_v, N = D twice, the
// same tensor work.
#include "diff_prefill.cuh"
#include "qtile.cuh"

namespace nk {

template <int KK, int KV, int D>
struct DiffQCfg {
  static constexpr int NCONV = 8, THREADS = 192 + 32 * NCONV;
  static constexpr int KCB = code_row_bytes<KK>(D), VCB = code_row_bytes<KV>(D);
  static constexpr int KSB = scale_row_bytes<KK>(D), VSB = scale_row_bytes<KV>(D);
  static constexpr int K_RB = KCB < 128 ? KCB : 128, V_RB = VCB < 128 ? VCB : 128;
  static constexpr int F16 = 64 * D * 2;  // one head's f16 page tile
  static constexpr bool K_SPLIT = KK == KIND_INT8;           // exact INT8 keys: two f16 tiles
  static constexpr bool K8MMA = KK == KIND_FP8 && D >= 128;  // raw E4M3 keys to the tensor cores
  static constexpr bool VAL_FAC = KV != KIND_NVFP4;          // weights take a factor per key and head
  static constexpr int K_STAGE = K_SPLIT ? 2 * F16 : F16, V_STAGE = 2 * F16;
  static constexpr int RK_CODES = (64 * KCB + 1023) / 1024 * 1024, RV_CODES = (64 * VCB + 1023) / 1024 * 1024;
  static constexpr int RK_STAGE = (RK_CODES + 64 * KSB + 1023) / 1024 * 1024;
  static constexpr int RV_HEAD = (RV_CODES + 64 * VSB + 1023) / 1024 * 1024, RV_STAGE = 2 * RV_HEAD;
  static constexpr int NF = 4;  // factor ring: 64 K factors, 2 x 64 V factors
  static constexpr int NK = K8MMA ? 0 : D == 64 ? 4 : K_SPLIT ? 2 : 3;
  static constexpr int NV = D == 64 ? 4 : K_SPLIT ? 2 : 3;
  static constexpr int NRK = 4;
  static constexpr int NRV = D == 64 ? 4 : K_SPLIT ? 2 : 3;
  static constexpr int NKF = K8MMA ? 0 : NK;
  static constexpr int OFF_V = NK * K_STAGE;
  static constexpr int OFF_RK = OFF_V + NV * V_STAGE;
  static constexpr int OFF_RV = OFF_RK + NRK * RK_STAGE;
  static constexpr int OFF_F = OFF_RV + NRV * RV_STAGE;
  static constexpr int OFF_BAR = OFF_F + NF * 768;
  static constexpr int NBAR = 2 * NKF + 2 * NV + 2 * NRK + 2 * NRV + 2 * NF + 6;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr uint32_t COL_S = 0, COL_Q = 128, COL_O = 256;
  static constexpr uint32_t ID_S = K8MMA ? tc::idesc_e4m3(128, 64) : tc::idesc_f16(128, 64, false, false);
  static constexpr uint32_t ID_O = tc::idesc_f16(128, VAL_FAC ? D : 2 * D, false, true);
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

template <int KK, int KV, int D>
__global__ void __launch_bounds__((DiffQCfg<KK, KV, D>::THREADS), 1)
    diff_qprefill_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                         DiffPrefillArgs a) {
  using Cfg = DiffQCfg<KK, KV, D>;
  constexpr int NK = Cfg::NK, NV = Cfg::NV, NRK = Cfg::NRK, NRV = Cfg::NRV, NF = Cfg::NF, NKF = Cfg::NKF;
  constexpr int NCT = 32 * Cfg::NCONV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + Cfg::OFF_V;
  uint8_t* sRK = smem + Cfg::OFF_RK;
  uint8_t* sRV = smem + Cfg::OFF_RV;
  float* sF = reinterpret_cast<float*>(smem + Cfg::OFF_F);  // [NF][192]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* k_empty = k_full + NKF;
  uint64_t* v_full = k_empty + NKF;
  uint64_t* v_empty = v_full + NV;
  uint64_t* rk_full = v_empty + NV;
  uint64_t* rk_empty = rk_full + NRK;
  uint64_t* rv_full = rk_empty + NRK;
  uint64_t* rv_empty = rv_full + NRV;
  uint64_t* f_full = rv_empty + NRV;
  uint64_t* f_empty = f_full + NF;
  uint64_t* s_full = f_empty + NF;  // [2]
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 1;
  uint64_t* q_ready = o_done + 1;
  uint64_t* drain = q_ready + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();
  griddep_launch_dependents();
  const DiffTile w = diff_tile(a);
  const int n = w.n;
  if (n < 0) return;
  const int F = w.prefix + w.chunk;  // keys >= F are stale
  const int32_t* table = a.tables + static_cast<int64_t>(w.row) * a.L + w.p_lo;

  if (tid == 0) {
    for (int i = 0; i < NKF; ++i) {
      mbar_init(&k_full[i], Cfg::NCONV);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], Cfg::NCONV);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NRK; ++i) {
      mbar_init(&rk_full[i], 1);
      mbar_init(&rk_empty[i], Cfg::K8MMA ? 1 + Cfg::NCONV : Cfg::NCONV);  // raw FP8 keys: the MMA's commit too
    }
    for (int i = 0; i < NRV; ++i) {
      mbar_init(&rv_full[i], 1);
      mbar_init(&rv_empty[i], Cfg::NCONV);
    }
    for (int i = 0; i < NF; ++i) {
      mbar_init(&f_full[i], Cfg::NCONV);
      mbar_init(&f_empty[i], 4);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_full, 4);
    mbar_init(o_done, 1);
    mbar_init(q_ready, 4);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  if (warp == 0) {
    tc::alloc(tslot, 512);
    tc::relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;

  if (warp == 4) {
    // ------------- TMA producer: raw code and scale tiles of each page -----------
    int gnext = 0, nk = 0, nv = 0;  // copies issued (lane 0)
    for (int j = 0; j < n; ++j) {
      if ((j & 31) == 0) gnext = (j + lane < n) ? table[j + lane] : 0;
      int g = __shfl_sync(0xffffffffu, gnext, j & 31);
      int stop = 0;
      if (lane == 0) {
        if (g < 0 || g >= a.M) {  // never copy from outside the pool
          set_status(a.status, NK_STATUS_PAGE_RANGE);
          g = 0;
        }
        const int y[2] = {static_cast<int>(tile_row(g, 2 * w.pair, a.H, a.M, a.head_major)),
                          static_cast<int>(tile_row(g, 2 * w.pair + 1, a.H, a.M, a.head_major))};
        const int rk = j % NRK, rv = j % NRV;
        if (j >= NRK && !mbar_wait_bounded(&rk_empty[rk], ((j / NRK) - 1) & 1, a.status)) stop = 1;
        if (!stop) {
          uint8_t* st = sRK + rk * Cfg::RK_STAGE;
          mbar_arrive_expect_tx(&rk_full[rk], 64 * Cfg::KCB + 64 * Cfg::KSB);
#pragma unroll
          for (int c = 0; c < Cfg::KCB / Cfg::K_RB; ++c)
            tma_load_2d(st + c * 64 * Cfg::K_RB, &tmk, c * Cfg::K_RB, y[w.map], &rk_full[rk]);
          bulk_load(st + Cfg::RK_CODES, a.ks + static_cast<int64_t>(y[w.map]) * Cfg::KSB, 64 * Cfg::KSB, &rk_full[rk]);
          ++nk;
        }
        if (!stop && j >= NRV && !mbar_wait_bounded(&rv_empty[rv], ((j / NRV) - 1) & 1, a.status)) stop = 1;
        if (!stop) {
          mbar_arrive_expect_tx(&rv_full[rv], 2 * (64 * Cfg::VCB + 64 * Cfg::VSB));
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            uint8_t* st = sRV + rv * Cfg::RV_STAGE + v * Cfg::RV_HEAD;
#pragma unroll
            for (int c = 0; c < Cfg::VCB / Cfg::V_RB; ++c)
              tma_load_2d(st + c * 64 * Cfg::V_RB, &tmv, c * Cfg::V_RB, y[v], &rv_full[rv]);
            bulk_load(st + Cfg::RV_CODES, a.vs + static_cast<int64_t>(y[v]) * Cfg::VSB, 64 * Cfg::VSB, &rv_full[rv]);
          }
          ++nv;
        }
        if (stop) *s_abort = 1;
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) break;
    }
    if (lane == 0) {  // every copy lands before the CTA may leave
      for (int j = max(0, nk - NRK); j < nk; ++j) mbar_wait_bounded(&rk_full[j % NRK], (j / NRK) & 1, a.status);
      for (int j = max(0, nv - NRV); j < nv; ++j) mbar_wait_bounded(&rv_full[j % NRV], (j / NRV) & 1, a.status);
    }
  } else if (warp >= 6) {
    // ------------- converters: K(0), K(1), V(0), K(2), V(1), ... -------------------
    const int ct = tid - 192;
    bool ok = true;
    for (int i = 0; ok && i <= n; ++i) {
      if (i < n) {  // K(i) and the factors of page i
        const int rk = i % NRK, rv = i % NRV, fs = i % NF;
        ok = mbar_wait_bounded(&rk_full[rk], (i / NRK) & 1, a.status) && !*s_abort;
        if (!ok) break;
        const uint8_t* raw = sRK + rk * Cfg::RK_STAGE;
        const int kvalid = F - 64 * (w.p_lo + i);
        const int key = ct & 63;
        const bool live = key < kvalid;
        // threads 0-63: the K factor, 64-127 and 128-191: those of the two V heads;
        // the K factor is read before its raw slot can be released
        float fac = 0.f;
        if (ct < 64 && live) fac = key_factor<KK, D>(raw + Cfg::RK_CODES, key) * a.scale_log2;
        if constexpr (!Cfg::K8MMA) {
          const int ks = i % NK;
          if (i >= NK) ok = mbar_wait_bounded(&k_empty[ks], ((i / NK) - 1) & 1, a.status) && !*s_abort;
          if (!ok) break;
          convert_tile<KK, D, Cfg::K_RB, NCT, Cfg::K_SPLIT>(raw, Cfg::RK_CODES, sK + ks * Cfg::K_STAGE, ct, kvalid);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            q_arrive(&rk_empty[rk]);
            q_arrive(&k_full[ks]);
          }
        }
        ok = mbar_wait_bounded(&rv_full[rv], (i / NRV) & 1, a.status) && !*s_abort;
        if (ok && i >= NF) ok = mbar_wait_bounded(&f_empty[fs], ((i / NF) - 1) & 1, a.status) && !*s_abort;
        if (!ok) break;
        if (ct >= 64 && ct < 192 && live)
          fac = key_factor<KV, D>(sRV + rv * Cfg::RV_STAGE + ((ct >> 6) - 1) * Cfg::RV_HEAD + Cfg::RV_CODES, key);
        if (ct < 192) sF[fs * 192 + ct] = fac;
        __syncwarp();
        if (lane == 0) {
          q_arrive(&f_full[fs]);
          if constexpr (Cfg::K8MMA) q_arrive(&rk_empty[rk]);
        }
      }
      if (i >= 1) {  // V(i - 1), both heads
        const int jj = i - 1, rv = jj % NRV, vs = jj % NV;
        ok = mbar_wait_bounded(&rv_full[rv], (jj / NRV) & 1, a.status) && !*s_abort;
        if (ok && jj >= NV) ok = mbar_wait_bounded(&v_empty[vs], ((jj / NV) - 1) & 1, a.status) && !*s_abort;
        if (!ok) break;
#pragma unroll
        for (int v = 0; v < 2; ++v)
          convert_tile<KV, D, Cfg::V_RB, NCT>(sRV + rv * Cfg::RV_STAGE + v * Cfg::RV_HEAD, Cfg::RV_CODES,
                                              sV + vs * Cfg::V_STAGE + v * Cfg::F16, ct, F - 64 * (w.p_lo + jj));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          q_arrive(&rv_empty[rv]);
          q_arrive(&v_full[vs]);
        }
      }
    }
    if (!ok) *s_abort = 1;
  } else if (warp == 5) {
    // ------------------------------ MMA issuer --------------------------------
    if (lane == 0) {
      bool ok = mbar_wait_bounded(q_ready, 0, a.status);
      tc::fence_after();
      for (int j = 0; ok && j <= n; ++j) {
        if (j < n) {  // S(j) into buffer j & 1
          const int sb = j & 1;
          if constexpr (Cfg::K8MMA) {  // q_hi in columns [COL_Q, COL_Q + D / 4), q_lo in the next D / 4
            const int rk = j % NRK;
            ok = mbar_wait_bounded(&rk_full[rk], (j / NRK) & 1, a.status) && !*s_abort;
            if (!ok) break;
            tc::fence_after();
            const uint64_t kd = tc::smem_desc(smem_u32(sRK + rk * Cfg::RK_STAGE), 16, 1024);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                tc::mma_ts_f8(tmem + Cfg::COL_S + 64 * sb, tmem + Cfg::COL_Q + part * (D / 4) + kk * 8,
                              kd + static_cast<uint64_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), Cfg::ID_S,
                              part > 0 || kk > 0);
            tc::commit(&s_full[sb]);
            tc::commit(&rk_empty[rk]);
          } else {
            const int ks = j % NK;
            ok = mbar_wait_bounded(&k_full[ks], (j / NK) & 1, a.status) && !*s_abort;
            if (!ok) break;
            tc::fence_after();
#pragma unroll
            for (int part = 0; part < (Cfg::K_SPLIT ? 2 : 1); ++part) {  // INT8-G64: Q k1^T - Q k2'^T
              const uint64_t kd = tc::smem_desc(smem_u32(sK + ks * Cfg::K_STAGE + part * Cfg::F16), 16, 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_ts(tmem + Cfg::COL_S + 64 * sb, tmem + Cfg::COL_Q + kk * 8,
                           kd + static_cast<uint64_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4),
                           part > 0 ? tc::idesc_negate_b(Cfg::ID_S) : Cfg::ID_S, part > 0 || kk > 0);
            }
            tc::commit(&s_full[sb]);
            tc::commit(&k_empty[ks]);
          }
        }
        if (j >= 1) {  // O += P(j - 1) V(j - 1)
          const int jj = j - 1, vs = jj % NV;
          ok = mbar_wait_bounded(&v_full[vs], (jj / NV) & 1, a.status) && !*s_abort;
          if (ok) ok = mbar_wait_bounded(p_full, jj & 1, a.status) && !*s_abort;
          if (!ok) break;
          tc::fence_after();
#pragma unroll
          for (int v = 0; v < (Cfg::VAL_FAC ? 2 : 1); ++v) {
            const uint64_t vd = tc::smem_desc(smem_u32(sV + vs * Cfg::V_STAGE + v * Cfg::F16), 8192, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_ts(tmem + Cfg::COL_O + v * D, tmem + Cfg::COL_S + 64 * (jj & 1) + 32 * v + kk * 8,
                         vd + static_cast<uint64_t>((kk * 2048) >> 4), Cfg::ID_O, (jj > 0 || kk > 0));
          }
          tc::commit(o_done);
          tc::commit(&v_empty[vs]);
        }
      }
      if (!ok) *s_abort = 1;
      tc::commit(drain);
    }
  } else {
    // ------------------------------ softmax warps -----------------------------
    const int m = tid;
    const int tl = m / a.G, g = m % a.G, token = w.t0 + tl;
    const bool valid = tl < a.TQ && token < w.chunk;
    const int pos = w.prefix + token;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    float rs = 1.f;  // 2^-e of this query row
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((static_cast<int64_t>(w.b) * a.Tc + token) * a.Hq + 2 * (w.pair * a.G + g) + w.map) * D);
      float mx = 0.f;
      if (valid)
        for (int u = 0; u < D / 8; ++u) {
          const uint4 x = src[u];
          const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&x);
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(__bfloat162float(e[k])));
        }
      int ex = 0;
      if (mx > 0.f) frexpf(mx, &ex);
      // f16 q: max|q| 2^e in [2^14, 2^15); E4M3 q: max|q| 2^e in [2^7, 2^8)
      const int e = mx > 0.f ? min((Cfg::K8MMA ? 8 : 15) - ex, 100) : 0;
      const float qf = ldexpf(1.f, e);
      rs = ldexpf(1.f, -e);
      if constexpr (Cfg::K8MMA) {  // q' = hi + lo in E4M3, as in qprefill.cu
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 64) {
          uint32_t hv[16], lv[16];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = valid ? src[c0 / 8 + u] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            uint32_t hp[4], lp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&xw[k]);
              const float x0 = __low2float(v) * qf, x1 = __high2float(v) * qf;
              const uint16_t h2 = f32x2_to_e4m3x2(x0, x1);
              const uint32_t h32 = e4m3x2_to_f16x2(h2);
              const __half2 hb = *reinterpret_cast<const __half2*>(&h32);
              hp[k] = h2;
              lp[k] = f32x2_to_e4m3x2(x0 - __low2float(hb), x1 - __high2float(hb));
            }
            hv[2 * u] = hp[0] | (hp[1] << 16);
            hv[2 * u + 1] = hp[2] | (hp[3] << 16);
            lv[2 * u] = lp[0] | (lp[1] << 16);
            lv[2 * u + 1] = lp[2] | (lp[3] << 16);
          }
          tc::st16(tmem + lane_base + Cfg::COL_Q + c0 / 4, hv);
          tc::st16(tmem + lane_base + Cfg::COL_Q + D / 4 + c0 / 4, lv);
        }
      } else {
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          uint32_t qv[32];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = valid ? src[c0 / 4 + u] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&xw[k]);
              qv[4 * u + k] = pack_f16x2(__low2float(v) * qf, __high2float(v) * qf);
            }
          }
          tc::st32(tmem + lane_base + Cfg::COL_Q + c0, qv);
        }
      }
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) q_arrive(q_ready);
    }
    float m_used = -INFINITY, l = 0.f;
    // FP8-row V: the weights, l and O carry 2^k_run (v_lift), one lift for both heads
    int k_run = KV == KIND_FP8 ? kVLiftInit : 0;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int sb = j & 1, fs = j % NF;
      ok = mbar_wait_bounded(&s_full[sb], (j / 2) & 1, a.status) && !*s_abort;
      if (ok) ok = mbar_wait_bounded(&f_full[fs], (j / NF) & 1, a.status) && !*s_abort;
      if (!ok) break;
      tc::fence_after();
      uint32_t sv[64];
      {
        uint32_t v0[32], v1[32];
        tc::ld32(tmem + lane_base + Cfg::COL_S + 64 * sb, v0);
        tc::ld32(tmem + lane_base + Cfg::COL_S + 64 * sb + 32, v1);
        tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) sv[c] = v0[c], sv[32 + c] = v1[c];
      }
      const float* ksc = sF + fs * 192;
      const float* vsc = ksc + 64;
      const int kmax = valid ? pos - 64 * (w.p_lo + j) : -1;
      constexpr bool KEY_FAC = KK != KIND_NVFP4;  // NVFP4 keys carry their scales
      const bool nomask = __all_sync(0xffffffffu, kmax >= 63);
      float rmax = -INFINITY;
#pragma unroll
      for (int c4 = 0; c4 < 16; ++c4) {
        float kf[4] = {a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2};
        if constexpr (KEY_FAC) {
          const float4 k0 = *reinterpret_cast<const float4*>(ksc + 4 * c4);
          kf[0] = k0.x, kf[1] = k0.y, kf[2] = k0.z, kf[3] = k0.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = 4 * c4 + u;
          float x = __uint_as_float(sv[c]) * kf[u];
          if (!nomask) x = c <= kmax ? x : -INFINITY;
          sv[c] = __float_as_uint(x);
          rmax = fmaxf(rmax, x);
        }
      }
      rmax = rmax == -INFINITY ? -INFINITY : rmax * rs;
      int knew = k_run;
      if constexpr (KV == KIND_FP8) {
        const float4 s4 = *reinterpret_cast<const float4*>(vsc + 4 * lane);  // both heads' 128 scales
        knew = v_lift(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fmaxf(s4.x, s4.y), fmaxf(s4.z, s4.w)))), k_run);
      }
      float factor = 1.f;
      const float mnew = fmaxf(m_used, rmax);
      bool resc = false;
      if (mnew != -INFINITY && (m_used == -INFINITY || mnew > m_used + kLazyThr || knew != k_run)) {
        factor = m_used == -INFINITY ? 0.f : ex2((m_used - mnew) + static_cast<float>(knew - k_run));
        m_used = mnew;
        resc = true;
      }
      k_run = knew;
      const float mu = m_used == -INFINITY ? 0.f : m_used - static_cast<float>(k_run);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        const float p = ex2(fmaf(__uint_as_float(sv[c]), rs, -mu));
        sum += p;
        sv[c] = __float_as_uint(p);
      }
      l = l * factor + sum;
      if (j >= 1) {
        ok = mbar_wait_bounded(o_done, (j - 1) & 1, a.status) && !*s_abort;
        if (!ok) break;
        tc::fence_after();
      }
      if (__any_sync(0xffffffffu, resc && j >= 1)) {
        const float f = (resc && j >= 1) ? factor : 1.f;
#pragma unroll 1
        for (int c0 = 0; c0 < 2 * D; c0 += 32) {
          uint32_t ov[32];
          tc::ld32(tmem + lane_base + Cfg::COL_O + c0, ov);
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * f);
          tc::st32(tmem + lane_base + Cfg::COL_O + c0, ov);
        }
      }
#pragma unroll
      for (int v = 0; v < (Cfg::VAL_FAC ? 2 : 1); ++v) {  // weights of head v, over the S that was read
        uint32_t pk[32];
#pragma unroll
        for (int c4 = 0; c4 < 16; ++c4) {
          float p[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) p[u] = __uint_as_float(sv[4 * c4 + u]);
          if constexpr (Cfg::VAL_FAC) {
            const float4 s = *reinterpret_cast<const float4*>(vsc + 64 * v + 4 * c4);
            p[0] *= s.x, p[1] *= s.y, p[2] *= s.z, p[3] *= s.w;
          }
          pk[2 * c4] = pack_f16x2(p[0], p[1]);
          pk[2 * c4 + 1] = pack_f16x2(p[2], p[3]);
        }
        tc::st32(tmem + lane_base + Cfg::COL_S + 64 * sb + 32 * v, pk);
      }
      __syncwarp();
      if (lane == 0) q_arrive(&f_empty[fs]);  // this warp is done with the page's factors
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) q_arrive(p_full);
    }
    if (ok && n > 0) ok = mbar_wait_bounded(o_done, (n - 1) & 1, a.status) && !*s_abort;
    tc::fence_after();
    if (ok) {
      const float m_eff = m_used == -INFINITY ? -INFINITY : m_used - static_cast<float>(k_run);
      diff_store<D>(a, w, tmem + lane_base + Cfg::COL_O, n > 0, valid, m, m_eff, l);
    }
  }

  // ---- teardown: every issued MMA has completed before TMEM is freed ---------
  if (tid == 0) mbar_wait_bounded(drain, 0, a.status, 200000000ull);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(tmem, 512);
}

template <int KK, int KV, int D>
static cudaError_t launch_diff_qprefill(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid,
                                        cudaStream_t s) {
  using Cfg = DiffQCfg<KK, KV, D>;
  auto k = diff_qprefill_kernel<KK, KV, D>;
  static std::atomic<uint64_t> granted{0};
  const cudaError_t e = grant_smem(granted, k, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, grid, dim3(Cfg::THREADS), Cfg::SMEM, s, p->tmap[layer * 2 + 0], p->tmap[layer * 2 + 1], a);
}

template <int KK, int KV>
static cudaError_t diff_qprefill_d(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid, cudaStream_t s) {
  return p->desc.head_dim == 64 ? launch_diff_qprefill<KK, KV, 64>(p, layer, a, grid, s)
                                : launch_diff_qprefill<KK, KV, 128>(p, layer, a, grid, s);
}

cudaError_t diff_prefill_quant(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid, cudaStream_t s) {
  switch (p->desc.profile) {
    case NK_INT8_G64: return diff_qprefill_d<KIND_INT8, KIND_INT8>(p, layer, a, grid, s);
    case NK_FP8_E4M3_ROW: return diff_qprefill_d<KIND_FP8, KIND_FP8>(p, layer, a, grid, s);
    case NK_NVFP4_G16: return diff_qprefill_d<KIND_NVFP4, KIND_NVFP4>(p, layer, a, grid, s);
    default: return diff_qprefill_d<KIND_FP8, KIND_NVFP4>(p, layer, a, grid, s);
  }
}

}  // namespace nk
