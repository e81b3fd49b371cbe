// diff_prefill.cu -- differential attention of prompt chunks over BF16 pages on
// the 5th-generation tensor cores, the join of all profiles' partials, and the
// host side (diff_qprefill.cu has the quantized pages).
//
// As in prefill.cu, keys advance one page at a time:
//   S = Q_m K_m^T   M 128 x N 64 x K D, A = Q in TMEM, B = the map's K tile;
//   P = exp2(S scale - m) in bf16 over the first half of the S buffer;
//   O += P V        M 128 x N 2 D x K 64, B = the two heads' V tiles side by
//                   side (their 64-dim blocks lie behind one another).
// A page then takes 2 D + 4 D flops per (query row, key), the least there is
// for two maps over one wide value, against 8 D with two plain calls per map.
// TMEM columns: S [0, 128), Q [128, 128 + D / 2), O [256, 256 + 2 D).
//
// Warps 0-3 softmax and the partial's store, 4 TMA producer, 5 MMA issuer.  All
// waits are bounded; a wait that runs out ends the CTA without results once the
// copies in flight have landed.
#include "diff_prefill.cuh"

namespace nk {

template <int D>
struct DiffPrefillCfg {
  static constexpr int THREADS = 192;
  static constexpr int K_BYTES = 64 * D * 2, V_BYTES = 2 * K_BYTES;
  static constexpr int NK = D == 128 ? 4 : 8, NV = D == 128 ? 4 : 8;
  static constexpr int OFF_V = NK * K_BYTES;
  static constexpr int OFF_BAR = OFF_V + NV * V_BYTES;
  static constexpr int NBAR = 2 * NK + 2 * NV + 6;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr uint32_t COL_S = 0, COL_Q = 128, COL_O = 256;
  static constexpr uint32_t ID_S = tc::idesc_bf16(128, 64, false, false);
  static constexpr uint32_t ID_O = tc::idesc_bf16(128, 2 * D, false, true);
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

__device__ __forceinline__ void dp_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D>
__global__ void __launch_bounds__(192, 1)
    diff_prefill_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        DiffPrefillArgs a) {
  using Cfg = DiffPrefillCfg<D>;
  constexpr int NK = Cfg::NK, NV = Cfg::NV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + Cfg::OFF_V;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* k_empty = k_full + NK;
  uint64_t* v_full = k_empty + NK;
  uint64_t* v_empty = v_full + NV;
  uint64_t* s_full = v_empty + NV;  // [2]
  uint64_t* p_full = s_full + 2;
  uint64_t* o_done = p_full + 1;
  uint64_t* q_ready = o_done + 1;
  uint64_t* drain = q_ready + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();
  const DiffTile w = diff_tile(a);
  const int n = w.n;
  if (n < 0) return;
  const int32_t* table = a.tables + static_cast<int64_t>(w.row) * a.L + w.p_lo;

  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
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
    // ------------------------------ TMA producer ------------------------------
    int gnext = 0, nk = 0, nv = 0;  // copies of K and V issued (lane 0)
    for (int j = 0; j < n; ++j) {
      if ((j & 31) == 0) gnext = (j + lane < n) ? table[j + lane] : 0;
      int g = __shfl_sync(0xffffffffu, gnext, j & 31);
      int stop = 0;
      if (lane == 0) {
        if (g < 0 || g >= a.M) {  // never copy from outside the pool
          set_status(a.status, NK_STATUS_PAGE_RANGE);
          g = 0;
        }
        const int ks = j % NK, vs = j % NV;
        const int y[2] = {static_cast<int>(tile_row(g, 2 * w.pair, a.H, a.M, a.head_major)),
                          static_cast<int>(tile_row(g, 2 * w.pair + 1, a.H, a.M, a.head_major))};
        if (j >= NK && !mbar_wait_bounded(&k_empty[ks], ((j / NK) - 1) & 1, a.status)) stop = 1;
        if (!stop) {
          mbar_arrive_expect_tx(&k_full[ks], Cfg::K_BYTES);
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_2d(sK + ks * Cfg::K_BYTES + kb * 8192, &tmk, kb * 128, y[w.map], &k_full[ks]);
          ++nk;
        }
        if (!stop && j >= NV && !mbar_wait_bounded(&v_empty[vs], ((j / NV) - 1) & 1, a.status)) stop = 1;
        if (!stop) {
          mbar_arrive_expect_tx(&v_full[vs], Cfg::V_BYTES);
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int kb = 0; kb < D / 64; ++kb)
              tma_load_2d(sV + vs * Cfg::V_BYTES + (v * (D / 64) + kb) * 8192, &tmv, kb * 128, y[v], &v_full[vs]);
          ++nv;
        }
        if (stop) *s_abort = 1;
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) break;
    }
    if (lane == 0) {  // every copy lands before the CTA may leave
      for (int j = max(0, nk - NK); j < nk; ++j) mbar_wait_bounded(&k_full[j % NK], (j / NK) & 1, a.status);
      for (int j = max(0, nv - NV); j < nv; ++j) mbar_wait_bounded(&v_full[j % NV], (j / NV) & 1, a.status);
    }
  } else if (warp == 5) {
    // ------------------------------ MMA issuer --------------------------------
    if (lane == 0) {
      bool ok = mbar_wait_bounded(q_ready, 0, a.status);
      tc::fence_after();
      for (int j = 0; ok && j <= n; ++j) {
        if (j < n) {  // S(j) into buffer j & 1
          const int ks = j % NK, sb = j & 1;
          ok = mbar_wait_bounded(&k_full[ks], (j / NK) & 1, a.status);
          if (!ok) break;
          tc::fence_after();
          const uint64_t kd = tc::smem_desc(smem_u32(sK + ks * Cfg::K_BYTES), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_ts(tmem + Cfg::COL_S + 64 * sb, tmem + Cfg::COL_Q + kk * 8,
                       kd + static_cast<uint64_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), Cfg::ID_S, kk > 0);
          tc::commit(&s_full[sb]);
          tc::commit(&k_empty[ks]);
        }
        if (j >= 1) {  // O += P(j - 1) V(j - 1)
          const int jj = j - 1, vs = jj % NV;
          ok = mbar_wait_bounded(&v_full[vs], (jj / NV) & 1, a.status);
          if (ok) ok = mbar_wait_bounded(p_full, jj & 1, a.status);
          if (!ok) break;
          tc::fence_after();
          const uint64_t vd = tc::smem_desc(smem_u32(sV + vs * Cfg::V_BYTES), 8192, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_ts(tmem + Cfg::COL_O, tmem + Cfg::COL_S + 64 * (jj & 1) + kk * 8,
                       vd + static_cast<uint64_t>((kk * 2048) >> 4), Cfg::ID_O, (jj > 0 || kk > 0));
          tc::commit(o_done);
          tc::commit(&v_empty[vs]);
        }
      }
      if (!ok) *s_abort = 1;
      tc::commit(drain);  // arrives once every MMA issued above has completed
    }
  } else {
    // ------------------------------ softmax warps -----------------------------
    const int m = tid;  // query row = TMEM lane
    const int tl = m / a.G, g = m % a.G, token = w.t0 + tl;
    const bool valid = tl < a.TQ && token < w.chunk;
    const int pos = w.prefix + token;  // keys <= pos are visible
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((static_cast<int64_t>(w.b) * a.Tc + token) * a.Hq + 2 * (w.pair * a.G + g) + w.map) * D);
#pragma unroll 1
      for (int c0 = 0; c0 < D / 2; c0 += 32) {
        uint32_t qv[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 x = valid ? src[c0 / 4 + u] : make_uint4(0u, 0u, 0u, 0u);
          qv[4 * u] = x.x, qv[4 * u + 1] = x.y, qv[4 * u + 2] = x.z, qv[4 * u + 3] = x.w;
        }
        tc::st32(tmem + lane_base + Cfg::COL_Q + c0, qv);
      }
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) dp_arrive(q_ready);
    }
    float m_used = -INFINITY, l = 0.f;
    const bool pos_scale = a.scale_log2 >= 0.f;
    const float fill = pos_scale ? -INFINITY : INFINITY;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int sb = j & 1;
      ok = mbar_wait_bounded(&s_full[sb], (j / 2) & 1, a.status) && !*s_abort;
      if (!ok) break;
      tc::fence_after();
      uint32_t v0[32], v1[32];
      tc::ld32(tmem + lane_base + Cfg::COL_S + 64 * sb, v0);
      tc::ld32(tmem + lane_base + Cfg::COL_S + 64 * sb + 32, v1);
      tc::wait_ld();
      // the largest raw score (the smallest for a negative scale); the causal
      // mask only where the page reaches past a row's last key
      const int kmax = valid ? pos - 64 * (w.p_lo + j) : -1;
      float rext = fill;
      if (!__all_sync(0xffffffffu, kmax >= 63)) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (c > kmax) v0[c] = __float_as_uint(fill);
          if (32 + c > kmax) v1[c] = __float_as_uint(fill);
        }
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const float x = __uint_as_float(v0[c]), y = __uint_as_float(v1[c]);
        rext = pos_scale ? fmaxf(rext, fmaxf(x, y)) : fminf(rext, fminf(x, y));
      }
      const float rmax = rext == fill ? -INFINITY : rext * a.scale_log2;
      float factor = 1.f;
      const float mnew = fmaxf(m_used, rmax);
      bool resc = false;
      if (mnew != -INFINITY && (m_used == -INFINITY || mnew > m_used + 8.f)) {
        factor = m_used == -INFINITY ? 0.f : ex2(m_used - mnew);
        m_used = mnew;
        resc = true;
      }
      const float mu = m_used == -INFINITY ? 0.f : m_used;
      uint32_t pk[32];
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float pa = ex2(fmaf(__uint_as_float(v0[2 * c]), a.scale_log2, -mu));
        const float pb = ex2(fmaf(__uint_as_float(v0[2 * c + 1]), a.scale_log2, -mu));
        const float pc = ex2(fmaf(__uint_as_float(v1[2 * c]), a.scale_log2, -mu));
        const float pd = ex2(fmaf(__uint_as_float(v1[2 * c + 1]), a.scale_log2, -mu));
        sum += (pa + pb) + (pc + pd);
        pk[c] = pack_bf16x2(pa, pb);
        pk[16 + c] = pack_bf16x2(pc, pd);
      }
      l = l * factor + sum;
      // PV(j - 1) is complete before a rescale (consumed every page: a parity
      // wait is sound one phase at a time)
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
      tc::st32(tmem + lane_base + Cfg::COL_S + 64 * sb, pk);
      tc::wait_st();
      // values past the row's frontier may be any bits; 0 * NaN would reach O
      const int kstale = w.prefix + w.chunk - 64 * (w.p_lo + j);
      if (kstale < 64) {
        const int vs = j % NV;
        ok = mbar_wait_bounded(&v_full[vs], (j / NV) & 1, a.status);
        if (!ok) break;
        uint8_t* vt = sV + vs * Cfg::V_BYTES;
        constexpr int CH = 2 * (D / 64) * 8;  // 16-byte chunks of a key
        for (int i = tid; i < (64 - kstale) * CH; i += 128) {
          const int rr = kstale + i / CH, rem = i % CH;
          *reinterpret_cast<uint4*>(vt + (rem >> 3) * 8192 + rr * 128 + (rem & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) dp_arrive(p_full);
    }
    if (ok && n > 0) ok = mbar_wait_bounded(o_done, (n - 1) & 1, a.status) && !*s_abort;
    tc::fence_after();
    if (ok) diff_store<D>(a, w, tmem + lane_base + Cfg::COL_O, n > 0, valid, m, m_used, l);
  }

  // ---- teardown: every issued MMA has completed before TMEM is freed ---------
  if (tid == 0) mbar_wait_bounded(drain, 0, a.status, 200000000ull);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::dealloc(tmem, 512);
}

template <int D>
static cudaError_t launch_diff_prefill(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid,
                                       cudaStream_t s) {
  using Cfg = DiffPrefillCfg<D>;
  auto k = diff_prefill_kernel<D>;
  static std::atomic<uint64_t> granted{0};
  const cudaError_t e = grant_smem(granted, k, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, grid, dim3(Cfg::THREADS), Cfg::SMEM, s, p->tmap[layer * 2 + 0], p->tmap[layer * 2 + 1], a);
}

cudaError_t diff_prefill_bf16(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid, cudaStream_t s) {
  return p->desc.head_dim == 64 ? launch_diff_prefill<64>(p, layer, a, grid, s)
                                : launch_diff_prefill<128>(p, layer, a, grid, s);
}

// ---- the join: one warp per (token, head), 2 D / 32 values a lane --------------
// Reads every partial once and writes bf16: bound by HBM / L2.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) diff_prefill_join_kernel(DiffPrefillArgs a) {
  constexpr int V = 2 * D / 128;  // float4 per lane
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, heads = a.Hq / 2, b = blockIdx.y;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int token = static_cast<int>(at / heads), head = static_cast<int>(at % heads);
  const int row = a.table_rows[b], prefix = a.prefix_len[b], chunk = a.chunk_len[b];
  if (token >= a.Tc || token >= chunk || chunk > a.Tc || row < 0 || row >= a.C || prefix < 0 ||
      static_cast<int64_t>(prefix) + chunk > static_cast<int64_t>(a.L) * 64)
    return;
  const int qt = token / a.TQ, m = (token - qt * a.TQ) * a.G + head % a.G;
  const int64_t part0 =
      ((static_cast<int64_t>(b) * (a.H / 2) + head / a.G) * a.tiles + qt) * a.nsplit * 2;
  float o[V][4], L[2], M[2];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const int64_t bt = static_cast<int64_t>(b) * a.Tc + token;
  const float lambda = a.o.lambda[bt * a.o.lambda_stride + head];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    // lane s holds range s's (m, l); nsplit <= 32
    const float2 ml = lane < a.nsplit ? a.ws_ml[(part0 + 2 * lane + map) * 128 + m] : make_float2(-INFINITY, 0.f);
    M[map] = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M[map] = fmaxf(M[map], __shfl_xor_sync(0xffffffffu, M[map], off));
    const float e = ml.y == 0.f ? 0.f : ex2(ml.x - M[map]);
    L[map] = e * ml.y;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L[map] += __shfl_xor_sync(0xffffffffu, L[map], off);
    const float f = L[map] == 0.f ? 0.f : (map ? -lambda : 1.f) * e / L[map];
    for (int s = 0; s < a.nsplit; ++s) {
      const float wgt = __shfl_sync(0xffffffffu, f, s);
      if (__shfl_sync(0xffffffffu, ml.y, s) == 0.f) continue;  // an empty range has no O
      const float* src = a.ws_o + ((part0 + 2 * s + map) * 128 + m) * (2 * D) + 4 * lane;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(src + 128 * i));
        o[i][0] = fmaf(wgt, v.x, o[i][0]);
        o[i][1] = fmaf(wgt, v.y, o[i][1]);
        o[i][2] = fmaf(wgt, v.z, o[i][2]);
        o[i][3] = fmaf(wgt, v.w, o[i][3]);
      }
    }
  }
  float f = a.o.out_scale;
  if (a.o.w) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = fmaf(o[i][k], o[i][k], sum);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    f *= rsqrtf(sum / (2 * D) + a.o.eps);
  }
  __nv_bfloat16* dst = a.o.out + (bt * heads + head) * (2 * D) + 4 * lane;
#pragma unroll
  for (int i = 0; i < V; ++i)
    *reinterpret_cast<uint2*>(dst + 128 * i) = diff_finish(o[i], f, a.o.w, 128 * i + 4 * lane);
  if (a.o.lse && lane < 2) {
    const float l = lane ? L[1] : L[0], mm = lane ? M[1] : M[0];
    a.o.lse[bt * a.Hq + 2 * head + lane] = l == 0.f ? -INFINITY : (mm + log2f(l)) * kDiffLn2;
  }
}

struct DiffPrefillPlan {
  int TQ, tiles, nsplit;
  size_t ml_bytes, bytes;
};

// Ranges per tile: the smallest count up to 16 that takes the fewest waves of
// one CTA per SM per unit of work.
static int diff_nsplit(int64_t ctas, int sms) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 16; ++s) {
    const double waves = static_cast<double>((ctas * s + sms - 1) / sms) / s;
    if (waves < 0.93 * least) {
      least = waves;
      best = s;
    }
  }
  return best;
}

static int diff_prefill_plan(const nk_pool* p, int B, int Tc, int Hq, DiffPrefillPlan* pl) {
  const int rc = check_diff_shape(p, B, Tc, Hq);
  if (rc) return rc;
  const int H = p->desc.num_kv_heads, G = Hq / H, D = p->desc.head_dim;
  if (G > 64) return fail(NK_ERR_UNSUPPORTED, "Hq / num_kv_heads must be <= 64");
  if (H / 2 > 65535) return fail(NK_ERR_UNSUPPORTED, "too many KV heads");
  pl->TQ = 128 / G;
  pl->tiles = (Tc - 1) / pl->TQ + 1;
  const int64_t work = static_cast<int64_t>(B) * (H / 2) * pl->tiles;
  if (work > (int64_t(1) << 24) || static_cast<int64_t>(Tc) * Hq > (int64_t(1) << 30))
    return fail(NK_ERR_SHAPE, "too many tokens in one chunk");
  pl->nsplit = diff_nsplit(2 * work, p->num_sms);
  const size_t rows = static_cast<size_t>(work) * pl->nsplit * 2 * 128;
  pl->ml_bytes = (rows * sizeof(float2) + 255) / 256 * 256;
  pl->bytes = pl->ml_bytes + rows * 2 * D * sizeof(float);
  return NK_OK;
}

}  // namespace nk

using namespace nk;

extern "C" int nk_diff_prefill_workspace_bytes(const nk_pool* pool, int32_t B, int32_t Tc, int32_t Hq, size_t* bytes) {
  clear_error();
  if (!pool || !bytes) return fail(NK_ERR_INVALID_ARG, "null argument");
  DiffPrefillPlan pl;
  const int rc = diff_prefill_plan(pool, B, Tc, Hq, &pl);
  if (rc) return rc;
  *bytes = pl.bytes;
  return NK_OK;
}

extern "C" int nk_paged_diff_prefill_attention(const void* q_chunk, int32_t Hq, const nk_pool* pool, int32_t layer,
                                               const int32_t* block_tables, const int32_t* table_rows,
                                               const int32_t* prefix_len, const int32_t* chunk_len, int32_t B,
                                               int32_t Tc, float softmax_scale, const nk_diff* diff, void* out,
                                               float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  DiffPrefillArgs a;
  if (!chunk_len) return fail(NK_ERR_INVALID_ARG, "null argument to nk_paged_diff_prefill_attention");
  int rc = check_diff("nk_paged_diff_prefill_attention", q_chunk, Hq, pool, layer, block_tables, table_rows, prefix_len,
                      B, Tc, softmax_scale, diff, out, lse, &a.o);
  if (rc) return rc;
  DiffPrefillPlan pl;
  if ((rc = diff_prefill_plan(pool, B, Tc, Hq, &pl))) return rc;
  if (!workspace || workspace_bytes < pl.bytes)
    return fail(NK_ERR_WORKSPACE, "workspace needs " + std::to_string(pl.bytes) + " bytes");
  if (!aligned16(workspace)) return fail(NK_ERR_ALIGN, "workspace must be 16-byte aligned");
  const int np = pool->n_planes;
  a.q = static_cast<const __nv_bfloat16*>(q_chunk);
  a.tables = block_tables;
  a.table_rows = table_rows;
  a.prefix_len = prefix_len;
  a.chunk_len = chunk_len;
  a.ks = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 2]) : nullptr;
  a.vs = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 3]) : nullptr;
  a.ws_ml = static_cast<float2*>(workspace);
  a.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.ml_bytes);
  a.status = pool->status;
  a.scale_log2 = softmax_scale * kDiffLog2e;
  // masked scores are infinities times the scale: 0 becomes the least normal
  // number, which no finite score makes visible
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.17549435e-38f;
  a.B = B;
  a.Tc = Tc;
  a.Hq = Hq;
  a.H = pool->desc.num_kv_heads;
  a.G = Hq / a.H;
  a.L = pool->L;
  a.M = pool->M;
  a.C = pool->desc.max_concurrency;
  a.TQ = pl.TQ;
  a.tiles = pl.tiles;
  a.nsplit = pl.nsplit;
  a.head_major = pool->desc.order == NK_HEAD_MAJOR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(2 * pl.tiles * pl.nsplit, a.H / 2, B);
  cudaError_t e = pool->desc.profile == NK_BF16 ? diff_prefill_bf16(pool, layer, a, grid, s)
                                                : diff_prefill_quant(pool, layer, a, grid, s);
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill launch");
  const dim3 join(static_cast<unsigned>((static_cast<int64_t>(Tc) * (Hq / 2) + kJoinThreads / 32 - 1) / (kJoinThreads / 32)),
                  B);
  e = pool->desc.head_dim == 64 ? launch_pdl(diff_prefill_join_kernel<64>, join, dim3(kJoinThreads), 0, s, a)
                                : launch_pdl(diff_prefill_join_kernel<128>, join, dim3(kJoinThreads), 0, s, a);
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill join launch");
  return NK_OK;
}
