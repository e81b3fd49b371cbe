// diff_prefill.cuh -- what the differential prefill kernels share: arguments,
// the store of a tile's partial result and the plan of the splits.
//
// A CTA owns 128 query rows of one map of one (row b, pair of KV heads), TQ =
// floor(128 / G) consecutive chunk tokens times the G heads that share the pair,
// and one range of key pages; its values are those of both KV heads (2 D wide).
// Every CTA leaves (m, l, O) of its rows in the workspace, and
// diff_prefill_join_kernel joins the ranges, takes the difference of the maps
// and norms it.
#pragma once

#include "diff.cuh"
#include "tcgen05.cuh"

namespace nk {

struct DiffPrefillArgs {
  const __nv_bfloat16* q;  // [B][Tc][Hq][D]
  const int32_t* tables;
  const int32_t* table_rows;
  const int32_t* prefix_len;
  const int32_t* chunk_len;
  const uint8_t* ks;  // scale planes of the layer (nullptr for BF16)
  const uint8_t* vs;
  float2* ws_ml;  // [B][pairs][tiles][nsplit][2][128] (m, l)
  float* ws_o;    // [B][pairs][tiles][nsplit][2][128][2 D]
  int* status;
  float scale_log2;  // softmax_scale * log2(e)
  int B, Tc, Hq, H, G, L, M, C;
  int TQ, tiles, nsplit;
  int head_major;
  DiffOut o;
};

// At least this many pages per range: shorter ones cost more in start-up and
// partials than they win.
constexpr int kDiffSplitPages = 4;

// What a CTA works on; n < 0: nothing.  Later tiles see more keys and are
// launched first; the two maps of a tile are neighbours.
struct DiffTile {
  int b, pair, map, qt, split, row, prefix, chunk, t0, p_lo, n;
};

__device__ __forceinline__ DiffTile diff_tile(const DiffPrefillArgs& a) {
  DiffTile w;
  w.map = blockIdx.x & 1;
  const int x = blockIdx.x >> 1;
  w.split = x % a.nsplit;
  w.qt = a.tiles - 1 - x / a.nsplit;
  w.pair = blockIdx.y;
  w.b = blockIdx.z;
  w.row = a.table_rows[w.b];
  w.prefix = a.prefix_len[w.b];
  w.chunk = a.chunk_len[w.b];
  w.n = -1;
  if (w.row < 0 || w.row >= a.C || w.prefix < 0 || w.chunk < 0 || w.chunk > a.Tc ||
      static_cast<int64_t>(w.prefix) + w.chunk > static_cast<int64_t>(a.L) * 64) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && w.pair == 0) set_status(a.status, NK_STATUS_FRONTIER);
    return w;
  }
  w.t0 = w.qt * a.TQ;
  if (w.t0 >= w.chunk) return w;
  const int last = min(w.t0 + a.TQ, w.chunk) - 1;
  const int pages = (w.prefix + last + 64) / 64;
  const int per = max((pages + a.nsplit - 1) / a.nsplit, kDiffSplitPages);
  w.p_lo = min(w.split * per, pages);
  w.n = min(w.p_lo + per, pages) - w.p_lo;
  return w;
}

// Row m's partial of this CTA (TMEM columns [tmem_o, + 2 D) of the thread's
// lane); has_o: a page was visited.
template <int D>
__device__ __forceinline__ void diff_store(const DiffPrefillArgs& a, const DiffTile& w, uint32_t tmem_o, bool has_o,
                                           bool valid, int m, float m_used, float l) {
  const int64_t part =
      (((static_cast<int64_t>(w.b) * (a.H / 2) + w.pair) * a.tiles + w.qt) * a.nsplit + w.split) * 2 + w.map;
  if (valid) a.ws_ml[part * 128 + m] = make_float2(has_o ? m_used : -INFINITY, has_o ? l : 0.f);
  if (!has_o) return;
  float* dst = a.ws_o + (part * 128 + m) * (2 * D);
#pragma unroll 1
  for (int c0 = 0; c0 < 2 * D; c0 += 32) {
    uint32_t v[32];
    tc::ld32(tmem_o + c0, v);
    tc::wait_ld();
    if (valid) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(dst + c0 + 4 * c) = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
  }
}

cudaError_t diff_prefill_bf16(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid, cudaStream_t s);
cudaError_t diff_prefill_quant(const nk_pool* p, int layer, const DiffPrefillArgs& a, dim3 grid, cudaStream_t s);

}  // namespace nk
