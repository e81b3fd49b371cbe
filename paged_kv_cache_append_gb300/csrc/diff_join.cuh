// diff_join.cuh -- joins the partials of the tile kernel (diff_tile.cuh), takes the
// difference of the maps and its norm.
//
// A CTA owns ROWS neighbouring query rows of a tile, both maps: lanes along the rows
// read 16 ROWS consecutive bytes of a partial (rows are its innermost index), threads
// of a row own every 4-dim slice from their own on.  Which partials a tile has follows
// from the lengths, which are read before the wait for the partials.  Every partial is
// read once and the output written once: bound by L2, after a chain of three loads.
#pragma once

#include "diff_tile.cuh"

namespace nk {

struct DiffTileJoinArgs {
  const int32_t* table_rows;
  const int32_t* lengths;    // chunks: prefix_len; decode: frontiers
  const int32_t* chunk_len;  // chunks
  const float2* ws_ml;
  const float* ws_o;
  int B, T, Hq, H, G, L, C;
  int TQ, tiles, cg;  // chunks: tokens of a CTA's tile, tiles of a cluster's tokens, CTAs of a cluster
  int ctas;           // clusters of the tile kernel (decode: CTAs per pair)
  DiffOut o;
};

constexpr int kDiffMaxPieces = 256;  // of one tile: at most one per CTA

template <int D, bool BOTH>
struct DiffJoinCfg {
  static constexpr int ROWS = BOTH && D == 128 ? 4 : 8;  // decode has few rows: more CTAs
  static constexpr int C4 = D / 2;                       // 4-dim slices of a row
  static constexpr int SL = 256 / ROWS < C4 ? 256 / ROWS : C4, V = C4 / SL, THREADS = ROWS * SL;
};

template <int D, bool BOTH>
__global__ void __launch_bounds__((DiffJoinCfg<D, BOTH>::THREADS)) diff_tile_join_kernel(DiffTileJoinArgs a) {
  using Cfg = DiffJoinCfg<D, BOTH>;
  constexpr int ROWS = Cfg::ROWS, SL = Cfg::SL, V = Cfg::V, NWARP = Cfg::THREADS / 32;
  __shared__ DiffChunkRows s_rows;
  __shared__ int64_t s_before;
  __shared__ float s_w[2][ROWS][kDiffMaxPieces];
  __shared__ float s_sum[NWARP][ROWS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pair = blockIdx.y, b = blockIdx.z;
  const int blocks = BOTH ? 1 : (a.TQ * a.G + ROWS - 1) / ROWS;
  const int qt = BOTH ? 0 : blockIdx.x / blocks, r0 = (blockIdx.x - qt * blocks) * ROWS;
  // ---- the partials of this tile (inputs of the call: complete since before the tile
  // kernel let this one start; read past L1, which the wait below has not renewed) ------
  const int cg = BOTH ? 1 : a.cg, TQ = a.TQ * cg, dt = qt / cg;  // a cluster's tile
  int64_t slot0[2];
  int np[2], tokens;
  if constexpr (BOTH) {
    const DiffRows rows = diff_rows(a.lengths, a.table_rows, a.B, a.L, a.C, a.ctas, nullptr);
    np[0] = np[1] = __shfl_sync(0xffffffffu, rows.ns, b);
    slot0[0] = slot0[1] = static_cast<int64_t>(pair) * a.ctas + __shfl_sync(0xffffffffu, rows.end, b) - np[0];
    tokens = a.T;
  } else {
    for (int i = warp; i < a.B; i += NWARP)
      s_rows.fill(a.table_rows, a.lengths, a.chunk_len, a.B, a.T, a.L, a.C, TQ, i, nullptr);
    __syncthreads();
    if (dt >= s_rows.tiles[b]) return;
    if (warp == 0) {
      const int64_t before = diff_tile_units(s_rows.prefix[b], s_rows.chunk[b], TQ, dt);
      if (lane == 0) s_before = before;
    }
    __syncthreads();
    const int64_t W = s_rows.total(a.B, a.H), ctas = diff_chunk_ctas(W, a.ctas);
    int64_t at = s_before + kDiffTileCost + 2 * pair * s_rows.units[b];  // unit of page 0, map 1
    for (int i = 0; i < b; ++i) at += s_rows.units[i] * a.H;
    const int pages = s_rows.tile_pages(b, dt, TQ);
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      const int64_t from = at + map * s_rows.units[b];
      const int c0 = static_cast<int>(((from + 1) * ctas - 1) / W), c1 = static_cast<int>(((from + pages) * ctas - 1) / W);
      np[map] = c1 - c0 + 1;
      slot0[map] = ((static_cast<int64_t>(b) * a.H + 2 * pair + map) * a.tiles + dt + c0) * a.cg + qt % a.cg;
    }
    tokens = s_rows.chunk[b];
  }
  const auto token_of = [&](int r) { return (BOTH ? 0 : qt * a.TQ) + r / a.G; };
  const auto there = [&](int r) { return (BOTH || r < a.TQ * a.G) && token_of(r) < tokens; };
  griddep_wait();  // the partials
  griddep_launch_dependents();

  // ---- weights: a warp per row -----------------------------------------------------------
  for (int rr = warp; rr < ROWS; rr += NWARP) {
    const int r = r0 + rr;
    if (!there(r)) continue;
    const int head = pair * a.G + r % a.G;
    const int64_t bt = static_cast<int64_t>(b) * a.T + token_of(r);
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      const float2* ml = a.ws_ml + slot0[map] * 128 + (BOTH ? 64 * map : 0) + r;
      float M = -INFINITY, L = 0.f;
      float2 first = make_float2(-INFINITY, 0.f);
      for (int s = lane; s < np[map]; s += 32) {
        const float2 x = ml[static_cast<int64_t>(s) * cg * 128];
        if (s < 32) first = x;
        M = fmaxf(M, x.x);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      for (int s = lane; s < np[map]; s += 32) {
        const float2 x = s < 32 ? first : ml[static_cast<int64_t>(s) * cg * 128];
        const float e = x.y == 0.f ? 0.f : ex2(x.x - M);  // a piece that saw no key weighs nothing
        s_w[map][rr][s] = e;
        L += e * x.y;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
      const float f = L == 0.f ? 0.f : (map ? -a.o.lambda[bt * a.o.lambda_stride + head] : 1.f) / L;
      for (int s = lane; s < np[map]; s += 32) s_w[map][rr][s] *= f;
      if (a.o.lse && lane == 0)
        a.o.lse[bt * a.Hq + 2 * head + map] = L == 0.f ? -INFINITY : (M + log2f(L)) * kDiffLn2;
    }
  }
  __syncthreads();

  // ---- o = sum over pieces of both maps, its norm, the output ------------------------------
  const int rr = tid % ROWS, sl = tid / ROWS, r = r0 + rr;
  const bool mine = there(r);
  float o[V][4];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
  if (mine) {
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      const float4* src = reinterpret_cast<const float4*>(a.ws_o) + slot0[map] * (Cfg::C4 * 128) + (BOTH ? 64 * map : 0) + r;
#pragma unroll 4
      for (int s = 0; s < np[map]; ++s) {
        const float w = s_w[map][rr][s];
        if (w != 0.f) {  // also what an empty piece has not written
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float4 v = __ldcs(src + (static_cast<int64_t>(s) * cg * Cfg::C4 + sl + k * SL) * 128);
            o[k][0] = fmaf(w, v.x, o[k][0]);
            o[k][1] = fmaf(w, v.y, o[k][1]);
            o[k][2] = fmaf(w, v.z, o[k][2]);
            o[k][3] = fmaf(w, v.w, o[k][3]);
          }
        }
      }
    }
  }
  float f = a.o.out_scale;
  if (a.o.w) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = fmaf(o[k][i], o[k][i], sum);
#pragma unroll
    for (int off = 16; off >= ROWS; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane < ROWS) s_sum[warp][lane] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < NWARP; ++w) sum += s_sum[w][rr];
    f *= rsqrtf(sum / (2 * D) + a.o.eps);
  }
  if (mine) {
    const int64_t bt = static_cast<int64_t>(b) * a.T + token_of(r);
    __nv_bfloat16* dst = a.o.out + (bt * (a.Hq / 2) + pair * a.G + r % a.G) * (2 * D);
#pragma unroll
    for (int k = 0; k < V; ++k)
      *reinterpret_cast<uint2*>(dst + 4 * (sl + k * SL)) = diff_finish(o[k], f, a.o.w, 4 * (sl + k * SL));
  }
}

template <bool BOTH>
inline cudaError_t launch_diff_tile_join(int D, const DiffTileJoinArgs& j, cudaStream_t s) {
  const auto go = [&](auto kernel, int rows, int threads) {
    const int blocks = BOTH ? (j.T * j.G + rows - 1) / rows : (j.TQ * j.G + rows - 1) / rows * j.tiles * j.cg;
    return launch_pdl(kernel, dim3(blocks, j.H / 2, j.B), dim3(threads), 0, s, j);
  };
  return D == 64 ? go(diff_tile_join_kernel<64, BOTH>, DiffJoinCfg<64, BOTH>::ROWS, DiffJoinCfg<64, BOTH>::THREADS)
                 : go(diff_tile_join_kernel<128, BOTH>, DiffJoinCfg<128, BOTH>::ROWS, DiffJoinCfg<128, BOTH>::THREADS);
}

}  // namespace nk
