// diff_join.cuh -- joins the partials of the tile kernel (diff_tile.cuh), takes the
// difference of the maps and its norm.
//
// A CTA owns ROWS neighbouring query rows of a tile, both maps: lanes along the rows
// read 16 ROWS consecutive bytes of a partial (rows are its innermost index), a thread
// owns V neighbouring 4-dim slices of its row.  Which partials a tile has follows
// from the lengths, which are read before the wait for the partials.  Every partial is
// read once and the output written once: bound by L2, after a chain of three loads (2048
// tokens of 8 heads, 52 MB of partials: 21 us with cold caches; with the weights of four
// rows one after the other in a warp, 29).
#pragma once

#include <type_traits>

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

constexpr int kDiffMaxPieces = 160;  // of one tile: at most one per cluster

template <int D, int ROWS>
struct DiffJoinCfg {
  static constexpr int C4 = D / 2;                       // 4-dim slices of a row
  static constexpr int SL = 256 / ROWS < C4 ? 256 / ROWS : C4, V = C4 / SL, THREADS = ROWS * SL;
};

template <int D, int ROWS, bool BOTH>
__global__ void __launch_bounds__((DiffJoinCfg<D, ROWS>::THREADS)) diff_tile_join_kernel(DiffTileJoinArgs a) {
  using Cfg = DiffJoinCfg<D, ROWS>;
  constexpr int SL = Cfg::SL, V = Cfg::V, NWARP = Cfg::THREADS / 32;
  constexpr int AHEAD = BOTH ? 8 : ROWS == 32 ? 0 : 2;  // pieces that are read ahead (32 rows have V slices in flight)
  __shared__ DiffChunkRows s_rows;
  __shared__ int64_t s_slot[2];
  __shared__ int s_np[2];
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
      if (lane < 2) {  // of map `lane`
        const int64_t W = s_rows.total(a.B, a.H), ctas = diff_chunk_ctas(W, a.ctas);
        int64_t from = before + kDiffTileCost + (2 * pair + lane) * s_rows.units[b];  // unit of page 0
        for (int i = 0; i < b; ++i) from += s_rows.units[i] * a.H;
        const int c0 = static_cast<int>(((from + 1) * ctas - 1) / W);
        const int c1 = static_cast<int>(((from + s_rows.tile_pages(b, dt, TQ)) * ctas - 1) / W);
        s_np[lane] = c1 - c0 + 1;
        s_slot[lane] = ((static_cast<int64_t>(b) * a.H + 2 * pair + lane) * a.tiles + dt + c0) * a.cg + qt % a.cg;
      }
    }
    __syncthreads();
#pragma unroll
    for (int map = 0; map < 2; ++map) {
      np[map] = s_np[map];
      slot0[map] = s_slot[map];
    }
    tokens = s_rows.chunk[b];
  }
  const auto token_of = [&](int r) { return (BOTH ? 0 : qt * a.TQ) + r / a.G; };
  const auto there = [&](int r) { return (BOTH || r < a.TQ * a.G) && token_of(r) < tokens; };
  griddep_wait();  // the partials
  griddep_launch_dependents();
  // the first pieces' values of this thread's row, while their weights are not known yet
  const int rr = tid % ROWS, sl = tid / ROWS, r = r0 + rr;
  const bool mine = there(r);
  const float4* src[2];
  float4 ahead[2][AHEAD > 0 ? AHEAD : 1][V];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    src[map] = reinterpret_cast<const float4*>(a.ws_o) + slot0[map] * (Cfg::C4 * 128) + (BOTH ? 64 * map : 0) + r;
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (mine && s < np[map])
          ahead[map][s][k] = __ldcs(src[map] + (static_cast<int64_t>(s) * cg * Cfg::C4 + sl * V + k) * 128);
  }

  // ---- weights: LP lanes per (map, row), every one at once --------------------------------
  {
    constexpr int LP = Cfg::THREADS / (2 * ROWS);
    static_assert(LP >= 1 && LP <= 32 && (LP & (LP - 1)) == 0, "lanes of a (map, row)");
    const int sub = tid % LP, map = tid / LP / ROWS, wr = tid / LP % ROWS, x = r0 + wr;
    const int pieces = there(x) ? (map ? np[1] : np[0]) : 0;
    const float2* ml = a.ws_ml + (map ? slot0[1] : slot0[0]) * 128 + (BOTH ? 64 * map : 0) + x;
    float M = -INFINITY, L = 0.f;
    float2 first = make_float2(-INFINITY, 0.f);
    for (int s = sub; s < pieces; s += LP) {
      const float2 v = ml[static_cast<int64_t>(s) * cg * 128];
      if (s < LP) first = v;
      M = fmaxf(M, v.x);
    }
#pragma unroll
    for (int off = LP / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    for (int s = sub; s < pieces; s += LP) {
      const float2 v = s < LP ? first : ml[static_cast<int64_t>(s) * cg * 128];
      const float e = v.y == 0.f ? 0.f : ex2(v.x - M);  // a piece that saw no key weighs nothing
      s_w[map][wr][s] = e;
      L += e * v.y;
    }
#pragma unroll
    for (int off = LP / 2; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (pieces > 0) {
      const int head = pair * a.G + x % a.G;
      const int64_t bt = static_cast<int64_t>(b) * a.T + token_of(x);
      const float f = L == 0.f ? 0.f : (map ? -a.o.lambda[bt * a.o.lambda_stride + head] : 1.f) / L;
      for (int s = sub; s < pieces; s += LP) s_w[map][wr][s] *= f;
      if (a.o.lse && sub == 0)
        a.o.lse[bt * a.Hq + 2 * head + map] = L == 0.f ? -INFINITY : (M + log2f(L)) * kDiffLn2;
    }
  }
  __syncthreads();

  // ---- o = sum over pieces of both maps, its norm, the output ------------------------------
  float o[V][4];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
  const auto add = [&](float w, const float4& v, float (&x)[4]) {
    x[0] = fmaf(w, v.x, x[0]);
    x[1] = fmaf(w, v.y, x[1]);
    x[2] = fmaf(w, v.z, x[2]);
    x[3] = fmaf(w, v.w, x[3]);
  };
  if (mine) {
#pragma unroll
    for (int map = 0; map < 2; ++map) {
#pragma unroll
      for (int s = 0; s < AHEAD; ++s) {
        const float w = s < np[map] ? s_w[map][rr][s] : 0.f;
        if (w != 0.f) {  // 0: also what an empty piece has not written
#pragma unroll
          for (int k = 0; k < V; ++k) add(w, ahead[map][s][k], o[k]);
        }
      }
#pragma unroll (BOTH ? 4 : 1)
      for (int s = AHEAD; s < np[map]; ++s) {
        const float w = s_w[map][rr][s];
        if (w != 0.f) {
#pragma unroll
          for (int k = 0; k < V; ++k)
            add(w, __ldcs(src[map] + (static_cast<int64_t>(s) * cg * Cfg::C4 + sl * V + k) * 128), o[k]);
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
      *reinterpret_cast<uint2*>(dst + 4 * (sl * V + k)) = diff_finish(o[k], f, a.o.w, 4 * (sl * V + k));
  }
}

// Rows of a CTA: 32 (512 bytes of a partial at a time, one plan for them) where that
// still makes a CTA per SM, else 8; a decode, of at most 64 rows, 4 or 8.  With 8 rows and
// with 32, us: 4 x 2048 tokens of 8 heads 85 and 68, 501 tokens of 2 heads 8 and 18.
template <bool BOTH>
inline cudaError_t launch_diff_tile_join(int D, int sms, const DiffTileJoinArgs& j, cudaStream_t s) {
  const auto blocks = [&](int rows) {
    return BOTH ? (j.T * j.G + rows - 1) / rows : (j.TQ * j.G + rows - 1) / rows * j.tiles * j.cg;
  };
  const auto go = [&](auto kernel, int rows, int threads) {
    return launch_pdl(kernel, dim3(blocks(rows), j.H / 2, j.B), dim3(threads), 0, s, j);
  };
  const auto pick = [&](auto dim) {
    constexpr int D_ = decltype(dim)::value, FEW = BOTH && D_ == 128 ? 4 : 8;
    if (!BOTH && static_cast<int64_t>(blocks(32)) * (j.H / 2) * j.B >= sms)
      return go(diff_tile_join_kernel<D_, BOTH ? FEW : 32, BOTH>, 32, DiffJoinCfg<D_, 32>::THREADS);
    return go(diff_tile_join_kernel<D_, FEW, BOTH>, FEW, DiffJoinCfg<D_, FEW>::THREADS);
  };
  return D == 64 ? pick(std::integral_constant<int, 64>{}) : pick(std::integral_constant<int, 128>{});
}

}  // namespace nk
