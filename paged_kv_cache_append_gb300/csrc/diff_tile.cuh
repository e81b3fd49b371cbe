// diff_tile.cuh -- differential attention of 128 query rows to a CTA on the
// 5th-generation tensor cores (kernel template; instantiated per profile in
// diff_tile_*.cu): prompt chunks, and decode / verify tokens of many query rows.
//
// Per page of 64 keys, for the query rows of a map m of a pair of KV heads:
//   S = Q_m K_m^T;   P = exp2(S - reference);   O += P [V1 V2]
// 2 D + 4 D flops per (query row, key): the least for two maps over one wide value.
//
// Chunks (BOTH = false).  A cluster of two CTAs owns 2 TQ consecutive tokens, TQ =
// floor(128 / G), of one map: 128 query rows in each CTA (TQ tokens times the G heads
// that share the pair), and every MMA is one of both (cta_group::2, M 256).  A CTA
// stages and converts one half of each operand: 32 of a page's keys, and the value head
// of its rank (FP8-row and INT8-G64 values: 64 of the dims of both heads, since each head
// has its own P; at head_dim 64 that half would be less than a swizzle atom, so there a
// CTA works alone, M 128).  With one CTA to an MMA a BF16 chunk read its pages at 8.3
// TB/s from L2, which bound it: 8192 tokens behind 0, 731 us, 500 in pairs.
// The grid is one cluster for every two SMs; the line of all tiles' pages is cut into equal
// parts (diff_chunk_first), so that a CTA sets up once and no wave is short: with a CTA
// to a tile and range, each started and drained for 10 us.
//
// Decode / verify (BOTH = true).  One CTA; lanes 0-63 are the (up to 64) query rows of map
// 1, lanes 64-127 those of map 2, so that every page is read and converted once:
//   S = [Q1; 0] K1^T + [0; Q2] K2^T, two MMAs (M 128) into one S.
//
// Tensor memory: NS S buffers of 64 columns, Q (D / 2 columns; BOTH: two operands), O
// [256, 256 + 2 D).  P goes over the S that its own warp computed it from: keys
// [32 h, +32) in columns [32 h, +16) of the buffer.
//
// Operands.  Scores: BF16 pages as they are; FP8-row keys of head_dim 128 as raw
// E4M3 codes with q in two E4M3 terms, other quantized keys as exact f16 tiles
// (INT8-G64: two), their per-key factors applied to the scores in fp32, as in
// qprefill.cu.  P is f16 for every profile, so that its weights keep 11 bits (bf16
// weights: an error of 0.0025 against 0.0017 over a BF16 chunk), and V therefore too:
//   * NVFP4 values carry their scales exactly; one P serves both heads, N = 2 D;
//   * FP8-row and INT8-G64 values leave a factor per key to the weights, so each
//     head has its own P (the second 16 columns further), N = D twice;
//   * BF16 values are rewritten in place, v 2^k with a power of two per strip of dims (a
//     converter warp's) that brings the strip's largest value so far below 2^15 and above
//     2^-3 (0 while it is there by itself): exact for every element from 2^-11 of the
//     largest on (2^-14 itself, where k = 0), and to 2^-19 of the largest below; infinities
//     and NaN have no part in k.  k only falls (then O is rescaled, in both CTAs of a
//     pair: the strips' factors are stored into both), and the store divides it out.
// Weights are stored lifted: 2^(s - reference) is at most 2^8, so 2^7 of it (with value factors,
// 2^k by the largest of them, v_lift) stays below 2^15, and the weights that f16 holds to 11 bits
// reach down to 2^-21 of a row's largest instead of 2^-14; below, they are within 2^-32 of it
// (beside one key of weight 1, keys of 2^-20 each were off by 3%).
//
// Warps (640 threads): 0-7 softmax, warp w lanes 32 (w & 3) of every second page, from
// w >> 2 on, a whole row to a thread; 8 TMA producer; 9 MMA issuer (CTA 1's tells CTA 0's
// when it could go); 10 idle (registers move by warpgroups); 11 factors of the keys'
// scales; 12-19 converters, for quantized pages in two groups on alternate pages.  A
// page's softmax is a chain of waits and tensor-memory trips of 1600-2000 cycles, longer
// than the MMAs of a page (800, head_dim 128): so two pages are in it at a time, S NS - 1
// pages ahead of PV.  A wait on a complete barrier takes 120-250 cycles beside 19 busy
// warps, most of it latency: a role's barriers of a page are tried together (K8V4 batch
// below: 1196 us one by one, 1104 together).
// The warps of a row hand on its reference maximum from page to page, right after the
// page's maximum; it moves lazily (by a score more than 2^8 above it).  The MMAs are
// issued by an elected lane of a warp that runs the loop as a whole: from a branch of one
// lane each issue took 47-54 cycles (M 128, N 64, A in tensor memory), from the whole
// warp the 33 of the tensor core.
//
// Measured (with the join, L2 cold): chunk of 2048 tokens behind 8150, 16 query heads,
// BF16: 210 us, 57% of the dense rate; 4 x 2048 behind 16384, K8V4: 1127 us, 66%; verify
// of 4 tokens of 32 heads over 8 x 131072, K8V4: 172 us, 57% of the copy rate.  A page of a
// chunk takes 1050 (K8V4) to 1350 cycles (BF16): what bounds it is the loop from S over the
// softmax to the PV that frees S's buffer, three pages long; two warps for S and PV, which
// shorten that of the issue, were 4 us faster for a BF16 chunk (head_dim 64: 17 of 250) and 7
// slower for the verify.  A piece of a tile costs 7 us beside its pages (queries, first
// scores, partial).  The verify's two MMAs for S, each with half of its rows zero, and M 128 of
// values are 8.4 MFLOP a page and pair whatever the rows: 110 us of those 172 at the dense rate.
// The roles' registers do not hold everything (-Xptxas -v): the chunk kernels spill 176 (BF16)
// to 280 bytes (INT8-G64) a thread, the decodes 0 to 72; executed, 16 local loads a CTA's page
// for BF16, 13 K8V4, 51 FP8-row, 55 INT8-G64, of 2900 to 5000 warp instructions.
//
// S(j) goes over the P that PV(j - NS) reads, with no wait between: the MMAs that one thread
// issues run in issue order, here also across kinds (E4M3 scores, f16 values), shapes and the
// two CTAs of a pair.
//
// All waits are bounded; a wait that ran out ends its warp's work (for all lanes, and for
// both softmax warps of a row), the others' waits run out too, and the CTA leaves without
// results once the copies in flight landed.
#pragma once

#include "diff.cuh"
#include "packed.cuh"
#include "qtile.cuh"
#include "tcgen05.cuh"

namespace nk {

struct DiffTileArgs {
  const __nv_bfloat16* q;  // [B][T][Hq][D]
  const int32_t* tables;
  const int32_t* table_rows;
  const int32_t* lengths;    // chunks: prefix_len; decode: frontiers
  const int32_t* chunk_len;  // chunks
  const uint8_t* ks;         // scale planes of the layer (nullptr for BF16)
  const uint8_t* vs;
  float2* ws_ml;  // [part][128] (m, l)
  float* ws_o;    // [part][D / 2][128][4]: neighbouring rows store next to each other
  int* status;
  float scale_log2;  // |softmax_scale| log2 e, > 0
  int negate;        // softmax_scale < 0: the queries change sign
  int B, T, Hq, H, G, L, M, C;
  int TQ, tiles;          // chunks
  int ctas;               // decode: CTAs per pair
  int head_major;
};

// CTAs to a tile of a chunk: a pair, but for profiles whose halves of a value would be
// less than the 64 dims of a swizzle atom.
constexpr int diff_chunk_group(int kind_v, int D) { return (kind_v == KIND_FP8 || kind_v == KIND_INT8) && D == 64 ? 1 : 2; }

// Chunks: the work of all tiles is one line, in order of (row b, pair, map, tile, page),
// a tile's pages after kDiffTileCost units for its start and end (queries, first scores,
// partial), and cluster c of n takes the units [c W / n, (c + 1) W / n): a tile that crosses
// a boundary has a partial from each of its clusters, numbered tile + cluster.  n is at
// most one CTA per SM and leaves each at least kDiffLeastUnits.  8192 tokens behind 0
// (many short tiles), us, by a tile's cost: 532 with 0, 434 with 6, 421 with 12, 434 with 18;
// 2 x 64 tokens behind 1000, by the least units: 26 with 5, 31 with 16, 34 with 24.
constexpr int kDiffTileCost = 12, kDiffLeastUnits = 5;

// Units of tiles [0, upto) of a row (a warp).
__device__ __forceinline__ int64_t diff_tile_units(int prefix, int chunk, int TQ, int upto) {
  int64_t sum = 0;
  for (int t = threadIdx.x & 31; t < upto; t += 32) sum += (prefix + min((t + 1) * TQ, chunk) + 63) / 64 + kDiffTileCost;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  return sum;
}

// The rows of a call, as every CTA of the chunk kernel and of its join sees them.
struct DiffChunkRows {
  int row[8], prefix[8], chunk[8], tiles[8];
  int64_t units[8];  // of one (pair, map)

  // Warp b fills row b; a refused row has no tiles.
  __device__ void fill(const int32_t* table_rows, const int32_t* prefix_len, const int32_t* chunk_len, int B, int T, int L,
                       int C, int TQ, int warp, int* report) {
    if (warp >= B) return;
    const int rw = __ldcg(table_rows + warp), pre = __ldcg(prefix_len + warp);
    int ch = __ldcg(chunk_len + warp);
    if (rw < 0 || rw >= C || pre < 0 || ch < 0 || ch > T ||
        static_cast<int64_t>(pre) + ch > static_cast<int64_t>(L) * 64) {
      if (report && (threadIdx.x & 31) == 0) set_status(report, NK_STATUS_FRONTIER);
      ch = 0;
    }
    const int n = (ch + TQ - 1) / TQ;
    const int64_t sum = diff_tile_units(pre, ch, TQ, n);
    if ((threadIdx.x & 31) == 0) {
      row[warp] = rw;
      prefix[warp] = pre;
      chunk[warp] = ch;
      tiles[warp] = n;
      units[warp] = sum;
    }
  }
  __device__ int64_t total(int B, int maps) const {
    int64_t w = 0;
    for (int b = 0; b < B; ++b) w += units[b] * maps;
    return w;
  }
  __device__ int tile_pages(int b, int qt, int TQ) const { return (prefix[b] + min((qt + 1) * TQ, chunk[b]) + 63) / 64; }
};

__device__ __forceinline__ int diff_chunk_ctas(int64_t W, int most) {
  return static_cast<int>(min(static_cast<int64_t>(most), max(W / kDiffLeastUnits, static_cast<int64_t>(1))));
}

template <int KK, int KV, int D, bool BOTH>
struct DiffTileCfg {
  static constexpr bool BF16 = KK == KIND_BF16;
  static constexpr int NSOFT = 8, NCONV = 8, THREADS = 32 * (NSOFT + 4 + NCONV);
  // Registers: 640 threads start with 96 each; the softmax warps (64 scores and 16 or 32
  // packed weights at a time) take over what the others do not need.
  static constexpr int R_SOFT = BOTH ? 144 : 136, R_MISC = BOTH ? 40 : 56, R_CONV = 72;
  // (two CTAs of an SM would not fit: each takes all of the tensor memory)
  static_assert(256 * R_SOFT + 128 * R_MISC + 256 * R_CONV <= 640 * 96, "registers of the CTA");
  static constexpr int KCB = BF16 ? 2 * D : code_row_bytes<KK>(D), VCB = BF16 ? 2 * D : code_row_bytes<KV>(D);
  static constexpr int KSB = scale_row_bytes<KK>(D), VSB = scale_row_bytes<KV>(D);
  static constexpr int K_RB = KCB < 128 ? KCB : 128, V_RB = VCB < 128 ? VCB : 128;
  static constexpr int F16 = 64 * D * 2;                     // one head's f16 page tile
  static constexpr bool K_SPLIT = KK == KIND_INT8;           // exact INT8 keys: two f16 tiles
  static constexpr bool K8MMA = KK == KIND_FP8 && D >= 128;  // raw E4M3 keys to the tensor cores
  static constexpr bool K_RAW = BF16 || K8MMA;               // the raw K tile is the operand
  static constexpr bool KEY_FAC = KK == KIND_FP8 || KK == KIND_INT8;  // scores take a factor per key
  static constexpr bool VAL_FAC = KV == KIND_FP8 || KV == KIND_INT8;  // weights take one per key and head
  static constexpr bool HAS_F = KEY_FAC || VAL_FAC || BF16;
  static constexpr int KH = BOTH ? 2 : 1;  // K tiles of a page
  static constexpr int CG = BOTH ? 1 : diff_chunk_group(KV, D);  // CTAs to an MMA
  static constexpr int KR = 64 / CG;                             // keys of a K tile in this CTA
  static constexpr int VH = CG == 2 && !VAL_FAC ? 1 : 2;         // value heads in this CTA
  static constexpr bool V_HALF = CG == 2 && VAL_FAC;             // 64 of the 128 dims of both
  static constexpr int VPART = V_HALF ? 64 * 64 * 2 : 64 * D * 2;  // f16 bytes of a value head here
  static constexpr int RK_CODES = (64 * KCB + 1023) / 1024 * 1024, RV_CODES = (64 * VCB + 1023) / 1024 * 1024;
  static constexpr int RK_HEAD = (RK_CODES + 64 * KSB + 1023) / 1024 * 1024, RK_STAGE = KH * RK_HEAD;
  static constexpr int RV_HEAD = (RV_CODES + 64 * VSB + 1023) / 1024 * 1024, RV_STAGE = BF16 ? 0 : VH * RV_HEAD;
  static constexpr int K_HEAD = K_SPLIT ? 2 * F16 : F16, K_STAGE = K_RAW ? 0 : KH * K_HEAD;
  static constexpr int V_STAGE = VH * VPART;
  // Groups of converter warps, on alternate pages; one where the f16 keys fit once
  // (INT8-G64 decode, head_dim 128), and for BF16, whose strips go from page to page.
  static constexpr int NCG = BF16 || (K_SPLIT && BOTH && D == 128) ? 1 : 2, CGW = NCONV / NCG;
  // Ring depths, as shared memory allows; a group's slots are its own.
  static constexpr int NRK = CG == 2 ? (K_SPLIT ? 4 : 6)
                           : D == 64 ? 4 : BF16 || (K8MMA && KV == KIND_NVFP4) ? 3 : K_SPLIT ? 2 : 4;
  static constexpr int NK = K_RAW ? 1 : CG == 2 ? (K_SPLIT ? 2 : 4) : D == 64 ? (K_SPLIT && BOTH ? 2 : 4) : K_SPLIT ? 1 : 2;
  static constexpr int NV = CG == 2 ? (BF16 ? 6 : K_SPLIT ? 2 : 4) : D == 64 ? 4 : BF16 ? 3 : K8MMA && KV == KIND_NVFP4 ? 4 : 2;
  static constexpr int NRV = BF16 ? NV : CG == 2 ? (K_SPLIT ? 2 : 4) : D == 64 ? 4 : K_SPLIT || (K8MMA && KV == KIND_NVFP4) ? 2 : 4;
  static_assert(NCG == 1 || (NV % 2 == 0 && NRV % 2 == 0 && (K_RAW || (NK % 2 == 0 && NRK % 2 == 0))), "a group's slots");
  static constexpr int NF = 4;  // factor ring: 1 KB per page
  static constexpr int OFF_V = NK * K_STAGE;
  static constexpr int OFF_RK = OFF_V + NV * V_STAGE;
  static constexpr int OFF_RV = OFF_RK + NRK * RK_STAGE;
  static constexpr int OFF_F = OFF_RV + NRV * RV_STAGE;
  static constexpr int NS = BOTH && D == 128 ? 2 : 3;  // S buffers
  static constexpr int OFF_X = OFF_F + NF * 1024;  // [2][128] references, [2][128] final (reference, sum)
  static constexpr int OFF_ROWS = OFF_X + 4096 + 256;  // [4][16] lifts of the BF16 strips
  static constexpr int OFF_BAR = OFF_ROWS + 256;
  static constexpr int NBAR = 2 * NK + 2 * NV + 2 * NRK + 2 * NRV + 2 * NF + 4 * NS + 2 + 8 + (K_RAW ? NRK : NK);
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64 + 1024;
  static constexpr uint32_t COL_S = 0, COL_Q = 64 * NS, COL_O = 256;
  static_assert(COL_Q + KH * (D / 2) <= COL_O, "tensor memory");
  static constexpr uint32_t ID_S = K8MMA  ? tc::idesc_e4m3(128 * CG, 64)
                                   : BF16 ? tc::idesc_bf16(128 * CG, 64, false, false)
                                          : tc::idesc_f16(128 * CG, 64, false, false);
  static constexpr uint32_t ID_O = tc::idesc_f16(128 * CG, VAL_FAC ? D : 2 * D, false, true);
  static constexpr int STRIPS = NCONV * CG, STRIP = 2 * D / STRIPS;  // a converter warp of BF16 values owns a strip of dims
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// What a CTA works on: pages [p_lo, p_lo + n) of one tile (n < 0: nothing).
struct DiffWork {
  int b, pm, qt, p_lo, n;  // pm = 2 pair + map
  int left;                // units of this cluster beyond these (the host bounds them)
};

// The pages of tile w.qt from its unit `u` on, as far as w.left goes.
__device__ __forceinline__ void diff_take(const DiffChunkRows& rows, int TQ, int u, DiffWork& w) {
  const int pages = rows.tile_pages(w.b, w.qt, TQ), take = min(pages + kDiffTileCost - u, w.left);
  w.p_lo = max(u - kDiffTileCost, 0);
  w.n = max(u + take - kDiffTileCost, 0) - w.p_lo;
  w.left -= take;
}

// The next piece with pages; TQ: tokens of a tile (of a cluster).
__device__ __forceinline__ bool diff_chunk_next(const DiffChunkRows& rows, int maps, int TQ, DiffWork& w) {
  do {
    if (w.left == 0) return false;
    if (++w.qt >= rows.tiles[w.b]) {
      w.qt = 0;
      if (++w.pm >= maps) {
        w.pm = 0;
        do ++w.b;
        while (rows.tiles[w.b] == 0);  // units are left: a row with tiles follows
      }
    }
    diff_take(rows, TQ, 0, w);
  } while (w.n == 0);
  return true;
}

// The first piece of cluster c of (at most) `most`; every warp computes it.
__device__ __forceinline__ DiffWork diff_chunk_first(const DiffChunkRows& rows, int B, int maps, int TQ, int c, int most) {
  DiffWork w;
  w.n = -1;
  const int lane = threadIdx.x & 31;
  const int64_t W = rows.total(B, maps);
  const int n = diff_chunk_ctas(W, most);
  if (W == 0 || c >= n) return w;
  const auto cut = [&](int k) {  // k W / n, in 32 bits where they do
    return W < (1 << 22) ? static_cast<int64_t>(static_cast<unsigned>(k) * static_cast<unsigned>(W) / static_cast<unsigned>(n))
                         : k * W / n;
  };
  int64_t at = cut(c);
  w.left = static_cast<int>(cut(c + 1) - at);
  w.b = 0;
  while (at >= rows.units[w.b] * maps) at -= rows.units[w.b++] * maps;
  w.pm = static_cast<int>(at / rows.units[w.b]);
  at -= w.pm * rows.units[w.b];
  for (w.qt = 0;; w.qt += 32) {  // the tile that holds unit `at`, 32 tiles at a time
    const int mine = w.qt + lane < rows.tiles[w.b] ? rows.tile_pages(w.b, w.qt + lane, TQ) + kDiffTileCost : 0;
    int64_t end = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, end, off);
      if (lane >= off) end += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, at < end);
    if (past) {
      const int k = __ffs(past) - 1;
      w.qt += k;
      at -= __shfl_sync(0xffffffffu, end - mine, k);
      break;
    }
    at -= __shfl_sync(0xffffffffu, end, 31);
  }
  diff_take(rows, TQ, static_cast<int>(at), w);
  if (w.n == 0 && !diff_chunk_next(rows, maps, TQ, w)) w.n = -1;
  return w;
}

// Decode: the CTA's split of the plan of all rows; the row as a chunk of T tokens
// after F - T.
__device__ __forceinline__ DiffWork diff_decode_work(const DiffTileArgs& a, DiffChunkRows* rows) {
  DiffWork w;
  const DiffSplit own = diff_split(diff_rows(a.lengths, a.table_rows, a.B, a.L, a.C, a.ctas,
                                             blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32 ? a.status : nullptr),
                                   a.B, blockIdx.x);
  w.b = own.b;
  w.pm = 2 * blockIdx.y;
  w.qt = 0;
  w.p_lo = own.p0;
  w.n = own.b < 0 ? -1 : own.n;  // 0 only for a row without keys
  w.left = 0;
  if (threadIdx.x == 0 && own.b >= 0) {
    rows->row[own.b] = own.row;
    rows->prefix[own.b] = own.F - a.T;
    rows->chunk[own.b] = a.T;
  }
  return w;
}

// ---- the other CTA of a pair ----------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_u32(const void* p, uint32_t rank) {  // p's place in CTA `rank`
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// What such an arrival announces lies in tensor memory, or in shared memory behind a proxy
// fence, for the tensor core: no release at cluster scope, which cost 1500 cycles a page.
__device__ __forceinline__ void peer_arrive(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_u32(bar, rank)) : "memory");
}
// 16 bytes to p's place in CTA `rank`, counted by the barrier at bar's place there.
__device__ __forceinline__ void peer_store(float4* p, float4 v, uint64_t* bar, uint32_t rank) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   peer_u32(p, rank)),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(peer_u32(bar, rank))
               : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// True in one lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t bf16x2_lift(uint32_t w, float f) {  // two bf16 values times f as f16x2
  return pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
}

// |v| 2^-112 of two bf16 values: the exponent field of an f16, for |v| < 2^16
// (below 2^-14 gradually, to 2^-21).
__device__ __forceinline__ uint32_t bf16x2_rebias(uint32_t w) {
  const uint32_t k = 0x07800780u;  // 2^-112
  const __nv_bfloat162 r =
      __hmul2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)), *reinterpret_cast<const __nv_bfloat162*>(&k));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The magnitudes of two bf16 values, 0 for an infinity or a NaN.
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t w) {
  const uint32_t infinity = 0x7F807F80u;
  w &= 0x7FFF7FFFu;
  return w & __hlt2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&infinity));
}

// The f16 pair of bf16 values w from their rebiased magnitudes.
__device__ __forceinline__ uint32_t f16x2_of(uint32_t rebiased, uint32_t w) {
  return (rebiased << 3) | (w & 0x80008000u);
}

// Converter warps of BF16 values: warp cw rewrites its strip of every staged V
// tile, bf16 -> f16 of v 2^k in place, and publishes what its k did.
template <int STRIP>
struct StripOf {
  static constexpr int CH = STRIP / 8;  // 16-byte chunks of the strip in a key's row
  static constexpr int ROWS = 32 / CH;  // keys that a warp access covers
  static constexpr int UNITS = 64 / ROWS;
};

// 2^k that takes the largest bf16 magnitude (its 15 bits) to [2^10, 2^11).
__device__ __forceinline__ int strip_lift(uint32_t bits) {
  const int e = static_cast<int>(bits >> 7);
  return max(-117, min(110, 137 - e));
}

template <int KK, int KV, int D, bool BOTH>
__global__ void __launch_bounds__((DiffTileCfg<KK, KV, D, BOTH>::THREADS), 1)
    diff_tile_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, DiffTileArgs a) {
  using Cfg = DiffTileCfg<KK, KV, D, BOTH>;
  constexpr int NK = Cfg::NK, NV = Cfg::NV, NRK = Cfg::NRK, NRV = Cfg::NRV, NF = Cfg::NF, KH = Cfg::KH, NS = Cfg::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = smem + Cfg::OFF_V;
  uint8_t* sRK = smem + Cfg::OFF_RK;
  uint8_t* sRV = Cfg::BF16 ? sV : smem + Cfg::OFF_RV;
  float* sF = reinterpret_cast<float*>(smem + Cfg::OFF_F);  // [NF][256]: K factors of 2 heads, V factors of 2 heads
  float2* sX = reinterpret_cast<float2*>(smem + Cfg::OFF_X);
  float* sDown = reinterpret_cast<float*>(smem + Cfg::OFF_X + 4096);
  DiffChunkRows* rows = reinterpret_cast<DiffChunkRows*>(smem + Cfg::OFF_ROWS);
  static_assert(sizeof(DiffChunkRows) <= 256, "rows");
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);  // f16 K tiles ready (converters)
  uint64_t* k_empty = k_full + NK;                                      // their S done (MMA commit)
  uint64_t* v_full = k_empty + NK;                                      // f16 V tiles ready
  uint64_t* v_empty = v_full + NV;
  uint64_t* rk_full = v_empty + NV;  // raw K landed (TMA)
  uint64_t* rk_empty = rk_full + NRK;
  uint64_t* rv_full = rk_empty + NRK;  // raw V landed
  uint64_t* rv_empty = rv_full + NRV;
  uint64_t* f_full = rv_empty + NRV;  // factors of a page written
  uint64_t* f_empty = f_full + NF;
  uint64_t* s_full = f_empty + NF;  // [NS]
  uint64_t* p_full = s_full + NS;   // [NS]
  uint64_t* o_done = p_full + NS;   // [NS] PV of the page in S buffer i complete
  uint64_t* q_ready = o_done + NS;
  uint64_t* drain = q_ready + 1;  // every MMA complete
  uint64_t* peer_v = drain + 1;  // [NS] of CTA 0: CTA 1 is ready for PV
  uint64_t* peer_k = peer_v + NS;  // [ring] and for S
  uint64_t* x_full = peer_k + (Cfg::K_RAW ? NRK : NK);  // [2][4] the references of 32 rows after a page are there
  uint32_t* tslot = reinterpret_cast<uint32_t*>(x_full + 8);

  constexpr int CG = Cfg::CG;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;  // this CTA's in its pair
  const int TQ = a.TQ * CG;                                         // tokens of a tile
  if (tid == 0) {
    for (int i = 0; i < NK; ++i) {
      mbar_init(&k_full[i], Cfg::CGW);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], Cfg::CGW);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NRK; ++i) {
      mbar_init(&rk_full[i], 1);
      // released by the converters, a raw operand by the MMA's commit; and where key
      // factors are read, by the warp that does
      mbar_init(&rk_empty[i], (Cfg::K_RAW ? 1 : Cfg::CGW) + (Cfg::KEY_FAC ? 1 : 0));
    }
    for (int i = 0; i < NRV; ++i) {
      mbar_init(&rv_full[i], 1);
      mbar_init(&rv_empty[i], Cfg::CGW + (Cfg::VAL_FAC ? 1 : 0));
    }
    for (int i = 0; i < NF; ++i) {
      mbar_init(&f_full[i], Cfg::BF16 ? Cfg::NCONV : 1);
      mbar_init(&f_empty[i], Cfg::NSOFT / 2 * (Cfg::BF16 ? CG : 1));
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], Cfg::NSOFT / 2);
      mbar_init(&o_done[i], 1);
      mbar_init(&peer_v[i], 1);
    }
    mbar_init(q_ready, Cfg::NSOFT);
    for (int i = 0; i < (Cfg::K_RAW ? NRK : NK); ++i) mbar_init(&peer_k[i], 1);
    mbar_init(drain, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&x_full[i], 1);
    fence_barrier_init();
    prefetch_tmap(&tmk);
    prefetch_tmap(&tmv);
  }
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the other CTA's barriers exist
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();
  DiffWork first;
  if constexpr (BOTH) {
    first = diff_decode_work(a, rows);
  } else {
    rows->fill(a.table_rows, a.lengths, a.chunk_len, a.B, a.T, a.L, a.C, TQ, warp, blockIdx.x == 0 ? a.status : nullptr);
    __syncthreads();
    first = diff_chunk_first(*rows, a.B, a.H, TQ, blockIdx.x / CG, gridDim.x / CG);
  }
  if (first.n < 0) return;  // a pair's CTAs alike

  if (warp == 0) {
    if constexpr (CG == 2) {
      tc::alloc2(tslot, 512);
      tc::relinquish2();
    } else {
      tc::alloc(tslot, 512);
      tc::relinquish();
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;
  // Every role goes through the CTA's pieces; `base` counts the pages of those before.
  const auto next = [&](DiffWork& w, int& base) {
    base += w.n;
    return !BOTH && diff_chunk_next(*rows, a.H, TQ, w);
  };
  const auto mma = [](uint32_t d, uint32_t am, uint64_t bd, uint32_t id, uint32_t acc) {
    if constexpr (CG == 2) tc::mma_ts2(d, am, bd, id, acc);
    else tc::mma_ts(d, am, bd, id, acc);
  };
  const auto mma_f8 = [](uint32_t d, uint32_t am, uint64_t bd, uint32_t id, uint32_t acc) {
    if constexpr (CG == 2) tc::mma_ts2_f8(d, am, bd, id, acc);
    else tc::mma_ts_f8(d, am, bd, id, acc);
  };
  const auto commit = [](uint64_t* bar) {  // in both CTAs
    if constexpr (CG == 2) tc::commit2(bar);
    else tc::commit(bar);
  };
  const auto wait = [&](uint64_t* bar, int use) { return mbar_wait_bounded(bar, use & 1, a.status); };
  // Two or three at once: a wait on a complete barrier is mostly its latency.
  const auto wait2 = [&](uint64_t* p, int up, uint64_t* q, int uq) {
    const bool x = mbar_try_wait(p, up & 1), y = mbar_try_wait(q, uq & 1);
    return (x & y) || (wait(p, up) && wait(q, uq));
  };
  const auto wait3 = [&](uint64_t* p, int up, uint64_t* q, int uq, uint64_t* r, int ur) {
    const bool x = mbar_try_wait(p, up & 1), y = mbar_try_wait(q, uq & 1), z = mbar_try_wait(r, ur & 1);
    return (x & y & z) || (wait(p, up) && wait(q, uq) && wait(r, ur));
  };

  if (warp >= Cfg::NSOFT && warp < Cfg::NSOFT + 4) {
   fewer_registers<Cfg::R_MISC>();
   if (warp == Cfg::NSOFT) {
    // ------------- TMA producer: code and scale tiles of each page ---------------
    int gnext = 0, nk = 0, nv = 0;  // copies issued (lane 0)
    DiffWork w = first;
    int base = 0, stop = 0;
    do {
     const int32_t* table = a.tables + static_cast<int64_t>(rows->row[w.b]) * a.L + w.p_lo;
     const int pair = w.pm >> 1;
     for (int i = 0; i < w.n; ++i) {
      const int j = base + i;
      if ((i & 31) == 0) gnext = (i + lane < w.n) ? table[i + lane] : 0;
      int g = __shfl_sync(0xffffffffu, gnext, i & 31);
      if (lane == 0) {
        if (g < 0 || g >= a.M) {  // never copy from outside the pool
          set_status(a.status, NK_STATUS_PAGE_RANGE);
          g = 0;
        }
        const int y[2] = {static_cast<int>(tile_row(g, 2 * pair, a.H, a.M, a.head_major)),
                          static_cast<int>(tile_row(g, 2 * pair + 1, a.H, a.M, a.head_major))};
        const int rk = j % NRK, rv = j % NRV;
        if (j >= NRK && !wait(&rk_empty[rk], j / NRK - 1)) stop = 1;
        if (!stop) {
          mbar_arrive_expect_tx(&rk_full[rk], KH * (Cfg::KR * Cfg::KCB + 64 * Cfg::KSB));
#pragma unroll
          for (int h = 0; h < KH; ++h) {
            uint8_t* st = sRK + rk * Cfg::RK_STAGE + h * Cfg::RK_HEAD;
            const int yk = y[BOTH ? h : w.pm & 1];
#pragma unroll
            for (int c = 0; c < Cfg::KCB / Cfg::K_RB; ++c)
              tma_load_2d(st + c * 64 * Cfg::K_RB, &tmk, c * Cfg::K_RB, yk + Cfg::KR * rank, &rk_full[rk]);
            if constexpr (Cfg::KSB > 0)
              bulk_load(st + Cfg::RK_CODES, a.ks + static_cast<int64_t>(yk) * Cfg::KSB, 64 * Cfg::KSB, &rk_full[rk]);
          }
          ++nk;
        }
        // BF16 values land where the MMA reads them: their slot is free once it has
        if (!stop && j >= NRV && !wait(Cfg::BF16 ? &v_empty[rv] : &rv_empty[rv], j / NRV - 1)) stop = 1;
        if (!stop) {
          mbar_arrive_expect_tx(&rv_full[rv], Cfg::VH * (64 * Cfg::VCB + 64 * Cfg::VSB));
#pragma unroll
          for (int v = 0; v < Cfg::VH; ++v) {
            uint8_t* st = Cfg::BF16 ? sV + rv * Cfg::V_STAGE + v * Cfg::F16 : sRV + rv * Cfg::RV_STAGE + v * Cfg::RV_HEAD;
            const int yv = y[Cfg::VH == 2 ? v : rank];
#pragma unroll
            for (int c = 0; c < Cfg::VCB / Cfg::V_RB; ++c)
              tma_load_2d(st + c * 64 * Cfg::V_RB, &tmv, c * Cfg::V_RB, yv, &rv_full[rv]);
            if constexpr (Cfg::VSB > 0)
              bulk_load(st + Cfg::RV_CODES, a.vs + static_cast<int64_t>(yv) * Cfg::VSB, 64 * Cfg::VSB, &rv_full[rv]);
          }
          ++nv;
        }
      }
      stop = __shfl_sync(0xffffffffu, stop, 0);
      if (stop) break;
     }
    } while (!stop && next(w, base));
    if (lane == 0) {  // every copy lands before the CTA may leave
      for (int j = max(0, nk - NRK); j < nk; ++j) mbar_wait_bounded(&rk_full[j % NRK], (j / NRK) & 1, a.status);
      for (int j = max(0, nv - NRV); j < nv; ++j) mbar_wait_bounded(&rv_full[j % NRV], (j / NRV) & 1, a.status);
    }
  } else if (warp == Cfg::NSOFT + 3) {
    // ------------- factors: per-key factors of the scores and of the weights -------------
    if constexpr (Cfg::KEY_FAC || Cfg::VAL_FAC) {
      bool ok = true;
      DiffWork w = first;
      int base = 0;
      do {
       const int F = rows->prefix[w.b] + rows->chunk[w.b];
       for (int i = base; i < base + w.n; ++i) {
        const int rk = i % NRK, rv = i % NRV, fs = i % NF, kvalid = F - 64 * (w.p_lo + i - base);
        float* slot = sF + fs * 256;
        if constexpr (Cfg::KEY_FAC && Cfg::VAL_FAC) ok = wait2(&rk_full[rk], i / NRK, &rv_full[rv], i / NRV);
        else if constexpr (Cfg::KEY_FAC) ok = wait(&rk_full[rk], i / NRK);
        else ok = wait(&rv_full[rv], i / NRV);
        if (ok && i >= NF) ok = wait(&f_empty[fs], i / NF - 1);
        ok = __all_sync(0xffffffffu, ok);  // the warp stops as one
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = lane + 32 * (k & 1), h = k >> 1;
          const bool in = key < kvalid;
          if constexpr (Cfg::KEY_FAC)
            if (h < KH)
              slot[64 * h + key] =
                  in ? key_factor<KK, D>(sRK + rk * Cfg::RK_STAGE + h * Cfg::RK_HEAD + Cfg::RK_CODES, key) * a.scale_log2 : 0.f;
          if constexpr (Cfg::VAL_FAC)
            slot[128 + 64 * h + key] =
                in ? key_factor<KV, D>(sRV + rv * Cfg::RV_STAGE + h * Cfg::RV_HEAD + Cfg::RV_CODES, key) : 0.f;
        }
        __syncwarp();
        if (lane == 0) {
          q_arrive(&f_full[fs]);
          if constexpr (Cfg::KEY_FAC) q_arrive(&rk_empty[rk]);
          if constexpr (Cfg::VAL_FAC) q_arrive(&rv_empty[rv]);
        }
       }
      } while (ok && next(w, base));
    }
  } else if (warp == Cfg::NSOFT + 1) {
    // ------------------------------ MMA issuer ---------------------------------
    bool ok = true;
    DiffWork w = first;
    int base = 0, piece = 0;
    do {
     ok = ok && wait(q_ready, piece++);  // and O of the piece before is stored: the same warps, in that order
     for (int i = 0; i < w.n + NS - 1; ++i) {  // S(i), then O += P V of page i - NS + 1
      if (i < w.n) {
        const int j = base + i;
        const int ring = Cfg::K_RAW ? NRK : NK, ks = j % ring, sb = j % NS;
        const uint32_t s_at = tmem + Cfg::COL_S + 64 * sb;
        // the operand, here and in the other CTA; P of the page before in this buffer is read
        // by MMAs issued before
        uint64_t* kb = Cfg::K_RAW ? &rk_full[ks] : &k_full[ks];
        if (CG == 2 && rank == 0) ok = ok && wait2(kb, j / ring, &peer_k[ks], j / ring);
        else ok = ok && wait(kb, j / ring);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc::fence_after();
        if (rank != 0) {  // CTA 0 issues for both
          tc::fence_before();
          if (lane == 0) peer_arrive(&peer_k[ks], 0);
        } else if (elect_one()) {
#pragma unroll
          for (int h = 0; h < KH; ++h) {
            const uint32_t qa = tmem + Cfg::COL_Q + h * (D / 2);
#pragma unroll
            for (int part = 0; part < (Cfg::K_SPLIT || Cfg::K8MMA ? 2 : 1); ++part) {
              const uint8_t* tile = Cfg::K_RAW ? sRK + ks * Cfg::RK_STAGE + h * Cfg::RK_HEAD
                                               : sK + ks * Cfg::K_STAGE + h * Cfg::K_HEAD + part * Cfg::F16;
              const uint64_t kd = tc::smem_desc(smem_u32(tile), 16, 1024);
              if constexpr (Cfg::K8MMA) {  // q_hi, then q_lo, in D / 4 columns each
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_f8(s_at, qa + part * (D / 4) + kk * 8,
                                kd + static_cast<uint64_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), Cfg::ID_S,
                                h > 0 || part > 0 || kk > 0);
              } else {  // INT8-G64: Q k1^T - Q k2'^T
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                  mma(s_at, qa + kk * 8, kd + static_cast<uint64_t>(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4),
                             part > 0 ? tc::idesc_negate_b(Cfg::ID_S) : Cfg::ID_S, h > 0 || part > 0 || kk > 0);
              }
            }
          }
          commit(&s_full[sb]);
          commit(Cfg::K_RAW ? &rk_empty[ks] : &k_empty[ks]);
        }
        __syncwarp();
      }
      if (i >= NS - 1) {
        const int j = base + i - (NS - 1);
        const int vs = j % NV, sb = j % NS;
        if (CG == 2 && rank == 0) ok = ok && wait3(&v_full[vs], j / NV, &p_full[sb], j / NS, &peer_v[sb], j / NS);
        else ok = ok && wait2(&v_full[vs], j / NV, &p_full[sb], j / NS);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc::fence_after();
        if (rank != 0) {
          tc::fence_before();
          if (lane == 0) peer_arrive(&peer_v[sb], 0);
        } else if (elect_one()) {
#pragma unroll
          for (int v = 0; v < (Cfg::VAL_FAC ? 2 : 1); ++v) {
            const uint64_t vd = tc::smem_desc(smem_u32(sV + vs * Cfg::V_STAGE + v * Cfg::VPART), 8192, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma(tmem + Cfg::COL_O + v * D, tmem + Cfg::COL_S + 64 * sb + 32 * (kk >> 1) + 16 * v + 8 * (kk & 1),
                         vd + static_cast<uint64_t>((kk * 2048) >> 4), Cfg::ID_O, (j > base || kk > 0));
          }
          commit(&o_done[sb]);
          commit(&v_empty[vs]);
        }
        __syncwarp();
      }
     }
    } while (__all_sync(0xffffffffu, ok) && next(w, base));
    __syncwarp();
    if (rank == 0 && elect_one()) commit(drain);  // arrives once every MMA issued above has completed
   }
  } else if (warp >= Cfg::NSOFT + 4) {
    fewer_registers<Cfg::R_CONV>();
    const int ct = tid - 32 * (Cfg::NSOFT + 4);
    // Lanes measure the time of a wait each for itself, and the warp stops as one, by a vote at
    // the end of a page: lanes that left alone would be missed at its next collective
    // instruction.  (INT8-G64, with a vote there and without any: 8 x 4 tokens of 32 heads over
    // 32768 140 us and 132, chunk of 2048 behind 8192 363 and 373; the other page types the same.)
    bool ok = true;
    if constexpr (Cfg::BF16) {
      // ------------- converters of BF16 values: a strip of dims per warp -----------
      using St = StripOf<Cfg::STRIP>;
      const int cw = ct >> 5, col = cw * Cfg::STRIP;
      const int blk = (col / D) * Cfg::F16 + (col % D) / 64 * 8192;
      // lane: chunk lane % CH of a key; the keys of eight lanes are apart, so that their
      // swizzled chunks lie in different banks
      const int row0 = St::CH == 4   ? (lane >> 3) + 4 * ((lane >> 2) & 1)
                       : St::CH == 2 ? ((lane >> 3) & 1) + 2 * ((lane >> 1) & 3) + 8 * (lane >> 4)
                                     : lane;
      const int strip = Cfg::NCONV * rank + cw;  // of all that O's dims have
      const int off0 = row0 * 128 + ((((col % 64) / 8 + lane % St::CH) ^ (row0 & 7)) << 4);
      DiffWork w = first;
      int base = 0;
      do {
       const int F = rows->prefix[w.b] + rows->chunk[w.b];
       int k = 0;
       for (int i = 0; ok && i < w.n; ++i) {
        const int j = base + i, vs = j % NV, fs = j % NF, kvalid = F - 64 * (w.p_lo + i);
        ok = j >= NF ? wait2(&rv_full[vs], j / NV, &f_empty[fs], j / NF - 1) : wait(&rv_full[vs], j / NV);
        uint8_t* tile = sV + vs * Cfg::V_STAGE + blk;
        uint4 v[St::UNITS];
#pragma unroll
        for (int u = 0; u < St::UNITS; ++u) v[u] = *reinterpret_cast<const uint4*>(tile + off0 + u * St::ROWS * 128);
        if (kvalid < 64) {  // stale keys are zeros
#pragma unroll
          for (int u = 0; u < St::UNITS; ++u)
            if (row0 + u * St::ROWS >= kvalid) v[u] = make_uint4(0u, 0u, 0u, 0u);
        }
        uint32_t top2 = 0u;  // largest rebiased magnitudes
#pragma unroll
        for (int u = 0; u < St::UNITS; ++u)
          top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(bf16x2_rebias(v[u].x), bf16x2_rebias(v[u].y)),
                                         __vmaxu2(bf16x2_rebias(v[u].z), bf16x2_rebias(v[u].w))));
        const uint32_t mine = max(top2 & 0xFFFFu, top2 >> 16);
        // k stays 0 while the strip's largest value lies in [2^-3, 2^15) (its first
        // page) and below 2^15 (later): no lift to apply.  (2^15 and 2^-3 rebiased.)
        const int was = k;
        const bool plain = k == 0 && !__any_sync(0xffffffffu, mine >= 0x0F00u) &&
                           (i > 0 || __any_sync(0xffffffffu, mine >= 0x0600u));
        if (plain) {
#pragma unroll
          for (int u = 0; u < St::UNITS; ++u)
            *reinterpret_cast<uint4*>(tile + off0 + u * St::ROWS * 128) =
                make_uint4(f16x2_of(bf16x2_rebias(v[u].x), v[u].x), f16x2_of(bf16x2_rebias(v[u].y), v[u].y),
                           f16x2_of(bf16x2_rebias(v[u].z), v[u].z), f16x2_of(bf16x2_rebias(v[u].w), v[u].w));
        } else {
          uint32_t raw2 = 0u;  // of the finite values: an infinity or a NaN leaves its neighbours' k alone
#pragma unroll
          for (int u = 0; u < St::UNITS; ++u)
            raw2 = __vmaxu2(raw2, __vmaxu2(__vmaxu2(bf16x2_finite(v[u].x), bf16x2_finite(v[u].y)),
                                           __vmaxu2(bf16x2_finite(v[u].z), bf16x2_finite(v[u].w))));
          const uint32_t most = __reduce_max_sync(0xffffffffu, max(raw2 & 0xFFFFu, raw2 >> 16));
          const int e = static_cast<int>(most >> 7) - 127;
          if (i == 0) k = strip_lift(most);
          else if (most && e + k >= 15) k = min(k, strip_lift(most));
          const float f = pow2i(k);
#pragma unroll
          for (int u = 0; u < St::UNITS; ++u)
            *reinterpret_cast<uint4*>(tile + off0 + u * St::ROWS * 128) =
                make_uint4(bf16x2_lift(v[u].x, f), bf16x2_lift(v[u].y, f), bf16x2_lift(v[u].z, f), bf16x2_lift(v[u].w, f));
        }
        if (lane == 0) {
          // of a strip: whether its k fell, O's factor for that, 2^-k.  O of the pair's other
          // CTA has these dims too.
          float4* slot = reinterpret_cast<float4*>(sF + fs * 256);
          const float4 x = make_float4(i > 0 && k != was ? 1.f : 0.f, pow2i(i > 0 ? max(k - was, -126) : 0), pow2i(-k), 0.f);
          slot[strip] = x;
          if constexpr (CG == 2)
            if (ok) peer_store(slot + strip, x, &f_full[fs], rank ^ 1);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (ok && lane == 0) {
          if (CG == 2 && cw == 0) mbar_arrive_expect_tx(&f_full[fs], 16 * Cfg::NCONV);  // and the other CTA's strips
          else q_arrive(&f_full[fs]);
          q_arrive(&v_full[vs]);
        }
        ok = __all_sync(0xffffffffu, ok);
       }
      } while (ok && next(w, base));
    } else {
      // ------------- converters: K(i), V(i) of the group's pages i -------------------
      constexpr int NCG = Cfg::NCG, NCT = 32 * Cfg::CGW;
      const int cg = ct / NCT, gt = ct % NCT;
      DiffWork w = first;
      int base = 0;
      do {
       const int F = rows->prefix[w.b] + rows->chunk[w.b];
       for (int i = base + (base + cg) % NCG; ok && i < base + w.n; i += NCG) {  // pages i = cg mod NCG
        const int kvalid = F - 64 * (w.p_lo + i - base);
        if constexpr (!Cfg::K_RAW) {
          const int rk = i % NRK, ks = i % NK;
          ok = i >= NK ? wait2(&rk_full[rk], i / NRK, &k_empty[ks], i / NK - 1) : wait(&rk_full[rk], i / NRK);
          if (ok) {
#pragma unroll
            for (int h = 0; h < KH; ++h)
              convert_tile<KK, D, Cfg::K_RB, NCT, Cfg::K_SPLIT, Cfg::KR>(
                  sRK + rk * Cfg::RK_STAGE + h * Cfg::RK_HEAD, Cfg::RK_CODES + Cfg::KR * rank * Cfg::KSB,
                  sK + ks * Cfg::K_STAGE + h * Cfg::K_HEAD, gt, kvalid - Cfg::KR * rank);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (ok && lane == 0) {
            q_arrive(&rk_empty[rk]);
            q_arrive(&k_full[ks]);
          }
        }
        const int rv = i % NRV, vs = i % NV;
        ok = ok && (i >= NV ? wait2(&rv_full[rv], i / NRV, &v_empty[vs], i / NV - 1) : wait(&rv_full[rv], i / NRV));
        if (ok) {
#pragma unroll
          for (int v = 0; v < Cfg::VH; ++v)
            convert_tile<KV, D, Cfg::V_RB, NCT, false, 64, Cfg::V_HALF ? 4 : D / 16>(
                sRV + rv * Cfg::RV_STAGE + v * Cfg::RV_HEAD, Cfg::RV_CODES, sV + vs * Cfg::V_STAGE + v * Cfg::VPART, gt,
                kvalid, Cfg::V_HALF ? 4 * rank : 0);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        if (ok && lane == 0) {
          q_arrive(&rv_empty[rv]);
          q_arrive(&v_full[vs]);
        }
        ok = __all_sync(0xffffffffu, ok);
       }
      } while (ok && next(w, base));
    }
  } else {
    // ------------------------------ softmax warps -----------------------------
    more_registers<Cfg::R_SOFT>();
    const int half = warp >> 2, quad32 = warp & 3, m = tid & 127;  // query row = TMEM lane; pages half, half + 2, ..
    const int r = BOTH ? m & 63 : m, tl = r / a.G, g = r % a.G;
    bool live = true;
    DiffWork w = first;
    int base = 0;
    do {
    const int n = w.n, map = BOTH ? m >> 6 : w.pm & 1, pair = w.pm >> 1, token = (w.qt * CG + rank) * a.TQ + tl;
    const bool valid = (BOTH || tl < a.TQ) && token < rows->chunk[w.b];
    const int pos = rows->prefix[w.b] + token;  // keys <= pos are visible
    const uint32_t quad = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float rs = 1.f;  // 2^-e of this query row
    {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + ((static_cast<int64_t>(w.b) * a.T + token) * a.Hq + 2 * (pair * a.G + g) + map) * D);
      const uint32_t flip = a.negate ? 0x80008000u : 0u;
      float qf = 1.f;
      if constexpr (!Cfg::BF16) {
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
        qf = ldexpf(1.f, e);
        rs = ldexpf(1.f, -e);
      }
      // this half's dims [half D / 2, +D / 2), 32 at a time; BOTH: zeros in the other map's operand
      const uint32_t q_at = quad + Cfg::COL_Q + (BOTH ? map * (D / 2) : 0);
      const uint32_t z_at = quad + Cfg::COL_Q + (map ^ 1) * (D / 2);
      const uint32_t zero[16] = {};
#pragma unroll
      for (int d0 = half * (D / 2); d0 < (half + 1) * (D / 2); d0 += (Cfg::K8MMA ? 64 : 32)) {
        if constexpr (Cfg::K8MMA) {  // q' = hi + lo in E4M3, as in qprefill.cu
          uint32_t hv[16], lv[16];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 x = valid ? src[d0 / 8 + u] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t xw[4] = {x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip};
            uint32_t hp[4], lp[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x0 = __uint_as_float(xw[k] << 16) * qf, x1 = __uint_as_float(xw[k] & 0xFFFF0000u) * qf;
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
          tc::st16(q_at + d0 / 4, hv);
          tc::st16(q_at + D / 4 + d0 / 4, lv);
          if constexpr (BOTH) {
            tc::st16(z_at + d0 / 4, zero);
            tc::st16(z_at + D / 4 + d0 / 4, zero);
          }
        } else {
          uint32_t qv[16];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 x = valid ? src[d0 / 8 + u] : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t xw[4] = {x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip};
#pragma unroll
            for (int k = 0; k < 4; ++k) qv[4 * u + k] = Cfg::BF16 ? xw[k] : bf16x2_lift(xw[k], qf);
          }
          tc::st16(q_at + d0 / 2, qv);
          if constexpr (BOTH) tc::st16(z_at + d0 / 2, zero);
        }
      }
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) q_arrive(q_ready);
    }
    // what turns a raw score into one in base 2: per key and row, or for all keys
    const float c_row = Cfg::KEY_FAC ? rs : fmaxf(a.scale_log2 * rs, 1.17549435e-38f);
    const F2 c2 = pack2(c_row, c_row);
    // of this warp's pages: sum, and the reference and lift of the weights that it carries
    // (without factors per key the reference itself lies kDiffWeightLift below the largest score)
    constexpr int kLift0 = Cfg::VAL_FAC ? kVLiftInit : 0;
    float l = 0.f, m_own = -INFINITY;
    int k_own = kLift0;
    float mu = 0.f;
    // Scores of 32 keys of the page: factors and mask.
    const auto finish = [&](uint32_t (&sv)[32], const float* ksc, int kmax) {
      if constexpr (Cfg::KEY_FAC) {
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(ksc + c);
          float x[4];
          unpack2(mul2(pack2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), pack2(k4.x, k4.y)), x[0], x[1]);
          unpack2(mul2(pack2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), pack2(k4.z, k4.w)), x[2], x[3]);
#pragma unroll
          for (int u = 0; u < 4; ++u) sv[c + u] = __float_as_uint(x[u]);
        }
      }
      if (!__all_sync(0xffffffffu, kmax >= 31)) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c > kmax) sv[c] = 0xFF800000u;  // -inf
      }
    };
    const auto top_of = [](const uint32_t (&sv)[32]) {
      float t4[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) t4[u] = fmaxf(__uint_as_float(sv[u]), __uint_as_float(sv[4 + u]));
#pragma unroll
      for (int c = 8; c < 32; c += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u) t4[u] = max3(t4[u], __uint_as_float(sv[c + u]), __uint_as_float(sv[c + 4 + u]));
      return fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
    };
    // The weights of 32 scores under the reference mu, to P's columns; returns their sum.
    const auto weights = [&](uint32_t (&sv)[32], const float* vsc, uint32_t p_at) {
      const F2 mu2 = pack2(-mu, -mu);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float x, y;
        unpack2(fma2(pack2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), c2, mu2), x, y);
        sv[c] = __float_as_uint(x);
        sv[c + 1] = __float_as_uint(y);
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) sv[c] = __float_as_uint(ex2(__uint_as_float(sv[c])));
      uint32_t pk[16];
#pragma unroll
      for (int v = 0; v < (Cfg::VAL_FAC ? 2 : 1); ++v) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          if constexpr (Cfg::VAL_FAC) {
            const float2 f = *reinterpret_cast<const float2*>(vsc + 64 * v + c);
            float x, y;
            unpack2(mul2(pack2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), pack2(f.x, f.y)), x, y);
            pk[c / 2] = pack_f16x2(x, y);
          } else {
            pk[c / 2] = pack_f16x2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
          }
        }
        tc::st16(p_at + 16 * v, pk);
      }
      F2 sum2[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) sum2[u] = pack2(__uint_as_float(sv[2 * u]), __uint_as_float(sv[2 * u + 1]));
#pragma unroll
      for (int c = 8; c < 32; c += 2)
        sum2[(c >> 1) & 3] = add2(sum2[(c >> 1) & 3], pack2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])));
      float s0, s1;
      unpack2(add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3])), s0, s1);
      return s0 + s1;
    };
    const bool any = __any_sync(0xffffffffu, valid);
    const int from = base + (base + half) % 2;  // this warp's first page
    if (!any)  // rows past the last query: P is whatever the buffers hold, and their O is not stored
      for (int j = from; live && j < base + n; j += 2) {
        live = wait(&s_full[j % NS], j / NS);
        if constexpr (Cfg::HAS_F) live = live && wait(&f_full[j % NF], j / NF);
        tc::fence_after();
        tc::fence_before();
        if (lane == 0) {
          q_arrive(&x_full[4 * (j & 1) + quad32]);
          q_arrive(&p_full[j % NS]);
          if constexpr (Cfg::HAS_F) q_arrive(&f_empty[j % NF]);
          if constexpr (Cfg::BF16 && CG == 2) peer_arrive(&f_empty[j % NF], rank ^ 1);
        }
      }
    for (int j = from; any && j < base + n; j += 2) {
      const int sb = j % NS, fs = j % NF;
      const uint32_t s_at = quad + Cfg::COL_S + 64 * sb;
      const float* ksc = sF + fs * 256 + (BOTH ? 64 * map : 0);
      const float* vsc = sF + fs * 256 + 128;
      const int kmax = valid ? pos - 64 * (w.p_lo + j - base) : -1;
      bool strips = false;  // BF16 values: a strip's k fell
      float most = 0.f;     // the largest value factor of the page
      // the scores, their factors, and the reference after the page before
      uint64_t* xb = &x_full[4 * ((j - 1) & 1) + quad32];
      if (j > base) {
        if constexpr (Cfg::HAS_F) live = live && wait3(&f_full[fs], j / NF, &s_full[sb], j / NS, xb, (j - 1) >> 1);
        else live = live && wait2(&s_full[sb], j / NS, xb, (j - 1) >> 1);
      } else {
        if constexpr (Cfg::HAS_F) live = live && wait2(&f_full[fs], j / NF, &s_full[sb], j / NS);
        else live = live && wait(&s_full[sb], j / NS);
      }
      if constexpr (Cfg::BF16) strips = lane < Cfg::STRIPS && sF[fs * 256 + 4 * lane] != 0.f;  // any lane's, below
      if constexpr (Cfg::VAL_FAC) {
        const float4 s4 = *reinterpret_cast<const float4*>(sF + fs * 256 + 128 + 4 * lane);  // both heads' 128 scales
        most = fmaxf(fmaxf(s4.x, s4.y), fmaxf(s4.z, s4.w));
      }
      tc::fence_after();
      uint32_t sv[2][32];
      tc::ld32(s_at, sv[0]);
      tc::ld32(s_at + 32, sv[1]);
      tc::wait_ldn(sv[0]);
      tc::wait_ldn(sv[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) finish(sv[h], ksc + 32 * h, kmax - 32 * h);
      const float top = fmaxf(top_of(sv[0]), top_of(sv[1]));
      // the reference and lift after the page before, from the warp of the other pages
      float m_was = -INFINITY;
      int k_was = kLift0, k_now = kLift0;
      if (j > base) {
        const float2 x = sX[((j - 1) & 1) * 128 + m];
        m_was = x.x;
        if constexpr (Cfg::VAL_FAC) k_was = __float_as_int(x.y);
      }
      if constexpr (Cfg::VAL_FAC) k_now = v_lift(__reduce_max_sync(0xffffffffu, __float_as_uint(most)), k_was);
      const float rmax = top == -INFINITY ? -INFINITY : fmaf(top, c_row, Cfg::VAL_FAC ? 0.f : -static_cast<float>(kDiffWeightLift));
      // lazy: the reference moves when a score passes it by more than 2^8, or the lift drops
      const float m_new = fmaxf(m_was, rmax);
      const bool resc = m_new != -INFINITY && (m_was == -INFINITY || m_new > m_was + kLazyThr || k_now != k_was);
      const float m_now = resc ? m_new : m_was;
      sX[(j & 1) * 128 + m] = make_float2(m_now, __int_as_float(k_now));
      __syncwarp();
      if (lane == 0) q_arrive(&x_full[4 * (j & 1) + quad32]);
      if (m_now != m_own || k_now != k_own) {
        l *= m_own == -INFINITY ? 0.f : ex2((m_own - m_now) + static_cast<float>(k_now - k_own));
        m_own = m_now;
        k_own = k_now;
      }
      mu = m_now == -INFINITY ? 0.f : m_now - static_cast<float>(k_now);
#pragma unroll
      for (int h = 0; h < 2; ++h) l += weights(sv[h], vsc + 32 * h, s_at + 32 * h);
      if (j > base && __any_sync(0xffffffffu, resc || strips || k_now != k_was)) {
        // O, once PV(j - 1) is complete
        const float factor = !resc ? 1.f : m_was == -INFINITY ? 0.f : ex2((m_was - m_now) + static_cast<float>(k_now - k_was));
        live = live && wait(&o_done[(j - 1) % NS], (j - 1) / NS);
        tc::fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < 2 * D; c0 += 16) {
          uint32_t ov[16];
          tc::ld16(quad + Cfg::COL_O + c0, ov);
          tc::wait_ld();
#pragma unroll
          for (int c8 = 0; c8 < 16; c8 += 8) {
            const float fc = Cfg::BF16 ? factor * sF[fs * 256 + 4 * ((c0 + c8) / Cfg::STRIP) + 1] : factor;
#pragma unroll
            for (int c = c8; c < c8 + 8; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * fc);
          }
          tc::st16(quad + Cfg::COL_O + c0, ov);
        }
      }
      if constexpr (Cfg::BF16)  // the strips' lifts that the piece ends with
        if (j == base + n - 1 && lane < Cfg::STRIPS) sDown[16 * quad32 + lane] = sF[fs * 256 + 4 * lane + 2];
      tc::wait_st();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) {
        q_arrive(&p_full[sb]);
        if constexpr (Cfg::HAS_F) q_arrive(&f_empty[fs]);  // this warp is done with the page's factors
        if constexpr (Cfg::BF16 && CG == 2) peer_arrive(&f_empty[fs], rank ^ 1);
      }
    }
    // ---- the piece's partial: (m, l) of the row, and O, the half's D dims -------------
    if (n > 0) live = live && wait(&o_done[(base + n - 1) % NS], (base + n - 1) / NS);  // every PV
    tc::fence_after();
    const float m_eff = m_own == -INFINITY ? -INFINITY : m_own - static_cast<float>(k_own);
    sX[256 + 128 * half + m] = make_float2(m_eff, l);
    // the two warps of these rows, which meet here once a piece: both go on to the next or neither
    live = barrier_and(1 + quad32, 64, live);
    const int64_t part = BOTH ? static_cast<int64_t>(pair) * a.ctas + blockIdx.x
                              : ((static_cast<int64_t>(w.b) * a.H + w.pm) * a.tiles + w.qt + blockIdx.x / CG) * CG + rank;
    if (live && valid && half == 0) {  // the sums, under the reference after the last page
      const int last_half = n > 0 ? (base + n - 1) & 1 : 0;
      const float2 last = sX[256 + 128 * last_half + m], other = sX[256 + 128 * (last_half ^ 1) + m];
      const float f = other.x == -INFINITY ? 0.f : ex2(other.x - last.x);
      a.ws_ml[part * 128 + m] = make_float2(last.x, fmaf(other.y, f, last.y));
    }
    if (live && n > 0 && any) {
      float4* dst = reinterpret_cast<float4*>(a.ws_o) + part * (D / 2) * 128 + m;
#pragma unroll 1
      for (int c0 = half * D; c0 < (half + 1) * D; c0 += 32) {
        uint32_t v[32];
        tc::ld32(quad + Cfg::COL_O + c0, v);
        tc::wait_ldn(v);
        if constexpr (Cfg::BF16) {
#pragma unroll
          for (int c8 = 0; c8 < 32; c8 += 8) {
            const float f = sDown[16 * quad32 + (c0 + c8) / Cfg::STRIP];
#pragma unroll
            for (int c = c8; c < c8 + 8; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * f);
          }
        }
        if (valid) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            dst[(c0 / 4 + c) * 128] = make_float4(__uint_as_float(v[4 * c]), __uint_as_float(v[4 * c + 1]),
                                                  __uint_as_float(v[4 * c + 2]), __uint_as_float(v[4 * c + 3]));
        }
      }
    }
    tc::fence_before();
    } while (live && next(w, base));
    if (CG == 2 && live && tid == 0) {  // the last commits that nobody else waits for have arrived
      constexpr int ring = Cfg::K_RAW ? NRK : NK;
      const int j = base - 1;
      wait(&v_empty[j % NV], j / NV);
      wait(Cfg::K_RAW ? &rk_empty[j % ring] : &k_empty[j % ring], j / ring);
    }
  }

  // ---- teardown: every issued MMA has completed before TMEM is freed ---------
  if (tid == 0) mbar_wait_bounded(drain, 0, a.status, 200000000ull);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if constexpr (CG == 2) {  // neither CTA leaves while the other may reach into it
    cluster_sync();
    if (warp == 0) tc::dealloc2(tmem, 512);
  } else {
    if (warp == 0) tc::dealloc(tmem, 512);
  }
}

template <int KK, int KV, int D, bool BOTH>
cudaError_t launch_diff_tile(const nk_pool* p, int layer, const DiffTileArgs& a, dim3 grid, cudaStream_t s) {
  using Cfg = DiffTileCfg<KK, KV, D, BOTH>;
  auto k = diff_tile_kernel<KK, KV, D, BOTH>;
  static std::atomic<uint64_t> granted{0};
  const cudaError_t e = grant_smem(granted, k, Cfg::SMEM);
  if (e != cudaSuccess) return e;
  if constexpr (Cfg::CG == 2)
    return launch_pdl_cluster(k, grid, dim3(Cfg::THREADS), Cfg::SMEM, s, 2, p->tmap_half[layer], p->tmap[layer * 2 + 1], a);
  else
    return launch_pdl(k, grid, dim3(Cfg::THREADS), Cfg::SMEM, s, p->tmap[layer * 2 + 0], p->tmap[layer * 2 + 1], a);
}

template <int KK, int KV>
cudaError_t diff_tile_dispatch(const nk_pool* p, int layer, const DiffTileArgs& a, bool both, dim3 grid, cudaStream_t s) {
  if (p->desc.head_dim == 64)
    return both ? launch_diff_tile<KK, KV, 64, true>(p, layer, a, grid, s)
                : launch_diff_tile<KK, KV, 64, false>(p, layer, a, grid, s);
  return both ? launch_diff_tile<KK, KV, 128, true>(p, layer, a, grid, s)
              : launch_diff_tile<KK, KV, 128, false>(p, layer, a, grid, s);
}

using DiffTileFn = cudaError_t (*)(const nk_pool*, int layer, const DiffTileArgs&, bool both, dim3 grid, cudaStream_t);
cudaError_t diff_tile_bf16(const nk_pool*, int, const DiffTileArgs&, bool, dim3, cudaStream_t);
cudaError_t diff_tile_int8(const nk_pool*, int, const DiffTileArgs&, bool, dim3, cudaStream_t);
cudaError_t diff_tile_fp8(const nk_pool*, int, const DiffTileArgs&, bool, dim3, cudaStream_t);
cudaError_t diff_tile_nvfp4(const nk_pool*, int, const DiffTileArgs&, bool, dim3, cudaStream_t);
cudaError_t diff_tile_k8v4(const nk_pool*, int, const DiffTileArgs&, bool, dim3, cudaStream_t);

// The instantiations of a profile, and the arguments that every call shares.
inline DiffTileFn diff_tile_for(int profile) {
  switch (profile) {
    case NK_BF16: return diff_tile_bf16;
    case NK_INT8_G64: return diff_tile_int8;
    case NK_FP8_E4M3_ROW: return diff_tile_fp8;
    case NK_NVFP4_G16: return diff_tile_nvfp4;
    default: return diff_tile_k8v4;
  }
}

inline DiffTileArgs diff_tile_args(const nk_pool* pool, int layer, const void* q, int Hq, const int32_t* tables,
                                   const int32_t* table_rows, const int32_t* lengths, int B, int T, float softmax_scale,
                                   void* ws, size_t ml_bytes) {
  DiffTileArgs a = {};
  const int np = pool->n_planes;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tables = tables;
  a.table_rows = table_rows;
  a.lengths = lengths;
  a.ks = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 2]) : nullptr;
  a.vs = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 3]) : nullptr;
  a.ws_ml = static_cast<float2*>(ws);
  a.ws_o = reinterpret_cast<float*>(static_cast<char*>(ws) + ml_bytes);
  a.status = pool->status;
  // masked scores are -inf times the scale: 0 becomes the least normal number,
  // which no finite score makes visible
  a.scale_log2 = fmaxf(fabsf(softmax_scale) * kDiffLog2e, 1.17549435e-38f);
  a.negate = softmax_scale < 0.f;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.H = pool->desc.num_kv_heads;
  a.G = Hq / a.H;
  a.L = pool->L;
  a.M = pool->M;
  a.C = pool->desc.max_concurrency;
  a.head_major = pool->desc.order == NK_HEAD_MAJOR;
  return a;
}

}  // namespace nk
