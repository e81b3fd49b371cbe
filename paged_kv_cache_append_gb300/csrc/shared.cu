// shared.cu -- decode / verify attention of a batch whose rows share a long
// prefix of pages: the prefix is attended once for all rows.
//
// softmax(q K^T) V over a row's keys is the log-sum-exp merge of the same over
// any partition of them.  Here the partition is the shared pages and the row's
// own:
//   prefix pass  the B T G query rows that read one KV head, of all rows of
//                the batch, are the rows of 128-row tensor-core tiles
//                (prefix.cu); the shared pages are cut into ranges, and every
//                range leaves a partial (m, l, O) for all query rows;
//   own pages    the decode kernels (decode.cuh, vdecode.cu) on each row's
//                pages behind the prefix, as partials too, after the prefix
//                pass or next to it (share_split, shared.cuh);
//   merge        M = max m, out = sum 2^(m - M) O / sum 2^(m - M) l, below.
// The shared pages cross HBM once per call instead of once per row.
#include <algorithm>
#include <cmath>

#include "decode.cuh"

namespace nk {

cudaError_t prefix_pass(const nk_pool* p, int layer, const void* q, const int32_t* tables, const int32_t* table_rows,
                        int Hq, float scale_log2, const PrefixParts& parts, const SharedPrefix& sh, cudaStream_t s);

constexpr int kMaxPrefixSplits = 128;

struct SharedPlan {
  DecodePlan own;  // the rows' own pages
  int tiles, nsplit;
  size_t sh_ml_bytes, sh_bytes, ws_bytes;
};

static int make_shared_plan(const nk_pool* p, int B, int T, int Hq, SharedPlan* pl) {
  int rc = make_plan(p, B, T, Hq, &pl->own);
  if (rc) return rc;
  const int H = p->desc.num_kv_heads, D = p->desc.head_dim, G = Hq / H;
  pl->tiles = (B * T * G + 127) / 128;
  // one CTA per SM; at head_dim 64 and 128 one CTA takes both tiles of a head
  const int fit = p->num_sms / (H * (D == 256 ? pl->tiles : 1));
  pl->nsplit = fit < 1 ? 1 : fit > kMaxPrefixSplits ? kMaxPrefixSplits : fit;
  const size_t parts = static_cast<size_t>(H) * pl->tiles * pl->nsplit * 128;
  pl->sh_ml_bytes = parts * sizeof(float2);
  pl->sh_bytes = pl->sh_ml_bytes + parts * D * sizeof(float);
  pl->ws_bytes = pl->sh_bytes + pl->own.ws_bytes;
  return NK_OK;
}

// Measured times of one page of a KV head on one SM, in us: a row's own decode
// of it, from L2 and (`cold`) from HBM, and the prefix pass's for its rows.
struct PageCosts {
  float own, own_cold, prefix;
  bool tensor;  // the tensor-core decode
};

static PageCosts page_costs(const nk_pool* p, int B, int R, int64_t page_bytes) {
  const int D = p->desc.head_dim;
  const float d = D == 64 ? 0.75f : D == 128 ? 1.f : 2.2f;
  PageCosts c;
  c.tensor = R > 16 && p->desc.profile != NK_BF16 && p->desc.profile != NK_INT8_G64;
  c.own = d * (R <= 8 ? 0.3f : R <= 16 ? 0.56f : c.tensor ? 0.68f : 0.85f);
  c.own_cold = fmaxf(D / 128.f * (R <= 8 ? 0.28f : R <= 16 ? 0.56f : c.tensor ? 0.72f : 1.35f), page_bytes / 40e3f);
  c.prefix = D == 256 ? 1.25f * ((B * R + 127) / 128) : B * R > 128 ? 1.3f : D == 64 ? 1.25f : 0.95f;
  if (p->desc.profile == NK_INT8_G64) c.prefix += 0.6f;  // two key tiles a page
  return c;
}

// When the prefix gets a pass of its own: where its pages cost the pass less than
// the rows by as much as its launch, its partials and their merge cost, about
// 4.5 us of the chip, or 1 over 16 query rows, where the plain decode has more of
// a start itself.  Crossings seen, in shared pages: 8 rows of FP8-row, BF16 at 2
// heads of 256: 90, 85; 4 rows of FP8-row there 120; 8 rows of K8V4, BF16 at 4
// heads of 128: 130, 150, and less than 16 for their 4-token verify; 8 rows at 8
// heads of 64: 195; 2 rows, and 3 of 2 query heads a KV head: never.
static int64_t share_least(const nk_pool* p, int B, int R, const PageCosts& c) {
  const float gain = p->desc.num_kv_heads * (B * c.own - c.prefix);
  return gain <= 0.f ? INT32_MAX : static_cast<int64_t>(p->num_sms * (R > 16 ? 1.f : 4.5f) / gain) + 1;
}

// The own-pages kernel without pages takes 3 to 10 us, behind the prefix pass up
// to 17 on the tensor cores (share_split).
static ShareShape share_shape(const nk_pool* p, const SharedPlan& pl, int B, int R, const PageCosts& c) {
  const int H = p->desc.num_kv_heads, D = p->desc.head_dim;
  ShareShape g;
  g.sms = p->num_sms;
  g.range_ctas = H * (D == 256 ? pl.tiles : 1);
  g.nsplit = pl.nsplit;
  g.ctas = pl.own.ctas;
  g.least = (B * H + pl.own.per_sm - 1) / pl.own.per_sm;
  g.step = static_cast<float>(B * H) / pl.own.per_sm;
  g.all_sms = fmaxf(floorf(p->num_sms / g.step), 1.f) * g.step;
  g.ranges_per_sm = 1.f / g.range_ctas;
  g.ctas_per_sm = static_cast<float>(pl.own.per_sm) / H;
  g.own_page = H * c.own_cold / 1.25f;
  g.own_start = c.tensor ? 8.f : (R <= 8 ? 4.f : R <= 16 ? 6.f : 8.f) * D / 128;
  g.turn_start = !c.tensor ? g.own_start : D == 256 ? 10.f : 14.f;
  return g;
}

struct SharedMergeArgs {
  DecodeArgs d;
  PrefixParts prefix;
};

constexpr int kMergeRows = 4;  // query rows of one merge CTA

// One CTA per (row, KV head, 4 query rows, 32 dims): the row's own splits
// followed by the prefix's, at most kMaxSplits + kMaxPrefixSplits partials a
// query row.  The plan (before the wait) overlaps the kernels before.  Bound by
// the latency of three dependent reads and, for many partials, by L2: the
// accumulators are read as whole 128-byte lines, eight loads of a thread in
// flight, the first eight before the weights are known.
template <int D, int SUB>
__global__ void __launch_bounds__(kMergeRows * 8 * SUB) shared_merge_kernel(const __grid_constant__ SharedMergeArgs m) {
  const DecodeArgs& a = m.d;
  constexpr int S_MAX = kMaxSplits + kMaxPrefixSplits, U = 8, THREADS = kMergeRows * 8 * SUB;
  __shared__ int s_F[8];
  __shared__ int s_row[8];
  __shared__ float s_w[kMergeRows * S_MAX];  // weights; -1: a partial without keys, which has no accumulators
  const int b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int d0 = (blockIdx.z % (D / 32)) * 32, q0 = (blockIdx.z / (D / 32)) * kMergeRows;
  const int warp = tid >> 5, lane = tid & 31;
  const int pages = *a.shared;
  if (tid < a.B) {
    const int F = a.frontiers[tid], row = a.table_rows[tid];
    const bool ok = F >= 0 && F <= a.L * 64 && row >= 0 && row < a.C;
    const int before = pages_before(a, F, row);
    s_F[tid] = ok ? F - 64 * before : 0;
    s_row[tid] = before > 0 ? row : -1;
  }
  __syncthreads();
  int total = 0, maxp = 0, first = -1;
  for (int bb = a.B - 1; bb >= 0; --bb) {
    const int np = (s_F[bb] + 63) >> 6;
    total += np;
    maxp = max(maxp, np);
    if (s_row[bb] >= 0) first = s_row[bb];
  }
  const ShareSplit split = share_split(a.shape, first >= 0 ? pages : 0, total);
  const int chunk = own_chunk(s_F, a, total, maxp, split.ctas);
  const int own = max(1, (((s_F[b] + 63) >> 6) + chunk - 1) / chunk);
  const bool part = s_row[b] >= 0;
  const int per = part ? (pages + split.nsplit - 1) / split.nsplit : 1;
  const int pre = part ? (pages + per - 1) / per : 0;
  if (h == 0 && blockIdx.z == 0) {  // the row's leading table entries are those the prefix pass read
    if (part && s_row[b] != first) {
      const int32_t* mine = a.tables + static_cast<int64_t>(s_row[b]) * a.L;
      const int32_t* read = a.tables + static_cast<int64_t>(first) * a.L;
      for (int i = tid; i < pages; i += THREADS)
        if (mine[i] != read[i]) set_status(a.status, NK_STATUS_PREFIX);
    }
  }
  const int R_all = a.T * a.G;
  const int R = R_all <= 8 ? 8 : R_all <= 16 ? 16 : 32;  // rows of an own partial's slot
  const int R_real = min(kMergeRows, R_all - q0);
  const int64_t own0 = (static_cast<int64_t>(b) * a.H + h) * a.target;  // the row's first own slot
  // slot of query row q0 + r in the first prefix partial of its tile; the next
  // partial is 128 slots on
  auto prefix0 = [&](int r) {
    const int flat = b * R_all + q0 + r;
    return (static_cast<int64_t>(h) * m.prefix.tiles + flat / 128) * m.prefix.nsplit * 128 + flat % 128;
  };
  griddep_wait();
  griddep_launch_dependents();

  // thread = (query row r, 4 dims, every SUB-th partial from `sub` on)
  const int sub = tid % SUB, r = tid / (8 * SUB), d = d0 + (tid / SUB % 8) * 4;
  const bool live = r < R_real;
  const int splits = own + pre;
  const float* own_o = a.ws_acc + (own0 * R + q0 + r) * D + d;
  const float* pre_o = m.prefix.o + (live ? prefix0(r) : 0) * D + d;
  auto acc_at = [&](int k) {
    const float* p = k < own ? own_o + static_cast<int64_t>(k) * R * D : pre_o + static_cast<int64_t>(k - own) * 128 * D;
    return __ldcg(reinterpret_cast<const float4*>(p));
  };
  float4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = live && sub + SUB * u < splits ? acc_at(sub + SUB * u) : make_float4(0.f, 0.f, 0.f, 0.f);

  for (int wr = warp; wr < R_real; wr += THREADS / 32) {  // the weights of query row q0 + wr, lanes over its partials
    const float2* own_ml = a.ws_ml + own0 * R + q0 + wr;
    const float2* pre_ml = m.prefix.ml + prefix0(wr);
    constexpr int N = S_MAX / 32;
    float2 w[N];
    float M = -INFINITY;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = lane + 32 * u;
      w[u] = k >= splits ? make_float2(-INFINITY, 0.f) : __ldcg(k < own ? own_ml + k * R : pre_ml + (k - own) * 128);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) M = fmaxf(M, w[u].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
#pragma unroll
    for (int u = 0; u < N; ++u) {  // (a NaN sum goes on into L and from there into every weight)
      w[u].x = w[u].y == 0.f ? -1.f : ex2(w[u].x - M);
      L += w[u].y == 0.f ? 0.f : w[u].y * w[u].x;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    const float inv = 1.f / L;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = lane + 32 * u;
      if (k < splits) s_w[wr * S_MAX + k] = w[u].x == -1.f ? -1.f : w[u].x * inv;
    }
    if (lane == 0 && a.lse && d0 == 0) {
      const int qr = q0 + wr;
      a.lse[(static_cast<int64_t>(b) * a.T + qr / a.G) * a.Hq + h * a.G + qr % a.G] =
          L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = sub; k0 < splits; k0 += SUB * U) {
    float4 nx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + SUB * (U + u);
      nx[u] = live && k < splits ? acc_at(k) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + SUB * u;
      const float w = live && k < splits ? s_w[r * S_MAX + k] : -1.f;
      if (w != -1.f) {
        acc.x = fmaf(w, v[u].x, acc.x);
        acc.y = fmaf(w, v[u].y, acc.y);
        acc.z = fmaf(w, v[u].z, acc.z);
        acc.w = fmaf(w, v[u].w, acc.w);
      }
      v[u] = nx[u];
    }
  }
#pragma unroll
  for (int off = 1; off < SUB; off <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
  }
  if (sub == 0 && live) {
    const int qr = q0 + r;
    __nv_bfloat16* dst = a.out + ((static_cast<int64_t>(b) * a.T + qr / a.G) * a.Hq + h * a.G + qr % a.G) * D + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  }
}

// SUB threads share 4 dims of a query row.  Over 16 query rows a row, with four
// times the CTAs, 2 take less than 4 (116 against 120 us for the 4-token verify
// of 8 rows); below, 8 take less than 4 (35.0 against 37.2 us for one token of 8
// rows; CTAs of 8 query rows 35.9 either way, 4 or 14 loads of a thread in
// flight 40.3 and 37.9; the two attention kernels in turn).
template <int SUB>
static cudaError_t launch_merge(int D, dim3 grid, cudaStream_t s, const SharedMergeArgs& m) {
  const dim3 block(kMergeRows * 8 * SUB);
  return D == 64    ? launch_pdl(shared_merge_kernel<64, SUB>, grid, block, 0, s, m)
         : D == 128 ? launch_pdl(shared_merge_kernel<128, SUB>, grid, block, 0, s, m)
                    : launch_pdl(shared_merge_kernel<256, SUB>, grid, block, 0, s, m);
}

}  // namespace nk

using namespace nk;

extern "C" int nk_shared_decode_workspace_bytes(const nk_pool* pool, int32_t B, int32_t T, int32_t Hq,
                                                size_t* bytes) {
  clear_error();
  if (!pool || !bytes) return fail(NK_ERR_INVALID_ARG, "null argument");
  SharedPlan pl;
  int rc = make_shared_plan(pool, B, T, Hq, &pl);
  if (rc) return rc;
  *bytes = pl.ws_bytes;
  return NK_OK;
}

extern "C" int nk_paged_shared_decode_attention(const void* q, int32_t Hq, const nk_pool* pool, int32_t layer,
                                                const int32_t* block_tables, const int32_t* table_rows,
                                                const int32_t* frontiers, const int32_t* shared_pages,
                                                int32_t B, int32_t T, float softmax_scale, void* out,
                                                float* lse, int64_t share_from, void* workspace,
                                                size_t workspace_bytes, void* stream) {
  clear_error();
  if (!q || !pool || !block_tables || !table_rows || !frontiers || !shared_pages || !out)
    return fail(NK_ERR_INVALID_ARG, "null argument to nk_paged_shared_decode_attention");
  if (!std::isfinite(softmax_scale)) return fail(NK_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (layer < 0 || layer >= pool->desc.num_layers) return fail(NK_ERR_SHAPE, "layer out of range");
  if (!aligned16(q) || !aligned16(out)) return fail(NK_ERR_ALIGN, "q / out must be 16-byte aligned");
  SharedPlan pl;
  int rc = make_shared_plan(pool, B, T, Hq, &pl);
  if (rc) return rc;
  if (!workspace || workspace_bytes < pl.ws_bytes)
    return fail(NK_ERR_WORKSPACE, "workspace needs " + std::to_string(pl.ws_bytes) + " bytes");
  if (!aligned16(workspace)) return fail(NK_ERR_ALIGN, "workspace must be 16-byte aligned");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != pool->device)
    return fail(NK_ERR_INVALID_ARG, "the pool belongs to device " + std::to_string(pool->device) +
                                        ", the current device is " + std::to_string(dev));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int64_t page_bytes = 0;
  for (int i = 0; i < pool->n_planes; ++i) page_bytes += int64_t(NK_PAGE_TOKENS) * pool->plane[i].row_bytes;
  const int R = T * (Hq / pool->desc.num_kv_heads);
  const PageCosts costs = page_costs(pool, B, R, page_bytes);
  const int64_t least = share_from < 0 ? share_least(pool, B, R, costs) : std::max<int64_t>(share_from, 1);
  if (least > pool->L)  // no row has that many pages
    return run_decode(q, Hq, pool, layer, block_tables, table_rows, frontiers, nullptr, nullptr, B, T, softmax_scale,
                      out, lse, workspace, workspace_bytes, s, "nk_paged_shared_decode_attention");
  char* ws = static_cast<char*>(workspace);
  SharedPrefix sh;
  sh.pages = shared_pages;
  sh.frontiers = frontiers;
  sh.B = B;
  sh.T = T;
  sh.least = static_cast<int>(least);
  sh.shape = share_shape(pool, pl, B, R, costs);
  const PrefixParts parts{pl.tiles, pl.nsplit, reinterpret_cast<float2*>(ws),
                          reinterpret_cast<float*>(ws + pl.sh_ml_bytes)};
  e = prefix_pass(pool, layer, q, block_tables, table_rows, Hq, softmax_scale * kLog2e, parts, sh, s);
  if (e != cudaSuccess) return cuda_fail(e, "prefix pass launch");
  SharedMergeArgs m;
  DecodeArgs& a = m.d;
  const int np = pool->n_planes;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tables = block_tables;
  a.table_rows = table_rows;
  a.frontiers = frontiers;
  a.ks = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 2]) : nullptr;
  a.vs = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 3]) : nullptr;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.ws_ml = reinterpret_cast<float2*>(ws + pl.sh_bytes);
  a.ws_acc = reinterpret_cast<float*>(ws + pl.sh_bytes + pl.own.ws_ml_bytes);
  a.status = pool->status;
  a.softmax_scale = softmax_scale;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.H = pool->desc.num_kv_heads;
  a.G = Hq / a.H;
  a.L = pool->L;
  a.M = pool->M;
  a.C = pool->desc.max_concurrency;
  a.target = pl.own.target;
  a.nseg = pl.own.nseg;
  a.ctas = pl.own.ctas;
  a.head_major = pool->desc.order == NK_HEAD_MAJOR;
  a.shared = shared_pages;
  a.shared_least = sh.least;
  a.shape = sh.shape;
  e = pl.own.fn(pool, layer, a, pl.own.nqt, dim3(pl.own.ctas, a.H), s);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  m.prefix = parts;
  const int D = pool->desc.head_dim;
  const dim3 grid(B, a.H, D / 32 * ((T * a.G + kMergeRows - 1) / kMergeRows));
  e = T * a.G > 16 ? launch_merge<2>(D, grid, s, m) : launch_merge<8>(D, grid, s, m);
  if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  return NK_OK;
}
