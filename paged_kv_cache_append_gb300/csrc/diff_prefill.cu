// diff_prefill.cu -- differential attention of prompt chunks: the join of the
// tiles' partials (diff_tile.cuh) and the host side.
#include "diff_tile.cuh"

namespace nk {

struct DiffChunkJoinArgs {
  const int32_t* table_rows;
  const int32_t* prefix_len;
  const int32_t* chunk_len;
  const float2* ws_ml;  // [B][pairs][tiles][nsplit][2][128]
  const float* ws_o;    // [B][pairs][tiles][nsplit][2][128][2 D]
  int Tc, Hq, H, G, L, C, TQ, tiles, nsplit;
  DiffOut o;
};

// ---- the join: one warp per (token, head), 2 D / 32 values a lane --------------
// Reads every partial once and writes bf16: bound by HBM / L2.
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) diff_prefill_join_kernel(DiffChunkJoinArgs a) {
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
  DiffOut o;
  if (!chunk_len) return fail(NK_ERR_INVALID_ARG, "null argument to nk_paged_diff_prefill_attention");
  int rc = check_diff("nk_paged_diff_prefill_attention", q_chunk, Hq, pool, layer, block_tables, table_rows, prefix_len,
                      B, Tc, softmax_scale, diff, out, lse, &o);
  if (rc) return rc;
  DiffPrefillPlan pl;
  if ((rc = diff_prefill_plan(pool, B, Tc, Hq, &pl))) return rc;
  if (!workspace || workspace_bytes < pl.bytes)
    return fail(NK_ERR_WORKSPACE, "workspace needs " + std::to_string(pl.bytes) + " bytes");
  if (!aligned16(workspace)) return fail(NK_ERR_ALIGN, "workspace must be 16-byte aligned");
  DiffTileArgs a = diff_tile_args(pool, layer, q_chunk, Hq, block_tables, table_rows, prefix_len, B, Tc, softmax_scale,
                                  workspace, pl.ml_bytes);
  a.chunk_len = chunk_len;
  a.TQ = pl.TQ;
  a.tiles = pl.tiles;
  a.nsplit = pl.nsplit;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = diff_tile_for(pool->desc.profile)(pool, layer, a, false, dim3(2 * pl.tiles * pl.nsplit, a.H / 2, B), s);
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill launch");
  const DiffChunkJoinArgs j{table_rows, prefix_len, chunk_len, a.ws_ml, a.ws_o, Tc, Hq, a.H, a.G,
                            a.L, a.C, pl.TQ, pl.tiles, pl.nsplit, o};
  const dim3 join(static_cast<unsigned>((static_cast<int64_t>(Tc) * (Hq / 2) + kJoinThreads / 32 - 1) / (kJoinThreads / 32)),
                  B);
  e = pool->desc.head_dim == 64 ? launch_pdl(diff_prefill_join_kernel<64>, join, dim3(kJoinThreads), 0, s, j)
                                : launch_pdl(diff_prefill_join_kernel<128>, join, dim3(kJoinThreads), 0, s, j);
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill join launch");
  return NK_OK;
}
