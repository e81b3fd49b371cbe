// diff_prefill.cu -- differential attention of prompt chunks: the host side
// (diff_tile.cuh, diff_join.cuh).
#include "diff_join.cuh"

namespace nk {

struct DiffPrefillPlan {
  int TQ, tiles, cg, ctas;  // tokens of a CTA's tile; tiles of a cluster, its CTAs; clusters
  size_t ml_bytes, bytes;
};

static int diff_prefill_plan(const nk_pool* p, int B, int Tc, int Hq, DiffPrefillPlan* pl) {
  const int rc = check_diff_shape(p, B, Tc, Hq);
  if (rc) return rc;
  const int H = p->desc.num_kv_heads, G = Hq / H, D = p->desc.head_dim;
  if (G > 64) return fail(NK_ERR_UNSUPPORTED, "Hq / num_kv_heads must be <= 64");
  if (H / 2 > 65535) return fail(NK_ERR_UNSUPPORTED, "too many KV heads");
  pl->TQ = 128 / G;
  const int profile = p->desc.profile;
  pl->cg = diff_chunk_group(profile == NK_INT8_G64 ? KIND_INT8 : profile == NK_FP8_E4M3_ROW ? KIND_FP8 : KIND_BF16, D);
  pl->tiles = (Tc - 1) / (pl->TQ * pl->cg) + 1;
  const int64_t work = static_cast<int64_t>(B) * (H / 2) * pl->tiles;
  const int64_t most = work * 2 * (p->L + kDiffTileCost);  // units of all tiles
  if (work > (int64_t(1) << 24) || most / p->num_sms >= (int64_t(1) << 30) || static_cast<int64_t>(Tc) * Hq > (int64_t(1) << 30))
    return fail(NK_ERR_SHAPE, "too many tokens in one chunk");
  pl->ctas = p->num_sms / pl->cg < kDiffMaxPieces ? p->num_sms / pl->cg : kDiffMaxPieces;
  const size_t rows = (static_cast<size_t>(work) * 2 + pl->ctas) * pl->cg * 128;  // partials are numbered tile + cluster
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = diff_tile_for(pool->desc.profile)(pool, layer, a, false, dim3(pl.ctas * pl.cg), s);
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill launch");
  const DiffTileJoinArgs j{table_rows, prefix_len, chunk_len, a.ws_ml, a.ws_o, B,       Tc,       Hq,
                           a.H,        a.G,        a.L,       a.C,     pl.TQ,  pl.tiles, pl.cg, pl.ctas, o};
  e = launch_diff_tile_join<false>(pool->desc.head_dim, pool->num_sms, j, s);
  if (e != cudaSuccess) return cuda_fail(e, "differential prefill join launch");
  return NK_OK;
}
