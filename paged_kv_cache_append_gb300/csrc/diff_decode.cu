// diff_decode.cu -- host side of the differential decode: checks, plan, launch.
#include "diff_decode.cuh"

namespace nk {

int check_diff_shape(const nk_pool* pool, int32_t B, int32_t T, int32_t Hq) {
  const int H = pool->desc.num_kv_heads, D = pool->desc.head_dim;
  if (D != 64 && D != 128) return fail(NK_ERR_UNSUPPORTED, "differential attention needs head_dim 64 or 128");
  if (H % 2) return fail(NK_ERR_SHAPE, "differential attention needs an even number of KV heads");
  if (Hq < 1 || Hq % H) return fail(NK_ERR_SHAPE, "Hq must be a positive multiple of num_kv_heads");
  if (B < 1 || B > pool->desc.max_concurrency) return fail(NK_ERR_SHAPE, "B must be in [1, C]");
  if (T < 1) return fail(NK_ERR_SHAPE, "T must be >= 1");
  return NK_OK;
}

int check_diff(const char* what, const void* q, int32_t Hq, const nk_pool* pool, int32_t layer, const int32_t* tables,
               const int32_t* table_rows, const int32_t* lengths, int32_t B, int32_t T, float scale, const nk_diff* diff,
               void* out, float* lse, DiffOut* o) {
  if (!q || !pool || !tables || !table_rows || !lengths || !diff || !out)
    return fail(NK_ERR_INVALID_ARG, std::string("null argument to ") + what);
  if (!diff->lambda) return fail(NK_ERR_INVALID_ARG, "lambda is NULL");
  if (!std::isfinite(scale)) return fail(NK_ERR_INVALID_ARG, "softmax_scale is not finite");
  if (!std::isfinite(diff->out_scale)) return fail(NK_ERR_INVALID_ARG, "out_scale is not finite");
  if (diff->norm_weight && (!std::isfinite(diff->eps) || diff->eps <= 0.f))
    return fail(NK_ERR_INVALID_ARG, "eps must be finite and > 0");
  const int rc = check_diff_shape(pool, B, T, Hq);
  if (rc) return rc;
  if (layer < 0 || layer >= pool->desc.num_layers) return fail(NK_ERR_SHAPE, "layer out of range");
  if (!aligned16(q) || !aligned16(out) || !aligned16(diff->norm_weight))
    return fail(NK_ERR_ALIGN, "q, out and the norm weight must be 16-byte aligned");
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != pool->device)
    return fail(NK_ERR_INVALID_ARG, "the pool belongs to device " + std::to_string(pool->device) +
                                        ", the current device is " + std::to_string(dev));
  *o = DiffOut{diff->lambda, diff->lambda_stride, static_cast<const __nv_bfloat16*>(diff->norm_weight), diff->eps,
               diff->out_scale, static_cast<__nv_bfloat16*>(out), lse};
  return NK_OK;
}

struct DiffPlan {
  DiffDecodeFn fn;
  int rows, blocks, ctas;
  size_t ml_bytes, bytes;
};

// Query rows of one pair go in blocks of 4, 8 or 16 (two maps of a block in one
// CTA); more rows take several blocks, which read the same pages side by side.
static int diff_plan(const nk_pool* p, int B, int T, int Hq, DiffPlan* pl) {
  const int rc = check_diff_shape(p, B, T, Hq);
  if (rc) return rc;
  const int H = p->desc.num_kv_heads, D = p->desc.head_dim;
  const int64_t rows = static_cast<int64_t>(T) * (Hq / H);
  if (rows > 64) return fail(NK_ERR_UNSUPPORTED, "T * Hq / num_kv_heads must be <= 64");
  switch (p->desc.profile) {
    case NK_BF16: pl->fn = diff_decode_bf16; break;
    case NK_INT8_G64: pl->fn = diff_decode_int8; break;
    case NK_FP8_E4M3_ROW: pl->fn = diff_decode_fp8; break;
    case NK_NVFP4_G16: pl->fn = diff_decode_nvfp4; break;
    default: pl->fn = diff_decode_k8v4; break;
  }
  pl->rows = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  pl->blocks = static_cast<int>((rows + pl->rows - 1) / pl->rows);
  int per_sm = 1;
  const cudaError_t e = pl->fn(p, 0, nullptr, pl->rows, &per_sm, nullptr);
  if (e != cudaSuccess) return cuda_fail(e, "occupancy query");
  const int target = p->num_sms * per_sm / (H / 2 * pl->blocks);
  pl->ctas = target > B ? target : B;
  const size_t slots = static_cast<size_t>(H / 2) * pl->blocks * pl->ctas * 2 * pl->rows;
  pl->ml_bytes = (slots * sizeof(float2) + 255) / 256 * 256;
  pl->bytes = pl->ml_bytes + slots * 2 * D * sizeof(float);
  return NK_OK;
}

}  // namespace nk

using namespace nk;

extern "C" int nk_diff_decode_workspace_bytes(const nk_pool* pool, int32_t B, int32_t T, int32_t Hq, size_t* bytes) {
  clear_error();
  if (!pool || !bytes) return fail(NK_ERR_INVALID_ARG, "null argument");
  DiffPlan pl;
  const int rc = diff_plan(pool, B, T, Hq, &pl);
  if (rc) return rc;
  *bytes = pl.bytes;
  return NK_OK;
}

extern "C" int nk_paged_diff_decode_attention(const void* q, int32_t Hq, const nk_pool* pool, int32_t layer,
                                              const int32_t* block_tables, const int32_t* table_rows,
                                              const int32_t* frontiers, int32_t B, int32_t T, float softmax_scale,
                                              const nk_diff* diff, void* out, float* lse, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  clear_error();
  DiffDecodeArgs a;
  int rc = check_diff("nk_paged_diff_decode_attention", q, Hq, pool, layer, block_tables, table_rows, frontiers, B, T,
                      softmax_scale, diff, out, lse, &a.o);
  if (rc) return rc;
  DiffPlan pl;
  if ((rc = diff_plan(pool, B, T, Hq, &pl))) return rc;
  if (!workspace || workspace_bytes < pl.bytes)
    return fail(NK_ERR_WORKSPACE, "workspace needs " + std::to_string(pl.bytes) + " bytes");
  if (!aligned16(workspace)) return fail(NK_ERR_ALIGN, "workspace must be 16-byte aligned");
  const int np = pool->n_planes;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tables = block_tables;
  a.table_rows = table_rows;
  a.frontiers = frontiers;
  a.ks = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 2]) : nullptr;
  a.vs = np == 4 ? static_cast<const uint8_t*>(pool->ptrs[layer * np + 3]) : nullptr;
  a.ws_ml = static_cast<float2*>(workspace);
  a.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.ml_bytes);
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
  a.ctas = pl.ctas;
  a.blocks = pl.blocks;
  a.head_major = pool->desc.order == NK_HEAD_MAJOR;
  const cudaError_t e = pl.fn(pool, layer, &a, pl.rows, nullptr, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "differential decode launch");
  return NK_OK;
}
