// diff_decode.cu -- differential decode: the join of the splits, and the host side
// (checks, plan, launches).
#include "diff_decode.cuh"
#include "diff_join.cuh"

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

struct DiffJoinArgs {
  const int32_t* table_rows;
  const int32_t* frontiers;
  const float2* ws_ml;  // [pair][ctas][2][RB]
  const float* ws_o;    // [pair][ctas][2][RB][2 D]
  int B, T, Hq, G, L, C, ctas, RB;
  DiffOut o;
};

// ---- the join of the splits, the difference and the norm -------------------------------
// One CTA per (row, token, head).  A thread owns 4 dims of one map and every
// LANES-th split; the shares are added in a fixed order in shared memory.
template <int D>
__global__ void __launch_bounds__(512) diff_join_kernel(DiffJoinArgs a) {
  constexpr int COLS = D;  // 2 maps x 2 D / 4
  constexpr int LANES = 512 / COLS, EACH = kDiffMaxSplits / LANES, STEP = 8;
  __shared__ float s_w[2][kDiffMaxSplits];
  __shared__ float4 s_acc[LANES][COLS];
  __shared__ float s_sum[16];
  __shared__ int s_any;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.x, bt = blockIdx.y, b = bt / a.T, t = bt % a.T;
  // Inputs of the call: complete since before the splits' kernel let this one start,
  // and not written by it (read past L1, which the wait below has not renewed).
  const DiffRows rows = diff_rows(a.frontiers, a.table_rows, a.B, a.L, a.C, a.ctas, nullptr);
  const int ns = __shfl_sync(0xffffffffu, rows.ns, b), at = __shfl_sync(0xffffffffu, rows.end, b) - ns;
  const float lambda = __ldcg(a.o.lambda + bt * a.o.lambda_stride + head);
  const int RB = a.RB, r = t * a.G + head % a.G;
  const int64_t slot0 = static_cast<int64_t>(head / a.G) * a.ctas + at;
  const int map = tid % COLS / (COLS / 2), d = tid % (COLS / 2) * 4, sub = tid / COLS;
  const float* src = a.ws_o + ((slot0 * 2 + map) * RB + r) * (2 * D) + d;
  const int64_t step = static_cast<int64_t>(2) * RB * 2 * D;
  griddep_wait();  // the partials
  griddep_launch_dependents();
  if (warp < 2) {  // weights of map `warp`
    float2 ml[kDiffMaxSplits / 32];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < kDiffMaxSplits / 32; ++k) {
      const int s = lane + 32 * k;
      ml[k] = s < ns ? a.ws_ml[((slot0 + s) * 2 + warp) * RB + r] : make_float2(-INFINITY, 0.f);
      M = fmaxf(M, ml[k].x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll
    for (int k = 0; k < kDiffMaxSplits / 32; ++k) {
      ml[k].x = ml[k].y == 0.f ? 0.f : ex2(ml[k].x - M);  // a split that saw no key weighs nothing
      L += ml[k].x * ml[k].y;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    const bool none = L == 0.f;
#pragma unroll
    for (int k = 0; k < kDiffMaxSplits / 32; ++k)
      if (lane + 32 * k < ns) s_w[warp][lane + 32 * k] = none ? 0.f : ml[k].x / L;
    if (lane == 0) {
      if (warp == 0) s_any = !none;
      if (a.o.lse) a.o.lse[static_cast<int64_t>(bt) * a.Hq + 2 * head + warp] = none ? -INFINITY : (M + log2f(L)) * kDiffLn2;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < EACH && sub + k0 * LANES < ns; k0 += STEP) {
    float4 v[STEP];
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
      const int s = sub + (k0 + k) * LANES;
      v[k] = s < ns ? *reinterpret_cast<const float4*>(src + s * step) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int k = 0; k < STEP; ++k) {
      const int s = sub + (k0 + k) * LANES;
      const float w = s < ns ? s_w[map][s] : 0.f;
      acc.x = fmaf(w, v[k].x, acc.x);
      acc.y = fmaf(w, v[k].y, acc.y);
      acc.z = fmaf(w, v[k].z, acc.z);
      acc.w = fmaf(w, v[k].w, acc.w);
    }
  }
  s_acc[sub][tid % COLS] = acc;
  __syncthreads();
  float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  if (tid < COLS / 2) {
    float x[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float4 v = s_acc[0][m * (COLS / 2) + tid];
#pragma unroll
      for (int k = 1; k < LANES; ++k) {
        const float4 y = s_acc[k][m * (COLS / 2) + tid];
        v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      }
      x[m][0] = v.x, x[m][1] = v.y, x[m][2] = v.z, x[m][3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = s_any ? fmaf(-lambda, x[1][i], x[0][i]) : 0.f;
      sum = fmaf(o[i], o[i], sum);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (tid < COLS / 2) {
    sum = s_sum[0];
#pragma unroll
    for (int w = 1; w < COLS / 64; ++w) sum += s_sum[w];
    const float f = a.o.w ? rsqrtf(sum / (2 * D) + a.o.eps) * a.o.out_scale : a.o.out_scale;
    __nv_bfloat16* dst = a.o.out + (static_cast<int64_t>(bt) * (a.Hq / 2) + head) * (2 * D) + tid * 4;
    *reinterpret_cast<uint2*>(dst) = diff_finish(o, f, a.o.w, tid * 4);
  }
}

struct DiffPlan {
  DiffDecodeFn fn;  // nullptr: the tensor-core tiles
  int RB, ctas;
  size_t ml_bytes, bytes;
};

// Up to 8 query rows a map the warp-level kernel (4 or 8 rows of both maps in
// one column tile or two), beyond that the 64-row tiles; both with one CTA per SM.
// 8 rows by the warps, and the tiles, whose time up to 64 rows is one (head_dim 128, 8
// requests up to 32768 tokens): FP8-row 55 and 76 us, INT8-G64 64 and 113; up to 131072,
// K8V4: 143 and 174.
static int diff_plan(const nk_pool* p, int B, int T, int Hq, DiffPlan* pl) {
  const int rc = check_diff_shape(p, B, T, Hq);
  if (rc) return rc;
  const int H = p->desc.num_kv_heads, D = p->desc.head_dim;
  const int64_t rows = static_cast<int64_t>(T) * (Hq / H);
  if (rows > 64) return fail(NK_ERR_UNSUPPORTED, "T * Hq / num_kv_heads must be <= 64");
  pl->RB = rows <= 4 ? 4 : rows <= 8 ? 8 : 64;
  pl->fn = nullptr;
  if (pl->RB < 64) {
    switch (p->desc.profile) {
      case NK_BF16: pl->fn = diff_decode_bf16; break;
      case NK_INT8_G64: pl->fn = diff_decode_int8; break;
      case NK_FP8_E4M3_ROW: pl->fn = diff_decode_fp8; break;
      case NK_NVFP4_G16: pl->fn = diff_decode_nvfp4; break;
      default: pl->fn = diff_decode_k8v4; break;
    }
  }
  const int target = p->num_sms / (H / 2);
  pl->ctas = target > B ? target : B;
  const size_t slots = static_cast<size_t>(H / 2) * pl->ctas * 2 * pl->RB;  // query rows of all partials
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
  DiffOut o;
  int rc = check_diff("nk_paged_diff_decode_attention", q, Hq, pool, layer, block_tables, table_rows, frontiers, B, T,
                      softmax_scale, diff, out, lse, &o);
  if (rc) return rc;
  DiffPlan pl;
  if ((rc = diff_plan(pool, B, T, Hq, &pl))) return rc;
  if (!workspace || workspace_bytes < pl.bytes)
    return fail(NK_ERR_WORKSPACE, "workspace needs " + std::to_string(pl.bytes) + " bytes");
  if (!aligned16(workspace)) return fail(NK_ERR_ALIGN, "workspace must be 16-byte aligned");
  const DiffTileArgs t = [&] {
    DiffTileArgs x = diff_tile_args(pool, layer, q, Hq, block_tables, table_rows, frontiers, B, T, softmax_scale,
                                    workspace, pl.ml_bytes);
    x.ctas = pl.ctas;
    return x;
  }();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (pl.fn) {
    const DiffDecodeArgs a{t.q, t.tables, t.table_rows, t.lengths, t.ks, t.vs, t.ws_ml, t.ws_o, t.status, softmax_scale,
                           t.B, t.T, t.Hq, t.H, t.G, t.L, t.M, t.C, t.ctas, t.head_major};
    e = pl.fn(pool, layer, a, pl.RB == 4, s);
  } else {
    e = diff_tile_for(pool->desc.profile)(pool, layer, t, true, dim3(pl.ctas, t.H / 2), s);
  }
  if (e != cudaSuccess) return cuda_fail(e, "differential decode launch");
  if (!pl.fn) {
    const DiffTileJoinArgs tj{t.table_rows, t.lengths, nullptr, t.ws_ml, t.ws_o, B, T, Hq, t.H, t.G, t.L, t.C, 0, 1, 1, pl.ctas, o};
    e = launch_diff_tile_join<true>(pool->desc.head_dim, pool->num_sms, tj, s);
    if (e != cudaSuccess) return cuda_fail(e, "differential decode join launch");
    return NK_OK;
  }
  const DiffJoinArgs j{t.table_rows, t.lengths, t.ws_ml, t.ws_o, B, T, Hq, t.G, t.L, t.C, pl.ctas, pl.RB, o};
  const dim3 grid(Hq / 2, B * T);
  e = pool->desc.head_dim == 64 ? launch_pdl(diff_join_kernel<64>, grid, dim3(512), 0, s, j)
                                : launch_pdl(diff_join_kernel<128>, grid, dim3(512), 0, s, j);
  if (e != cudaSuccess) return cuda_fail(e, "differential decode join launch");
  return NK_OK;
}
