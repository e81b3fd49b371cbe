// rope.cu -- per-head RMS norm and position rotation of queries and keys:
// on their own (nk_qk_norm_rope) and on the way into the paged cache
// (nk_paged_kv_append_rope, with the step's queries in the same launch).
//
// Both are one pass over the data, bound by HBM for long inputs and by the
// launch and two dependent loads for a decode step.  A warp holds 32 / (D/8)
// rows (rope.cuh).  Units of work are (token, group of HPU heads of one
// operand); a lane loads the position's angles once for the HPU heads.  The
// units are laid out operand by operand (all q, then k, then v), each operand
// padded to whole warps, so a warp never mixes operands.
#include <cmath>

#include "rope.cuh"

namespace nk {

static int check_rope(const nk_rope* r, int D, RopeArgs* o) {
  if (!r) return fail(NK_ERR_INVALID_ARG, "rope is NULL");
  if (r->rotary_dim < 0 || r->rotary_dim > D || r->rotary_dim % 16)
    return fail(NK_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 in [0, head_dim]");
  if (r->layout != NK_ROPE_HALVES && r->layout != NK_ROPE_PAIRS)
    return fail(NK_ERR_INVALID_ARG, "rope layout must be NK_ROPE_HALVES or NK_ROPE_PAIRS");
  if (r->positions < 1) return fail(NK_ERR_SHAPE, "rope positions must be >= 1");
  if (r->rotary_dim && !r->cos_sin) return fail(NK_ERR_INVALID_ARG, "cos_sin is NULL");
  if (!aligned16(r->cos_sin) || !aligned16(r->q_weight) || !aligned16(r->k_weight))
    return fail(NK_ERR_ALIGN, "cos_sin and the norm weights must be 16-byte aligned");
  if (!std::isfinite(r->eps) || r->eps < 0.f || !std::isfinite(r->weight_offset))
    return fail(NK_ERR_INVALID_ARG, "eps must be finite and >= 0, weight_offset finite");
  *o = RopeArgs{static_cast<const float*>(r->cos_sin), r->positions, r->rotary_dim, r->layout == NK_ROPE_PAIRS,
                r->eps, r->weight_offset};
  return NK_OK;
}

// Rows of an operand: 16-byte loads need an aligned base and strides that are
// multiples of 8 elements.
static int check_rows(const nk_rows* r, const char* name) {
  if (!r->ptr) return fail(NK_ERR_INVALID_ARG, std::string(name) + " rows are NULL");
  if (!aligned16(r->ptr) || r->token_stride % 8 || r->head_stride % 8)
    return fail(NK_ERR_ALIGN, std::string(name) + " rows need a 16-byte aligned base and strides of 8 elements");
  return NK_OK;
}

static RowsIn rows_in(const nk_rows* r) {
  return r ? RowsIn{static_cast<const __nv_bfloat16*>(r->ptr), r->token_stride, r->head_stride}
           : RowsIn{nullptr, 0, 0};
}

struct NormRopeArgs {
  RowsIn in[2];           // q, k
  RowsIn out[2];          // written
  const __nv_bfloat16* w[2];
  const int32_t* positions;
  int heads[2], groups[2];
  int64_t units[2];       // padded to whole warps
  int N;
  int* status;
  RopeArgs rp;
};

// Which unit a group of LPR lanes takes: returns false past the last unit of
// its operand (padding lanes stay in the warp for its shuffles).
struct Unit {
  int token, head0;
  bool live;
};

template <int HPU>
__device__ __forceinline__ Unit unit_of(int64_t u, int tokens, int groups) {
  Unit x;
  const int64_t t = u / groups;
  x.live = t < tokens;
  x.token = x.live ? static_cast<int>(t) : 0;
  x.head0 = static_cast<int>(u - t * groups) * HPU;
  return x;
}

template <int D, int HPU>
__global__ void __launch_bounds__(128) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPR;
  int64_t u = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5)) * RPW;  // the warp's first unit
  const int op = u >= a.units[0];
  if (op) u -= a.units[0];
  if (u >= a.units[op]) return;
  const Unit x = unit_of<HPU>(u + lane / LPR, a.N, a.groups[op]);
  const int pos = x.live ? a.positions[x.token] : 0;
  const bool ok = x.live && pos >= 0 && pos < a.rp.positions;
  if (x.live && !ok && l == 0) set_status(a.status, NK_STATUS_FRONTIER);
  const RowsIn in = a.in[op], out = a.out[op];
  const int heads = a.heads[op];
  const int64_t base = x.token * in.token_stride + x.head0 * in.head_stride + 8 * l;
  uint4 raw[HPU];
#pragma unroll
  for (int i = 0; i < HPU; ++i)
    raw[i] = ok && x.head0 + i < heads ? *reinterpret_cast<const uint4*>(in.ptr + base + i * in.head_stride)
                                       : make_uint4(0u, 0u, 0u, 0u);
  Angles ang;
  load_angles(a.rp, ok ? pos : 0, l, ang);
  const int src = partner_lane(a.rp, lane, l);
  Weights w;
  load_weights(a.rp, a.w[op], lane, l, src, w);
  __nv_bfloat16* dst = const_cast<__nv_bfloat16*>(out.ptr) + x.token * out.token_stride + x.head0 * out.head_stride + 8 * l;
#pragma unroll
  for (int i = 0; i < HPU; ++i) {
    float y[8];
    norm_rotate<LPR>(raw[i], a.rp, ang, w, src, y);
    if (ok && x.head0 + i < heads) *reinterpret_cast<uint4*>(dst + i * out.head_stride) = pack8_bf16(y);
  }
}

// Heads per unit: 4 once the launch has several waves of units (the angles of
// a position are then read once for 4 heads and a lane keeps four 16-byte
// loads in flight); 1 below, where spreading the rows over the SMs counts.
static int heads_per_unit(int64_t rows, int lpr, int sms) { return rows * lpr >= int64_t(sms) * 8192 ? 4 : 1; }

static int64_t padded(int64_t units, int rpw) { return (units + rpw - 1) / rpw * rpw; }

template <int D>
static cudaError_t launch_norm_rope(NormRopeArgs a, int sms, cudaStream_t s) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int hpu = heads_per_unit(static_cast<int64_t>(a.N) * (a.heads[0] + a.heads[1]), LPR, sms);
  for (int i = 0; i < 2; ++i) {
    a.groups[i] = (a.heads[i] + hpu - 1) / hpu;
    a.units[i] = padded(static_cast<int64_t>(a.N) * a.groups[i], RPW);
  }
  const int64_t warps = (a.units[0] + a.units[1]) / RPW;
  const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
  return hpu == 4 ? launch_pdl(norm_rope_kernel<D, 4>, grid, dim3(128), 0, s, a)
                  : launch_pdl(norm_rope_kernel<D, 1>, grid, dim3(128), 0, s, a);
}

// ---- append with the rotation on the way ------------------------------------

struct AppendRopeArgs {
  RowsIn in[3];  // q (may be absent), k, v; token index b * T + t
  __nv_bfloat16* q_out;
  const __nv_bfloat16* w[2];  // q, k norm weights
  const int32_t* tables;
  const int32_t* table_rows;
  const int32_t* write_pos;
  const int32_t* counts;
  uint8_t *kc, *vc, *ks, *vs;
  int* status;
  int heads[3], groups[3];
  int64_t units[3];
  int B, T, L, M, C, head_major;
  RopeArgs rp;
};

template <int KK, int KV, int D, int HPU>
__global__ void __launch_bounds__(128) append_rope_kernel(const __grid_constant__ AppendRopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPR;
  int64_t u = (static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5)) * RPW;
  int op = 0;
  while (op < 3 && u >= a.units[op]) u -= a.units[op++];
  if (op == 3) return;
  const Unit x = unit_of<HPU>(u + lane / LPR, a.B * a.T, a.groups[op]);
  const int b = x.token / a.T, t = x.token - b * a.T;
  const int H = a.heads[1];
  bool ok = x.live && t < (a.counts ? a.counts[b] : a.T);
  int row = 0, pos = 0;
  if (ok) {
    row = a.table_rows[b];
    pos = a.write_pos[b] + t;
    // rows and positions out of range are skipped, never written
    if (row < 0 || row >= a.C || pos < 0 || pos >= a.L * 64 || pos >= a.rp.positions) {
      if (l == 0) set_status(a.status, NK_STATUS_FRONTIER);
      ok = false;
    }
  }
  const RowsIn in = a.in[op];
  const int heads = a.heads[op];
  const int64_t base = x.token * in.token_stride + x.head0 * in.head_stride + 8 * l;
  uint4 raw[HPU];
#pragma unroll
  for (int i = 0; i < HPU; ++i)
    raw[i] = ok && x.head0 + i < heads ? *reinterpret_cast<const uint4*>(in.ptr + base + i * in.head_stride)
                                       : make_uint4(0u, 0u, 0u, 0u);
  int64_t tile0 = 0;  // first plane row of the token for head 0, and the heads' distance
  int64_t pitch = 0;
  if (op > 0 && ok) {
    const int g = a.tables[static_cast<int64_t>(row) * a.L + (pos >> 6)];
    if (g < 0 || g >= a.M) {
      if (l == 0) set_status(a.status, NK_STATUS_PAGE_RANGE);
      ok = false;
    } else {
      tile0 = tile_row(g, 0, H, a.M, a.head_major) + (pos & 63);
      pitch = a.head_major ? static_cast<int64_t>(a.M) * 64 : 64;
    }
  }
  if (op == 2) {  // values: the codec alone
#pragma unroll
    for (int i = 0; i < HPU; ++i) {
      const bool live = ok && x.head0 + i < heads;
      const int64_t r = tile0 + (x.head0 + i) * pitch;
      if constexpr (KV == KIND_BF16) {  // the bits unchanged
        if (live) *reinterpret_cast<uint4*>(a.vc + r * (2 * D) + 16 * l) = raw[i];
      } else {
        float y[8];
        unpack8(raw[i], y);
        encode8<KV, D>(y, a.vc + r * code_row_bytes<KV>(D), a.vs + r * scale_row_bytes<KV>(D), l, live);
      }
    }
    return;
  }
  Angles ang;
  load_angles(a.rp, ok ? pos : 0, l, ang);
  const int src = partner_lane(a.rp, lane, l);
  Weights w;
  load_weights(a.rp, a.w[op], lane, l, src, w);
#pragma unroll
  for (int i = 0; i < HPU; ++i) {
    const bool live = ok && x.head0 + i < heads;
    float y[8];
    norm_rotate<LPR>(raw[i], a.rp, ang, w, src, y);
    if (op == 0) {
      if (live)
        *reinterpret_cast<uint4*>(a.q_out + (static_cast<int64_t>(x.token) * heads + x.head0 + i) * D + 8 * l) =
            pack8_bf16(y);
    } else {
      const int64_t r = tile0 + (x.head0 + i) * pitch;
      encode8<KK, D>(y, a.kc + r * code_row_bytes<KK>(D), a.ks + r * scale_row_bytes<KK>(D), l, live);
    }
  }
}

template <int KK, int KV, int D>
static cudaError_t launch_append_rope(AppendRopeArgs a, int sms, cudaStream_t s) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int64_t n = static_cast<int64_t>(a.B) * a.T;
  const int hpu = heads_per_unit(n * (a.heads[0] + a.heads[1] + a.heads[2]), LPR, sms);
  int64_t warps = 0;
  for (int i = 0; i < 3; ++i) {
    a.groups[i] = (a.heads[i] + hpu - 1) / hpu;
    a.units[i] = padded(n * a.groups[i], RPW);
    warps += a.units[i] / RPW;
  }
  const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
  return hpu == 4 ? launch_pdl(append_rope_kernel<KK, KV, D, 4>, grid, dim3(128), 0, s, a)
                  : launch_pdl(append_rope_kernel<KK, KV, D, 1>, grid, dim3(128), 0, s, a);
}

template <int KK, int KV>
static cudaError_t append_rope_d(int D, const AppendRopeArgs& a, int sms, cudaStream_t s) {
  return D == 64    ? launch_append_rope<KK, KV, 64>(a, sms, s)
         : D == 128 ? launch_append_rope<KK, KV, 128>(a, sms, s)
                    : launch_append_rope<KK, KV, 256>(a, sms, s);
}

}  // namespace nk

using namespace nk;

extern "C" int nk_qk_norm_rope(const nk_rope* rope, int32_t head_dim, const nk_rows* q, int32_t Hq,
                               const nk_rows* k, int32_t H, const int32_t* positions, int32_t N,
                               const nk_rows* q_out, const nk_rows* k_out, void* stream) {
  clear_error();
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(NK_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256, got " + std::to_string(head_dim));
  NormRopeArgs a;
  int rc = check_rope(rope, head_dim, &a.rp);
  if (rc) return rc;
  if (!positions || (!q && !k)) return fail(NK_ERR_INVALID_ARG, "null argument to nk_qk_norm_rope");
  if ((q != nullptr) != (q_out != nullptr) || (k != nullptr) != (k_out != nullptr))
    return fail(NK_ERR_INVALID_ARG, "q and q_out, k and k_out come together");
  if (N < 1) return fail(NK_ERR_SHAPE, "N must be >= 1");
  if ((q && Hq < 1) || (k && H < 1)) return fail(NK_ERR_SHAPE, "head counts must be >= 1");
  const nk_rows* rows[4] = {q, k, q_out, k_out};
  const char* names[4] = {"q", "k", "q_out", "k_out"};
  for (int i = 0; i < 4; ++i)
    if (rows[i] && (rc = check_rows(rows[i], names[i]))) return rc;
  const int heads = (q ? Hq : 0) + (k ? H : 0);
  if (static_cast<int64_t>(N) * heads > (int64_t(1) << 30)) return fail(NK_ERR_SHAPE, "too many head rows in one call");
  a.in[0] = rows_in(q);
  a.in[1] = rows_in(k);
  a.out[0] = rows_in(q_out);
  a.out[1] = rows_in(k_out);
  a.w[0] = static_cast<const __nv_bfloat16*>(rope->q_weight);
  a.w[1] = static_cast<const __nv_bfloat16*>(rope->k_weight);
  a.positions = positions;
  a.heads[0] = q ? Hq : 0;
  a.heads[1] = k ? H : 0;
  a.N = N;
  a.status = status_word();
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int sms = device_sm_count(dev);
  if (!a.status || !sms) return fail(NK_ERR_CUDA, "device query failed (status word / SM count)");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = head_dim == 64    ? launch_norm_rope<64>(a, sms, s)
      : head_dim == 128 ? launch_norm_rope<128>(a, sms, s)
                        : launch_norm_rope<256>(a, sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "norm and rotation launch");
  return NK_OK;
}

extern "C" int nk_paged_kv_append_rope(nk_pool* pool, int32_t layer, const int32_t* block_tables,
                                       const int32_t* table_rows, const int32_t* write_pos,
                                       const int32_t* counts, const nk_rope* rope, const nk_rows* k,
                                       const nk_rows* v, const nk_rows* q, int32_t Hq, void* q_out,
                                       int32_t B, int32_t T, void* stream) {
  clear_error();
  if (!pool || !block_tables || !table_rows || !write_pos || !k || !v)
    return fail(NK_ERR_INVALID_ARG, "null argument to nk_paged_kv_append_rope");
  const int D = pool->desc.head_dim, H = pool->desc.num_kv_heads;
  AppendRopeArgs a;
  int rc = check_rope(rope, D, &a.rp);
  if (rc) return rc;
  if (layer < 0 || layer >= pool->desc.num_layers) return fail(NK_ERR_SHAPE, "layer out of range");
  if (B < 1 || B > pool->desc.max_concurrency) return fail(NK_ERR_SHAPE, "B must be in [1, C]");
  if (T < 1) return fail(NK_ERR_SHAPE, "T must be >= 1");
  if ((q != nullptr) != (q_out != nullptr)) return fail(NK_ERR_INVALID_ARG, "q and q_out come together");
  if (q && Hq < 1) return fail(NK_ERR_SHAPE, "Hq must be >= 1");
  if ((rc = check_rows(k, "k")) || (rc = check_rows(v, "v")) || (q && (rc = check_rows(q, "q")))) return rc;
  if (!aligned16(q_out)) return fail(NK_ERR_ALIGN, "q_out must be 16-byte aligned");
  if (static_cast<int64_t>(B) * T * (2 * static_cast<int64_t>(H) + (q ? Hq : 0)) > (int64_t(1) << 30))
    return fail(NK_ERR_SHAPE, "too many head rows in one append");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != pool->device)
    return fail(NK_ERR_INVALID_ARG, "the pool belongs to device " + std::to_string(pool->device) +
                                        ", the current device is " + std::to_string(dev));
  const int np = pool->n_planes;
  a.in[0] = rows_in(q);
  a.in[1] = rows_in(k);
  a.in[2] = rows_in(v);
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.w[0] = static_cast<const __nv_bfloat16*>(rope->q_weight);
  a.w[1] = static_cast<const __nv_bfloat16*>(rope->k_weight);
  a.tables = block_tables;
  a.table_rows = table_rows;
  a.write_pos = write_pos;
  a.counts = counts;
  a.kc = static_cast<uint8_t*>(pool->ptrs[layer * np + 0]);
  a.vc = static_cast<uint8_t*>(pool->ptrs[layer * np + 1]);
  a.ks = np == 4 ? static_cast<uint8_t*>(pool->ptrs[layer * np + 2]) : nullptr;
  a.vs = np == 4 ? static_cast<uint8_t*>(pool->ptrs[layer * np + 3]) : nullptr;
  a.status = pool->status;
  a.heads[0] = q ? Hq : 0;
  a.heads[1] = a.heads[2] = H;
  a.B = B;
  a.T = T;
  a.L = pool->L;
  a.M = pool->M;
  a.C = pool->desc.max_concurrency;
  a.head_major = pool->desc.order == NK_HEAD_MAJOR;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (pool->desc.profile) {
    case NK_BF16: e = append_rope_d<KIND_BF16, KIND_BF16>(D, a, pool->num_sms, s); break;
    case NK_INT8_G64: e = append_rope_d<KIND_INT8, KIND_INT8>(D, a, pool->num_sms, s); break;
    case NK_FP8_E4M3_ROW: e = append_rope_d<KIND_FP8, KIND_FP8>(D, a, pool->num_sms, s); break;
    case NK_NVFP4_G16: e = append_rope_d<KIND_NVFP4, KIND_NVFP4>(D, a, pool->num_sms, s); break;
    default: e = append_rope_d<KIND_FP8, KIND_NVFP4>(D, a, pool->num_sms, s); break;
  }
  if (e != cudaSuccess) return cuda_fail(e, "append with rotation launch");
  return NK_OK;
}
