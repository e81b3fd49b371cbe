// rope.cu -- per-head RMS norm and position rotation of queries and keys:
// on their own (nk_qk_norm_rope) and on the way into the paged cache
// (nk_paged_kv_append_rope, with the step's queries in the same launch).
//
// Both are one pass over the data, bound by HBM for long inputs and by the
// launch and two dependent loads for a decode step.  A warp holds 32 / (D/16)
// rows (rope.cuh).  Units of work are (token, group of heads of one operand); a
// lane reads the position's angles once for the heads of its unit.  The units
// are laid out operand by operand (all of q, then k and v), each operand padded
// to whole warps, so a warp never mixes operands.
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

// No element is written twice: the rows of a token lie behind one another and
// the tokens do, or the other way round.
static bool rows_apart(const nk_rows* r, int64_t tokens, int64_t heads, int D) {
  using Wide = __int128;
  const Wide t = r->token_stride < 0 ? -Wide(r->token_stride) : Wide(r->token_stride);
  const Wide h = r->head_stride < 0 ? -Wide(r->head_stride) : Wide(r->head_stride);
  if (tokens == 1) return heads == 1 || h >= D;
  if (heads == 1) return t >= D;
  return (h >= D && t >= (heads - 1) * h + D) || (t >= D && h >= (tokens - 1) * t + D);
}

static RowsIn rows_in(const nk_rows* r) {
  return r ? RowsIn{static_cast<const __nv_bfloat16*>(r->ptr), r->token_stride, r->head_stride}
           : RowsIn{nullptr, 0, 0};
}

constexpr int kRopeThreads = 128;
// Long inputs are bound by HBM and close behind by the issue rate.  Rows of a
// lane in flight, blocks per SM and warps per SM below which the heads of a
// token are spread over more units, with the times of 32749 tokens of 32 + 4
// heads of 128, an append of 8 x 2048 ragged tokens of 16 + 2 + 2 heads of 256
// and 2048 tokens of 16 + 2 heads of 256, in us (the copy rate gives 91.5, 42.3
// and 5.9):
//   4 rows, 5 blocks, 8 warps    94.5  52.4   9.2   (taken)
//   2 rows                       97.3  55.3
//   4 blocks / 6 blocks          94.4  55.8  /  95.4  51.3
//   16 warps / 32 warps                       10.6  /  14.9
constexpr int kRing = 4, kRopeBlocks = 5, kRopeWarps = 8;

// Work of one operand: units of `hpu` heads of one token, padded to whole
// warps; a warp of rpw rows takes rpw units.
struct Work {
  int heads, hpu;
  uint32_t groups, units;
};

// The unit of a group of LPR lanes; not live past the last one of its operand
// (padding lanes stay in the warp for its shuffles).
struct Unit {
  int token, head0, heads;  // heads [head0, head0 + heads)
  bool live;
};

__device__ __forceinline__ Unit unit_of(uint32_t u, uint32_t tokens, const Work& w) {
  Unit x;
  const uint32_t t = w.groups == 1 ? u : u / w.groups;
  x.live = t < tokens;
  x.token = x.live ? static_cast<int>(t) : 0;
  x.head0 = static_cast<int>(u - t * w.groups) * w.hpu;
  x.heads = min(w.hpu, w.heads - x.head0);
  return x;
}

__device__ __forceinline__ void copy_async16(uint32_t smem, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(p) : "memory");
}

// Rows 0 .. n - 1 of this lane (n alike in the warp): `src(i)` is the row's
// address or nullptr, `begin()` runs while the first are on their way, then
// `body(i, chunks)` for every row.  RING: a private ring of 16-byte slots in
// shared memory, filled by cp.async kRing rows ahead (the bytes in flight cost
// no registers, and a lane reads only what it copied, so no barrier is needed).
// Otherwise, for up to two rows, plain loads.
template <bool RING, class Src, class Begin, class Body>
__device__ __forceinline__ void for_rows(uint4* slots, int n, const Chunks& ch, Src src, Begin begin, Body body) {
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (RING) {
    const uint32_t at = smem_u32(slots);
    auto fetch = [&](int i) {
      const __nv_bfloat16* p = i < n ? src(i) : nullptr;
      if (p) {
        copy_async16(at + (2 * (i % kRing)) * (kRopeThreads * 16), p + ch.a);
        copy_async16(at + (2 * (i % kRing) + 1) * (kRopeThreads * 16), p + ch.b);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch(i);
    begin();
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      uint4 v[2] = {zero, zero};
      if (src(i)) {
        v[0] = slots[(2 * (i % kRing)) * kRopeThreads];
        v[1] = slots[(2 * (i % kRing) + 1) * kRopeThreads];
      }
      body(i, v);
      fetch(i + kRing);
    }
  } else {
    uint4 v[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __nv_bfloat16* p = i < n ? src(i) : nullptr;
      v[i][0] = p ? *reinterpret_cast<const uint4*>(p + ch.a) : zero;
      v[i][1] = p ? *reinterpret_cast<const uint4*>(p + ch.b) : zero;
    }
    begin();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i < n) body(i, v[i]);
  }
}

struct NormRopeArgs {
  RowsIn in[2];   // q, k
  RowsIn out[2];  // written
  const __nv_bfloat16* w[2];
  const int32_t* positions;
  Work work[2];
  int N;
  int* status;
  RopeArgs rp;
};

template <int D, bool RING>
__global__ void __launch_bounds__(kRopeThreads, RING ? kRopeBlocks : 1) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  __shared__ uint4 ring[RING ? 2 * kRing * kRopeThreads : 1];
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPR;
  uint32_t u = (blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5)) * RPW;  // the warp's first unit
  const int op = u >= a.work[0].units;
  if (op) u -= a.work[0].units;
  if (u >= a.work[op].units) return;
  const Unit x = unit_of(u + lane / LPR, a.N, a.work[op]);
  const RowsIn in = a.in[op], out = a.out[op];
  const Chunks ch = chunks_of(a.rp, l);
  const __nv_bfloat16* src = in.ptr + x.token * in.token_stride + x.head0 * in.head_stride;
  __nv_bfloat16* dst = const_cast<__nv_bfloat16*>(out.ptr) + x.token * out.token_stride + x.head0 * out.head_stride;
  Turn t;
  bool ok = false;
  for_rows<RING>(
      ring + threadIdx.x, a.work[op].hpu, ch,
      [&](int i) { return x.live && i < x.heads ? src + i * in.head_stride : nullptr; },
      [&] {
        const int pos = x.live ? a.positions[x.token] : 0;
        ok = x.live && pos >= 0 && pos < a.rp.positions;
        if (x.live && !ok && l == 0) set_status(a.status, NK_STATUS_FRONTIER);
        load_turn(a.rp, a.w[op], ok ? pos : 0, ch, t);
      },
      [&](int i, const uint4 (&raw)[2]) {
        Row16 y;
        norm_rotate<LPR>(raw, a.rp, ch, t, y);
        if (ok && i < x.heads) {
          *reinterpret_cast<uint4*>(dst + i * out.head_stride + ch.a) = pack8_bf16(y);
          *reinterpret_cast<uint4*>(dst + i * out.head_stride + ch.b) = pack8_bf16(y + 4);
        }
      });
}

// Heads per unit.  A unit reads its position's angles and weights once, so
// long inputs take all heads of an operand in one unit; below that the heads
// are spread over more units until the launch has about `want` warps.
static void plan_work(Work* w, int heads, int64_t tokens, int rpw, int64_t want) {
  w->heads = heads;
  w->hpu = heads > 0 ? heads : 1;
  auto units = [&] { return tokens * ((heads + w->hpu - 1) / w->hpu); };
  while (w->hpu > 1 && units() / rpw < want) w->hpu = w->hpu > 8 ? 8 : w->hpu > 4 ? 4 : 1;
  w->groups = heads > 0 ? (heads + w->hpu - 1) / w->hpu : 1;
  w->units = static_cast<uint32_t>(heads > 0 ? (units() + rpw - 1) / rpw * rpw : 0);
}

template <int D>
static cudaError_t launch_norm_rope(NormRopeArgs a, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / (D / 16);
  uint32_t warps = 0;
  bool ring = false;
  for (int i = 0; i < 2; ++i) {
    plan_work(&a.work[i], a.work[i].heads, a.N, RPW, int64_t(kRopeWarps) * sms);
    warps += a.work[i].units / RPW;
    ring = ring || a.work[i].hpu > 1;
  }
  const dim3 grid((warps + 3) / 4);
  return ring ? launch_pdl(norm_rope_kernel<D, true>, grid, dim3(kRopeThreads), 0, s, a)
              : launch_pdl(norm_rope_kernel<D, false>, grid, dim3(kRopeThreads), 0, s, a);
}

// ---- append with the rotation on the way ------------------------------------

struct AppendRopeArgs {
  RowsIn q, k, v;  // q may be absent; token index b * T + t
  __nv_bfloat16* q_out;
  const __nv_bfloat16* w[2];  // q, k norm weights
  const int32_t* tables;
  const int32_t* table_rows;
  const int32_t* write_pos;
  const int32_t* counts;
  uint8_t *kc, *vc, *ks, *vs;
  int* status;
  Work work[2];  // q heads; KV heads (a unit's keys, then its values)
  int B, T, L, M, C, head_major;
  RopeArgs rp;
};

template <int KK, int KV, int D, bool RING>
__global__ void __launch_bounds__(kRopeThreads, RING ? kRopeBlocks : 1)
    append_rope_kernel(const __grid_constant__ AppendRopeArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  __shared__ uint4 ring[RING ? 2 * kRing * kRopeThreads : 1];
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, l = lane % LPR;
  uint32_t u = (blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5)) * RPW;
  const int op = u >= a.work[0].units;
  if (op) u -= a.work[0].units;
  if (u >= a.work[op].units) return;
  const Unit x = unit_of(u + lane / LPR, a.B * a.T, a.work[op]);
  const int b = x.token / a.T, t = x.token - b * a.T;
  bool ok = x.live && t < (a.counts ? a.counts[b] : a.T);
  const int hpu = a.work[op].hpu;
  const Chunks ch = chunks_of(a.rp, l);
  Turn turn;
  int row = 0, pos = 0;
  auto begin = [&] {
    const bool read = ok;
    if (ok) {
      row = a.table_rows[b];
      pos = a.write_pos[b] + t;
      // rows and positions out of range are skipped, never written
      ok = row >= 0 && row < a.C && pos >= 0 && pos < a.L * 64 && pos < a.rp.positions;
    }
    if (read && !ok && l == 0) set_status(a.status, NK_STATUS_FRONTIER);
    load_turn(a.rp, a.w[op], ok ? pos : 0, ch, turn);
  };
  const bool read = ok;
  if (op == 0) {
    const __nv_bfloat16* src = a.q.ptr + x.token * a.q.token_stride + x.head0 * a.q.head_stride;
    __nv_bfloat16* dst = a.q_out + (static_cast<int64_t>(x.token) * a.work[0].heads + x.head0) * D;
    for_rows<RING>(
        ring + threadIdx.x, hpu, ch, [&](int i) { return read && i < x.heads ? src + i * a.q.head_stride : nullptr; },
        begin,
        [&](int i, const uint4 (&raw)[2]) {
          Row16 y;
          norm_rotate<LPR>(raw, a.rp, ch, turn, y);
          if (ok && i < x.heads) {
            *reinterpret_cast<uint4*>(dst + i * D + ch.a) = pack8_bf16(y);
            *reinterpret_cast<uint4*>(dst + i * D + ch.b) = pack8_bf16(y + 4);
          }
        });
    return;
  }
  const __nv_bfloat16* ksrc = a.k.ptr + x.token * a.k.token_stride + x.head0 * a.k.head_stride;
  const __nv_bfloat16* vsrc = a.v.ptr + x.token * a.v.token_stride + x.head0 * a.v.head_stride;
  constexpr bool GROUPS = KK == KIND_INT8 || KV == KIND_NVFP4;  // scales of part of a row
  __shared__ float s_max[GROUPS ? kRopeThreads * 2 : 1];
  float* maxima = GROUPS ? s_max + (threadIdx.x / LPR) * (D / 8) : s_max;
  int64_t tile0 = 0, pitch = 0;  // plane row of the token for the unit's first head, and the heads' distance
  for_rows<RING>(
      ring + threadIdx.x, 2 * hpu, ch,
      [&](int i) -> const __nv_bfloat16* {
        const int h = i < hpu ? i : i - hpu;
        if (!read || h >= x.heads) return nullptr;
        return i < hpu ? ksrc + h * a.k.head_stride : vsrc + h * a.v.head_stride;
      },
      [&] {
        begin();
        if (!ok) return;
        const int g = a.tables[static_cast<int64_t>(row) * a.L + (pos >> 6)];
        if (g < 0 || g >= a.M) {
          if (l == 0) set_status(a.status, NK_STATUS_PAGE_RANGE);
          ok = false;
          return;
        }
        tile0 = tile_row(g, x.head0, a.work[1].heads, a.M, a.head_major) + (pos & 63);
        pitch = a.head_major ? static_cast<int64_t>(a.M) * 64 : 64;
      },
      [&](int i, const uint4 (&raw)[2]) {
        Row16 y;
        if (i < hpu) {
          const int64_t r = tile0 + i * pitch;
          norm_rotate<LPR>(raw, a.rp, ch, turn, y);
          encode16<KK, D>(y, a.kc + r * code_row_bytes<KK>(D), a.ks + r * scale_row_bytes<KK>(D), ch, l,
                          ok && i < x.heads, maxima);
        } else {  // values: the codec alone
          const bool live = ok && i - hpu < x.heads;
          const int64_t r = tile0 + (i - hpu) * pitch;
          if constexpr (KV == KIND_BF16) {  // the bits unchanged
            if (live) {
              *reinterpret_cast<uint4*>(a.vc + r * (2 * D) + 2 * ch.a) = raw[0];
              *reinterpret_cast<uint4*>(a.vc + r * (2 * D) + 2 * ch.b) = raw[1];
            }
          } else {
            unpack8(raw[0], y);
            unpack8(raw[1], y + 4);
            encode16<KV, D>(y, a.vc + r * code_row_bytes<KV>(D), a.vs + r * scale_row_bytes<KV>(D), ch, l, live, maxima);
          }
        }
      });
}

template <int KK, int KV, int D>
static cudaError_t launch_append_rope(AppendRopeArgs a, int sms, cudaStream_t s) {
  constexpr int RPW = 32 / (D / 16);
  uint32_t warps = 0;
  bool ring = false;
  for (int i = 0; i < 2; ++i) {
    plan_work(&a.work[i], a.work[i].heads, static_cast<int64_t>(a.B) * a.T, RPW, int64_t(kRopeWarps) * sms);
    warps += a.work[i].units / RPW;
    ring = ring || a.work[i].hpu > 1;
  }
  const dim3 grid((warps + 3) / 4);
  return ring ? launch_pdl(append_rope_kernel<KK, KV, D, true>, grid, dim3(kRopeThreads), 0, s, a)
              : launch_pdl(append_rope_kernel<KK, KV, D, false>, grid, dim3(kRopeThreads), 0, s, a);
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
  if ((q && !rows_apart(q_out, N, Hq, head_dim)) || (k && !rows_apart(k_out, N, H, head_dim)))
    return fail(NK_ERR_SHAPE, "output rows overlap");
  const int heads = (q ? Hq : 0) + (k ? H : 0);
  if (static_cast<int64_t>(N) * heads > (int64_t(1) << 30)) return fail(NK_ERR_SHAPE, "too many head rows in one call");
  a.in[0] = rows_in(q);
  a.in[1] = rows_in(k);
  a.out[0] = rows_in(q_out);
  a.out[1] = rows_in(k_out);
  a.w[0] = static_cast<const __nv_bfloat16*>(rope->q_weight);
  a.w[1] = static_cast<const __nv_bfloat16*>(rope->k_weight);
  a.positions = positions;
  a.work[0].heads = q ? Hq : 0;
  a.work[1].heads = k ? H : 0;
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
  a.q = rows_in(q);
  a.k = rows_in(k);
  a.v = rows_in(v);
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
  a.work[0].heads = q ? Hq : 0;
  a.work[1].heads = H;
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
