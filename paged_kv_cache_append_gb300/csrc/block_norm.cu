// block_norm.cu -- the norms before and after a block with its gate and the
// scales of the residual, in one pass (nk_residual_norm):
//   u = post(y), h = residual_scale r + scale act(g) u, x = norm(h).
//
// Bound by HBM: every operand crosses once, a row stays in registers between
// its two sums of squares.  A row is held by a group of threads with VPT vectors
// of 8 elements each; groups of up to a warp share a CTA and reduce by shuffles,
// wider rows take a CTA of whole warps and one shared-memory exchange for each
// sum.  The loads of y, the gate and the residual are issued before the first sum; the
// weight's, which L2 holds after the first rows, only before the second: held from the
// start it cost 10-14 registers a thread, and with them a CTA of an SM's (2048 rows of
// 4096, gated: 28.7 us against 22.5; 32749 rows of 2560, fp32 residual: 178 against 170,
// 87% of the copy rate).
#include <cmath>

#include "device.cuh"
#include "internal.h"

namespace nk {

struct NormArgs {
  const __nv_bfloat16* y;
  const __nv_bfloat16* gate;
  const void* res;
  void* res_out;
  __nv_bfloat16* x_out;
  const __nv_bfloat16* w;
  const __nv_bfloat16* post;
  int64_t ys, gs, rs, ros, xs;  // row strides in elements
  float eps, offset, scale, residual_scale, inv_dim;
  int sigmoid, N, vecs;  // vecs = dim / 8
};

__device__ __forceinline__ void unpack_bf16(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// x / (1 + e^-g).  With e^-|g| = t^2 the divisor stays in [1, 2], where __fdividef holds, and a
// gate far below 0 scales x by t twice: the factor by itself would leave fp32's range from -87 on,
// where an x of 2^127 still gives results of ordinary size (2048 gated rows of 4096: 20.5 us with
// 1 / (1 + e^-g) at once, 21.3 so).
__device__ __forceinline__ float gated(float x, float g) {
  const float t = ex2(-0.7213475204f * fabsf(g));  // log2(e) / 2
  if (g < 0.f) x = x * t * t;
  return __fdividef(x, fmaf(t, t, 1.f));
}

// Sum over the group of `lanes` (a power of two up to 32) or, beyond a warp,
// over the CTA; `part` is one slot per warp.
__device__ __forceinline__ float group_sum(float v, int lanes, float* part) {
  for (int off = min(lanes, 32) >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (lanes <= 32) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int VPT, bool WIDE>
__global__ void __launch_bounds__(512) block_norm_kernel(NormArgs a, int lanes) {
  __shared__ float part[2][32];
  const int groups = lanes > 32 ? 1 : blockDim.x / lanes;
  const int t = lanes > 32 ? threadIdx.x : threadIdx.x % lanes;
  const int n = blockIdx.x * groups + (lanes > 32 ? 0 : threadIdx.x / lanes);
  const bool row = n < a.N;
  griddep_wait();
  griddep_launch_dependents();
  float h[VPT][8], u[VPT][8];
  uint4 gv[VPT], pv[VPT];
  bool in[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = t + i * lanes;
    in[i] = row && v < a.vecs;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 yv = zero;
    gv[i] = pv[i] = zero;
#pragma unroll
    for (int k = 0; k < 8; ++k) h[i][k] = 0.f;
    if (in[i]) {
      if (a.y) yv = __ldcs(reinterpret_cast<const uint4*>(a.y + n * a.ys) + v);
      if constexpr (WIDE) {
        const float4* r = reinterpret_cast<const float4*>(static_cast<const float*>(a.res) + n * a.rs) + 2 * v;
        const float4 lo = __ldcs(r), hi = __ldcs(r + 1);
        h[i][0] = lo.x, h[i][1] = lo.y, h[i][2] = lo.z, h[i][3] = lo.w;
        h[i][4] = hi.x, h[i][5] = hi.y, h[i][6] = hi.z, h[i][7] = hi.w;
      } else {
        unpack_bf16(__ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.res) + n * a.rs) + v), h[i]);
      }
      if (a.gate) gv[i] = *(reinterpret_cast<const uint4*>(a.gate + n * a.gs) + v);
      if (a.post) pv[i] = __ldg(reinterpret_cast<const uint4*>(a.post) + v);
    }
    unpack_bf16(yv, u[i]);
  }
  if (a.y) {
    float f = 1.f;
    if (a.post) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) s = fmaf(u[i][k], u[i][k], s);
      f = rsqrtf(group_sum(s, lanes, part[0]) * a.inv_dim + a.eps);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float p[8], g[8];
      unpack_bf16(pv[i], p);
      unpack_bf16(gv[i], g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float x = u[i][k];
        if (a.post) x *= f * (p[k] + a.offset);
        if (a.gate) x = a.sigmoid ? gated(x, g[k]) : x * g[k];
        h[i][k] = fmaf(a.scale, x, a.residual_scale * h[i][k]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] *= a.residual_scale;
  }
  if (a.res_out) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!in[i]) continue;
      const int v = t + i * lanes;
      if constexpr (WIDE) {
        float4* r = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + n * a.ros) + 2 * v;
        r[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
        r[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
      } else {
        *(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.res_out) + n * a.ros) + v) = pack_bf16(h[i]);
      }
    }
  }
  if (!a.w) return;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(h[i][k], h[i][k], s);
  uint4 wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) wv[i] = in[i] ? __ldg(reinterpret_cast<const uint4*>(a.w) + t + i * lanes) : make_uint4(0u, 0u, 0u, 0u);
  const float f = rsqrtf(group_sum(s, lanes, part[1]) * a.inv_dim + a.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if (!in[i]) continue;
    float w[8], x[8];
    unpack_bf16(wv[i], w);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = h[i][k] * f * (w[k] + a.offset);
    *(reinterpret_cast<uint4*>(a.x_out + n * a.xs) + t + i * lanes) = pack_bf16(x);
  }
}

template <int VPT>
static cudaError_t launch_block_norm(const NormArgs& a, bool wide, int lanes, cudaStream_t s) {
  const int threads = lanes > 32 ? lanes : 128, groups = lanes > 32 ? 1 : threads / lanes;
  const dim3 grid((a.N + groups - 1) / groups);
  return wide ? launch_pdl(block_norm_kernel<VPT, true>, grid, dim3(threads), 0, s, a, lanes)
              : launch_pdl(block_norm_kernel<VPT, false>, grid, dim3(threads), 0, s, a, lanes);
}

static int check_operand(const void* p, int64_t stride, const char* name) {
  if (!aligned16(p) || stride % 8)
    return fail(NK_ERR_ALIGN, std::string(name) + " needs a 16-byte aligned base and a stride of 8 elements");
  return NK_OK;
}

}  // namespace nk

using namespace nk;

extern "C" int nk_residual_norm(const nk_block_norm* norm, int32_t dim, int32_t N, const void* y, int64_t y_stride,
                                const void* gate, int64_t gate_stride, const void* residual, int64_t residual_stride,
                                void* residual_out, int64_t residual_out_stride, void* x_out, int64_t x_stride,
                                void* stream) {
  clear_error();
  if (!norm || !residual) return fail(NK_ERR_INVALID_ARG, "null argument to nk_residual_norm");
  if (!residual_out && !x_out) return fail(NK_ERR_INVALID_ARG, "nk_residual_norm without an output");
  if ((norm->weight != nullptr) != (x_out != nullptr)) return fail(NK_ERR_INVALID_ARG, "weight and x_out come together");
  if (!y && (gate || norm->post_weight)) return fail(NK_ERR_INVALID_ARG, "a gate and post_weight need y");
  if (dim < 8 || dim > 16384 || dim % 8) return fail(NK_ERR_UNSUPPORTED, "dim must be a multiple of 8 in [8, 16384]");
  if (N < 1) return fail(NK_ERR_SHAPE, "N must be >= 1");
  if (!std::isfinite(norm->eps) || norm->eps <= 0.f || !std::isfinite(norm->weight_offset) ||
      !std::isfinite(norm->scale) || !std::isfinite(norm->residual_scale))
    return fail(NK_ERR_INVALID_ARG, "eps must be finite and > 0, the scales and weight_offset finite");
  if (norm->sigmoid_gate < 0 || norm->sigmoid_gate > 1 || norm->residual_fp32 < 0 || norm->residual_fp32 > 1)
    return fail(NK_ERR_INVALID_ARG, "sigmoid_gate and residual_fp32 must be 0 or 1");
  int rc;
  if ((rc = check_operand(norm->weight, 0, "weight")) || (rc = check_operand(norm->post_weight, 0, "post_weight")) ||
      (rc = check_operand(y, y ? y_stride : 0, "y")) || (rc = check_operand(gate, gate ? gate_stride : 0, "gate")) ||
      (rc = check_operand(residual, residual_stride, "residual")) ||
      (rc = check_operand(residual_out, residual_out ? residual_out_stride : 0, "residual_out")) ||
      (rc = check_operand(x_out, x_out ? x_stride : 0, "x_out")))
    return rc;
  const auto apart = [&](int64_t stride) { return N == 1 || stride >= dim || stride <= -dim; };
  if ((residual_out && !apart(residual_out_stride)) || (x_out && !apart(x_stride)))
    return fail(NK_ERR_SHAPE, "output rows overlap");
  NormArgs a{static_cast<const __nv_bfloat16*>(y), static_cast<const __nv_bfloat16*>(gate), residual, residual_out,
             static_cast<__nv_bfloat16*>(x_out), static_cast<const __nv_bfloat16*>(norm->weight),
             static_cast<const __nv_bfloat16*>(norm->post_weight), y_stride, gate_stride, residual_stride,
             residual_out_stride, x_stride, norm->eps, norm->weight_offset, norm->scale, norm->residual_scale,
             1.f / static_cast<float>(dim), norm->sigmoid_gate, N, dim / 8};
  // Threads of a row: one vector each while that is a warp or less, then whole
  // warps with one vector each up to 256 threads, two up to 512 (1024 rows and more of
  // 2560 dims: 170 us with two, 178 with one; of 4096, equal), else four: 16384 dims
  // would need 1024 threads of 64 registers with two.
  const bool wide = norm->residual_fp32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int lanes = 1;
  while (lanes < 32 && lanes < a.vecs) lanes *= 2;
  cudaError_t e;
  if (a.vecs <= 32) {
    e = launch_block_norm<1>(a, wide, lanes, s);
  } else {
    const auto warps = [&](int vpt) { return ((a.vecs + vpt - 1) / vpt + 31) / 32 * 32; };
    if (a.vecs <= 256) e = launch_block_norm<1>(a, wide, warps(1), s);
    else if (a.vecs <= 1024) e = launch_block_norm<2>(a, wide, warps(2), s);
    else e = launch_block_norm<4>(a, wide, warps(4), s);
  }
  if (e != cudaSuccess) return cuda_fail(e, "residual norm launch");
  return NK_OK;
}
