// verify.cu -- verification of drafted tokens against the target model's
// probabilities, from given random numbers.
//
// Sequence b has K_b <= K drafts x_0 .. x_{K_b - 1}, the target's rows p_0 ..
// p_{K_b} and the draft model's rows q_0 .. q_{K_b - 1} (without them each
// draft is taken as certain: q_i is 1 at x_i).  Draft i is accepted iff
//   u_i q_i(x_i) < p_i(x_i)
// (compared exactly: the fp64 product of two fp32 values has no rounding); n
// is the first draft that is not, K_b if there is none.  The next token is
// drawn by inverse transform from the weights
//   d_j = max(p_n(j) - q_n(j), 0)  (n < K_b),   d_j = p_n(j)  (n = K_b):
// the least j with d_0 + .. + d_j > u_K (d_0 + .. + d_{V-1}).
//
// The sums decide at borders whose distance is a token's own probability, so
// they are held in more than fp32: a thread adds its fp32 differences, with
// the rounding error of each difference and of each addition, as an unevaluated
// pair of fp32 values (Knuth's TwoSum; about 48 bits, at the fp32 rate, where
// this chip's fp64 units are a small fraction of it), and everything above a
// thread in fp64.
//
// One cluster of CTAs works on a sequence, each CTA on a contiguous slice of
// the vocabulary, staged tile by tile in shared memory with coalesced loads
// (rows of an odd vocabulary are not 16-byte aligned) and then read back as
// one contiguous run per thread, so that the thread sums are in vocabulary
// order.  The slice sums meet over distributed shared memory; every CTA then
// knows which slice holds the border, and that one finds the tile, warp, lane
// and element.  Only the two rows that are needed are read, once.
#include <cooperative_groups.h>

#include <cfloat>

#include "device.cuh"
#include "internal.h"

namespace cg = cooperative_groups;

namespace nk {

struct VerifyArgs {
  const float* target;   // [B][K + 1] rows of target_stride
  const float* draft;    // [B][K] rows of draft_stride, or nullptr
  const int32_t* tokens;  // [B][K]
  const int32_t* draft_len;
  const float* u;  // [B][K + 1]
  const int32_t* frontiers;
  int32_t* accepted;
  int32_t* out;  // [B][K + 1]
  int32_t* frontiers_out;
  int* status;
  int64_t target_stride, draft_stride;
  int K, V;
};

constexpr int kVThreads = 512, kVWarps = kVThreads / 32;
constexpr int kVRun = 25;                       // elements of a thread's run (odd: no bank conflicts)
constexpr int kVTile = kVThreads * kVRun;       // elements of a staged tile
constexpr int kVMaxTiles = 128;                 // tiles of a slice
constexpr int kVMaxVocab = 1 << 24;
constexpr size_t kVSmem = 2ull * kVTile * sizeof(float);

// d = max(p - q, 0) as s + e exactly (s the rounded difference); weights that
// are not finite count as 0.
__device__ __forceinline__ void weight(float p, float q, float& s, float& e) {
  s = p - q;
  const float bb = s - p;
  e = (p - (s - bb)) - (q + bb);
  if (!(s > 0.f && s <= FLT_MAX)) s = e = 0.f;
}

// The first position whose running sum passes the threshold and whose own sum
// is positive; the last positive one where rounding leaves none; -1 for no
// positive one.
__device__ __forceinline__ int pick(uint32_t over, uint32_t positive) {
  const uint32_t m = over & positive;
  return m ? __ffs(m) - 1 : positive ? 31 - __clz(positive) : -1;
}

// Inclusive scan over the warp's lanes.
__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

__global__ void __launch_bounds__(kVThreads, 1) verify_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / nc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  extern __shared__ float smem_v[];
  float* sp = smem_v;
  float* sq = smem_v + kVTile;
  __shared__ double s_slice;              // this CTA's slice sum, read by the cluster
  __shared__ double s_warp[kVWarps];
  __shared__ double s_tile[kVMaxTiles];
  __shared__ int s_n;
  griddep_wait();  // launched with programmatic stream serialization
  griddep_launch_dependents();

  // ---- acceptance (every CTA for itself) --------------------------------------
  const int K = a.K, V = a.V;
  int Kb = a.draft_len ? a.draft_len[b] : K;
  Kb = min(max(Kb, 0), K);
  const float* prow0 = a.target + static_cast<int64_t>(b) * (K + 1) * a.target_stride;
  const float* qrow0 = a.draft ? a.draft + static_cast<int64_t>(b) * K * a.draft_stride : nullptr;
  const float* u = a.u + static_cast<int64_t>(b) * (K + 1);
  if (warp == 0) {
    int n = Kb;
    for (int i0 = 0; i0 < Kb; i0 += 32) {
      const int i = i0 + lane;
      bool ok = false;
      if (i < Kb) {
        const int x = a.tokens[static_cast<int64_t>(b) * K + i];
        if (x >= 0 && x < V) {
          const float p = prow0[i * a.target_stride + x];
          const float q = qrow0 ? qrow0[i * a.draft_stride + x] : 1.f;
          ok = static_cast<double>(u[i]) * static_cast<double>(q) < static_cast<double>(p);
        } else if (rank == 0) {
          set_status(a.status, NK_STATUS_TOKEN_RANGE);
        }
      }
      const uint32_t no = __ballot_sync(0xffffffffu, !ok && i < Kb);
      if (no) {
        n = i0 + __ffs(no) - 1;
        break;
      }
    }
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  const bool cut = n < Kb;
  const float* prow = prow0 + n * a.target_stride;
  const float* qrow = cut && qrow0 ? qrow0 + n * a.draft_stride : nullptr;
  const int certain = cut && !qrow0 ? a.tokens[static_cast<int64_t>(b) * K + n] : -1;  // weight 0

  // ---- this CTA's slice ---------------------------------------------------------
  const int per = (V + nc - 1) / nc;
  const int lo = min(rank * per, V), hi = min(lo + per, V);
  const int tiles = (hi - lo + kVTile - 1) / kVTile;

  // Stages tile t; elements past the slice weigh 0.
  auto stage = [&](int t, bool residual) {
    const int at = lo + t * kVTile;
#pragma unroll 5
    for (int k = 0; k < kVRun; ++k) {
      const int j = at + k * kVThreads + tid;
      const bool in = j < hi && !(residual && j == certain);
      sp[k * kVThreads + tid] = in ? prow[j] : 0.f;
      sq[k * kVThreads + tid] = in && residual && qrow ? qrow[j] : 0.f;
    }
  };
  // The sum of this thread's run of the staged tile.
  auto run_sum = [&]() {
    float h = 0.f, l = 0.f;
#pragma unroll 5
    for (int k = 0; k < kVRun; ++k) {
      float s, e;
      weight(sp[tid * kVRun + k], sq[tid * kVRun + k], s, e);
      const float t = h + s, bb = t - h;
      l += (h - (t - bb)) + (s - bb) + e;
      h = t;
    }
    return static_cast<double>(h) + static_cast<double>(l);
  };

  int token = -1;
  // The residual weights; where they are all zero (p_n and q_n equal in every
  // token they give weight to) the target's own.
  for (int pass = 0; pass < 2; ++pass) {
    const bool residual = pass == 0 && cut;
    double mine = 0.0;   // sum of the last staged tile's run
    double scan = 0.0;   // inclusive scan of the runs in this warp
    double slice = 0.0;
    for (int t = 0; t < tiles; ++t) {
      stage(t, residual);
      __syncthreads();
      mine = run_sum();
      scan = warp_scan(mine, lane);
      if (lane == 31) s_warp[warp] = scan;
      __syncthreads();
      double tile = 0.0;
#pragma unroll
      for (int w = 0; w < kVWarps; ++w) tile += s_warp[w];
      if (tid == 0) s_tile[t] = tile;
      slice += tile;
      if (t + 1 < tiles) __syncthreads();  // s_warp and the tile are read before they are overwritten
    }
    if (tid == 0) s_slice = slice;
    cluster.sync();
    // the slice sums of the cluster, one per lane, scanned by every warp alike
    const double part = lane < nc ? *cluster.map_shared_rank(&s_slice, lane) : 0.0;
    const double incl = warp_scan(part, lane);
    const double total = __shfl_sync(0xffffffffu, incl, 31);
    const double border = static_cast<double>(u[K]) * total;
    const int owner = pick(__ballot_sync(0xffffffffu, incl > border), __ballot_sync(0xffffffffu, part > 0.0));
    const double before_owner = __shfl_sync(0xffffffffu, incl - part, max(owner, 0));
    cluster.sync();  // every slice sum has been read before a second pass or an exit
    if (owner >= 0) {
      if (owner == rank) {
        // the tile that holds the border (all threads alike)
        double base = before_owner;
        int t = -1, last = -1;
        double last_base = base;
        for (int k = 0; k < tiles; ++k) {
          const double x = s_tile[k];
          if (x > 0.0) {
            last = k;
            last_base = base;
            if (base + x > border) {
              t = k;
              break;
            }
          }
          base += x;
        }
        if (t < 0) t = last, base = last_base;
        if (t != tiles - 1) {  // not the staged one any more
          __syncthreads();
          stage(t, residual);
          __syncthreads();
          mine = run_sum();
          scan = warp_scan(mine, lane);
          if (lane == 31) s_warp[warp] = scan;
          __syncthreads();
        }
        const double ws = lane < kVWarps ? s_warp[lane] : 0.0;
        const double wincl = warp_scan(ws, lane);
        const int w = pick(__ballot_sync(0xffffffffu, base + wincl > border), __ballot_sync(0xffffffffu, ws > 0.0));
        const double wbase = base + __shfl_sync(0xffffffffu, wincl - ws, max(w, 0));
        if (warp == w) {
          const int ln = pick(__ballot_sync(0xffffffffu, wbase + scan > border), __ballot_sync(0xffffffffu, mine > 0.0));
          const double lbase = wbase + __shfl_sync(0xffffffffu, scan - mine, max(ln, 0));
          // that lane's run, one element per lane
          const int e0 = (warp * 32 + max(ln, 0)) * kVRun;
          float s = 0.f, e = 0.f;
          if (lane < kVRun) weight(sp[e0 + lane], sq[e0 + lane], s, e);
          const double d = static_cast<double>(s) + static_cast<double>(e);
          const double dincl = warp_scan(d, lane);
          const int el = pick(__ballot_sync(0xffffffffu, lbase + dincl > border), __ballot_sync(0xffffffffu, d > 0.0));
          token = lo + t * kVTile + e0 + max(el, 0);
          if (lane == 0) a.out[static_cast<int64_t>(b) * (K + 1) + n] = token;
        }
      }
      token = 0;  // found (by the owner)
      break;
    }
    if (!cut) break;
  }

  if (rank == 0) {
    for (int i = tid; i <= K; i += kVThreads) {
      int32_t* o = a.out + static_cast<int64_t>(b) * (K + 1) + i;
      if (i < n) *o = a.tokens[static_cast<int64_t>(b) * K + i];
      else if (i > n) *o = -1;
      else if (token < 0) *o = -1;  // no weight anywhere
    }
    if (tid == 0) {
      a.accepted[b] = n;
      if (a.frontiers_out) a.frontiers_out[b] = a.frontiers[b] - (Kb - n);
      if (token < 0) set_status(a.status, NK_STATUS_TOKEN_RANGE);
    }
  }
}

}  // namespace nk

using namespace nk;

extern "C" int nk_verify_drafts(const float* target, int64_t target_stride, const float* draft,
                                int64_t draft_stride, const int32_t* tokens, const int32_t* draft_len,
                                const float* uniforms, const int32_t* frontiers, int32_t B, int32_t K,
                                int32_t V, int32_t* accepted, int32_t* out_tokens, int32_t* frontiers_out,
                                void* stream) {
  clear_error();
  if (!target || !uniforms || !accepted || !out_tokens)
    return fail(NK_ERR_INVALID_ARG, "null argument to nk_verify_drafts");
  if ((frontiers != nullptr) != (frontiers_out != nullptr))
    return fail(NK_ERR_INVALID_ARG, "frontiers and frontiers_out come together");
  if (B < 1 || B > (1 << 20)) return fail(NK_ERR_SHAPE, "B must be in [1, 2^20]");
  if (K < 0 || K > 1024) return fail(NK_ERR_SHAPE, "K must be in [0, 1024]");
  if (V < 1 || V > kVMaxVocab) return fail(NK_ERR_SHAPE, "V must be in [1, 2^24]");
  if (K > 0 && !tokens) return fail(NK_ERR_INVALID_ARG, "drafted tokens are NULL");
  if (target_stride < V || (draft && draft_stride < V))
    return fail(NK_ERR_SHAPE, "row strides must be at least V");
  VerifyArgs a;
  a.target = target;
  a.draft = K > 0 ? draft : nullptr;
  a.tokens = tokens;
  a.draft_len = draft_len;
  a.u = uniforms;
  a.frontiers = frontiers;
  a.accepted = accepted;
  a.out = out_tokens;
  a.frontiers_out = frontiers_out;
  a.status = status_word();
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.K = K;
  a.V = V;
  if (!a.status) return fail(NK_ERR_CUDA, "status word address unavailable");
  cudaError_t e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kVSmem));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return cuda_fail(e, "verify attributes");
  // CTAs per sequence: enough that a slice is one tile, at most 16
  int nc = 1;
  while (nc < 16 && static_cast<int64_t>(nc) * kVTile < V) nc *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * nc);
  cfg.blockDim = dim3(kVThreads);
  cfg.dynamicSmemBytes = kVSmem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, verify_kernel, a);
  if (e != cudaSuccess) return cuda_fail(e, "verify launch");
  return NK_OK;
}
