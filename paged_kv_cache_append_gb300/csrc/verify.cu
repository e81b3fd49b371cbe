// verify.cu -- verification of drafted tokens against the target model's
// probabilities, from given random numbers.
//
// Sequence b has K_b <= K drafts x_0 .. x_{K_b - 1}, the target's rows p_0 ..
// p_{K_b} and the draft model's rows q_0 .. q_{K_b - 1} (without them each
// draft is taken as certain: q_i is 1 at x_i).  Draft i is accepted iff
//   u_i q_i(x_i) < p_i(x_i)
// (compared exactly: the rounded product and its error); n is the first draft
// that is not, K_b if there is none.  The next token is drawn by inverse
// transform from the weights
//   d_j = max(p_n(j) - q_n(j), 0)  (n < K_b),   d_j = p_n(j)  (n = K_b):
// the least j with d_0 + .. + d_j > u_K (d_0 + .. + d_{V-1}).
//
// The sums decide at borders whose distance is a token's own probability, so
// they are held in more than fp32, as unevaluated pairs of fp32 values (Knuth's
// TwoSum on every difference and every addition), two elements to a packed
// instruction; a lane's sum over many blocks has a third value.  With u = 2^-24
// and every addition of two pairs of positive values good to 3 u^2, a lane's
// blocks are off by at most 13 u^2 of their sum, whatever their number; its two
// halves and the tail, the five levels over a warp, the four over its CTA and the
// three over the cluster add 43 to that, the steps of the search and the last 8
// tokens 36, and the border has the first 56 and 3 of its own: a running sum and
// its border are compared to within 2^-40 of the total.  Where roundings do not
// conspire it is 2^-47 (log-normal weights, up to 2^24 tokens).
//
// One cluster of CTAs works on a sequence.  Its warps take contiguous chunks of
// the vocabulary and read them with coalesced 4-byte loads (rows of an odd
// vocabulary are not 16-byte aligned), every lane adding its own stride, so
// nothing is staged and the loads of many warps are in flight.  The CTAs' sums
// meet over distributed shared memory.  What follows is serial and short, so
// one warp does it: it finds whose slice holds the border and, in that CTA,
// the warp chunk from the chunk sums that were kept; the chunk is read again
// (some KB, from L2), a long one in W contiguous parts by all warps; and the
// last part is scanned 256 elements at a time, 8 consecutive ones a lane.
#include <cfloat>

#include <cooperative_groups.h>

#include "device.cuh"
#include "internal.h"
#include "packed.cuh"

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

constexpr int kVMaxWarps = 16;
constexpr int kVMaxVocab = 1 << 24;

// A sum held as an unevaluated pair of fp32 values.
struct Pair {
  float h, l;
};

__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const float t = a.h + b.h, bb = t - a.h;
  const float l = ((a.h - (t - bb)) + (b.h - bb)) + (a.l + b.l);
  const float h = t + l;
  return Pair{h, l - (h - t)};
}

__device__ __forceinline__ bool pair_greater(Pair a, Pair b) {
  const float t = a.h - b.h, bb = t - a.h;
  return t + (((a.h - (t - bb)) - (b.h + bb)) + (a.l - b.l)) > 0.f;
}

// u * a: the rounding error of the first product is in the second value.
__device__ __forceinline__ Pair pair_scale(Pair a, float u) {
  const float t = u * a.h, e = fmaf(u, a.h, -t) + u * a.l;
  const float h = t + e;
  return Pair{h, e - (h - t)};
}

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
__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, x.h, off), __shfl_up_sync(0xffffffffu, x.l, off)};
    if (lane >= off) x = pair_add(y, x);
  }
  return x;
}

__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    x = pair_add(x, Pair{__shfl_xor_sync(0xffffffffu, x.h, off), __shfl_xor_sync(0xffffffffu, x.l, off)});
  return x;
}

__device__ __forceinline__ Pair shuffle(Pair x, int lane) {
  return Pair{__shfl_sync(0xffffffffu, x.h, lane), __shfl_sync(0xffffffffu, x.l, lane)};
}

// One level of the search, done alike by every warp that calls it: lane i holds
// the sum of part i and all parts follow `base`.  Returns the part with the
// border (-1 for none with weight) and moves `base` to where it begins.
__device__ __forceinline__ int find(Pair part, Pair border, int lane, Pair& base) {
  const Pair at = pair_add(base, warp_scan(part, lane));
  const uint32_t over = __ballot_sync(0xffffffffu, pair_greater(at, border));
  const int i = pick(over, __ballot_sync(0xffffffffu, part.h > 0.f));
  const Pair before = shuffle(at, max(i - 1, 0));
  if (i > 0) base = before;
  return i;
}

// u q < p without rounding: the product and its error, or fp64 where they
// could underflow.
__device__ __forceinline__ bool accepts(float u, float q, float p) {
  const float t = u * q;
  if (fabsf(t) < 1e-30f) return static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
  return t < p || (t == p && fmaf(u, q, -t) < 0.f);
}

// The weights of one sequence's next token.
struct Weights {
  const float* p;
  const float* q;  // nullptr: none is taken off
  int zero;        // a token without weight (-1: none)

  __device__ __forceinline__ void at(int j, int end, float& s, float& e) const {
    const bool in = j < end && j != zero;
    weight(in ? p[j] : 0.f, in && q ? q[j] : 0.f, s, e);
  }
};

// a + b as the rounded sum (returned) and its error.
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float t = a + b, bb = t - a;
  err = (a - (t - bb)) + (b - bb);
  return t;
}

__device__ __forceinline__ F2 two_sum(F2 a, F2 b, F2& err) {
  const F2 minus = pack2(-1.f, -1.f), t = add2(a, b), bb = fma2(a, minus, t);
  err = add2(fma2(fma2(bb, minus, t), minus, a), fma2(bb, minus, b));
  return t;
}

__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ F2 plus(F2 a, F2 b) { return add2(a, b); }

// A lane's running sum h + l + c of float or, two at once, F2, without rounding
// but in c, which holds what l lost: a pair would lose what is below 2^-24 of its
// second value, in every addition anew (up to 2^-30 of the sum over the 2048
// additions of a lane of the largest vocabulary: a few heavy tokens, then a
// long light tail).
template <class T>
struct Running {
  T h = T(0), l = T(0), c = T(0);

  __device__ __forceinline__ void add(T s, T e) {
    T e0, e1, e2;
    h = two_sum(h, s, e0);
    l = two_sum(l, e, e1);
    l = two_sum(l, e0, e2);
    c = plus(c, plus(e1, e2));
  }
};

__device__ __forceinline__ Pair pair_of(float h, float l, float c) {
  const float t = h + l;
  return Pair{t, (l - (t - h)) + c};
}

// h + l += s + e, exactly but for the last bits of l.
__device__ __forceinline__ void pair_acc(float& h, float& l, float s, float e) {
  float err;
  h = two_sum(h, s, err);
  l += err + e;
}

// The sum of one lane over its stride of [lo, hi), any elements, four at a time.
__device__ __forceinline__ Pair lane_sum(const Weights& w, int lo, int hi, int lane) {
  constexpr int U = 4;
  Running<float> sum;
  for (int j = lo + lane; j < hi; j += 32 * U) {
    float s[U], e[U], h = 0.f, l = 0.f;
#pragma unroll
    for (int k = 0; k < U; ++k) w.at(j + 32 * k, hi, s[k], e[k]);
#pragma unroll
    for (int k = 0; k < U; ++k) pair_acc(h, l, s[k], e[k]);
    if (j - lane == lo) sum.h = h, sum.l = l;
    else sum.add(h, l);
  }
  return pair_of(sum.h, sum.l, sum.c);
}

// The sum over [lo, hi) of one warp, in every lane.  Whole blocks of 256
// elements take the packed path: with m = max(p, q), m - q is the weight, 0
// where p <= q or p is NaN.  A lane adds the block's elements to a pair of its
// own, whose few roundings are below 2^-44 of the block, and the pair to its
// running sum.  Entries that are not finite leave a sum that is not, and the
// warp then does it over, element by element.
template <bool Q>
__device__ __forceinline__ Pair chunk_sum(const Weights& w, int lo, int hi, int lane) {
  constexpr int U = 8;
  Pair sum{0.f, 0.f};
  int j = lo;
  if (w.zero < lo || w.zero >= hi) {
    const F2 minus = pack2(-1.f, -1.f);
    Running<F2> run;
    for (; j + 32 * U <= hi; j += 32 * U) {
      float x[U], y[U];
#pragma unroll
      for (int k = 0; k < U; ++k) x[k] = __ldcs(w.p + j + 32 * k + lane);
#pragma unroll
      for (int k = 0; k < U; ++k) y[k] = Q ? __ldcs(w.q + j + 32 * k + lane) : 0.f;
      F2 bh = 0ull, bl = 0ull;  // the block
#pragma unroll
      for (int k = 0; k < U; k += 2) {
        const F2 m = pack2(fmaxf(x[k], y[k]), fmaxf(x[k + 1], y[k + 1]));
        F2 s = m, e = 0ull;
        if constexpr (Q) {
          const F2 q = pack2(y[k], y[k + 1]);
          s = fma2(q, minus, m);
          const F2 bb = fma2(m, minus, s);
          e = fma2(add2(q, bb), minus, fma2(fma2(bb, minus, s), minus, m));
        }
        if (k == 0) {
          bh = s;
          bl = e;
        } else {
          F2 err;
          bh = two_sum(bh, s, err);
          bl = add2(bl, Q ? add2(err, e) : err);
        }
      }
      if (j == lo) run.h = bh, run.l = bl;
      else run.add(bh, bl);
    }
    float h[2], l[2], c[2];
    unpack2(run.h, h[0], h[1]);
    unpack2(run.l, l[0], l[1]);
    unpack2(run.c, c[0], c[1]);
    sum = pair_add(pair_of(h[0], l[0], c[0]), pair_of(h[1], l[1], c[1]));
    if (!__all_sync(0xffffffffu, fabsf(sum.h) <= FLT_MAX && fabsf(sum.l) <= FLT_MAX)) {
      sum = Pair{0.f, 0.f};
      j = lo;
    }
  }
  if (j < hi) sum = pair_add(sum, lane_sum(w, j, hi, lane));
  return warp_sum(sum);
}

__device__ __forceinline__ Pair chunk_sum(const Weights& w, int lo, int hi, int lane) {
  return w.q ? chunk_sum<true>(w, lo, hi, lane) : chunk_sum<false>(w, lo, hi, lane);
}

// The token of [lo, hi) where the running sum from `base` on passes the border
// (the last one with weight if none does, -1 without weight), by one warp.
__device__ __forceinline__ int scan_token(const Weights& w, int lo, int hi, Pair base, Pair border, int lane) {
  constexpr int E = 8;
  int token = -1;
  Running<float> done;  // the blocks before j
  for (int j = lo; j < hi; j += 32 * E) {
    float s[E], e[E];
    Pair sum{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < E; ++k) w.at(j + E * lane + k, hi, s[k], e[k]);
#pragma unroll
    for (int k = 0; k < E; ++k) sum = pair_add(sum, Pair{s[k], e[k]});
    const Pair scan = warp_scan(sum, lane), start = pair_add(base, pair_of(done.h, done.l, done.c)), at = pair_add(start, scan);
    const uint32_t positive = __ballot_sync(0xffffffffu, sum.h > 0.f);
    const uint32_t over = __ballot_sync(0xffffffffu, pair_greater(at, border)) & positive;
    if (positive) {
      const int i = over ? __ffs(over) - 1 : 31 - __clz(positive);  // the lane that holds it
      const Pair before = shuffle(at, max(i - 1, 0));
      Pair run = i > 0 ? before : start;
      int last = -1, first = -1;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        run = pair_add(run, Pair{s[k], e[k]});
        if (s[k] > 0.f) {
          last = k;
          if (first < 0 && pair_greater(run, border)) first = k;
        }
      }
      token = j + E * i + __shfl_sync(0xffffffffu, first >= 0 ? first : last, i);
    }
    if (over) break;
    const Pair block = shuffle(scan, 31);
    done.add(block.h, block.l);
  }
  return token;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// CTAs of 32 W threads, W <= 16, in clusters that share a sequence.
__global__ void __launch_bounds__(512, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / nc;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, W = blockDim.x >> 5;
  __shared__ Pair s_slice;              // this CTA's sum, read by the cluster
  __shared__ Pair s_chunk[kVMaxWarps];  // the warp chunks' sums
  __shared__ Pair s_part[kVMaxWarps];   // the parts' sums of the chunk with the border
  __shared__ int s_owner, s_where;      // slice and warp chunk with the border
  griddep_wait();  // launched with programmatic stream serialization

  // ---- acceptance (every warp for itself) ---------------------------------------
  const int K = a.K, V = a.V;
  const float* prow0 = a.target + static_cast<int64_t>(b) * (K + 1) * a.target_stride;
  const float* qrow0 = a.draft ? a.draft + static_cast<int64_t>(b) * K * a.draft_stride : nullptr;
  const float* u = a.u + static_cast<int64_t>(b) * (K + 1);
  const int32_t* drafts = a.tokens + static_cast<int64_t>(b) * K;
  int Kb = a.draft_len ? a.draft_len[b] : K;
  Kb = min(max(Kb, 0), K);
  int n = Kb;
  for (int i0 = 0; i0 < K; i0 += 32) {
    const int i = i0 + lane;
    bool ok = false;
    if (i < K) {
      const int x = drafts[i];
      const float ui = u[i];
      if (x >= 0 && x < V) {
        const bool used = i < Kb;  // rows behind the last draft are not read
        const float p = used ? prow0[i * a.target_stride + x] : 0.f;
        const float q = !used ? 0.f : qrow0 ? qrow0[i * a.draft_stride + x] : 1.f;
        ok = accepts(ui, q, p);
      } else if (i < Kb && rank == 0 && warp == 0) {
        set_status(a.status, NK_STATUS_TOKEN_RANGE);
      }
    }
    const uint32_t no = __ballot_sync(0xffffffffu, !ok && i < Kb);
    if (no) {
      n = i0 + __ffs(no) - 1;
      break;
    }
  }
  const bool cut = n < Kb;
  // The trimmed length goes out before the next kernel may start: the fused
  // append + decode reads its frontiers while this one still runs.  The fence
  // makes it visible to the whole GPU first (the reader takes it from L2).
  if (tid == 0) {
    if (rank == 0 && a.frontiers_out) {
      a.frontiers_out[b] = a.frontiers[b] - (Kb - n);
      __threadfence();
    }
    griddep_launch_dependents();
  }

  // ---- this warp's chunk of this CTA's slice ----------------------------------------
  const int per = (V + nc - 1) / nc;
  const int lo = min(rank * per, V), hi = min(lo + per, V);
  const int cper = (hi - lo + W - 1) / W;
  const int c_lo = min(lo + warp * cper, hi), c_hi = min(c_lo + cper, hi);
  const bool parts = cper > 512;  // a chunk that one warp would scan for too long

  bool found = false;
  // The residual weights; where they are all zero (p_n and q_n equal in every
  // token they give weight to) the target's own.
  for (int pass = 0; pass < 2; ++pass) {
    const bool residual = pass == 0 && cut;
    Weights w;
    w.p = prow0 + n * a.target_stride;
    w.q = residual && qrow0 ? qrow0 + n * a.draft_stride : nullptr;
    w.zero = residual && !qrow0 ? drafts[n] : -1;
    const Pair sum = chunk_sum(w, c_lo, c_hi, lane);
    if (lane == 0) s_chunk[warp] = sum;
    __syncthreads();
    const Pair none{0.f, 0.f};
    Pair border = none, base = none, chunk = none;
    if (warp == 0) {
      chunk = lane < W ? s_chunk[lane] : none;
      const Pair all = warp_sum(chunk);
      if (lane == 0) s_slice = all;
    }
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      const Pair slice = lane < nc ? *cluster.map_shared_rank(&s_slice, lane) : none;
      border = pair_scale(warp_sum(slice), u[K]);
      const int owner = find(slice, border, lane, base);
      const int c = owner == rank ? max(find(chunk, border, lane, base), 0) : 0;
      if (lane == 0) {
        s_owner = owner;
        s_where = c;
      }
    }
    __syncthreads();
    cluster_arrive_relaxed();  // this CTA has read the slice sums
    const int owner = s_owner;
    found = owner >= 0;
    if (owner == rank) {
      const int b_lo = min(lo + s_where * cper, hi), b_hi = min(b_lo + cper, hi);  // the chunk with the border
      int p_lo = b_lo, p_hi = b_hi;
      if (parts) {
        const int pper = (b_hi - b_lo + W - 1) / W;
        const int m_lo = min(b_lo + warp * pper, b_hi);
        const Pair mine = chunk_sum(w, m_lo, min(m_lo + pper, b_hi), lane);
        if (lane == 0) s_part[warp] = mine;
        __syncthreads();
        if (warp == 0) {
          const int r = max(find(lane < W ? s_part[lane] : none, border, lane, base), 0);
          p_lo = min(b_lo + r * pper, b_hi);
          p_hi = min(p_lo + pper, b_hi);
        }
      }
      if (warp == 0) {
        const int token = scan_token(w, p_lo, p_hi, base, border, lane);
        if (lane == 0) a.out[static_cast<int64_t>(b) * (K + 1) + n] = token;
      }
    }
    cluster_wait();  // every CTA has read this one's sum: it may change, or the CTA end
    if (found || !cut) break;
  }

  if (rank == 0) {
    for (int i = tid; i <= K; i += 32 * W) {
      int32_t* o = a.out + static_cast<int64_t>(b) * (K + 1) + i;
      if (i < n) *o = drafts[i];
      else if (i > n || !found) *o = -1;  // i == n: no weight anywhere
    }
    if (tid == 0) {
      a.accepted[b] = n;
      if (!found) set_status(a.status, NK_STATUS_TOKEN_RANGE);
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
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int sms = device_sm_count(dev);
  // CTAs of 16 warps; 8 of them per sequence while all run at once, 4 beyond
  // (fewer, longer chunks: 64 sequences of 200003 tokens took 25.0 us with 4
  // and 28.7 with 8, 8 sequences of 131072 took 12.1 and 9.4), and fewer where
  // a warp would get less than 64 tokens
  constexpr int W = 16;
  int nc = static_cast<int64_t>(B) * 8 <= sms ? 8 : 4;
  while (nc > 1 && static_cast<int64_t>(nc) * W * 64 > V) nc /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B) * nc);
  cfg.blockDim = dim3(32 * W);
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
