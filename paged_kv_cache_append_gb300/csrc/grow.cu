// grow.cu -- the pages of a step from the requests' lengths: block tables,
// frontiers, positions and slot maps on the device (nk_pages_grow).
//
// At most 8 rows take part, so the plan (how many pages each row returns or
// takes, and where on the stack) is eight lanes' work: one warp loads the rows'
// numbers and walks the batch with shuffles.  With
//   top0 = free pages before, top1 = top0 + all returned pages,
// page p of a returning row lands at base_b + (mapped_b - 1 - p), and the j-th
// page that row b takes is entry top_b - 1 - j of that virtual stack; entries
// from top0 on are still in the tables of the rows that returned them.  No entry
// that a thread reads is one that another writes: taken entries lie below top0
// or in returning rows' tables, written ones from top0 on or in taking rows'.
//
// What bounds it: the chain launch -> table_rows -> mapped -> pages, and for
// prompts the moves of the pages, row after row in the one CTA that does the tables
// (8 rows of 2048 pages: 12.4 us; of 64: 7.0), where a load of a page id waits for the
// store before it.  Slots of more tokens than that CTA writes in the time of a launch
// go to a second kernel.
#include "device.cuh"
#include "internal.h"

namespace nk {

struct GrowArgs {
  int32_t* tables;
  const int32_t* table_rows;
  const int32_t* committed;
  const int32_t* counts;  // nullptr: T each
  const int32_t* keep;    // nullptr: 0
  const int32_t* mapped;
  int32_t* mapped_out;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* frontiers;
  int32_t* positions;
  int64_t* slots;
  int* status;
  int B, T, L, M, C;
};

constexpr int kGrowThreads = 512;

// Position and slot of token t of a row with frontier F (0: refused) and n new
// tokens, whose table is `table`.
__device__ __forceinline__ void write_token(const GrowArgs& a, int64_t at, int t, int F, int n, const int32_t* table) {
  const bool live = F > 0 && t < n;
  const int pos = live ? F - n + t : -1;
  if (a.positions) a.positions[at] = pos;
  if (a.slots) a.slots[at] = live ? static_cast<int64_t>(table[pos >> 6]) * 64 + (pos & 63) : -1;
}

__global__ void __launch_bounds__(kGrowThreads) grow_kernel(GrowArgs a, bool tokens, bool last) {
  __shared__ int s_row[8], s_F[8], s_n[8], s_have[8], s_gone[8], s_base[8], s_take[8], s_top[8];
  __shared__ int s_top0;
  const int tid = threadIdx.x, lane = tid & 31;
  griddep_wait();  // lengths and tables may come from the kernel ahead
  // The fused append + decode reads tables and frontiers before its wait: the
  // kernel behind may start early only where it is the token kernel.
  if (!last) griddep_launch_dependents();
  if (tid < 32) {
    const bool in = lane < a.B;
    const int row = in ? a.table_rows[lane] : -1;
    const int64_t have = in ? a.committed[lane] : 0;
    const int n = in ? (a.counts ? a.counts[lane] : a.T) : 0;
    const int freed0 = *a.free_count;
    bool ok = in && row >= 0 && row < a.C;
    const int mapped = ok ? a.mapped[row] : 0;
    const int keep = ok && a.keep ? a.keep[row] : 0;
    // every row's value, read by all before any is written (the arrays may be the same)
    const int old = lane < a.C ? a.mapped[lane] : 0;
    for (int i = 0; i < a.B; ++i) {
      const int other = __shfl_sync(0xffffffffu, row, i);
      if (i < lane && other == row) ok = false;
    }
    ok = ok && have >= 0 && n >= 0 && n <= a.T && have + n <= static_cast<int64_t>(a.L) * 64 && mapped >= 0 &&
         mapped <= a.L;
    if (in && !ok) set_status(a.status, NK_STATUS_FRONTIER);
    const bool stack = freed0 >= 0 && freed0 <= a.M;
    if (lane == 0 && !stack) set_status(a.status, NK_STATUS_PAGE_RANGE);
    const int top0 = stack ? freed0 : 0;
    const int need = ok ? static_cast<int>((have + n + 63) >> 6) : 0;
    int gone = ok ? max(0, mapped - max(need, keep)) : 0;
    int take = ok ? max(0, need - mapped) : 0;
    int top = top0, base = 0, from = 0;
    for (int i = a.B - 1; i >= 0; --i) {
      const int g = __shfl_sync(0xffffffffu, gone, i);
      const bool fits = stack && g <= a.M - top;  // more pages than the pool has: an inconsistent stack
      if (lane == i) {
        base = top;
        if (!fits && g) {
          gone = 0;
          set_status(a.status, NK_STATUS_PAGE_RANGE);
        }
      }
      if (fits) top += g;
    }
    for (int i = 0; i < a.B; ++i) {
      const int want = __shfl_sync(0xffffffffu, take, i);
      if (want > top) {
        if (lane == i) {
          ok = false;
          take = 0;
          set_status(a.status, NK_STATUS_PAGES);
        }
      } else {
        if (lane == i) from = top;
        top -= want;
      }
    }
    if (in) {
      s_row[lane] = row;
      s_F[lane] = ok ? static_cast<int>(have) + n : 0;
      s_n[lane] = n;
      s_have[lane] = mapped;
      s_gone[lane] = gone;
      s_base[lane] = base;
      s_take[lane] = take;
      s_top[lane] = from;
      a.frontiers[lane] = s_F[lane];
    }
    if (lane == 0) {
      s_top0 = top0;
      *a.free_count_out = stack ? top : freed0;
    }
    int now = old;
    for (int i = 0; i < a.B; ++i) {
      const int r = __shfl_sync(0xffffffffu, row, i);
      const int v = __shfl_sync(0xffffffffu, mapped - gone + take, i);
      const bool moved = __shfl_sync(0xffffffffu, static_cast<int>(gone | take), i) != 0;
      if (moved && r == lane) now = v;
    }
    if (lane < a.C) a.mapped_out[lane] = now;
  }
  __syncthreads();
  for (int b = 0; b < a.B; ++b) {
    int32_t* table = a.tables + static_cast<int64_t>(s_row[b]) * a.L;  // read and written where a row is served
    const int have = s_have[b], gone = s_gone[b], take = s_take[b];
    for (int i = tid; i < gone; i += kGrowThreads) a.free_pages[s_base[b] + i] = table[have - 1 - i];
    for (int i = tid; i < take; i += kGrowThreads) {
      const int at = s_top[b] - 1 - i;
      int page;
      if (at < s_top0) {
        page = a.free_pages[at];
      } else {
        page = 0;
        for (int r = 0; r < a.B; ++r)
          if (at >= s_base[r] && at < s_base[r] + s_gone[r])
            page = a.tables[static_cast<int64_t>(s_row[r]) * a.L + s_have[r] - 1 - (at - s_base[r])];
      }
      table[have + i] = page;
    }
  }
  if (tokens) {
    __syncthreads();  // this CTA's own table entries
    for (int i = tid; i < a.B * a.T; i += kGrowThreads) {
      const int b = i / a.T;
      write_token(a, i, i - b * a.T, s_F[b], s_n[b], a.tables + static_cast<int64_t>(s_row[b]) * a.L);
    }
  }
  __threadfence();  // in L2 before the kernel behind starts
}

constexpr int kTokenThreads = 256, kTokenEach = 4;

// Positions and slots of one row, from the tables and frontiers just written.
__global__ void __launch_bounds__(kTokenThreads) grow_tokens_kernel(GrowArgs a) {
  griddep_wait();  // and lets nothing start before its end, for the same reason
  const int b = blockIdx.y;
  const int F = a.frontiers[b], row = a.table_rows[b], n = a.counts ? a.counts[b] : a.T;
  const int32_t* table = a.tables + static_cast<int64_t>(F > 0 ? row : 0) * a.L;
  const int t0 = blockIdx.x * (kTokenThreads * kTokenEach) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kTokenEach; ++i) {
    const int t = t0 + i * kTokenThreads;
    if (t < a.T) write_token(a, static_cast<int64_t>(b) * a.T + t, t, F, n, table);
  }
}

// Up to here the one CTA of the tables writes the tokens too.  Fresh rows, us a call, one
// launch and two: 8 x 128 tokens 5.4 and 5.8, 8 x 256 6.2 and 6.1, 8 x 512 7.1 and 6.3,
// 8 x 4096 16.5 and 7.0.
constexpr int64_t kTokensInOne = 2048;

}  // namespace nk

using namespace nk;

extern "C" int nk_pages_grow(const nk_pool* pool, int32_t* block_tables, const int32_t* table_rows,
                             const int32_t* committed, const int32_t* counts, const int32_t* keep,
                             const int32_t* mapped, int32_t* mapped_out, int32_t* free_pages,
                             const int32_t* free_count, int32_t* free_count_out, int32_t B, int32_t T,
                             int32_t* frontiers, int32_t* positions, int64_t* slots, void* stream) {
  clear_error();
  if (!pool || !block_tables || !table_rows || !committed || !mapped || !mapped_out || !free_pages || !free_count ||
      !free_count_out || !frontiers)
    return fail(NK_ERR_INVALID_ARG, "null argument to nk_pages_grow");
  if (B < 1 || B > pool->desc.max_concurrency) return fail(NK_ERR_SHAPE, "B must be in [1, C]");
  if (T < 0 || static_cast<int64_t>(B) * T > (int64_t(1) << 30)) return fail(NK_ERR_SHAPE, "T must be >= 0, B * T <= 2^30");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != pool->device)
    return fail(NK_ERR_INVALID_ARG, "the pool belongs to device " + std::to_string(pool->device) +
                                        ", the current device is " + std::to_string(dev));
  const GrowArgs a{block_tables, table_rows, committed, counts, keep, mapped, mapped_out, free_pages, free_count,
                   free_count_out, frontiers, positions, slots, pool->status, B, T, pool->L, pool->M,
                   pool->desc.max_concurrency};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t n = positions || slots ? static_cast<int64_t>(B) * T : 0;
  const bool in_one = n <= kTokensInOne;
  e = launch_pdl(grow_kernel, dim3(1), dim3(kGrowThreads), 0, s, a, n > 0 && in_one, in_one);
  if (e == cudaSuccess && !in_one) {
    const int per = kTokenThreads * kTokenEach;
    e = launch_pdl(grow_tokens_kernel, dim3((T + per - 1) / per, B), dim3(kTokenThreads), 0, s, a);
  }
  if (e != cudaSuccess) return cuda_fail(e, "page growth launch");
  return NK_OK;
}
