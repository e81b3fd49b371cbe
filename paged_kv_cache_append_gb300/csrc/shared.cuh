// shared.cuh -- what the kernels of the shared-prefix attention agree on.
//
// A batch's rows share their first `pages` pages.  Row b takes part iff there
// are enough of them to gain by it and every one of its query tokens sees all
// of them (F_b - T >= 64 * pages); its keys
// are then the shared pages, attended once for all rows by the prefix pass,
// and its own pages from there on, attended by the decode kernels with the
// row's table and frontier moved by `pages`.  A row that does not take part
// is attended by the decode kernels alone, from its first page.
#pragma once

#include "device.cuh"

namespace nk {

struct SharedPrefix {
  const int32_t* pages = nullptr;  // device, one value; nullptr: no shared prefix
  const int32_t* frontiers = nullptr;
  int B = 0, T = 0;
  int least = 1;  // fewer shared pages than this are not worth a pass of their own
};

// Where the prefix pass leaves its partials: of page range `split` of `nsplit`
// and tile of 128 query rows, for every KV head.
struct PrefixParts {
  int tiles, nsplit;
  float2* ml;  // [H][tiles][nsplit][128] (m, l), O relative to 2^m
  float* o;    // [H][tiles][nsplit][128][D]
};

__device__ __forceinline__ bool takes_part(int pages, int least, int F, int row, int T, int L, int C) {
  return pages >= least && pages <= L && F >= T && F <= L * 64 && F - T >= 64 * pages && row >= 0 && row < C;
}

// The table row whose pages the prefix pass reads: the first one that takes
// part (they all name the same pages), -1 for none.
__device__ __forceinline__ int prefix_row(const SharedPrefix& sh, const int32_t* table_rows, int pages, int L, int C) {
  int F[8], row[8], found = -1;
#pragma unroll
  for (int b = 0; b < 8; ++b) {  // no load waits for another
    F[b] = b < sh.B ? sh.frontiers[b] : 0;
    row[b] = b < sh.B ? table_rows[b] : -1;
  }
#pragma unroll
  for (int b = 7; b >= 0; --b)
    if (takes_part(pages, sh.least, F[b], row[b], sh.T, L, C)) found = row[b];
  return found;
}

}  // namespace nk
