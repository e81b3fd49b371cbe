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

// How a call divides the SMs, which all of its kernels work out for themselves
// from the same lengths: the prefix pass and the rows' own pages one after the
// other on all SMs, or at once, each on SMs of its own (their CTAs do not fit
// one SM together), where that is expected to take less time.  At once hides
// the start and the tail of one behind the other: 8 rows of one token over 480
// FP8-row pages and 2000 own tokens take 26.5 us against 30.6, 4 tokens over 1920
// K8V4 pages and 8000 own tokens 107 against 112, over 128 pages and 700 own
// tokens 28.4 against 36.8; but 225 against 189 over 2000 NVFP4 pages of
// head_dim 256 and 64 own tokens, whose rows need 32 SMs for their CTAs alone.
// Working this out costs about 1 us a call.
struct ShareShape {
  int sms = 0;
  int range_ctas = 0;  // prefix CTAs of a page range: KV heads, times tiles where a CTA takes one
  int nsplit = 0;      // page ranges at most
  int ctas = 0;        // own-pages CTAs of a KV head at most
  int least = 0;       // SMs on which every row has a CTA per head
  float ranges_per_sm = 0.f, ctas_per_sm = 0.f;  // 1 / range_ctas; own-pages CTAs of a head per SM
  // rows of equal length use whole multiples of `step` SMs, of all SMs all_sms
  float step = 0.f, all_sms = 0.f;
  // in units of the prefix pass's time for a page: own_page of a row's own page
  // of all heads on one SM, own_start of the own-pages kernel without any page,
  // turn_start of it when it follows the prefix pass
  float own_page = 0.f, own_start = 0.f, turn_start = 0.f;
};

struct SharedPrefix {
  const int32_t* pages = nullptr;  // device, one value; nullptr: no shared prefix
  const int32_t* frontiers = nullptr;
  int B = 0, T = 0;
  int least = 1;  // fewer shared pages than this are not worth a pass of their own
  ShareShape shape;
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

// Pages of row (F, row) that the decode kernels attend, the first `pages` of a
// row that takes part (`part`) being the prefix pass's.
__device__ __forceinline__ int own_pages(int pages, bool part, int F, int row, int L, int C) {
  return F < 0 || F > L * 64 || row < 0 || row >= C ? 0 : ((F + 63) >> 6) - (part ? pages : 0);
}

struct ShareSplit {
  int nsplit;  // page ranges
  int ctas;    // own-pages CTAs of a KV head
};

// (No operation here may be contracted with another: the kernels have to agree.
// Half a unit on top keeps the quotients of small whole numbers away from whole
// numbers.)
__device__ __forceinline__ ShareSplit share_split(const ShareShape& g, int pages, int own) {
  if (pages <= 0) return ShareSplit{g.nsplit, g.ctas};
  constexpr float kPrefixStart = 4.f, kTail = 3.f;
  const float pre_work = __fmul_rn(pages, g.range_ctas), own_work = __fmul_rn(own, g.own_page);
  const int give = max(__float2int_rz(__fdividef(__fmul_rn(g.sms, own_work), __fadd_rn(pre_work, own_work))) + 1, g.least);
  const int nsplit = min(__float2int_rz(__fmul_rn(__fadd_rn(g.sms - give, 0.5f), g.ranges_per_sm)), g.nsplit);
  if (nsplit < 1) return ShareSplit{g.nsplit, g.ctas};
  const int per = (pages + nsplit - 1) / nsplit, used = (pages + per - 1) / per;
  const int left = g.sms - used * g.range_ctas;
  const float busy = __fmul_rn(floorf(__fdividef(__fadd_rn(left, 0.01f), g.step)), g.step);
  const float at_once = __fadd_rn(
      kTail, fmaxf(__fadd_rn(kPrefixStart, per), __fadd_rn(g.own_start, __fdividef(own_work, busy))));
  const float in_turn = __fadd_rn(__fadd_rn(kPrefixStart, __fdividef(pages, g.nsplit)),
                                  __fadd_rn(g.turn_start, __fdividef(own_work, g.all_sms)));
  if (!(at_once < in_turn)) return ShareSplit{g.nsplit, g.ctas};
  return ShareSplit{nsplit, min(__float2int_rz(__fmul_rn(__fadd_rn(left, 0.001f), g.ctas_per_sm)), g.ctas)};
}

// The table row whose pages the prefix pass reads: the first one that takes
// part (they all name the same pages), -1 for none; and all rows' own pages.
__device__ __forceinline__ int prefix_row(const SharedPrefix& sh, const int32_t* table_rows, int pages, int L, int C,
                                          int& own) {
  int F[8], row[8], found = -1;
#pragma unroll
  for (int b = 0; b < 8; ++b) {  // no load waits for another
    F[b] = b < sh.B ? sh.frontiers[b] : 0;
    row[b] = b < sh.B ? table_rows[b] : -1;
  }
  own = 0;
#pragma unroll
  for (int b = 7; b >= 0; --b) {
    const bool part = takes_part(pages, sh.least, F[b], row[b], sh.T, L, C);
    if (part) found = row[b];
    own += own_pages(pages, part, F[b], row[b], L, C);
  }
  return found;
}

// A row of the batch as the own-pages kernels take it.
struct OwnRow {
  int F, row, before;  // frontier, table row, pages that the prefix pass attends
};

// Lane b's row, and the own-pages CTAs of a KV head, by a whole warp before
// anything is set up: a CTA that gets nothing leaves at once (it may start only
// when the prefix pass ends, and the merge waits for it).
__device__ __forceinline__ OwnRow own_row(const ShareShape& g, const int32_t* shared, int least,
                                          const int32_t* frontiers, const int32_t* table_rows, int B, int T, int L,
                                          int C, int lane, int& ctas) {
  const int pages = *shared, F = lane < B ? frontiers[lane] : 0, row = lane < B ? table_rows[lane] : -1;
  const bool part = lane < B && takes_part(pages, least, F, row, T, L, C);
  const int own = __reduce_add_sync(0xffffffffu, own_pages(pages, part, F, row, L, C));
  ctas = share_split(g, __any_sync(0xffffffffu, part) ? pages : 0, own).ctas;
  return OwnRow{F, row, part ? pages : 0};
}

}  // namespace nk
