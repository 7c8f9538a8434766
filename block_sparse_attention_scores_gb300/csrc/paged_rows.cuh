// The first work of the attentions over the paged cache: the workspace's header
// and the counters of finished parts are cleared, every new row's sequence and
// position found, and the rows that lead a tile listed. A row whose position lies
// outside the page table (or, behind a shared prefix, inside the prefix) is
// reported and left out.
//
// In front of the index scores a block of their kernel does this: nobody else in
// it needs the rows, and a kernel of its own costs two to four microseconds. The
// blocks there must not write the error word, which this clears: they leave what
// they find in `flags`, a word per block, and a later kernel reports it (so do
// the shared prefix's blocks).
#pragma once

#include "paged.h"
#include "paged_math.cuh"
#include "pdl.cuh"
#include "sm100.cuh"

namespace msa {

struct RowsArgs {
  const int32_t *row_start, *seq_len, *page_table;
  int4 *rows, *lead, *runs;
  int *arrived, *header;
  int S, N, n_arrived, max_blocks, prefix, tile_rows, run_rows;
  int check;  // pages of a shared prefix that are compared here, as no kernel of their own does
};

inline RowsArgs rows_args(const PagedProb& p, const PagedCachePtrs& c, uint8_t* ws, const PagedWs& L) {
  RowsArgs a;
  a.row_start = c.row_start;
  a.seq_len = c.seq_len;
  a.page_table = c.page_table;
  a.rows = reinterpret_cast<int4*>(ws + L.rows);
  a.lead = reinterpret_cast<int4*>(ws + L.lead);
  a.runs = reinterpret_cast<int4*>(ws + L.runs);
  a.arrived = reinterpret_cast<int*>(ws + L.arrived);
  a.header = reinterpret_cast<int*>(ws);
  a.S = p.S;
  a.N = p.N;
  a.n_arrived = L.splits > 1 ? p.N * p.G * 3 : 0;  // (few rows: others are not cut)
  a.max_blocks = p.max_blocks;
  a.prefix = p.prefix;
  a.tile_rows = L.tile_rows;
  a.run_rows = L.run_rows;
  a.check = p.prefix - L.prefix;
  return a;
}

constexpr int kStaged = 4000;  // sequence starts kept in shared memory
struct RowsShared {
  int staged[kStaged];
  int sums[32];
};

// The sequence of row r: the last s with row_start[s] <= r (the first counts as 0); S behind the last sequence.
template <class Start>
__device__ __forceinline__ int bisect_rows(const Start& start, int S, int r) {
  int lo = 0, hi = S + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same by a whole warp, 32 probes a step.
__device__ __forceinline__ int find_sequence(const int32_t* row_start, int S, int r, int lane) {
  int lo = 0, n = S + 1;  // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool in = lane == 0 || (lane * step < n && ld_in(row_start + at) <= r);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const int last = 31 - __clz(m);
    const int left = n - last * step;
    lo += last * step;
    n = left < step ? left : step;
  }
  return lo;
}

// By `threads` threads (whole warps, tid counted among them), which `sync` brings together.
template <class Sync>
__device__ __forceinline__ void line_up_rows(const RowsArgs& a, RowsShared& sh, int tid, int threads, const Sync& sync) {
  const int lane = tid & 31, warp = tid >> 5;
  const bool all = a.S + 1 <= kStaged;
  for (int i = tid; i < 64; i += threads) a.header[i] = 0;
  if (all)
    for (int i = tid; i <= a.S; i += threads) sh.staged[i] = ld_in(a.row_start + i);
  for (int i = tid; i < a.n_arrived; i += threads) a.arrived[i] = 0;
  sync();
  auto start = [&](int i) { return all ? sh.staged[i] : ld_in(a.row_start + i); };
  if (a.check) {
    const int ref = bisect_rows(start, a.S, 0);  // the first sequence with rows
    bool bad = false;
    for (int i = tid; ref < a.S && i < a.S * a.check; i += threads) {
      const int s = i / a.check, c = i % a.check;
      if (start(s + 1) > start(s))
        bad |= ld_in(a.page_table + (size_t)s * a.max_blocks + c) != ld_in(a.page_table + (size_t)ref * a.max_blocks + c);
    }
    if (bad) dev_fail(a.header, kDevBadIndex, 1512);
  }
  int leads = 0, runs = 0;
  for (int r0 = 0; r0 < a.N; r0 += threads) {
    const int r = r0 + tid;
    int4 out = make_int4(-1, 0, 0, 0);
    if (r < a.N) {
      const int s = bisect_rows(start, a.S, r);
      if (s < a.S) {
        const int len = ld_in(a.seq_len + s), begin = start(s), end = start(s + 1);
        if (len < end - r + a.prefix * 128 || len > a.max_blocks * 128) {
          out.x = -2;
          dev_fail(a.header, kDevBadIndex, 1211);
        } else {
          out = make_int4(s, len - (end - r), r - begin, (end < a.N ? end : a.N) - r);
        }
      }
      a.rows[r] = out;
    }
    // the rows that lead a tile, in order
    auto list = [&](int rows, int4* to, int& count) {
      const bool lead = out.x >= 0 && out.z % rows == 0;
      const unsigned m = __ballot_sync(0xffffffffu, lead);
      if (lane == 0) sh.sums[warp] = __popc(m);
      sync();
      int before = count;
      for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) before += sh.sums[w];
        count += sh.sums[w];
      }
      if (lead) to[before + __popc(m & ((1u << lane) - 1))] = make_int4(out.x, out.y, r, min(rows, out.w));
      sync();
    };
    if (a.tile_rows > 1 && !a.run_rows) list(a.tile_rows, a.lead, leads);
    if (a.run_rows) list(a.run_rows, a.runs, runs);
  }
  if (tid == 0) {
    a.header[kLeadCount] = leads;
    a.header[kRunCount] = runs;
  }
}

// What the blocks of the kernel before found wrong; by one warp.
__device__ __forceinline__ void report_flags(const int* flags, int n, int* err, int lane) {
  for (int i = lane; i < n; i += 32) {
    const int flag = ld_in(flags + i);
    if (flag) dev_fail(err, flag / 65536, flag % 65536);
  }
}

}  // namespace msa
