// Full attention by 128-row tiles: of a batch's new rows over the pages that all
// its sequences share, in one pass over those pages for the whole batch, and of
// the several new rows of a sequence over its own pages.
//
// The rows of every sequence times the heads of a group fill 128-row tiles
// (128 / h_g rows each), so the shared part is a matrix product with as many
// rows as the batch has, whatever the sequences' lengths: tcgen05, two tiles
// per CTA against each K/V page, which arrives once for both.
//   S_t = Q_t K^T (TMEM);  P_t = exp2(S_t scale log2 e - m), bf16 over S_t's
//   columns;  O_t += P_t V (P_t from TMEM, O_t in TMEM)
// for the tiles t = 0, 1 in turn, so that the tensor core computes one tile's
// products while the softmax warps of the other work (the scheme of the full
// causal forward, without masks: every row sees every shared token). P is
// rounded to bf16 as there: the MMA takes both operands in V's type, and the
// row sum is taken before the rounding. The running maximum moves only when a
// page raises it by more than 2^8 (an O_t rescale is a TMEM round trip).
//
// What bounds it is the chain S -> softmax -> PV -> next S of a tile: its two
// products take 1,100 cycles, and the softmax should fit into the other tile's.
// So two warps share each row, 64 keys each, and do not wait for each other:
// both compute P under the row's common maximum, and only a warp that finds a
// value 2^8 above it calls the other (which is then still waiting for the next
// S), after which both raise the maximum, rescale O and compute P again.
//
// Work of the shared part: all (group, page) pairs in a line, cut into `teams`
// runs of equal length; a run is walked by `pairs` CTAs at once, one per pair of
// tiles, so that a page is read from HBM once and from L2 by the others. A run
// leaves one partial O (fp32, normalised) and log-sum-exp per row and group.
//
// A sequence's own pages (kRuns): a run is up to 256 / h_g of its rows, a group
// and some pages, taken as they come. Where its rows fill one tile only, the
// second tile is the same rows of the next group against that group's pages: a
// tile alone would leave the tensor core idle during its softmax and the memory
// during both (32 sequences of 4 rows, 64 heads over 8 groups, 2000 tokens: 109
// us against 92). What differs from the shared part:
//   - P as the sum of two positive bf16 values, side by side over S (the second
//     product costs little where the memory bounds: with one row or two the same
//     result comes from the mma.sync path, which does that too);
//   - masks, on the pages that not every row sees all of, and V cleaned there by
//     a warp of its own before the tensor core may read it: a zero of P does not
//     keep an infinity or a NaN of a later row's V from an earlier row;
//   - K and V have a producer and barriers each, and the runs' descriptions go
//     round in shared memory.
//
// Measured: the shared part of 128 sequences x 2 rows x 32 heads over 128K tokens
// 385 us on 136 SMs, 1430 TFLOP/s (0.74 of what a library product reaches on all);
// own pages of 16 x 4 rows x 64 heads over 3000 tokens 50 us, 4.1 TB/s; the whole
// call for 32 x 4 rows x 64 heads over 2000 tokens 63 us, for 300 rows x 32 heads
// over 4 groups and 8000 tokens 64 us (610 TFLOP/s, P's second product not counted).
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr float kHeadroom = 8.f;  // P = exp2(s - m) stays <= 2^kHeadroom
// warp 0 TMA, warp 1 UMMA + TMEM, 2 and 3 V of own pages, 4-11 and 12-19 softmax of tiles 0 and 1
constexpr int kThreads = 640;
constexpr int kTile = 32768;      // 128 rows x 128 bf16, two 64-column SW128 chunks
constexpr int kChunk = 16384;
constexpr int kStages = 2;        // K/V ring
constexpr int oQ = 0, oK = 2 * kTile, oV = oK + kStages * kTile;
constexpr int kSmem = oV + kStages * kTile + 1024;

// One run: pages of one group against up to two tiles of rows.
struct Run {
  int row0, rows;   // the tiles' first row, and how many rows there are for them
  int g, pages;     // (pages 0: the end)
  int slot;         // of the rows' partials
  int own;          // a sequence's own pages: P as the sum of two bf16, masks
  int twin;         // the second tile is the same rows of group g + 1, against that group's pages
  int seq, first;   // whose pages, from which block
  int pos;          // own: position of the first row
  int masked;       // the first page that not every row sees all of
};

struct PrefixArgs {
  int* flags;  // [blocks] what a block found wrong (the error word is cleared meanwhile; the merge reports it)
  const int32_t *page_table, *row_start;
  float *part_o, *part_lse;
  const int4* runs;
  const __nv_bfloat16* V;
  int* header;
  int S, N, Hq, G, hg, prefix, pairs, teams, num_pages, max_blocks;
  int run_rows, per_run, rslots, pslots;
  float scale_log2;
};

struct PrefixShared {
  int flag;
  Run run[2];
  int odd[2];  // a run's V has infinities or NaN among the rows' own tokens
  uint64_t run_full[2], run_empty[2], k_full[kStages], v_clean[kStages];  // (kRuns)
  uint64_t q_full, q_empty;
  uint64_t k0_full, kv_full[kStages];  // the first page's K; then a page's V with the next one's K
  uint64_t k_empty[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t pair[2][4];           // the two warps of a tile's 32 rows
  float row_max[2][2][128];      // [tile][half][row] of the page's scores (at the end: the row's sums)
  int raised[2][2][4];           // [tile][half][quarter] the page (counted from 1) at which this warp called the other
  uint32_t tmem_base;
};

// (x0, x1) * a + b, two at a time.
__device__ __forceinline__ void fma2(float& x0, float& x1, float a, float b) {
  asm("{\n\t.reg .b64 x, m, n;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 m, {%2, %2};\n\tmov.b64 n, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, m, n;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a), "f"(b));
}
// (s0, s1) += (x0, x1)
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  asm("{\n\t.reg .b64 s, x;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\tadd.rn.f32x2 s, s, x;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}
// Eight floats to a 32-byte boundary in one store.
__device__ __forceinline__ void st_global8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
               "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// kShared: the call has a shared prefix. Without one every page is a sequence's own, and its P has both parts: told at run
// time, as where there are both kinds, it costs 2 % (32 x 4 rows x 64 heads over 2000 tokens 63.3 -> 64.9 us).
template <bool kRuns, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    paged_prefix_kernel(PrefixArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PrefixShared sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int team = a.pairs ? blockIdx.x / a.pairs : 0, pair = a.pairs ? blockIdx.x % a.pairs : 0;
  const int units = a.G * a.prefix;
  int u_begin = 0, u_end = 0;
  if (!kRuns || team < a.teams) {  // (with runs there may be more CTAs than the prefix has work for)
    u_begin = team_start(team, units, a.teams);
    u_end = team_start(team + 1, units, a.teams);
  }
  const int tile_rows = 128 / a.hg;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 8);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.o_free[i], 8);
      for (int j = 0; j < 4; ++j) mbar_init(&sh.pair[i][j], 2);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.k_empty[i], 1);
      mbar_init(&sh.v_empty[i], 1);
    }
    if (kRuns) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.run_full[i], 1);
        mbar_init(&sh.run_empty[i], 19);
        mbar_init(&sh.k_full[i], 1);
        mbar_init(&sh.v_clean[i], 1);
      }
    }
    mbar_init(&sh.k0_full, 1);
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 16; ++i) sh.raised[i >> 3][(i >> 2) & 1][i & 3] = 0;
    sh.flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_release();  // (not before: the kernel that starts on the SMs left over reads what the one before this wrote)
  // the first sequence with rows: its table holds the shared pages
  const int ref = a.prefix ? find_sequence(a.row_start, a.S, 0, lane) : a.S;
  int* const err = &sh.flag;
  if (ref >= a.S) u_begin = u_end;  // no rows at all
  const uint32_t tmem = sh.tmem_base;  // S_0 [0,128), S_1 [128,256), O_0 [256,384), O_1 [384,512)

  // The next run (false: the end, or a wait that ran out). Without kRuns everybody counts for himself.
  int n_run = 0, u = u_begin;
  auto next_run = [&](Run& run) {
    if constexpr (kRuns) {
      if (!mbar_wait(&sh.run_full[n_run & 1], (n_run >> 1) & 1, err, 1505)) return false;
      run = sh.run[n_run & 1];
      ++n_run;
      return run.pages > 0;
    } else {
      if (u >= u_end) return false;
      const int g = u / a.prefix, stop = min(u_end, (g + 1) * a.prefix);
      run = {2 * pair * tile_rows, a.N, g, stop - u, team - team_of(g * a.prefix, units, a.teams)};
      u = stop;
      return true;
    }
  };

  auto run_done = [&](bool solo) {  // solo: said by one thread of the warp
    if constexpr (kRuns) {
      if (!solo) __syncwarp();
      if (solo || lane == 0) mbar_arrive(&sh.run_empty[(n_run - 1) & 1]);
    }
  };

  // Row of the pools' tensor maps of the run's page i.
  auto table_row = [&](const Run& run, int i) {
    if (i >= run.pages) return 0;
    int page = ld_in(a.page_table + (size_t)run.seq * a.max_blocks + run.first + i);
    if (page < 0 || page >= a.num_pages) {
      dev_fail(err, kDevBadIndex, 1511);
      page = 0;
    }
    return (page * a.G + run.g) * 128;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
    auto load_tile = [&](int at, const CUtensorMap* map, uint64_t* bar, int y) {
      tma_load_2d(smem + at, map, bar, 0, y);
      tma_load_2d(smem + at + kChunk, map, bar, 64, y);
    };
    auto load_kv = [&](int at, const CUtensorMap* map, uint64_t* bar, int y) {
      mbar_arrive_expect_tx(bar, kTile);
      load_tile(at, map, bar, y);
    };
    if constexpr (kRuns) {
      // The prefix's runs first, as below, then the sequences' own ones as they come. A run's first 32 pages are looked
      // up ahead, one step a page: the number, the rows, the pages.
      struct Ahead {
        Run run;
        int y;  // of this lane's page
      };
      int u = u_begin, id = 0, taken = 0, own = -1;  // own: runs of its own that this CTA has asked for
      const int pair_g = a.G % 2 ? 1 : 2;  // groups of an item: both tiles' at once, or one after the other
      const int items = a.run_rows ? ld_in(a.header + kRunCount) * a.rslots * (a.G / pair_g) : 0;
      bool second = false;  // the item's second group is still to come
      bool own_now = false;
      int4 lead = make_int4(0, 0, 0, 0);
      auto step1 = [&]() {
        own_now = second || u >= u_end;
        if (!own_now || second) return;
        if (++own > 0 && lane == 0) taken = atomicAdd(a.header + kRunNext, 1);
      };
      auto step2 = [&]() {
        if (!own_now || second) return;
        id = own ? gridDim.x + __shfl_sync(0xffffffffu, taken, 0) : blockIdx.x;
        if (id < items) lead = ld_in(a.runs + id / (a.rslots * (a.G / pair_g)));
      };
      auto step3 = [&](Ahead& h) {
        h.run.pages = 0;
        if (!own_now) {
          const int g = u / a.prefix, stop = min(u_end, (g + 1) * a.prefix);
          const int row0 = 2 * pair * tile_rows;
          h.run = {row0, min(a.N - row0, 2 * tile_rows), g, stop - u, team - team_of(g * a.prefix, units, a.teams), 0, 0, ref,
                   u - g * a.prefix, 0, 1 << 30};
          u = stop;
        } else if (id < items) {
          const int pairs_g = a.G / pair_g, part = id % (a.rslots * pairs_g), split = part / pairs_g;
          const int twin = pair_g == 2 && lead.w <= tile_rows;
          const int first = a.prefix + split * a.per_run, own_pages = (lead.y + lead.w - 1) / 128 + 1 - first;
          h.run = {lead.z, lead.w, part % pairs_g * pair_g + second, max(0, min(a.per_run, own_pages)), a.pslots + split, 1,
                   twin, lead.x, first, lead.y, max(0, (lead.y + 1) / 128 - first)};
          second = pair_g == 2 && !twin && !second && h.run.pages;
        }
        h.y = table_row(h.run, lane);
      };
      Ahead now, next;
      now.run.pages = next.run.pages = 0;
      auto find = [&](Ahead& h, int step) {  // the next run with pages (or the end), or one step on the way there
        if (step == 0) step1();
        else if (step == 1) step2();
        else if (step == 2) step3(h);
      };
      auto more = [&] { return u < u_end || second || id < items; };  // what step 3 of the last one leaves to be asked for
      for (int s = 0; s < 3; ++s) find(now, s);
      int n_run = 0;
      uint32_t kc = 0;
      bool ok = true;
      while (ok) {
        const bool end = now.run.pages == 0;
        if (end && more()) {  // a run without pages: on to the next one
          for (int s = 0; s < 3; ++s) find(now, s);
          continue;
        }
        const int slot = n_run & 1;
        if (!mbar_wait(&sh.run_empty[slot], ((n_run >> 1) & 1) ^ 1, err, 1501)) break;
        if (lane == 0) {
          sh.run[slot] = now.run;
          mbar_arrive(&sh.run_full[slot]);
        }
        __syncwarp();
        if (end) break;
        int y = now.y, step = 0;
        const int tiles = now.run.twin || now.run.rows > tile_rows ? 2 : 1;
        const int streams = now.run.twin ? 2 : 1;  // of pages
        for (int i = 0; i < now.run.pages * streams; ++i, ++kc) {
          const int page = now.run.twin ? i >> 1 : i, other = now.run.twin ? (i & 1) * 128 : 0;
          if (page && !other && (page & 31) == 0) y = table_row(now.run, page + lane);
          const int st = kc % kStages, at = __shfl_sync(0xffffffffu, y, page & 31) + other;
          const uint32_t par = ((kc / kStages) & 1) ^ 1;
          if (!mbar_wait(&sh.k_empty[st], par, err, 1503)) { ok = false; break; }
          if (lane == 0) load_kv(oK + st * kTile, &map_k, &sh.k_full[st], at);
          __syncwarp();
          if (i == 0 && !mbar_wait(&sh.q_empty, (n_run & 1) ^ 1, err, 1502)) { ok = false; break; }
          if (i == 0 && lane == 0) {  // (the first K may come while the run before still needs its queries)
            mbar_arrive_expect_tx(&sh.q_full, tiles * kTile);
            for (int t = 0; t < tiles; ++t) {
              const int row0 = now.run.row0 + (now.run.twin ? 0 : t * tile_rows);  // rows past N arrive as zeros
              const int head = (now.run.g + (now.run.twin ? t : 0)) * a.hg;
              tma_load_3d(smem + oQ + t * kTile, &map_q, &sh.q_full, 0, head, row0);
              tma_load_3d(smem + oQ + t * kTile + kChunk, &map_q, &sh.q_full, 64, head, row0);
            }
          }
          __syncwarp();
          if (step < 3) find(next, step++);
        }
        ++n_run;
        for (; step < 3; ++step) find(next, step);
        now = next;
      }
    } else {
      const int n = u_end - u_begin;
      // row of the pool's tensor map of the CTA's page i + lane
      auto rows_of = [&](int i) {
        const int u = u_begin + i + lane;
        if (u >= u_end) return 0;
        const int g = u / a.prefix;
        int page = ld_in(a.page_table + (size_t)ref * a.max_blocks + (u - g * a.prefix));
        if (page < 0 || page >= a.num_pages) {
          dev_fail(err, kDevBadIndex, 1511);
          page = 0;
        }
        return (page * a.G + g) * 128;
      };
      auto load_q = [&](int g) {
        mbar_arrive_expect_tx(&sh.q_full, 2 * kTile);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row0 = (2 * pair + t) * tile_rows;  // rows past N arrive as zeros
          tma_load_3d(smem + oQ + t * kTile, &map_q, &sh.q_full, 0, g * a.hg, row0);
          tma_load_3d(smem + oQ + t * kTile + kChunk, &map_q, &sh.q_full, 64, g * a.hg, row0);
        }
      };
      int cur = rows_of(0), ahead = rows_of(32), seg = 0;
      if (n > 0 && lane == 0) {
        load_q(u_begin / a.prefix);
        mbar_arrive_expect_tx(&sh.k0_full, kTile);
        load_tile(oK, &map_k, &sh.k0_full, cur);
      }
      for (int i = 0; i < n; ++i) {
        const int st = i % kStages, st1 = (i + 1) % kStages;
        const int y = __shfl_sync(0xffffffffu, cur, i & 31);
        const int y1 = (i & 31) == 31 ? __shfl_sync(0xffffffffu, ahead, 0) : __shfl_sync(0xffffffffu, cur, (i & 31) + 1);
        const bool more = i + 1 < n;
        if (!mbar_wait(&sh.v_empty[st], ((i / kStages) & 1) ^ 1, err, 1504)) break;
        if (more && !mbar_wait(&sh.k_empty[st1], (((i + 1) / kStages) & 1) ^ 1, err, 1503)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.kv_full[st], more ? 2 * kTile : kTile);
          load_tile(oV + st * kTile, &map_v, &sh.kv_full[st], y);
          if (more) load_tile(oK + st1 * kTile, &map_k, &sh.kv_full[st], y1);
        }
        __syncwarp();
        const int g1 = (u_begin + i + 1) / a.prefix;
        if (more && g1 != (u_begin + i) / a.prefix) {  // the next page is another group's: its queries
          if (!mbar_wait(&sh.q_empty, seg & 1, err, 1502)) break;
          ++seg;
          if (lane == 0) load_q(g1);
          __syncwarp();
        }
        if ((i & 31) == 31) {
          cur = ahead;
          ahead = rows_of(i + 33);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- UMMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = make_idesc_bf16(128, 128, false, false);  // Q, K both K-major
      constexpr uint32_t id_o = make_idesc_bf16(128, 128, false, true);   // P from TMEM, V MN-major
      // the operands' descriptors as 32-bit words: one add per instruction, so that the issuing thread keeps up
      constexpr uint32_t hi = sdesc_hi_sw128_sbo1024();
      const uint32_t q_lo = sdesc_lo(smem_u32(smem + oQ), 16), k_lo = sdesc_lo(smem_u32(smem + oK), 16);
      const uint32_t v_lo = sdesc_lo(smem_u32(smem + oV), kChunk);
      uint32_t kc = 0;
      bool ok = true;
      auto issue_s = [&](int t, int st) {
        const uint32_t qa = q_lo + t * (kTile >> 4), ka = k_lo + st * (kTile >> 4), d = tmem + t * 128;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t off = ((ks >> 2) * kChunk + (ks & 3) * 32) >> 4;
          umma_bf16_ss_w(d, qa + off, ka + off, hi, id_s, ks > 0);
        }
        umma_commit(&sh.s_full[t]);
      };
      auto issue_o = [&](int t, int st, bool acc, bool own) {
        const uint32_t va = v_lo + st * (kTile >> 4), d = tmem + 256 + t * 128, p = tmem + t * 128;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          umma_bf16_ts_w(d, p + (ks >> 2) * 64 + (ks & 3) * 8, va + ks * (2048 >> 4), hi, id_o, ks > 0 ? 1u : (uint32_t)acc);
        if (kRuns && own)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_bf16_ts_w(d, p + (ks >> 2) * 64 + 32 + (ks & 3) * 8, va + ks * (2048 >> 4), hi, id_o, 1u);
      };
      // pages and runs of each tile (the second one has none in a run of few rows)
      uint32_t pages_of[2] = {0, 0}, runs_of[2] = {0, 0};
      Run run;
      for (int seg = 0; ok && next_run(run); ++seg) {
        run_done(true);
        const bool twin = kRuns && run.twin;
        const int pages = run.pages, last_t = !kRuns || twin || run.rows > tile_rows, streams = twin ? 2 : 1;
        if (!mbar_wait(&sh.q_full, seg & 1, err, 1520)) { ok = false; break; }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t > last_t) break;
          const uint32_t kk = kc + (twin ? t : 0), st = kk % kStages;
          if (kRuns) {
            if ((t == 0 || twin) && !mbar_wait(&sh.k_full[st], (kk / kStages) & 1, err, 1513)) { ok = false; break; }
          } else {
            // (a later run's first K came with the V of the page before it)
            if (kc == 0 && t == 0 && !mbar_wait(&sh.k0_full, 0, err, 1513)) { ok = false; break; }
          }
          tc_fence_after();
          issue_s(t, st);
          if (twin || t == last_t) umma_commit(&sh.k_empty[st]);
        }
        if (pages == 1) umma_commit(&sh.q_empty);
        for (int c = 0; c < pages && ok; ++c, kc += streams) {
          const bool last = c == pages - 1;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t > last_t) break;
            const uint32_t kk = kc + (twin ? t : 0), st = kk % kStages, kk1 = kk + streams, st1 = kk1 % kStages;
            // the page's V and the next one's K first: nothing then stands between P_t and its products
            if (c == 0 && !mbar_wait(&sh.o_free[t], (runs_of[t] & 1) ^ 1, err, 1516 + t)) { ok = false; break; }
            if ((t == 0 || twin) && !mbar_wait(&sh.kv_full[st], (kk / kStages) & 1, err, 1518)) { ok = false; break; }
            if (kRuns && (t == 0 || twin) && !mbar_wait(&sh.v_clean[st], (kk / kStages) & 1, err, 1519)) { ok = false; break; }
            // P_t of this page written (and O_t rescaled if its row maximum moved)
            if (!mbar_wait(&sh.p_full[t], pages_of[t] & 1, err, 1514 + t)) { ok = false; break; }
            ++pages_of[t];
            tc_fence_after();
            issue_o(t, st, c > 0, run.own);
            if (twin || t == last_t) umma_commit(&sh.v_empty[st]);
            if (!last) {
              // the next page's S_t: after this PV_t in issue order, so it overwrites P_t only once read
              if (kRuns && (t == 0 || twin)) {
                if (!mbar_wait(&sh.k_full[st1], (kk1 / kStages) & 1, err, 1513)) { ok = false; break; }
                tc_fence_after();
              }
              issue_s(t, st1);
              if (twin || t == last_t) umma_commit(&sh.k_empty[st1]);
              if (t == last_t && c + 1 == pages - 1) umma_commit(&sh.q_empty);
            } else {
              umma_commit(&sh.o_full[t]);
              ++runs_of[t];
            }
          }
        }
      }
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------------- V of the sequences' own pages
    if constexpr (kRuns) {
      // Two warps for V. The first loads it; K has a producer of its own (and arrives a softmax earlier), so that neither
      // waits for the other's stages. The second looks at V of pages that not every row sees all of: what lies behind the
      // last row's end is cleared, and infinities and NaN among the rows' own tokens, which would reach the rows before
      // them as 0 * x; where there are any, each row's own ones are added at the end.
      uint32_t kc = 0;
      Run run;
      bool ok = true;
      while (ok && next_run(run)) {
        const int streams = run.twin ? 2 : 1;
        int y = 0;
        if (warp == 2) y = table_row(run, lane);
        else if (lane == 0) sh.odd[(n_run - 1) & 1] = 0;
        __syncwarp();
        for (int i = 0; i < run.pages * streams; ++i, ++kc) {
          const int st = kc % kStages, page = run.twin ? i >> 1 : i, other = run.twin ? i & 1 : 0;
          const uint32_t par = (kc / kStages) & 1;
          if (warp == 2) {
            if (page && !other && (page & 31) == 0) y = table_row(run, page + lane);
            const int at = __shfl_sync(0xffffffffu, y, page & 31) + other * 128;
            if (!mbar_wait(&sh.v_empty[st], par ^ 1, err, 1504)) { ok = false; break; }
            if (lane == 0) {
              mbar_arrive_expect_tx(&sh.kv_full[st], kTile);
              tma_load_2d(smem + oV + st * kTile, &map_v, &sh.kv_full[st], 0, at);
              tma_load_2d(smem + oV + st * kTile + kChunk, &map_v, &sh.kv_full[st], 64, at);
            }
            __syncwarp();
            continue;
          }
          if (!mbar_wait(&sh.kv_full[st], par, err, 1506)) { ok = false; break; }
          if (page >= run.masked) {
            // 16 lanes per key, 8 dims each: first the rows' own tokens, then what is behind them
            const int token0 = (run.first + page) * 128, chunk = lane & 15;
            const int own = max(0, run.pos + 1 - token0), behind = min(128, max(0, run.pos + run.rows - token0));
            uint8_t* tile = smem + oV + st * kTile + (chunk >> 3) * kChunk;
            bool odd = false;
            for (int key = own + lane / 16; key < behind; key += 2) {
              uint4* at = reinterpret_cast<uint4*>(tile + sw128_off(key, chunk & 7));
              uint4 v = *at;
              bool bad = false;
              auto check = [&](uint32_t& w) {
                if ((w & 0x7f80u) == 0x7f80u) { w &= 0xffff0000u; bad = true; }
                if ((w & 0x7f800000u) == 0x7f800000u) { w &= 0xffffu; bad = true; }
              };
              check(v.x); check(v.y); check(v.z); check(v.w);
              if (bad) *at = v;
              odd |= bad;
            }
#pragma unroll 8
            for (int key = behind + lane / 16; key < 128; key += 2)
              *reinterpret_cast<uint4*>(tile + sw128_off(key, chunk & 7)) = make_uint4(0, 0, 0, 0);
            if (odd) sh.odd[(n_run - 1) & 1] = 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.v_clean[st]);
        }
        run_done(false);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax (thread = one head of one new row, 64 keys)
    const int t = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_at = tmem + lane_off + t * 128 + half * 64;        // this warp's scores, and P over their first half
    const uint32_t o_at = tmem + lane_off + 256 + t * 128 + half * 64;  // the columns of O that it rescales and reads out
    {
      // while the first pages are on their way: is the prefix the same one for every sequence with rows?
      bool bad = false;
      const long long cells = (long long)a.S * a.prefix;
      for (long long i = (long long)blockIdx.x * 512 + threadIdx.x - 128; ref < a.S && i < cells; i += (long long)gridDim.x * 512) {
        const int s = (int)(i / a.prefix), c = (int)(i % a.prefix);
        const int32_t* table = a.page_table + c;
        if (ld_in(a.row_start + s + 1) > ld_in(a.row_start + s))
          bad |= ld_in(table + (size_t)s * a.max_blocks) != ld_in(table + (size_t)ref * a.max_blocks);
      }
      if (bad) dev_fail(err, kDevBadIndex, 1512);
    }
    uint32_t kc = 0, pair_ph = 0;
    bool ok = true;
    Run run;
    for (int seg = 0; ok && next_run(run);) {
      if (kRuns && t && !run.twin && run.rows <= tile_rows) {  // no second tile
        run_done(false);
        continue;
      }
      const bool twin = kRuns && run.twin;
      const int in = (twin ? 0 : t * tile_rows) + lrow / a.hg, row = run.row0 + in;
      const int pages = run.pages;
      float m_run = -INFINITY, l_run = 0.f;  // the maximum is the row's, the sum that of this warp's keys
      if (!mbar_wait(&sh.s_full[t], kc & 1, err, 1522 + t)) { ok = false; break; }
      for (int c = 0; c < pages && ok; ++c, ++kc) {
        tc_fence_after();
        float sv[64], mq[2];
        tmem_ld32_max(s_at, *reinterpret_cast<float(*)[32]>(sv), mq[0]);
        tmem_ld32_max(s_at + 32, *reinterpret_cast<float(*)[32]>(sv + 32), mq[1]);
        tmem_wait_ld();
        if (kRuns && c >= run.masked) {
          const int seen = run.pos + in + 1 - (run.first + c) * 128 - half * 64;  // keys of this warp's before the row's end
          mq[0] = mq[1] = -INFINITY;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            if (i >= seen) sv[i] = -INFINITY;
            mq[i & 1] = fmaxf(mq[i & 1], sv[i]);
          }
        }
        const float m_blk = fmaxf(mq[0], mq[1]) * a.scale_log2;
        sh.row_max[t][half][lrow] = m_blk;
        bool mine = c == 0 || __any_sync(0xffffffffu, m_blk > m_run + kHeadroom);  // this warp calls the other
        float l_add = 0.f;
        auto write_p = [&]() {
          float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
          const float base = m_run == -INFINITY ? 0.f : m_run;  // (nothing but -infinity so far: exp2(-inf - 0) = 0)
          if (kRuns && (!kShared || run.own)) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t pk[8], rest[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) {
                float p0 = sv[16 * h + 2 * z], p1 = sv[16 * h + 2 * z + 1];
                fma2(p0, p1, a.scale_log2, -base);
                p0 = fast_exp2(p0);
                p1 = fast_exp2(p1);
                if (z & 1) add2(t0, t1, p0, p1);
                else add2(s0, s1, p0, p1);
                pk[z] = bf16_cut(p0, p1);
                rest[z] = bf16_rest(p0, p1, pk[z]);
              }
              tmem_st8(s_at + 8 * h, pk);
              tmem_st8(s_at + 32 + 8 * h, rest);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t pk[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) {
                float p0 = sv[16 * h + 2 * z], p1 = sv[16 * h + 2 * z + 1];
                fma2(p0, p1, a.scale_log2, -base);
                p0 = fast_exp2(p0);
                p1 = fast_exp2(p1);
                if (z & 1) add2(t0, t1, p0, p1);
                else add2(s0, s1, p0, p1);
                pk[z] = pack_bf16(p0, p1);
              }
              tmem_st8(s_at + 8 * h, pk);
            }
          }
          l_add = (s0 + s1) + (t0 + t1);
        };
        if (!mine) {
          write_p();
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[t]);
        } else if (c > 0) {
          __syncwarp();
          if (lane == 0) *static_cast<volatile int*>(&sh.raised[t][half][quarter]) = (int)kc + 1;
        }
        // what comes next: the other warp's call, or the next page's scores (after the last page, O)
        uint64_t* next = c + 1 < pages ? &sh.s_full[t] : &sh.o_full[t];
        const uint32_t next_ph = c + 1 < pages ? (kc + 1) & 1 : seg & 1;
        bool redo = mine;
        if (!mine) {
          const uint32_t bar = smem_u32(next);
          const volatile int* call = &sh.raised[t][half ^ 1][quarter];
          unsigned long long since = 0;
          for (uint32_t i = 1;; ++i) {
            redo = __any_sync(0xffffffffu, *call == (int)kc + 1);
            if (redo) break;
            if (__all_sync(0xffffffffu, mbar_test(bar, next_ph))) break;
            if ((i & 255u) == 0) {
              const unsigned long long at = global_ns();
              if (!since) since = at;
              if (__any_sync(0xffffffffu, at - since > kWaitLimitNs)) {
                dev_fail(err, kDevTimeout, 1524 + t);
                ok = false;
                break;
              }
            }
          }
          if (!ok) break;
        }
        if (redo) {
          if (!warps_sync(&sh.pair[t][quarter], pair_ph, err, 1526 + t)) { ok = false; break; }
          const float m_new = fmaxf(m_blk, sh.row_max[t][half ^ 1][lrow]);
          const bool need = m_new > m_run + kHeadroom;
          const float alpha = need ? fast_exp2(m_run - m_new) : 1.f;
          if (need) m_run = m_new;
          l_run *= alpha;
          if (c > 0) {
            // O_t to the new maximum: PV_t of the previous page is done (it was issued before this page's S_t)
#pragma unroll 1
            for (int z = 0; z < 8; ++z) {
              float o[8];
              tmem_ld8(o_at + z * 8, o);
              tmem_wait_ld();
              uint32_t ob[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) ob[i] = __float_as_uint(o[i] * alpha);
              tmem_st8(o_at + z * 8, ob);
            }
          }
          write_p();
          tmem_wait_st();
          tc_fence_before();
          // both warps are through before the one that called (or both) hands P on
          if (!warps_sync(&sh.pair[t][quarter], pair_ph, err, 1528 + t)) { ok = false; break; }
          if (mine) {
            tc_fence_after();
            tc_fence_before();
            if (lane == 0) mbar_arrive(&sh.p_full[t]);
          }
          if (!mbar_wait(next, next_ph, err, 1530 + t)) { ok = false; break; }
        }
        l_run += l_add;
      }
      if (!ok) break;
      // ---- the run's end in this group: the row's partial
      sh.row_max[t][half][lrow] = l_run;
      if (!warps_sync(&sh.pair[t][quarter], pair_ph, err, 1532 + t)) { ok = false; break; }
      const float l = half ? sh.row_max[t][0][lrow] + l_run : l_run + sh.row_max[t][1][lrow];
      if (!warps_sync(&sh.pair[t][quarter], pair_ph, err, 1534 + t)) { ok = false; break; }
      tc_fence_after();
      const bool valid = kRuns ? in < run.rows : row < a.N;
      const int group = run.g + (twin ? t : 0);
      const size_t at = ((size_t)run.slot * a.N + row) * a.Hq + group * a.hg + lrow % a.hg;
      const bool odd = kRuns && run.own && sh.odd[(n_run - 1) & 1];
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (a run behind the row's end, or scores of -infinity)
      float* dst = a.part_o + at * 128 + half * 64;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        float o[16];
        tmem_ld16(o_at + z * 16, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] *= inv;
        if (odd && valid) {  // infinities and NaN of the own tokens that this row sees, and of this run's
          const int begin = max(run.pos + 1, run.first * 128), end = min(run.pos + in + 1, (run.first + run.pages) * 128);
          for (int k = begin; k < end; ++k) {
            const int page = ld_in(a.page_table + (size_t)run.seq * a.max_blocks + k / 128);
            if (page < 0 || page >= a.num_pages) continue;
            const __nv_bfloat16* v = a.V + (((size_t)page * a.G + group) * 128 + k % 128) * 128 + half * 64 + z * 16;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = __bfloat162float(v[i]);
              if (!(fabsf(x) < INFINITY)) o[i] += x;
            }
          }
        }
        if (valid) {
          st_global8(dst + 16 * z, o);
          st_global8(dst + 16 * z + 8, o + 8);
        }
      }
      if (valid && half == 0) a.part_lse[at] = m_run + log2f(l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free[t]);
      ++seg;
      run_done(false);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = sh.flag;
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <bool kRuns, bool kShared>
cudaError_t launch_prefix(const PrefixArgs& a, int blocks, const CUtensorMap& mq, const PoolMaps& maps, cudaStream_t st) {
  static bool attr[kMaxDevices] = {};
  const int dslot = device_slot();
  if (!attr[dslot]) {
    cudaError_t e =
        cudaFuncSetAttribute(paged_prefix_kernel<kRuns, kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr[dslot] = true;
  }
  count_launches(1);
  return launch_dependent(paged_prefix_kernel<kRuns, kShared>, blocks, kThreads, kSmem, st, a, mq, maps.k, maps.v);
}

}  // namespace

cudaError_t launch_paged_prefix(const PagedProb& p, const PagedCachePtrs& c, const PoolMaps& maps, const void* Q,
                                uint8_t* ws, const PagedWs& L, cudaStream_t st) {
  CUtensorMap mq;
  {
    // a tile's rows times the heads of one group: box {64 d, h_g heads, 128 / h_g rows}
    const uint64_t dims[3] = {128, (uint64_t)p.Hq, (uint64_t)p.N};
    const uint64_t strides[2] = {256, (uint64_t)p.Hq * 256};
    const uint32_t box[3] = {64, (uint32_t)p.hg, (uint32_t)(128 / p.hg)};
    if (!encode_tmap(&mq, const_cast<void*>(Q), 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  PrefixArgs a;
  a.flags = reinterpret_cast<int*>(ws + L.flags);
  a.page_table = c.page_table;
  a.row_start = c.row_start;
  a.S = p.S;
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + L.part_lse);
  a.N = p.N;
  a.Hq = p.Hq;
  a.G = p.G;
  a.hg = p.hg;
  a.prefix = L.prefix;
  a.pairs = L.pairs;
  a.teams = L.teams;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.scale_log2 = p.scale * kLog2e;
  a.runs = reinterpret_cast<const int4*>(ws + L.runs);
  a.V = static_cast<const __nv_bfloat16*>(c.V);
  a.header = reinterpret_cast<int*>(ws);
  a.run_rows = L.run_rows;
  a.per_run = L.per_run;
  a.rslots = L.rslots;
  a.pslots = L.pslots;
  if (!L.run_rows) return launch_prefix<false, true>(a, L.n_flags, mq, maps, st);
  if (L.prefix) return launch_prefix<true, true>(a, L.n_flags, mq, maps, st);
  return launch_prefix<true, false>(a, L.n_flags, mq, maps, st);
}

}  // namespace msa
