// Attention of new tokens over pages of the cache: the selected pages of each
// (row, group), or a sequence's own pages behind a shared prefix.
//
// Few query columns against streamed keys: 64 KB of K and V per page and group
// serve at most 8 columns, so the time is the memory's. One persistent
// CTA per SM: a producer warp keeps three whole pages in flight (192 KB, TMA
// boxes of half a page each), eight warps take 16 keys of every page each:
//   S^T = K q^T   (mma.sync, keys in rows, columns = rows of the sequence x heads of the group)
//   P   = exp2(S scale log2 e - m), m the warp's own running maximum per column
//   O^T += V^T P^T, P as a sum of two bf16 values (16 bits of it: the rounding
//          of P would otherwise be as large as the output's own), both positive,
//          so that an infinity of V comes out as such
// with the warp's own maximum, sum and O in registers; the warps meet once per
// item (a run of pages of one (row tile, group)). The CTA whose item is done
// last of its (row tile, group) joins the fp32 parts in their order, so the
// result does not depend on which one it is; warps of their own do that, so
// that the next pages are not kept waiting by its loads. Behind a shared prefix
// the merge kernel below joins them with the prefix's.
//
// Measured: 60 rows x 8 groups x 16 selected pages, 503 MB in 81 us, 6.2 TB/s,
// 0.93 of a plain copy; one row's 128 pages 10.7 us, of which the memory takes 1.3.
// Equal runs of pages for every CTA, cut anywhere, cost more at their seams than
// their balance gained (a row at 128K tokens 36 us against 30).
//
// Masked places: a page is masked per column only where it crosses a row's end.
// There, each row of the tile is accumulated on its own with the values behind
// its end cleared, so that nothing stored behind a row's end (another row's
// tokens, stale cache lines, NaN or infinities) reaches it through 0 * x.
#include "mma_sync.cuh"
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr int kWarps = 8;                          // consumers; then the producer and the joining warps
constexpr int kJoinWarps = 3;
constexpr int kThreads = (kWarps + 1 + kJoinWarps) * 32;
constexpr int kHalf = 16384;                       // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kTile = 2 * kHalf;                   // K or V of a page and group
constexpr int kStages = 3;
// The joining warps may have nothing to do until the kernel's end: 20 s, and 20 us for every page that a CTA takes if it
// takes them all in turn (it takes 1.5).
constexpr unsigned long long kIdleNs = 20000000000ull, kIdlePageNs = 20000ull;

constexpr int kQStride = 272;                      // bytes between the queries' rows in shared memory (no bank conflicts)

constexpr int kCols = 8;                           // query columns of a tile
constexpr int kSmem = kStages * 2 * kTile + 2 * kCols * kQStride + 1024;

struct AttnArgs {
  const int4* rows;
  const int4* lead;                       // the rows that lead a tile (null: every row does)
  int* header;                            // of the workspace: kLeadCount, kWorkNext
  const __nv_bfloat16* Q;
  const int32_t *page_table, *block_idx;  // block_idx null: the sequence's own pages from block `prefix` on
  float *part_o, *part_lse;
  int* arrived;                           // [N, G, kJoinWarps] items of a (row tile, group) that are done
  __nv_bfloat16* O;
  float* LSE;
  int N, Hq, G, hg, hg_log2, k, num_pages, max_blocks, prefix, splits, per_split, tile_rows, items, slot0, join;
  int beside;                             // the prefix kernel may still be running (what it writes is not read here)
  float scale_log2;
  const int* flags;                       // [n_flags] of the first kernel's blocks
  int n_flags;
  int* err;
  unsigned long long idle_ns;
};

struct AttnItem {
  int row, g, split, pages;  // pages -1: the end
  int parts;                 // items of this (row tile, group)
  int pos, rows;             // position of the first row; rows of the tile
};

struct AttnShared {
  uint64_t k_full[kStages], v_full[kStages], empty[kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t meet;              // the consumer warps' rendezvous
  uint64_t j_full[2], j_empty[2];
  AttnItem item[2];
  AttnItem join[2];           // for the joining warps; parts 0: the end
  int token0[kStages];        // first token of the stage's page
  float m[kWarps][kCols], l[kWarps][kCols];  // maximum and sum of a warp's columns
  float inv[kCols], lse[kCols];            // of all warps together: 1 / sum, and log2 of the sum
};

// The bf16 pairs of keys t, t + 1 (x) and t + 8, t + 9 (y) that lie before `end`.
__device__ __forceinline__ uint2 keep_keys(int t, int end) {
  return make_uint2((t < end ? 0xffffu : 0u) | (t + 1 < end ? 0xffff0000u : 0u),
                    (t + 8 < end ? 0xffffu : 0u) | (t + 9 < end ? 0xffff0000u : 0u));
}

// What the producer knows about an item, fetched in steps while earlier items
// are on their way: what a step loads is first looked at in the next one, so
// that no load's latency (microseconds while the pages' traffic fills the
// memory's queues) holds up the pages.
struct Fetch {
  int row, split, g;   // row -1: no item
  int4 info;
  int id, before;      // sparse: this lane's block id and the one in front of it
  int ids[4];          // the row's ids lane, lane + 32, ...
  int pages, parts;
  int block, page;     // of this lane's page (the item's first 32)
};

// Items: (row tile, split, group), group fastest.
__device__ __forceinline__ void fetch_row(const AttnArgs& a, int item, int items, int lane, Fetch& f) {
  f.row = -1;
  if (item >= items) return;
  f.g = item % a.G;
  const int t = item / a.G;
  f.split = t % a.splits;
  f.row = t / a.splits;
  f.info = __ldcg((a.lead ? a.lead : a.rows) + f.row);
  if (a.block_idx) {
    const int32_t* ids = a.block_idx + ((size_t)f.row * a.G + f.g) * a.k;
    const int at = f.split * a.per_split + lane;
    f.id = at < a.k ? __ldcg(ids + at) : -1;
    f.before = at > 0 && at < a.k ? __ldcg(ids + at - 1) : -1;
#pragma unroll
    for (int c = 0; c < 4; ++c) f.ids[c] = c * 32 + lane < a.k ? __ldcg(ids + c * 32 + lane) : -1;
  }
}

__device__ __forceinline__ void fetch_pages(const AttnArgs& a, int lane, Fetch& f) {
  f.page = -1;
  if (f.row < 0) return;
  if (f.info.x < 0) {
    f.row = -1;
    return;
  }
  if (a.lead) f.row = f.info.z;
  if (a.block_idx) {
    int have = 0;  // ids stand at the front of the list
#pragma unroll
    for (int c = 0; c < 4; ++c) have += __popc(__ballot_sync(0xffffffffu, f.ids[c] >= 0));
    if (have > a.splits * a.per_split) {  // more ids than the table has columns: the parts are counted for no more
      if (lane == 0) dev_fail(a.err, kDevBadIndex, 1411);
      have = a.splits * a.per_split;
    }
    f.parts = max(1, (have + a.per_split - 1) / a.per_split);
    f.pages = min(a.per_split, have - f.split * a.per_split);
    if (f.pages <= 0 && f.split) f.row = -1;  // a row without any block has one item, without pages
    f.pages = max(f.pages, 0);
    f.block = f.id;
  } else {
    const int rows = min(a.tile_rows, f.info.w);
    const int own = (f.info.y + rows - 1) / 128 + 1 - a.prefix;  // pages up to the own one of the tile's last row
    f.parts = (own + a.per_split - 1) / a.per_split;
    f.pages = min(a.per_split, own - f.split * a.per_split);
    if (f.pages <= 0) f.row = -1;
    f.block = a.prefix + f.split * a.per_split + lane;
  }
  if (f.row < 0 || lane >= f.pages) f.block = -1;
  else if (f.block >= 0 && f.block <= f.info.y / 128 + a.tile_rows)
    f.page = __ldcg(a.page_table + (size_t)f.info.x * a.max_blocks + min(f.block, a.max_blocks - 1));
}

// The page as it was read, or -1 (reported) where it may not be: ids ascend up to the row's own block, pages lie in
// the pool. `before`: the list's id in front of this one, or -1.
__device__ __forceinline__ int checked_page(const AttnArgs& a, const int4& info, int block, int before, int page) {
  if (a.block_idx && (block < 0 || block > info.y / 128 || before >= block)) {
    dev_fail(a.err, kDevBadIndex, 1411);
    return -1;
  }
  if (page < 0 || page >= a.num_pages) {
    dev_fail(a.err, kDevBadIndex, 1412);
    return -1;
  }
  return page;
}

// Joins an item's (row tile, group), every kJoinWarps-th column from `first`
// on: the parts in their order, two columns and eight parts in flight.
__device__ __forceinline__ void join_parts(const AttnArgs& a, const AttnItem& item, int first, int lane) {
  const size_t step = (size_t)a.N * a.Hq;
  const int cols = item.rows * a.hg;
  for (int c0 = first; c0 < cols; c0 += 2 * kJoinWarps) {
    size_t at[2];
    float mm[2], den[2] = {0.f, 0.f};
    float4 acc[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int col = min(c0 + x * kJoinWarps, cols - 1);
      at[x] = (size_t)(item.row + (col >> a.hg_log2)) * a.Hq + item.g * a.hg + (col & (a.hg - 1));
      mm[x] = -INFINITY;
      acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = lane; i < item.parts; i += 32) mm[x] = fmaxf(mm[x], __ldcg(a.part_lse + i * step + at[x]));
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int o = 16; o; o >>= 1) mm[x] = fmaxf(mm[x], __shfl_xor_sync(0xffffffffu, mm[x], o));
#pragma unroll 8
    for (int i = 0; i < item.parts; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float lse = __ldcg(a.part_lse + i * step + at[x]);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + (i * step + at[x]) * 128) + lane);
        const float w = lse == -INFINITY ? 0.f : fast_exp2(lse - mm[x]);
        den[x] += w;
        acc[x].x = fmaf(w, v.x, acc[x].x);
        acc[x].y = fmaf(w, v.y, acc[x].y);
        acc[x].z = fmaf(w, v.z, acc[x].z);
        acc[x].w = fmaf(w, v.w, acc[x].w);
      }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      if (c0 + x * kJoinWarps >= cols) break;
      const bool none = den[x] == 0.f;  // (NaN scores: a maximum of -infinity, too, but a sum of NaN)
      const float inv = none ? 0.f : 1.f / den[x];
      reinterpret_cast<uint2*>(a.O + at[x] * 128)[lane] =
          make_uint2(pack_bf16(acc[x].x * inv, acc[x].y * inv), pack_bf16(acc[x].z * inv, acc[x].w * inv));
      if (lane == 0) a.LSE[at[x]] = none ? -INFINITY : (mm[x] + log2f(den[x])) * 0.6931471805599453f;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(AttnArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ AttnShared sh;
  uint8_t* s_q = smem + kStages * 2 * kTile;  // [2][kCols][kQStride]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.k_full[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.q_full[i], 1);
      mbar_init(&sh.q_empty[i], kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.j_full[i], kWarps);
      mbar_init(&sh.j_empty[i], kJoinWarps);
    }
    mbar_init(&sh.meet, kWarps);
    fence_barrier_init();
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  pdl_release();
  __syncthreads();
  if (!a.beside) pdl_wait();

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    uint32_t st = 0, st_ph = 0;  // stage and its parity
    int n_item = 0;              // items handed over
    bool ok = true;
    // Items are taken as they come, the first one by the CTA's number: their lengths differ. The next one is looked for
    // when the last four pages are being asked for, one step a page: its number, its row, its pages.
    const int items = a.lead ? __ldcg(a.header + kLeadCount) * a.splits * a.G : a.items;
    int id = blockIdx.x, id_next = 0, taken = 0, step = 0;
    Fetch now, next;
    auto advance = [&]() {
      if (step == 0) {
        if (lane == 0) taken = atomicAdd(a.header + kWorkNext, 1);
      } else if (step == 1) {
        id_next = gridDim.x + __shfl_sync(0xffffffffu, taken, 0);
        fetch_row(a, id_next, items, lane, next);
      } else if (step == 2) {
        fetch_pages(a, lane, next);
      }
      ++step;
    };
    fetch_row(a, id, items, lane, now);
    fetch_pages(a, lane, now);
    for (; ok && id < items; id = id_next, now = next) {
      step = 0;
      if (now.row >= 0) {
        const int rows = min(a.tile_rows, now.info.w), qs = n_item & 1;
        if (!mbar_wait(&sh.q_empty[qs], ((n_item >> 1) & 1) ^ 1, a.err, 1401)) { ok = false; break; }
        if (lane == 0) {
          sh.item[qs] = {now.row, now.g, now.split, now.pages, now.parts, now.info.y, rows};
          mbar_arrive_expect_tx(&sh.q_full[qs], rows * a.hg * 256);
        }
        __syncwarp();
        if (lane < rows * a.hg)  // one column each
          bulk_load(s_q + (qs * kCols + lane) * kQStride,
                    a.Q + ((size_t)(now.row + (lane >> a.hg_log2)) * a.Hq + now.g * a.hg + (lane & (a.hg - 1))) * 128, 256,
                    &sh.q_full[qs]);
        ++n_item;
        for (int j0 = 0; j0 < now.pages && ok; j0 += 32) {
          int block = now.block, page = now.page, before = now.before;
          const int j = j0 + lane;
          if (j0 && j < now.pages) {  // past the fetched ones
            const int at = now.split * a.per_split + j;
            const int32_t* ids = a.block_idx ? a.block_idx + ((size_t)now.row * a.G + now.g) * a.k + at : nullptr;
            block = ids ? ld_in(ids) : a.prefix + at;
            before = ids ? ld_in(ids - 1) : -1;
            page = block >= 0 && block < a.max_blocks
                       ? ld_in(a.page_table + (size_t)now.info.x * a.max_blocks + block)
                       : -1;
          }
          if (j < now.pages) page = checked_page(a, now.info, block, before, page);
          const int here = min(32, now.pages - j0);
          for (int i = 0; i < here; ++i) {
            const int pg = __shfl_sync(0xffffffffu, page, i), bl = __shfl_sync(0xffffffffu, block, i);
            if (!mbar_wait(&sh.empty[st], st_ph ^ 1, a.err, 1402)) { ok = false; break; }
            if (lane == 0) {
              // a page that may not be read counts as one whose tokens all lie behind the row's end
              sh.token0[st] = pg >= 0 ? bl * 128 : 0x3fffff00;
              const int y = (max(pg, 0) * a.G + now.g) * 128;
              uint8_t* d = smem + st * 2 * kTile;
              mbar_arrive_expect_tx(&sh.k_full[st], kTile);
              tma_load_2d(d, &map_k, &sh.k_full[st], 0, y);
              tma_load_2d(d + kHalf, &map_k, &sh.k_full[st], 64, y);
              mbar_arrive_expect_tx(&sh.v_full[st], kTile);
              tma_load_2d(d + kTile, &map_v, &sh.v_full[st], 0, y);
              tma_load_2d(d + kTile + kHalf, &map_v, &sh.v_full[st], 64, y);
            }
            __syncwarp();
            if (++st == kStages) {
              st = 0;
              st_ph ^= 1;
            }
            if (now.pages - (j0 + i) <= 4) advance();
          }
        }
      }
      while (step < 3) advance();
    }
    // the end
    const int qs = n_item & 1;
    if (ok && mbar_wait(&sh.q_empty[qs], ((n_item >> 1) & 1) ^ 1, a.err, 1403)) {
      if (lane == 0) {
        sh.item[qs].pages = -1;
        mbar_arrive(&sh.q_full[qs]);
      }
    }
  } else if (warp > kWarps) {
    // ---------------------------------------------------------------- joining warps
    if (blockIdx.x == 0 && warp == kWarps + 1) report_flags(a.flags, a.n_flags, a.err, lane);
    for (int n_join = 0;; ++n_join) {
      const int js = n_join & 1;
      if (!mbar_wait(&sh.j_full[js], (n_join >> 1) & 1, a.err, 1431, a.idle_ns)) break;
      const AttnItem item = sh.join[js];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.j_empty[js]);
      if (item.parts == 0) break;
      // each warp counts for itself: the one that finds all parts done joins its columns
      int done = 0;
      if (lane == 0) {
        __threadfence();
        done = atomicAdd(a.arrived + ((size_t)item.row * a.G + item.g) * kJoinWarps + warp - kWarps - 1, 1);
      }
      if (__shfl_sync(0xffffffffu, done, 0) != item.parts - 1) continue;
      __threadfence();
      join_parts(a, item, warp - kWarps - 1, lane);
    }
    if (a.beside) pdl_wait();  // the kernel after this one takes both to be done
  } else {
    // ---------------------------------------------------------------- consumers
    const int r = lane >> 2, q = lane & 3;
    uint32_t st = 0, st_ph = 0, meet_ph = 0;
    int n_join = 0;  // items handed to the joining warps
    bool ok = true;
    for (int n_item = 0; ok; ++n_item) {
      const int qs = n_item & 1;
      if (!mbar_wait(&sh.q_full[qs], (n_item >> 1) & 1, a.err, 1421)) { ok = false; break; }
      const AttnItem item = sh.item[qs];
      if (item.pages < 0) break;
      const int cols = item.rows * a.hg;
      // query fragments: column r, dims 16 ks + 2 q, + 1 and + 8, + 9
      uint32_t qb[8][2];
      {
        const uint8_t* src = s_q + (qs * kCols + r) * kQStride;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qb[ks][0] = r < cols ? *reinterpret_cast<const uint32_t*>(src + ks * 32 + q * 4) : 0u;
          qb[ks][1] = r < cols ? *reinterpret_cast<const uint32_t*>(src + ks * 32 + 16 + q * 4) : 0u;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[qs]);
      const int lim_lo = item.pos + 1;
      int lim[2];  // first token that columns 2 q, + 1 do not see
#pragma unroll
      for (int z = 0; z < 2; ++z) lim[z] = lim_lo + ((2 * q + z) >> a.hg_log2);

      float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int z = 0; z < 4; ++z) o[mt][z] = 0.f;

      for (int j = 0; j < item.pages; ++j) {
        if (!mbar_wait(&sh.k_full[st], st_ph, a.err, 1422)) { ok = false; break; }
        const int token0 = sh.token0[st] + warp * 16;  // of this warp's keys
        const uint32_t kaddr = smem_u32(smem + st * 2 * kTile), vaddr = kaddr + kTile;
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};  // even and odd steps of the sum over d
        {
          const int key = warp * 16 + (lane & 15);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t f[4];
            ldmatrix_x4(f, kaddr + (ks >> 2) * kHalf + sw128_off(key, (ks & 3) * 2 + (lane >> 4)));
            mma_16816(ks & 1 ? sd : sc, f[0], f[1], f[2], f[3], qb[ks][0], qb[ks][1]);
          }
        }
        const bool masked = token0 + 16 > lim_lo;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          float v = (sc[z] + sd[z]) * a.scale_log2;
          if (masked && token0 + r + (z >> 1) * 8 >= lim[z & 1]) v = -INFINITY;
          sc[z] = v;
          mx[z & 1] = fmaxf(mx[z & 1], v);
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1)
#pragma unroll
          for (int z = 0; z < 2; ++z) mx[z] = fmaxf(mx[z], __shfl_xor_sync(0xffffffffu, mx[z], x));
        bool moved = false;
        float alpha[2], base[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float m_new = fmaxf(m_run[z], mx[z]);
          moved |= m_new > m_run[z];
          base[z] = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: exp2(-inf - 0) = 0
          alpha[z] = fast_exp2(m_run[z] - base[z]);
          m_run[z] = m_new;
        }
        if (__any_sync(0xffffffffu, moved)) {
          l_run[0] *= alpha[0];
          l_run[1] *= alpha[1];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int z = 0; z < 4; ++z) o[mt][z] *= alpha[z & 1];
        }
        // P as hi + lo, turned so that a lane holds two neighbouring keys of one column
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float p0 = fast_exp2(sc[2 * y] - base[0]);
          const float p1 = fast_exp2(sc[2 * y + 1] - base[1]);
          l_run[0] += p0;
          l_run[1] += p1;
          const uint32_t h = bf16_cut(p0, p1);
          ph[y] = movmatrix_trans(h);
          pl[y] = movmatrix_trans(bf16_rest(p0, p1, h));
        }
        if (!mbar_wait(&sh.v_full[st], st_ph, a.err, 1423)) { ok = false; break; }
        const int key = warp * 16 + (lane & 7) + ((lane >> 4) << 3);
        if (!masked || item.rows == 1) {
          const uint2 keep = keep_keys(token0 + 2 * q, masked ? lim_lo : 0x7fffffff);
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t f[4];
            ldmatrix_x4_trans(f, vaddr + (mt >> 2) * kHalf + sw128_off(key, (mt & 3) * 2 + ((lane >> 3) & 1)));
            const uint32_t v[4] = {f[0] & keep.x, f[1] & keep.x, f[2] & keep.y, f[3] & keep.y};
            mma_16816(o[mt], v[0], v[1], v[2], v[3], ph[0], ph[1]);
            mma_16816(o[mt], v[0], v[1], v[2], v[3], pl[0], pl[1]);
          }
        } else {
          // each row of the tile on its own: values behind its end cleared, and only its own columns kept
#pragma unroll 1
          for (int i = 0; i < item.rows; ++i) {
            const int end = lim_lo + i;
            if (token0 >= end) continue;
            const uint2 keep = keep_keys(token0 + 2 * q, end);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              uint32_t f[4];
              ldmatrix_x4_trans(f, vaddr + (mt >> 2) * kHalf + sw128_off(key, (mt & 3) * 2 + ((lane >> 3) & 1)));
              float t[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16816(t, f[0] & keep.x, f[1] & keep.x, f[2] & keep.y, f[3] & keep.y, ph[0], ph[1]);
              mma_16816(t, f[0] & keep.x, f[1] & keep.x, f[2] & keep.y, f[3] & keep.y, pl[0], pl[1]);
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (lim[z & 1] == end) o[mt][z] += t[z];
            }
          }
        }
        if (j + 1 == item.pages) break;  // the last page's stage is kept: the warps' results meet in it
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[st]);
        if (++st == kStages) {
          st = 0;
          st_ph ^= 1;
        }
      }
      if (!ok) break;

      // ---- the warps' results meet: each scales its O to the maximum of all and puts it into the last page's stage
      // ([warp][column][d], d exchanged by column against bank conflicts), and all 256 threads add up the eight
      const bool joined = a.join && item.parts > 1;
      const int d = threadIdx.x & 127;  // one dim of every other column
      auto put = [&](int col, float val, float lse) {
        const size_t at = (size_t)(item.row + (col >> a.hg_log2)) * a.Hq + item.g * a.hg + (col & (a.hg - 1));
        if (a.join && !joined) {
          a.O[at * 128 + d] = __float2bfloat16_rn(val);
          if (d == 0) a.LSE[at] = lse * 0.6931471805599453f;
        } else {
          const size_t pt = (size_t)(a.slot0 + item.split) * a.N * a.Hq + at;
          a.part_o[pt * 128 + d] = val;
          if (d == 0) a.part_lse[pt] = lse;
        }
      };
      if (item.pages == 0) {  // nothing selected
        for (int col = threadIdx.x >> 7; col < cols; col += 2) put(col, 0.f, -INFINITY);
      } else {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float l = l_run[z];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
          if (r == 0) {
            sh.m[warp][2 * q + z] = m_run[z];
            sh.l[warp][2 * q + z] = l;
          }
        }
        if (!warps_sync(&sh.meet, meet_ph, a.err, 1425)) { ok = false; break; }
        float* s_o = reinterpret_cast<float*>(smem + st * 2 * kTile);
        float* mine = s_o + warp * kCols * 128;
        float f[2];  // what this warp's O counts for (0 where no warp saw a key)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float mm = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][2 * q + z]);
          f[z] = fast_exp2(m_run[z] - (mm == -INFINITY ? 0.f : mm));
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            mine[(2 * q + (z & 1)) * 128 + ((mt * 16 + r + (z >> 1) * 8) ^ (q << 3))] = o[mt][z] * f[z & 1];
        {
          // this warp's column's sum: lane w % 8 has warp w's
          const float m = sh.m[lane & 7][warp];
          float mm = m;
#pragma unroll
          for (int x = 1; x < 8; x <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
          float den = fast_exp2(m - (mm == -INFINITY ? 0.f : mm)) * sh.l[lane & 7][warp];
#pragma unroll
          for (int x = 1; x < 8; x <<= 1) den += __shfl_xor_sync(0xffffffffu, den, x);
          if (lane == 0) {  // nothing but NaN scores: a maximum of -infinity and a sum of NaN, which stays
            sh.inv[warp] = den == 0.f ? 0.f : __fdividef(1.f, den);
            sh.lse[warp] = den == 0.f ? -INFINITY : mm + __log2f(den);
          }
        }
        if (!warps_sync(&sh.meet, meet_ph, a.err, 1426)) { ok = false; break; }
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          const int col = c + (threadIdx.x >> 7);
          if (col >= cols) break;
          float val = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) val += s_o[(w * kCols + col) * 128 + (d ^ ((col & 6) << 2))];
          put(col, val * sh.inv[col], sh.lse[col]);
        }
        fence_proxy_async_smem();  // the stage goes back to TMA
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[st]);
        if (++st == kStages) {
          st = 0;
          st_ph ^= 1;
        }
      }
      if (!ok) break;
      if (joined) {
        const int js = n_join & 1;
        if (!mbar_wait(&sh.j_empty[js], ((n_join >> 1) & 1) ^ 1, a.err, 1427)) { ok = false; break; }
        if (threadIdx.x == 0) sh.join[js] = item;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.j_full[js]);
        ++n_join;
      }
    }
    // the joining warps' end
    const int js = n_join & 1;
    if (mbar_wait(&sh.j_empty[js], ((n_join >> 1) & 1) ^ 1, a.err, 1428)) {
      if (threadIdx.x == 0) sh.join[js].parts = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.j_full[js]);
    }
  }
}

// ---------------------------------------------------------------------------
// Joins a row's parts: those of its sequence's own pages (the attention's splits,
// or the runs of the tcgen05 path) and the shared prefix's (one per run of pages
// that reaches into the group's), in that order.
// One warp per row and head. Nothing but latency costs anything here (29 MB from
// L2 at most among the measured cases), so eight parts are asked for at a time,
// their sums with them, and the maximum is kept as they come. Measured: 9 us for 256
// rows x 32 heads of six parts each.
struct MergeArgs {
  const int4* rows;
  const float *part_o, *part_lse;
  __nv_bfloat16* O;
  float* LSE;
  int N, Hq, G, hg, prefix, per_split, tile_rows, teams, pslots;
  const int* flags;  // [n_flags] of the prefix kernel's blocks
  int n_flags;
  int* err;
};

constexpr int kMergeThreads = 128;

__global__ void __launch_bounds__(kMergeThreads, 6) paged_merge_kernel(MergeArgs a) {
  pdl_release();
  const int lane = threadIdx.x % 32;
  const long long item = (long long)blockIdx.x * (kMergeThreads / 32) + threadIdx.x / 32;
  if (item >= (long long)a.N * a.Hq) return;
  const int row = (int)(item / a.Hq), g = (int)(item % a.Hq) / a.hg;
  const int units = a.G * a.prefix;
  const int pre = units ? team_of((g + 1) * a.prefix - 1, units, a.teams) - team_of(g * a.prefix, units, a.teams) + 1 : 0;
  pdl_wait();
  if (item == 0) report_flags(a.flags, a.n_flags, a.err, lane);
  const int4 info = ld_in(a.rows + row);
  if (info.x < 0) return;  // behind the last sequence, or left out
  // the last row of its tile (or pair of tiles) decides how far the items went
  const int lead = info.z % a.tile_rows, rows = min(a.tile_rows, info.w + lead);
  const int own = ((info.y - lead + rows - 1) / 128 - a.prefix) / a.per_split + 1, n = own + pre;
  const size_t step = (size_t)a.N * a.Hq;
  float m = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 8) {
    float lse[8];
    float4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j;
      const size_t at = (size_t)(i < own ? a.pslots + i : i - own) * step + item;
      lse[j] = -INFINITY;
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < n) {
        lse[j] = ld_in(a.part_lse + at);
        v[j] = ld_in(reinterpret_cast<const float4*>(a.part_o + at * 128) + lane);
      }
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, lse[j]);
    const float base = top == -INFINITY ? 0.f : top;  // (parts whose scores are all -infinity)
    const float old = fast_exp2(m - base);
    m = top;
    den *= old;
    acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w = fast_exp2(lse[j] - base);
      den += w;
      acc.x = fmaf(w, v[j].x, acc.x);
      acc.y = fmaf(w, v[j].y, acc.y);
      acc.z = fmaf(w, v[j].z, acc.z);
      acc.w = fmaf(w, v[j].w, acc.w);
    }
  }
  const float inv = 1.f / den;
  const uint2 out = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  reinterpret_cast<uint2*>(a.O + (size_t)item * 128)[lane] = out;
  if (lane == 0) a.LSE[item] = (m + log2f(den)) * 0.6931471805599453f;
}

cudaError_t launch_attn(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  static bool attr[kMaxDevices] = {};
  const int dslot = device_slot();
  if (!attr[dslot]) {
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem);
    if (e != cudaSuccess) return e;
    attr[dslot] = true;
  }
  count_launches(1);
  return launch_dependent(paged_attn_kernel, std::min(a.items, num_sms()), kThreads, kSmem, st, a, mk, mv);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedProb& p, const PagedCachePtrs& c, const PoolMaps& maps, const void* Q,
                              const int32_t* block_idx, void* O, float* LSE, uint8_t* ws, const PagedWs& L,
                              cudaStream_t st) {
  AttnArgs a;
  a.rows = reinterpret_cast<const int4*>(ws + L.rows);
  a.lead = L.tile_rows > 1 ? reinterpret_cast<const int4*>(ws + L.lead) : nullptr;
  a.header = reinterpret_cast<int*>(ws);
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.page_table = c.page_table;
  a.block_idx = block_idx;
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + L.part_lse);
  a.N = p.N;
  a.Hq = p.Hq;
  a.G = p.G;
  a.hg = p.hg;
  a.hg_log2 = p.hg == 8 ? 3 : p.hg == 4 ? 2 : p.hg - 1;
  a.k = p.k;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.prefix = L.prefix;
  a.splits = L.splits;
  a.per_split = L.per_split;
  a.tile_rows = L.tile_rows;
  a.items = p.N * L.splits * p.G;  // at most 2^28: more than one split only where N * G is small
  a.slot0 = L.pslots;
  a.join = L.pslots == 0;
  a.arrived = reinterpret_cast<int*>(ws + L.arrived);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.LSE = LSE;
  a.scale_log2 = p.scale * kLog2e;
  a.flags = reinterpret_cast<const int*>(ws + L.flags);
  a.beside = L.pslots > 0;
  a.n_flags = a.beside ? 0 : L.n_flags;
  a.err = reinterpret_cast<int*>(ws);
  a.idle_ns = kIdleNs + kIdlePageNs * L.per_split * (a.items / std::min(a.items, num_sms()) + 1);
  return launch_attn(a, maps.k, maps.v, st);
}

cudaError_t launch_paged_merge(const PagedProb& p, void* O, float* LSE, uint8_t* ws, const PagedWs& L,
                               cudaStream_t st) {
  MergeArgs a;
  a.rows = reinterpret_cast<const int4*>(ws + L.rows);
  a.part_o = reinterpret_cast<const float*>(ws + L.part_o);
  a.part_lse = reinterpret_cast<const float*>(ws + L.part_lse);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.LSE = LSE;
  a.N = p.N;
  a.Hq = p.Hq;
  a.G = p.G;
  a.hg = p.hg;
  a.prefix = L.prefix;
  a.per_split = L.per_split;
  a.tile_rows = L.tile_rows;
  a.teams = L.teams;
  a.pslots = L.pslots;
  if (L.run_rows) {
    a.per_split = L.per_run;
    a.tile_rows = L.run_rows;
  }
  a.flags = reinterpret_cast<const int*>(ws + L.flags);
  a.n_flags = L.n_flags;
  a.err = reinterpret_cast<int*>(ws);
  const long long items = (long long)p.N * p.Hq;
  count_launches(1);
  return launch_dependent(paged_merge_kernel, (unsigned)((items + 3) / 4), kMergeThreads, 0, st, a);
}

}  // namespace msa
