// Attention of new tokens over pages of the cache: the selected pages of each
// (row, group), or a sequence's own pages behind a shared prefix.
//
// Few query columns against streamed keys: 64 KB of K and V per page and group
// serve at most 8 (or 16) columns, so the time is the memory's. One persistent
// CTA per SM: a producer warp keeps three whole pages in flight (192 KB, TMA
// boxes of half a page each), four warps take 32 keys of every page each:
//   S^T = K q^T   (mma.sync, keys in rows, columns = rows of the sequence x heads of the group)
//   P   = exp2(S scale log2 e - m), m the warp's own running maximum per column
//   O^T += V^T P^T, P as a sum of two bf16 values (16 bits of it: the rounding
//          of P would otherwise be as large as the output's own)
// with the warp's own maximum, sum and O in registers; the four warps meet once
// per item (a run of pages of one (row tile, group)), whose normalised O and
// log-sum-exp leave in fp32 for the merge.
//
// Masked places: a page is masked per column only where it crosses a row's end.
// There, each row of the tile is accumulated on its own with the values behind
// its end cleared, so that nothing stored behind a row's end (another row's
// tokens, stale cache lines, NaN or infinities) reaches it through 0 * x.
#include "mma_sync.cuh"
#include "paged.h"
#include "sm100.cuh"

namespace msa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;                          // consumers; the producer is warp kWarps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kHalf = 16384;                       // 128 rows x 64 bf16, 128-byte swizzle
constexpr int kTile = 2 * kHalf;                   // K or V of a page and group
constexpr int kStages = 3;
constexpr int kOStride = 132;                      // floats between columns of the warps' O (no bank conflicts)

template <int NT>
constexpr int smem_bytes() {
  return kStages * 2 * kTile + kWarps * 8 * kOStride * 4 + 2 * NT * 8 * 256 + 1024;
}

struct AttnArgs {
  const int4* rows;
  const __nv_bfloat16* Q;
  const int32_t *page_table, *block_idx;  // block_idx null: the sequence's own pages from block `prefix` on
  float *part_o, *part_lse;
  int N, Hq, G, hg, k, num_pages, max_blocks, prefix, splits, per_split, tile_rows, items, slot0;
  float scale_log2;
  int* err;
};

struct AttnShared {
  uint64_t k_full[kStages], v_full[kStages], empty[kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t meet;              // the consumer warps' rendezvous
  int4 item[2];               // row, group, split, pages (0: the end)
  int4 info[2];               // the first row's entry of the row table
  int token0[kStages];        // first token of the stage's page
  float m[kWarps][16], l[kWarps][16];
  int abort;
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Items: (row, split, group), group fastest. A row that does not lead its tile has none.
__device__ __forceinline__ void decode_item(int id, const AttnArgs& a, int& row, int& split, int& g) {
  g = id % a.G;
  const int t = id / a.G;
  split = t % a.splits;
  row = t / a.splits;
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(AttnArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ AttnShared sh;
  float* s_o = reinterpret_cast<float*>(smem + kStages * 2 * kTile);  // [warp][8 columns][kOStride]
  uint8_t* s_q = smem + kStages * 2 * kTile + kWarps * 8 * kOStride * 4;  // [2][NT * 8][256 bytes]
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
    mbar_init(&sh.meet, kWarps);
    sh.abort = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort_flag = &sh.abort;

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
    }
    uint32_t st = 0, st_ph = 0;  // stage and its parity
    int n_item = 0;              // items handed over
    bool ok = true;
    for (int id = blockIdx.x; ok && id < a.items; id += gridDim.x) {
      int row, split, g;
      decode_item(id, a, row, split, g);
      const int4 info = __ldg(a.rows + row);
      if (info.x < 0 || info.z % a.tile_rows) continue;
      const int rows = min(a.tile_rows, info.w);
      // the item's pages
      int first, count;
      if (a.block_idx) {
        // ids stand at the front of the list: as many as are >= 0
        first = split * a.per_split;
        const int32_t* ids = a.block_idx + ((size_t)row * a.G + g) * a.k;
        int have = 0;
        for (int j0 = 0; j0 < a.k; j0 += 32) {
          const int b = j0 + lane < a.k ? __ldg(ids + j0 + lane) : -1;
          have += __popc(__ballot_sync(0xffffffffu, b >= 0));
        }
        count = min(a.per_split, have - first);
      } else {
        const int last = (info.y + rows - 1) / 128;  // own block of the tile's last row
        first = a.prefix + split * a.per_split;
        count = min(a.per_split, last + 1 - first);
      }
      if (count <= 0) continue;
      const int qs = n_item & 1;
      if (!mbar_wait(&sh.q_empty[qs], ((n_item >> 1) & 1) ^ 1, a.err, 1401)) { ok = false; break; }
      if (lane == 0) {
        sh.item[qs] = make_int4(row, g, split, count);
        sh.info[qs] = info;
        mbar_arrive_expect_tx(&sh.q_full[qs], rows * a.hg * 256);
        for (int i = 0; i < rows; ++i)
          bulk_load(s_q + (qs * NT * 8 + i * a.hg) * 256, a.Q + ((size_t)(row + i) * a.Hq + g * a.hg) * 128,
                    a.hg * 256, &sh.q_full[qs]);
      }
      __syncwarp();
      ++n_item;
      for (int j0 = 0; j0 < count && ok; j0 += 32) {
        const int j = j0 + lane;
        int block = -1, page = -1;
        if (j < count) {
          block = a.block_idx ? __ldg(a.block_idx + ((size_t)row * a.G + g) * a.k + first + j) : first + j;
          // ids ascend, each one once, up to the row's own block
          if (a.block_idx &&
              (block < 0 || block > info.y / 128 ||
               (first + j > 0 && __ldg(a.block_idx + ((size_t)row * a.G + g) * a.k + first + j - 1) >= block))) {
            dev_fail(a.err, kDevBadIndex, 1411);
            block = -1;
          }
          if (block >= 0) page = __ldg(a.page_table + (size_t)info.x * a.max_blocks + block);
          if (block >= 0 && (page < 0 || page >= a.num_pages)) {
            dev_fail(a.err, kDevBadIndex, 1412);
            page = -1;
          }
        }
        const int here = min(32, count - j0);
        for (int i = 0; i < here; ++i) {
          const int pg = __shfl_sync(0xffffffffu, page, i), bl = __shfl_sync(0xffffffffu, block, i);
          if (!mbar_wait(&sh.empty[st], st_ph ^ 1, a.err, 1402)) { ok = false; break; }
          if (lane == 0) {
            // a page that may not be read counts as one whose tokens all lie behind the row's end
            sh.token0[st] = pg >= 0 ? bl * 128 : 0x3fffff00;
            const int y = (max(pg, 0) * a.G + g) * 128;
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
        }
      }
    }
    if (!ok) *abort_flag = 1;
    // the end: an item without pages
    const int qs = n_item & 1;
    if (ok && mbar_wait(&sh.q_empty[qs], ((n_item >> 1) & 1) ^ 1, a.err, 1403)) {
      if (lane == 0) {
        sh.item[qs] = make_int4(0, 0, 0, 0);
        mbar_arrive(&sh.q_full[qs]);
      }
    }
  } else {
    // ---------------------------------------------------------------- consumers
    const int r = lane >> 2, q = lane & 3;
    uint32_t st = 0, st_ph = 0, meet_ph = 0;
    bool ok = true;
    for (int n_item = 0; ok; ++n_item) {
      const int qs = n_item & 1;
      if (!mbar_wait(&sh.q_full[qs], (n_item >> 1) & 1, a.err, 1421)) { ok = false; break; }
      const int4 item = sh.item[qs], info = sh.info[qs];
      const int count = item.w;
      if (count == 0) break;
      const int rows = min(a.tile_rows, info.w), cols = rows * a.hg;
      // query fragments: column 8 nt + r, dims 16 ks + 2 q, + 1 and + 8, + 9
      uint32_t qb[NT][8][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = 8 * nt + r;
        const uint8_t* src = s_q + (qs * NT * 8 + col) * 256;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qb[nt][ks][0] = col < cols ? *reinterpret_cast<const uint32_t*>(src + ks * 32 + q * 4) : 0u;
          qb[nt][ks][1] = col < cols ? *reinterpret_cast<const uint32_t*>(src + ks * 32 + 16 + q * 4) : 0u;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[qs]);
      // first token that columns 8 nt + 2 q, + 1 do not see
      int lim[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int z = 0; z < 2; ++z) lim[nt][z] = info.y + 1 + (8 * nt + 2 * q + z) / a.hg;
      const int lim_lo = info.y + 1;

      float m_run[NT][2], l_run[NT][2], o[NT][8][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          m_run[nt][z] = -INFINITY;
          l_run[nt][z] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int z = 0; z < 4; ++z) o[nt][mt][z] = 0.f;
      }

      for (int j = 0; j < count; ++j) {
        if (!mbar_wait(&sh.k_full[st], st_ph, a.err, 1422)) { ok = false; break; }
        const int token0 = sh.token0[st];
        const uint32_t kaddr = smem_u32(smem + st * 2 * kTile), vaddr = kaddr + kTile;
        float sc[2][NT][4];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 4; ++z) sc[kt][nt][z] = 0.f;
          const int key = warp * 32 + kt * 16 + (lane & 15);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t f[4];
            ldmatrix_x4(f, kaddr + (ks >> 2) * kHalf + sw128_off(key, (ks & 3) * 2 + (lane >> 4)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(sc[kt][nt], f[0], f[1], f[2], f[3], qb[nt][ks][0], qb[nt][ks][1]);
          }
        }
        const bool masked = token0 + 128 > lim_lo;
        float mx[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              float v = sc[kt][nt][z] * a.scale_log2;
              if (masked && token0 + warp * 32 + kt * 16 + r + (z >> 1) * 8 >= lim[nt][z & 1]) v = -INFINITY;
              sc[kt][nt][z] = v;
              mx[nt][z & 1] = fmaxf(mx[nt][z & 1], v);
            }
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int z = 0; z < 2; ++z) mx[nt][z] = fmaxf(mx[nt][z], __shfl_xor_sync(0xffffffffu, mx[nt][z], x));
        bool moved = false;
        float alpha[NT][2], base[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float m_new = fmaxf(m_run[nt][z], mx[nt][z]);
            moved |= m_new > m_run[nt][z];
            base[nt][z] = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: exp2(-inf - 0) = 0
            alpha[nt][z] = fast_exp2(m_run[nt][z] - base[nt][z]);
            m_run[nt][z] = m_new;
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            l_run[nt][0] *= alpha[nt][0];
            l_run[nt][1] *= alpha[nt][1];
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
              for (int z = 0; z < 4; ++z) o[nt][mt][z] *= alpha[nt][z & 1];
          }
        }
        // P as hi + lo, turned so that a lane holds two neighbouring keys of one column
        uint32_t ph[2][NT][2], pl[2][NT][2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float p0 = fast_exp2(sc[kt][nt][2 * y] - base[nt][0]);
              const float p1 = fast_exp2(sc[kt][nt][2 * y + 1] - base[nt][1]);
              l_run[nt][0] += p0;
              l_run[nt][1] += p1;
              const uint32_t h = pack_bf16(p0, p1);
              ph[kt][nt][y] = movmatrix_trans(h);
              pl[kt][nt][y] = movmatrix_trans(pack_bf16(p0 - __uint_as_float(h << 16),
                                                        p1 - __uint_as_float(h & 0xffff0000u)));
            }
        if (!mbar_wait(&sh.v_full[st], st_ph, a.err, 1423)) { ok = false; break; }
        if (!masked) {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            const int key = warp * 32 + kt * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              uint32_t f[4];
              ldmatrix_x4_trans(f, vaddr + (mt >> 2) * kHalf + sw128_off(key, (mt & 3) * 2 + ((lane >> 3) & 1)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16816(o[nt][mt], f[0], f[1], f[2], f[3], ph[kt][nt][0], ph[kt][nt][1]);
                mma_16816(o[nt][mt], f[0], f[1], f[2], f[3], pl[kt][nt][0], pl[kt][nt][1]);
              }
            }
          }
        } else {
          // each row on its own: values behind its end cleared, and only its own columns kept
#pragma unroll 1
          for (int i = 0; i < rows; ++i) {
            const int end = lim_lo + i;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
              const int kbase = token0 + warp * 32 + kt * 16;
              if (kbase >= end) continue;
              const int key = warp * 32 + kt * 16 + (lane & 7) + ((lane >> 4) << 3);
              const int t0 = kbase + 2 * q;  // this lane's keys: t0, t0 + 1 (f0, f1) and t0 + 8, t0 + 9 (f2, f3)
              const uint32_t keep0 = (t0 < end ? 0xffffu : 0u) | (t0 + 1 < end ? 0xffff0000u : 0u);
              const uint32_t keep1 = (t0 + 8 < end ? 0xffffu : 0u) | (t0 + 9 < end ? 0xffff0000u : 0u);
#pragma unroll
              for (int mt = 0; mt < 8; ++mt) {
                uint32_t f[4];
                ldmatrix_x4_trans(f, vaddr + (mt >> 2) * kHalf + sw128_off(key, (mt & 3) * 2 + ((lane >> 3) & 1)));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_16816(t, f[0] & keep0, f[1] & keep0, f[2] & keep1, f[3] & keep1, ph[kt][nt][0], ph[kt][nt][1]);
                  mma_16816(t, f[0] & keep0, f[1] & keep0, f[2] & keep1, f[3] & keep1, pl[kt][nt][0], pl[kt][nt][1]);
#pragma unroll
                  for (int z = 0; z < 4; ++z)
                    if ((8 * nt + 2 * q + (z & 1)) / a.hg == i) o[nt][mt][z] += t[z];
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[st]);
        if (++st == kStages) {
          st = 0;
          st_ph ^= 1;
        }
      }
      if (!ok) break;

      // ---- the four warps' results meet, eight columns at a time
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float l = l_run[nt][z];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
          if (r == 0) {
            sh.m[warp][8 * nt + 2 * q + z] = m_run[nt][z];
            sh.l[warp][8 * nt + 2 * q + z] = l;
          }
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float* mine = s_o + warp * 8 * kOStride;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int z = 0; z < 4; ++z) mine[(2 * q + (z & 1)) * kOStride + mt * 16 + r + (z >> 1) * 8] = o[nt][mt][z];
        if (!warps_sync(&sh.meet, meet_ph, a.err, 1424)) { ok = false; break; }
        const int d = threadIdx.x;  // 128 consumers: one dim each
        for (int c = 0; c < 8; ++c) {
          const int col = 8 * nt + c;
          if (col >= cols) break;
          float mm = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sh.m[w][col]);
          float num = 0.f, den = 0.f;
          if (mm > -INFINITY) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float f = fast_exp2(sh.m[w][col] - mm);
              num = fmaf(f, s_o[(w * 8 + c) * kOStride + d], num);
              den = fmaf(f, sh.l[w][col], den);
            }
          }
          const int row = item.x + col / a.hg, head = item.y * a.hg + col % a.hg;
          const size_t at = ((size_t)(a.slot0 + item.z) * a.N + row) * a.Hq + head;
          a.part_o[at * 128 + d] = mm > -INFINITY ? num / den : 0.f;
          if (d == 0) a.part_lse[at] = mm > -INFINITY ? mm + log2f(den) : -INFINITY;
        }
        if (!warps_sync(&sh.meet, meet_ph, a.err, 1425)) { ok = false; break; }
      }
    }
    if (!ok) *abort_flag = 1;
  }
}

// ---------------------------------------------------------------------------
// Joins a row's partials: the shared prefix's (one per run of pages that
// reaches into the group's) and the own pages' splits, in that order.
struct MergeArgs {
  const int4* rows;
  const int32_t* block_idx;
  const float *part_o, *part_lse;
  __nv_bfloat16* O;
  float* LSE;
  int N, Hq, G, hg, k, prefix, per_split, tile_rows, teams, pslots;
};

constexpr int kMergeThreads = 256;

__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(MergeArgs a) {
  const int lane = threadIdx.x % 32;
  const long long item = (long long)blockIdx.x * (kMergeThreads / 32) + threadIdx.x / 32;
  if (item >= (long long)a.N * a.Hq) return;
  const int row = (int)(item / a.Hq), head = (int)(item % a.Hq), g = head / a.hg;
  const int4 info = __ldg(a.rows + row);
  if (info.x < 0) return;  // behind the last sequence, or left out
  int own;                 // partials of the own pages
  if (a.block_idx) {
    int have = 0;
    for (int j0 = 0; j0 < a.k; j0 += 32) {
      const int b = j0 + lane < a.k ? __ldg(a.block_idx + ((size_t)row * a.G + g) * a.k + j0 + lane) : -1;
      have += __popc(__ballot_sync(0xffffffffu, b >= 0));
    }
    own = (have + a.per_split - 1) / a.per_split;
  } else {
    // the tile's last row decides how far its items went
    const int lead = info.z % a.tile_rows, rows = min(a.tile_rows, info.w + lead);
    const int last = (info.y - lead + rows - 1) / 128;
    own = (last - a.prefix) / a.per_split + 1;
  }
  int shared_parts = 0;
  if (a.teams) {
    const int units = a.G * a.prefix;
    shared_parts = team_of((g + 1) * a.prefix - 1, units, a.teams) - team_of(g * a.prefix, units, a.teams) + 1;
  }
  const int n = shared_parts + own;
  const size_t step = (size_t)a.N * a.Hq;
  auto slot = [&](int i) { return (size_t)(i < shared_parts ? i : a.pslots + i - shared_parts) * step + item; };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, a.part_lse[slot(i)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  if (m > -INFINITY) {
    for (int i = 0; i < n; ++i) {
      const size_t at = slot(i);
      const float w = fast_exp2(__ldg(a.part_lse + at) - m);
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.part_o + at * 128) + lane);
      den += w;
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint2 out = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  reinterpret_cast<uint2*>(a.O + (size_t)item * 128)[lane] = out;
  if (lane == 0) a.LSE[item] = m > -INFINITY ? (m + log2f(den)) * 0.6931471805599453f : -INFINITY;
}

template <int NT>
cudaError_t launch_attn(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  static bool attr[kMaxDevices] = {};
  const int dslot = device_slot();
  if (!attr[dslot]) {
    cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes<NT>());
    if (e != cudaSuccess) return e;
    attr[dslot] = true;
  }
  paged_attn_kernel<NT><<<std::min(a.items, num_sms()), kThreads, smem_bytes<NT>(), st>>>(a, mk, mv);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

bool encode_pool_map(CUtensorMap* m, const PagedProb& p, void* pool) {
  const uint64_t dims[2] = {128, (uint64_t)p.num_pages * p.G * 128};
  const uint64_t strides[1] = {256};
  const uint32_t box[2] = {64, 128};
  return encode_tmap(m, pool, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t launch_paged_attn(const PagedProb& p, const PagedCachePtrs& c, const void* Q, const int32_t* block_idx,
                              void* O, float* LSE, uint8_t* ws, const PagedWs& L, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!encode_pool_map(&mk, p, c.K) || !encode_pool_map(&mv, p, c.V)) return cudaErrorInvalidValue;
  AttnArgs a;
  a.rows = reinterpret_cast<const int4*>(ws + L.rows);
  a.Q = static_cast<const __nv_bfloat16*>(Q);
  a.page_table = c.page_table;
  a.block_idx = block_idx;
  a.part_o = reinterpret_cast<float*>(ws + L.part_o);
  a.part_lse = reinterpret_cast<float*>(ws + L.part_lse);
  a.N = p.N;
  a.Hq = p.Hq;
  a.G = p.G;
  a.hg = p.hg;
  a.k = p.k;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.prefix = p.prefix;
  a.splits = L.splits;
  a.per_split = L.per_split;
  a.tile_rows = L.tile_rows;
  a.items = p.N * L.splits * p.G;  // at most 2^28: more than one split only where N * G is small
  a.slot0 = L.pslots;
  a.scale_log2 = p.scale * kLog2e;
  a.err = reinterpret_cast<int*>(ws);
  return L.tile_rows * p.hg > 8 ? launch_attn<2>(a, mk, mv, st) : launch_attn<1>(a, mk, mv, st);
}

cudaError_t launch_paged_merge(const PagedProb& p, const int32_t* block_idx, void* O, float* LSE, uint8_t* ws,
                               const PagedWs& L, cudaStream_t st) {
  MergeArgs a;
  a.rows = reinterpret_cast<const int4*>(ws + L.rows);
  a.block_idx = block_idx;
  a.part_o = reinterpret_cast<const float*>(ws + L.part_o);
  a.part_lse = reinterpret_cast<const float*>(ws + L.part_lse);
  a.O = static_cast<__nv_bfloat16*>(O);
  a.LSE = LSE;
  a.N = p.N;
  a.Hq = p.Hq;
  a.G = p.G;
  a.hg = p.hg;
  a.k = p.k;
  a.prefix = p.prefix;
  a.per_split = L.per_split;
  a.tile_rows = L.tile_rows;
  a.teams = L.teams;
  a.pslots = L.pslots;
  const long long items = (long long)p.N * p.Hq;
  paged_merge_kernel<<<(unsigned)((items + 7) / 8), kMergeThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace msa
