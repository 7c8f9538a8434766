// Full attention of a batch's new rows over the pages that all its sequences
// share: one pass over those pages for the whole batch.
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
// Work: all (group, page) pairs in a line, cut into `teams` runs of equal
// length; a run is walked by `pairs` CTAs at once, one per pair of tiles, so
// that a page is read from HBM once and from L2 by the others. A run leaves
// one partial O (fp32, normalised) and log-sum-exp per row and group.
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHeadroom = 8.f;  // P = exp2(s - m) stays <= 2^kHeadroom
constexpr int kThreads = 640;     // warp 0 TMA, warp 1 UMMA + TMEM; 2, 3 the rows; warps 4-11 and 12-19 softmax of tiles 0 and 1
constexpr int kTile = 32768;      // 128 rows x 128 bf16, two 64-column SW128 chunks
constexpr int kChunk = 16384;
constexpr int kStages = 2;        // K/V ring
constexpr int oQ = 0, oK = 2 * kTile, oV = oK + kStages * kTile;
constexpr int kSmem = oV + kStages * kTile + 1024;

struct PrefixArgs {
  RowsArgs lineup;
  int* flags;  // [blocks] what a block found wrong (the error word is cleared meanwhile; the merge reports it)
  const int32_t *page_table, *row_start;
  float *part_o, *part_lse;
  int S, N, Hq, G, hg, prefix, pairs, teams, num_pages, max_blocks;
  float scale_log2;
};

struct PrefixShared {
  int flag;
  uint64_t q_full, q_empty;
  uint64_t k0_full, kv_full[kStages];  // the first page's K; then a page's V with the next one's K
  uint64_t k_empty[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t pair[2][4];           // the two warps of a tile's 32 rows
  float row_max[2][2][128];      // [tile][half][row] of the page's scores (at the end: the row's sums)
  int raised[2][2][4];           // [tile][half][quarter] the page (counted from 1) at which this warp called the other
  uint32_t tmem_base;
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_prefix_kernel(PrefixArgs a, const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PrefixShared sh;
  __shared__ RowsShared sh_rows;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int team = blockIdx.x / a.pairs, pair = blockIdx.x % a.pairs;
  const int units = a.G * a.prefix;
  int u_begin = team_start(team, units, a.teams);
  const int u_end = team_start(team + 1, units, a.teams);
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
  pdl_release();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  // the first sequence with rows: its table holds the shared pages
  const int ref = find_sequence(a.row_start, a.S, 0, lane);
  int* const err = &sh.flag;
  if (ref >= a.S) u_begin = u_end;  // no rows at all
  const uint32_t tmem = sh.tmem_base;  // S_0 [0,128), S_1 [128,256), O_0 [256,384), O_1 [384,512)

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
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
    auto load_tile = [&](int at, const CUtensorMap* map, uint64_t* bar, int y) {
      tma_load_2d(smem + at, map, bar, 0, y);
      tma_load_2d(smem + at + kChunk, map, bar, 64, y);
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
      auto issue_o = [&](int t, int st, bool acc) {
        const uint32_t va = v_lo + st * (kTile >> 4), d = tmem + 256 + t * 128, p = tmem + t * 128;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          umma_bf16_ts_w(d, p + (ks >> 2) * 64 + (ks & 3) * 8, va + ks * (2048 >> 4), hi, id_o, ks > 0 ? 1u : (uint32_t)acc);
      };
      int seg = 0;
      for (int u = u_begin; u < u_end && ok; ++seg) {
        const int g = u / a.prefix, stop = min(u_end, (g + 1) * a.prefix), pages = stop - u;
        if (!mbar_wait(&sh.q_full, seg & 1, err, 1520)) { ok = false; break; }
        {
          const int st = kc % kStages;
          // (a later run's first K came with the V of the page before it)
          if (kc == 0 && !mbar_wait(&sh.k0_full, 0, err, 1513)) { ok = false; break; }
          tc_fence_after();
          issue_s(0, st);
          issue_s(1, st);
          umma_commit(&sh.k_empty[st]);
          if (pages == 1) umma_commit(&sh.q_empty);
        }
        for (int c = 0; c < pages && ok; ++c, ++kc) {
          const int st = kc % kStages, st1 = (kc + 1) % kStages;
          const uint32_t par = (kc / kStages) & 1;
          const bool last = c == pages - 1;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            // the page's V and the next one's K first: nothing then stands between P_t and its products
            if (c == 0 && !mbar_wait(&sh.o_free[t], (seg & 1) ^ 1, err, 1516 + t)) { ok = false; break; }
            if (t == 0 && !mbar_wait(&sh.kv_full[st], par, err, 1518)) { ok = false; break; }
            // P_t of this page written (and O_t rescaled if its row maximum moved)
            if (!mbar_wait(&sh.p_full[t], kc & 1, err, 1514 + t)) { ok = false; break; }
            tc_fence_after();
            issue_o(t, st, c > 0);
            if (t == 1) umma_commit(&sh.v_empty[st]);
            if (!last) {
              // the next page's S_t: after this PV_t in issue order, so it overwrites P_t only once read
              issue_s(t, st1);
              if (t == 1) {
                umma_commit(&sh.k_empty[st1]);
                if (c + 1 == pages - 1) umma_commit(&sh.q_empty);
              }
            } else {
              umma_commit(&sh.o_full[t]);
            }
          }
        }
        u = stop;
      }
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------------- rows, for the kernels after this one
    if (blockIdx.x == 0)
      line_up_rows(a.lineup, sh_rows, threadIdx.x - 64, 64, [] { asm volatile("bar.sync 1, 64;" ::: "memory"); });
  } else {
    // ---------------------------------------------------------------- softmax (thread = one head of one new row, 64 keys)
    const int t = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;
    const int quarter = warp & 3;
    const int lrow = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_at = tmem + lane_off + t * 128 + half * 64;        // this warp's scores, and P over their first half
    const uint32_t o_at = tmem + lane_off + 256 + t * 128 + half * 64;  // the columns of O that it rescales and reads out
    const int row = (2 * pair + t) * tile_rows + lrow / a.hg;
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
    int seg = 0;
    for (int u = u_begin; u < u_end && ok; ++seg) {
      const int g = u / a.prefix, stop = min(u_end, (g + 1) * a.prefix), pages = stop - u;
      float m_run = -INFINITY, l_run = 0.f;  // the maximum is the row's, the sum that of this warp's keys
      if (!mbar_wait(&sh.s_full[t], kc & 1, err, 1522 + t)) { ok = false; break; }
      for (int c = 0; c < pages && ok; ++c, ++kc) {
        tc_fence_after();
        float sv[64], mq[2];
        tmem_ld32_max(s_at, *reinterpret_cast<float(*)[32]>(sv), mq[0]);
        tmem_ld32_max(s_at + 32, *reinterpret_cast<float(*)[32]>(sv + 32), mq[1]);
        tmem_wait_ld();
        const float m_blk = fmaxf(mq[0], mq[1]) * a.scale_log2;
        sh.row_max[t][half][lrow] = m_blk;
        bool mine = c == 0 || __any_sync(0xffffffffu, m_blk > m_run + kHeadroom);  // this warp calls the other
        float l_add = 0.f;
        auto write_p = [&]() {
          float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              float p0 = sv[16 * h + 2 * z], p1 = sv[16 * h + 2 * z + 1];
              fma2(p0, p1, a.scale_log2, -m_run);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              if (z & 1) add2(t0, t1, p0, p1);
              else add2(s0, s1, p0, p1);
              pk[z] = pack_bf16(p0, p1);
            }
            tmem_st8(s_at + 8 * h, pk);
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
      const int slot = team - team_of(g * a.prefix, units, a.teams);
      const size_t at = ((size_t)slot * a.N + row) * a.Hq + g * a.hg + lrow % a.hg;
      const float inv = 1.f / l;
      float* dst = a.part_o + at * 128 + half * 64;
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        float o[16];
        tmem_ld16(o_at + z * 16, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] *= inv;
        if (row < a.N) {
          st_global8(dst + 16 * z, o);
          st_global8(dst + 16 * z + 8, o + 8);
        }
      }
      if (row < a.N && half == 0) a.part_lse[at] = m_run + log2f(l);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free[t]);
      u = stop;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = sh.flag;
  if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

cudaError_t launch_paged_prefix(const PagedProb& p, const PagedCachePtrs& c, const void* Q, uint8_t* ws,
                                const PagedWs& L, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  {
    // a tile's rows times the heads of one group: box {64 d, h_g heads, 128 / h_g rows}
    const uint64_t dims[3] = {128, (uint64_t)p.Hq, (uint64_t)p.N};
    const uint64_t strides[2] = {256, (uint64_t)p.Hq * 256};
    const uint32_t box[3] = {64, (uint32_t)p.hg, (uint32_t)(128 / p.hg)};
    if (!encode_tmap(&mq, const_cast<void*>(Q), 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if (!encode_pool_map(&mk, p, c.K) || !encode_pool_map(&mv, p, c.V)) return cudaErrorInvalidValue;
  PrefixArgs a;
  a.lineup = rows_args(p, c, ws, L);
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
  a.prefix = p.prefix;
  a.pairs = L.pairs;
  a.teams = L.teams;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.scale_log2 = p.scale * kLog2e;
  static bool attr[kMaxDevices] = {};
  const int dslot = device_slot();
  if (!attr[dslot]) {
    cudaError_t e = cudaFuncSetAttribute(paged_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr[dslot] = true;
  }
  count_launches(1);
  return launch_dependent(paged_prefix_kernel, L.teams * L.pairs, kThreads, kSmem, st, a, mq, mk, mv);
}

}  // namespace msa
