// Index branch for new tokens over the paged cache: block maxima of the index
// scores, and each (row, group)'s own block plus its best k - 1 earlier ones.
//
// paged_scores_kernel reads every index key of a sequence once: a producer keeps
// twelve pages (128 keys x 64, 16 KB by TMA) in flight per SM, and each of twelve
// warps takes a whole page and multiplies it with the sequence's index queries
// (rows x groups, eight columns at a time, mma.sync): the memory's time, at a
// tenth of the tensor pipe's. Measured: two sequences of 2^20 tokens, 268 MB of
// keys in 44 us, 6.1 TB/s, 0.91 of a plain copy. The selection after it is all
// latency: 5 us for a row over 1,024 blocks, 15 over 8,192, 10.5 for 480 rows and
// groups over up to 256 each.
//
// All columns (rows x groups) of a sequence go through one warp a page: made for
// tokens and drafts. 16 rows x 8 groups over 8K tokens take the whole call 45 us, 256
// rows 437, and a prompt of 8,192 rows 13 ms (each row reads its own pages, too),
// where the training calls need 0.64 for the whole sequence.
//
// The selection has to be exact, not exact up to the rounding of fp32: the
// order of two blocks decides whole pages. An fp32 maximum v_c differs from
// the exact one by at most e_c = kErr * |q|_1 * max|k_c|, so the blocks whose
// interval [v_c - e_c, v_c + e_c] lies clear of the border are decided, and
// only the others (usually none) are scored again, exactly. kErr is
// 68 * 2^-23: each of the 64 products and four partial sums of a score may be
// cut off at fp32's step at the size of the largest of them, which |q|_1 max|k|
// bounds (measured: one large product among 63 small ones loses 2^-19.3 of it,
// normally distributed values 2^-24.5).
#include "mma_sync.cuh"
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr float kErr = 68.f / 8388608.f;
constexpr float kTiny = 1e-35f;               // products below the normal range may count as zero
constexpr int kScoreWarps = 12;
constexpr int kScoreThreads = (kScoreWarps + 1) * 32;  // the last warp loads
constexpr int kScoreStages = 12;
// page n lies in stage n % stages and is warp n % warps's: a stage is always the same warp's, so that nobody waits for a
// stage's next page before the one in it has been taken (a barrier's parity tells only two pages apart)
static_assert(kScoreStages % kScoreWarps == 0, "a stage belongs to one warp");
constexpr int kScorePage = 16384;
constexpr int kScoreQ = 8 * 128;  // the first eight columns' queries, which come with each page
constexpr int kScoreSmem = kScoreStages * (kScorePage + kScoreQ) + 1024;
constexpr int kScoreRun = 6;    // pages of a work item
constexpr int kScoreBatch = 5;  // items whose description is fetched at once (a lane per page)

struct ScoreArgs {
  const __nv_bfloat16* q_idx;
  const int32_t *page_table, *row_start, *seq_len;
  float2* pooled;
  int S, N, G, num_pages, max_blocks, runs, items;
  int* flags;  // [blocks but the last] what a block found wrong
  RowsArgs rows;
  unsigned long long wait_ns;  // a stage may be held for as long as a page takes a warp: the longer, the more columns
};


struct ScoreShared {
  uint64_t full[kScoreStages], empty[kScoreStages];
  int4 info[kScoreStages];  // sequence (-1: the end), block (its complement where the page may not be read), first row, columns
  int flag;
};

// The last block lines up the rows for the kernels after this one.
__global__ void __launch_bounds__(kScoreThreads, 1)
    paged_scores_kernel(ScoreArgs a, const __grid_constant__ CUtensorMap map_k) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (blockIdx.x == gridDim.x - 1) {
    pdl_release();
    pdl_wait();
    line_up_rows(a.rows, *reinterpret_cast<RowsShared*>(smem), threadIdx.x, kScoreThreads, [] { __syncthreads(); });
    return;
  }
  __shared__ ScoreShared sh;
  uint8_t* s_q = smem + kScoreStages * kScorePage;  // [stage][8][128]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ctas = gridDim.x - 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kScoreStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    sh.flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_k);
  }
  pdl_release();
  __syncthreads();
  pdl_wait();

  if (warp == kScoreWarps) {
    // ---------------------------------------------------------------- producer
    // An item is a run of pages of one sequence. Five of them are described by 30 lanes, one page each, and the next
    // five are fetched meanwhile.
    struct Batch {
      int s, c, begin, end, len, page;
    } now, next;
    const int step = ctas;
    auto fetch = [&](int first, Batch& f) {
      const int id = first + lane / kScoreRun * step;
      f.s = -1;
      f.c = f.begin = f.end = f.len = f.page = 0;
      if (lane >= kScoreRun * kScoreBatch || id >= a.items) return;
      f.s = id / a.runs;
      f.c = id % a.runs * kScoreRun + lane % kScoreRun;
      f.begin = ld_in(a.row_start + f.s);
      f.end = ld_in(a.row_start + f.s + 1);
      f.len = ld_in(a.seq_len + f.s);
      if (f.c < a.max_blocks) f.page = ld_in(a.page_table + (size_t)f.s * a.max_blocks + f.c);
    };
    int n = 0;  // pages handed over
    bool ok = true;
    fetch(blockIdx.x, now);
    for (int id = blockIdx.x; id < a.items && ok; id += kScoreBatch * step, now = next) {
      fetch(id + kScoreBatch * step, next);
      const int rows = min(now.end, a.N) - now.begin;
      // blocks before the last row's own one
      const bool want = now.s >= 0 && now.begin >= 0 && rows > 0 && now.len > 0 && now.len <= a.max_blocks * 128 &&
                        now.c < (now.len - 1) / 128;
      const bool bad = want && (now.page < 0 || now.page >= a.num_pages);
      if (bad) dev_fail(&sh.flag, kDevBadIndex, 1301);
      const int page = bad ? 0 : now.page, cols = rows * a.G;
      for (unsigned m = __ballot_sync(0xffffffffu, want); m; m &= m - 1, ++n) {
        const int from = __ffs(m) - 1, st = n % kScoreStages;
        if (!mbar_wait(&sh.empty[st], ((n / kScoreStages) & 1) ^ 1, &sh.flag, 1302, a.wait_ns)) { ok = false; break; }
        if (lane == from) {
          sh.info[st] = make_int4(now.s, bad ? ~now.c : now.c, now.begin, cols);
          const int first = min(cols, 8);
          mbar_arrive_expect_tx(&sh.full[st], kScorePage + first * 128);
          tma_load_2d(smem + st * kScorePage, &map_k, &sh.full[st], 0, page * 128);
          // (one copy: eight of 128 bytes that avoid bank conflicts took longer to issue than the page to arrive)
          bulk_load(s_q + st * kScoreQ, a.q_idx + (size_t)now.begin * a.G * 64, first * 128, &sh.full[st]);
        }
        __syncwarp();
      }
    }
    for (int i = 0; i < kScoreWarps && ok; ++i, ++n) {  // the end, for every warp
      const int st = n % kScoreStages;
      ok = mbar_wait(&sh.empty[st], ((n / kScoreStages) & 1) ^ 1, &sh.flag, 1302, a.wait_ns);
      if (ok && lane == 0) {
        sh.info[st].x = -1;
        mbar_arrive(&sh.full[st]);
      }
    }
  } else {
    // ---------------------------------------------------------------- one page per warp
    const int r = lane >> 2, q = lane & 3;
    for (int n = warp;; n += kScoreWarps) {
      const int st = n % kScoreStages;
      if (!mbar_wait(&sh.full[st], (n / kScoreStages) & 1, &sh.flag, 1303, a.wait_ns)) break;
      const int4 info = sh.info[st];
      if (info.x < 0) break;
      const bool bad = info.y < 0;
      const int c = bad ? ~info.y : info.y, cols = info.w;
      const uint32_t base = smem_u32(smem + st * kScorePage);
      const uint32_t* qp = reinterpret_cast<const uint32_t*>(a.q_idx + (size_t)info.z * a.G * 64);
      uint32_t top = 0;  // largest magnitude, two bf16 at a time (after the first columns: of all)
      for (int n0 = 0; n0 < cols; n0 += 8) {
        uint32_t b[4][2];  // queries' column n0 + r, dims 16 ks + 2 q, + 1 and + 8, + 9
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = ks * 8 + h * 4 + q;
            b[ks][h] = n0 + r >= cols ? 0u
                       : n0           ? ld_in(qp + (size_t)(n0 + r) * 32 + at)
                                      : *reinterpret_cast<const uint32_t*>(s_q + st * kScoreQ + r * 128 + at * 4);
          }
        float best0 = -INFINITY, best1 = -INFINITY;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            uint32_t f[4];
            ldmatrix_x4(f, base + sw128_off(m * 16 + (lane & 15), ks * 2 + (lane >> 4)));
            mma_16816(d, f[0], f[1], f[2], f[3], b[ks][0], b[ks][1]);
            if (n0 == 0)
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(f[0] & 0x7fff7fffu, f[1] & 0x7fff7fffu),
                                           __vmaxu2(f[2] & 0x7fff7fffu, f[3] & 0x7fff7fffu)));
          }
          best0 = fmaxf(best0, fmaxf(d[0], d[2]));  // a NaN score counts as -infinity (fmaxf leaves it out)
          best1 = fmaxf(best1, fmaxf(d[1], d[3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, o));
          best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, o));
        }
        if (n0 == 0) top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16)) << 16;
        if (r == 0) {
          const size_t col = (size_t)info.z * a.G + n0 + 2 * q;
          if (n0 + 2 * q < cols) a.pooled[col * a.max_blocks + c] = make_float2(bad ? -INFINITY : best0, __uint_as_float(top));
          if (n0 + 2 * q + 1 < cols) 
            a.pooled[(col + 1) * a.max_blocks + c] = make_float2(bad ? -INFINITY : best1, __uint_as_float(top));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = sh.flag;
}

// ---------------------------------------------------------------------------
struct SelectArgs {
  const int4* rows;
  const float2* pooled;
  const __nv_bfloat16 *q_idx, *k_idx;
  const int32_t* page_table;
  int32_t* block_idx;
  int G, k, num_pages, max_blocks;
};

struct SelectShared {
  uint2 count[2][32];
  uint32_t kmax[32], kmin[32];
  float emax[32];
  int n_in, n_open;
  uint32_t chosen[256];  // one bit per block
  int scan[32];
};

// Order of floats as unsigned numbers.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// Products of a query and a block's keys (exact in fp32) as integers, in units of 2^-57 of `most`, the largest that they
// could have, so that 64 of them stay below 2^63. `cut` says that one is not a whole number of units.
struct Units {
  float scale;
  double unit;
  __device__ __forceinline__ explicit Units(float most) {
    const int up = 56 - ((int)(__float_as_uint(most) >> 23) - 127);
    scale = __uint_as_float((uint32_t)(up + 127) << 23);
    unit = __longlong_as_double((long long)(1023 - up) << 52);
  }
  __device__ __forceinline__ long long of(float q, float k, bool& cut) const {
    const float x = q * k * scale;
    cut |= x != truncf(x);
    return __float2ll_rz(x);
  }
};

// The largest of a block's scores for a query (64 bf16 at q), by one warp, a key per lane. NaN where a product is cut.
__device__ __noinline__ double integer_max(const __nv_bfloat16* page, const __nv_bfloat16* q, float most, int lane) {
  const Units units(most);
  long long top = -0x7fffffffffffffffll;
  bool cut = false;
#pragma unroll 1
  for (int key = lane; key < 128; key += 32) {
    long long sum = 0;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      const uint4 w = ld_in(reinterpret_cast<const uint4*>(q) + c);
      const uint4 k = ld_in(reinterpret_cast<const uint4*>(page + key * 64) + c);
      const uint32_t wv[4] = {w.x, w.y, w.z, w.w}, kv[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) sum += units.of(lo_f(wv[z]), lo_f(kv[z]), cut) + units.of(hi_f(wv[z]), hi_f(kv[z]), cut);
    }
    top = max(top, sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  return __any_sync(0xffffffffu, cut) ? (double)NAN : (double)top * units.unit;
}

// s + e += t + f, with s the rounded sum and e what it lacks.
__device__ __forceinline__ void add_exactly(double& s, double& e, double t, double f) {
  const double sum = s + t, z = sum - s;
  e += f + ((s - (sum - z)) + (t - z));
  s = sum;
}

// The largest score among the keys of `near` (of lane i: the keys 32 i + bit), by one warp, two dims per lane.
__device__ __noinline__ double double_max(const __nv_bfloat16* page, uint32_t qq, unsigned near, int lane) {
  double top = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 4; ++i)
#pragma unroll 1
    for (unsigned m = __shfl_sync(0xffffffffu, near, i); m; m &= m - 1) {
      const uint32_t kk = ld_in(reinterpret_cast<const uint32_t*>(page + (__ffs(m) - 1 + 32 * i) * 64) + lane);
      double t = (double)lo_f(qq) * (double)lo_f(kk), e = 0.;
      add_exactly(t, e, (double)hi_f(qq) * (double)hi_f(kk), 0.);
#pragma unroll
      for (int o = 16; o; o >>= 1)
        add_exactly(t, e, __shfl_xor_sync(0xffffffffu, t, o), __shfl_xor_sync(0xffffffffu, e, o));
      top = fmax(top, e == e ? t + e : t);  // (e is NaN where t is not finite)
    }
  return top;
}

// The block's exact maximum for a query, rounded once, by one warp: a lane scores
// four keys in fp32, and the keys within `margin` of the best one are summed again.
// 64 fused steps are off by 64 * 2^-24 of the products' magnitudes at worst, so a
// difference of two scores by less than kErr of them.
//
// Those sums are of 64-bit integers: of few keys (as a rule one) with two dims per
// lane, of many, as where all keys of a block are the same (one token over and
// over: then every block is undecided, too), with a key per lane. Where products
// lie too far apart for that, or are not finite, of doubles with what their
// additions lose. A score is the same number in whichever way: one that was
// rounded in between could part equal keys.
__device__ __noinline__ double exact_max(const __nv_bfloat16* page, const __nv_bfloat16* q, float margin, float qmax,
                                         float kmax, int lane) {
  float s32[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 k[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        k[i][c] = ld_in(reinterpret_cast<const uint4*>(page + (lane + 32 * i) * 64 + 32 * h) + c);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 w = ld_in(reinterpret_cast<const uint4*>(q + 32 * h) + c);
      const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t kv[4] = {k[i][c].x, k[i][c].y, k[i][c].z, k[i][c].w};
#pragma unroll
        for (int z = 0; z < 4; ++z) s32[i] = fmaf(hi_f(wv[z]), hi_f(kv[z]), fmaf(lo_f(wv[z]), lo_f(kv[z]), s32[i]));
      }
    }
  }
  float best = fmaxf(fmaxf(s32[0], s32[1]), fmaxf(s32[2], s32[3]));
#pragma unroll
  for (int o = 16; o; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  unsigned near = 0;  // lane i: which keys 32 i + bit (the comparison is false for NaN: such a key is looked at again)
  int many = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned m = __ballot_sync(0xffffffffu, !(s32[i] < best - margin));
    if (lane == i) near = m;
    many += __popc(m);
  }
  const uint32_t qq = ld_in(reinterpret_cast<const uint32_t*>(q) + lane);
  const float most = qmax * kmax;
  double t = NAN;
  if (most >= 0x1p-60f && most <= 0x1p90f) {
    if (many > 8) {
      t = integer_max(page, q, most, lane);
    } else {
      const Units units(most);
      long long top = -0x7fffffffffffffffll;
      bool cut = false;
#pragma unroll 1
      for (int i = 0; i < 4; ++i)
#pragma unroll 1
        for (unsigned m = __shfl_sync(0xffffffffu, near, i); m; m &= m - 1) {
          const uint32_t kk = ld_in(reinterpret_cast<const uint32_t*>(page + (__ffs(m) - 1 + 32 * i) * 64) + lane);
          long long sum = units.of(lo_f(qq), lo_f(kk), cut) + units.of(hi_f(qq), hi_f(kk), cut);
#pragma unroll
          for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          top = max(top, sum);
        }
      if (!__any_sync(0xffffffffu, cut)) t = (double)top * units.unit;
    }
  }
  return t == t ? t : double_max(page, qq, near, lane);
}

// One block per (row, group). A thread keeps its blocks' lower bounds (as
// ordered keys) and errors in registers; shared memory has room for the list of
// undecided blocks and their scores.
template <int kThreads, int kSelItems>
__global__ void __launch_bounds__(kThreads) paged_select_kernel(SelectArgs a) {
  pdl_release();
  pdl_wait();
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SelectShared sh;
  const int rg = blockIdx.x, row = rg / a.G, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const __nv_bfloat16* q = a.q_idx + (size_t)rg * 64;
  const uint32_t qq = ld_in(reinterpret_cast<const uint32_t*>(q) + lane);
  const float2* v = a.pooled + (size_t)rg * a.max_blocks;
  float x[kSelItems], e[kSelItems];
#pragma unroll
  for (int z = 0; z < kSelItems; ++z) {  // (before it is known how many of them there are)
    const int i = z * kThreads + tid;
    const float2 f = a.k > 1 && i < a.max_blocks - 1 ? ld_in(v + i) : make_float2(-INFINITY, 0.f);
    x[z] = f.x;
    e[z] = f.y;
  }
  const int4 info = ld_in(a.rows + row);
  if (info.x < 0) return;
  const int n = info.y / 128;  // earlier blocks
  const int want = min(a.k - 1, n);
  int32_t* out = a.block_idx + (size_t)rg * a.k;
  if (want == n) {  // every earlier block is kept
    for (int i = tid; i < a.k; i += kThreads) out[i] = i <= n ? i : -1;
    return;
  }
  if (want == 0) {
    for (int i = tid; i < a.k; i += kThreads) out[i] = i == 0 ? n : -1;
    return;
  }
  double* score = reinterpret_cast<double*>(dyn);               // [n] of the open blocks
  int* open = reinterpret_cast<int*>(score + a.max_blocks);     // [n]

  if (tid == 0) sh.n_in = sh.n_open = 0;
  for (int i = tid; i < kThreads * kSelItems / 32; i += kThreads) sh.chosen[i] = 0;
  float l1 = fabsf(lo_f(qq)) + fabsf(hi_f(qq));  // |q|_1
#pragma unroll
  for (int o = 16; o; o >>= 1) l1 += __shfl_xor_sync(0xffffffffu, l1, o);
  const float err_q = l1 * kErr;

  uint32_t key[kSelItems], kmax = 0, kmin = 0xffffffffu;
  float emax = 0.f;
#pragma unroll
  for (int z = 0; z < kSelItems; ++z) {
    key[z] = 0u;
    if (z * kThreads >= n) continue;
    const bool in = z * kThreads + tid < n;
    const float t = fmaf(err_q, e[z], kTiny);
    e[z] = t < 1e30f ? t : INFINITY;  // not finite, or so large that fp32 may have overflowed: undecided
    key[z] = in ? order_key(e[z] < INFINITY ? x[z] - e[z] : -INFINITY) : 0u;  // 0: below every value
    if (in) {
      kmax = max(kmax, key[z]);
      kmin = min(kmin, key[z]);
      emax = fmaxf(emax, e[z]);
    }
  }
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  emax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(emax)));  // (not negative)
  if (lane == 0) {
    sh.kmax[warp] = kmax;
    sh.kmin[warp] = kmin;
    sh.emax[warp] = emax;
  }
  __syncthreads();
  kmax = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.kmax[lane] : 0u);
  kmin = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.kmin[lane] : 0xffffffffu);
  emax = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < kWarps ? __float_as_uint(sh.emax[lane]) : 0u));

  // A threshold that `want` keys reach: lo is reached by enough, hi + 1 by too few; three probes a step.
  uint32_t lo = kmin, hi = kmax;
  for (int step = 0; lo < hi; ++step) {
    const uint32_t w = ((hi - lo) >> 2) + 1, t1 = lo + w, t2 = min(t1 + w, hi), t3 = min(t2 + w, hi);
    uint32_t c12 = 0, c3 = 0;  // counts of t1 (low half), t2 (high half), t3
#pragma unroll
    for (int z = 0; z < kSelItems; ++z) {
      if (z * kThreads >= n) break;
      c12 += (key[z] >= t1 ? 1u : 0u) + (key[z] >= t2 ? 0x10000u : 0u);
      c3 += key[z] >= t3 ? 1u : 0u;
    }
    c12 = __reduce_add_sync(0xffffffffu, c12);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    if (lane == 0) sh.count[step & 1][warp] = make_uint2(c12, c3);
    __syncthreads();
    if (kWarps <= 8) {
      c12 = c3 = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const uint2 c = sh.count[step & 1][i];
        c12 += c.x;
        c3 += c.y;
      }
    } else {
      const uint2 c = sh.count[step & 1][lane];
      c12 = __reduce_add_sync(0xffffffffu, c.x);
      c3 = __reduce_add_sync(0xffffffffu, c.y);
    }
    const int n1 = c12 & 0xffff, n2 = c12 >> 16, n3 = c3;
    int got;
    if (n3 >= want) {
      lo = t3;
      got = n3;
    } else if (n2 >= want) {
      lo = t2;
      hi = t3 - 1;
      got = n2;
    } else if (n1 >= want) {
      lo = t1;
      hi = t2 - 1;
      got = n1;
    } else {
      hi = t1 - 1;
      got = -1;
    }
    if (got == want) break;  // lo parts exactly `want` blocks from the rest
  }
  const float theta = from_key(lo);  // `want` blocks have lower bounds >= theta, so no block with v + e < theta is chosen
  const float clear = theta + 2.f * emax;  // and one with v - e above this is: fewer than `want` upper bounds reach it
#pragma unroll
  for (int z = 0; z < kSelItems; ++z) {
    const int i = z * kThreads + tid;
    if (z * kThreads >= n) break;
    int kind = 0;
    if (i < n) {
      if (!(e[z] < INFINITY)) kind = 2;
      else if (x[z] - e[z] > clear) kind = 1;
      else if (x[z] + e[z] >= theta) kind = 2;
    }
    const unsigned in = __ballot_sync(0xffffffffu, kind == 1), op = __ballot_sync(0xffffffffu, kind == 2);
    int at = 0;
    if (lane == 0) {
      if (in) {
        sh.chosen[i / 32] = in;
        atomicAdd(&sh.n_in, __popc(in));
      }
      if (op) at = atomicAdd(&sh.n_open, __popc(op));
    }
    at = __shfl_sync(0xffffffffu, at, 0);
    if (kind == 2) open[at + __popc(op & ((1u << lane) - 1))] = i;
  }
  __syncthreads();
  const int n_open = sh.n_open, need = want - sh.n_in;
  if (n_open == need) {
    for (int i = tid; i < n_open; i += kThreads) atomicOr(&sh.chosen[open[i] / 32], 1u << (open[i] % 32));
  } else {
    // the border runs through the open blocks: their exact maxima decide, equal ones by the lower id
    float qmax = fmaxf(fabsf(lo_f(qq)), fabsf(hi_f(qq)));
    if (!(l1 < INFINITY)) qmax = INFINITY;  // (a NaN as well)
#pragma unroll
    for (int o = 16; o; o >>= 1) qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, o));
    for (int i = warp; i < n_open; i += kWarps) {
      const int c = open[i], page = ld_in(a.page_table + (size_t)info.x * a.max_blocks + c);
      const float top = ld_in(v + c).y, t0 = fmaf(err_q, top, kTiny), margin = t0 < 1e30f ? t0 : INFINITY;
      double t = -INFINITY;
      if (page < 0 || page >= a.num_pages) t = -INFINITY;  // (reported)
      else if ((qmax == 0.f || top == 0.f) && qmax < INFINITY && top < INFINITY) t = 0.;  // nothing but zeros
      else t = exact_max(a.k_idx + (size_t)page * 128 * 64, q, margin, qmax, top, lane);
      if (lane == 0) score[i] = t;
    }
    __syncthreads();
    for (int i = tid; i < n_open; i += kThreads) {
      const double t = score[i];
      const int c = open[i];
      int before = 0;
      for (int j = 0; j < n_open && before < need; ++j) before += score[j] > t || (score[j] == t && open[j] < c);
      if (before < need) atomicOr(&sh.chosen[c / 32], 1u << (c % 32));
    }
  }
  __syncthreads();
  // ascending ids, the own block after them, then -1
  static_assert(kSelItems <= 32, "a thread has a word of the chosen ones");
  uint32_t w = tid < kThreads * kSelItems / 32 ? sh.chosen[tid] : 0;
  int before = __popc(w);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) sh.scan[warp] = before;
  __syncthreads();
  before += (int)__reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)sh.scan[lane] : 0u) - __popc(w);
  for (; w; w &= w - 1, ++before)
    if (before < want) out[before] = tid * 32 + __ffs(w) - 1;
  for (int i = want + tid; i < a.k; i += kThreads) out[i] = i == want ? n : -1;
}

// As few threads as hold every block with eight each, fewer warps to wait for: 1,200 rows and groups of 40 blocks take
// 199 us in all with 128 threads, 211 with 256. (One warp, or half the threads with twice the blocks, is slower: a row
// over 8,192 blocks 72 us with 1,024 threads, 83 with 512, 89 with 256.)
template <int kThreads, int kSelItems>
cudaError_t launch_select(const PagedProb& p, const SelectArgs& a, cudaStream_t st) {
  static bool attr[kMaxDevices] = {};
  const int dslot = device_slot();
  if (!attr[dslot]) {
    cudaError_t e = cudaFuncSetAttribute(paged_select_kernel<kThreads, kSelItems>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (kThreads * kSelItems + 1) * 12);
    if (e != cudaSuccess) return e;
    attr[dslot] = true;
  }
  count_launches(1);
  return launch_dependent(paged_select_kernel<kThreads, kSelItems>, p.N * p.G, kThreads, p.max_blocks * 12, st, a);
}

// The rows alone, where no index scores are wanted and no prefix is shared.
constexpr int kRowThreads = 1024;  // 256 for up to as many rows: a smaller block starts sooner

__global__ void __launch_bounds__(kRowThreads) paged_rows_kernel(RowsArgs a) {
  __shared__ RowsShared sh;
  pdl_release();
  pdl_wait();
  line_up_rows(a, sh, threadIdx.x, blockDim.x, [] { __syncthreads(); });
}

}  // namespace

cudaError_t launch_paged_rows(const PagedProb& p, const PagedCachePtrs& c, uint8_t* ws, const PagedWs& L,
                              cudaStream_t st) {
  count_launches(1);
  return launch_dependent(paged_rows_kernel, 1, p.N <= 256 ? 256 : kRowThreads, 0, st, rows_args(p, c, ws, L));
}

cudaError_t launch_paged_index(const PagedProb& p, const PagedCachePtrs& c, const void* q_idx, int32_t* block_idx,
                               uint8_t* ws, const PagedWs& L, cudaStream_t st) {
  ScoreArgs a;
  a.q_idx = static_cast<const __nv_bfloat16*>(q_idx);
  a.page_table = c.page_table;
  a.row_start = c.row_start;
  a.seq_len = c.seq_len;
  a.pooled = reinterpret_cast<float2*>(ws + L.pooled);
  a.S = p.S;
  a.N = p.N;
  a.G = p.G;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.flags = reinterpret_cast<int*>(ws + L.flags);
  a.rows = rows_args(p, c, ws, L);
  a.wait_ns = kWaitLimitNs + 1000ull * p.N * p.G;  // eight columns take under a microsecond
  if (L.n_flags > 0) {
    CUtensorMap mk;
    const uint64_t dims[2] = {64, (uint64_t)p.num_pages * 128};
    const uint64_t strides[1] = {128};
    const uint32_t box[2] = {64, 128};
    if (!encode_tmap(&mk, c.k_idx, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
    a.runs = (p.max_blocks - 1 + kScoreRun - 1) / kScoreRun;
    a.items = p.S * a.runs;
    static bool attr[kMaxDevices] = {};
    const int dslot = device_slot();
    cudaError_t e;
    if (!attr[dslot]) {
      e = cudaFuncSetAttribute(paged_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem);
      if (e != cudaSuccess) return e;
      attr[dslot] = true;
    }
    count_launches(1);
    e = launch_dependent(paged_scores_kernel, L.n_flags + 1, kScoreThreads, kScoreSmem, st, a, mk);
    if (e != cudaSuccess) return e;
  } else {
    const cudaError_t e = launch_paged_rows(p, c, ws, L, st);
    if (e != cudaSuccess) return e;
  }
  SelectArgs b;
  b.rows = reinterpret_cast<const int4*>(ws + L.rows);
  b.pooled = a.pooled;
  b.q_idx = a.q_idx;
  b.k_idx = static_cast<const __nv_bfloat16*>(c.k_idx);
  b.page_table = c.page_table;
  b.block_idx = block_idx;
  b.G = p.G;
  b.k = p.k;
  b.num_pages = p.num_pages;
  b.max_blocks = p.max_blocks;
  const int n = p.max_blocks - 1;
  if (n <= 256) return launch_select<128, 2>(p, b, st);
  return n <= 2048 ? launch_select<256, 8>(p, b, st) : launch_select<1024, 8>(p, b, st);
}

}  // namespace msa
