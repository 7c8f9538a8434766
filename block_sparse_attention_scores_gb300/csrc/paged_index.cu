// Index branch for new tokens over the paged cache: block maxima of the index
// scores, and each (row, group)'s own block plus its best k - 1 earlier ones.
//
// paged_scores_kernel reads every index key of a sequence once: a warp holds
// one page (128 keys x 64) in registers, straight from 16-byte loads, and
// multiplies it with the sequence's index queries (rows x groups, eight
// columns at a time). The sum over the 64 dims may run in any order, so the
// pieces that a thread loads serve as its matrix fragments as they are: no
// shared memory, no shuffles before the maximum.
//
// The selection has to be exact, not exact up to the rounding of fp32: the
// order of two blocks decides whole pages. An fp32 maximum v_c differs from
// the exact one by at most e_c = kErr * |q|_1 * max|k_c|, so the blocks whose
// interval [v_c - e_c, v_c + e_c] lies clear of the border are decided, and
// only the others (usually none) are scored again in 64 bits. kErr is 2^-20:
// four 16-deep products accumulated in fp32 lose a few 2^-24 of the sum of
// the products' magnitudes, which |q|_1 max|k| bounds.
#include "mma_sync.cuh"
#include "paged.h"
#include "sm100.cuh"

namespace msa {
namespace {

constexpr float kErr = 9.5367431640625e-07f;  // 2^-20
constexpr float kTiny = 1e-35f;               // products below the normal range may count as zero
constexpr int kScoreThreads = 128;
constexpr int kScorePages = kScoreThreads / 32;

struct ScoreArgs {
  const __nv_bfloat16 *q_idx, *k_idx;
  const int32_t *page_table, *row_start, *seq_len;
  float *pooled, *amax;
  int S, N, G, num_pages, max_blocks;
  int* err;
};

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__global__ void __launch_bounds__(kScoreThreads, 3) paged_scores_kernel(ScoreArgs a) {
  const int s = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int c = blockIdx.x * kScorePages + warp;
  const int begin = __ldg(a.row_start + s);
  int rows = __ldg(a.row_start + s + 1) - begin;
  if (begin < 0 || rows <= 0 || begin >= a.N) return;
  rows = min(rows, a.N - begin);
  // blocks before the last row's own one; all their tokens exist
  const int len = min(__ldg(a.seq_len + s), a.max_blocks * 128);
  if (len <= 0 || c >= (len - 1) / 128) return;
  const int page = __ldg(a.page_table + (size_t)s * a.max_blocks + c);
  const bool bad = page < 0 || page >= a.num_pages;
  if (bad && lane == 0) dev_fail(a.err, kDevBadIndex, 1301);
  const int r = lane >> 2, q = lane & 3;

  // key 16 m + r (x) and 16 m + 8 + r (y): dims 8 q .. 8 q + 7 and 32 + 8 q .. (one piece per h)
  uint4 x[8][2], y[8][2];
  const uint4* kp = reinterpret_cast<const uint4*>(a.k_idx + (size_t)(bad ? 0 : page) * 128 * 64) + r * 8 + q;
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[m][h] = ld_stream(kp + m * 128 + h * 4);
      y[m][h] = ld_stream(kp + m * 128 + 64 + h * 4);
    }
  uint32_t top = 0;  // largest magnitude, two bf16 at a time
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = x[m][h], v = y[m][h];
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                   __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                   __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
    }
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  if (lane == 0) a.amax[(size_t)s * a.max_blocks + c] = __uint_as_float(top << 16);

  const int cols = rows * a.G;
  const uint4* qp = reinterpret_cast<const uint4*>(a.q_idx + (size_t)begin * a.G * 64);
  for (int n0 = 0; n0 < cols; n0 += 8) {
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (n0 + r < cols) {
      w[0] = __ldg(qp + (size_t)(n0 + r) * 8 + q);
      w[1] = __ldg(qp + (size_t)(n0 + r) * 8 + 4 + q);
    }
    float best0 = -INFINITY, best1 = -INFINITY;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_16816(d, x[m][h].x, y[m][h].x, x[m][h].y, y[m][h].y, w[h].x, w[h].y);
        mma_16816(d, x[m][h].z, y[m][h].z, x[m][h].w, y[m][h].w, w[h].z, w[h].w);
      }
      best0 = fmaxf(best0, fmaxf(d[0], d[2]));  // a NaN score counts as -infinity (fmaxf leaves it out)
      best1 = fmaxf(best1, fmaxf(d[1], d[3]));
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, o));
      best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, o));
    }
    if (r == 0) {
      const size_t col = (size_t)begin * a.G + n0 + 2 * q;
      if (n0 + 2 * q < cols) a.pooled[col * a.max_blocks + c] = bad ? -INFINITY : best0;
      if (n0 + 2 * q + 1 < cols) a.pooled[(col + 1) * a.max_blocks + c] = bad ? -INFINITY : best1;
    }
  }
}

// ---------------------------------------------------------------------------
constexpr int kSelThreads = 128;
constexpr int kSelWarps = kSelThreads / 32;

struct SelectArgs {
  const int4* rows;
  const float *pooled, *amax;
  const __nv_bfloat16 *q_idx, *k_idx;
  const int32_t* page_table;
  int32_t* block_idx;
  int G, k, num_pages, max_blocks;
};

struct SelectShared {
  int count[2][kSelWarps];
  uint32_t word[kSelWarps];
  float fval[kSelWarps];
  int n_in, n_open;
  uint32_t chosen[256];  // one bit per block
  int scan[kSelWarps];
  float q[64];
};

// Order of floats as unsigned numbers.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float bf(const __nv_bfloat16 v) { return __bfloat162float(v); }

// The block's exact maximum for the query in sh.q, by one warp: keys whose
// fp32 score is within `margin` of the best one are summed in 64 bits.
__device__ double exact_max(const __nv_bfloat16* page, const float* q, float margin, int lane) {
  float s32[4];
  float best = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat16* k = page + (lane + 32 * i) * 64;
    float s = 0.f;
    for (int e = 0; e < 64; ++e) s = fmaf(q[e], bf(k[e]), s);
    s32[i] = s;
    best = fmaxf(best, s);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  double top = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    if (s32[i] < best - margin) continue;  // false for NaN: such a key is looked at in 64 bits
    const __nv_bfloat16* k = page + (lane + 32 * i) * 64;
    double t[4] = {0., 0., 0., 0.};
    for (int e = 0; e < 64; e += 4)
#pragma unroll
      for (int z = 0; z < 4; ++z) t[z] = fma((double)q[e + z], (double)bf(k[e + z]), t[z]);
    top = fmax(top, (t[0] + t[1]) + (t[2] + t[3]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

// One block per (row, group). Shared memory: the blocks' lower bounds as
// ordered keys, and room for the list of undecided blocks and their scores.
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(SelectArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SelectShared sh;
  const int rg = blockIdx.x, row = rg / a.G, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int4 info = a.rows[row];
  if (info.x < 0) return;
  const int n = info.y / 128;  // earlier blocks
  const int want = min(a.k - 1, n);
  int32_t* out = a.block_idx + (size_t)rg * a.k;
  if (want == n) {  // every earlier block is kept
    for (int i = tid; i < a.k; i += kSelThreads) out[i] = i <= n ? i : -1;
    return;
  }
  if (want == 0) {
    for (int i = tid; i < a.k; i += kSelThreads) out[i] = i == 0 ? n : -1;
    return;
  }
  double* score = reinterpret_cast<double*>(dyn);                             // [n] of the open blocks
  uint32_t* key = reinterpret_cast<uint32_t*>(score + a.max_blocks);          // [n]
  int* open = reinterpret_cast<int*>(key + a.max_blocks);                     // [n]
  const float* v = a.pooled + (size_t)rg * a.max_blocks;
  const float* am = a.amax + (size_t)info.x * a.max_blocks;

  // |q|_1
  if (tid < 64) sh.q[tid] = bf(a.q_idx[(size_t)rg * 64 + tid]);
  if (tid == 0) sh.n_in = sh.n_open = 0;
  for (int i = tid; i < 256; i += kSelThreads) sh.chosen[i] = 0;
  __syncthreads();
  float l1 = fabsf(sh.q[lane]) + fabsf(sh.q[lane + 32]);
#pragma unroll
  for (int o = 16; o; o >>= 1) l1 += __shfl_xor_sync(0xffffffffu, l1, o);
  const float err_q = l1 * kErr;
  auto err_of = [&](float amax) {
    const float e = fmaf(err_q, amax, kTiny);
    return e < 1e30f ? e : INFINITY;  // not finite, or so large that fp32 may have overflowed: undecided
  };

  uint32_t kmax = 0, kmin = 0xffffffffu;
  float emax = 0.f;
  for (int i = tid; i < n; i += kSelThreads) {
    const float e = err_of(am[i]), x = v[i];
    const uint32_t u = order_key(e < INFINITY ? x - e : -INFINITY);
    key[i] = u;
    kmax = max(kmax, u);
    kmin = min(kmin, u);
    emax = fmaxf(emax, e);
  }
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  kmin = __reduce_min_sync(0xffffffffu, kmin);
#pragma unroll
  for (int o = 16; o; o >>= 1) emax = fmaxf(emax, __shfl_xor_sync(0xffffffffu, emax, o));
  if (lane == 0) {
    sh.word[warp] = kmax;
    sh.fval[warp] = emax;
    sh.count[0][warp] = (int)kmin;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    kmax = max(kmax, sh.word[i]);
    kmin = min(kmin, (uint32_t)sh.count[0][i]);
    emax = fmaxf(emax, sh.fval[i]);
  }
  __syncthreads();

  // The largest threshold that at least `want` keys reach: lo is reached by enough, hi + 1 by too few.
  uint32_t lo = kmin, hi = kmax;
  for (int step = 0; lo < hi; ++step) {
    const uint32_t mid = lo + ((hi - lo + 1) >> 1);
    int cnt = 0;
    for (int i = tid; i < n; i += kSelThreads) cnt += key[i] >= mid;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) sh.count[step & 1][warp] = cnt;
    __syncthreads();
    cnt = 0;
#pragma unroll
    for (int i = 0; i < kSelWarps; ++i) cnt += sh.count[step & 1][i];
    if (cnt >= want) lo = mid;
    else hi = mid - 1;
    if (cnt == want) break;  // lo parts exactly `want` blocks from the rest
  }
  __syncthreads();
  const float theta = from_key(lo);  // `want` blocks have lower bounds >= theta, so no block with v + e < theta is chosen
  const float clear = theta + 2.f * emax;  // and one with v - e above this is: fewer than `want` upper bounds reach it
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    int kind = 0;
    if (i < n) {
      const float e = err_of(am[i]), x = v[i];
      if (!(e < INFINITY)) kind = 2;
      else if (x - e > clear) kind = 1;
      else if (x + e >= theta) kind = 2;
    }
    const unsigned in = __ballot_sync(0xffffffffu, kind == 1), op = __ballot_sync(0xffffffffu, kind == 2);
    int at = 0;
    if (lane == 0) {
      if (i < n) sh.chosen[i / 32] = in;
      if (in) atomicAdd(&sh.n_in, __popc(in));
      if (op) at = atomicAdd(&sh.n_open, __popc(op));
    }
    at = __shfl_sync(0xffffffffu, at, 0);
    if (kind == 2) open[at + __popc(op & ((1u << lane) - 1))] = i;
  }
  __syncthreads();
  const int n_open = sh.n_open, need = want - sh.n_in;
  if (n_open == need) {
    for (int i = tid; i < n_open; i += kSelThreads) atomicOr(&sh.chosen[open[i] / 32], 1u << (open[i] % 32));
  } else {
    // the border runs through the open blocks: their exact maxima decide, equal ones by the lower id
    for (int i = warp; i < n_open; i += kSelWarps) {
      const int c = open[i], page = a.page_table[(size_t)info.x * a.max_blocks + c];
      const float e = err_of(am[c]);
      double t = -INFINITY;
      if (page >= 0 && page < a.num_pages) t = exact_max(a.k_idx + (size_t)page * 128 * 64, sh.q, 2.f * e, lane);
      if (lane == 0) score[i] = t;
    }
    __syncthreads();
    for (int i = tid; i < n_open; i += kSelThreads) {
      const double t = score[i];
      const int c = open[i];
      int before = 0;
      for (int j = 0; j < n_open; ++j) before += score[j] > t || (score[j] == t && open[j] < c);
      if (before < need) atomicOr(&sh.chosen[c / 32], 1u << (c % 32));
    }
  }
  __syncthreads();
  // ascending ids, the own block after them, then -1
  const uint32_t w0 = sh.chosen[2 * tid], w1 = sh.chosen[2 * tid + 1];
  const int mine = __popc(w0) + __popc(w1);
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) sh.scan[warp] = before;
  __syncthreads();
  before -= mine;
  for (int i = 0; i < warp; ++i) before += sh.scan[i];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    for (uint32_t w = h ? w1 : w0; w; w &= w - 1) {
      if (before < want) out[before] = (2 * tid + h) * 32 + __ffs(w) - 1;
      ++before;
    }
  for (int i = want + tid; i < a.k; i += kSelThreads) out[i] = i == want ? n : -1;
}

}  // namespace

cudaError_t launch_paged_index(const PagedProb& p, const PagedCachePtrs& c, const void* q_idx, int32_t* block_idx,
                               uint8_t* ws, const PagedWs& L, cudaStream_t st) {
  ScoreArgs a;
  a.q_idx = static_cast<const __nv_bfloat16*>(q_idx);
  a.k_idx = static_cast<const __nv_bfloat16*>(c.k_idx);
  a.page_table = c.page_table;
  a.row_start = c.row_start;
  a.seq_len = c.seq_len;
  a.pooled = reinterpret_cast<float*>(ws + L.pooled);
  a.amax = reinterpret_cast<float*>(ws + L.amax);
  a.S = p.S;
  a.N = p.N;
  a.G = p.G;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.err = reinterpret_cast<int*>(ws);
  if (p.max_blocks > 1 && p.k > 1) {
    paged_scores_kernel<<<dim3((p.max_blocks - 1 + kScorePages - 1) / kScorePages, p.S), kScoreThreads, 0, st>>>(a);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  SelectArgs b;
  b.rows = reinterpret_cast<const int4*>(ws + L.rows);
  b.pooled = a.pooled;
  b.amax = a.amax;
  b.q_idx = a.q_idx;
  b.k_idx = a.k_idx;
  b.page_table = c.page_table;
  b.block_idx = block_idx;
  b.G = p.G;
  b.k = p.k;
  b.num_pages = p.num_pages;
  b.max_blocks = p.max_blocks;
  const int smem = p.max_blocks * 16;
  static bool attr[kMaxDevices] = {};
  const int dslot = device_slot();
  if (!attr[dslot]) {
    cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 8192 * 16);
    if (e != cudaSuccess) return e;
    attr[dslot] = true;
  }
  paged_select_kernel<<<p.N * p.G, kSelThreads, smem, st>>>(b);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace msa
