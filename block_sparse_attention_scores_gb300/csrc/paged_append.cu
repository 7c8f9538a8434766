// New tokens into the paged cache: rotation of K, Q and the index branch's
// keys and queries by their positions, and the copy of V, in one pass.
//
// Rotation of the pair (a, b) with frequency f at position t:
//   (a cos(t f) - b sin(t f),  b cos(t f) + a sin(t f)).
// The angle is kept as a fraction of a turn in 64-bit fixed point:
// frac(f / 2 pi) * 2^64 times t, modulo 2^64, is exact in t, so a position of
// a million costs no accuracy (a product in 32 bits is off by 0.06 radians
// there); the top 32 bits then give sin and cos in fp32.
//
// Every value is read and written once; nothing else moves. One block per new
// row: a row's K, V, Q and index vectors are cut into items of two 16-byte
// pieces (the two halves of eight pairs, or two neighbours), one thread each.
#include "paged.h"
#include "pdl.cuh"
#include "sm100.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 2;  // items a thread has loaded before it needs the angles

struct AppendArgs {
  RopeRows r;
  __nv_bfloat16 *K, *V, *k_idx;
  const int32_t *page_table, *row_start, *seq_len;
  int S, N, Hq, G, num_pages, max_blocks;
  int* err;
};

// Largest s with row_start[s] <= r, by the whole warp: 32 probes a step.
__device__ __forceinline__ int find_sequence(const int32_t* row_start, int S, int r, int lane) {
  int lo = 0, n = S + 1;  // the answer lies in [lo, lo + n); row_start[0] counts as 0
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool in = lane == 0 || (lane * step < n && __ldg(row_start + at) <= r);
    const unsigned m = __ballot_sync(0xffffffffu, in);
    const int last = 31 - __clz(m);
    const int left = n - last * step;
    lo += last * step;
    n = left < step ? left : step;
  }
  return lo;
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Item j of a vector: which two 16-byte pieces, and whether (and from which pair on) they are rotated.
__device__ __forceinline__ void item_pieces(int j, int rot, int interleaved, int& a, int& b, int& pair) {
  const bool turned = 16 * j < rot;
  if (turned && !interleaved) {
    a = j;
    b = j + rot / 16;
  } else {
    a = 2 * j;
    b = 2 * j + 1;
  }
  pair = turned ? 8 * j : -1;
}

__device__ __forceinline__ void rotate(uint4& x, uint4& y, const float2* cs, int interleaved) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&x);
  uint32_t* v = reinterpret_cast<uint32_t*>(&y);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[i], d = cs[4 + i];
      const float a0 = lo_f(u[i]), b0 = hi_f(u[i]), a1 = lo_f(v[i]), b1 = hi_f(v[i]);
      u[i] = pack(a0 * c.x - b0 * c.y, b0 * c.x + a0 * c.y);
      v[i] = pack(a1 * d.x - b1 * d.y, b1 * d.x + a1 * d.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[2 * i], d = cs[2 * i + 1];
      const float a0 = lo_f(u[i]), a1 = hi_f(u[i]), b0 = lo_f(v[i]), b1 = hi_f(v[i]);
      u[i] = pack(a0 * c.x - b0 * c.y, a1 * d.x - b1 * d.y);
      v[i] = pack(b0 * c.x + a0 * c.y, b1 * d.x + a1 * d.y);
    }
  }
}

__global__ void __launch_bounds__(kThreads) paged_append_kernel(AppendArgs a) {
  __shared__ float2 turn[64 + 32];  // cos, sin of the row's pairs: d, then d_idx
  __shared__ int place[3];          // sequence found, page (-1: not to be written), slot
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31;

  // the row's sequence and position; every warp looks them up, so that no warp waits for another's loads
  const int s = find_sequence(a.row_start, a.S, r, lane);
  if (s >= a.S) return;  // behind the last sequence
  const int len = __ldg(a.seq_len + s), end = __ldg(a.row_start + s + 1);
  if (len < end - r || len > a.max_blocks * 128) {
    if (tid == 0) dev_fail(a.err, kDevBadIndex, 1201);
    return;
  }
  const int pos = len - (end - r);
  if (tid == 0) {
    int page = __ldg(a.page_table + (size_t)s * a.max_blocks + (pos >> 7));
    if (page < 0 || page >= a.num_pages) {
      dev_fail(a.err, kDevBadIndex, 1202);
      page = -1;
    }
    place[1] = page;
    place[2] = pos & 127;
  }
  const int half = a.r.rot / 2, half_idx = a.r.rot_idx / 2;
  if (tid < 96) {
    const bool idx = tid >= 64;
    const int i = idx ? tid - 64 : tid;
    if (i < (idx ? half_idx : half)) {
      const double turns = (double)__ldg((idx ? a.r.inv_freq_idx : a.r.inv_freq) + i) * 0.15915494309189533577;
      const unsigned long long f = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
      const unsigned long long phase = f * (unsigned long long)pos;
      float sn, cs;
      sincospif((float)(int)(uint32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);  // the top 32 bits, in half turns
      turn[tid] = make_float2(cs, sn);
    }
  }

  // vectors: Hq queries, G keys, G values (8 items each), then G index queries and the index key (4 items each)
  const int n_q = a.r.Q ? 8 * a.Hq : 0, n_k = 8 * a.G, n_v = 8 * a.G;
  const int n_qi = a.r.q_idx ? 4 * a.G : 0, n_ki = a.r.k_idx ? 4 : 0;
  const int n = n_q + n_k + n_v + n_qi + n_ki;
  bool synced = false;
  for (int base = 0; base < n; base += kThreads * kInFlight) {
    uint4 x[kInFlight], y[kInFlight];
    int pa[kInFlight], pb[kInFlight], pair[kInFlight], kind[kInFlight], vec[kInFlight];
#pragma unroll
    for (int z = 0; z < kInFlight; ++z) {
      int it = base + z * kThreads + tid;
      kind[z] = -1;
      if (it >= n) continue;
      const __nv_bfloat16* src;
      if (it < n_q) {
        kind[z] = 0;
        src = static_cast<const __nv_bfloat16*>(a.r.Q) + (size_t)r * a.r.ld_Q;
      } else if ((it -= n_q) < n_k) {
        kind[z] = 1;
        src = static_cast<const __nv_bfloat16*>(a.r.K) + (size_t)r * a.r.ld_K;
      } else if ((it -= n_k) < n_v) {
        kind[z] = 2;
        src = static_cast<const __nv_bfloat16*>(a.r.V) + (size_t)r * a.r.ld_V;
      } else if ((it -= n_v) < n_qi) {
        kind[z] = 3;
        src = static_cast<const __nv_bfloat16*>(a.r.q_idx) + (size_t)r * a.r.ld_q_idx;
      } else {
        it -= n_qi;
        kind[z] = 4;
        src = static_cast<const __nv_bfloat16*>(a.r.k_idx) + (size_t)r * a.r.ld_k_idx;
      }
      const bool idx = kind[z] >= 3;
      vec[z] = idx ? it >> 2 : it >> 3;
      item_pieces(idx ? it & 3 : it & 7, kind[z] == 2 ? 0 : (idx ? a.r.rot_idx : a.r.rot), a.r.interleaved, pa[z],
                  pb[z], pair[z]);
      const uint4* v = reinterpret_cast<const uint4*>(src + (size_t)vec[z] * (idx ? 64 : 128));
      x[z] = v[pa[z]];
      y[z] = v[pb[z]];
    }
    if (!synced) {
      __syncthreads();
      synced = true;
    }
    const int page = place[1], slot = place[2];
#pragma unroll
    for (int z = 0; z < kInFlight; ++z) {
      if (kind[z] < 0) continue;
      const bool idx = kind[z] >= 3;
      if (pair[z] >= 0) rotate(x[z], y[z], turn + (idx ? 64 : 0) + pair[z], a.r.interleaved);
      __nv_bfloat16* dst;
      if (kind[z] == 0) {
        dst = static_cast<__nv_bfloat16*>(a.r.Q_out) + ((size_t)r * a.Hq + vec[z]) * 128;
      } else if (kind[z] == 3) {
        dst = static_cast<__nv_bfloat16*>(a.r.q_idx_out) + ((size_t)r * a.G + vec[z]) * 64;
      } else {
        if (page < 0) continue;
        if (kind[z] == 4)
          dst = a.k_idx + ((size_t)page * 128 + slot) * 64;
        else
          dst = (kind[z] == 1 ? a.K : a.V) + (((size_t)page * a.G + vec[z]) * 128 + slot) * 128;
      }
      reinterpret_cast<uint4*>(dst)[pa[z]] = x[z];
      reinterpret_cast<uint4*>(dst)[pb[z]] = y[z];
    }
  }
}

// ---------------------------------------------------------------------------
// First launch of the attentions: clears the error word and the counters of
// finished parts, and finds every new row's sequence and position. A row whose
// position lies outside the page table (or, behind a shared prefix, inside the
// prefix) is marked; the attention reports it and leaves it out.
struct RowsArgs {
  const int32_t *row_start, *seq_len;
  int4* rows;
  int *arrived, *err;
  int S, N, G, max_blocks, prefix;
};

constexpr int kStaged = 4096;  // sequence starts kept in shared memory

__global__ void __launch_bounds__(kThreads) paged_rows_kernel(RowsArgs a) {
  __shared__ int staged[kStaged];
  // released after the wait: the index scores, launched then, have only this kernel's own work to wait for (at their end)
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0 && tid < 64) a.err[tid] = 0;
  const bool all = a.S + 1 <= kStaged;
  if (all) {
    for (int i = tid; i <= a.S; i += kThreads) staged[i] = ld_in(a.row_start + i);
    __syncthreads();
  }
  auto start = [&](int i) { return all ? staged[i] : ld_in(a.row_start + i); };
  const int r = blockIdx.x * kThreads + tid;
  if (r >= a.N) return;
  for (int i = 0; i < 3 * a.G; ++i) a.arrived[(size_t)r * 3 * a.G + i] = 0;
  int lo = 0, hi = a.S + 1;  // start(lo) <= r (the first counts as 0), start(hi) > r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= r) lo = mid;
    else hi = mid;
  }
  int4 out = make_int4(-1, 0, 0, 0);
  if (lo < a.S) {
    const int len = ld_in(a.seq_len + lo), begin = start(lo), end = start(lo + 1);
    if (len < end - r + a.prefix * 128 || len > a.max_blocks * 128)
      out.x = -2;
    else
      out = make_int4(lo, len - (end - r), r - begin, (end < a.N ? end : a.N) - r);
  }
  a.rows[r] = out;
}

}  // namespace

cudaError_t launch_paged_append(const PagedProb& p, const PagedCachePtrs& c, const RopeRows& r, uint8_t* ws,
                                cudaStream_t st) {
  AppendArgs a;
  a.r = r;
  a.K = static_cast<__nv_bfloat16*>(c.K);
  a.V = static_cast<__nv_bfloat16*>(c.V);
  a.k_idx = static_cast<__nv_bfloat16*>(c.k_idx);
  a.page_table = c.page_table;
  a.row_start = c.row_start;
  a.seq_len = c.seq_len;
  a.S = p.S;
  a.N = p.N;
  a.Hq = p.Hq;
  a.G = p.G;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.err = reinterpret_cast<int*>(ws);
  paged_append_kernel<<<p.N, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_paged_rows(const PagedProb& p, const PagedCachePtrs& c, uint8_t* ws, const PagedWs& L,
                              cudaStream_t st) {
  RowsArgs a;
  a.row_start = c.row_start;
  a.seq_len = c.seq_len;
  a.rows = reinterpret_cast<int4*>(ws + L.rows);
  a.arrived = reinterpret_cast<int*>(ws + L.arrived);
  a.err = reinterpret_cast<int*>(ws);
  a.S = p.S;
  a.N = p.N;
  a.G = p.G;
  a.max_blocks = p.max_blocks;
  a.prefix = p.prefix;
  count_launches(1);
  return launch_dependent(paged_rows_kernel, (p.N + kThreads - 1) / kThreads, kThreads, 0, st, a);
}

}  // namespace msa
