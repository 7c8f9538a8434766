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
// Every value is read and written once; nothing else moves. A block takes one
// new row, or up to four where there are many short ones (the frequencies are then
// turned into fixed point once for all of them): a row's K, V, Q and index vectors are cut
// into items of two 16-byte pieces (the two halves of eight pairs, or two
// neighbours), one thread each, whose loads are on their way before the row's
// place and angles are looked up.
//
// Measured: 32,764 rows of 32 + 2 x 8 heads (881 MB) 139 us, 6.3 TB/s, 0.93 of a
// plain copy; one row 3 us in a graph, which is a launch's time. Into 8 bits 812 MB
// in 162 us (0.74): twice the instructions for K and V, and what bounds is issuing
// them.
//
// Positions with several axes (kind of token: time, height, width): a pair turns
// with the position on its own axis, position[r][axis[i]] * f, while the row's
// place in the cache stays its number in the sequence. Nothing else changes: the
// positions come with the row's place, one look-up for all axes.
//
// A cache in 8 bits (kBytes): K, V and k_idx become codes and a power of two
// (paged_fp8.cuh). Eight neighbouring threads hold a vector (four an index key),
// so its largest magnitude takes three shuffles, and the values are quantised in
// the registers in which they were rotated, from fp32, rounded once.
#include "paged_fp8.cuh"
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr int kInFlight = 2;  // items a thread loads at a time
constexpr int kMaxRows = 4;   // rows of a block
constexpr int kPairs = 64 + 32;
// Eight pairs' turns lie together, 80 bytes from the next eight's: the eight threads that rotate a vector meet in no bank
// (64 bytes apart they met four at a time).
constexpr int kTurns = kPairs / 8 * 10;
__device__ __forceinline__ int turn_at(int pair) { return pair + pair / 8 * 2; }
struct Turns {
  float2 c[8];
  __device__ __forceinline__ explicit Turns(const float2* at) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(at)[i];
      c[2 * i] = make_float2(v.x, v.y);
      c[2 * i + 1] = make_float2(v.z, v.w);
    }
  }
};
constexpr int kMaxAxes = 8;

struct AppendArgs {
  RopeRows r;
  void *K, *V, *k_idx;
  uint8_t *K_exp, *V_exp, *k_idx_exp;  // (kBytes)
  const int32_t *page_table, *row_start, *seq_len;
  int S, N, Hq, G, num_pages, max_blocks;
  int rows;                      // of a block
  int report;                    // the last block checks every row and writes the error word; the others write none
  int n_q, n_k, n_qi, n_ki;      // items of a row: queries, keys (values as many), index queries, its index key
  int items;                     // all (kBytes: made a multiple of eight, so that no vector's threads are in two warps)
  float inv_items;
  int* err;
};


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

__device__ __forceinline__ void rotate(uint4& x, uint4& y, const float2* at, int interleaved) {
  const Turns turns(at);
  const float2* cs = turns.c;
  uint32_t* u = reinterpret_cast<uint32_t*>(&x);
  uint32_t* v = reinterpret_cast<uint32_t*>(&y);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[i], d = cs[4 + i];
      const float a0 = lo_f(u[i]), b0 = hi_f(u[i]), a1 = lo_f(v[i]), b1 = hi_f(v[i]);
      u[i] = pack_bf16(a0 * c.x - b0 * c.y, b0 * c.x + a0 * c.y);
      v[i] = pack_bf16(a1 * d.x - b1 * d.y, b1 * d.x + a1 * d.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 c = cs[2 * i], d = cs[2 * i + 1];
      const float a0 = lo_f(u[i]), a1 = hi_f(u[i]), b0 = lo_f(v[i]), b1 = hi_f(v[i]);
      u[i] = pack_bf16(a0 * c.x - b0 * c.y, a1 * d.x - b1 * d.y);
      v[i] = pack_bf16(b0 * c.x + a0 * c.y, b1 * d.x + a1 * d.y);
    }
  }
}

// The rotated values of both pieces (pair < 0: as they are), not rounded: the first one's eight, then the second one's.
__device__ __forceinline__ void rotated_values(const uint4& x, const uint4& y, int pair, const float2* at, int interleaved,
                                               float (&v)[16]) {
  const uint32_t u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = lo_f(u[i]);
    v[2 * i + 1] = hi_f(u[i]);
  }
  if (pair < 0) return;
  const Turns turns(at);
  const float2* cs = turns.c;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 c = cs[i];
      const float a = v[2 * i], b = v[2 * i + 1];
      v[2 * i] = a * c.x - b * c.y;
      v[2 * i + 1] = b * c.x + a * c.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 c = cs[i];
      const float a = v[i], b = v[8 + i];
      v[i] = a * c.x - b * c.y;
      v[8 + i] = b * c.x + a * c.y;
    }
  }
}

// What an item is: kind 0 Q, 1 K, 2 V, 3 q_idx, 4 k_idx, 7 none; its vector, and pieces a and b of it, rotated from `pair` on.
struct What {
  int kind, row, vec, a, b, pair;
};
struct Piece {
  uint4 x, y;
  uint32_t what;  // packed (kind 3 bits, row 2, item of the vector 3, vector 24), so that the values have the registers
};
__device__ __forceinline__ What what_of(const AppendArgs& a, uint32_t what) {
  What w;
  w.kind = what >> 29;
  w.row = what >> 27 & 3;
  w.vec = what & 0xffffff;
  item_pieces(what >> 24 & 7, w.kind == 2 ? 0 : w.kind >= 3 ? a.r.rot_idx : a.r.rot, a.r.interleaved, w.a, w.b, w.pair);
  return w;
}

// Item `it` of the block's rows: which vector's pieces, and their loads.
__device__ __forceinline__ void load_piece(const AppendArgs& a, long long r0, int it, Piece& p) {
  p.what = 7u << 29;
  const int row = (int)(((float)it + 0.5f) * a.inv_items);
  it -= row * a.items;
  if (row >= a.rows || r0 + row >= a.N) return;
  int kind;
  const __nv_bfloat16* src;
  if (it < a.n_q) {
    kind = 0;
    src = static_cast<const __nv_bfloat16*>(a.r.Q) + r0 * a.r.ld_Q + row * a.r.ld_Q;
  } else if ((it -= a.n_q) < a.n_k) {
    kind = 1;
    src = static_cast<const __nv_bfloat16*>(a.r.K) + r0 * a.r.ld_K + row * a.r.ld_K;
  } else if ((it -= a.n_k) < a.n_k) {
    kind = 2;
    src = static_cast<const __nv_bfloat16*>(a.r.V) + r0 * a.r.ld_V + row * a.r.ld_V;
  } else if ((it -= a.n_k) < a.n_qi) {
    kind = 3;
    src = static_cast<const __nv_bfloat16*>(a.r.q_idx) + r0 * a.r.ld_q_idx + row * a.r.ld_q_idx;
  } else {
    it -= a.n_qi;
    if (it >= a.n_ki) return;  // (past the row's own items)
    kind = 4;
    src = static_cast<const __nv_bfloat16*>(a.r.k_idx) + r0 * a.r.ld_k_idx + row * a.r.ld_k_idx;
  }
  const bool idx = kind >= 3;
  p.what = (uint32_t)kind << 29 | row << 27 | (idx ? it & 3 : it & 7) << 24 | (idx ? it >> 2 : it >> 3);
  const What w = what_of(a, p.what);
  const uint4* v = reinterpret_cast<const uint4*>(src) + w.vec * (idx ? 8 : 16);
  p.x = v[w.a];
  p.y = v[w.b];
}

// Place of row r in a sequence of length len with `left` rows from r on, or a code for what is wrong with it.
__device__ __forceinline__ int place_row(const AppendArgs& a, int s, int len, int left, int& pos, int& page) {
  pos = page = -1;
  if (len < left || len > a.max_blocks * 128) return 1201;
  pos = len - left;
  page = ld_in(a.page_table + (size_t)s * a.max_blocks + (pos >> 7));
  if (page >= 0 && page < a.num_pages) return 0;
  page = -1;
  return 1202;
}

// What the axes of pair t (index pairs from 64 on) are: its own one, 0 (and `bad`) where there is none of that number.
__device__ __forceinline__ int pair_axis(const AppendArgs& a, int t, bool& bad) {
  const int32_t* axis = t < 64 ? a.r.axis : a.r.axis_idx;
  const int x = axis ? __ldg(axis + (t & 63)) : 0;
  if (x >= 0 && x < a.r.axes) return x;
  bad = true;
  return 0;
}

// A vector's codes and its power of two into the cache, by whole warps. `code`: this thread has a piece of such a vector,
// of which eight neighbouring threads (four: an index key) have one each. cs: the row's turns.
__device__ __forceinline__ void quantise_piece(const AppendArgs& a, const Piece& p, const What& e, bool code, int pos, int page,
                                               const float2* cs) {
  const bool idx = e.kind == 4;
  float v[16], most = 0.f;
  if (code && pos >= 0) {
    rotated_values(p.x, p.y, e.pair, cs + turn_at((idx ? 64 : 0) + max(e.pair, 0)), a.r.interleaved, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(v[i]));  // (leaves NaN out)
  }
  const auto over_vector = [&] {
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, most, o);
      if (o < 4 || !idx) most = fmaxf(most, other);
    }
  };
  over_vector();
  if (__any_sync(0xffffffffu, most == INFINITY)) {  // they become NaN and count for nothing in the scale
    most = 0.f;
    if (code && pos >= 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (!(fabsf(v[i]) < INFINITY)) v[i] = NAN;
        most = fmaxf(most, fabsf(v[i]));
      }
    }
    over_vector();
  }
  if (!code || pos < 0 || page < 0) return;
  const int byte = exp_byte(most), slot = pos & 127;
  const float scale = exp_inverse(byte);
  const uint32_t at = (idx ? page : page * a.G + e.vec) * 128 + slot;  // (pages times groups are below 2^24)
  uint8_t* dst = static_cast<uint8_t*>(idx ? a.k_idx : e.kind == 1 ? a.K : a.V) + (size_t)at * (idx ? 64 : 128);
  const uint2 lo = make_uint2(four_codes(v[0], v[1], v[2], v[3], scale), four_codes(v[4], v[5], v[6], v[7], scale));
  const uint2 hi = make_uint2(four_codes(v[8], v[9], v[10], v[11], scale), four_codes(v[12], v[13], v[14], v[15], scale));
  reinterpret_cast<uint2*>(dst)[e.a] = lo;
  reinterpret_cast<uint2*>(dst)[e.b] = hi;
  if (e.a == 0) (idx ? a.k_idx_exp : e.kind == 1 ? a.K_exp : a.V_exp)[at] = (uint8_t)byte;
}

template <bool kBytes, int kThreads>
__global__ void __launch_bounds__(kThreads, (kBytes ? 1024 : 1280) / kThreads) paged_append_kernel(AppendArgs a) {
  const int half = a.r.rot / 2, half_idx = a.r.rot_idx / 2;
  if (a.report && blockIdx.x == gridDim.x - 1) {
    int bad = 0;
    const auto start = [&](int i) { return ld_in(a.row_start + i); };
    for (int r = threadIdx.x; r < a.N; r += kThreads) {
      const int s = bisect_rows(start, a.S, r);
      int pos, page;
      if (s < a.S) bad = max(bad, place_row(a, s, ld_in(a.seq_len + s), start(s + 1) - r, pos, page));
    }
    bool axis = false;
    if (a.r.axes && threadIdx.x < kPairs) {
      const int t = threadIdx.x;
      if (t < 64 ? t < half : t - 64 < half_idx) pair_axis(a, t, axis);
    }
    const int second = __syncthreads_or(bad == 1202), first = __syncthreads_or(bad == 1201), third = __syncthreads_or(axis);
    const int where = first ? 1201 : second ? 1202 : third ? 1203 : 0;
    if (threadIdx.x == 0) *a.err = where ? kDevBadIndex * 65536 + where : kDevOk;
    return;
  }
  __shared__ unsigned long long turns_of[kPairs];  // frequency as a fraction of a turn per position
  __shared__ __align__(16) float2 turn[kMaxRows][kTurns];  // cos, sin of a row's pairs: d, then d_idx
  __shared__ int pos_of[kMaxRows], page_of[kMaxRows];  // -1: no row, or not to be written
  __shared__ int axis_of[kPairs], at_axis[kMaxRows][kMaxAxes];  // a pair's axis, and a row's positions on each
  const int r0 = blockIdx.x * a.rows, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Piece p[kInFlight];
#pragma unroll
  for (int z = 0; z < kInFlight; ++z) load_piece(a, r0, z * kThreads + tid, p[z]);

  if (tid >= kThreads - kPairs) {  // the last three warps
    const int t = tid - (kThreads - kPairs);
    const bool idx = t >= 64;
    const int i = idx ? t - 64 : t;
    if (i < (idx ? half_idx : half)) {
      const double turns = (double)__ldg((idx ? a.r.inv_freq_idx : a.r.inv_freq) + i) * 0.15915494309189533577;
      turns_of[t] = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
      if (a.r.axes) {
        bool bad = false;
        axis_of[t] = pair_axis(a, t, bad);
        if (bad && !a.report) dev_fail(a.err, kDevBadIndex, 1203);
      }
    }
  }
  if (warp < a.rows) {  // the rows' sequences, positions and pages, a warp each
    const int r = r0 + warp;
    int pos = -1, page = -1;
    if (r < a.N && lane < a.r.axes) at_axis[warp][lane] = __ldg(a.r.positions + (size_t)r * a.r.axes + lane);
    const int s = r < a.N ? find_sequence(a.row_start, a.S, r, lane) : a.S;
    if (s < a.S) {  // not behind the last sequence
      const int bad = place_row(a, s, ld_in(a.seq_len + s), ld_in(a.row_start + s + 1) - r, pos, page);
      if (bad && !a.report && lane == 0) dev_fail(a.err, kDevBadIndex, bad);
    }
    if (lane == 0) {
      pos_of[warp] = pos;
      page_of[warp] = page;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.rows * kPairs; i += kThreads) {
    const int row = i / kPairs, t = i - row * kPairs, pos = pos_of[row];
    if (pos >= 0 && (t < 64 ? t < half : t - 64 < half_idx)) {
      const long long at = a.r.axes ? at_axis[row][axis_of[t]] : pos;  // (modulo 2^64 a negative one turns backward)
      const unsigned long long phase = turns_of[t] * (unsigned long long)at;
      float sn, cs;
      sincospif((float)(int)(uint32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);  // the top 32 bits, in half turns
      turn[row][turn_at(t)] = make_float2(cs, sn);
    }
  }
  __syncthreads();

  for (int base = 0; base < a.rows * a.items; base += kThreads * kInFlight) {
    if (base) {
#pragma unroll
      for (int z = 0; z < kInFlight; ++z) load_piece(a, r0, base + z * kThreads + tid, p[z]);
    }
#pragma unroll
    for (int z = 0; z < kInFlight; ++z) {
      const What e = what_of(a, p[z].what);
      if constexpr (kBytes) {
        const bool code = e.kind == 1 || e.kind == 2 || e.kind == 4;
        if (__any_sync(0xffffffffu, code)) quantise_piece(a, p[z], e, code, pos_of[e.row], page_of[e.row], turn[e.row]);
        if (code) continue;
      }
      if (e.kind == 7) continue;
      const int pos = pos_of[e.row], page = page_of[e.row];
      if (pos < 0) continue;
      const bool idx = e.kind >= 3;
      if (e.pair >= 0) rotate(p[z].x, p[z].y, turn[e.row] + turn_at((idx ? 64 : 0) + e.pair), a.r.interleaved);
      const uint32_t r = r0 + e.row;  // (rows times heads are at most 2^28, pages times groups below 2^24)
      __nv_bfloat16* dst;
      if (e.kind == 0) {
        dst = static_cast<__nv_bfloat16*>(a.r.Q_out) + (size_t)(r * a.Hq + e.vec) * 128;
      } else if (e.kind == 3) {
        dst = static_cast<__nv_bfloat16*>(a.r.q_idx_out) + (size_t)(r * a.G + e.vec) * 64;
      } else {
        if (page < 0) continue;
        const int slot = pos & 127;
        if (e.kind == 4)
          dst = static_cast<__nv_bfloat16*>(a.k_idx) + (size_t)(page * 128u + slot) * 64;
        else
          dst = static_cast<__nv_bfloat16*>(e.kind == 1 ? a.K : a.V) + (size_t)((uint32_t)(page * a.G + e.vec) * 128 + slot) * 128;
      }
      reinterpret_cast<uint4*>(dst)[e.a] = p[z].x;
      reinterpret_cast<uint4*>(dst)[e.b] = p[z].y;
    }
  }
}

}  // namespace

template <bool kBytes, int kThreads>
static cudaError_t launch_append(const PagedProb& p, AppendArgs& a, cudaStream_t st) {
  // Rows for two rounds of a block's loads, so that its look-ups are shared, as long as every SM gets three blocks. 38,610
  // rows of 4 + 2 x 4 heads take 97 us with one row a block and 57 with four; 6,710 rows of 64 + 2 x 8, whose blocks are long
  // enough with one, 64 and 68; 2,400 rows of 8 + 2 x 2 heads 12 and 8.
  a.rows = std::min(kMaxRows, std::max(1, 2 * kInFlight * kThreads / a.items));
  while (a.rows > 1 && p.N < 3 * kCutSms * a.rows) --a.rows;
  paged_append_kernel<kBytes, kThreads><<<(p.N + a.rows - 1) / a.rows + a.report, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedProb& p, const PagedCachePtrs& c, const RopeRows& r, uint8_t* ws,
                                cudaStream_t st) {
  AppendArgs a;
  a.r = r;
  a.K = c.K;
  a.V = c.V;
  a.k_idx = c.k_idx;
  a.K_exp = c.K_exp;
  a.V_exp = c.V_exp;
  a.k_idx_exp = c.k_idx_exp;
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
  a.n_q = r.Q ? 8 * p.Hq : 0;
  a.n_k = 8 * p.G;
  a.n_qi = r.q_idx ? 4 * p.G : 0;
  a.n_ki = r.k_idx ? 4 : 0;
  a.items = a.n_q + 2 * a.n_k + a.n_qi + a.n_ki;
  if (c.bytes()) a.items = (a.items + 7) / 8 * 8;
  a.inv_items = 1.f / (float)a.items;
  // Few rows: a block of its own checks them and writes the error word, so that nothing has to clear it first (256 rows in
  // a graph: 3.0 us against 6.2 with a memset). For many rows it would be the last to end: 1024 sequences' rows 9.1 us
  // against 9.7, 2000 sequences' 16.8 against 12.3.
  a.report = p.N <= 1024;
  if (!a.report) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
    if (e != cudaSuccess) return e;
  }
  // Blocks of 128 threads for many long rows, whose waits for one another are shorter then: 32,764 rows of 32 + 2 x 8 heads
  // take 146 us with 256 threads and 139 with 128 in bf16, 170 and 162 in 8 bits; but 64 of them 4.0 and 5.0 us in a graph, and
  // 2,400 of 8 + 2 x 2 heads, of which a block has four, 8.4 and 10.4.
  const bool small = !a.report && a.items >= 256;
  if (c.bytes()) return small ? launch_append<true, 128>(p, a, st) : launch_append<true, 256>(p, a, st);
  return small ? launch_append<false, 128>(p, a, st) : launch_append<false, 256>(p, a, st);
}

}  // namespace msa
