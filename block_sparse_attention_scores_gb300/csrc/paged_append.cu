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
// Measured: 32,764 rows of 32 + 2 x 8 heads (881 MB) 150 us, 5.9 TB/s, 0.88 of a
// plain copy; one row 3 us in a graph, which is a launch's time.
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 2;  // items a thread loads at a time
constexpr int kMaxRows = 4;   // rows of a block
constexpr int kPairs = 64 + 32;

struct AppendArgs {
  RopeRows r;
  __nv_bfloat16 *K, *V, *k_idx;
  const int32_t *page_table, *row_start, *seq_len;
  int S, N, Hq, G, num_pages, max_blocks;
  int rows;                      // of a block
  int report;                    // the last block checks every row and writes the error word; the others write none
  int n_q, n_k, n_qi, items;     // items of a row: queries, keys (values as many), index queries; all
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

__device__ __forceinline__ void rotate(uint4& x, uint4& y, const float2* cs, int interleaved) {
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

struct Piece {
  uint4 x, y;
  int row, kind, vec, a, b, pair;  // kind -1: none; 0 Q, 1 K, 2 V, 3 q_idx, 4 k_idx
};

// Item `it` of the block's rows: which vector's pieces, and their loads.
__device__ __forceinline__ void load_piece(const AppendArgs& a, int r0, int it, Piece& p) {
  p.kind = -1;
  const int row = (int)(((float)it + 0.5f) * a.inv_items);
  it -= row * a.items;
  if (row >= a.rows || r0 + row >= a.N) return;
  p.row = row;
  const __nv_bfloat16* src;
  const size_t r = r0 + row;
  if (it < a.n_q) {
    p.kind = 0;
    src = static_cast<const __nv_bfloat16*>(a.r.Q) + r * a.r.ld_Q;
  } else if ((it -= a.n_q) < a.n_k) {
    p.kind = 1;
    src = static_cast<const __nv_bfloat16*>(a.r.K) + r * a.r.ld_K;
  } else if ((it -= a.n_k) < a.n_k) {
    p.kind = 2;
    src = static_cast<const __nv_bfloat16*>(a.r.V) + r * a.r.ld_V;
  } else if ((it -= a.n_k) < a.n_qi) {
    p.kind = 3;
    src = static_cast<const __nv_bfloat16*>(a.r.q_idx) + r * a.r.ld_q_idx;
  } else {
    it -= a.n_qi;
    p.kind = 4;
    src = static_cast<const __nv_bfloat16*>(a.r.k_idx) + r * a.r.ld_k_idx;
  }
  const bool idx = p.kind >= 3;
  p.vec = idx ? it >> 2 : it >> 3;
  item_pieces(idx ? it & 3 : it & 7, p.kind == 2 ? 0 : (idx ? a.r.rot_idx : a.r.rot), a.r.interleaved, p.a, p.b, p.pair);
  const uint4* v = reinterpret_cast<const uint4*>(src + (size_t)p.vec * (idx ? 64 : 128));
  p.x = v[p.a];
  p.y = v[p.b];
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

__global__ void __launch_bounds__(kThreads) paged_append_kernel(AppendArgs a) {
  if (a.report && blockIdx.x == gridDim.x - 1) {
    int bad = 0;
    const auto start = [&](int i) { return ld_in(a.row_start + i); };
    for (int r = threadIdx.x; r < a.N; r += kThreads) {
      const int s = bisect_rows(start, a.S, r);
      int pos, page;
      if (s < a.S) bad = max(bad, place_row(a, s, ld_in(a.seq_len + s), start(s + 1) - r, pos, page));
    }
    const int second = __syncthreads_or(bad == 1202), first = __syncthreads_or(bad == 1201);
    if (threadIdx.x == 0) *a.err = first ? kDevBadIndex * 65536 + 1201 : second ? kDevBadIndex * 65536 + 1202 : kDevOk;
    return;
  }
  __shared__ unsigned long long turns_of[kPairs];  // frequency as a fraction of a turn per position
  __shared__ float2 turn[kMaxRows][kPairs];        // cos, sin of a row's pairs: d, then d_idx
  __shared__ int pos_of[kMaxRows], page_of[kMaxRows];  // -1: no row, or not to be written
  const int r0 = blockIdx.x * a.rows, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Piece p[kInFlight];
#pragma unroll
  for (int z = 0; z < kInFlight; ++z) load_piece(a, r0, z * kThreads + tid, p[z]);

  const int half = a.r.rot / 2, half_idx = a.r.rot_idx / 2;
  if (tid >= kThreads - kPairs) {  // the last three warps
    const int t = tid - (kThreads - kPairs);
    const bool idx = t >= 64;
    const int i = idx ? t - 64 : t;
    if (i < (idx ? half_idx : half)) {
      const double turns = (double)__ldg((idx ? a.r.inv_freq_idx : a.r.inv_freq) + i) * 0.15915494309189533577;
      turns_of[t] = (unsigned long long)((turns - floor(turns)) * 18446744073709551616.0);
    }
  } else if (warp < a.rows) {  // the rows' sequences, positions and pages, a warp each
    const int r = r0 + warp;
    int pos = -1, page = -1;
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
      const unsigned long long phase = turns_of[t] * (unsigned long long)pos;
      float sn, cs;
      sincospif((float)(int)(uint32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);  // the top 32 bits, in half turns
      turn[row][t] = make_float2(cs, sn);
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
      Piece& e = p[z];
      if (e.kind < 0) continue;
      const int pos = pos_of[e.row], page = page_of[e.row];
      if (pos < 0) continue;
      const bool idx = e.kind >= 3;
      if (e.pair >= 0) rotate(e.x, e.y, turn[e.row] + (idx ? 64 : 0) + e.pair, a.r.interleaved);
      const size_t r = r0 + e.row;
      __nv_bfloat16* dst;
      if (e.kind == 0) {
        dst = static_cast<__nv_bfloat16*>(a.r.Q_out) + (r * a.Hq + e.vec) * 128;
      } else if (e.kind == 3) {
        dst = static_cast<__nv_bfloat16*>(a.r.q_idx_out) + (r * a.G + e.vec) * 64;
      } else {
        if (page < 0) continue;
        const int slot = pos & 127;
        if (e.kind == 4)
          dst = a.k_idx + ((size_t)page * 128 + slot) * 64;
        else
          dst = (e.kind == 1 ? a.K : a.V) + (((size_t)page * a.G + e.vec) * 128 + slot) * 128;
      }
      reinterpret_cast<uint4*>(dst)[e.a] = e.x;
      reinterpret_cast<uint4*>(dst)[e.b] = e.y;
    }
  }
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
  a.n_q = r.Q ? 8 * p.Hq : 0;
  a.n_k = 8 * p.G;
  a.n_qi = r.q_idx ? 4 * p.G : 0;
  a.items = a.n_q + 2 * a.n_k + a.n_qi + (r.k_idx ? 4 : 0);
  a.inv_items = 1.f / (float)a.items;
  // Rows for two rounds of a block's loads, so that its look-ups are shared, as long as every SM gets three blocks. 38,610
  // rows of 4 + 2 x 4 heads take 97 us with one row a block and 57 with four; 6,710 rows of 64 + 2 x 8, whose blocks are long
  // enough with one, 64 and 68; 2,400 rows of 8 + 2 x 2 heads 12 and 8.
  a.rows = std::min(kMaxRows, std::max(1, 2 * kInFlight * kThreads / a.items));
  while (a.rows > 1 && p.N < 3 * kCutSms * a.rows) --a.rows;
  // Few rows: a block of its own checks them and writes the error word, so that nothing has to clear it first (256 rows in
  // a graph: 3.0 us against 6.2 with a memset). For many rows it would be the last to end: 1024 sequences' rows 9.1 us
  // against 9.7, 2000 sequences' 16.8 against 12.3.
  a.report = p.N <= 1024;
  if (!a.report) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
    if (e != cudaSuccess) return e;
  }
  paged_append_kernel<<<(p.N + a.rows - 1) / a.rows + a.report, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace msa
