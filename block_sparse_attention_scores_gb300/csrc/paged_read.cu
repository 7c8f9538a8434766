// Tokens of the cache in 8 bits back as bf16 rows: value = code * 2^e, exact in
// bf16, so that a page which is read and quantised again holds the same values.
//
// 129 bytes of a vector are read and 256 written, and nothing else moves. A block
// takes 32 rows of the result: their sequences and pages are looked up by one
// warp, a lane each, then the block goes over the (tensor, group)s, eight threads
// a vector, 16 codes each, so that a warp reads four tokens' neighbouring 128
// bytes and writes 256 each. Four vectors a thread are in flight.
//
// Measured: 129,974 tokens of 8 groups with their index keys (661 MB) 106 us, 6.2
// TB/s, 0.92 of a plain copy; 701 tokens 3.3 us in a graph, launch and look-ups.
#include "paged_fp8.cuh"
#include "paged_rows.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;     // of the result, a block
constexpr int kInFlight = 4;  // loads of a thread

struct ReadArgs {
  const uint8_t *K, *V, *k_idx, *K_exp, *V_exp, *k_idx_exp;
  const int32_t *page_table, *seq_len, *first, *out_start;
  __nv_bfloat16 *K_out, *V_out, *k_idx_out;
  int S, M, G, num_pages, max_blocks, parts, per_part;
  int report;  // the last block checks every row and writes the error word; the others write none
  int* err;
};

// Place in the pools (page * 128 + slot) of row r of the result, which is one of sequence s or a later one; -1 before the
// first sequence and behind the last one, or where there is no such token (what is wrong: bad).
__device__ __forceinline__ int place_of(const ReadArgs& a, int s, int r, int& bad) {
  const auto start = [&](int i) { return __ldg(a.out_start + i); };
  bad = 0;
  if (r >= a.M || s >= a.S) return -1;
  if (start(s + 1) <= r) s = bisect_rows(start, a.S, r);
  if (s >= a.S || r < start(s)) return -1;  // (the searches take the first start for 0)
  const long long token = (a.first ? (long long)__ldg(a.first + s) : 0LL) + r - start(s);
  if (token < 0 || token >= __ldg(a.seq_len + s) || token >= a.max_blocks * 128) {
    bad = 1221;
    return -1;
  }
  const int page = __ldg(a.page_table + (size_t)s * a.max_blocks + token / 128);
  if (page >= 0 && page < a.num_pages) return page * 128 + (int)(token % 128);
  bad = 1222;
  return -1;
}

// 16 codes at `src` as bf16 at `dst` (32 bytes).
__device__ __forceinline__ void write_values(__nv_bfloat16* dst, uint4 codes, uint32_t byte) {
  const float pow2 = exp_value(byte);
  const uint4 lo = eight_bf16(make_uint2(codes.x, codes.y), pow2), hi = eight_bf16(make_uint2(codes.z, codes.w), pow2);
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w),
               "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

__global__ void __launch_bounds__(kThreads) paged_read_kernel(ReadArgs a) {
  __shared__ int at_of[kRows];  // token's place in the pools, -1: none
  const int tid = threadIdx.x, lane = tid & 31;
  if (a.report && blockIdx.x == gridDim.x - 1) {
    int worst = 0;
    for (int r0 = tid & ~31; r0 < a.M; r0 += kThreads) {
      int bad;
      place_of(a, find_sequence(a.out_start, a.S, r0, lane), r0 + lane, bad);
      if (!worst) worst = bad;
    }
    const int first = __syncthreads_or(worst == 1221), second = __syncthreads_or(worst != 0);
    if (tid == 0) *a.err = second ? kDevBadIndex * 65536 + (first ? 1221 : 1222) : kDevOk;
    return;
  }
  const int r0 = blockIdx.x / a.parts * kRows, part = blockIdx.x % a.parts;
  if (tid < 32) {  // (most rows are of the first one's sequence)
    int bad;
    at_of[tid] = place_of(a, find_sequence(a.out_start, a.S, r0, tid), r0 + tid, bad);
    if (bad && !a.report) dev_fail(a.err, kDevBadIndex, bad);
  }
  __syncthreads();
  const int row = tid >> 3, piece = tid & 7;
  const int at = at_of[row];
  if (at < 0) return;
  const size_t slot = (size_t)(at >> 7) * a.G * 128 + (at & 127), out = (size_t)(r0 + row) * a.G;
  const int begin = part * a.per_part, end = min(2 * a.G, begin + a.per_part);  // K's groups, then V's
  for (int v0 = begin; v0 < end; v0 += kInFlight) {
    uint4 codes[kInFlight];
    uint32_t byte[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int v = min(v0 + i, end - 1), g = v < a.G ? v : v - a.G;
      const size_t from = slot + (size_t)g * 128;
      codes[i] = __ldcs(reinterpret_cast<const uint4*>((v < a.G ? a.K : a.V) + from * 128) + piece);
      byte[i] = __ldg((v < a.G ? a.K_exp : a.V_exp) + from);
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int v = v0 + i, g = v < a.G ? v : v - a.G;
      if (v < end) write_values((v < a.G ? a.K_out : a.V_out) + (out + g) * 128 + piece * 16, codes[i], byte[i]);
    }
  }
  if (a.k_idx_out && part == a.parts - 1 && piece < 4)
    write_values(a.k_idx_out + (size_t)(r0 + row) * 64 + piece * 16,
                 __ldcs(reinterpret_cast<const uint4*>(a.k_idx + (size_t)at * 64) + piece), __ldg(a.k_idx_exp + at));
}

}  // namespace

cudaError_t launch_paged_read(const PagedProb& p, const PagedCachePtrs& c, const ReadRows& r, uint8_t* ws, cudaStream_t st) {
  ReadArgs a;
  a.K = static_cast<const uint8_t*>(c.K);
  a.V = static_cast<const uint8_t*>(c.V);
  a.k_idx = static_cast<const uint8_t*>(c.k_idx);
  a.K_exp = c.K_exp;
  a.V_exp = c.V_exp;
  a.k_idx_exp = c.k_idx_exp;
  a.page_table = c.page_table;
  a.seq_len = c.seq_len;
  a.first = r.first;
  a.out_start = r.out_start;
  a.K_out = static_cast<__nv_bfloat16*>(r.K);
  a.V_out = static_cast<__nv_bfloat16*>(r.V);
  a.k_idx_out = static_cast<__nv_bfloat16*>(r.k_idx);
  a.S = p.S;
  a.M = r.M;
  a.G = p.G;
  a.num_pages = p.num_pages;
  a.max_blocks = p.max_blocks;
  a.err = reinterpret_cast<int*>(ws);
  // As the append does it: few rows are checked by a block of their own, which writes the error word, so that nothing has to
  // clear it first (701 tokens in a graph 6.2 us with a memset, 3.3 without).
  a.report = r.M <= 2048;
  if (!a.report) {
    const cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
    if (e != cudaSuccess) return e;
  }
  // Few rows: their vectors are spread over several blocks, three for each SM at most.
  const int tiles = (r.M + kRows - 1) / kRows;
  a.parts = std::min(2 * p.G, std::max(1, 3 * kCutSms / tiles));
  a.per_part = (2 * p.G + a.parts - 1) / a.parts;
  a.parts = (2 * p.G + a.per_part - 1) / a.per_part;
  paged_read_kernel<<<tiles * a.parts + a.report, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace msa
