// Tokens of the cache in 8 bits back as bf16 rows: value = code * 2^e, exact in
// bf16, so that a page which is read and quantised again holds the same values.
//
// 129 bytes of a vector are read and 256 written, and nothing else moves. A block
// takes 32 rows of the result: their sequences and pages are looked up by one
// warp, a lane each, then the block goes over the (tensor, group)s, eight threads
// a vector, 16 codes each, so that a warp reads four tokens' neighbouring 128
// bytes and writes 256 each. Four vectors a thread are in flight.
//
// Measured: see the launcher.
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
  int* err;
};

// 16 codes at `src` as bf16 at `dst` (32 bytes).
__device__ __forceinline__ void write_values(__nv_bfloat16* dst, uint4 codes, uint32_t byte) {
  const float pow2 = exp_value(byte);
  const uint4 lo = eight_bf16(make_uint2(codes.x, codes.y), pow2), hi = eight_bf16(make_uint2(codes.z, codes.w), pow2);
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w),
               "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w)
               : "memory");
}

__global__ void __launch_bounds__(kThreads) paged_read_kernel(ReadArgs a) {
  __shared__ int at_of[kRows];  // token's place in the pools (page * 128 + slot), -1: none
  const int r0 = blockIdx.x / a.parts * kRows, part = blockIdx.x % a.parts, tid = threadIdx.x;
  if (tid < 32) {
    const int r = r0 + tid;
    const auto start = [&](int i) { return __ldg(a.out_start + i); };
    int s = find_sequence(a.out_start, a.S, r0, tid);  // of the first row; most others are of the same one
    int at = -1;
    if (r < a.M && s < a.S) {
      if (start(s + 1) <= r) s = bisect_rows(start, a.S, r);
      if (s < a.S) {  // not behind the last sequence
        const long long token = (a.first ? (long long)__ldg(a.first + s) : 0) + (r - start(s));
        if (token < 0 || token >= __ldg(a.seq_len + s) || token >= a.max_blocks * 128) {
          dev_fail(a.err, kDevBadIndex, 1221);
        } else {
          const int page = __ldg(a.page_table + (size_t)s * a.max_blocks + token / 128);
          if (page < 0 || page >= a.num_pages) dev_fail(a.err, kDevBadIndex, 1222);
          else at = page * 128 + (int)(token % 128);
        }
      }
    }
    at_of[tid] = at;
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
  const cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
  if (e != cudaSuccess) return e;
  // Few rows: their vectors are spread over several blocks, three for each SM at most.
  const int tiles = (r.M + kRows - 1) / kRows;
  a.parts = std::min(2 * p.G, std::max(1, 3 * kCutSms / tiles));
  a.per_part = (2 * p.G + a.parts - 1) / a.parts;
  a.parts = (2 * p.G + a.per_part - 1) / a.per_part;
  paged_read_kernel<<<tiles * a.parts, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace msa
