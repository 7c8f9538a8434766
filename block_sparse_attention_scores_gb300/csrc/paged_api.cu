// C ABI of the paged cache: argument checks, workspace layout and launch
// order. See include/msa.h for the contract of each call.
#include <math.h>

#include "paged.h"

namespace msa {

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Cuts `pages` pages of each of `tiles` row tiles into runs of equal length. An
// item costs `extra` pages more than its pages (its row, pages and queries to
// look up, the warps' meeting, its part of O), and parts that the kernel joins
// itself `join` more; SMs take items as they come, so the end is half an item
// long. Measured for what the mma.sync path joins (6 and 8): 64 rows of 16 pages
// and 8 groups 125 us, 127 where an item counts for one page more and the join for
// nothing (which cuts in two), 57 rows of 9 pages and 2 groups 15.3 and 22.9; a
// row's 128 pages 23.7 us, 28.6 uncut; 16000 tokens of 8 groups 22.7 us, 84.7 uncut.
// Where the merge kernel joins (1 and 0): 64 sequences behind 32K tokens 94 us, 97
// with two pages. 128-row tiles (3 and 0): 300 rows x 32 heads over 4 groups and
// 8000 tokens 64 us, 84 with one and 93 with eight pages.
static void cut_pages(long long tiles, int pages, double extra, double join, int* per_split, int* n_splits) {
  tiles = std::max(1LL, tiles);
  pages = std::max(1, pages);
  double best = 0;
  for (int i = -2; i <= 8; ++i) {
    // two and three runs, and what gives every SM one, two, ... items
    const long long want = i < 0 ? 1 - i : i == 0 ? 1 : std::max(1LL, i * (long long)kCutSms / tiles);
    const int per = (int)((pages + std::min<long long>(want, pages) - 1) / std::min<long long>(want, pages));
    const int splits = (pages + per - 1) / per;
    const double cost = (std::max(1.0, (double)tiles * splits / kCutSms) + 0.5) * (per + extra) + (splits > 1 ? join : 0);
    if (best == 0 || cost < best) {
      best = cost;
      *per_split = per;
      *n_splits = splits;
    }
  }
}

PagedWs paged_ws_layout(const PagedProb& p, int which) {
  PagedWs L;
  size_t off = 256;  // header: error word
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align256(off + bytes);
    return o;
  };
  if (which == MSA_WS_PAGED_APPEND) {
    L.total = off;
    return L;
  }
  L.rows = take((size_t)p.N * 16);
  L.lead = take((size_t)p.N * 16);
  L.arrived = take((size_t)p.N * p.G * 12);
  if (which == MSA_WS_PAGED_SPARSE) {
    if (p.k > 1 && p.max_blocks > 1) L.pooled = take((size_t)p.N * p.G * p.max_blocks * 8);
    if (p.k > 1) L.n_flags = (int)std::min<long long>((long long)p.S * ((p.max_blocks + 4) / 6), kCutSms - 1);
    L.flags = take(kCutSms * 4);
    cut_pages((long long)p.N * p.G, std::min(p.k, p.max_blocks), 6, 8, &L.per_split, &L.splits);
  } else {
    L.tile_rows = 8 / p.hg;
    // More than nine columns (rows x heads) a sequence on average and more than a page each: 128-row tiles, tcgen05. Padded
    // rows count, as nothing here tells them from others: the ninth column is for a pad of up to an eighth. Against eight
    // columns at a time: 32 sequences of 2 rows x 64 heads over 2000 tokens 63 -> 60 us, of 8 rows 135 -> 69, 300 rows x 32
    // heads over 4 groups and 8000 tokens 274 -> 64; the other way for one page (8 rows x 64 heads over 100 tokens 17 -> 10).
    const bool runs = (long long)p.N * p.hg > 9LL * p.S && p.max_blocks - p.prefix > 1;
    // A shared prefix of ten pages an SM (13 where a sequence has several tiles of eight columns), counted for every such
    // tile, is read as own pages: it stays in L2, and two kernels do with it what four do. 4 sequences of 32 heads over 8
    // groups behind 16 pages 15 us against 19, 16 behind 8 pages 14 and 19, 8 of 4 rows behind 12 pages (1536) 17 and 21,
    // one of 16 rows x 64 heads over 8 groups behind 10 pages (1280) 15 and 21, of 64 x 32 heads behind 6 (1536) 19 and
    // 23; beyond: 16 rows x 64 heads behind 50 pages (6400) 50 and 29, 64 behind 10 (5120) 40 and 30, 128 behind 10
    // (10240) 66 and 41, behind 180 (1,440 pages, read 128 times) 797 and 99.
    const long long tiles = std::max(p.N / L.tile_rows, std::min(p.S, p.N));
    // (Idle sequences count too: their tables are looked at by the one block that lines up the rows.)
    const long long readers = std::max<long long>(tiles, p.S);
    const bool fold = !runs && readers * p.prefix * p.G <= (readers > p.S ? 2000 : 1500);
    L.prefix = fold ? 0 : p.prefix;
    if (runs) {
      L.run_rows = 256 / p.hg;
      L.runs = take((size_t)p.N * 16);
      cut_pages((long long)std::max(p.N / L.run_rows, std::min(p.S, p.N)) * p.G, p.max_blocks - p.prefix, 3, 0, &L.per_run,
                &L.rslots);
      L.splits = 0;
      L.n_flags = kCutSms;
    } else {
      cut_pages(tiles * p.G, p.max_blocks - L.prefix, L.prefix ? 1 : 6, L.prefix ? 0 : 8, &L.per_split, &L.splits);
    }
    if (L.prefix > 0) {
      L.pairs = (int)(((long long)p.N * p.hg + 255) / 256);
      const int units = p.G * p.prefix;
      // The own pages' kernel runs beside: its CTAs start on the SMs left over, the others as the prefix's end, so that the
      // memory is busy while the tensor core is. Both are estimated (a page takes a pair of tiles 2,750 cycles, a row tile
      // 2,000; own pages: half of what the table holds), and the prefix has half of the SMs at least, lest a poor estimate
      // make it the longer one. 64 sequences behind 32K tokens with up to 2K of their own: 112 us one after the other,
      // 100 with two thirds, 94 with half, 102 with 0.35 of the SMs; 100 sequences with 2000 each: 67, 49, 48, 48.
      const double own = (double)tiles * p.G * (p.max_blocks - p.prefix + 1) / 2 * 2000;
      const double shared = (double)units * L.pairs * 2750;
      const int sms = L.run_rows ? kCutSms : (int)(kCutSms * std::max(0.5, shared / (shared + own)));
      L.teams = std::min(units, std::max(1, sms / L.pairs));
      L.n_flags = std::max(L.n_flags, L.teams * L.pairs);
      for (int g = 0; g < p.G; ++g)
        L.pslots = std::max(L.pslots, team_of((g + 1) * p.prefix - 1, units, L.teams) -
                                          team_of(g * p.prefix, units, L.teams) + 1);
    }
    L.flags = take((size_t)L.n_flags * 4);
  }
  // (a row's only part, which no other joins, is its result)
  const int slots = L.pslots + L.rslots + (L.pslots || L.splits > 1 ? L.splits : 0);
  const size_t rows = (size_t)slots * p.N * p.Hq;
  L.part_o = take(rows * 128 * 4);
  L.part_lse = take(rows * 4);
  L.total = off;
  return L;
}

static msa_status validate_paged(const msa_paged_shape* s, PagedProb* p) {
  if (!s) return fail(MSA_ERR_INVALID_ARG, "shape is NULL");
  if (s->S < 1 || s->N < 1 || s->Hq < 1 || s->G < 1 || s->d < 1 || s->d_idx < 1 || s->Bk < 1 || s->k < 1 ||
      s->num_pages < 1 || s->max_blocks < 1 || s->prefix_blocks < 0)
    return fail(MSA_ERR_INVALID_ARG,
                "shape fields must be positive (S=%d N=%d Hq=%d G=%d d=%d d_idx=%d Bk=%d k=%d num_pages=%d max_blocks=%d "
                "prefix_blocks=%d)",
                s->S, s->N, s->Hq, s->G, s->d, s->d_idx, s->Bk, s->k, s->num_pages, s->max_blocks, s->prefix_blocks);
  if (s->Hq % s->G) return fail(MSA_ERR_INVALID_ARG, "Hq=%d is not a multiple of G=%d", s->Hq, s->G);
  if (s->prefix_blocks >= s->max_blocks)
    return fail(MSA_ERR_INVALID_ARG, "prefix_blocks=%d leaves no block of max_blocks=%d for the new rows",
                s->prefix_blocks, s->max_blocks);
  const int hg = s->Hq / s->G;
  if (s->d != 128) return fail(MSA_ERR_UNSUPPORTED, "d=%d: only head dim 128 is supported", s->d);
  if (s->d_idx != 64) return fail(MSA_ERR_UNSUPPORTED, "d_idx=%d: only index dim 64 is supported", s->d_idx);
  if (s->Bk != 128) return fail(MSA_ERR_UNSUPPORTED, "Bk=%d: only 128-token pages are supported", s->Bk);
  if (!(hg == 1 || hg == 2 || hg == 4 || hg == 8))
    return fail(MSA_ERR_UNSUPPORTED, "Hq/G=%d: heads per group must be 1, 2, 4 or 8", hg);
  if (s->k > 128) return fail(MSA_ERR_UNSUPPORTED, "k=%d exceeds 128", s->k);
  if (s->S > 65535) return fail(MSA_ERR_UNSUPPORTED, "S=%d exceeds 65535 sequences", s->S);
  if (s->max_blocks > 8192) return fail(MSA_ERR_UNSUPPORTED, "max_blocks=%d exceeds 8192 (2^20 tokens)", s->max_blocks);
  if (s->N > (1 << 20)) return fail(MSA_ERR_UNSUPPORTED, "N=%d exceeds 2^20 rows", s->N);
  // (items of a row's vectors are counted in fp32 and 32 bits, pages times groups in 32)
  if (s->Hq > 65536) return fail(MSA_ERR_UNSUPPORTED, "Hq=%d exceeds 65536 heads", s->Hq);
  if ((long long)s->N * s->Hq > (1LL << 28)) return fail(MSA_ERR_UNSUPPORTED, "N*Hq too large");
  if ((long long)s->num_pages * s->G > (1LL << 24) - 1)
    return fail(MSA_ERR_UNSUPPORTED, "num_pages*G=%lld: at most 2^24 - 1 page tiles are addressed",
                (long long)s->num_pages * s->G);
  const float sc = s->scale > 0 ? s->scale : 1.0f / sqrtf((float)s->d);
  if (!(sc > 0) || !isfinite(sc)) return fail(MSA_ERR_INVALID_ARG, "scale must be finite");
  p->S = s->S;
  p->N = s->N;
  p->Hq = s->Hq;
  p->G = s->G;
  p->hg = hg;
  p->k = s->k;
  p->num_pages = s->num_pages;
  p->max_blocks = s->max_blocks;
  p->prefix = s->prefix_blocks;
  p->scale = sc;
  return MSA_OK;
}

static msa_status check_cache(const msa_paged_cache* c, bool index, PagedCachePtrs* out) {
  msa_status s;
  if (!c) return fail(MSA_ERR_INVALID_ARG, "cache is NULL");
  if ((s = check_ptr(c->K, "cache.K", 16)) != MSA_OK) return s;
  if ((s = check_ptr(c->V, "cache.V", 16)) != MSA_OK) return s;
  if (index && (s = check_ptr(c->k_idx, "cache.k_idx", 16)) != MSA_OK) return s;
  if ((s = check_ptr(c->page_table, "cache.page_table", 4)) != MSA_OK) return s;
  if ((s = check_ptr(c->row_start, "cache.row_start", 4)) != MSA_OK) return s;
  if ((s = check_ptr(c->seq_len, "cache.seq_len", 4)) != MSA_OK) return s;
  *out = {c->K, c->V, c->k_idx, c->page_table, c->row_start, c->seq_len};
  return MSA_OK;
}

static msa_status encode_pools(const PagedProb& p, const PagedCachePtrs& c, PoolMaps* m) {
  const uint64_t dims[2] = {128, (uint64_t)p.num_pages * p.G * 128};
  const uint64_t strides[1] = {256};
  const uint32_t box[2] = {64, 128};
  if (encode_tmap(&m->k, c.K, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
      encode_tmap(&m->v, c.V, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return MSA_OK;
  return fail(MSA_ERR_CUDA, "tensor maps of the pools could not be encoded");
}

static msa_status check_paged_ws(const PagedProb& p, int which, void* ws, size_t bytes, PagedWs* L) {
  *L = paged_ws_layout(p, which);
  if (!ws) return fail(MSA_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(MSA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (bytes < L->total) return fail(MSA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", bytes, L->total);
  return MSA_OK;
}

// One new-row input: present with its output, 16-byte rows.
static msa_status check_rows(const void* ptr, const char* name, int64_t* ld, int64_t packed) {
  msa_status s;
  if ((s = check_ptr(ptr, name, 16)) != MSA_OK) return s;
  if (*ld == 0) *ld = packed;
  if (*ld < packed || *ld % 8)
    return fail(MSA_ERR_INVALID_ARG, "row stride of %s is %lld: at least %lld and a multiple of 8 are needed", name,
                (long long)*ld, (long long)packed);
  return MSA_OK;
}

static msa_status check_rot(int rot, int dim, const float* freq, const char* name) {
  if (rot < 0 || rot > dim || rot % 16)
    return fail(MSA_ERR_INVALID_ARG, "%s=%d: a multiple of 16 in [0, %d] is needed", name, rot, dim);
  if (rot > 0) return check_ptr(freq, rot && dim == 64 ? "inv_freq_idx" : "inv_freq", 4);
  return MSA_OK;
}

}  // namespace msa

using namespace msa;

extern "C" {

size_t msa_paged_workspace_size(const msa_paged_shape* shape, int which) {
  PagedProb p{};
  if (which < MSA_WS_PAGED_APPEND || which > MSA_WS_PAGED_DENSE) return 0;
  if (validate_paged(shape, &p) != MSA_OK) return 0;
  if (which != MSA_WS_PAGED_DENSE) p.prefix = 0;
  return paged_ws_layout(p, which).total;
}

msa_status msa_paged_append(const msa_paged_shape* shape, const msa_paged_cache* cache, const msa_rope* rope,
                            const msa_new_rows* rows, void* Q_out, void* q_idx_out, void* workspace,
                            size_t workspace_bytes, msa_stream_t stream) {
  PagedProb p{};
  PagedCachePtrs c;
  PagedWs L;
  msa_status s;
  if ((s = validate_paged(shape, &p)) != MSA_OK) return s;
  p.prefix = 0;
  if (!rows) return fail(MSA_ERR_INVALID_ARG, "rows is NULL");
  if (!rope) return fail(MSA_ERR_INVALID_ARG, "rope is NULL");
  if ((s = check_cache(cache, rows->k_idx != nullptr, &c)) != MSA_OK) return s;
  msa_new_rows n = *rows;
  if ((s = check_rows(n.K, "K", &n.ld_K, (int64_t)p.G * 128)) != MSA_OK) return s;
  if ((s = check_rows(n.V, "V", &n.ld_V, (int64_t)p.G * 128)) != MSA_OK) return s;
  if ((n.Q == nullptr) != (Q_out == nullptr) || (n.q_idx == nullptr) != (q_idx_out == nullptr))
    return fail(MSA_ERR_INVALID_ARG, "give Q with Q_out and q_idx with q_idx_out, or neither of a pair");
  if (n.Q) {
    if ((s = check_rows(n.Q, "Q", &n.ld_Q, (int64_t)p.Hq * 128)) != MSA_OK) return s;
    if ((s = check_ptr(Q_out, "Q_out", 16)) != MSA_OK) return s;
  }
  if (n.q_idx) {
    if ((s = check_rows(n.q_idx, "q_idx", &n.ld_q_idx, (int64_t)p.G * 64)) != MSA_OK) return s;
    if ((s = check_ptr(q_idx_out, "q_idx_out", 16)) != MSA_OK) return s;
  }
  if (n.k_idx && (s = check_rows(n.k_idx, "k_idx", &n.ld_k_idx, 64)) != MSA_OK) return s;
  if ((s = check_rot(rope->rot_dim, 128, rope->inv_freq, "rot_dim")) != MSA_OK) return s;
  const bool index = n.q_idx || n.k_idx;
  if (index && (s = check_rot(rope->rot_dim_idx, 64, rope->inv_freq_idx, "rot_dim_idx")) != MSA_OK) return s;
  if ((s = check_paged_ws(p, MSA_WS_PAGED_APPEND, workspace, workspace_bytes, &L)) != MSA_OK) return s;
  if ((s = check_device()) != MSA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  RopeRows r;
  r.Q = n.Q;
  r.K = n.K;
  r.V = n.V;
  r.q_idx = n.q_idx;
  r.k_idx = n.k_idx;
  r.ld_Q = n.ld_Q;
  r.ld_K = n.ld_K;
  r.ld_V = n.ld_V;
  r.ld_q_idx = n.ld_q_idx;
  r.ld_k_idx = n.ld_k_idx;
  r.Q_out = Q_out;
  r.q_idx_out = q_idx_out;
  r.inv_freq = rope->inv_freq;
  r.inv_freq_idx = rope->inv_freq_idx;
  r.rot = rope->rot_dim;
  r.rot_idx = index ? rope->rot_dim_idx : 0;
  r.interleaved = rope->interleaved != 0;
  return cuda_status(launch_paged_append(p, c, r, static_cast<uint8_t*>(workspace), st), "paged append launch");
}

msa_status msa_paged_sparse_attn(const msa_paged_shape* shape, const msa_paged_cache* cache, const void* Q,
                                 const void* q_idx, int32_t* block_idx, void* O, float* LSE, void* workspace,
                                 size_t workspace_bytes, msa_stream_t stream) {
  PagedProb p{};
  PagedCachePtrs c;
  PagedWs L;
  msa_status s;
  if ((s = validate_paged(shape, &p)) != MSA_OK) return s;
  p.prefix = 0;
  if ((s = check_cache(cache, q_idx != nullptr, &c)) != MSA_OK) return s;
  if ((s = check_ptr(Q, "Q", 16)) != MSA_OK) return s;
  if (q_idx && (s = check_ptr(q_idx, "q_idx", 16)) != MSA_OK) return s;
  if ((s = check_ptr(block_idx, "block_idx", 4)) != MSA_OK) return s;
  if ((s = check_ptr(O, "O", 16)) != MSA_OK) return s;
  if ((s = check_ptr(LSE, "LSE", 4)) != MSA_OK) return s;
  if ((s = check_paged_ws(p, MSA_WS_PAGED_SPARSE, workspace, workspace_bytes, &L)) != MSA_OK) return s;
  if ((s = check_device()) != MSA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  PoolMaps maps;
  if ((s = encode_pools(p, c, &maps)) != MSA_OK) return s;
  if (!q_idx) L.n_flags = 0;
  if ((s = cuda_status(q_idx ? launch_paged_index(p, c, q_idx, block_idx, w, L, st) : launch_paged_rows(p, c, w, L, st),
                       "paged index launch")) != MSA_OK)
    return s;
  return cuda_status(launch_paged_attn(p, c, maps, Q, block_idx, O, LSE, w, L, st), "paged attention launch");
}

msa_status msa_paged_dense_attn(const msa_paged_shape* shape, const msa_paged_cache* cache, const void* Q, void* O,
                                float* LSE, void* workspace, size_t workspace_bytes, msa_stream_t stream) {
  PagedProb p{};
  PagedCachePtrs c;
  PagedWs L;
  msa_status s;
  if ((s = validate_paged(shape, &p)) != MSA_OK) return s;
  if ((s = check_cache(cache, false, &c)) != MSA_OK) return s;
  if ((s = check_ptr(Q, "Q", 16)) != MSA_OK) return s;
  if ((s = check_ptr(O, "O", 16)) != MSA_OK) return s;
  if ((s = check_ptr(LSE, "LSE", 4)) != MSA_OK) return s;
  if ((s = check_paged_ws(p, MSA_WS_PAGED_DENSE, workspace, workspace_bytes, &L)) != MSA_OK) return s;
  if ((s = check_device()) != MSA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  PoolMaps maps;
  if ((s = encode_pools(p, c, &maps)) != MSA_OK) return s;
  const bool parts = L.prefix || L.run_rows;
  if ((s = cuda_status(launch_paged_rows(p, c, w, L, st), "paged rows launch")) != MSA_OK) return s;
  if (parts && (s = cuda_status(launch_paged_prefix(p, c, maps, Q, w, L, st), "paged prefix launch")) != MSA_OK) return s;
  if (!L.run_rows &&
      (s = cuda_status(launch_paged_attn(p, c, maps, Q, nullptr, O, LSE, w, L, st), "paged attention launch")) != MSA_OK)
    return s;
  return parts ? cuda_status(launch_paged_merge(p, O, LSE, w, L, st), "paged merge launch") : MSA_OK;
}

}  // extern "C"
