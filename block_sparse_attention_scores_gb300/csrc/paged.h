// Host-side internals of the paged-cache entry points: the validated batch,
// the workspace layout, and the launchers.
#pragma once

#include "msa_internal.h"

namespace msa {

// SMs the work is cut for. A constant, so that a workspace's size does not
// depend on the machine that asks for it (any SM count runs the same cuts).
constexpr int kCutSms = 152;

// Words of a workspace's header behind the error word.
constexpr int kLeadCount = 16;  // rows in PagedWs::lead
constexpr int kWorkNext = 17;   // items that attention CTAs have taken beyond their first ones
constexpr int kRunCount = 18;   // entries of PagedWs::runs
constexpr int kRunNext = 19;    // runs that have been taken beyond the CTAs' first ones

struct PagedProb {
  int S, N, Hq, G, hg, k;
  int num_pages, max_blocks, prefix;
  float scale;
};

// Workspace regions (byte offsets, 256-aligned) and how the work is cut.
struct PagedWs {
  size_t rows = 0;      // int4 [N]  per new row: sequence (-1: none, -2: refused), position, rows of its sequence before
                        //           it, and from it on
  size_t lead = 0;      // int4 [N]  the rows that lead a tile of the mma.sync path: sequence, position, row, rows of the tile
  size_t runs = 0;      // int4 [N]  the rows that lead a pair of 128-row tiles: sequence, position, row, rows of the pair
  size_t flags = 0;     // int32 [n_flags] what the blocks of the index scores or of the shared prefix found wrong
  int n_flags = 0;      // those blocks
  size_t arrived = 0;   // int32 [N, G, 3] parts of a (row tile, group) that are done, as each joining warp counts them
  size_t pooled = 0;    // fp32 [N, G, max_blocks, 2] block maxima of the index scores, and the block's largest |key| value
                        //      (none where nothing is chosen: one block kept, or one column)
  size_t part_o = 0;    // fp32 [pslots + rslots or splits, N, Hq, d] partial outputs (normalised; none for a single split)
  size_t part_lse = 0;  // fp32 [pslots + rslots or splits, N, Hq]    their log2-sum-exp2
  size_t total = 256;
  int splits = 1;       // partials a row's own pages are cut into ...
  int per_split = 1;    // ... of this many pages
  int tile_rows = 1;    // new rows of one sequence that share the key tiles (mma.sync path)
  int prefix = 0;       // pages that are read once for the batch (0 where a small shared prefix is read as own pages)
  int pairs = 0;        // shared prefix: pairs of 128-row query tiles
  int teams = 0;        // shared prefix: runs of pages, each walked by `pairs` CTAs
  int pslots = 0;       // shared prefix: partials per row
  int run_rows = 0;     // new rows of one sequence in a pair of 128-row tiles of the tcgen05 path, which takes a sequence's
                        // own pages where this is not 0
  int per_run = 1;      // pages of such a pair's runs ...
  int rslots = 0;       // ... and how many runs at most: partials per row
};

PagedWs paged_ws_layout(const PagedProb& p, int which);

// Units (group, page) of the shared prefix, cut into `teams` runs of nearly
// equal length: run j holds [j U / teams, (j + 1) U / teams).
__host__ __device__ inline int team_start(int j, int units, int teams) { return (int)((long long)j * units / teams); }
__host__ __device__ inline int team_of(int u, int units, int teams) {
  return (int)((((long long)u + 1) * teams - 1) / units);
}

struct PagedCachePtrs {
  void *K, *V, *k_idx;
  const int32_t *page_table, *row_start, *seq_len;
};

// Tensor maps over the K and V pools as rows of 128 values: boxes of 64 columns x 128 rows (half a page of one group).
struct PoolMaps {
  CUtensorMap k, v;
};

struct RopeRows {
  const void *Q, *K, *V, *q_idx, *k_idx;
  long long ld_Q, ld_K, ld_V, ld_q_idx, ld_k_idx;  // elements between consecutive rows
  void *Q_out, *q_idx_out;
  const float *inv_freq, *inv_freq_idx;
  int rot, rot_idx, interleaved;
};

cudaError_t launch_paged_append(const PagedProb& p, const PagedCachePtrs& c, const RopeRows& r, uint8_t* ws,
                                cudaStream_t st);
// The call's first work (paged_rows.cuh) as a kernel of its own (the index scores' kernel does it itself).
cudaError_t launch_paged_rows(const PagedProb& p, const PagedCachePtrs& c, uint8_t* ws, const PagedWs& L,
                              cudaStream_t st);
cudaError_t launch_paged_index(const PagedProb& p, const PagedCachePtrs& c, const void* q_idx, int32_t* block_idx,
                               uint8_t* ws, const PagedWs& L, cudaStream_t st);
// Attention of every new row over its selected pages (block_idx) or, with
// block_idx null, over its sequence's pages behind the shared prefix.
cudaError_t launch_paged_attn(const PagedProb& p, const PagedCachePtrs& c, const PoolMaps& maps, const void* Q,
                              const int32_t* block_idx, void* O, float* LSE, uint8_t* ws, const PagedWs& L, cudaStream_t st);
// Shared prefix, and runs of the sequences' own pages. The attention kernel may start while it still runs.
cudaError_t launch_paged_prefix(const PagedProb& p, const PagedCachePtrs& c, const PoolMaps& maps, const void* Q,
                                uint8_t* ws, const PagedWs& L, cudaStream_t st);
// Joins the parts of the shared prefix and of the own pages (without a prefix the attention does).
cudaError_t launch_paged_merge(const PagedProb& p, void* O, float* LSE, uint8_t* ws, const PagedWs& L,
                               cudaStream_t st);


}  // namespace msa
