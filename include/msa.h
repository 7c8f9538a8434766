/*
 * msa.h -- C ABI of the GB300 (sm_103a) MiniMax Sparse Attention (MSA)
 * training hot path on one GQA layer.
 *
 * The method (itinai.ru "How to solve the memory problem with MiniMax Sparse
 * Attention", sections "Two-stage process", "How the indexer works" and
 * "Training sparse attention"; dothoosh.com "how Flash-MSA cuts
 * million-token training cost", sections "Block-sparsity mechanism",
 * "Kernel design and execution" and "Fixing the KL-divergence bottleneck"):
 *
 *   1. msa_index_topk  -- index branch: every causally visible token is scored
 *      with the group's index query against the shared index key, scores are
 *      max-pooled over Bk-token KV blocks, and each (group, query) keeps k
 *      blocks: its own block plus the best k-1 earlier ones.
 *   2. msa_sparse_fwd  -- main branch: exact causal softmax attention over the
 *      selected blocks only; writes O and the log-sum-exp kept for the backward.
 *   3. msa_bwd         -- fused backward: dQ, dK, dV of the main branch and the
 *      KL-alignment gradient of the index branch, whose score gradient is
 *      p_px - p_main (index softmax over the selected tokens minus the
 *      head-averaged, detached main softmax), giving dq_idx and dk_idx.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers owned by the caller; the library
 *   never allocates device memory. Scratch comes from the caller's workspace,
 *   sized by msa_workspace_size() (256-byte aligned base required).
 * - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *   stream). Host-side argument checks run before anything is enqueued; on a
 *   non-OK status nothing was launched and msa_last_error() describes why.
 * - bf16 tensors are passed as `void*` holding IEEE bfloat16 values; the
 *   backward's gradients are fp32 (`float*`), accumulated and written in fp32.
 * - Layouts (row-major, innermost last):
 *     Q, O, dO            [B, T, Hq, d]      bf16      dQ      fp32
 *     K, V                [B, T, G, d]       bf16      dK, dV  fp32 (one KV head per group)
 *     q_idx               [B, T, G, d_idx]   bf16      dq_idx  fp32
 *     k_idx               [B, T, d_idx]      bf16      dk_idx  fp32 (shared by all groups)
 *     block_idx           [B, G, T, k]       int32  (ascending ids, -1 padded)
 *     LSE                 [B, T, Hq]         fp32   (natural log, scaled scores)
 *     KL                  [B, G, T]          fp32   (one KL term per query)
 *   Head h belongs to group h / (Hq / G).
 * - Supported shapes (MSA_ERR_UNSUPPORTED otherwise): d = 128, d_idx = 64,
 *   Bk = 128, Hq / G in {1, 2, 4, 8} with Hq % G == 0, T % 128 == 0,
 *   1 <= T <= 2^20, 1 <= k <= 128, B >= 1, scale and scale_idx > 0 after
 *   defaulting; the index top-k (msa_index_topk, msa_index_topk_fp8,
 *   msa_index_topk_noalloc, and the MSA_WS_TOPK / MSA_WS_TOPK_FP8 workspace
 *   sizes) keeps at most k = 64 blocks per row. Kernels need an sm_100-family
 *   GPU (built for sm_103a).
 * - Device-side checks (bounded waits, block ids out of range) write an error
 *   word in the workspace; msa_check_device_status() reads it.
 */
#ifndef MSA_H
#define MSA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define MSA_API __attribute__((visibility("default")))
#else
#define MSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *msa_stream_t;

typedef enum msa_status {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, bad enum       */
  MSA_ERR_UNSUPPORTED = 2, /* shape outside the supported set above, or no GPU */
  MSA_ERR_WORKSPACE = 3,   /* workspace missing, misaligned or too small      */
  MSA_ERR_CUDA = 4,        /* a CUDA runtime call failed (see msa_last_error) */
  MSA_ERR_DEVICE = 5       /* a kernel reported a timeout or a bad block id   */
} msa_status;

typedef struct msa_shape {
  int32_t B;       /* batch                                                 */
  int32_t T;       /* sequence length                                       */
  int32_t Hq;      /* query heads                                           */
  int32_t G;       /* GQA groups = KV heads = index queries per position    */
  int32_t d;       /* head dim of Q/K/V                                     */
  int32_t d_idx;   /* index dim of q_idx/k_idx                              */
  int32_t Bk;      /* tokens per KV block                                   */
  int32_t k;       /* blocks kept per (group, query), own block included    */
  float scale;     /* main softmax scale; <= 0 selects 1/sqrt(d)            */
  float scale_idx; /* index score scale; <= 0 selects 1/sqrt(d_idx)         */
} msa_shape;

/* Which entry point a workspace is sized for. */
enum { MSA_WS_TOPK = 0, MSA_WS_FWD = 1, MSA_WS_BWD = 2, MSA_WS_TOPK_FP8 = 3, MSA_WS_DENSE = 4 };

/* Bytes of device workspace the entry point `which` needs for `shape`
 * (0 if the shape is invalid or unsupported). A workspace sized for
 * MSA_WS_BWD also serves MSA_WS_TOPK and MSA_WS_FWD; MSA_WS_TOPK_FP8 is
 * sized on its own (its E4M3 copies start right after the header). */
MSA_API size_t msa_workspace_size(const msa_shape *shape, int which);

/*
 * Index branch (itinai.ru "How the indexer works"; dothoosh.com Flash-MSA,
 * "Block-sparsity mechanism" and "Kernel design and execution": the proxy
 * pass accumulates no output, only scores and the running top-k).
 *
 * For every (b, g, t) with own block c_t = t / Bk:
 *   s[j]  = <q_idx[b,t,g,:], k_idx[b,j,:]>            for j <= t (fp32 sums of
 *           exact bf16 products; the positive scale_idx does not change order)
 *   pool[c] = max_{j in block c} s[j]                  for c < c_t
 *   block_idx[b,g,t,:] = {c_t} U top-(k-1) of pool under (score descending,
 *           block id ascending), written in ascending order, then -1 padding.
 * No T x T (or T x n_blocks) tensor is materialised.
 *
 * q_idx: [B,T,G,d_idx] bf16, k_idx: [B,T,d_idx] bf16 (both 16-byte aligned).
 * block_idx: [B,G,T,k] int32, fully written.
 */
MSA_API msa_status msa_index_topk(const msa_shape *shape, const void *q_idx, const void *k_idx, int32_t *block_idx,
                          void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* msa_index_topk with a low-precision indexer (dothoosh.com "how Flash-MSA
 * cuts million-token training cost", "Current limits and future scaling":
 * training the indexer in low precision, as at inference). The index scores
 * are computed from E4M3 copies of q_idx and k_idx made inside the call: one
 * scale per q_idx row (b, t, g) and one per 128-key block of k_idx (b, c);
 * each value is multiplied by 448 / amax in fp32 and rounded to the nearest
 * E4M3 value (ties to even, saturating at +-448); the scale is amax / 448
 * (1 when amax = 0). Pooling and selection are those of msa_index_topk on
 * the scores (q8 * sq) . (k8 * sk) * scale_idx, so block_idx can differ from
 * msa_index_topk's where quantization reorders blocks. `workspace` is sized
 * with MSA_WS_TOPK_FP8 (it holds the E4M3 copies: B*T*(G+1)*d_idx bytes plus
 * one float per key block); same arguments and errors as msa_index_topk. */
MSA_API msa_status msa_index_topk_fp8(const msa_shape *shape, const void *q_idx, const void *k_idx,
                                      int32_t *block_idx, void *workspace, size_t workspace_bytes,
                                      msa_stream_t stream);

/*
 * Main branch forward (itinai.ru "Two-stage process": exact softmax over the
 * selected tokens only; dothoosh.com Flash-MSA, "Kernel design and
 * execution": keep the LSE for the backward; dothoosh.com "how FlashAttention
 * cuts GPU memory traffic", "Online-softmax trick": the (m, l, a) merge).
 *
 * For head h in group g and query t, over S(g,t) = { j <= t : j / Bk listed in
 * block_idx[b,g,t,:] }:
 *   s_j = scale * <Q[b,t,h,:], K[b,j,g,:]>,  LSE = ln sum_j exp(s_j),
 *   O[b,t,h,:] = sum_j exp(s_j - LSE) V[b,j,g,:].
 * block_idx may come from msa_index_topk or from anywhere else, but every row
 * must hold distinct ids in [0, t / Bk] in ascending order followed by -1s
 * and must include t / Bk (violations set the device error word and the
 * offending row's outputs are unspecified).
 *
 * O: [B,T,Hq,d] bf16, LSE: [B,T,Hq] fp32, both fully written.
 */
MSA_API msa_status msa_sparse_fwd(const msa_shape *shape, const void *Q, const void *K, const void *V,
                          const int32_t *block_idx, void *O, float *LSE, void *workspace,
                          size_t workspace_bytes, msa_stream_t stream);

/*
 * Fused backward (dothoosh.com Flash-MSA, "Kernel design and execution": one
 * backward over proxy and main branch, scheduled through the inverted
 * block -> query map; "Fixing the KL-divergence bottleneck": d KL / d s_px =
 * p_px - p_main; itinai.ru "Training sparse attention": KL alignment to the
 * head-averaged main softmax, gradient detached from the backbone;
 * dothoosh.com FlashAttention page, "Training and the backward pass").
 *
 * Main branch, with P = exp(s - LSE) rebuilt from the saved LSE:
 *   D = rowsum(dO * O), dP = dO V^T, dS = P (dP - D),
 *   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO.
 * Index branch, per (b, g, t) over S(g,t):
 *   p_main_j = mean over the group's heads of P_h,j (detached),
 *   p_px_j   = softmax_j(scale_idx <q_idx[b,t,g,:], k_idx[b,j,:]>),
 *   KL[b,g,t] = sum_j p_main_j (ln p_main_j - ln p_px_j),
 *   gs_j = kl_weight (p_px_j - p_main_j),
 *   dq_idx[b,t,g,:] = scale_idx sum_j gs_j k_idx[b,j,:],
 *   dk_idx[b,j,:]  += scale_idx sum_{g,t} gs_j q_idx[b,t,g,:].
 * The loss is kl_weight * sum over rows of KL (pass 1/(B*G*T) for a mean).
 * No KL gradient reaches Q, K, V and no dO gradient reaches q_idx, k_idx.
 *
 * Inputs as in msa_sparse_fwd; O and LSE are the forward's outputs for the
 * same block_idx. Outputs dQ, dK, dV, dq_idx, dk_idx and KL (all fp32) are
 * fully written: every key block is selected at least by its own queries, so
 * every dK/dV/dk_idx row receives its sum (rows of a block whose queries all
 * had invalid block_idx rows are unspecified, as is everything else when the
 * device error word is set). Every sum runs in a fixed order (per-slot and
 * per-group partials, merged in order; no floating-point atomics), so the
 * outputs, like those of msa_index_topk and msa_sparse_fwd, are the same bits
 * in every run on the same inputs.
 */
MSA_API msa_status msa_bwd(const msa_shape *shape, const void *Q, const void *K, const void *V, const void *O,
                   const void *dO, const float *LSE, const void *q_idx, const void *k_idx,
                   const int32_t *block_idx, float kl_weight, float *dQ, float *dK, float *dV, float *dq_idx,
                   float *dk_idx, float *KL, void *workspace, size_t workspace_bytes, msa_stream_t stream);

/*
 * Index top-k for callers that cannot allocate device memory. The method's
 * description has no counterpart to this call; it computes exactly what
 * msa_index_topk does.
 *
 * Some callers cannot call cudaMalloc: a plugin inside a host application
 * that owns every byte of device memory and hands the plugin no allocator,
 * or code on a latency-critical path where cudaMalloc's implicit device-wide
 * synchronisation is not acceptable. This variant needs no workspace: its
 * scratch (the kernel's error word and work counter, 256 bytes) lives in a
 * static device array of MSA_NOALLOC_SCRATCH_BYTES bytes inside the library,
 * which every GPU that loads the library holds until the process exits.
 *
 * - Each GPU has its own copy of the array. The first call on a device looks
 *   up the address of that device's copy (once per device, with the device
 *   current) and the library keeps it; make that first call before any stream
 *   capture. The address belongs to the device's primary context: after
 *   cudaDeviceReset() on that device, reload the library before calling
 *   this function again.
 * - Every call clears the scratch it relies on (asynchronously, on `stream`)
 *   and then reuses it: calls that overlap on the same GPU (for example on
 *   two streams of one device) race on it. Serialise them; calls on
 *   different GPUs use different copies and do not race.
 * - A shape whose scratch would exceed MSA_NOALLOC_SCRATCH_BYTES is rejected
 *   with MSA_ERR_UNSUPPORTED.
 * - check != 0 synchronises `stream` and returns MSA_ERR_DEVICE if the kernel
 *   reported a timeout; check == 0 returns without waiting (device-side
 *   errors then go unreported).
 * No cudaMalloc, cudaFree or allocating library routine is called.
 */
#define MSA_NOALLOC_SCRATCH_BYTES 4096
MSA_API msa_status msa_index_topk_noalloc(const msa_shape *shape, const void *q_idx, const void *k_idx,
                                          int32_t *block_idx, int32_t check, msa_stream_t stream);

/* IndexShare: one selection shared by several layers (dothoosh.com "how
 * Flash-MSA cuts million-token training cost", "Current limits and future
 * scaling": sharing the proxy (index) heads across layers, so later layers
 * reuse an earlier layer's block indices). msa_block_map
 * builds the inverted block -> query map of `block_idx` once, into a
 * MSA_WS_BWD-sized `workspace`, with the work items of both the forward and
 * the backward; msa_sparse_fwd_mapped and msa_bwd_mapped then run on that map
 * instead of building their own (same arguments, results and errors as
 * msa_sparse_fwd and msa_bwd). The map stays valid for as long as `block_idx`
 * and the workspace's map region are unchanged: msa_index_topk,
 * msa_sparse_fwd and msa_bwd on the same workspace overwrite it, the mapped
 * calls do not. The caller guarantees that the `block_idx` passed to the
 * mapped calls is the one the map was built from; rows that fail validation
 * are reported by msa_block_map (device error word). */
MSA_API msa_status msa_block_map(const msa_shape *shape, const int32_t *block_idx, void *workspace,
                                 size_t workspace_bytes, msa_stream_t stream);
MSA_API msa_status msa_sparse_fwd_mapped(const msa_shape *shape, const void *Q, const void *K, const void *V,
                                         const int32_t *block_idx, void *O, float *LSE, void *workspace,
                                         size_t workspace_bytes, msa_stream_t stream);
MSA_API msa_status msa_bwd_mapped(const msa_shape *shape, const void *Q, const void *K, const void *V,
                                  const void *O, const void *dO, const float *LSE, const void *q_idx,
                                  const void *k_idx, const int32_t *block_idx, float kl_weight, float *dQ, float *dK,
                                  float *dV, float *dq_idx, float *dk_idx, float *KL, void *workspace,
                                  size_t workspace_bytes, msa_stream_t stream);

/* Indexer warmup (itinai.ru "How to solve the memory problem with MiniMax
 * Sparse Attention", "Training sparse attention": the first iterations run
 * full attention so that the indexer learns before it routes). Writes into
 * `block_idx` [B,G,T,k] int32 (device, caller-owned) the selection of full
 * causal attention: row (b, g, t) holds the blocks 0 .. t / Bk ascending,
 * then -1. Given it, msa_sparse_fwd computes dense causal attention and
 * msa_bwd the KL of the index branch against the dense teacher (the head mean
 * of the full attention weights) over every visible token, with its gradients
 * to q_idx and k_idx. No index scores are computed and no workspace is used.
 * MSA_ERR_UNSUPPORTED unless k >= T / Bk (so at most T = 128 * Bk). */
MSA_API msa_status msa_warmup_block_idx(const msa_shape *shape, int32_t *block_idx, msa_stream_t stream);

/*
 * Full attention at any T: the forward and backward that msa_sparse_fwd and
 * msa_bwd compute for the selection msa_warmup_block_idx writes (every
 * visible block), without a block list and without per-(query, block)
 * scratch, so that the indexer warmup (itinai.ru "How to solve the memory
 * problem with MiniMax Sparse Attention", "Training sparse attention": the
 * first iterations run full attention) reaches the sequence lengths of the
 * sparse path. For head h in group g and query t, over every j <= t:
 *   O, LSE as msa_sparse_fwd with S(g,t) = { 0 .. t };
 *   dQ, dK, dV, dq_idx, dk_idx, KL as msa_bwd over the same set (the KL of
 *   the index softmax over every visible token against the head mean of the
 *   full attention weights).
 * Same tensors, layouts and scales as msa_sparse_fwd / msa_bwd; no block_idx.
 * shape->k is not used (any value is accepted). Supported: Hq / G in {4, 8}
 * (MSA_ERR_UNSUPPORTED otherwise: 1 or 2 heads per group take
 * msa_warmup_block_idx with the sparse calls, T <= 128 * Bk), and the other
 * limits of the common conventions. Workspace: MSA_WS_DENSE (msa_dense_fwd
 * needs only its 256-byte header).
 *
 * msa_dense_fwd is query-outer (the running maximum, sum and O of each row
 * stay on chip) and writes O and LSE once; deterministic.
 * msa_dense_bwd overwrites its six outputs with sums accumulated by fp32
 * atomic and TMA reduce-add operations from concurrent CTAs: the summation
 * order, hence the last bits, varies from run to run. O and LSE must be
 * msa_dense_fwd's outputs (or the sparse forward's under the full selection).
 */
MSA_API msa_status msa_dense_fwd(const msa_shape *shape, const void *Q, const void *K, const void *V, void *O,
                                 float *LSE, void *workspace, size_t workspace_bytes, msa_stream_t stream);
MSA_API msa_status msa_dense_bwd(const msa_shape *shape, const void *Q, const void *K, const void *V, const void *O,
                                 const void *dO, const float *LSE, const void *q_idx, const void *k_idx,
                                 float kl_weight, float *dQ, float *dK, float *dV, float *dq_idx, float *dk_idx,
                                 float *KL, void *workspace, size_t workspace_bytes, msa_stream_t stream);

/*
 * Serving: the layer's new tokens over a paged cache.
 *
 * The method's description stops at training; a model trained with it is
 * decoded with the three calls below. A page holds one KV block (Bk tokens) of
 * every group, so the block ids of the selection (itinai.ru "How the indexer
 * works") are columns of the page table, and a selected block is one
 * contiguous run of K and of V per group.
 *
 * A batch is S sequences with N rows (new tokens) in all, in sequence order:
 * sequence s has the rows row_start[s] .. row_start[s+1] - 1 (any count, none
 * included), and row r of it the position
 *   t = seq_len[s] - (row_start[s+1] - r),
 * seq_len[s] being the sequence's tokens with its new ones. Rows from
 * row_start[S] on (a padded batch) are left alone: nothing of theirs is read
 * into a result, and their outputs stay as they were.
 *
 * The batch description (row_start, seq_len, page_table, block_idx) is read on
 * the device when the kernels run; a call's launches depend on `shape` and on
 * which pointers are NULL only, so a captured call can be replayed on another
 * batch of the same shape. Kernels check it: a position outside the page table
 * (or, with a shared prefix, inside the prefix), a page id outside
 * [0, num_pages), prefix pages that differ between sequences, or a block list
 * that is not ascending ids up to the row's own block sets the error word, and
 * the outputs of the sequences concerned (of all, for the prefix) are
 * unspecified; nothing is read or written out of range.
 *
 * Supported: d = 128, d_idx = 64, Bk = 128, Hq / G in {1, 2, 4, 8},
 * 1 <= k <= 128, S <= 65535, N <= 2^20, Hq <= 65536 (N * Hq <= 2^28),
 * max_blocks <= 8192 (2^20 tokens), num_pages * G < 2^24. Two calls may run at the same time if
 * they have workspaces of their own. All results are the same bits in every
 * run on the same inputs.
 *
 * Values that are not finite, where a row sees them: an infinity in V gives
 * that infinity in O (both signs, or NaN, give NaN), in the dims that have it
 * alone, unless the token's probability is below 2^-100; a NaN score gives NaN
 * in the row's O and LSE. Scores s_j are expected below 2^30 in magnitude: full
 * attention of several rows a sequence may lose rows with larger ones (NaN, or as
 * if they saw nothing).
 */
typedef struct msa_paged_shape {
  int32_t S;             /* sequences                                            */
  int32_t N;             /* rows the tensors of new tokens have                  */
  int32_t Hq;            /* query heads                                          */
  int32_t G;             /* GQA groups = KV heads = index queries per row        */
  int32_t d;             /* head dim                                             */
  int32_t d_idx;         /* index dim                                            */
  int32_t Bk;            /* tokens per page                                      */
  int32_t k;             /* blocks kept per (row, group), own block included     */
  int32_t num_pages;     /* pages of the pools                                   */
  int32_t max_blocks;    /* columns of the page table                            */
  int32_t prefix_blocks; /* msa_paged_dense_attn: leading pages that all
                            sequences share (0: none); ignored by the others     */
  float scale;           /* softmax scale; <= 0 selects 1/sqrt(d)                */
} msa_paged_shape;

/* The cache and the batch's description, all in device memory. */
typedef struct msa_paged_cache {
  void *K, *V;               /* pools [num_pages, G, Bk, d] bf16                 */
  void *k_idx;               /* pool  [num_pages, Bk, d_idx] bf16; NULL in a
                                layer without an index branch of its own         */
  const int32_t *page_table; /* [S, max_blocks] pages of block 0, 1, ...; columns
                                past a sequence's last block are not read        */
  const int32_t *row_start;  /* [S + 1], row_start[0] = 0, non-decreasing        */
  const int32_t *seq_len;    /* [S]                                              */
} msa_paged_cache;

/* Which entry point a workspace is sized for. */
enum {
  MSA_WS_PAGED_APPEND = 0, /* the appends and msa_paged_read_fp8 */
  MSA_WS_PAGED_SPARSE = 1,
  MSA_WS_PAGED_DENSE = 2,
  MSA_WS_PAGED_SPARSE_FP8 = 4,
  MSA_WS_PAGED_DENSE_FP8 = 5
};

/* Bytes of device workspace the entry point `which` needs for `shape` (0 if
 * the shape is invalid or unsupported). */
MSA_API size_t msa_paged_workspace_size(const msa_paged_shape *shape, int which);

/* Position rotation: pair i of a vector at position t turns by the angle
 * t * inv_freq[i]. The pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) with
 * `interleaved` != 0; values from rot_dim on stay as they are. */
typedef struct msa_rope {
  const float *inv_freq;     /* [rot_dim / 2] radians per position (device)      */
  const float *inv_freq_idx; /* [rot_dim_idx / 2]                                */
  int32_t rot_dim;           /* of Q and K: a multiple of 16 up to d; 0: none    */
  int32_t rot_dim_idx;       /* of q_idx and k_idx: a multiple of 16 up to d_idx */
  int32_t interleaved;
} msa_rope;

/* New rows as the projections leave them. ld_*: elements between consecutive
 * rows (0: packed), so the pieces of one fused projection can be given as they
 * lie; each row is packed, starts on a 16-byte boundary, and ld is a multiple
 * of 8. */
typedef struct msa_new_rows {
  const void *Q;     /* [N, Hq, d] bf16, or NULL with Q_out          */
  const void *K, *V; /* [N, G, d] bf16                               */
  const void *q_idx; /* [N, G, d_idx] bf16, or NULL with q_idx_out   */
  const void *k_idx; /* [N, d_idx] bf16, or NULL                     */
  int64_t ld_Q, ld_K, ld_V, ld_q_idx, ld_k_idx;
} msa_new_rows;

/*
 * Appends new tokens: row r of sequence s, position t, goes to slot t % Bk of
 * page page_table[s][t / Bk], K and k_idx rotated by their position, V as it
 * is; Q_out [N, Hq, d] and q_idx_out [N, G, d_idx] (packed) get the rotated
 * queries. The rotation is computed in fp32 from angles that are exact to fp32
 * at any position, and rounded once. Q_out may be Q, and q_idx_out q_idx, when
 * they are packed. A page that receives rows must belong to one sequence.
 */
MSA_API msa_status msa_paged_append(const msa_paged_shape *shape, const msa_paged_cache *cache, const msa_rope *rope,
                                    const msa_new_rows *rows, void *Q_out, void *q_idx_out, void *workspace,
                                    size_t workspace_bytes, msa_stream_t stream);

/*
 * The MSA layer for new tokens: msa_index_topk's selection and msa_sparse_fwd's
 * attention for each row over its sequence's pages, for a row at position t
 * with own block c_t = t / Bk:
 *   pool[c] = max_{j in block c} <q_idx[r,g,:], k_idx[j,:]>,  c < c_t,
 *   block_idx[r,g,:] = {c_t} U top-(k-1) of pool under (score descending, id
 *     ascending), written in ascending order, then -1;
 *   s_j = scale <Q[r,h,:], K[j,g,:]> over the tokens j <= t of those blocks,
 *   LSE = ln sum_j exp(s_j),  O[r,h,:] = sum_j exp(s_j - LSE) V[j,g,:].
 * The selection is that of the exact scores (blocks that fp32 sums cannot tell
 * apart are summed again without rounding); a NaN score counts as -infinity. What
 * lies in the pages behind a row's position reaches no result. Made for few rows
 * a sequence (a token, a draft): each row reads its own pages, and the scores of
 * a page are one warp's work for all rows of its sequence, so a prompt's rows
 * are right but take a multiple of the training calls' time.
 *
 * Q [N, Hq, d], q_idx [N, G, d_idx] bf16 -> block_idx [N, G, k] int32, O
 * [N, Hq, d] bf16, LSE [N, Hq] fp32. With q_idx NULL the layer reuses a
 * selection (IndexShare): block_idx is read, not written, and may come from
 * anywhere; a row whose list is empty (all -1) gives O = 0, LSE = -infinity.
 */
MSA_API msa_status msa_paged_sparse_attn(const msa_paged_shape *shape, const msa_paged_cache *cache, const void *Q,
                                         const void *q_idx, int32_t *block_idx, void *O, float *LSE, void *workspace,
                                         size_t workspace_bytes, msa_stream_t stream);

/*
 * Full attention for new tokens (msa_dense_fwd's result for each row, over all
 * tokens j <= t): the layers and training stages without a selection. The
 * first shape->prefix_blocks pages of every sequence must be the same (a
 * prompt that the batch shares); they are read once for the whole batch (a few
 * pages once a sequence, from L2, where that is quicker), and every row's
 * position must lie behind them. prefix_blocks = 0 shares nothing.
 *
 * Probabilities are multiplied with V in 16 bits. Where pages are shared, they
 * may be rounded to bf16 against those (O then differs by up to 2^-8 of
 * sum p |v|, as msa_dense_fwd's does), which depends on the shape alone; a
 * caller who wants 16 bits throughout gives prefix_blocks = 0.
 */
MSA_API msa_status msa_paged_dense_attn(const msa_paged_shape *shape, const msa_paged_cache *cache, const void *Q,
                                        void *O, float *LSE, void *workspace, size_t workspace_bytes,
                                        msa_stream_t stream);

/*
 * Positions with several axes (itself not part of the method): tokens of images
 * and videos turn by their time, line and column, each pair of a vector on one of
 * them: pair i of row r by the angle positions[r][axis[i]] * inv_freq[i]. A row's
 * place in the cache, and what it sees, still go by its position in its sequence.
 */
typedef struct msa_axes {
  const int32_t *positions; /* [N, axes] (device), any sign                         */
  const int32_t *axis;      /* [rot_dim / 2] each pair's axis; NULL: all on axis 0  */
  const int32_t *axis_idx;  /* [rot_dim_idx / 2] the same for q_idx and k_idx       */
  int32_t axes;             /* 1 .. 8                                               */
} msa_axes;

/* msa_paged_append with positions of several axes (axes NULL: msa_paged_append).
 * An axis outside [0, axes) is reported in the error word, and its pairs turn in
 * no specified way. */
MSA_API msa_status msa_paged_append_axes(const msa_paged_shape *shape, const msa_paged_cache *cache, const msa_rope *rope,
                                         const msa_axes *axes, const msa_new_rows *rows, void *Q_out, void *q_idx_out,
                                         void *workspace, size_t workspace_bytes, msa_stream_t stream);

/*
 * Serving from a cache in 8 bits: half the bytes of msa_paged_cache, so twice the
 * tokens, and less time for tokens and few rows over long contexts, where the
 * memory's speed is what counts (full attention of many rows takes as long or longer).
 *
 * Each vector of the cache (a token's K or V of one group, a token's index key) is
 * held as E4M3 codes and one power of two, its exponent + 127 in a byte (E8M0); it
 * stands for the values code * 2^e. Written is, for a vector x in fp32 (after its
 * rotation),
 *   e = the smallest with max |x_i| <= 448 * 2^e, in [-117, 120],
 *   code_i = x_i * 2^-e rounded to nearest, ties to even,
 * so a value is off by 2^-4 of itself at most (2^-10 * 2^e where that is more).
 * Values that are not finite become NaN (E4M3 has no infinity) and count for
 * nothing in e. The values are exact in bf16, but for magnitudes from 248 * 2^120 on
 * (bf16 ends at 255 * 2^120): they round to 256 * 2^120 = 2^128, which is read back
 * as an infinity. A row that sees such a key may have any result, one that sees
 * such a value of V any in that dim; other rows and dims are not reached by it.
 * Bytes other than 10 .. 247 (those e) are not supported.
 *
 * The calls below are the ones above over such a cache, their results those of the
 * values it stands for: same batches, limits, errors and NaN. Workspaces are sized
 * with the _FP8 values (the append's with MSA_WS_PAGED_APPEND).
 * Powers of two of a query and a key (a value) whose product leaves fp32's range
 * may give infinities or zeros where the exact score would not.
 */
typedef struct msa_paged_cache_fp8 {
  void *K, *V;               /* pools [num_pages, G, Bk, d] E4M3                    */
  void *K_exp, *V_exp;       /* pools [num_pages, G, Bk] E8M0, 16-byte aligned      */
  void *k_idx, *k_idx_exp;   /* pools [num_pages, Bk, d_idx] E4M3, [num_pages, Bk]
                                E8M0; NULL as in msa_paged_cache                    */
  const int32_t *page_table; /* as in msa_paged_cache                               */
  const int32_t *row_start;
  const int32_t *seq_len;
} msa_paged_cache_fp8;

/* msa_paged_append: K, V and k_idx quantised as they are written, from the fp32
 * values of the rotation; Q and q_idx stay bf16. axes may be NULL. */
MSA_API msa_status msa_paged_append_fp8(const msa_paged_shape *shape, const msa_paged_cache_fp8 *cache,
                                        const msa_rope *rope, const msa_axes *axes, const msa_new_rows *rows, void *Q_out,
                                        void *q_idx_out, void *workspace, size_t workspace_bytes, msa_stream_t stream);

/*
 * Tokens back as bf16, exactly the values that the cache stands for: row r of the
 * M rows, out_start[s] <= r < out_start[s+1], is token first[s] + r - out_start[s]
 * of sequence s (first NULL: from the first token on), K_out and V_out [M, G, d],
 * k_idx_out [M, d_idx] (NULL: not wanted), all bf16 and 32-byte aligned. Rows before
 * out_start[0] and from out_start[S] on are left alone. A token past seq_len[s] or a page outside the
 * pools is reported in the error word and its row left alone. cache->row_start and
 * shape->N, Hq, k are not used. M <= 2^28. first and out_start [S], [S + 1] are
 * device memory.
 */
MSA_API msa_status msa_paged_read_fp8(const msa_paged_shape *shape, const msa_paged_cache_fp8 *cache, const int32_t *first,
                                      const int32_t *out_start, int32_t M, void *K_out, void *V_out, void *k_idx_out,
                                      void *workspace, size_t workspace_bytes, msa_stream_t stream);

/* msa_paged_sparse_attn: the selection is that of the exact scores of the index
 * keys that the cache stands for. */
MSA_API msa_status msa_paged_sparse_attn_fp8(const msa_paged_shape *shape, const msa_paged_cache_fp8 *cache, const void *Q,
                                             const void *q_idx, int32_t *block_idx, void *O, float *LSE, void *workspace,
                                             size_t workspace_bytes, msa_stream_t stream);

/* msa_paged_dense_attn. Probabilities are multiplied with V in fp16, whatever the
 * batch's shape: each is off by 2^-11 of itself at most, or, times its page's
 * largest power of two of V, by 2^-32 of the largest such product in its row where
 * that is more (in a page whose powers of two lie more than 2^14 apart, times its
 * own one). A vector of V with the least power of two, 2^-117, may count as zeros
 * beside larger ones in its page. */
MSA_API msa_status msa_paged_dense_attn_fp8(const msa_paged_shape *shape, const msa_paged_cache_fp8 *cache, const void *Q,
                                            void *O, float *LSE, void *workspace, size_t workspace_bytes,
                                            msa_stream_t stream);

/* Message describing the last non-OK status returned on this thread. */
MSA_API const char *msa_last_error(void);

/* Synchronises `stream`, then reads and clears the device error word of
 * `workspace` (the one the last call on it used). MSA_ERR_DEVICE if a kernel
 * gave up on a wait or met a block id out of range; msa_last_error() says
 * which kernel and where. */
MSA_API msa_status msa_check_device_status(const void *workspace, msa_stream_t stream);

/* Failure-detection self-test: launches one block whose wait on an mbarrier
 * that nothing ever arrives at is bounded by `limit_us` microseconds
 * (1..1000000). The wait runs out, the kernel records a timeout in the error
 * word of `workspace` (>= 256 bytes, device memory) and returns; a following
 * msa_check_device_status() reports MSA_ERR_DEVICE. Exercises the same bounded
 * wait every kernel uses, without faulting or hanging the GPU. */
MSA_API msa_status msa_selftest_wait_timeout(void *workspace, int32_t limit_us, msa_stream_t stream);

/* Kernel timing for benchmarks. The main kernel of one stage: */
enum {
  MSA_TIME_INDEX_TOPK = 0, /* index_topk_kernel (msa_index_topk, msa_index_topk_fp8, the no-workspace call) */
  MSA_TIME_SPARSE_FWD = 1, /* sparse_fwd_kernel (msa_sparse_fwd, msa_sparse_fwd_mapped), not the map or merge */
  MSA_TIME_BWD = 2,        /* the fused backward kernel (msa_bwd, msa_bwd_mapped), not the pre-passes or merges */
  MSA_TIME_DENSE_FWD = 3,  /* dense_fwd_kernel (msa_dense_fwd) */
  MSA_TIME_DENSE_BWD = 4   /* the backward kernel of msa_dense_bwd, not D or the index LSE */
};

/* While set, every launch of kernel `which` is bracketed by
 * cudaEventRecord(start_event) and cudaEventRecord(stop_event) on the call's
 * stream, so that the caller can read the kernel's own duration with
 * cudaEventElapsedTime. The events are the caller's cudaEvent_t handles (created
 * with timing enabled, on this device) and stay the caller's; each launch
 * re-records them. Both NULL stops the recording. The setting is process-wide
 * and not synchronised between threads. MSA_ERR_INVALID_ARG for an unknown
 * `which` or for exactly one NULL event. */
MSA_API msa_status msa_set_timing_events(int32_t which, void *start_event, void *stop_event);

/* Number of kernels this library has launched in the calling process since it
 * was loaded (monotonic; for accounting in benchmarks and tests). */
MSA_API int64_t msa_kernel_launches(void);

/* ABI version: (major << 16) | minor. */
MSA_API int32_t msa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H */
