/*
 * misa.h -- C ABI of the B200 (sm_100a) MISA indexer library.
 *
 * The operations are those of "MISA: Mixture of Indexer Sparse Attention for
 * Long-Context LLM Inference" (picx.dev summary page, Methodology sections 1-2):
 * block pooling of indexer keys (Eq. 4), the block-pooled head router
 * (Eqs. 7-8), routed token scoring with top-k selection (Eqs. 9-10), the dense
 * DSA indexer the method replaces (Introduction, Eqs. 1-2), and the
 * hierarchical MISA-dagger re-rank (Eqs. 11-12); and what uses their selection: attention
 * over a paged key-value cache, with the upkeep of that cache ("Paged key-value cache" below).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers.  Every tensor pointer is a DEVICE pointer on the current CUDA
 *   device.  bf16 tensors are passed as their 16-bit patterns (uint16_t).
 *   q, k and k_pool must be 16-byte aligned; all tensors are dense, row-major
 *   (last index fastest), with no padding.
 * Shapes.  nseq independent sequences; T query rows per sequence; L keys per
 *   sequence; H = H^I indexer heads; d = head dim (only d = 128 is built);
 *   B = router block size; h = routed heads; topk = k; kprime = k'.
 *     q      bf16  [nseq, T, H, d]    indexer queries q^I
 *     w      fp32  [nseq, T, H]       head weights w^I
 *     k      bf16  [nseq, L, d]       indexer keys k^I (one key stream per sequence)
 *     pos    int32 [nseq, T]          absolute position of each query; query (n, t)
 *                                     sees keys s = 0 .. pos[n,t] (prefix P = pos+1);
 *                                     -1: a padded row, which sees nothing: its idx is all
 *                                     -1, its heads are those of position 0
 *     k_pool fp32  [nseq, ceil(L/B), d]
 *     heads  int32 [nseq, T, h]
 *     E      fp32  [nseq, T, H]
 *     idx    int32 [nseq, T, topk]    selected token indices
 *     vals   fp32  [nseq, T, topk]    their scores
 * Ownership.  The caller owns every buffer.  The library never allocates or
 *   frees device memory and keeps no state between calls.  Scratch space is a
 *   caller-provided workspace of at least misa_workspace_size(...) bytes; it must
 *   be zero-filled once after allocation (its first 256 bytes hold a sticky
 *   device status word) and must not be used by two calls that overlap on the GPU.
 * Streams.  `stream` is a cudaStream_t (NULL = legacy default stream).  Calls only
 *   enqueue work; none of them synchronises, except misa_check_device_status.
 * Errors.  Every call returns a status (MISA_OK = 0).  Arguments are validated on
 *   the host before anything is enqueued; an invalid call enqueues nothing.
 *   Conditions only the GPU can see (a pos[] entry outside [-1, L), a candidate outside its
 *   query's prefix, a bounded wait that expired) are recorded in the workspace
 *   status word; the affected values are clamped or skipped, never read out of
 *   bounds.  misa_check_device_status() reports and clears that word.
 * Ordering.  idx rows list tokens by descending score, equal scores by ascending
 *   token index, and are padded with -1 (vals -inf) when fewer than topk tokens
 *   exist.  heads rows list heads by descending E, equal E by ascending head index.
 */
#ifndef MISA_B200_MISA_H
#define MISA_B200_MISA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define MISA_OK                      0
#define MISA_ERR_INVALID_ARG         1  /* bad pointer, alignment, shape or parameter   */
#define MISA_ERR_UNSUPPORTED         2  /* valid but not built (e.g. d != 128)          */
#define MISA_ERR_CUDA                3  /* a CUDA runtime call or launch failed          */
#define MISA_ERR_DEVICE_TIMEOUT      4  /* a bounded device-side wait expired            */
#define MISA_ERR_WORKSPACE_TOO_SMALL 5  /* ws_bytes < misa_workspace_size(...)            */
#define MISA_ERR_BAD_DEVICE_INPUT    6  /* device data out of range (pos >= L, cand)     */
#define MISA_ERR_STATIC_SCRATCH_TOO_SMALL 7  /* call larger than the fixed scratch of
                                                misa_score_topk_noalloc                 */
#define MISA_ERR_OUT_OF_PAGES        8  /* misa_pages_resize: not enough free pages      */

/* Operation ids for misa_workspace_size. */
#define MISA_OP_ROUTE_HEADS   1
#define MISA_OP_SCORE_TOPK    2
#define MISA_OP_DSA_TOPK      3
#define MISA_OP_DAGGER_RERANK 4
#define MISA_OP_SCORE_ROWS    5
#define MISA_OP_HISA_TOPK     6
/* Operation ids for misa_pages_workspace_size. */
#define MISA_OP_PAGES_RESIZE  7
#define MISA_OP_PAGES_FORK    8
#define MISA_OP_PAGES_COMPACT 9

/* Limits of this build (larger values return MISA_ERR_UNSUPPORTED). */
#define MISA_HEAD_DIM        128
#define MISA_MAX_HEADS       128
#define MISA_MAX_ROUTED      128  /* h <= H <= MISA_MAX_HEADS */
#define MISA_MAX_TOPK        16384
#define MISA_MAX_POOLS       256  /* pools of one misa_pages_* call */

/* Element types of the paged cache. */
#define MISA_DTYPE_BF16 0
#define MISA_DTYPE_FP16 1

/*
 * Bytes of workspace the operation `op` needs for these sizes (0 on invalid
 * arguments).  Arguments an operation does not use are ignored.  Host-only.
 */
size_t misa_workspace_size(int op, int nseq, int T, int H, int d, int64_t L, int B,
                           int h, int topk, int kprime);

/*
 * Block pooling of the indexer keys, Eq. (4) (Methodology section 1), with Pool
 * read as the arithmetic mean: k_pool[n, b, :] = mean of k[n, s, :] over
 * s in [b*B, min((b+1)*B, L)).  The last block may be partial and is then the
 * mean of its valid keys.  Output fp32 [nseq, ceil(L/B), d].  No workspace.
 */
int misa_pool_keys(const uint16_t* k, int nseq, int64_t L, int d, int B, float* k_pool,
                   void* stream);

/*
 * Refresh of the pooled keys after keys changed: recomputes, for every sequence,
 * exactly the blocks of Eq. (4) that meet the token range [s_begin, s_end) and
 * leaves every other block of k_pool as it is.  The pages count the router as
 * O(H * M) per query, which presumes the pooled keys are kept rather than rebuilt;
 * in decode a step appends one key, so the caller refreshes [pos, pos + 1) and only
 * that key's block is re-read (B keys instead of L).  Same layout as
 * misa_pool_keys; 0 <= s_begin <= s_end <= L, else MISA_ERR_INVALID_ARG; an empty
 * range launches nothing.  No workspace.
 */
int misa_pool_keys_range(const uint16_t* k, int nseq, int64_t L, int d, int B,
                         int64_t s_begin, int64_t s_end, float* k_pool, void* stream);

/*
 * Block-pooled head router, Eqs. (7)-(8) (Methodology section 1).  For query
 * (n, t) with prefix P = pos+1 and M = ceil(P/B) blocks of that prefix:
 *   A[j, b] = w[j] * ReLU(q[j] . kp_b),   E[j] = (1/M) * sum_b |A[j, b]|,
 *   heads   = the h largest E[j].
 * kp_b is k_pool[n, b] for blocks that lie wholly inside the prefix; when P is
 * not a multiple of B the last block is the mean of keys (M-1)*B .. P-1, read
 * from k.  E may be NULL.  Needs misa_workspace_size(MISA_OP_ROUTE_HEADS, ...).
 */
int misa_route_heads(const uint16_t* q, const float* w, const uint16_t* k,
                     const float* k_pool, const int32_t* pos, int nseq, int T, int H,
                     int d, int64_t L, int B, int h, int32_t* heads, float* E, void* ws,
                     size_t ws_bytes, void* stream);

/*
 * Routed token scoring and selection, Eqs. (9)-(10) (Methodology section 1):
 *   Ihat[s] = sum_{r < h} w[heads[r]] * ReLU(q[heads[r]] . k[s]),  s = 0 .. pos,
 *   idx = TopK_s(Ihat, topk).
 * With topk = k' this is also the MISA-dagger coarse stage, Eq. (11).  vals and
 * scores may be NULL; scores, when given, is fp32 [nseq, T, L] and receives Ihat
 * for s <= pos (later entries are left untouched).  Head ids outside [0, H) are
 * recorded as bad device input and skipped.
 * Needs misa_workspace_size(MISA_OP_SCORE_TOPK, ...).
 */
int misa_score_topk(const uint16_t* q, const float* w, const uint16_t* k,
                    const int32_t* heads, const int32_t* pos, int nseq, int T, int H,
                    int d, int64_t L, int h, int topk, int32_t* idx, float* vals,
                    float* scores, void* ws, size_t ws_bytes, void* stream);

/*
 * Dense DSA indexer, Eqs. (1)-(2) (Introduction): the same as misa_score_topk
 * with all H heads.  Needs misa_workspace_size(MISA_OP_DSA_TOPK, ...).
 */
int dsa_score_topk(const uint16_t* q, const float* w, const uint16_t* k,
                   const int32_t* pos, int nseq, int T, int H, int d, int64_t L, int topk,
                   int32_t* idx, float* vals, float* scores, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * Token scores without selection: Eq. (9) over each query's prefix when heads is given
 * (h heads per query), Eq. (1) with all H heads when heads is NULL.  scores is fp32
 * [nseq, T, L]; entries s > pos are left untouched (but for entry 0 of a padded
 * row, which is not defined).  This is the scoring kernel of
 * misa_score_topk / dsa_score_topk on its own (same launch configuration), for callers
 * that select tokens themselves or inspect the scores.
 * Needs misa_workspace_size(MISA_OP_SCORE_ROWS, ...) (h = H when heads is NULL).
 */
int misa_score_rows(const uint16_t* q, const float* w, const uint16_t* k, const int32_t* heads,
                    const int32_t* pos, int nseq, int T, int H, int d, int64_t L, int h,
                    float* scores, void* ws, size_t ws_bytes, void* stream);

/*
 * MISA-dagger fine stage, Eq. (12) (Methodology section 2): for each query,
 * re-score the candidate tokens cand[n, t, 0 .. kprime-1] (int32, any order;
 * -1 = empty slot; a repeated id counts once) with all H heads,
 * I[s] = sum_j w[j] * ReLU(q[j] . k[s]), and return the topk best (ties: lower
 * token index).  Candidates outside [0, pos] are recorded as bad device input and
 * skipped.
 * Needs misa_workspace_size(MISA_OP_DAGGER_RERANK, ...).
 */
int misa_dagger_rerank(const uint16_t* q, const float* w, const uint16_t* k,
                       const int32_t* pos, const int32_t* cand, int nseq, int T, int H,
                       int d, int64_t L, int kprime, int topk, int32_t* idx, float* vals,
                       void* ws, size_t ws_bytes, void* stream);

/*
 * HISA-style token-axis block filter, the variant the pages contrast MISA with
 * ("Key distinction from HISA", Methodology section 1; the HISA abstract's
 * block-level coarse filter followed by token-level refinement).  Both use the
 * router's affinities A[j, b] = w[j] * ReLU(q[j] . kp_b) over the blocks of the
 * query's prefix (partial last block as in misa_route_heads); this one reduces
 * them across heads, G[b] = sum_j A[j, b], keeps the m blocks with the largest G
 * (ties: lower b), scores the tokens of the kept blocks with all H heads (Eq. 1),
 * and returns their topk best in idx / vals (order and padding as elsewhere).
 * k_pool must hold the pooled keys for this B (misa_pool_keys).  blocks (nullable,
 * int32 [nseq, T, m]) receives the kept blocks by descending G, -1 padded.
 * 1 <= m, m * B <= MISA_MAX_TOPK.
 * Needs misa_workspace_size(MISA_OP_HISA_TOPK, ..., B, m (as h), topk, 0).
 */
int hisa_block_filter_topk(const uint16_t* q, const float* w, const uint16_t* k,
                           const float* k_pool, const int32_t* pos, int nseq, int T, int H,
                           int d, int64_t L, int B, int m, int topk, int32_t* idx, float* vals,
                           int32_t* blocks, void* ws, size_t ws_bytes, void* stream);

/*
 * misa_score_topk without any allocation or workspace.  The paper has no
 * counterpart of this entry point; it serves callers that cannot allocate device
 * memory or pass a workspace (code running inside an allocator-free region of a
 * serving engine, or a plugin whose host framework owns every allocation).
 *
 * Computes exactly what misa_score_topk computes (Ihat and its top-k; vals may be
 * NULL).  Its scratch is a fixed array inside the library's device image: 16 MiB
 * on every GPU that loads the library, held until the process exits, enough for
 * nseq * T * L <= 4,194,304 scores; larger calls return
 * MISA_ERR_STATIC_SCRATCH_TOO_SMALL and enqueue nothing.  All calls on a device
 * share that array and it keeps the last call's contents, so calls whose GPU work
 * overlaps (other streams, other host threads) race and must be serialised by the
 * caller.  Every call looks up the array's address with the caller's device
 * current; the first call on a device also loads the library there, so make it
 * before any stream capture.  Pointers are checked like misa_score_topk's (on the
 * current device, aligned, long enough); a bad one returns MISA_ERR_INVALID_ARG.  device_status (nullable,
 * device int32) receives this call's device-side status word (MISA_OK or
 * MISA_ERR_BAD_DEVICE_INPUT), as misa_check_device_status would report it.
 * Calls no cudaMalloc, cudaFree or allocating library routine.
 */
int misa_score_topk_noalloc(const uint16_t* q, const float* w, const uint16_t* k,
                            const int32_t* heads, const int32_t* pos, int nseq, int T, int H,
                            int d, int64_t L, int h, int topk, int32_t* idx, float* vals,
                            int32_t* device_status, void* stream);

/*
 * Paged key-value cache
 * ---------------------
 * A pool holds num_pages pages of page_size tokens; sequence n keeps its tokens
 * i * page_size .. (i + 1) * page_size - 1 in page page_table[n, i].
 *     k_cache, v_cache  16-bit [num_pages, page_size, Hkv, d]  (MISA_DTYPE_*; d = 64 or 128)
 *     page_table        int32  [nseq, max_pages], -1: no page
 *     refs              int32  [num_pages], the table entries that name the page; 0: free
 * Any page_size from 1 on; max_pages * page_size, nseq * max_pages and num_pages <= 2^30,
 * num_pages * page_size < 2^31.  Tensors whose rows are moved (q, k_new, v_new, out, caches,
 * pools) are 16-byte aligned.
 * Scratch and status differ from the calls above in one way, so that calls on different
 * streams and captured graphs share nothing: `ws` is scratch only (256-byte aligned, any
 * contents, not used by two calls that overlap on the GPU), and conditions that only the GPU can
 * see go to device_status (nullable; int32 on the device, zeroed once by the caller, the first
 * condition wins and stays until misa_check_device_status(device_status, stream)).
 */

/*
 * Attention of new tokens over a paged cache: for query row (n, t) and head j,
 *   z[s] = scale * (q[n, t, j] . k[s, j / (Hq / Hkv)]),  p = softmax of z over the tokens seen,
 *   out[n, t, j] = sum_s p[s] v[s, j / (Hq / Hkv)],      lse[n, t, j] = ln sum_s exp z[s].
 * Tokens seen: idx NULL (topk 0): the prefix s = 0 .. pos[n, t].  Otherwise the tokens
 * idx[n, t, 0 .. topk) (as written by misa_score_topk, dsa_score_topk, misa_dagger_rerank and
 * hisa_block_filter_topk): any order, -1 = empty slot, each in [0, pos]; a token that is listed
 * twice counts twice.  Hq must be a multiple of Hkv.
 * pos = -1 marks a padded row, which sees nothing.  A row that sees nothing (or only scores of
 * -inf) gets out 0 and lse -inf; cache rows that no query sees are not read, so they may hold
 * anything.  Reported and skipped: idx entries outside their query's prefix, tokens whose page
 * entry is not in [0, num_pages).  Reported and clamped: pos outside [-1, max_pages *
 * page_size).  q, out: dtype, [nseq, T, Hq, d]; lse (nullable) fp32 [nseq, T, Hq].  out may be
 * q itself; otherwise what is written (out, lse, ws, device_status) must not overlap anything else.
 * Sums and softmax statistics are fp32; the weights p are rounded to dtype for their product with
 * v.  In fp16 those down to 2^-25 of their row's largest keep the type's precision, those below
 * 2^-36 of it count as 0 there.  A row whose largest score is beyond what they hold (2^30 / log2 e =
 * 7e8 in magnitude, in fp16 2^26 / log2 e = 4e7) is NaN.
 * A NaN or infinite key or value shows in the queries that see it, and in no other.  (An infinite
 * value whose weight is 0, by a score of -inf or one that vanishes in fp32, may show as itself, as
 * NaN or not at all.)
 * Made for few queries per sequence (decode, drafts): 128 / (Hq / Hkv) queries share one
 * reading of the cache.  How the work is split follows from max_pages * page_size, taken for the
 * longest sequence; a table no wider than needed is quickest for short ones.
 * ws: misa_paged_attention_workspace_size(...) bytes (0 where few or short items need none, and on
 * invalid arguments; ws may then be NULL).
 */
size_t misa_paged_attention_workspace_size(int nseq, int T, int Hq, int Hkv, int d,
                                           int page_size, int max_pages, int topk);
int misa_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* page_table, const int32_t* pos, const int32_t* idx,
                         int dtype, int nseq, int T, int Hq, int Hkv, int d, int num_pages,
                         int page_size, int max_pages, int topk, float scale, void* out,
                         float* lse, int32_t* device_status, void* ws, size_t ws_bytes,
                         void* stream);

/*
 * The keys and values of new tokens into their pages: row (n, t) of k_new / v_new (dtype,
 * [nseq, T, Hkv, d]) becomes token pos[n, t] of sequence n; pos = -1 skips the row (padding).
 * Everything else in the caches stays.  The rows of a call must name different cache rows
 * (with two for one, which of them each 16 bytes come from is undefined), and a page that others
 * hold too is theirs as well: misa_pages_resize copies it first.  Reported and skipped: pos
 * outside [-1, max_pages * page_size), page entries outside [0, num_pages).  No workspace.
 * What is written (the caches, device_status) must not overlap one another, pos or page_table, and
 * no row written may be one of k_new or v_new.
 */
int misa_paged_append(const void* k_new, const void* v_new, const int32_t* pos,
                      const int32_t* page_table, int dtype, int nseq, int T, int Hkv, int d,
                      int num_pages, int page_size, int max_pages, void* k_cache, void* v_cache,
                      int32_t* device_status, void* stream);

/*
 * Upkeep of the pages.  Each call reads page_table and refs and writes out_table and out_refs,
 * which may be the same buffers (in place); otherwise nothing that a call writes may overlap another
 * of its buffers.  `pools` (a host array of npools device pointers; NULL with npools 0) lists every
 * pool that the table pages, e.g. the k_cache and v_cache of all layers: pool i is [num_pages,
 * page_bytes[i]], page_bytes[i] a multiple of 16.  ws: misa_pages_workspace_size(op, ...) bytes (0,
 * and ws may be NULL, where none is needed; 0 on invalid arguments too).
 */
size_t misa_pages_workspace_size(int op, int nseq, int max_pages, int num_pages);

/*
 * Gives every sequence the pages for new_len[n] tokens, where it held those for old_len[n]
 * (int32 [nseq], 0 .. max_pages * page_size; entries from ceil(old_len / page_size) on count as
 * empty).  new_len 0 ends a sequence.
 *   - Growing: slots ceil(old / page_size) .. ceil(new / page_size) - 1 take free pages.  A
 *     partly filled last page that others hold too (refs > 1) is replaced by a copy of its
 *     contents in every pool, so that the new tokens may be written; where all its holders grow
 *     in this call, the one with the highest n keeps the page itself.
 *   - Shrinking: the slots from ceil(new / page_size) on become -1 and let go of their pages.
 * Pages are taken lowest first, in the order (sequence, slot), from those that are free before
 * the call; pages let go of are free after it.  When too few are free, MISA_ERR_OUT_OF_PAGES is
 * reported and nothing changes.  Reported, the row stays as it is: lengths out of range.
 */
int misa_pages_resize(const int32_t* page_table, const int32_t* refs, const int32_t* old_len,
                      const int32_t* new_len, int nseq, int max_pages, int num_pages,
                      int page_size, void* const* pools, const int64_t* page_bytes, int npools,
                      int32_t* out_table, int32_t* out_refs, int32_t* device_status, void* ws,
                      size_t ws_bytes, void* stream);

/*
 * Row n takes the pages of row parent[n] as they were before the call (int32 [nseq]; n: the row
 * stays, -1: it holds nothing afterwards), all rows at once, as a beam search reorders its
 * beams.  No page is copied: refs counts the holders.  Reported, the row stays: a parent outside
 * [-1, nseq).
 */
int misa_pages_fork(const int32_t* page_table, const int32_t* refs, const int32_t* parent,
                    int nseq, int max_pages, int num_pages, int32_t* out_table,
                    int32_t* out_refs, int32_t* device_status, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * Moves the pages in use to the front of the pools: with n_live pages in use, the i-th lowest
 * of those at or above n_live moves into the i-th lowest free page below it (contents of every
 * pool, table entries and counts).  n_live (nullable) receives n_live on the device; the pages
 * from there on are free afterwards.  Reported, left as they are: table entries outside
 * [-1, num_pages), or naming a page at or above n_live that refs says is free.
 */
int misa_pages_compact(const int32_t* page_table, const int32_t* refs, int nseq, int max_pages,
                       int num_pages, void* const* pools, const int64_t* page_bytes, int npools,
                       int32_t* out_table, int32_t* out_refs, int32_t* n_live,
                       int32_t* device_status, void* ws, size_t ws_bytes, void* stream);

/* Static text for a status code.  Host-only. */
const char* misa_status_string(int status);

/*
 * Synchronise `stream`, read the workspace status word (or a device_status word), clear it,
 * and return it (MISA_OK when no device-side condition was recorded).
 */
int misa_check_device_status(void* ws, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MISA_B200_MISA_H */
