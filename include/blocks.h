/*
 * Attention over selected blocks of a KV cache (libattn.so; C ABI): bounds of a
 * block's keys, selection of blocks for each query by a score that needs only the
 * bounds, and attention over the selected blocks.
 *
 * A decode step of attn.h reads the whole cache of a request (concept chapter
 * section 4.3: decode is bound by memory bandwidth; its section 2.6 lists ways to
 * read less of it).  Here a query reads the bounds of every block, 4 D bytes
 * instead of the 2 * block_size * D entries, and then the entries of at most `keep`
 * blocks.
 *
 * Block i of a request is its positions [i * block_size, (i + 1) * block_size);
 * block_size is 64, 128 or 256, and at most page_size in a paged cache (a block
 * lies in one page).  The step of a layer, for chunks of prompts and single
 * tokens alike:
 *   attn_prefill_prepare (or attn_qkv_proj_prepare, _axes)   K, V appended, prepared Q
 *   attn_block_bounds    bounds of the blocks that these tokens fill
 *   attn_block_select    the blocks of each query: list [N, Hkv, keep]
 *   attn_block_attend    out [N, Hq * D]
 * A list may also come from elsewhere.
 *
 * q is the prepared Q [N, Hq, D] of attn_prefill_prepare: bf16, f16 next to an E4M3
 * or E2M1 cache; 16-byte aligned.  cu_seqlens: int32 [B + 1] as for attn_prefill;
 * NULL: one token per request (N == B), which spares every kernel the search for a
 * token's request.  cache_lens are the lengths before the tokens were appended,
 * as in the calls of attn.h: the token j of request b is at position c_b + j.
 *
 * The calls are asynchronous on `stream`, allocate nothing, may be recorded by
 * stream capture, and report what only the device sees in the workspace's status
 * word (attn_get_status): ATTN_STATUS_CAPACITY for a request whose region cannot
 * hold c_b + n_b entries (skipped: nothing of it is written) and for a page outside
 * the cache (it reads as zeros) or a row outside the bounds (not written, reads as
 * zeros); ATTN_STATUS_SEQLENS for tokens of no request; ATTN_STATUS_BOUNDS for a
 * request longer than max_kv_len (attn_block_select: its lists are left unwritten);
 * ATTN_STATUS_TIMEOUT for a pipeline wait that gave up (attn_block_attend: an internal
 * error, the token's output for that KV head is left unwritten).
 */
#ifndef GB300_BLOCKS_H
#define GB300_BLOCKS_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bounds of the keys of one layer's blocks (host struct holding device pointers).
 * bounds: bf16 [num_rows, Hkv, 2, D], 16-byte aligned: row r holds for each KV head
 * the lowest, then the highest entry of each component over the keys of a block.
 * The entries are those that attn_kv_gather gives (bf16; codes as the bf16 nearest
 * to their value); a component with a NaN has NaN bounds.
 * Block i of request b has the row
 *   paged cache:      (slot of position i * block_size) / block_size, num_rows >=
 *                     num_slots / block_size: pages that requests share have their
 *                     bounds in common; row_base is not used (may be NULL);
 *   contiguous cache: row_base[b] + i (int64 [B] on the device).
 * num_rows is below 2^31.
 * Only blocks that are full have bounds: a query always takes the block of its own
 * position.  attn_pages_fork, _copy and _compact move entries and not bounds: make
 * those anew with `start` (below; after a fork from the first position of the copied
 * page, after a compaction from 0). */
typedef struct attn_blocks {
  void* bounds;
  int64_t num_rows;
  const int64_t* row_base;
  int32_t block_size;
} attn_blocks_t;

/* Workspace bytes for the calls below with at most max_tokens tokens, max_kv_len
 * keys per request (c_b + n_b) and lists of `keep` blocks; covers smaller calls too.
 * It holds a 256-byte header (status word) and, for attn_block_select, 12 bytes per token,
 * KV head and block of max_kv_len, with a little per 512 of those blocks: a call with many
 * tokens over long caches can take a chunk's tokens in parts to need less.
 * 256-byte aligned, caller-owned, initialised by attn_workspace_init.  0 for invalid
 * arguments. */
ATTN_API size_t attn_block_workspace_size(const attn_config_t* cfg, int32_t max_tokens, int32_t max_kv_len,
                                          int32_t block_size, int32_t keep);

/* Bounds of the blocks of each request that hold a position in [start[b], c_b + n_b)
 * and are full (their last position is below c_b + n_b), from the cache, which
 * already holds the tokens.  start: int32 [B] on the device, or NULL for c_b: the
 * blocks that this call's tokens reach.  A negative start counts as 0.  With n_b = 0
 * and a start, bounds are made anew.  The other rows are left as they were.  The
 * workspace needs only its 256-byte header.  Every request has the same share of the grid,
 * so a long prompt among many single tokens is faster in a call of its own. */
ATTN_API int attn_block_bounds(const attn_config_t* cfg, const attn_kv_t* kv, const attn_blocks_t* blocks,
                               const int32_t* start, const int32_t* cu_seqlens, int32_t B, void* workspace,
                               size_t ws_bytes, void* stream);

/* The blocks of each query.  list: int32 [N, Hkv, keep] on the device (output).
 * The query of a token at position p sees the blocks 0 .. p / block_size, n in all.
 * With n <= keep the list of each KV head holds all of them; else the `first` first
 * ones, the `last` last ones (last >= 1: the query's own block is among them) and of
 * the others the keep - first - last with the largest score
 *   sum over d < D of M_d * lo_d + P_d * hi_d,
 *   M_d, P_d: the sums of min(q_hd, 0) and max(q_hd, 0) over the group's query heads h,
 * an upper bound of the heads' summed q . k over the block's keys as attn_kv_gather gives
 * them.  (Codes times a k_scale that is no power of two are rounded to bf16 there and in
 * the bounds, so of the values that attention takes it is one to within 2^-8 of the
 * products' magnitudes.)  Blocks of equal
 * score: the lower one first; a score that is no number counts as the largest.  The
 * scores are compared as 64-bit arithmetic gives them (fp32 sums with a bound on their error
 * decide, and what that leaves open is summed in fp64), so a list does not depend on
 * the order of fp32 sums.  Lists ascend and end with -1 where they are shorter.
 * 1 <= keep <= 4096, first >= 0, first + last <= keep.  max_kv_len >= every c_b + n_b
 * (host value; sizes the workspace and the grid). */
ATTN_API int attn_block_select(const attn_config_t* cfg, const void* q, const int32_t* cu_seqlens, int32_t B,
                               int32_t N, int32_t max_kv_len, const attn_kv_t* kv, const attn_blocks_t* blocks,
                               int32_t first, int32_t last, int32_t keep, int32_t* list, void* workspace,
                               size_t ws_bytes, void* stream);

/* Causal attention of each query over the listed blocks of its KV head:
 *   out[t, h] = softmax(q . K^T / sqrt(D)) V over the positions <= p of the blocks
 *   list[t, h / (Hq / Hkv), :]
 * out: bf16 [N, Hq * D], 16-byte aligned.  Entries of the list may come in any order;
 * a negative one and one past the query's own block are skipped, and a block listed
 * twice counts twice.  A query whose list leaves no key gets zeros.  The workspace needs
 * only its 256-byte header.  The softmax probabilities enter the second product as two
 * bf16, within 2^-16, next to an E4M3 or E2M1 cache as one f16, within 2^-11 (attn.h).
 * Every query reads its own blocks: 1.1 us a token with 64 blocks of 64 bf16 keys (Hq 32,
 * Hkv 8, D 128), however long the cache is.  attn_prefill_attend, which reads a key once
 * for many queries, is faster for a chunk of 256 tokens up to about 25 000 keys and for
 * 1000 tokens and more up to about 105 000 (the selection's time counted). */
ATTN_API int attn_block_attend(const attn_config_t* cfg, const void* q, const int32_t* cu_seqlens, int32_t B,
                               int32_t N, const attn_kv_t* kv, int32_t block_size, const int32_t* list,
                               int32_t keep, void* out, void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_BLOCKS_H */
