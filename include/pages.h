/*
 * Pages of a paged KV cache (libattn.so; C ABI): handing them out, sharing
 * them between requests, copying, compacting and giving them back, on the
 * device and without a host round trip.
 *
 * The transformer-basics page's cache (past_key_values) grows by append; a
 * served batch holds many such caches in one pool of pages (attn.h, paged
 * layout).  These calls keep the three arrays that describe the pool:
 *   page_table [num_rows, pages_per_req]  row b lists request b's pages in
 *       position order, -1 where it has none;
 *   ref_count [num_pages]  in how many table entries a page is listed; 0: free;
 *   cache_lens [num_rows]  entries cached per request.
 * All of it is the caller's device memory (int32) and may be read or written by
 * the caller between calls as long as the three agree.  num_pages = num_slots /
 * page_size.  The pages handed out are always the lowest-numbered free ones, in
 * the order the call states, so results do not depend on timing.
 *
 * A call changes the table and the counts and moves the bytes of the one attn_kv_t
 * that it is given.  So the layers of a model share a pool: one attn_kv_t over all
 * their slots, layer l of request b being row l * requests + b.  One call then
 * reserves, forks, frees or compacts all layers by one plan, and the attention of
 * layer l takes the rows [l * requests, (l + 1) * requests) of page_table,
 * cache_lens and slot_capacity (and that layer's k_scale and v_scale).  With a pool
 * per layer, each has a table, counts and lengths of its own.
 *
 * The calls are asynchronous on `stream`, allocate nothing, may be recorded by
 * stream capture, and report problems that only the device sees by
 * ATTN_STATUS_PAGES in the workspace's status word (attn_get_status).  Calls on
 * one pool, and calls that share a workspace, must be ordered on one stream.
 * Host-side checks: ATTN_EINVAL for NULL pointers, negative counts, a cache that
 * is not paged, num_rows < 1, more than 2^24 pages or 2^24 rows, lists longer
 * than num_rows (reserve, fork), or more than 2^31 - 1 units of 32 KB in the n
 * pages of a fork or copy; ATTN_EWORKSPACE, ATTN_EDEVICE, ATTN_ELAUNCH as in
 * attn.h.  A call with n == 0 does nothing (its lists may be NULL).
 */
#ifndef GB300_PAGES_H
#define GB300_PAGES_H

#include "attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pool's bookkeeping (host struct holding device pointers).  page_size,
 * pages_per_req and num_slots come from the attn_kv_t of the same call, whose
 * own page_table and cache_lens are not used (they normally are these). */
typedef struct attn_pages {
  int32_t* page_table; /* [num_rows, pages_per_req] */
  int32_t* ref_count;  /* [num_slots / page_size] */
  int32_t* cache_lens; /* [num_rows] */
  int32_t num_rows;
} attn_pages_t;

/* Workspace bytes for the calls below on a pool of at most max_pages pages and
 * max_rows rows: a 256-byte header (status word, see attn_workspace_init) and
 * int32 scratch.  256-byte aligned, caller-owned.  0 for invalid arguments. */
ATTN_API size_t attn_pages_workspace_size(int64_t max_pages, int32_t max_rows);

/* Room for new_tokens[i] more entries in request rows[i], i < n (int32 [n] on
 * the device): of its entries [ceil(c / page_size), ceil((c + new) / page_size)),
 * c = cache_lens, those that are -1 get a page each (reference count 1).  Pages
 * go to i = 0, 1, ... in turn and within a row by position.  All or nothing:
 * when too few pages are free, a row is out of range or listed twice, a length
 * is negative or needs more than pages_per_req pages, nothing changes and
 * ATTN_STATUS_PAGES is set. */
ATTN_API int attn_pages_reserve(const attn_kv_t* kv, const attn_pages_t* pages, const int32_t* rows,
                                const int32_t* new_tokens, int32_t n, void* workspace, size_t ws_bytes,
                                void* stream);

/* Row dst_rows[i] becomes a copy of the request in row src_rows[i], i < n: the
 * floor(c / page_size) full pages are shared (reference counts rise), and the
 * first c % page_size entries of the page after them, if any, are copied into a
 * page of the row's own (K, V and block scales; the page's other entries are
 * left as they were), so that both requests can append.  cache_lens[dst] = c,
 * the other entries of its table row -1.  Pages go to i = 0, 1, ... in turn.
 * A source may be forked several times in one call; a destination must be empty
 * (its first entry -1), listed once, and no source of the call.  All or nothing
 * as for attn_pages_reserve, also when an entry of a source is no page. */
ATTN_API int attn_pages_fork(const attn_config_t* cfg, const attn_kv_t* kv, const attn_pages_t* pages,
                             const int32_t* src_rows, const int32_t* dst_rows, int32_t n, void* workspace,
                             size_t ws_bytes, void* stream);

/* Requests rows[i] end: the reference count of every page listed in the row
 * falls by one, the row's entries become -1 and its cache_lens 0.  A row out of
 * range is skipped (ATTN_STATUS_PAGES), so is an entry that is no page or whose
 * count is already 0; a row listed twice is emptied once. */
ATTN_API int attn_pages_free(const attn_kv_t* kv, const attn_pages_t* pages, const int32_t* rows, int32_t n,
                             void* workspace, size_t ws_bytes, void* stream);

/* Page dst_pages[i] becomes a copy of page src_pages[i] (K, V and block
 * scales), i < n.  Destinations must differ from each other and from every
 * source (else those pages hold a mixture).  A pair with a number outside the
 * pool is skipped (ATTN_STATUS_PAGES).  Tables and counts are not touched. */
ATTN_API int attn_pages_copy(const attn_config_t* cfg, const attn_kv_t* kv, const int32_t* src_pages,
                             const int32_t* dst_pages, int32_t n, void* workspace, size_t ws_bytes,
                             void* stream);

/* Moves the pages in use to the front of the pool.  With L pages in use, those
 * numbered >= L, in ascending order, move to the free pages numbered < L, in
 * ascending order (K, V and block scales); every table entry and count follows.
 * Afterwards pages [0, L) are in use and the rest are free (their contents
 * are left). */
ATTN_API int attn_pages_compact(const attn_config_t* cfg, const attn_kv_t* kv, const attn_pages_t* pages,
                                void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_PAGES_H */
