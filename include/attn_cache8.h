/*
 * attn_cache8.h -- C ABI of the paged key/value cache in 8 bits (its append, its read-back and
 * attention of one new token over it) and of pages that sequences share (forking, freeing, room
 * for new tokens, copies of pages).  The conventions are those of attn_cache.h: caller-owned
 * buffers, asynchronous calls on `stream` that can be captured into CUDA graphs, what lies in
 * device memory is checked by the kernels and reported by attn_check_device_status.
 */
#ifndef ATTN_CACHE8_GB300_H
#define ATTN_CACHE8_GB300_H

#include "attn_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A cache in 8 bits.  kv.k and kv.v hold codes of one byte (strides in codes, multiples of 16;
 * head_dim a multiple of 16): ATTN_E4M3 (4 bits of exponent, 3 of mantissa, largest value 448, no
 * infinities) or ATTN_INT8 (-127 .. 127).  Each block of `block` neighbouring slots of a page
 * (page_size is a multiple of it) has a factor for each head: slot j of a page holds for head h
 * the values code * k_scale[page * k_scale_page + (j / block) * k_scale_block + h * k_scale_head],
 * and v alike.  Factors are 0 or lie in [2^-60, 2^60] (attn_decode8 takes a factor of v beyond that
 * for the nearest bound); the append makes powers of two.  A block has at most 2^26 slots, a call
 * at most 2^31 - 65536 tokens.
 * attn_cache_evict moves single slots between blocks and does not take such a cache.
 */
enum { ATTN_E4M3 = 0, ATTN_INT8 = 1 };
typedef struct {
  attn_paged_kv kv;
  float* k_scale;         /* device fp32 */
  float* v_scale;
  int64_t k_scale_page, k_scale_block, k_scale_head; /* strides, entries */
  int64_t v_scale_page, v_scale_block, v_scale_head;
  int block;              /* slots that share a factor */
  int kind;               /* ATTN_E4M3 or ATTN_INT8 */
} attn_paged_kv8;

/*
 * attn_cache_append8 -- attn_cache_append for a cache in 8 bits (dtype: that of q, k and v).  A
 * block's factor becomes the smallest power of two s in [2^-60, 2^60] with |x| <= 448 s (int8:
 * 127 s) for every finite new value x of the block and head, but not less than the factor that
 * the block's earlier slots (below seqlens[b]) have; where it grows, their codes are rounded to
 * it again.  A block without earlier slots takes its factor from the new tokens alone.  Codes are
 * the nearest ones, ties to even; what lies beyond the largest code becomes it, a NaN stays one
 * in e4m3 and becomes 0 in int8.  k is rounded once, from its rotation in fp32.  Tokens whose
 * slot or page is bad are left out and reported as there.  cu_seqlens that do not ascend, or
 * pass `tokens`, are reported and their sequences left out.
 */
int attn_cache_append8(const attn_tensor* q, const attn_tensor* oq, const attn_tensor* k,
                       const attn_tensor* v, int dtype, int tokens, int batch, int h_q, int h_k,
                       int head_dim, const attn_paged_kv8* cache, const int* seqlens,
                       const int* cu_seqlens, const attn_rotary* rotary, attn_stream_t stream);

/*
 * attn_cache_load8 -- reads slots of a cache in 8 bits back: row t of the packed k, v [tokens,
 * H_k, D] (dtype) that is the i-th of sequence b (cu_seqlens[b] <= t = cu_seqlens[b] + i <
 * cu_seqlens[b+1]) becomes the values of slot starts[b] + i, each rounded once.  So a prefix is
 * attended by the next chunk of its prompt (attn_fwd takes packed keys).  A row whose slot or page
 * is bad becomes 0 and is reported; rows from cu_seqlens[batch] on, and rows of offsets that do
 * not ascend (reported), stay as they were.
 */
int attn_cache_load8(const attn_tensor* k, const attn_tensor* v, int dtype, int tokens, int batch,
                     int h_k, int head_dim, const attn_paged_kv8* cache, const int* starts,
                     const int* cu_seqlens, attn_stream_t stream);

/*
 * attn_decode8 -- attn_decode over a cache in 8 bits, with all its arguments but the weights:
 *     s_j = scale q . (k_j ks_j),  o = softmax(s) (v vs)
 * for codes k_j, v_j and the factors ks_j, vs_j of their blocks.  The codes' products are summed
 * in fp32.  workspace: attn_decode_workspace_size(..., with_weights = 0).
 */
int attn_decode8(const attn_tensor* q, const attn_tensor* o, float* lse, int dtype, int batch,
                 int h_q, int h_k, int head_dim, float scale, const attn_paged_kv8* cache,
                 const int* seqlens, int max_seqlen, const attn_opts* opts, void* workspace,
                 size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_cache_fork -- sequences that share pages: forks, reorders and frees the rows of a block
 * table, counts references and finds room for new tokens.  refs[p] is the number of table entries
 * that name page p (of this and other tables; 0: free); an entry outside [0, num_pages) names
 * none.  Row b of the new table is made from row parents[b] of the old one (parents NULL: b
 * itself), of length n = seqlens[parents[b]]; a negative parent frees the row (all entries -1,
 * length 0).
 *   - The first row (lowest b) of a parent goes on with all its pages, also those beyond n.  If, once
 *     all rows have let go and shared, others hold one of those that it is to write (the partly full
 *     one, the room's; so after seqlens was lowered into a shared page), it gives up its pages from
 *     there on (references - 1): the partly full one is copied to a fresh page, the room's are fresh.
 *     Pages given up are not among the fresh ones of the same call.
 *   - Every other row shares the full pages (references + 1) and gets a fresh page for one that
 *     is partly full; with share == 0 it gets a fresh page for each.  (source, fresh page) is
 *     written to copies, in the order of rows and entries, for attn_cache_copy.
 *   - Entries of slots [n, n + room[b]) that name no page get a fresh one (room NULL: room_all).
 *     Room beyond max_pages * page_size is left out and reported.
 *   - Pages of rows that no row goes on with lose a reference.
 * So no slot of [n, n + room), nor any of a partly full page, lies in a page that others hold as well;
 * after seqlens was lowered a fork (parents NULL) has to run before the next append.
 * Fresh pages are the lowest ones without references then, in the order of rows and entries; where they
 * run out, entries become -1, are not copied, and are reported.  counts[0] becomes the
 * number of copies, counts[1] that of the pages without references.  copies: pairs, room for rows of
 * them (share == 0: rows * max_pages); further ones are left as they were.  A parent >= rows is
 * reported and taken for b, a bad length for 0, a shared entry without a page stays without one
 * (reported).  Outputs may be the inputs themselves (the same pointer and stride), other overlaps
 * are not allowed.  rows * max_pages and num_pages stay below 2^31 - 2^20.  workspace:
 * attn_cache_fork_workspace_size bytes, 256-byte aligned, not shared by calls that may overlap.  The
 * copies have to run (attn_cache_copy, for every cache of the table) before anything is appended.
 * attn_cache_evict moves slots within all pages of a sequence, also those that others share: rows that
 * are to be evicted are forked with share == 0 from the start (a row that goes on keeps the full pages
 * that it shares already, whatever share is).  Per-slot state (weights, slot positions) is the caller's to
 * reorder.
 */
size_t attn_cache_fork_workspace_size(int rows, int max_pages, int num_pages);
int attn_cache_fork(const int* block_table, int64_t table_stride, int* table_out,
                    int64_t out_stride, const int* seqlens, int* seqlens_out, const int* refs,
                    int* refs_out, int num_pages, int rows, int max_pages, int page_size,
                    const int* parents, const int* room, int room_all, int share, int* copies,
                    int* counts, void* workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_cache_copy -- copies pages: for i < num_pairs (count given: i < *count, too) page
 * pairs[2 i + 1] of the cache becomes page pairs[2 i], keys, values and, where k_scale and
 * v_scale are given, factors.  element_size: 2 (fp16, bf16) or 1 (8 bits).  cache->kv's table is
 * not used.  A page that is a target must be neither a source nor another target.  A pair that
 * names no page is left out and reported.
 */
int attn_cache_copy(const attn_paged_kv8* cache, int element_size, int h_k, int head_dim,
                    const int* pairs, const int* count, int num_pairs, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_CACHE8_GB300_H */
