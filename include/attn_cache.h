/*
 * attn_cache.h -- C ABI of the serving operators of libattn_gb300.so: rotary
 * positions (with their gradient), a paged key/value cache with its append,
 * attention of one new token over the cache, and eviction by accumulated
 * attention weight.  They share attn_bwd.h's conventions: fp16 or bf16, a head
 * dimension that is a multiple of 8 in [8, 256], tensors as attn_tensor (base
 * pointers 16-byte aligned, strides of dimensions longer than one positive
 * multiples of 8 elements, the head dimension contiguous), caller-owned
 * buffers, asynchronous calls on `stream`, 0 or a negative attn_status with a
 * message in attn_last_error().  Sums, softmax statistics, weights and LSE are
 * fp32.  Every call can be captured into a CUDA graph.
 *
 * The cache.  Keys and values live in pages: k and v are [num_pages,
 * page_size, H_k, D] (stride_b between pages, stride_s between the slots of a
 * page, stride_h between heads, so a [num_pages, H_k, page_size, D] allocation
 * is passed by its strides).  Slot j of sequence b is slot j % page_size of
 * page block_table[b * table_stride + j / page_size].  Any page size >= 1.
 * Pages that a call writes (append, evict) must belong to one sequence only, and stand
 * once in its row of the table.
 *
 * Device-side checks.  Lengths, block tables and offsets live in device
 * memory, so the kernels check them: a page outside [0, num_pages) is never
 * read or written (its keys take no part in attention, rows for it are not
 * stored), a sequence whose length is negative or above what the call allows
 * is treated as described at each call.  Each such case is reported by
 * attn_check_device_status as ATTN_ERR_ARG.  Unlike a failed cu_seqlens check
 * of attn_bwd.h's calls it does not stop later calls.
 */
#ifndef ATTN_CACHE_GB300_H
#define ATTN_CACHE_GB300_H

#include "attn_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged key/value cache and the block table of a batch. */
typedef struct {
  attn_tensor k;          /* [num_pages, page_size, H_k, D] */
  attn_tensor v;
  const int* block_table; /* device int32 [batch][table_stride], max_pages used */
  int64_t table_stride;   /* entries between the rows of two sequences */
  int num_pages;
  int page_size;
  int max_pages;          /* pages a sequence may have: its slots are [0, max_pages * page_size) */
} attn_paged_kv;

/*
 * Rotary positions.  Frequency i (of n_freq) belongs to axis a when
 * sections[0] + .. + sections[a-1] <= i < sections[0] + .. + sections[a];
 * token t turns its pair i by the angle positions[a * axis_stride + t] *
 * inv_freq[i]: (x, y) -> (x cos - y sin, x sin + y cos).  The pair is
 * (x_i, x_{i + n_freq}), or (x_{2i}, x_{2i+1}) when interleaved != 0; elements
 * from 2 * n_freq on are copied.  inverse != 0 turns by the negative angle,
 * which is also the backward pass (the rotation's transpose).  For
 * |inv_freq| <= 1 the angle is exact to about 2^-24 of a turn at every int32
 * position (it is reduced in 64-bit fixed point); inv_freq must be finite.
 */
typedef struct {
  const int* positions;   /* device int32, n_axes rows of one entry per token */
  int64_t axis_stride;    /* entries between the rows of two axes */
  const float* inv_freq;  /* device fp32 [n_freq] */
  int n_freq;             /* 1 .. head_dim / 2 */
  int n_axes;             /* 1 .. 4 */
  int sections[4];        /* frequencies of each axis; the sum is n_freq */
  int interleaved;
  int inverse;
} attn_rotary;

/*
 * attn_rope -- rotates q [B, S, H_q, D] and k [B, S, H_k, D] into oq and ok in
 * one launch (k->ptr NULL: q only).  Token t of positions is b * seqlen + s;
 * packed tensors pass batch = 1.  An output may be its input itself (the same
 * pointer and strides); other overlaps are not allowed.
 */
int attn_rope(const attn_tensor* q, const attn_tensor* k, const attn_tensor* oq,
              const attn_tensor* ok, int dtype, int batch, int seqlen, int h_q, int h_k,
              int head_dim, const attn_rotary* rotary, attn_stream_t stream);

/*
 * attn_cache_append -- stores the new tokens' keys and values: token t of the
 * packed k, v [tokens, H_k, D] that is the i-th of sequence b
 * (cu_seqlens[b] <= t = cu_seqlens[b] + i < cu_seqlens[b+1]) goes to slot
 * seqlens[b] + i.  cu_seqlens NULL: one token a sequence (tokens == batch).
 * Tokens from cu_seqlens[batch] on belong to no sequence and are left out.
 * rotary (NULL: none) rotates k on its way, and q [tokens, H_q, D] into oq when
 * q and oq are given (both or neither; with rotary NULL q must be NULL;
 * inverse is refused here).  oq may be q itself.
 * slot_positions (NULL: none), int32 [batch][H_k][slots_stride]: slot j of each
 * head receives the token's number seen[b] + i (attn_cache_evict's recency).
 * A token whose slot lies outside [0, max_pages * page_size) (or outside
 * [0, slots_stride) when slot_positions is given) or on a bad page is not
 * stored and reported; so are tokens of offsets that do not ascend.  seqlens
 * is not advanced: the caller adds the new tokens.
 */
int attn_cache_append(const attn_tensor* q, const attn_tensor* oq, const attn_tensor* k,
                      const attn_tensor* v, int dtype, int tokens, int batch, int h_q, int h_k,
                      int head_dim, const attn_paged_kv* cache, const int* seqlens,
                      const int* cu_seqlens, const attn_rotary* rotary, int* slot_positions,
                      int64_t slots_stride, const int* seen, attn_stream_t stream);

/*
 * attn_decode -- attention of one new token a sequence over its cached keys:
 *     s_j = scale q . k_j (capped as softcap * tanh(s_j / softcap)),
 *     o = softmax(s) v,  lse = log sum_j exp(s_j)  (natural log)
 * for query head h with key/value head h / (H_q / H_k), over slots
 * j < seqlens[b], the new token's own (appended) key being the last.
 * q, o: [batch, H_q, D] as attn_tensor with stride_b and stride_h (stride_s
 * unused).  lse: fp32 [batch][H_q] or NULL.  opts (NULL: none): window_left
 * >= 0 keeps the slots j >= seqlens[b] - 1 - window_left; window_right is
 * checked but leaves nothing out (no slot lies behind the last); softcap as in
 * attn_fwd_ex; seqused_q/k must be NULL.  A sequence of length 0 gets o = 0 and
 * lse = +inf, as a row without keys does in attn_fwd; so does one whose length
 * is negative or above max_seqlen (and it is reported).
 * weights_in / weights_out (both or neither), fp32 [batch][H_k][weights_stride]
 * with weights_stride >= max_seqlen: weights_out[b][g][j] = weights_in[b][g][j]
 * + the sum over the group's query heads of softmax(s)_j, for j < seqlens[b];
 * further entries are left as they were.  They may be the same array.
 * max_seqlen: bound on seqlens, at most max_pages * page_size and 2^31 - 8192 (the logits
 * kept for the weights make the workspace grow with it).
 * workspace: at least attn_decode_workspace_size(...) bytes, 256-byte aligned,
 * not shared by calls that may overlap on the GPU.  It needs no clearing.  The size
 * is 0 (workspace may be NULL) for small batches with max_seqlen <= 256 without weights.
 * The result does not depend on timing: the same call gives the same bits.
 */
size_t attn_decode_workspace_size(int batch, int h_q, int h_k, int head_dim, int max_seqlen,
                                  int with_weights);
int attn_decode(const attn_tensor* q, const attn_tensor* o, float* lse, int dtype, int batch,
                int h_q, int h_k, int head_dim, float scale, const attn_paged_kv* cache,
                const int* seqlens, int max_seqlen, const attn_opts* opts,
                const float* weights_in, float* weights_out, int64_t weights_stride,
                void* workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_cache_evict -- cuts every sequence to `budget` slots, each head by its
 * own choice.  For sequence b with n = seqlens[b] > budget and head g the kept
 * slots are the `budget` of largest rank, equal ranks in favour of the lower
 * slot: rank = +inf for slots with positions_in[b][g][j] >= seen[b] - recent,
 * else weights_in[b][g][j] (a NaN ranks below everything).  Kept slots below
 * `budget` stay; the i-th kept slot at or above it moves into the i-th freed
 * slot below (its key, value, weight and position), so only rows that have to
 * move are copied and the order of the slots is not that of the tokens:
 * attention over rotated keys does not depend on it (a window does).
 * seqlens_out[b] = min(n, budget).  weights_out / positions_out receive the
 * moved state of slots < n, with 0 and -1 in slots [budget, n); further
 * entries are left as they were.  Sequences with n <= budget keep everything
 * (their state is copied when the outputs are other arrays).  Outputs may be
 * the inputs themselves, but seqlens_out must overlap neither seqlens nor seen.
 * The state arrays are [batch][H_k][state_stride], state_stride >= max_seqlen.
 * positions_in and positions_out are given both or neither; recent > 0 needs
 * them and seen.  0 < budget, 0 <= recent <= budget; max_seqlen as in attn_decode.
 * A sequence whose length is negative or above max_seqlen is left as it is, with
 * seqlens_out[b] = 0, and reported; a row whose page is bad is not copied.
 * Pages from ceil(budget / page_size) on are free for the caller afterwards.
 */
size_t attn_cache_evict_workspace_size(int batch, int h_k, int budget, int max_seqlen);
int attn_cache_evict(const attn_paged_kv* cache, int dtype, int batch, int h_k, int head_dim,
                     const int* seqlens, int* seqlens_out, int max_seqlen, int budget, int recent,
                     const int* seen, const float* weights_in, float* weights_out,
                     const int* positions_in, int* positions_out, int64_t state_stride,
                     void* workspace, size_t workspace_bytes, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_CACHE_GB300_H */
