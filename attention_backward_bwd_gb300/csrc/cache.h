// Parameter blocks, launchers and the device-side page lookup of the serving
// operators (include/attn_cache.h, attn_cache8.h).  Not part of the public C ABI.
#pragma once

#include "../../include/attn_cache8.h"
#include "internal.h"

namespace attn {

// x / d for 0 <= x < 2^31 by a multiplication: q = (umulhi(x, mul) + x) >> shift with
// shift = ceil(log2 d) and mul = floor(2^32 (2^shift - d) / d) + 1 (the round-up
// method; the sum stays below 2^32 because x < 2^31).
struct FastDiv {
  uint32_t d, mul, shift;
  void set(uint32_t div) {
    d = div;
    shift = 0;
    while (shift < 31 && (1u << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return (__umulhi(x, mul) + x) >> shift; }
#endif
};

// Bits of the device status word of these operators (status_word()[2]).
constexpr unsigned int kBadLength = 1u;   // seqlens / slots out of range
constexpr unsigned int kBadPage = 2u;     // block_table entry outside [0, num_pages)
constexpr unsigned int kBadOffsets = 4u;  // cu_seqlens of an append or a read-back
constexpr unsigned int kBadParent = 8u;   // parents of a fork
constexpr unsigned int kNoPage = 16u;     // no free page left for a fork

// Longest sequence of a decode or an eviction.  Their kernels count slots in 32 bits and step past
// the last one by up to 8 * 512 slots (evict.cu: a head's threads) or a tile.
constexpr int kMaxLength = INT32_MAX - 8191;
// Tokens of a call on the 8-bit cache, slots of one of its blocks (a block's codes are counted in 32
// bits, 16 of them at once), entries and pages of a fork: a grid's step (append8.cu: 8 blocks of 8 warps
// an SM; pages.cu: 2 of 512 threads, times 8 entries) past the last stays below 2^31.
constexpr int kMaxTokens = INT32_MAX - 65535;
constexpr int kMaxBlock = 1 << 26;
constexpr int kMaxEntries = INT32_MAX - (1 << 20);

struct PagedArg {
  TensorArg k, v;  // sb: page, ss: slot, sh: head
  const int* table;
  int64_t table_stride;
  int num_pages, max_pages;
  FastDiv page;    // by page_size
};

struct RotaryArg {
  const int* positions;  // nullptr: no rotation
  int64_t axis_stride;
  const float* inv_freq;
  int n_freq, n_axes;
  int end[4];            // first frequency behind each axis
  int interleaved;
  float sign;            // -1: inverse
};

struct RopeParams {
  TensorArg q, k, v, oq, ok;  // ptr nullptr: absent; v only with the cache
  RotaryArg rot;
  int64_t tokens;
  int seqlen;                 // rows of one batch entry (tokens of a packed tensor)
  int h_q, h_k, head_dim;
  // append
  PagedArg cache;
  const int* seqlens;
  const int* cu;              // nullptr: token t is sequence t
  int batch;
  int* slot_positions;
  int64_t slots_stride;
  const int* seen;
  unsigned int* status;
};

struct DecodeParams {
  TensorArg q, o;  // sb, sh used
  PagedArg cache;
  float* lse;
  const int* seqlens;
  int batch, h_q, h_k, group, head_dim;
  int max_seqlen, win_left;
  float scale_log2, softcap, cap_in, cap_out;
  const float* w_in;
  float* w_out;
  int64_t w_stride;
  float* lse2;     // workspace: [batch][h_q] base-2 log-sum-exp (+inf: no keys)
  float* logits;   // workspace: [batch][h_q][logit_stride] base-2 logits from the first
                   // key seen on (weights only, else nullptr)
  int64_t logit_stride;
  float* parts;    // workspace: two partials of each run of tiles
  int64_t part_stride;  // floats of a partial
  int part_rows;        // its rows of O (maxima and sums follow them)
  int head_tiles;       // 16-row tiles of a group
  int chunks;           // 16-byte chunks of a row
  int lines;            // lines of tiles: one, or one a head tile
  unsigned int* status;
  int whole;            // one block a segment, nothing to join
  int tile_log2;        // keys of a tile
};

struct EvictParams {
  PagedArg cache;
  int batch, h_k, head_dim;
  const int* seqlens;
  int* seqlens_out;
  int max_seqlen, budget, recent;
  const int* seen;
  const float* w_in;
  float* w_out;
  const int* pos_in;
  int* pos_out;
  int64_t stride;
  int* from;    // workspace: [batch * h_k][move_cap] source slots
  int* to;      // workspace: the slots they move to
  int move_cap;
  unsigned int* status;
};

// Codes of 8 bits and their factors.
struct Cache8Arg {
  PagedArg pages;              // strides in bytes
  float *k_scale, *v_scale;
  int64_t ks[3], vs[3];        // strides of page, block of tokens, head
  FastDiv block;               // by the tokens of a block
  int int8;                    // 0: e4m3
};

struct Append8Params {
  TensorArg q, oq, k, v;
  RotaryArg rot;
  int bf16;
  int tokens, batch, h_q, h_k, head_dim;
  Cache8Arg cache;
  const int* seqlens;
  const int* cu;               // nullptr: token t is sequence t
  unsigned int* status;
};

struct Load8Params {
  TensorArg k, v;              // outputs, ss and sh used
  int bf16;
  int tokens, batch, h_k, head_dim;
  Cache8Arg cache;
  const int* starts;
  const int* cu;
  unsigned int* status;
};

struct Decode8Params : DecodeParams {
  float *k_scale, *v_scale;
  int64_t ks[3], vs[3];
  FastDiv block;
  int bf16;
};

struct ForkParams {
  const int* table;            // may be table_out
  int64_t table_stride;
  int* table_out;
  int64_t out_stride;
  const int* seqlens;
  int* seqlens_out;
  const int* refs;
  int* refs_out;
  int num_pages, rows, max_pages, page_size;
  const int* parents;          // nullptr: every row its own
  const int* room;             // nullptr: room_all for every row
  int room_all;
  int share;
  int* copies;                 // pairs of pages
  int* counts;                 // copies made, pages left free
  int* ws;                     // fork_ws() bytes
  unsigned int* status;
};

struct CopyParams {
  TensorArg k, v;              // strides in bytes: page, the rows of rows[0], those of rows[1]
  int rows[2], chunks;         // a page is rows[0] x rows[1] rows of 16-byte pieces
  float *k_scale, *v_scale;
  int64_t ks[3], vs[3];
  int blocks, heads;
  const int* pairs;
  const int* count;            // nullptr: all
  int num_pairs, num_pages;
  unsigned int* status;
};

cudaError_t launch_append8(const Append8Params& p, cudaStream_t stream);
cudaError_t launch_load8(const Load8Params& p, cudaStream_t stream);
cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream);
cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream);
size_t fork_ws(int rows, int max_pages, int num_pages);
cudaError_t launch_decode8(const Decode8Params& p, int int8, cudaStream_t stream);

cudaError_t launch_rope(const RopeParams& p, int dtype, bool append, cudaStream_t stream);
cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, int dtype, cudaStream_t stream);

// Geometry of a decode with tiles of 1 << tile_log2 keys: how the groups are cut into head
// tiles, the lines, their runs (0: no keys) and whether segments are taken whole.
cudaError_t shape_decode(DecodeParams& p, int tile_log2, int blocks_per_sm, int* runs);
// Joins the partials that a decode's `runs` blocks left (not after whole segments).  far: values
// may differ by more than fp32's exponents hold beside their weights.
cudaError_t launch_join(const DecodeParams& p, int dtype, int runs, bool far, cudaStream_t stream);

// ---- checks of arguments (cache_api.cu)

inline TensorArg arg(const attn_tensor* t) { return TensorArg{t->ptr, t->stride_b, t->stride_s, t->stride_h}; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// A tensor with `n` entries along batch / sequence / head: strides of dimensions longer than one
// are positive multiples of `unit` elements (16 bytes).
int check_rows(const attn_tensor* t, const char* name, int64_t nb, int64_t ns, int64_t nh, int unit = 8);
int check_heads(int dtype, int batch, int h_q, int h_k, int head_dim);
int check_cache(const attn_paged_kv* c, int batch, int h_k, PagedArg* out, int unit = 8);
int check_length(const attn_paged_kv* c, int max_seqlen);
int check_rotary(const attn_rotary* r, int64_t tokens, int head_dim, RotaryArg* out);
// The operators' device status word (separate from the one that stops later varlen calls).
int status_of(unsigned int** out);
int check_workspace(const void* ws, size_t given, size_t need);

// Moves of one head are at most the slots above the budget, and at most the budget.
inline int evict_move_cap(int budget, int max_seqlen) {
  const int above = max_seqlen > budget ? max_seqlen - budget : 0;
  return above < budget ? above : budget;
}

struct DecodeWs {
  size_t off_lse2, off_parts, off_logits, total;
  int64_t logit_stride;
};
DecodeWs decode_ws(int batch, int h_q, int h_k, int head_dim, int max_seqlen, bool weights);

#ifdef __CUDACC__
__device__ __forceinline__ void report(unsigned int* status, unsigned int bit) { atomicOr(status, bit); }

// Page and slot within it of slot j (0 <= j < max_pages * page_size) of a
// sequence's table row; false (and reported) when the table names no page.
__device__ __forceinline__ bool page_of(const PagedArg& c, const int* row, int j, int& page,
                                        int& within, unsigned int* status) {
  const int n = static_cast<int>(c.page.div(static_cast<uint32_t>(j)));
  within = j - n * static_cast<int>(c.page.d);
  page = row[n];
  if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages)) return true;
  report(status, kBadPage);
  return false;
}
#endif

}  // namespace attn
