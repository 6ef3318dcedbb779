// Parameter blocks, launchers and the device-side page lookup of the serving
// operators (include/attn_cache.h).  Not part of the public C ABI.
#pragma once

#include "../../include/attn_cache.h"
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
constexpr unsigned int kBadOffsets = 4u;  // cu_seqlens of an append

// Longest sequence of a decode or an eviction.  Their kernels count slots in 32 bits and step past
// the last one by up to 8 * 512 slots (evict.cu: a head's threads) or a tile.
constexpr int kMaxLength = INT32_MAX - 8191;

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

cudaError_t launch_rope(const RopeParams& p, int dtype, bool append, cudaStream_t stream);
cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, int dtype, cudaStream_t stream);

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
