// Host side of the serving operators' C ABI (include/attn_cache.h): argument
// checks, workspace layout and launches.  Arguments are checked before anything
// is launched; what lies in device memory is checked by the kernels.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "cache.h"

namespace attn {

namespace {

// A tensor with `n` entries along batch / sequence / head: strides of
// dimensions longer than one are positive multiples of 8 elements.
int check_rows(const attn_tensor* t, const char* name, int64_t nb, int64_t ns, int64_t nh) {
  if (t == nullptr || t->ptr == nullptr) return fail(ATTN_ERR_NULL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(t->ptr) % 16 != 0)
    return fail(ATTN_ERR_ALIGN, "%s: base pointer must be 16-byte aligned", name);
  const int64_t n[3] = {nb, ns, nh};
  const int64_t st[3] = {t->stride_b, t->stride_s, t->stride_h};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (st[i] <= 0 || st[i] % 8 != 0))
      return fail(ATTN_ERR_STRIDE,
                  "%s: strides must be positive multiples of 8 elements (got b=%lld s=%lld h=%lld)",
                  name, static_cast<long long>(t->stride_b), static_cast<long long>(t->stride_s),
                  static_cast<long long>(t->stride_h));
  if (nh > 1 && t->stride_h > INT32_MAX)
    return fail(ATTN_ERR_STRIDE, "%s: the head stride must stay below 2^31 elements", name);
  return ATTN_OK;
}

TensorArg arg(const attn_tensor* t) { return TensorArg{t->ptr, t->stride_b, t->stride_s, t->stride_h}; }

int check_heads(int dtype, int batch, int h_q, int h_k, int head_dim) {
  return check_common(dtype, batch, 0, 0, h_q, h_k, head_dim, 1.f, nullptr, nullptr, 0, 0);
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check_cache(const attn_paged_kv* c, int batch, int h_k, PagedArg* out) {
  if (c == nullptr) return fail(ATTN_ERR_NULL, "cache is NULL");
  if (c->num_pages <= 0 || c->page_size <= 0 || c->max_pages <= 0)
    return fail(ATTN_ERR_SHAPE, "num_pages (%d), page_size (%d) and max_pages (%d) must be positive",
                c->num_pages, c->page_size, c->max_pages);
  if (static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX)
    return fail(ATTN_ERR_SHAPE, "max_pages * page_size must stay below 2^31");
  int rc;
  if ((rc = check_rows(&c->k, "k cache", c->num_pages, c->page_size, h_k))) return rc;
  if ((rc = check_rows(&c->v, "v cache", c->num_pages, c->page_size, h_k))) return rc;
  // the kernels hold page and slot strides in 16-byte units of 32 bits (64 GiB a page)
  for (const attn_tensor* t : {&c->k, &c->v})
    if ((c->num_pages > 1 && t->stride_b / 8 > UINT32_MAX) ||
        (c->page_size > 1 && t->stride_s / 8 > UINT32_MAX))
      return fail(ATTN_ERR_STRIDE, "page and slot strides must stay below 2^35 elements");
  if (c->block_table == nullptr) return fail(ATTN_ERR_NULL, "block_table is NULL");
  if (!aligned(c->block_table, 4)) return fail(ATTN_ERR_ALIGN, "block_table must be 4-byte aligned");
  if (batch > 1 && c->table_stride < c->max_pages)
    return fail(ATTN_ERR_STRIDE, "table_stride (%lld) must be at least max_pages (%d)",
                static_cast<long long>(c->table_stride), c->max_pages);
  out->k = arg(&c->k);
  out->v = arg(&c->v);
  out->table = c->block_table;
  out->table_stride = c->table_stride;
  out->num_pages = c->num_pages;
  out->max_pages = c->max_pages;
  out->page.set(static_cast<uint32_t>(c->page_size));
  return ATTN_OK;
}

int check_length(const attn_paged_kv* c, int max_seqlen) {
  if (max_seqlen < 0 || max_seqlen > static_cast<int64_t>(c->max_pages) * c->page_size)
    return fail(ATTN_ERR_ARG, "max_seqlen (%d) must lie in [0, max_pages * page_size]", max_seqlen);
  if (max_seqlen > kMaxLength)
    return fail(ATTN_ERR_ARG, "max_seqlen (%d) must be at most 2^31 - 8192", max_seqlen);
  return ATTN_OK;
}

int check_rotary(const attn_rotary* r, int64_t tokens, int head_dim, RotaryArg* out) {
  if (r->n_freq < 1 || 2 * r->n_freq > head_dim)
    return fail(ATTN_ERR_SHAPE, "n_freq must lie in [1, head_dim / 2 = %d], got %d", head_dim / 2,
                r->n_freq);
  if (r->n_axes < 1 || r->n_axes > 4)
    return fail(ATTN_ERR_SHAPE, "n_axes must lie in [1, 4], got %d", r->n_axes);
  int sum = 0;
  for (int a = 0; a < 4; ++a) {
    if (a < r->n_axes) {
      if (r->sections[a] < 0 || r->sections[a] > r->n_freq)
        return fail(ATTN_ERR_SHAPE, "sections must lie in [0, n_freq], got %d", r->sections[a]);
      sum += r->sections[a];
    }
    out->end[a] = sum;
  }
  if (sum != r->n_freq)
    return fail(ATTN_ERR_SHAPE, "sections add up to %d, n_freq is %d", sum, r->n_freq);
  if (r->positions == nullptr || r->inv_freq == nullptr)
    return fail(ATTN_ERR_NULL, "positions and inv_freq must be given");
  if (!aligned(r->positions, 4) || !aligned(r->inv_freq, 4))
    return fail(ATTN_ERR_ALIGN, "positions and inv_freq must be 4-byte aligned");
  if (r->n_axes > 1 && r->axis_stride < tokens)
    return fail(ATTN_ERR_STRIDE, "axis_stride (%lld) must be at least the tokens (%lld)",
                static_cast<long long>(r->axis_stride), static_cast<long long>(tokens));
  out->positions = r->positions;
  out->axis_stride = r->axis_stride;
  out->inv_freq = r->inv_freq;
  out->n_freq = r->n_freq;
  out->n_axes = r->n_axes;
  out->interleaved = r->interleaved ? 1 : 0;
  out->sign = r->inverse ? -1.f : 1.f;
  return ATTN_OK;
}

// The operators' device status word (separate from the one that stops later
// varlen calls).
int status_of(unsigned int** out) {
  unsigned int* st = status_word();
  if (st == nullptr) return fail(ATTN_ERR_CUDA, "cannot resolve the device status word");
  *out = st + 2;
  return ATTN_OK;
}

int check_workspace(const void* ws, size_t given, size_t need) {
  if (need == 0) return ATTN_OK;
  if (ws == nullptr) return fail(ATTN_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(ATTN_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (given < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace too small: %zu bytes given, %zu needed", given, need);
  return ATTN_OK;
}

struct EvictWs {
  size_t off_to, total;
};

EvictWs evict_ws(int batch, int h_k, int budget, int max_seqlen) {
  const size_t heads = static_cast<size_t>(batch) * h_k;
  const size_t list = heads * evict_move_cap(budget, max_seqlen) * sizeof(int);
  EvictWs w;
  w.off_to = align256(list);
  w.total = w.off_to + align256(list > 0 ? list : 1);
  return w;
}

}  // namespace

}  // namespace attn

using namespace attn;

extern "C" {

int attn_rope(const attn_tensor* q, const attn_tensor* k, const attn_tensor* oq,
              const attn_tensor* ok, int dtype, int batch, int seqlen, int h_q, int h_k,
              int head_dim, const attn_rotary* rotary, attn_stream_t stream) {
  clear_error();
  const bool with_k = k != nullptr && k->ptr != nullptr;
  int rc = check_heads(dtype, batch, h_q, with_k ? h_k : h_q, head_dim);
  if (rc) return rc;
  if (seqlen < 0) return fail(ATTN_ERR_SHAPE, "seqlen must be >= 0, got %d", seqlen);
  if (rotary == nullptr) return fail(ATTN_ERR_NULL, "rotary is NULL");
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.tokens = static_cast<int64_t>(batch) * seqlen;
  if (p.tokens > INT32_MAX) return fail(ATTN_ERR_SHAPE, "batch * seqlen must stay below 2^31");
  if (p.tokens == 0) return ATTN_OK;
  if ((rc = check_rotary(rotary, p.tokens, head_dim, &p.rot))) return rc;
  if ((rc = check_rows(q, "q", batch, seqlen, h_q))) return rc;
  if ((rc = check_rows(oq, "oq", batch, seqlen, h_q))) return rc;
  p.q = arg(q);
  p.oq = arg(oq);
  if (with_k) {
    if ((rc = check_rows(k, "k", batch, seqlen, h_k))) return rc;
    if ((rc = check_rows(ok, "ok", batch, seqlen, h_k))) return rc;
    p.k = arg(k);
    p.ok = arg(ok);
  }
  p.seqlen = seqlen;
  p.batch = batch;
  p.h_q = h_q;
  p.h_k = with_k ? h_k : 0;
  p.head_dim = head_dim;
  const cudaError_t e = launch_rope(p, dtype, false, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "rope launch");
}

int attn_cache_append(const attn_tensor* q, const attn_tensor* oq, const attn_tensor* k,
                      const attn_tensor* v, int dtype, int tokens, int batch, int h_q, int h_k,
                      int head_dim, const attn_paged_kv* cache, const int* seqlens,
                      const int* cu_seqlens, const attn_rotary* rotary, int* slot_positions,
                      int64_t slots_stride, const int* seen, attn_stream_t stream) {
  clear_error();
  const bool with_q = q != nullptr && q->ptr != nullptr;
  if (with_q != (oq != nullptr && oq->ptr != nullptr))
    return fail(ATTN_ERR_ARG, "q and oq must both be given or both be NULL");
  if (with_q && rotary == nullptr)
    return fail(ATTN_ERR_ARG, "q is only taken to be rotated: give rotary, or no q");
  int rc = check_heads(dtype, batch, with_q ? h_q : h_k, h_k, head_dim);
  if (rc) return rc;
  if (tokens < 0) return fail(ATTN_ERR_SHAPE, "tokens must be >= 0, got %d", tokens);
  if (cu_seqlens == nullptr && tokens != batch)
    return fail(ATTN_ERR_ARG, "without cu_seqlens there is one token a sequence: got %d tokens, %d "
                "sequences", tokens, batch);
  if (rotary != nullptr && rotary->inverse)
    return fail(ATTN_ERR_ARG, "keys enter the cache rotated forward: inverse must be 0");
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = check_cache(cache, batch, h_k, &p.cache))) return rc;
  if (seqlens == nullptr) return fail(ATTN_ERR_NULL, "seqlens is NULL");
  if (slot_positions != nullptr) {
    if (seen == nullptr) return fail(ATTN_ERR_NULL, "slot_positions needs seen");
    if (slots_stride <= 0) return fail(ATTN_ERR_STRIDE, "slots_stride must be positive");
    if (!aligned(slot_positions, 4) || !aligned(seen, 4))
      return fail(ATTN_ERR_ALIGN, "slot_positions and seen must be 4-byte aligned");
  }
  if (!aligned(seqlens, 4) || !aligned(cu_seqlens, 4))
    return fail(ATTN_ERR_ALIGN, "seqlens and cu_seqlens must be 4-byte aligned");
  if (tokens == 0) return ATTN_OK;
  if (rotary != nullptr && (rc = check_rotary(rotary, tokens, head_dim, &p.rot))) return rc;
  if ((rc = check_rows(k, "k", 1, tokens, h_k))) return rc;
  if ((rc = check_rows(v, "v", 1, tokens, h_k))) return rc;
  p.k = arg(k);
  p.v = arg(v);
  if (with_q) {
    if ((rc = check_rows(q, "q", 1, tokens, h_q))) return rc;
    if ((rc = check_rows(oq, "oq", 1, tokens, h_q))) return rc;
    p.q = arg(q);
    p.oq = arg(oq);
  }
  p.tokens = tokens;
  p.seqlen = tokens;
  p.h_q = with_q ? h_q : 0;
  p.h_k = h_k;
  p.head_dim = head_dim;
  p.seqlens = seqlens;
  p.cu = cu_seqlens;
  p.batch = batch;
  p.slot_positions = slot_positions;
  p.slots_stride = slots_stride;
  p.seen = seen;
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_rope(p, dtype, true, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "append launch");
}

size_t attn_decode_workspace_size(int batch, int h_q, int h_k, int head_dim, int max_seqlen,
                                  int with_weights) {
  if (batch <= 0 || h_k <= 0 || h_q <= 0 || h_q % h_k != 0 || head_dim <= 0 || max_seqlen < 0 ||
      max_seqlen > kMaxLength)
    return 0;
  return decode_ws(batch, h_q, h_k, head_dim, max_seqlen, with_weights != 0).total;
}

int attn_decode(const attn_tensor* q, const attn_tensor* o, float* lse, int dtype, int batch,
                int h_q, int h_k, int head_dim, float scale, const attn_paged_kv* cache,
                const int* seqlens, int max_seqlen, const attn_opts* opts_in,
                const float* weights_in, float* weights_out, int64_t weights_stride,
                void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  clear_error();
  int rc = check_common(dtype, batch, 0, 0, h_q, h_k, head_dim, scale, nullptr, nullptr, 0, 0);
  if (rc) return rc;
  attn_opts opts;
  if ((rc = resolve_opts(opts_in, &opts))) return rc;
  if (opts.seqused_q != nullptr || opts.seqused_k != nullptr)
    return fail(ATTN_ERR_ARG, "seqused_q/k must be NULL: seqlens gives the used lengths");
  DecodeParams p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = check_cache(cache, batch, h_k, &p.cache))) return rc;
  if ((rc = check_length(cache, max_seqlen))) return rc;
  if ((rc = check_rows(q, "q", batch, 1, h_q))) return rc;
  if ((rc = check_rows(o, "o", batch, 1, h_q))) return rc;
  if (seqlens == nullptr) return fail(ATTN_ERR_NULL, "seqlens is NULL");
  if ((weights_in == nullptr) != (weights_out == nullptr))
    return fail(ATTN_ERR_ARG, "weights_in and weights_out must both be given or both be NULL");
  if (weights_in != nullptr && weights_stride < max_seqlen)
    return fail(ATTN_ERR_STRIDE, "weights_stride (%lld) must be at least max_seqlen (%d)",
                static_cast<long long>(weights_stride), max_seqlen);
  if (!aligned(seqlens, 4) || !aligned(lse, 4) || !aligned(weights_in, 4) || !aligned(weights_out, 4))
    return fail(ATTN_ERR_ALIGN, "seqlens, lse and the weights must be 4-byte aligned");
  const DecodeWs w = decode_ws(batch, h_q, h_k, head_dim, max_seqlen, weights_in != nullptr);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  char* ws = static_cast<char*>(workspace);
  p.q = arg(q);
  p.o = arg(o);
  p.lse = lse;
  p.seqlens = seqlens;
  p.batch = batch;
  p.h_q = h_q;
  p.h_k = h_k;
  p.group = h_q / h_k;
  p.head_dim = head_dim;
  p.max_seqlen = max_seqlen;
  p.win_left = opts.window_left;
  p.softcap = opts.softcap;
  p.cap_in = opts.softcap > 0.f ? scale / opts.softcap : 0.f;
  p.cap_out = opts.softcap * 1.4426950408889634f;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.w_in = weights_in;
  p.w_out = weights_out;
  p.w_stride = weights_stride;
  p.lse2 = weights_in != nullptr ? reinterpret_cast<float*>(ws + w.off_lse2) : nullptr;
  p.parts = reinterpret_cast<float*>(ws + w.off_parts);
  p.logits = weights_in != nullptr ? reinterpret_cast<float*>(ws + w.off_logits) : nullptr;
  p.logit_stride = w.logit_stride;
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_decode(p, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "decode launch");
}

size_t attn_cache_evict_workspace_size(int batch, int h_k, int budget, int max_seqlen) {
  if (batch <= 0 || h_k <= 0 || budget <= 0 || max_seqlen < 0 || max_seqlen > kMaxLength) return 0;
  return evict_ws(batch, h_k, budget, max_seqlen).total;
}

int attn_cache_evict(const attn_paged_kv* cache, int dtype, int batch, int h_k, int head_dim,
                     const int* seqlens, int* seqlens_out, int max_seqlen, int budget, int recent,
                     const int* seen, const float* weights_in, float* weights_out,
                     const int* positions_in, int* positions_out, int64_t state_stride,
                     void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  clear_error();
  int rc = check_heads(dtype, batch, h_k, h_k, head_dim);
  if (rc) return rc;
  EvictParams p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = check_cache(cache, batch, h_k, &p.cache))) return rc;
  if ((rc = check_length(cache, max_seqlen))) return rc;
  if (budget <= 0 || recent < 0 || recent > budget)
    return fail(ATTN_ERR_ARG, "budget (%d) must be positive and recent (%d) in [0, budget]", budget,
                recent);
  if (seqlens == nullptr || seqlens_out == nullptr || weights_in == nullptr || weights_out == nullptr)
    return fail(ATTN_ERR_NULL, "seqlens, seqlens_out, weights_in and weights_out must be given");
  // blocks of one sequence read them while another writes its length
  for (const int* in : {seqlens, seen})
    if (in != nullptr && in < seqlens_out + batch && seqlens_out < in + batch)
      return fail(ATTN_ERR_ARG, "seqlens_out must not overlap seqlens or seen");
  if ((positions_in == nullptr) != (positions_out == nullptr))
    return fail(ATTN_ERR_ARG, "positions_in and positions_out must both be given or both be NULL");
  if (recent > 0 && (positions_in == nullptr || seen == nullptr))
    return fail(ATTN_ERR_ARG, "recent > 0 needs the positions and seen");
  if (state_stride < max_seqlen || state_stride <= 0)
    return fail(ATTN_ERR_STRIDE, "state_stride (%lld) must be positive and at least max_seqlen (%d)",
                static_cast<long long>(state_stride), max_seqlen);
  if (!aligned(seqlens, 4) || !aligned(seqlens_out, 4) || !aligned(weights_in, 4) ||
      !aligned(weights_out, 4) || !aligned(positions_in, 4) || !aligned(positions_out, 4) ||
      !aligned(seen, 4))
    return fail(ATTN_ERR_ALIGN, "the arrays must be 4-byte aligned");
  const EvictWs w = evict_ws(batch, h_k, budget, max_seqlen);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  char* ws = static_cast<char*>(workspace);
  p.batch = batch;
  p.h_k = h_k;
  p.head_dim = head_dim;
  p.seqlens = seqlens;
  p.seqlens_out = seqlens_out;
  p.max_seqlen = max_seqlen;
  p.budget = budget;
  p.recent = recent;
  p.seen = seen;
  p.w_in = weights_in;
  p.w_out = weights_out;
  p.pos_in = positions_in;
  p.pos_out = positions_out;
  p.stride = state_stride;
  p.from = reinterpret_cast<int*>(ws);
  p.to = reinterpret_cast<int*>(ws + w.off_to);
  p.move_cap = evict_move_cap(budget, max_seqlen);
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_evict(p, dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "evict launch");
}

}  // extern "C"
