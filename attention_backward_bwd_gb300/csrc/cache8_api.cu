// Host side of the C ABI of the cache in 8 bits and of shared pages (include/attn_cache8.h):
// argument checks and launches, as in cache_api.cu.
#include <cuda_runtime.h>

#include <cstring>

#include "cache.h"

namespace attn {

namespace {

// Strides of factors: positive wherever a dimension is longer than one; those of pages and blocks
// are held in 32 bits.
int check_factors(const float* s, const char* name, const int64_t (&st)[3], int64_t pages, int64_t blocks,
                  int64_t heads) {
  if (s == nullptr) return fail(ATTN_ERR_NULL, "%s is NULL", name);
  if (!aligned(s, 4)) return fail(ATTN_ERR_ALIGN, "%s must be 4-byte aligned", name);
  const int64_t n[3] = {pages, blocks, heads};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && st[i] <= 0)
      return fail(ATTN_ERR_STRIDE, "%s: strides must be positive (got page=%lld block=%lld head=%lld)", name,
                  static_cast<long long>(st[0]), static_cast<long long>(st[1]), static_cast<long long>(st[2]));
  for (int i = 0; i < 2; ++i)
    if (n[i] > 1 && st[i] > UINT32_MAX)
      return fail(ATTN_ERR_STRIDE, "%s: page and block strides must stay below 2^32", name);
  return ATTN_OK;
}

int check_cache8(const attn_paged_kv8* c, int batch, int h_k, int head_dim, Cache8Arg* out) {
  if (c == nullptr) return fail(ATTN_ERR_NULL, "cache is NULL");
  if (head_dim % 16 != 0)
    return fail(ATTN_ERR_SHAPE, "head_dim must be a multiple of 16 for a cache in 8 bits, got %d", head_dim);
  if (c->kind != ATTN_E4M3 && c->kind != ATTN_INT8)
    return fail(ATTN_ERR_DTYPE, "kind must be ATTN_E4M3 or ATTN_INT8, got %d", c->kind);
  int rc = check_cache(&c->kv, batch, h_k, &out->pages, 16);
  if (rc) return rc;
  if (c->block <= 0 || c->kv.page_size % c->block != 0)
    return fail(ATTN_ERR_SHAPE, "block (%d) must be positive and divide page_size (%d)", c->block, c->kv.page_size);
  if (c->block > kMaxBlock) return fail(ATTN_ERR_SHAPE, "block must be at most 2^26, got %d", c->block);
  out->ks[0] = c->k_scale_page;
  out->ks[1] = c->k_scale_block;
  out->ks[2] = c->k_scale_head;
  out->vs[0] = c->v_scale_page;
  out->vs[1] = c->v_scale_block;
  out->vs[2] = c->v_scale_head;
  const int blocks = c->kv.page_size / c->block;
  if ((rc = check_factors(c->k_scale, "k_scale", out->ks, c->kv.num_pages, blocks, h_k))) return rc;
  if ((rc = check_factors(c->v_scale, "v_scale", out->vs, c->kv.num_pages, blocks, h_k))) return rc;
  out->k_scale = c->k_scale;
  out->v_scale = c->v_scale;
  out->block.set(static_cast<uint32_t>(c->block));
  out->int8 = c->kind == ATTN_INT8;
  return ATTN_OK;
}

// Whether [a, a + n) and [b, b + m) share an entry.
bool overlap(const int* a, int64_t n, const int* b, int64_t m) {
  return a != nullptr && b != nullptr && a < b + m && b < a + n;
}

}  // namespace

}  // namespace attn

using namespace attn;

extern "C" {

int attn_cache_append8(const attn_tensor* q, const attn_tensor* oq, const attn_tensor* k,
                       const attn_tensor* v, int dtype, int tokens, int batch, int h_q, int h_k,
                       int head_dim, const attn_paged_kv8* cache, const int* seqlens,
                       const int* cu_seqlens, const attn_rotary* rotary, attn_stream_t stream) {
  clear_error();
  const bool with_q = q != nullptr && q->ptr != nullptr;
  if (with_q != (oq != nullptr && oq->ptr != nullptr))
    return fail(ATTN_ERR_ARG, "q and oq must both be given or both be NULL");
  if (with_q && rotary == nullptr)
    return fail(ATTN_ERR_ARG, "q is only taken to be rotated: give rotary, or no q");
  int rc = check_heads(dtype, batch, with_q ? h_q : h_k, h_k, head_dim);
  if (rc) return rc;
  if (static_cast<int64_t>(h_q) + 2 * static_cast<int64_t>(h_k) > INT32_MAX / 2)
    return fail(ATTN_ERR_SHAPE, "h_q + 2 h_k must stay below 2^30");
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(ATTN_ERR_SHAPE, "tokens must lie in [0, 2^31 - 65536], got %d", tokens);
  if (cu_seqlens == nullptr && tokens != batch)
    return fail(ATTN_ERR_ARG, "without cu_seqlens there is one token a sequence: got %d tokens, %d "
                "sequences", tokens, batch);
  if (rotary != nullptr && rotary->inverse)
    return fail(ATTN_ERR_ARG, "keys enter the cache rotated forward: inverse must be 0");
  Append8Params p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = check_cache8(cache, batch, h_k, head_dim, &p.cache))) return rc;
  if (seqlens == nullptr) return fail(ATTN_ERR_NULL, "seqlens is NULL");
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
  p.bf16 = dtype == ATTN_BF16;
  p.tokens = tokens;
  p.batch = batch;
  p.h_q = with_q ? h_q : 0;
  p.h_k = h_k;
  p.head_dim = head_dim;
  p.seqlens = seqlens;
  p.cu = cu_seqlens;
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_append8(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "append8 launch");
}

int attn_cache_load8(const attn_tensor* k, const attn_tensor* v, int dtype, int tokens, int batch,
                     int h_k, int head_dim, const attn_paged_kv8* cache, const int* starts,
                     const int* cu_seqlens, attn_stream_t stream) {
  clear_error();
  int rc = check_heads(dtype, batch, h_k, h_k, head_dim);
  if (rc) return rc;
  if (tokens < 0 || tokens > kMaxTokens)
    return fail(ATTN_ERR_SHAPE, "tokens must lie in [0, 2^31 - 65536], got %d", tokens);
  if (static_cast<int64_t>(h_k) * head_dim > INT32_MAX) return fail(ATTN_ERR_SHAPE, "h_k * head_dim must stay below 2^31");
  Load8Params p;
  std::memset(&p, 0, sizeof(p));
  if ((rc = check_cache8(cache, batch, h_k, head_dim, &p.cache))) return rc;
  if (starts == nullptr || cu_seqlens == nullptr)
    return fail(ATTN_ERR_NULL, "starts and cu_seqlens must be given");
  if (!aligned(starts, 4) || !aligned(cu_seqlens, 4))
    return fail(ATTN_ERR_ALIGN, "starts and cu_seqlens must be 4-byte aligned");
  if (tokens == 0) return ATTN_OK;
  if ((rc = check_rows(k, "k", 1, tokens, h_k))) return rc;
  if ((rc = check_rows(v, "v", 1, tokens, h_k))) return rc;
  p.k = arg(k);
  p.v = arg(v);
  p.bf16 = dtype == ATTN_BF16;
  p.tokens = tokens;
  p.batch = batch;
  p.h_k = h_k;
  p.head_dim = head_dim;
  p.starts = starts;
  p.cu = cu_seqlens;
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_load8(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "load8 launch");
}

int attn_decode8(const attn_tensor* q, const attn_tensor* o, float* lse, int dtype, int batch,
                 int h_q, int h_k, int head_dim, float scale, const attn_paged_kv8* cache,
                 const int* seqlens, int max_seqlen, const attn_opts* opts_in, void* workspace,
                 size_t workspace_bytes, attn_stream_t stream) {
  clear_error();
  int rc = check_common(dtype, batch, 0, 0, h_q, h_k, head_dim, scale, nullptr, nullptr, 0, 0);
  if (rc) return rc;
  attn_opts opts;
  if ((rc = resolve_opts(opts_in, &opts))) return rc;
  if (opts.seqused_q != nullptr || opts.seqused_k != nullptr)
    return fail(ATTN_ERR_ARG, "seqused_q/k must be NULL: seqlens gives the used lengths");
  Decode8Params p;
  std::memset(&p, 0, sizeof(p));
  Cache8Arg c;
  if ((rc = check_cache8(cache, batch, h_k, head_dim, &c))) return rc;
  if ((rc = check_length(&cache->kv, max_seqlen))) return rc;
  if ((rc = check_rows(q, "q", batch, 1, h_q))) return rc;
  if ((rc = check_rows(o, "o", batch, 1, h_q))) return rc;
  if (seqlens == nullptr) return fail(ATTN_ERR_NULL, "seqlens is NULL");
  if (!aligned(seqlens, 4) || !aligned(lse, 4))
    return fail(ATTN_ERR_ALIGN, "seqlens and lse must be 4-byte aligned");
  const DecodeWs w = decode_ws(batch, h_q, h_k, head_dim, max_seqlen, false);
  if ((rc = check_workspace(workspace, workspace_bytes, w.total))) return rc;
  p.q = arg(q);
  p.o = arg(o);
  p.cache = c.pages;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  std::memcpy(p.ks, c.ks, sizeof(p.ks));
  std::memcpy(p.vs, c.vs, sizeof(p.vs));
  p.block = c.block;
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
  p.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + w.off_parts);
  p.bf16 = dtype == ATTN_BF16;
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_decode8(p, c.int8, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "decode8 launch");
}

size_t attn_cache_fork_workspace_size(int rows, int max_pages, int num_pages) {
  if (rows <= 0 || max_pages <= 0 || num_pages <= 0 || static_cast<int64_t>(rows) * max_pages > kMaxEntries ||
      num_pages > kMaxEntries)
    return 0;
  return fork_ws(rows, max_pages, num_pages);
}

int attn_cache_fork(const int* block_table, int64_t table_stride, int* table_out,
                    int64_t out_stride, const int* seqlens, int* seqlens_out, const int* refs,
                    int* refs_out, int num_pages, int rows, int max_pages, int page_size,
                    const int* parents, const int* room, int room_all, int share, int* copies,
                    int* counts, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  clear_error();
  if (rows <= 0 || num_pages <= 0 || page_size <= 0 || max_pages <= 0)
    return fail(ATTN_ERR_SHAPE, "rows (%d), num_pages (%d), page_size (%d) and max_pages (%d) must be positive", rows,
                num_pages, page_size, max_pages);
  if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX)
    return fail(ATTN_ERR_SHAPE, "max_pages * page_size must stay below 2^31");
  const int64_t entries = static_cast<int64_t>(rows) * max_pages;
  if (entries > kMaxEntries || num_pages > kMaxEntries)
    return fail(ATTN_ERR_SHAPE, "rows * max_pages and num_pages must stay below 2^31 - 2^20");
  for (const void* ptr : {static_cast<const void*>(block_table), static_cast<const void*>(table_out),
                          static_cast<const void*>(seqlens), static_cast<const void*>(seqlens_out),
                          static_cast<const void*>(refs), static_cast<const void*>(refs_out),
                          static_cast<const void*>(copies), static_cast<const void*>(counts)}) {
    if (ptr == nullptr)
      return fail(ATTN_ERR_NULL, "the table, seqlens and refs, their outputs, copies and counts must be given");
    if (!aligned(ptr, 4)) return fail(ATTN_ERR_ALIGN, "the arrays must be 4-byte aligned");
  }
  if (!aligned(parents, 4) || !aligned(room, 4))
    return fail(ATTN_ERR_ALIGN, "parents and room must be 4-byte aligned");
  if (rows > 1 && (table_stride < max_pages || out_stride < max_pages))
    return fail(ATTN_ERR_STRIDE, "the table's strides (%lld, %lld) must be at least max_pages (%d)",
                static_cast<long long>(table_stride), static_cast<long long>(out_stride), max_pages);
  if (room == nullptr && room_all < 0) return fail(ATTN_ERR_ARG, "room_all must be >= 0, got %d", room_all);
  // what an array takes, from its first entry to its last
  const int64_t span = rows > 1 ? (rows - 1) * table_stride + max_pages : max_pages;
  const int64_t out_span = rows > 1 ? (rows - 1) * out_stride + max_pages : max_pages;
  const int64_t most = share ? rows : entries;
  struct Range {
    const int* at;
    int64_t n;
  };
  const Range in[] = {{block_table, span}, {seqlens, rows}, {refs, num_pages}, {parents, rows}, {room, rows}};
  const Range out[] = {{table_out, out_span}, {seqlens_out, rows}, {refs_out, num_pages}, {copies, 2 * most}, {counts, 2}};
  for (int o = 0; o < 5; ++o) {
    for (int i = 0; i < 5; ++i) {
      if (i == o && i < 3 && in[i].at == out[o].at && (i > 0 || rows == 1 || table_stride == out_stride)) continue;
      if (overlap(in[i].at, in[i].n, out[o].at, out[o].n))
        return fail(ATTN_ERR_ARG, "an output overlaps an input without being its own");
    }
    for (int i = 0; i < o; ++i)
      if (overlap(out[i].at, out[i].n, out[o].at, out[o].n)) return fail(ATTN_ERR_ARG, "two outputs overlap");
  }
  int rc = check_workspace(workspace, workspace_bytes, fork_ws(rows, max_pages, num_pages));
  if (rc) return rc;
  ForkParams p;
  std::memset(&p, 0, sizeof(p));
  p.table = block_table;
  p.table_stride = table_stride;
  p.table_out = table_out;
  p.out_stride = out_stride;
  p.seqlens = seqlens;
  p.seqlens_out = seqlens_out;
  p.refs = refs;
  p.refs_out = refs_out;
  p.num_pages = num_pages;
  p.rows = rows;
  p.max_pages = max_pages;
  p.page_size = page_size;
  p.parents = parents;
  p.room = room;
  p.room_all = room_all;
  p.share = share != 0;
  p.copies = copies;
  p.counts = counts;
  p.ws = static_cast<int*>(workspace);
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_fork(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "fork launch");
}

int attn_cache_copy(const attn_paged_kv8* cache, int element_size, int h_k, int head_dim,
                    const int* pairs, const int* count, int num_pairs, attn_stream_t stream) {
  clear_error();
  if (cache == nullptr) return fail(ATTN_ERR_NULL, "cache is NULL");
  if (element_size != 1 && element_size != 2)
    return fail(ATTN_ERR_DTYPE, "element_size must be 1 or 2, got %d", element_size);
  const attn_paged_kv& kv = cache->kv;
  const int unit = 16 / element_size;
  if (kv.num_pages <= 0 || kv.page_size <= 0 || h_k <= 0 || head_dim <= 0)
    return fail(ATTN_ERR_SHAPE, "num_pages (%d), page_size (%d), h_k (%d) and head_dim (%d) must be positive", kv.num_pages,
                kv.page_size, h_k, head_dim);
  if (head_dim > 256 || head_dim % unit != 0)
    return fail(ATTN_ERR_SHAPE, "head_dim must be a multiple of %d of at most 256, got %d", unit, head_dim);
  if (static_cast<int64_t>(kv.page_size) * h_k > (1 << 30) / (head_dim / unit))
    return fail(ATTN_ERR_SHAPE, "a page must stay below 2^30 pieces of 16 bytes");
  if (num_pairs < 0) return fail(ATTN_ERR_SHAPE, "num_pairs must be >= 0, got %d", num_pairs);
  int rc;
  if ((rc = check_rows(&kv.k, "k cache", kv.num_pages, kv.page_size, h_k, unit))) return rc;
  if ((rc = check_rows(&kv.v, "v cache", kv.num_pages, kv.page_size, h_k, unit))) return rc;
  CopyParams p;
  std::memset(&p, 0, sizeof(p));
  if ((cache->k_scale == nullptr) != (cache->v_scale == nullptr))
    return fail(ATTN_ERR_ARG, "k_scale and v_scale must both be given or both be NULL");
  if (cache->k_scale != nullptr) {
    if (cache->block <= 0 || kv.page_size % cache->block != 0)
      return fail(ATTN_ERR_SHAPE, "block (%d) must be positive and divide page_size (%d)", cache->block, kv.page_size);
    const int64_t ks[3] = {cache->k_scale_page, cache->k_scale_block, cache->k_scale_head};
    const int64_t vs[3] = {cache->v_scale_page, cache->v_scale_block, cache->v_scale_head};
    p.blocks = kv.page_size / cache->block;
    if ((rc = check_factors(cache->k_scale, "k_scale", ks, kv.num_pages, p.blocks, h_k))) return rc;
    if ((rc = check_factors(cache->v_scale, "v_scale", vs, kv.num_pages, p.blocks, h_k))) return rc;
    std::memcpy(p.ks, ks, sizeof(ks));
    std::memcpy(p.vs, vs, sizeof(vs));
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
  }
  if (num_pairs == 0) return ATTN_OK;
  if (pairs == nullptr) return fail(ATTN_ERR_NULL, "pairs is NULL");
  if (!aligned(pairs, 4) || !aligned(count, 4)) return fail(ATTN_ERR_ALIGN, "pairs and count must be 4-byte aligned");
  // Rows of k and v that lie behind one another are one row, where they do in both.
  const attn_tensor* t[2] = {&kv.k, &kv.v};
  int outer = kv.page_size, inner = h_k;
  int64_t row = head_dim;       // codes of a row
  bool slots_inside = false;    // the rows of rows[1] are slots, those of rows[0] heads
  auto both = [&](auto f) { return f(*t[0]) && f(*t[1]); };
  if (both([&](const attn_tensor& x) { return h_k == 1 || x.stride_h == row; })) {
    row *= h_k;
    inner = 1;
    if (both([&](const attn_tensor& x) { return outer == 1 || x.stride_s == row; })) {
      row *= outer;
      outer = 1;
    }
  } else if (both([&](const attn_tensor& x) { return kv.page_size == 1 || x.stride_s == row; })) {
    slots_inside = true;
    row *= kv.page_size;
    outer = h_k;
    inner = 1;
    if (both([&](const attn_tensor& x) { return x.stride_h == row; })) {
      row *= h_k;
      outer = 1;
    }
  }
  p.rows[0] = outer;
  p.rows[1] = inner;
  p.chunks = static_cast<int>(row / unit);
  TensorArg* a[2] = {&p.k, &p.v};
  for (int i = 0; i < 2; ++i) {
    a[i]->ptr = t[i]->ptr;
    a[i]->sb = t[i]->stride_b * element_size;
    a[i]->ss = (slots_inside ? t[i]->stride_h : t[i]->stride_s) * element_size;
    a[i]->sh = t[i]->stride_h * element_size;
  }
  p.heads = h_k;
  p.pairs = pairs;
  p.count = count;
  p.num_pairs = num_pairs;
  p.num_pages = kv.num_pages;
  if ((rc = status_of(&p.status))) return rc;
  const cudaError_t e = launch_copy(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e, "copy launch");
}

}  // extern "C"
