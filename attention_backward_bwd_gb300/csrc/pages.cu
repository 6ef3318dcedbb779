// Pages that sequences share: forking, freeing and room for new tokens (attn_cache_fork), and the
// copy of pages (attn_cache_copy).
//
// attn_cache_fork works on the block table and the pages' counts of references alone.  One cluster
// of blocks takes it in steps that the cluster's barrier parts: who goes on with which row, the
// references that go and come and what each row needs, prefix sums over rows and the number of free
// pages in each block's part of the pool, the list of the lowest free pages, the new rows.  Which
// page a row gets follows from its place alone, so that the result does not depend on timing.  It
// is bound by the chain of these steps and of loads behind them.
// attn_cache_copy moves whole pages, 16 bytes a thread, several in flight: bound by the memory.
#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kForkThreads = 1024;
constexpr int kCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Workspace of a fork: per row the first row that takes it over, its parent, its length, the
// pages and copies it needs and their prefix sums; per block its free pages; the sums; then the
// list of free pages and, where the table is its own output, the old table.
struct ForkWs {
  int *who, *parent, *len, *fresh, *copied, *fresh_before, *copied_before, *free_of, *sums, *list, *old;
};
__host__ __device__ inline ForkWs fork_layout(int* ws, int64_t rows, int64_t list) {
  ForkWs w;
  w.who = ws;
  w.parent = w.who + rows;
  w.len = w.parent + rows;
  w.fresh = w.len + rows;
  w.copied = w.fresh + rows;
  w.fresh_before = w.copied + rows;
  w.copied_before = w.fresh_before + rows;
  w.free_of = w.copied_before + rows;
  w.sums = w.free_of + kCluster;
  w.list = w.sums + 8;
  w.old = w.list + list;
  return w;
}

// Block-wide exclusive prefix sum; `total` of all threads.
__device__ __forceinline__ int block_prefix(int mine, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = warp_sums[lane];
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, i);
    if (lane >= i) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  return (warp == 0 ? 0 : before) + x - mine;
}

// What a row of the new table is made of.
struct Row {
  int parent, n;      // -1: none; its length
  int full, used, need;  // entries of full pages, of pages with slots, with the room
  bool heir;          // goes on with its parent's pages
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kForkThreads) fork_kernel(ForkParams p, ForkWs w) {
  __shared__ int s_sums[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int at = rank * kForkThreads + tid, step = kCluster * kForkThreads;
  const int gw = at >> 5, warps = step >> 5;
  const bool in_place = p.table == p.table_out;
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  auto valid = [&](int page) { return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages); };

  // ---- lengths, the old table out of the way, the counts where they will be
  for (int b = at; b < p.rows; b += step) {
    int n = p.seqlens[b];
    if (n < 0 || n > cap) {
      report(p.status, kBadLength);
      n = 0;
    }
    w.len[b] = n;
    w.who[b] = p.rows;
  }
  if (in_place)
    for (int b = gw; b < p.rows; b += warps)
      for (int i = lane; i < p.max_pages; i += 32)
        w.old[static_cast<int64_t>(b) * p.max_pages + i] = p.table[b * p.table_stride + i];
  if (p.refs != p.refs_out)
    for (int i = at; i < p.num_pages; i += step) p.refs_out[i] = p.refs[i];
  if (at == 0) w.sums[2] = 0;
  cluster_sync();

  // ---- the first row of each parent goes on with its pages
  for (int b = at; b < p.rows; b += step) {
    int s = p.parents == nullptr ? b : p.parents[b];
    if (s >= p.rows) {
      report(p.status, kBadParent);
      s = b;
    }
    w.parent[b] = s;
    if (s >= 0) atomicMin(w.who + s, b);
  }
  cluster_sync();

  auto old_row = [&](int b) -> const int* {
    return in_place ? w.old + static_cast<int64_t>(b) * p.max_pages : p.table + b * p.table_stride;
  };
  auto row_of = [&](int b, bool tell) {
    Row r;
    r.parent = __ldcg(w.parent + b);
    r.n = r.parent < 0 ? 0 : __ldcg(w.len + r.parent);
    r.heir = r.parent >= 0 && __ldcg(w.who + r.parent) == b;
    r.full = r.n / p.page_size;
    r.used = r.full + (r.n % p.page_size != 0 ? 1 : 0);
    const int room = r.parent < 0 ? 0 : (p.room == nullptr ? p.room_all : p.room[b]);
    int64_t slots = static_cast<int64_t>(r.n) + (room > 0 ? room : 0);
    if (slots > cap) {
      if (tell) report(p.status, kBadLength);
      slots = cap;
    }
    r.need = static_cast<int>((slots + p.page_size - 1) / p.page_size);
    return r;
  };
  // Entry i of a row: the parent's page, whether it is shared, copied, or a fresh one is needed.
  struct Entry {
    int page;
    bool shared, copied, fresh, bad;
  };
  auto entry_of = [&](const Row& r, const int* old, int i) {
    Entry e{-1, false, false, false, false};
    if (r.parent < 0 || i >= p.max_pages) return e;
    const int page = __ldcg(old + i);
    if (r.heir) {
      e.page = valid(page) ? page : -1;
      e.fresh = e.page < 0 && i >= r.used && i < r.need;
    } else if (i < r.used) {
      e.bad = !valid(page);
      e.page = e.bad ? -1 : page;
      e.shared = !e.bad && p.share && i < r.full;
      e.copied = e.fresh = !e.bad && !e.shared;
    } else {
      e.fresh = i < r.need;
    }
    return e;
  };

  // ---- references that go and come; what each row needs
  for (int b = gw; b < p.rows; b += warps) {
    const int* own = old_row(b);
    if (__ldcg(w.who + b) == p.rows)
      for (int i = lane; i < p.max_pages; i += 32) {
        const int page = __ldcg(own + i);
        if (valid(page)) atomicSub(p.refs_out + page, 1);
      }
    const Row r = row_of(b, lane == 0);
    const int* old = r.parent < 0 ? own : old_row(r.parent);
    int fresh = 0, copied = 0;
    const int from = r.heir ? r.used : 0, end = max(r.used, r.need);
    for (int i = from + lane; i < end; i += 32) {
      const Entry e = entry_of(r, old, i);
      if (e.bad) report(p.status, kBadPage);
      if (e.shared) atomicAdd(p.refs_out + e.page, 1);
      fresh += e.fresh;
      copied += e.copied;
    }
    fresh = __reduce_add_sync(0xffffffffu, fresh);
    copied = __reduce_add_sync(0xffffffffu, copied);
    if (lane == 0) {
      w.fresh[b] = fresh;
      w.copied[b] = copied;
    }
  }
  cluster_sync();

  // ---- prefix sums over the rows (the first block); free pages of each block's part
  if (rank == 0) {
    int fresh0 = 0, copied0 = 0;
    for (int b0 = 0; b0 < p.rows; b0 += kForkThreads) {
      const int b = b0 + tid;
      int total;
      const int fresh = b < p.rows ? __ldcg(w.fresh + b) : 0, copied = b < p.rows ? __ldcg(w.copied + b) : 0;
      const int f = block_prefix(fresh, s_sums, total);
      if (b < p.rows) w.fresh_before[b] = fresh0 + f;
      fresh0 += total;
      const int c = block_prefix(copied, s_sums, total);
      if (b < p.rows) w.copied_before[b] = copied0 + c;
      copied0 += total;
    }
    if (tid == 0) w.sums[0] = fresh0;
  }
  const int page0 = static_cast<int>(static_cast<int64_t>(p.num_pages) * rank / kCluster);
  const int page1 = static_cast<int>(static_cast<int64_t>(p.num_pages) * (rank + 1) / kCluster);
  int free_here = 0;
  for (int i = page0 + tid; i < page1; i += kForkThreads) free_here += __ldcg(p.refs_out + i) == 0;
  int total;
  block_prefix(free_here, s_sums, total);
  if (tid == 0) w.free_of[rank] = total;
  cluster_sync();

  // ---- the lowest free pages, as many as are needed
  const int wanted = __ldcg(w.sums);
  int first = 0, all = 0;
#pragma unroll
  for (int c = 0; c < kCluster; ++c) {
    const int n = __ldcg(w.free_of + c);
    first += c < rank ? n : 0;
    all += n;
  }
  const int granted = min(wanted, all);
  for (int i0 = page0; i0 < page1 && first < granted; i0 += kForkThreads) {
    const int i = i0 + tid;
    const bool is_free = i < page1 && __ldcg(p.refs_out + i) == 0;
    int n;
    const int k = first + block_prefix(is_free, s_sums, n);
    if (is_free && k < granted) w.list[k] = i;
    first += n;
  }
  cluster_sync();

  // ---- the new rows
  for (int b = gw; b < p.rows; b += warps) {
    const Row r = row_of(b, false);
    const int* old = old_row(r.parent < 0 ? b : r.parent);
    int* out = p.table_out + b * p.out_stride;
    int fresh0 = __ldcg(w.fresh_before + b), copied0 = __ldcg(w.copied_before + b), made = 0;
    for (int i0 = 0; i0 < p.max_pages; i0 += 32) {
      const int i = i0 + lane;
      const Entry e = entry_of(r, old, i);
      const uint32_t fresh = __ballot_sync(0xffffffffu, e.fresh), copied = __ballot_sync(0xffffffffu, e.copied);
      const uint32_t below = (1u << lane) - 1;
      int page = e.page;
      if (e.fresh) {
        const int k = fresh0 + __popc(fresh & below);
        page = k < granted ? __ldcg(w.list + k) : -1;
        if (page >= 0) p.refs_out[page] = 1;
        else report(p.status, kNoPage);
        if (e.copied && page >= 0) {
          int* pair = p.copies + 2 * static_cast<int64_t>(copied0 + __popc(copied & below));
          pair[0] = e.page;
          pair[1] = page;
          ++made;
        }
      }
      if (i < p.max_pages) out[i] = page;
      fresh0 += __popc(fresh);
      copied0 += __popc(copied);
    }
    made = __reduce_add_sync(0xffffffffu, made);
    if (lane == 0) {
      p.seqlens_out[b] = r.n;
      if (made > 0) atomicAdd(w.sums + 2, made);
    }
  }
  cluster_sync();
  if (at == 0) {
    p.counts[0] = __ldcg(w.sums + 2);
    p.counts[1] = all - granted;
  }
}

constexpr int kCopyThreads = 256;
constexpr int kFlight = 4;  // 16-byte pieces of a thread in flight

// A block takes a part of a page of k or of v, and with a page's first part its factors.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(CopyParams p, FastDiv run, FastDiv row, int parts) {
  const int n = p.count == nullptr ? p.num_pairs : min(max(*p.count, 0), p.num_pairs);
  const int64_t items = static_cast<int64_t>(n) * 2 * parts;
  const int total = p.rows[0] * p.rows[1] * p.chunks;  // pieces of a page
  constexpr int kPart = kCopyThreads * kFlight;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t both = item / parts;
    const int part = static_cast<int>(item - both * parts), pair = static_cast<int>(both >> 1), is_v = static_cast<int>(both & 1);
    const int src = p.pairs[2 * static_cast<int64_t>(pair)], dst = p.pairs[2 * static_cast<int64_t>(pair) + 1];
    if (static_cast<unsigned>(src) >= static_cast<unsigned>(p.num_pages) ||
        static_cast<unsigned>(dst) >= static_cast<unsigned>(p.num_pages)) {
      if (threadIdx.x == 0) report(p.status, kBadPage);
      continue;
    }
    if (src == dst) continue;
    const TensorArg& t = is_v ? p.v : p.k;
    char* base = static_cast<char*>(const_cast<void*>(t.ptr));
    const char* from = base + src * t.sb;
    char* to = base + dst * t.sb;
    uint4 x[kFlight];
    int64_t off[kFlight];
    const int i0 = part * kPart + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int i = i0 + k * kCopyThreads;
      if (i >= total) break;
      const int r = static_cast<int>(run.div(i)), c = i - r * p.chunks;
      const int r0 = static_cast<int>(row.div(r)), r1 = r - r0 * p.rows[1];
      off[k] = r0 * t.ss + r1 * t.sh + static_cast<int64_t>(c) * 16;
      x[k] = __ldcs(reinterpret_cast<const uint4*>(from + off[k]));
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (i0 + k * kCopyThreads >= total) break;
      __stcs(reinterpret_cast<uint4*>(to + off[k]), x[k]);
    }
    if (part == 0 && p.k_scale != nullptr) {
      float* s = is_v ? p.v_scale : p.k_scale;
      const int64_t* st = is_v ? p.vs : p.ks;
      for (int i = threadIdx.x; i < p.blocks * p.heads; i += kCopyThreads) {
        const int blk = i / p.heads, h = i - blk * p.heads;
        const int64_t at = blk * st[1] + h * st[2];
        s[dst * st[0] + at] = s[src * st[0] + at];
      }
    }
  }
}

}  // namespace

size_t fork_ws(int rows, int max_pages, int num_pages) {
  const int64_t entries = static_cast<int64_t>(rows) * max_pages;
  const int64_t list = entries < num_pages ? entries : num_pages;
  return align256((7 * static_cast<int64_t>(rows) + kCluster + 8 + list + entries) * sizeof(int));
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.rows) * p.max_pages;
  const int64_t list = entries < p.num_pages ? entries : p.num_pages;
  fork_kernel<<<kCluster, kForkThreads, 0, stream>>>(p, fork_layout(p.ws, p.rows, list));
  return cudaGetLastError();
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream) {
  FastDiv run, row;
  run.set(static_cast<uint32_t>(p.chunks));
  row.set(static_cast<uint32_t>(p.rows[1]));
  const int parts = ceil_div(p.rows[0] * p.rows[1] * p.chunks, kCopyThreads * kFlight);
  const int64_t items = static_cast<int64_t>(p.num_pairs) * 2 * parts, most = static_cast<int64_t>(num_sms()) * 8;
  copy_kernel<<<static_cast<unsigned>(items < most ? items : most), kCopyThreads, 0, stream>>>(p, run, row, parts);
  return cudaGetLastError();
}

}  // namespace attn
