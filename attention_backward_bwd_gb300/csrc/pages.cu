// Pages that sequences share: forking, freeing and room for new tokens (attn_cache_fork), and the
// copy of pages (attn_cache_copy).
//
// attn_cache_fork works on the block table and the pages' counts of references alone, in steps: the
// references that go and come and what each row needs; prefix sums over the rows and the number of
// free pages in each block's part of the pool; the list of the lowest free pages; the new rows.
// Who goes on with which row is worked out by every block for itself, in shared memory.  Which page
// a row gets follows from its place alone, so that the result does not depend on timing.  A row that
// goes on and would write a page that others hold too (the settled references say so) gives up its
// pages from there on; they lose their references in the last step, after the free pages were listed,
// since the copies still read them.  A warp takes kChunk entries of a row.  Small tables and pools are
// one launch of one cluster, whose barrier parts the steps: bound by their chain, each some loads long.
// Large ones (kLarge) take a launch a step, with all of the GPU for the references and the rows (512
// rows of 1001 pages, 770000 entries and pages: 85 us in one cluster, 19 in launches).
// attn_cache_copy moves whole pages, 16 bytes a thread, several in flight: bound by the memory.
#include <atomic>

#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kForkThreads = 512;
constexpr int kForkWarps = kForkThreads / 32;
constexpr int kCluster = 8;    // blocks
constexpr int kEntries = 8;    // of a lane in flight
constexpr int kChunk = 32 * kEntries;
// Rows whose state is kept in shared memory: 12 bytes each, and 8 more for the prefix sums.
constexpr int kRows = 8192;
// Entries and pages from which every step has a launch of its own (the cluster and the launches:
// 6600 10.7 and 12.6 us, 23300 15.4 and 13.0, 132000 26.5 and 14.4).
constexpr int64_t kLarge = 16000;

// Steps of a launch.
enum { kRefs = 1, kList = 2, kWrite = 4, kAllSteps = 7 };

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Workspace of a fork: per row the pages and copies it needs, their prefix sums (the pages' below 0
// where the row gives pages up) and what it holds of pages that it would write (kNoneHeld, one page's
// number, kSomeHeld); beyond kRows rows also the first row that takes it over, its parent and its
// length; per block its free pages; the pages needed and those granted; then the list of free pages and,
// where the table is its own output, the old table.
struct ForkWs {
  int *fresh, *copied, *who, *parent, *len, *fresh_before, *copied_before, *held, *free_of, *sums, *list, *old;
};
enum { kNoneHeld = -1, kSomeHeld = -2 };
__host__ __device__ inline ForkWs fork_layout(int* ws, int64_t rows, int64_t list) {
  ForkWs w;
  w.fresh = ws;
  w.copied = w.fresh + rows;
  w.who = w.copied + rows;
  w.parent = w.who + rows;
  w.len = w.parent + rows;
  w.fresh_before = w.len + rows;
  w.copied_before = w.fresh_before + rows;
  w.held = w.copied_before + rows;
  w.free_of = w.held + rows;
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
  int s = lane < kForkWarps ? warp_sums[lane] : 0;
#pragma unroll
  for (int i = 1; i < kForkWarps; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, i);
    if (lane >= i) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, kForkWarps - 1);
  const int before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  return (warp == 0 ? 0 : before) + x - mine;
}

// What a row of the new table is made of.
struct Row {
  int parent, n;      // -1: none; its length
  int full, used, need;  // entries of full pages, of pages with slots, with the room
  bool heir;          // goes on with its parent's pages
  bool gives;         // but not with those from `full` on, which others hold
};

template <int STEPS>
__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkParams p, ForkWs w, int copy_refs) {
  __shared__ int s_sums[kForkWarps];
  extern __shared__ int s_state[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank()), blocks = static_cast<int>(cluster_blocks());
  const int at = blockIdx.x * kForkThreads + tid, step = gridDim.x * kForkThreads;
  auto sync = [&]() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  const bool in_place = p.table == p.table_out, few = p.rows <= kRows;
  int* const saved_len = w.len;  // from the references' launch to the rows': seqlens may be its own output
  if (STEPS == kRefs || STEPS == kList) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (STEPS == kList || STEPS == kWrite) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (few) {
    w.who = s_state;
    w.parent = w.who + p.rows;
    w.len = w.parent + p.rows;
    if (STEPS == kAllSteps) {
      w.fresh_before = w.len + p.rows;
      w.copied_before = w.fresh_before + p.rows;
    }
  }
  const int64_t cap = static_cast<int64_t>(p.max_pages) * p.page_size;
  auto valid = [&](int page) { return static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages); };

  if (STEPS != kList) {
    // ---- lengths and parents; the first row of each parent goes on with its pages.  Of few rows
    // every block sets all up.
    const bool tell = STEPS & kRefs && (!few || blockIdx.x == 0);
    const int b0 = few ? tid : at, bs = few ? kForkThreads : step;
    for (int b = b0; b < p.rows; b += bs) {
      int n = STEPS == kWrite ? __ldcg(saved_len + b) : p.seqlens[b], s = p.parents == nullptr ? b : p.parents[b];
      if (n < 0 || n > cap) {
        if (tell) report(p.status, kBadLength);
        n = 0;
      }
      if (s >= p.rows) {
        if (tell) report(p.status, kBadParent);
        s = b;
      }
      w.len[b] = n;
      if (STEPS == kRefs && blockIdx.x == 0) saved_len[b] = n;
      w.parent[b] = s;
      w.who[b] = p.rows;
    }
    if (STEPS & kRefs && copy_refs)
      for (int i0 = at; i0 < p.num_pages; i0 += step * kEntries) {
        int x[kEntries];
#pragma unroll
        for (int k = 0; k < kEntries; ++k)
          if (i0 + k * step < p.num_pages) x[k] = p.refs[i0 + k * step];
#pragma unroll
        for (int k = 0; k < kEntries; ++k)
          if (i0 + k * step < p.num_pages) p.refs_out[i0 + k * step] = x[k];
      }
    if (few) __syncthreads();
    else sync();
    for (int b = b0; b < p.rows; b += bs)
      if (w.parent[b] >= 0) atomicMin(w.who + w.parent[b], b);
    // (one launch: the references are where they will be, too)
    if (STEPS == kAllSteps && (copy_refs || !few)) sync();
    else __syncthreads();
  }

  auto shape_of = [&](int b, int parent, int n, bool tell) {
    Row r;
    r.parent = parent;
    r.n = n;
    r.heir = r.gives = false;
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
  auto row_of = [&](int b, bool tell) {
    const int parent = w.parent[b];
    Row r = shape_of(b, parent, parent < 0 ? 0 : w.len[parent], tell);
    r.heir = parent >= 0 && w.who[parent] == b;
    return r;
  };
  // Entry i of a row: its page, whether that is the parent's shared one, one to be copied, missing.
  struct Entry {
    int page;
    bool shared, copied, fresh, bad;
  };
  auto entry_of = [&](const Row& r, int page, int i) {
    Entry e{-1, false, false, false, false};
    if (r.parent < 0 || i >= p.max_pages) return e;
    if (r.heir && (!r.gives || i < r.full)) {
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
  // Where a row's missing entries start (and end: at max(used, need)), and those that it may give up.
  auto lack_from = [&](const Row& r) { return r.heir || p.share ? r.full : 0; };
  // Entries i0 + 32 k + lane below `end`, as they are.
  auto load = [&](const int* row, int i0, int end, int (&page)[kEntries]) {
#pragma unroll
    for (int k = 0; k < kEntries; ++k) {
      const int i = i0 + 32 * k + lane;
      page[k] = i < end ? __ldcg(row + i) : -1;
    }
  };
  // Missing entries and copies of [from, end), by a warp; of an heir also what it holds there.
  auto count = [&](const Row& r, const int* old, int from, int end, int& fresh, int& copied, int& held) {
    fresh = copied = 0;
    int pages = 0, most = kNoneHeld;
    for (int i0 = from; i0 < end; i0 += kChunk) {
      int page[kEntries];
      load(old, i0, end, page);
#pragma unroll
      for (int k = 0; k < kEntries; ++k)
        if (i0 + 32 * k + lane < end) {
          const Entry e = entry_of(r, page[k], i0 + 32 * k + lane);
          fresh += e.fresh;
          copied += e.copied;
          pages += e.page >= 0;
          most = max(most, e.page);
        }
    }
    fresh = __reduce_add_sync(0xffffffffu, fresh);
    copied = __reduce_add_sync(0xffffffffu, copied);
    held = __reduce_add_sync(0xffffffffu, pages) > 1 ? static_cast<int>(kSomeHeld) : __reduce_max_sync(0xffffffffu, most);
  };
  const int chunks = (p.max_pages + kChunk - 1) / kChunk;
  const int64_t items = static_cast<int64_t>(p.rows) * chunks;

  if (STEPS & kRefs) {
    // ---- references that go and come; what each row needs (the table is as it was until the last step)
    for (int64_t item = at >> 5; item < items; item += step >> 5) {
      const int b = static_cast<int>(item / chunks), i0 = static_cast<int>(item - static_cast<int64_t>(b) * chunks) * kChunk;
      const bool left = w.who[b] == p.rows;
      const Row r = row_of(b, lane == 0 && i0 == 0);
      const int* old = p.table + (r.parent < 0 ? b : r.parent) * p.table_stride;
      int own[kEntries], page[kEntries];
      if (left || in_place) load(p.table + b * p.table_stride, i0, p.max_pages, own);
      const int shared = r.heir || !p.share ? 0 : r.full;
      if (i0 < shared) load(old, i0, shared, page);
      if (left || in_place)
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
          const int i = i0 + 32 * k + lane;
          if (in_place && i < p.max_pages) w.old[static_cast<int64_t>(b) * p.max_pages + i] = own[k];
          if (left && valid(own[k])) atomicSub(p.refs_out + own[k], 1);
        }
      if (i0 < shared)
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
          const int i = i0 + 32 * k + lane;
          if (i < shared) {
            if (valid(page[k])) atomicAdd(p.refs_out + page[k], 1);
            else report(p.status, kBadPage);
          }
        }
      if (i0 == 0) {
        int fresh, copied, held;
        count(r, old, lack_from(r), max(r.used, r.need), fresh, copied, held);
        if (lane == 0) {
          w.fresh[b] = fresh;
          w.copied[b] = copied;
          w.held[b] = r.heir ? held : static_cast<int>(kNoneHeld);
          // pages of slots that cannot be copied: what is neither copied nor the room's
          if (r.parent >= 0 && !r.heir && copied < r.used - lack_from(r)) report(p.status, kBadPage);
        }
      }
    }
  }
  if (STEPS == kAllSteps) sync();

  int all = 0, granted = 0;
  if (STEPS & kList) {
    // ---- free pages of each block's part; prefix sums over the rows
    const int page0 = static_cast<int>(static_cast<int64_t>(p.num_pages) * rank / blocks);
    const int page1 = static_cast<int>(static_cast<int64_t>(p.num_pages) * (rank + 1) / blocks);
    const bool here = STEPS == kAllSteps && few;  // the prefix sums are each block's own
    int fresh = 0, copied = 0, held = kNoneHeld;
    auto ask = [&](int b) {
      fresh = b < p.rows ? __ldcg(w.fresh + b) : 0;
      copied = b < p.rows ? __ldcg(w.copied + b) : 0;
      held = b < p.rows ? __ldcg(w.held + b) : static_cast<int>(kNoneHeld);
    };
    if (here || rank == 0) ask(tid);  // (on their way while the counts are read)
    int free_here = 0;
    for (int i0 = page0 + tid; i0 < page1; i0 += kForkThreads * kEntries) {
      int x[kEntries];
#pragma unroll
      for (int k = 0; k < kEntries; ++k) x[k] = i0 + k * kForkThreads < page1 ? __ldcg(p.refs_out + i0 + k * kForkThreads) : 1;
#pragma unroll
      for (int k = 0; k < kEntries; ++k) free_here += x[k] == 0;
    }
    int total, wanted = 0, copied0 = 0;
    if (here || rank == 0) {
      for (int r0 = 0; r0 < p.rows; r0 += kForkThreads) {
        const int b = r0 + tid;
        if (r0 > 0) ask(b);
        bool gives = held >= 0 && __ldcg(p.refs_out + held) > 1;
        if (held != kNoneHeld && (gives || held == kSomeHeld)) {
          int s = p.parents == nullptr ? b : p.parents[b];
          s = s >= p.rows ? b : s;
          const Row r = shape_of(b, s, STEPS == kAllSteps ? w.len[s] : __ldcg(saved_len + s), false);
          const int* old = p.table + s * p.table_stride;
          for (int i = r.full; i < max(r.used, r.need) && !gives; ++i) {
            const int page = __ldcg(old + i);
            gives = valid(page) && __ldcg(p.refs_out + page) > 1;
          }
          if (gives) {  // its partly full page is copied, the room's are new
            copied = r.used > r.full && valid(__ldcg(old + r.full)) ? 1 : 0;
            fresh = copied + max(r.need - r.used, 0);
          }
        }
        const int f = block_prefix(fresh, s_sums, total);
        if (b < p.rows) w.fresh_before[b] = gives ? ~(wanted + f) : wanted + f;
        wanted += total;
        const int c = block_prefix(copied, s_sums, total);
        if (b < p.rows) w.copied_before[b] = copied0 + c;
        copied0 += total;
      }
      if (rank == 0 && tid == 0) w.sums[1] = wanted;
    }
    block_prefix(free_here, s_sums, total);
    if (tid == 0) w.free_of[rank] = total;
    sync();

    // ---- the lowest free pages, as many as are needed
    if (!here) wanted = __ldcg(w.sums + 1);
    int first = 0;
    for (int c = 0; c < blocks; ++c) {
      const int n = __ldcg(w.free_of + c);
      first += c < rank ? n : 0;
      all += n;
    }
    granted = min(wanted, all);
    for (int i0 = page0; i0 < page1 && first < granted; i0 += kForkThreads * 4) {
      int x[4], n, mine = 0;  // four neighbouring pages a thread
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + tid * 4 + k;
        x[k] = i < page1 ? __ldcg(p.refs_out + i) : 1;
        mine += x[k] == 0;
      }
      int k0 = first + block_prefix(mine, s_sums, n);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (x[k] == 0) {
          if (k0 < granted) w.list[k0] = i0 + tid * 4 + k;
          ++k0;
        }
      first += n;
    }
    if (rank == 0 && tid == 0) {
      w.sums[2] = granted;
      p.counts[0] = granted == wanted ? copied0 : 0;  // where pages run out the rows count their copies
      p.counts[1] = all - granted;
    }
  }
  if (STEPS == kAllSteps) sync();

  if (STEPS & kWrite) {
    // ---- the new rows
    if (STEPS == kWrite) granted = __ldcg(w.sums + 2);
    const bool run_out = __ldcg(w.sums + 2) < __ldcg(w.sums + 1);
    for (int64_t item = at >> 5; item < items; item += step >> 5) {
      const int b = static_cast<int>(item / chunks), i0 = static_cast<int>(item - static_cast<int64_t>(b) * chunks) * kChunk;
      Row r = row_of(b, false);
      r.gives = w.fresh_before[b] < 0;
      const int from = r.parent < 0 ? b : r.parent;
      const int* old = in_place ? w.old + static_cast<int64_t>(from) * p.max_pages : p.table + from * p.table_stride;
      int* out = p.table_out + b * p.out_stride;
      int page[kEntries];
      load(old, i0, r.heir ? p.max_pages : r.used, page);  // entries that the parent has a say in
      int fresh0 = r.gives ? ~w.fresh_before[b] : w.fresh_before[b], copied0 = w.copied_before[b], made = 0, freed = 0;
      if (i0 > lack_from(r) && i0 < max(r.used, r.need)) {
        int fresh, copied, held;
        count(r, old, lack_from(r), i0, fresh, copied, held);
        fresh0 += fresh;
        copied0 += copied;
      }
#pragma unroll
      for (int k = 0; k < kEntries; ++k) {
        const int i = i0 + 32 * k + lane;
        if (i - lane >= p.max_pages) break;
        const Entry e = entry_of(r, page[k], i);
        int now = e.page;
        const uint32_t fresh = __ballot_sync(0xffffffffu, e.fresh);
        if (fresh != 0) {
          const uint32_t copied = __ballot_sync(0xffffffffu, e.copied), below = (1u << lane) - 1;
          if (e.fresh) {
            const int nth = fresh0 + __popc(fresh & below);
            now = nth < granted ? __ldcg(w.list + nth) : -1;
            if (now >= 0) p.refs_out[now] = 1;
            else report(p.status, kNoPage);
            if (e.copied && now >= 0) {
              int* pair = p.copies + 2 * static_cast<int64_t>(copied0 + __popc(copied & below));
              pair[0] = e.page;
              pair[1] = now;
              ++made;
            }
          }
          fresh0 += __popc(fresh);
          copied0 += __popc(copied);
        }
        if (i < p.max_pages) {
          out[i] = now;
          if (r.gives && i >= r.full && valid(page[k])) freed += atomicSub(p.refs_out + page[k], 1) == 1;
        }
      }
      made = __reduce_add_sync(0xffffffffu, made);
      if (r.gives) freed = __reduce_add_sync(0xffffffffu, freed);
      if (lane == 0) {
        if (i0 == 0) p.seqlens_out[b] = r.n;
        if (run_out && made > 0) atomicAdd(p.counts, made);
        if (freed > 0) atomicAdd(p.counts + 1, freed);
      }
    }
  }
}

__global__ void __launch_bounds__(kForkThreads) copy_refs_kernel(const int* from, int* to, int n) {
  for (int i = blockIdx.x * kForkThreads + threadIdx.x; i < n; i += gridDim.x * kForkThreads) to[i] = from[i];
}

constexpr int kCopyThreads = 256;
// Copies of more than this are marked to leave the L2 first, with eight 16-byte pieces of a thread in
// flight; less stays there, with four (4000 pages of 128 KB 168 us and, the other way, 185; 48 pages of 256 KB
// 6.3 and 4.4).
constexpr int64_t kPassing = 64 << 20;

// A block takes a part of a page of k or of v, and with a page's first part its factors.
template <int kFlight, bool kPass>
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
      const uint4* at = reinterpret_cast<const uint4*>(from + off[k]);
      x[k] = kPass ? __ldcs(at) : *at;
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (i0 + k * kCopyThreads >= total) break;
      uint4* at = reinterpret_cast<uint4*>(to + off[k]);
      if (kPass) __stcs(at, x[k]);
      else *at = x[k];
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
  return align256((8 * static_cast<int64_t>(rows) + kCluster + 8 + list + entries) * sizeof(int));
}

namespace {

template <int STEPS>
cudaError_t launch_steps(const ForkParams& p, int cluster, int blocks, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.rows) * p.max_pages;
  const int64_t list = entries < p.num_pages ? entries : p.num_pages;
  const size_t smem = STEPS == kList || p.rows > kRows ? 0 : static_cast<size_t>(p.rows) * (STEPS == kAllSteps ? 20 : 12);
  static std::atomic<unsigned long long> done{0};  // devices with the attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit) || bit == 0) {
    e = cudaFuncSetAttribute(fork_kernel<STEPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRows * 20);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attrs[2];
  int n = 0;
  if (cluster > 1) {
    attrs[n].id = cudaLaunchAttributeClusterDimension;
    attrs[n].val.clusterDim.x = cluster;
    attrs[n].val.clusterDim.y = attrs[n].val.clusterDim.z = 1;
    ++n;
  }
  if (STEPS == kList || STEPS == kWrite) {  // launched early, waits for the launch before it
    attrs[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kForkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, fork_kernel<STEPS>, p, fork_layout(p.ws, p.rows, list),
                            STEPS == kAllSteps && p.refs != p.refs_out ? 1 : 0);
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.rows) * p.max_pages;
  if (entries + p.num_pages < kLarge || p.rows > kRows) return launch_steps<kAllSteps>(p, kCluster, kCluster, stream);
  const int64_t items = static_cast<int64_t>(p.rows) * ceil_div(p.max_pages, kChunk);
  const int64_t fit = (items + kForkWarps - 1) / kForkWarps, most = 2 * static_cast<int64_t>(num_sms());
  const int blocks = static_cast<int>(fit < most ? fit : most);
  if (p.refs != p.refs_out)
    copy_refs_kernel<<<static_cast<unsigned>(most), kForkThreads, 0, stream>>>(p.refs, p.refs_out, p.num_pages);
  cudaError_t e = launch_steps<kRefs>(p, 1, blocks, stream);
  if (e == cudaSuccess) e = launch_steps<kList>(p, kCluster, kCluster, stream);
  if (e == cudaSuccess) e = launch_steps<kWrite>(p, 1, blocks, stream);
  return e;
}

cudaError_t launch_copy(const CopyParams& p, cudaStream_t stream) {
  FastDiv run, row;
  run.set(static_cast<uint32_t>(p.chunks));
  row.set(static_cast<uint32_t>(p.rows[1]));
  const int64_t pieces = static_cast<int64_t>(p.rows[0]) * p.rows[1] * p.chunks;
  const bool pass = pieces > kPassing / 64 / p.num_pairs;  // k and v, read and written
  const int flight = pass ? 8 : 4, parts = static_cast<int>((pieces + kCopyThreads * flight - 1) / (kCopyThreads * flight));
  const int64_t items = static_cast<int64_t>(p.num_pairs) * 2 * parts, most = static_cast<int64_t>(num_sms()) * 8;
  const unsigned grid = static_cast<unsigned>(items < most ? items : most);
  if (pass) copy_kernel<8, true><<<grid, kCopyThreads, 0, stream>>>(p, run, row, parts);
  else copy_kernel<4, false><<<grid, kCopyThreads, 0, stream>>>(p, run, row, parts);
  return cudaGetLastError();
}

}  // namespace attn
