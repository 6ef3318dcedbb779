// Eviction from the paged cache by accumulated attention weight
// (attn_cache_evict), in one launch.
//
// A cluster of blocks takes one (sequence, head); every block owns a run of its slots,
// every warp a run of the block's.  Selection: the rank of a slot is a 32-bit key that
// orders as the floats do, kept in shared memory.  Up to four passes over its 8-bit digits
// find the key of the budget-th largest and how many of its equals stay: each block
// counts digits, and all blocks of the cluster read each other's counts (one bin a thread;
// with three passes of 2048 bins those reads took 200 us).
// Places: ballots along each warp's run, and sums over the warps and blocks before it,
// turn "kept" into indices; the i-th kept slot at or above the budget moves into the i-th
// freed slot below it.  Sources and targets are disjoint ranges of slots, so the moves
// need no order.  Then the cluster's threads move state and rows, 16 bytes a thread.
//
// The bytes are few (n weights and positions a head, and the rows that move); what
// bounds short heads is the chain of dependent steps.  Of 18.6 us for 1024 heads of 1025 to
// 1088 slots cut to 1024, the launch and the keys take 6.2, the selection 2.7, the places
// 3.4, the moves 6 (34 MB in all, 5.1 us at the memory's speed); of 23 us for 32 heads of
// 5000 to 16000 slots 4.8, 5.5, 3.4 and 8.  Heads that move much are bound by the moves: 1024
// heads of 8192 slots cut to 4096 take 334 us for 1.3 GB, 57 % of the copy bandwidth, since rows
// of 128 bytes lie in any order and each thread goes from the lists to the table to its rows.
// The loops are short: a form with the keys in registers and every loop unrolled spent 52 %
// of its warps' time fetching instructions.
#include <cooperative_groups.h>

#include "cache.h"
#include "common.cuh"

namespace cg = cooperative_groups;

namespace attn {

namespace {

constexpr int kBins = 256;
// keys of a block in shared memory; further ones are worked out again
template <int T>
constexpr int kCap = T == 512 ? 8192 : 4096;
constexpr int kMaxCluster = 8;
constexpr int kLeast = 1024;  // slots of a block where a head of the greatest length has several

// Unsigned key in the order of the ranks: NaN lowest, then the floats (-0 = +0).
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kInfKey = 0xFF800000u;  // rank_key(+inf): the rank of a recent slot

// kSpread: a head has several blocks.  (One form for both made single blocks 2 us slower.)
template <int T, bool kSpread>
__global__ void __launch_bounds__(T, T == 128 ? 7 : 1024 / T)
    evict_kernel(EvictParams p, int blocks_log2, FastDiv chunks) {
  constexpr int W = T / 32;
  constexpr int kOwn = T < kBins ? kBins / T : 1;  // bins of a thread
  constexpr int kSums = kBins / kOwn / 32;         // warps that have some
  __shared__ uint32_t s_key[kCap<T>];
  __shared__ int hist[4][kBins];
  __shared__ int s_sums[kSums];
  __shared__ int2 s_warp[W];        // counts of each warp's run: ties; or holes and movers
  __shared__ int2 s_tot[2];         // the block's, read by the cluster
  __shared__ int s_digit, s_left, s_equal;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = kSpread ? blockIdx.x >> blocks_log2 : blockIdx.x;
  const int rank = kSpread ? blockIdx.x & ((1 << blocks_log2) - 1) : 0;
  const int b = bh / p.h_k, h = bh - b * p.h_k;
  const int n = p.seqlens[b];
  if (n < 0 || n > p.max_seqlen) {
    if (tid == 0 && rank == 0) {
      report(p.status, kBadLength);
      if (h == 0) p.seqlens_out[b] = 0;
    }
    return;
  }
  // The launch knows the bound of the lengths alone: of a shorter sequence's blocks as many
  // leave as would have less than 512 slots (the cluster's barrier does not wait for them):
  // 1024 heads of 1088 slots with a bound of 32768 take 39 us, 118 with all blocks at work.
  int cs_log2 = kSpread ? blocks_log2 : 0;
  while (cs_log2 > 0 && n >> cs_log2 < kLeast / 2) --cs_log2;
  const int cs = kSpread ? 1 << cs_log2 : 1;
  if (rank >= cs) return;
  auto sync_all = [&]() {  // the blocks of this head
    if (cs == 1) __syncthreads(); else cluster.sync();
  };
  const int64_t base = static_cast<int64_t>(bh) * p.stride;
  const float* w = p.w_in + base;
  float* w_out = p.w_out + base;
  const int* pos = p.pos_in != nullptr ? p.pos_in + base : nullptr;
  int* pos_out = p.pos_out != nullptr ? p.pos_out + base : nullptr;
  const bool copy_w = w_out != w, copy_pos = pos != nullptr && pos_out != pos;
  if (tid == 0 && rank == 0 && h == 0) p.seqlens_out[b] = min(n, p.budget);
  if (n <= p.budget) {
    for (int j = rank * T + tid; j < n; j += cs * T) {
      if (copy_w) w_out[j] = w[j];
      if (copy_pos) pos_out[j] = pos[j];
    }
    return;
  }

  // ---- runs: the block's slots are [first, last), the warp's [from_slot, to_slot)
  const int per = (n + cs - 1) >> cs_log2;
  const int first = min(n, rank * per), last = min(n, first + per);
  const int run = ((last - first + W - 1) / W + 31) & ~31;
  const int from_slot = min(last, first + warp * run), to_slot = min(last, from_slot + run);
  const long long recent_from = p.recent > 0 ? static_cast<long long>(p.seen[b]) - p.recent : 0;
  for (int i = tid; i < 4 * kBins; i += T) (&hist[0][0])[i] = 0;
  __syncthreads();

  // ---- keys, with the first digit's counts.  State that goes to other arrays is copied
  // at once: slots below the budget as they are (a freed one gets its new tenant's later),
  // cleared ones above it.
#pragma unroll 4
  for (int j = from_slot + lane; j < to_slot; j += 32) {
    const float x = w[j];
    const int q = pos != nullptr ? pos[j] : 0;
    const uint32_t k = p.recent > 0 && q >= recent_from ? kInfKey : rank_key(x);
    if (j - first < kCap<T>) s_key[j - first] = k;
    atomicAdd(&hist[0][k >> 24], 1);
    if (copy_w) w_out[j] = j < p.budget ? x : 0.f;
    if (copy_pos) pos_out[j] = j < p.budget ? q : -1;
  }
  auto key = [&](int j) -> uint32_t {
    if (j - first < kCap<T>) return s_key[j - first];
    return p.recent > 0 && pos[j] >= recent_from ? kInfKey : rank_key(w[j]);
  };

  // ---- key of the budget-th largest, digit by digit
  uint32_t prefix = 0;
  int need = p.budget, equal = 0;  // still to be found among the `equal` keys that share `prefix`
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    if (pass > 0)
#pragma unroll 2
      for (int j = from_slot + lane; j < to_slot; j += 32) {
        const uint32_t k = key(j);
        if (((k ^ prefix) >> (shift + 8)) == 0) atomicAdd(&hist[pass][(k >> shift) & 255u], 1);
      }
    sync_all();
    // a thread kOwn bins, the highest first
    int bins[kOwn], mine = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) bins[i] = 0;
    if (tid < kBins / kOwn) {
      const int at = kBins - kOwn * (tid + 1);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < cs) {
          const int* from = cs == 1 ? &hist[pass][at] : cluster.map_shared_rank(&hist[pass][at], r);
#pragma unroll
          for (int i = 0; i < kOwn; ++i) bins[i] += from[kOwn - 1 - i];
        }
#pragma unroll
      for (int i = 0; i < kOwn; ++i) mine += bins[i];
    }
    int x = mine;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, i);
      if (lane >= i) x += y;
    }
    if (lane == 31 && warp < kSums) s_sums[warp] = x;
    __syncthreads();
    int above = x - mine;
#pragma unroll
    for (int v = 0; v < kSums - 1; ++v) above += v < warp ? s_sums[v] : 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (above < need && above + bins[i] >= need) {
        s_digit = kBins - 1 - kOwn * tid - i;
        s_left = need - above;
        s_equal = bins[i];
      }
      above += bins[i];
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_left;
    equal = s_equal;
    if (equal == need) break;  // all of them stay, whatever their further digits
  }
  // Kept: the keys from `prefix` on, if all of its equals stay; else the first `need` of
  // those, in slot order.
  const bool all_ties = equal == need;
  const uint32_t below = (1u << lane) - 1;
  // Counts of the warps before this one in the cluster; `all`: of every warp.
  auto before = [&](int2 mine, int which, int2& all) {
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int2 sum = make_int2(0, 0), block = make_int2(0, 0);
#pragma unroll
    for (int v = 0; v < W; ++v) {
      const int2 c = s_warp[v];
      if (v < warp) {
        sum.x += c.x;
        sum.y += c.y;
      }
      block.x += c.x;
      block.y += c.y;
    }
    if (tid == 0) s_tot[which] = block;
    sync_all();
    all = make_int2(0, 0);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      int2 c = make_int2(0, 0);
      if (r < cs) c = cs == 1 ? s_tot[which] : *cluster.map_shared_rank(&s_tot[which], r);
      if (r < rank) {
        sum.x += c.x;
        sum.y += c.y;
      }
      all.x += c.x;
      all.y += c.y;
    }
    return sum;
  };
  int2 all;
  int ties0 = 0;
  if (!all_ties) {
    int mine = 0;
#pragma unroll 1
    for (int j0 = from_slot; j0 < to_slot; j0 += 32)
      mine += __popc(__ballot_sync(0xffffffffu, j0 + lane < to_slot && key(j0 + lane) == prefix));
    ties0 = before(make_int2(mine, 0), 0, all).x;
  }
  // Whether slot j of the warp's 32 from j0 on stays; `ties`: equal keys before them.
  auto stays = [&](int j, int& ties) {
    const bool in = j < to_slot;
    const uint32_t k = in ? key(j) : 0u;
    if (all_ties) return in && k >= prefix;
    const bool tie = in && k == prefix;
    const uint32_t t = __ballot_sync(0xffffffffu, tie);
    const bool keep = in && (k > prefix || (tie && ties + __popc(t & below) < need));
    ties += __popc(t);
    return keep;
  };

  // ---- freed slots below the budget (holes) and kept ones above it (movers)
  int holes = 0, movers = 0, ties = ties0;
#pragma unroll 1
  for (int j0 = from_slot; j0 < to_slot; j0 += 32) {
    const int j = j0 + lane;
    const bool keep = stays(j, ties);
    holes += __popc(__ballot_sync(0xffffffffu, j < to_slot && j < p.budget && !keep));
    movers += __popc(__ballot_sync(0xffffffffu, j >= p.budget && keep));
  }
  const int2 start = before(make_int2(holes, movers), 1, all);
  const int moves = all.y;  // as many as there are holes
  int* from = p.from + static_cast<int64_t>(bh) * p.move_cap;
  int* to = p.to + static_cast<int64_t>(bh) * p.move_cap;
  holes = start.x;
  movers = start.y;
  ties = ties0;
#pragma unroll 1
  for (int j0 = from_slot; j0 < to_slot; j0 += 32) {
    const int j = j0 + lane;
    const bool keep = stays(j, ties);
    const bool hole = j < to_slot && j < p.budget && !keep, mover = j >= p.budget && keep;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, mover);
    if (hole) to[holes + __popc(hb & below)] = j;
    if (mover) from[movers + __popc(mb & below)] = j;
    holes += __popc(hb);
    movers += __popc(mb);
    if (j < to_slot && j >= p.budget && !keep) {
      if (!copy_w) w_out[j] = 0.f;
      if (pos != nullptr && !copy_pos) pos_out[j] = -1;
    }
  }
  sync_all();  // the lists are complete

  // ---- moves: state, then rows, a thread the same chunk of k and of v
#pragma unroll 1
  for (int i = rank * T + tid; i < moves; i += cs * T) {
    const int s = from[i], t = to[i];
    const float x = w[s];
    w_out[t] = x;
    w_out[s] = 0.f;
    if (pos != nullptr) {
      const int q = pos[s];
      pos_out[t] = q;
      pos_out[s] = -1;
    }
  }
  // strides in 16-byte units: a page's offset is one 32 x 32 bit product
  const uint32_t kpage = static_cast<uint32_t>(p.cache.k.sb / 8), kslot = static_cast<uint32_t>(p.cache.k.ss / 8);
  const uint32_t vpage = static_cast<uint32_t>(p.cache.v.sb / 8), vslot = static_cast<uint32_t>(p.cache.v.ss / 8);
  uint4* kp = static_cast<uint4*>(const_cast<void*>(p.cache.k.ptr)) + h * (p.cache.k.sh / 8);
  uint4* vp = static_cast<uint4*>(const_cast<void*>(p.cache.v.ptr)) + h * (p.cache.v.sh / 8);
  const int* row = p.cache.table + b * p.cache.table_stride;
  const int64_t units = static_cast<int64_t>(moves) * chunks.d, stride = static_cast<int64_t>(cs) * T;
  constexpr int kUnroll = 2;  // chunks in flight of a thread, of k and of v each
#pragma unroll 1
  for (int64_t u0 = rank * T + tid; u0 < units; u0 += kUnroll * stride) {
    uint4 x[kUnroll], y[kUnroll];
    uint64_t kto[kUnroll], vto[kUnroll];
    bool good[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t u = u0 + k * stride;
      good[k] = u < units;
      if (!good[k]) continue;
      const int i = units <= INT32_MAX ? static_cast<int>(chunks.div(static_cast<uint32_t>(u)))
                                       : static_cast<int>(u / chunks.d);
      const uint32_t c = static_cast<uint32_t>(u - static_cast<int64_t>(i) * chunks.d);
      const int s = from[i], t = to[i];
      int sp, sw, tp, tw;
      good[k] = page_of(p.cache, row, s, sp, sw, p.status) & page_of(p.cache, row, t, tp, tw, p.status);
      if (!good[k]) continue;
      auto at = [](int page, uint32_t ps, int within, uint32_t ss) {
        return static_cast<uint64_t>(static_cast<uint32_t>(page)) * ps +
               static_cast<uint64_t>(static_cast<uint32_t>(within)) * ss;
      };
      x[k] = kp[at(sp, kpage, sw, kslot) + c];
      y[k] = vp[at(sp, vpage, sw, vslot) + c];
      kto[k] = at(tp, kpage, tw, kslot) + c;
      vto[k] = at(tp, vpage, tw, vslot) + c;
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (good[k]) {
        kp[kto[k]] = x[k];
        vp[vto[k]] = y[k];
      }
  }
}

template <int T>
cudaError_t launch_t(const EvictParams& p, int cs_log2, cudaStream_t stream) {
  FastDiv chunks;
  chunks.set(static_cast<uint32_t>(p.head_dim / 8));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((static_cast<unsigned>(p.batch) * p.h_k) << cs_log2);
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1u << cs_log2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = cs_log2 > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, cs_log2 > 0 ? evict_kernel<T, true> : evict_kernel<T, false>, p, cs_log2,
                            chunks);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int dtype, cudaStream_t stream) {
  (void)dtype;  // rows are moved as 16-byte chunks
  const int64_t heads = static_cast<int64_t>(p.batch) * p.h_k;
  if (heads * kMaxCluster > INT32_MAX) return cudaErrorInvalidValue;
  // Blocks of a head: as many as keep its keys in shared memory (320 heads of 16000 slots:
  // 457 us with one block, 133 with four), then while all blocks fit the device at once and
  // each has 1024 slots (32 heads of 8192: 32 us with two, 21 with eight; of 1088: 10.0 with
  // one, 11.6 with two).
  const int64_t sms = num_sms();
  int log2 = 0;
  while ((1 << log2) < kMaxCluster &&
         (p.max_seqlen >> log2 > kCap<128> ||
          (heads << (log2 + 1) <= 4 * sms && p.max_seqlen >> (log2 + 1) >= kLeast)))
    ++log2;
  // Threads of a block: most where there are few blocks; fewer where there are many, which
  // then pass their barriers side by side (1024 heads of 1088 slots: 34 us with 512, 26 with
  // 256, 23 with 128; 400 heads: 14.0, 10.6, 13.0; 160 heads of 8192, two blocks each: 57,
  // 49, 75).  Where there are many blocks of many slots the three come close, and 128 is not
  // always the least: 1024 heads of 4000 133, 137, 136; of 8192, two blocks each, 357, 337,
  // 336; but 320 heads of 16000, four blocks each, 125, 115, 131.
  const int64_t blocks = heads << log2;
  if (blocks <= 2 * sms || p.max_seqlen >> log2 > kCap<256>) return launch_t<512>(p, log2, stream);
  if (blocks <= 4 * sms) return launch_t<256>(p, log2, stream);
  return launch_t<128>(p, log2, stream);
}

}  // namespace attn
