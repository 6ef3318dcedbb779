// Eviction from the paged cache by accumulated attention weight
// (attn_cache_evict), in one launch.
//
// A cluster of blocks takes one (sequence, head); every block owns a run of its slots.
// Selection: the rank of a slot is a 32-bit key that orders as the floats do.  Four
// passes over its 8-bit digits find the key of the budget-th largest and how many of its
// equals stay: each block counts digits in its shared memory, and all blocks of the
// cluster read each other's counts (one bin a thread; with three passes of 2048 bins those
// reads took 200 us).  Up to 8 keys a thread stay in
// registers; further ones are read again from the L2 in each pass.
// Places: warp ballots and prefix sums over them, in slot order, turn "kept" into indices;
// the i-th kept slot at or above the budget moves into the i-th freed slot below it.
// Sources and targets are disjoint ranges of slots, so the moves need no order.
// Copy: the cluster's threads move state and rows of k and v, 16 bytes a thread.
//
// The bytes are few (n weights and positions a head, and the rows that move); what
// bounds it is the chain of passes, so a head is spread over up to eight blocks while the
// device has room for them.
#include <cooperative_groups.h>

#include "cache.h"
#include "common.cuh"

namespace cg = cooperative_groups;

namespace attn {

namespace {

constexpr int kBins = 256;
constexpr int kKeep = 8;  // keys of a thread in registers
constexpr int kMaxCluster = 8;

// Unsigned key in the order of the ranks: NaN lowest, then the floats (-0 = +0).
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kInfKey = 0xFF800000u;  // rank_key(+inf): the rank of a recent slot

struct Totals {
  int ties, holes, movers;
};

template <int T>
__global__ void __launch_bounds__(T) evict_kernel(EvictParams p, int cs, FastDiv per_move) {
  constexpr int W = T / 32;
  __shared__ int hist[4][kBins];
  __shared__ int s_sums[W];
  __shared__ int s_cnt[kKeep * W];   // of a batch: per round and warp, then their prefixes
  __shared__ int s_cnt2[kKeep * W];
  __shared__ int s_digit, s_left, s_equal;
  __shared__ Totals s_tot;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x / cs, rank = blockIdx.x - bh * cs;
  const int b = bh / p.h_k, h = bh - b * p.h_k;
  const int n = p.seqlens[b];
  if (n < 0 || n > p.max_seqlen) {
    if (tid == 0 && rank == 0) {
      report(p.status, kBadLength);
      if (h == 0) p.seqlens_out[b] = 0;
    }
    return;
  }
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

  // ---- keys: this block's slots are [first, last), round i of a batch T of them
  const int per = ((n + cs - 1) / cs + T - 1) / T * T;
  const int first = min(n, rank * per), last = min(n, first + per);
  const int batches = (last - first + kKeep * T - 1) / (kKeep * T);
  const long long recent_from = p.recent > 0 ? static_cast<long long>(p.seen[b]) - p.recent : 0;
  auto slot = [&](int batch, int i) { return first + (batch * kKeep + i) * T + tid; };
  auto load = [&](int batch, uint32_t (&key)[kKeep]) {
    float x[kKeep];
    int q[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int j = slot(batch, i);
      x[i] = j < last ? w[j] : 0.f;
      q[i] = p.recent > 0 && j < last ? pos[j] : 0;
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) key[i] = p.recent > 0 && q[i] >= recent_from ? kInfKey : rank_key(x[i]);
  };
  for (int i = tid; i < 4 * kBins; i += T) (&hist[0][0])[i] = 0;
  if (tid == 0) s_tot = Totals{0, 0, 0};
  uint32_t key[kKeep];
  load(0, key);
  __syncthreads();

  // ---- key of the budget-th largest, digit by digit
  uint32_t prefix = 0;
  int need = p.budget, equal = 0;  // still to be found among the `equal` keys that share `prefix`
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    const uint32_t mask = pass == 0 ? 0u : ~0u << (shift + 8);
    for (int bt = 0; bt < batches; ++bt) {
      if (bt > 0) load(bt, key);
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (slot(bt, i) < last && (key[i] & mask) == prefix)
          atomicAdd(&hist[pass][(key[i] >> shift) & 255u], 1);
    }
    if (batches > 1) load(0, key);
    cluster.sync();
    // thread t: bin 255 - t, the highest first
    int mine = 0;
    if (tid < kBins)
      for (int r = 0; r < cs; ++r) mine += cluster.map_shared_rank(&hist[pass][0], r)[kBins - 1 - tid];
    int x = mine;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, i);
      if (lane >= i) x += y;
    }
    if (lane == 31) s_sums[warp] = x;
    __syncthreads();
    int above = x - mine;
#pragma unroll
    for (int v = 0; v < kBins / 32 - 1; ++v) above += v < warp ? s_sums[v] : 0;
    if (above < need && above + mine >= need) {
      s_digit = kBins - 1 - tid;
      s_left = need - above;
      s_equal = mine;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_digit) << shift;
    need = s_left;
    equal = s_equal;
  }

  // Exclusive prefixes of the counts of a batch, in slot order (round by round, warp by
  // warp); returns the batch's total.  Starts and ends with a barrier.
  auto scan_counts = [&](int* cnt) -> int {
    __syncthreads();
    if (warp == 0) {
      constexpr int kPer = kKeep * W / 32;
      int v[kPer], sum = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        v[i] = cnt[lane * kPer + i];
        sum += v[i];
      }
      int x = sum;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, i);
        if (lane >= i) x += y;
      }
      int at = x - sum;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        cnt[lane * kPer + i] = at;
        at += v[i];
      }
      if (lane == 31) s_sums[0] = x;
    }
    __syncthreads();
    const int total = s_sums[0];
    return total;
  };
  // The block totals of the blocks before this one, and of all.
  auto exchange = [&](Totals& all) {
    cluster.sync();
    Totals before{0, 0, 0};
    all = Totals{0, 0, 0};
    for (int r = 0; r < cs; ++r) {
      const Totals t = *cluster.map_shared_rank(&s_tot, r);
      if (r < rank) {
        before.ties += t.ties;
        before.holes += t.holes;
        before.movers += t.movers;
      }
      all.ties += t.ties;
      all.holes += t.holes;
      all.movers += t.movers;
    }
    return before;
  };
  const uint32_t below = (1u << lane) - 1;

  // ---- which of the equal keys stay: the lower slots
  const bool all_ties = equal == need;
  Totals all;
  int tie_base = 0;
  if (!all_ties) {
    int mine = 0;
    for (int bt = 0; bt < batches; ++bt) {
      if (bt > 0) load(bt, key);
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        mine += __popc(__ballot_sync(0xffffffffu, slot(bt, i) < last && key[i] == prefix));
    }
    if (batches > 1) load(0, key);
    if (lane == 0) atomicAdd(&s_tot.ties, mine);
    tie_base = exchange(all).ties;
  }
  // Bit i: the batch's key i stays.  `ties`: equal keys before the batch; advanced.
  auto kept = [&](int bt, int& ties) -> uint32_t {
    uint32_t keep = 0;
    if (all_ties) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i) keep |= (slot(bt, i) < last && key[i] >= prefix ? 1u : 0u) << i;
      return keep;
    }
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const uint32_t t = __ballot_sync(0xffffffffu, slot(bt, i) < last && key[i] == prefix);
      if (lane == 0) s_cnt[i * W + warp] = __popc(t);
    }
    const int total = scan_counts(s_cnt);
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const bool in = slot(bt, i) < last, tie = in && key[i] == prefix;
      const uint32_t t = __ballot_sync(0xffffffffu, tie);
      const int place = ties + s_cnt[i * W + warp] + __popc(t & below);
      keep |= ((in && key[i] > prefix) || (tie && place < need) ? 1u : 0u) << i;
    }
    __syncthreads();
    ties += total;
    return keep;
  };

  // ---- freed slots below the budget and kept ones above it, over the blocks
  {
    int holes = 0, movers = 0, ties = tie_base;
    for (int bt = 0; bt < batches; ++bt) {
      if (bt > 0) load(bt, key);
      const uint32_t keep = kept(bt, ties);
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int j = slot(bt, i);
        const bool k = (keep >> i) & 1u;
        holes += __popc(__ballot_sync(0xffffffffu, j < last && j < p.budget && !k));
        movers += __popc(__ballot_sync(0xffffffffu, j < last && j >= p.budget && k));
      }
    }
    if (batches > 1) load(0, key);
    if (lane == 0) {
      atomicAdd(&s_tot.holes, holes);
      atomicAdd(&s_tot.movers, movers);
    }
  }
  const Totals before = exchange(all);
  const int moves = all.movers;  // as many as there are holes
  int2* from = p.from + static_cast<int64_t>(bh) * p.move_cap;
  int2* to = p.to + static_cast<int64_t>(bh) * p.move_cap;
  const int* row = p.cache.table + b * p.cache.table_stride;
  auto place = [&](int j) {  // slot and its page, -1 for a bad one
    const int page = row[p.cache.page.div(static_cast<uint32_t>(j))];
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.cache.num_pages)) return make_int2(j, page);
    report(p.status, kBadPage);
    return make_int2(j, -1);
  };
  {
    int hole = before.holes, mover = before.movers, ties = tie_base;
    for (int bt = 0; bt < batches; ++bt) {
      if (bt > 0) load(bt, key);
      const uint32_t keep = kept(bt, ties);
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int j = slot(bt, i);
        const bool k = (keep >> i) & 1u;
        const uint32_t hb = __ballot_sync(0xffffffffu, j < last && j < p.budget && !k);
        const uint32_t mb = __ballot_sync(0xffffffffu, j < last && j >= p.budget && k);
        if (lane == 0) {
          s_cnt[i * W + warp] = __popc(hb);
          s_cnt2[i * W + warp] = __popc(mb);
        }
      }
      const int all_holes = scan_counts(s_cnt), all_movers = scan_counts(s_cnt2);
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int j = slot(bt, i);
        const bool k = (keep >> i) & 1u;
        const bool is_hole = j < last && j < p.budget && !k, is_mover = j < last && j >= p.budget && k;
        const uint32_t hb = __ballot_sync(0xffffffffu, is_hole), mb = __ballot_sync(0xffffffffu, is_mover);
        if (is_hole) to[hole + s_cnt[i * W + warp] + __popc(hb & below)] = place(j);
        if (is_mover) from[mover + s_cnt2[i * W + warp] + __popc(mb & below)] = place(j);
        // state of slots that stay, and of those that go
        if (j < last && j < p.budget && k) {
          if (copy_w) w_out[j] = w[j];
          if (copy_pos) pos_out[j] = pos[j];
        } else if (j < last && j >= p.budget && !k) {
          w_out[j] = 0.f;
          if (pos != nullptr) pos_out[j] = -1;
        }
      }
      __syncthreads();
      hole += all_holes;
      mover += all_movers;
    }
  }
  cluster.sync();  // the lists are complete

  // ---- moves: state, then rows: unit c of a move is a chunk of k, then of v
  for (int i = rank * T + tid; i < moves; i += cs * T) {
    const int s = from[i].x, t = to[i].x;
    const float x = w[s];
    w_out[t] = x;
    w_out[s] = 0.f;
    if (pos != nullptr) {
      const int y = pos[s];
      pos_out[t] = y;
      pos_out[s] = -1;
    }
  }
  const int chunks = p.head_dim / 8;
  uint4* kp = static_cast<uint4*>(const_cast<void*>(p.cache.k.ptr));
  uint4* vp = static_cast<uint4*>(const_cast<void*>(p.cache.v.ptr));
  const int64_t units = static_cast<int64_t>(moves) * per_move.d, stride = static_cast<int64_t>(cs) * T;
  auto address = [&](int2 at, int c) -> uint4* {  // nullptr for a bad page
    if (at.y < 0) return nullptr;
    const int within = at.x - static_cast<int>(p.cache.page.div(static_cast<uint32_t>(at.x)) * p.cache.page.d);
    const TensorArg& t = c < chunks ? p.cache.k : p.cache.v;
    return (c < chunks ? kp + c : vp + (c - chunks)) + (at.y * t.sb + within * t.ss + h * t.sh) / 8;
  };
  constexpr int kUnroll = 4;  // units in flight of a thread
  for (int64_t u0 = rank * T + tid; u0 < units; u0 += kUnroll * stride) {
    uint4* src[kUnroll];
    uint4* dst[kUnroll];
    uint4 x[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int64_t u = u0 + k * stride;
      src[k] = dst[k] = nullptr;
      if (u < units) {
        const int i = units <= INT32_MAX ? static_cast<int>(per_move.div(static_cast<uint32_t>(u)))
                                         : static_cast<int>(u / per_move.d);
        const int c = static_cast<int>(u - static_cast<int64_t>(i) * per_move.d);
        src[k] = address(from[i], c);
        dst[k] = address(to[i], c);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (src[k] != nullptr && dst[k] != nullptr) x[k] = *src[k];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (src[k] != nullptr && dst[k] != nullptr) *dst[k] = x[k];
  }
}

template <int T>
cudaError_t launch_t(const EvictParams& p, int cs, cudaStream_t stream) {
  FastDiv per_move;
  per_move.set(static_cast<uint32_t>(p.head_dim / 8 * 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * p.h_k * cs);
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_kernel<T>, p, cs, per_move);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int dtype, cudaStream_t stream) {
  (void)dtype;  // rows are moved as 16-byte chunks
  const int64_t heads = static_cast<int64_t>(p.batch) * p.h_k;
  if (heads * kMaxCluster > INT32_MAX) return cudaErrorInvalidValue;
  // blocks of a head: while all of them fit the device at once and each has 512 slots
  int cs = 1;
  while (cs < kMaxCluster && heads * cs * 2 <= 4 * static_cast<int64_t>(num_sms()) &&
         p.max_seqlen / (cs * 2) >= 512)
    cs *= 2;
  return ceil_div(p.max_seqlen, cs) <= 256 * kKeep ? launch_t<256>(p, cs, stream)
                                                   : launch_t<1024>(p, cs, stream);
}

}  // namespace attn
