// Eviction from the paged cache by accumulated attention weight
// (attn_cache_evict), in two launches.
//
// Selection, one block per (sequence, head): the rank of a slot is a 32-bit key
// that orders as the floats do; four passes of 8 bits with a histogram in shared
// memory find the key of the budget-th largest and how many of its equals stay.
// Each thread then owns a run of neighbouring slots, and block-wide prefix sums
// over the threads turn "kept" into places: the i-th kept slot above the budget
// moves into the i-th freed slot below it.  Sources and targets are disjoint
// ranges of slots, so the moves need no order among each other.
//
// Copy: the listed rows of k and v, 16 bytes a thread.
#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kSelThreads = 1024;

// Unsigned key in the order of the ranks: NaN lowest, then the floats (-0 = +0).
__device__ __forceinline__ uint32_t rank_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kInfKey = 0xFF800000u;  // rank_key(+inf): the rank of a recent slot

// Exclusive prefix sum of v over the block; total in `sum`.
__device__ int block_scan(int v, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, i);
      if (lane >= i) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  sum = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(EvictParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sums[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x;
  const int bh = blockIdx.x, b = bh / p.h_k;
  const int n = p.seqlens[b];
  if (n < 0 || n > p.max_seqlen) {
    if (tid == 0) {
      report(p.status, kBadLength);
      p.count[bh] = 0;
      if (bh == b * p.h_k) p.seqlens_out[b] = 0;
    }
    return;
  }
  const int64_t base = static_cast<int64_t>(bh) * p.stride;
  const float* w = p.w_in + base;
  float* w_out = p.w_out + base;
  const int* pos = p.pos_in != nullptr ? p.pos_in + base : nullptr;
  int* pos_out = p.pos_out != nullptr ? p.pos_out + base : nullptr;
  const int m = min(n, p.budget);
  if (tid == 0 && bh == b * p.h_k) p.seqlens_out[b] = m;
  if (n <= p.budget) {
    if (tid == 0) p.count[bh] = 0;
    for (int j = tid; j < n; j += kSelThreads) {
      if (w_out != w) w_out[j] = w[j];
      if (pos != nullptr && pos_out != pos) pos_out[j] = pos[j];
    }
    return;
  }
  const long long recent_from =
      p.recent > 0 ? static_cast<long long>(p.seen[b]) - p.recent : 0;
  auto key_of = [&](int j) -> uint32_t {
    if (p.recent > 0 && pos[j] >= recent_from) return kInfKey;
    return rank_key(w[j]);
  };

  // ---- key of the budget-th largest
  uint32_t prefix = 0;
  int need = p.budget;  // still to be found among keys that share `prefix`
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int j = tid; j < n; j += kSelThreads) {
      const uint32_t k = key_of(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int left = need, bin = 255;
      for (; bin > 0 && hist[bin] < left; --bin) left -= hist[bin];
      s_prefix = prefix | (static_cast<uint32_t>(bin) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }

  // ---- places: thread t owns slots [j0, j1)
  const int per = (n + kSelThreads - 1) / kSelThreads;
  const int j0 = min(n, tid * per), j1 = min(n, j0 + per);
  int ties = 0;
  for (int j = j0; j < j1; ++j) ties += key_of(j) == prefix ? 1 : 0;
  int sum;
  const int ties_before = block_scan(ties, warp_sums, sum);
  int seen_ties = ties_before, holes = 0, movers = 0;
  for (int j = j0; j < j1; ++j) {
    const uint32_t k = key_of(j);
    const bool keep = k > prefix || (k == prefix && seen_ties++ < need);
    if (j < p.budget) holes += keep ? 0 : 1;
    else movers += keep ? 1 : 0;
  }
  int n_holes, n_movers;
  int hole = block_scan(holes, warp_sums, n_holes);
  int mover = block_scan(movers, warp_sums, n_movers);
  int* from = p.from + static_cast<int64_t>(bh) * p.move_cap;
  int* to = p.to + static_cast<int64_t>(bh) * p.move_cap;
  seen_ties = ties_before;
  for (int j = j0; j < j1; ++j) {
    const uint32_t k = key_of(j);
    const bool keep = k > prefix || (k == prefix && seen_ties++ < need);
    if (j < p.budget) {
      if (!keep) to[hole++] = j;
    } else if (keep) {
      from[mover++] = j;
    }
  }
  if (tid == 0) p.count[bh] = n_movers;
  __syncthreads();

  // ---- state: kept slots stay, moved ones follow, the rest is cleared
  if (w_out != w)
    for (int j = tid; j < p.budget; j += kSelThreads) w_out[j] = w[j];
  if (pos != nullptr && pos_out != pos)
    for (int j = tid; j < p.budget; j += kSelThreads) pos_out[j] = pos[j];
  __syncthreads();
  for (int i = tid; i < n_movers; i += kSelThreads) {
    w_out[to[i]] = w[from[i]];
    if (pos != nullptr) pos_out[to[i]] = pos[from[i]];
  }
  __syncthreads();
  for (int j = p.budget + tid; j < n; j += kSelThreads) {
    w_out[j] = 0.f;
    if (pos != nullptr) pos_out[j] = -1;
  }
}

// Rows of k and v from their old slots into the freed ones.
__global__ void __launch_bounds__(256) move_kernel(EvictParams p, int chunks) {
  const int bh = blockIdx.x, b = bh / p.h_k, h = bh - b * p.h_k;
  const int moves = p.count[bh];
  const int* row = p.cache.table + b * p.cache.table_stride;
  const int* from = p.from + static_cast<int64_t>(bh) * p.move_cap;
  const int* to = p.to + static_cast<int64_t>(bh) * p.move_cap;
  const uint4* k = static_cast<const uint4*>(p.cache.k.ptr);
  const uint4* v = static_cast<const uint4*>(p.cache.v.ptr);
  const int64_t total = static_cast<int64_t>(moves) * chunks;
  for (int64_t u = blockIdx.y * 256 + threadIdx.x; u < total; u += gridDim.y * 256) {
    const int i = static_cast<int>(u / chunks), c = static_cast<int>(u - static_cast<int64_t>(i) * chunks);
    int p0, w0, p1, w1;
    const bool good = page_of(p.cache, row, from[i], p0, w0, p.status) &
                      page_of(p.cache, row, to[i], p1, w1, p.status);
    if (!good) continue;
    const TensorArg &ka = p.cache.k, &va = p.cache.v;
    const uint4 x = k[(p0 * ka.sb + w0 * ka.ss + h * ka.sh) / 8 + c];
    const uint4 y = v[(p0 * va.sb + w0 * va.ss + h * va.sh) / 8 + c];
    const_cast<uint4*>(k)[(p1 * ka.sb + w1 * ka.ss + h * ka.sh) / 8 + c] = x;
    const_cast<uint4*>(v)[(p1 * va.sb + w1 * va.ss + h * va.sh) / 8 + c] = y;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, int dtype, cudaStream_t stream) {
  (void)dtype;  // rows are moved as 16-byte chunks
  const unsigned heads = static_cast<unsigned>(p.batch) * p.h_k;
  select_kernel<<<heads, kSelThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.move_cap == 0) return e;
  const int chunks = p.head_dim / 8;
  const int64_t most = (static_cast<int64_t>(p.move_cap) * chunks + 255) / 256;
  int64_t y = (8 * static_cast<int64_t>(num_sms()) + heads - 1) / heads;
  if (y > most) y = most;
  move_kernel<<<dim3(heads, static_cast<unsigned>(y < 1 ? 1 : y)), 256, 0, stream>>>(p, chunks);
  return cudaGetLastError();
}

}  // namespace attn
