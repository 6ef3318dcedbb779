// What the single-token attention kernels share: the line of key tiles and where it is cut,
// the rows without keys, the partials of cut segments, and small copies and loads.
#pragma once

#include "cache.h"
#include "common.cuh"

namespace attn {

constexpr int kMaxRows = 16;    // query heads of a block
constexpr int kLens = 256;      // lengths kept in shared memory
// Runs at most: sizes the partials without asking a device.
constexpr int kMaxRuns = 320;
// Up to this length, and while the blocks suffice, sequences are taken whole (5.5 us against
// 6.9 for one of 128 keys; but 2048 segments of 63 to 256 keys 39.7 us against 31.5).
constexpr int kWholeKeys = 256;

// Columns that the kernels of a head dimension work on.
inline int pad_dim(int d) { return d <= 64 ? 64 : (d <= 96 ? 96 : (d <= 128 ? 128 : (d <= 192 ? 192 : 256))); }

// Of a tile of the line: it begins / ends a segment of this run, which is a whole one; it is of
// the run's second segment; there is no tile.
enum { kBegin = 1, kEnd = 2, kFull = 4, kSecond = 8, kNone = 16 };

// Keys that sequence length n leaves to attend: [first, n).
__device__ __forceinline__ int first_key(const DecodeParams& p, int n) {
  return p.win_left >= 0 ? max(0, n - 1 - p.win_left) : 0;
}
__device__ __forceinline__ int clean_len(const DecodeParams& p, int n, bool tell) {
  if (n >= 0 && n <= p.max_seqlen) return n;
  if (tell) report(p.status, kBadLength);
  return 0;
}
__device__ __forceinline__ int tiles_of(const DecodeParams& p, int n) {
  return (n - first_key(p, n) + (1 << p.tile_log2) - 1) >> p.tile_log2;
}

// Where a line of tiles is cut.  Run i of `runs` is [i * total / runs, (i + 1) * total / runs).
struct Cut {
  long long total;
  int runs;
  __device__ __forceinline__ long long start(int i) const { return total * i / runs; }
  __device__ __forceinline__ int run_of(long long tile) const {
    return static_cast<int>(((tile + 1) * runs - 1) / total);
  }
};

// Block-wide exclusive prefix of the tiles of the sequences: every thread owns `per`
// neighbouring ones.  Returns this thread's prefix.  Ends with a barrier.  (The launch
// checks that the sum stays below 2^31.)
template <int N>
__device__ __forceinline__ int scan_tiles(const DecodeParams& p, bool tell, int* lens,
                                          int* warp_sums, int per, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b >= p.batch) break;
    const int n = clean_len(p, p.seqlens[b], tell);
    if (lens != nullptr && b < kLens) lens[b] = n;
    mine += tiles_of(p, n);
  }
  int x = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < N / 32; ++w) {
    before += w < warp ? warp_sums[w] : 0;
    total += warp_sums[w];
  }
  return before + x - mine;
}

// (Without an L2 cache policy: three variants of these kernels whose copies had one, all gone, ended
// with an illegal instruction.  What caused it was not found.)
__device__ __forceinline__ void cp_async16(uint32_t dst, long long src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or 16 zeros.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, long long src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Partial of a block (of its run's first or second cut segment): rows of O, then maxima
// and sums.
__device__ __forceinline__ float* partial(const DecodeParams& p, int block, int second) {
  return p.parts + (static_cast<int64_t>(block) * 2 + second) * p.part_stride;
}

// The sequence that tile `r0` of the line lies in, and the tiles (of one head) before it.
template <int N, typename Len>
__device__ __forceinline__ int find_sequence(const DecodeParams& p, const int* pre, int per, int hv_n,
                                             long long r0, Len len_of, int& before) {
  int lo = 0, hi = N - 1;  // the last thread whose sequences start at or before r0
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<long long>(pre[mid]) * hv_n <= r0) lo = mid; else hi = mid - 1;
  }
  before = pre[lo];
  for (int b = lo * per;; ++b) {
    const int t = tiles_of(p, len_of(b));
    if (b + 1 >= p.batch || r0 < static_cast<long long>(before + t) * hv_n) return b;
    before += t;
  }
}

// Rows of head tile hv of a sequence without keys.
template <typename T>
__device__ __forceinline__ void no_keys(const DecodeParams& p, int b, int hv) {
  const int g = hv / p.head_tiles, ht = hv - g * p.head_tiles;
  const int h0 = g * p.group + ht * kMaxRows, hn = min(kMaxRows, p.group - ht * kMaxRows);
  T* out = static_cast<T*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + h0 * p.o.sh;
  const int chunks = p.head_dim / 8;
  for (int i = threadIdx.x; i < hn * chunks; i += blockDim.x)
    *reinterpret_cast<uint4*>(out + (i / chunks) * p.o.sh + (i % chunks) * 8) = make_uint4(0, 0, 0, 0);
  if (p.lse != nullptr)
    for (int i = threadIdx.x; i < hn; i += blockDim.x)
      p.lse[static_cast<int64_t>(b) * p.h_q + h0 + i] = INFINITY;
}

}  // namespace attn
