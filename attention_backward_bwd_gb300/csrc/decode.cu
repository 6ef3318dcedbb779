// Attention of one new token a sequence over the paged cache (attn_decode).
//
// For each (sequence, key/value head) the query heads of the group share every key and
// value, so the work is one pass over the cached rows: bound by the memory they lie in.
// With up to 16 query heads as the M rows of an m16n8k16 product, S = Q K^T and O += P V
// take a few per cent of the tensor pipe at full memory speed, whatever the group, so the
// products are kept small and synchronous and the design goes into the loads.
//
// Split.  Keys come in tiles of 64.  All tiles of all (sequence, head) segments form one
// line, cut into equal runs, one per resident block: ragged lengths balance by
// themselves, and one long sequence uses every SM.  A segment that lies inside one block
// is finished there; one that is cut leaves (O, maximum, sum) partials which a second
// small kernel joins.  The cut depends on the lengths alone, so results do not depend on
// timing.
//
// Block.  Four warps; tiles pass through a ring of shared-memory stages filled by 16-byte
// asynchronous copies, several tiles ahead.  Rows are padded by 16 bytes so that ldmatrix
// meets no bank conflict.  In a tile each warp takes the logits of 16 keys; the warps
// share the running maximum and P through shared memory; then each warp takes a quarter
// of the head dimension of O over all 64 keys, so the warps never join their O.
// Row addresses (page lookups) are worked out by two warps ahead of the copies.
//
// P is rounded to the inputs' type for the P V product (half a step of relative error
// on each, averaged by the sum); the sum itself, maxima and logits stay fp32.
#include <atomic>

#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kTile = 64;       // keys of a tile
constexpr int kThreads = 128;
constexpr int kMaxRows = 16;    // query heads of a block
constexpr int kLens = 512;      // lengths kept in shared memory
constexpr int kPPitch = 144;    // bytes of a P row (64 keys and 16 bytes)

// Stages: what fits twice on an SM up to 128 columns, once above (two blocks keep the
// loads going while one of them synchronises; wider rows have fewer, larger tiles).
template <int DP>
struct Cfg {
  static constexpr int kPitch = DP * 2 + 16;
  static constexpr int kStageBytes = 2 * kTile * kPitch;
  static constexpr int kStages = DP == 64 ? 5 : (DP == 128 ? 3 : (DP == 192 ? 4 : 3));
  static constexpr int kBlocks = DP <= 128 ? 2 : 1;
  static constexpr int kSlots = kStages + 2;
  static constexpr int kSmem = kStages * kStageBytes + kSlots * (kTile * 16 + 32) +
                               kMaxRows * kPPitch + 2 * 4 * kMaxRows * 4 + kLens * 4;
};

struct TileDesc {
  int b, hv, rel;  // sequence, head tile, first key of the tile (from the first seen)
  int flags;
  uint32_t valid[2];  // bit per key of the tile
  int pad[2];
};
enum { kBegin = 1, kEnd = 2, kWhole = 4, kSecond = 8 };

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
  return (n - first_key(p, n) + kTile - 1) / kTile;
}

// Where the line of tiles is cut.  Run i of `runs` is [i * total / runs, (i + 1) * total / runs).
struct Cut {
  long long total;
  int runs;
  __device__ __forceinline__ long long start(int i) const { return total * i / runs; }
  __device__ __forceinline__ int run_of(long long tile) const {
    return static_cast<int>(((tile + 1) * runs - 1) / total);
  }
};

// Block-wide exclusive prefix of the tiles of the sequences: every thread owns `per`
// neighbouring ones.  Returns this thread's prefix; `mine` its own tiles.  Starts and
// ends with a barrier.
__device__ __forceinline__ long long scan_tiles(const DecodeParams& p, bool tell, int* lens,
                                                long long* warp_sums, int per, long long& mine,
                                                long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = threadIdx.x * per + i;
    if (b >= p.batch) break;
    const int n = clean_len(p, p.seqlens[b], tell);
    if (lens != nullptr && b < kLens) lens[b] = n;
    mine += tiles_of(p, n);
  }
  long long x = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? warp_sums[w] : 0;
    total += warp_sums[w];
  }
  return before + x - mine;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
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
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (Pack<T>::kIsBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Partial of run c (its first or second cut segment): rows of O, then maxima and sums.
__device__ __forceinline__ float* partial(const DecodeParams& p, int c, int second) {
  return p.parts + (static_cast<int64_t>(c) * 2 + second) * p.part_stride;
}

template <typename T, int DP, bool EXACT>
__global__ void __launch_bounds__(kThreads, Cfg<DP>::kBlocks)
    decode_kernel(DecodeParams p) {
  using C = Cfg<DP>;
  constexpr int S = C::kStages, kPitch = C::kPitch, kSlots = C::kSlots;
  constexpr int kSteps = DP / 16;      // k-steps of Q K^T
  constexpr int kCols = DP / 4;        // columns of O of a warp
  constexpr int kNt = kCols / 8;       // their n-tiles
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_sums[kThreads / 32];
  __shared__ long long s_before;
  __shared__ int s_b;
  unsigned char* ring = smem;
  longlong2* rows = reinterpret_cast<longlong2*>(ring + S * C::kStageBytes);
  TileDesc* desc = reinterpret_cast<TileDesc*>(rows + kSlots * kTile);
  unsigned char* pbuf = reinterpret_cast<unsigned char*>(desc + kSlots);
  float* smax = reinterpret_cast<float*>(pbuf + kMaxRows * kPPitch);
  float* ssum = smax + 4 * kMaxRows;
  int* lens = reinterpret_cast<int*>(ssum + 4 * kMaxRows);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hv_n = p.h_k * p.head_tiles;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this block's run of tiles
  const int per = (p.batch + kThreads - 1) / kThreads;
  long long mine, total;
  const long long before = scan_tiles(p, true, lens, s_sums, per, mine, total);
  Cut cut;
  cut.total = total * hv_n;
  cut.runs = static_cast<int>(min(static_cast<long long>(gridDim.x), cut.total));
  if (static_cast<int>(blockIdx.x) >= cut.runs) return;
  const long long r0 = cut.start(blockIdx.x), r1 = cut.start(blockIdx.x + 1);
  if (r0 >= before * hv_n && r0 < (before + mine) * hv_n) {
    long long at = before;
    int b = tid * per;
    for (;; ++b) {
      const int t = tiles_of(p, clean_len(p, p.seqlens[b], false));
      if (r0 < (at + t) * hv_n) break;
      at += t;
    }
    s_b = b;
    s_before = at;
  }
  // columns that no copy writes stay zero
  if (!EXACT) {
    const int c0 = p.head_dim / 8, nc = DP / 8 - c0;
    for (int i = tid; i < S * 2 * kTile * nc; i += kThreads)
      *reinterpret_cast<uint4*>(ring + (i / nc) * kPitch + (c0 + i % nc) * 16) = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  // ---- the planner (warps 0 and 1, one key of a tile each): walks the run
  int left = static_cast<int>(min(r1 - r0, 0x7fffffffLL));
  const int n_tiles = left;
  int cb = s_b, ch, ct, cn, cfirst, cnt;
  bool seg_from_start;
  int nth = 0;  // segment of the run: 0 first, then 1
  auto load_seq = [&]() {
    cn = cb < kLens ? lens[cb] : clean_len(p, p.seqlens[cb], false);
    cfirst = first_key(p, cn);
    cnt = (cn - cfirst + kTile - 1) / kTile;
  };
  load_seq();
  {
    const long long in = r0 - s_before * hv_n;
    ch = static_cast<int>(in / cnt);
    ct = static_cast<int>(in - static_cast<long long>(ch) * cnt);
    seg_from_start = ct == 0;
  }
  int begin = 1;
  // what plan() saw, for store_plan()
  int pend_page = -1, pend_within = 0, pend_head = 0;
  bool pend_live = false;
  TileDesc pend;
  auto plan = [&]() {  // looks one tile up and moves on
    if (left == 0) return;
    const int j = cfirst + ct * kTile + tid;
    pend_live = j < cn;
    pend_head = ch / p.head_tiles;
    if (pend_live) {
      const int n = static_cast<int>(p.cache.page.div(static_cast<uint32_t>(j)));
      pend_within = j - n * static_cast<int>(p.cache.page.d);
      pend_page = p.cache.table[cb * p.cache.table_stride + n];
    }
    const bool at_end = ct == cnt - 1;
    pend.b = cb;
    pend.hv = ch;
    pend.rel = ct * kTile;
    pend.flags = (begin ? kBegin : 0) | (at_end || left == 1 ? kEnd : 0) |
                 (at_end && seg_from_start ? kWhole : 0) | (nth ? kSecond : 0);
    begin = 0;
    --left;
    if (left == 0) return;
    if (!at_end) {
      ++ct;
      return;
    }
    ct = 0;
    begin = 1;
    nth = 1;
    seg_from_start = true;
    if (++ch == hv_n) {
      ch = 0;
      do {
        ++cb;
        load_seq();
      } while (cnt == 0);
    }
  };
  auto store_plan = [&](int slot) {
    bool ok = pend_live;
    if (ok && static_cast<unsigned>(pend_page) >= static_cast<unsigned>(p.cache.num_pages)) {
      report(p.status, kBadPage);
      ok = false;
    }
    longlong2 o = make_longlong2(-1, -1);
    if (ok) {
      o.x = pend_page * p.cache.k.sb + pend_within * p.cache.k.ss + pend_head * p.cache.k.sh;
      o.y = pend_page * p.cache.v.sb + pend_within * p.cache.v.ss + pend_head * p.cache.v.sh;
    }
    rows[slot * kTile + tid] = o;
    const uint32_t bits = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) desc[slot].valid[warp] = bits;
    if (tid == 0) {
      desc[slot].b = pend.b;
      desc[slot].hv = pend.hv;
      desc[slot].rel = pend.rel;
      desc[slot].flags = pend.flags;
    }
  };
  const T* kbase = static_cast<const T*>(p.cache.k.ptr);
  const T* vbase = static_cast<const T*>(p.cache.v.ptr);
  const uint32_t ring_u = smem_u32(ring);
  auto fetch = [&](int tile) {  // issues the copies of one tile
    const longlong2* r = rows + (tile % kSlots) * kTile;
    const uint32_t dst = ring_u + (tile % S) * C::kStageBytes;
    if (EXACT) {
      constexpr int kCh = DP / 8, kIter = kTile * kCh / kThreads;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int u = tid + i * kThreads, row = u / kCh, c = u % kCh;
        const longlong2 o = r[row];
        const bool ok = o.x >= 0;
        cp_async16(dst + row * kPitch + c * 16, kbase + (ok ? o.x + c * 8 : 0), ok);
        cp_async16(dst + (kTile + row) * kPitch + c * 16, vbase + (ok ? o.y + c * 8 : 0), ok);
      }
    } else {
      const int total_u = kTile * static_cast<int>(p.chunks.d);
      for (int u = tid; u < total_u; u += kThreads) {
        const int row = static_cast<int>(p.chunks.div(u)), c = u - row * static_cast<int>(p.chunks.d);
        const longlong2 o = r[row];
        const bool ok = o.x >= 0;
        cp_async16(dst + row * kPitch + c * 16, kbase + (ok ? o.x + c * 8 : 0), ok);
        cp_async16(dst + (kTile + row) * kPitch + c * 16, vbase + (ok ? o.y + c * 8 : 0), ok);
      }
    }
  };

  // ---- prologue: plans for the first S tiles, copies for S - 1
  if (warp < 2)
    for (int t = 0; t < S; ++t) {
      plan();
      if (t < n_tiles) store_plan(t);
      if (t == S - 1) plan();  // tile S waits in the registers
    }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < S - 1; ++t) {
    if (t < n_tiles) fetch(t);
    cp_commit();
  }

  uint32_t qf[kSteps][4];
  float o[kNt][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int row0 = lane >> 2, col2 = (lane & 3) * 2;

  for (int t = 0; t < n_tiles; ++t) {
    const TileDesc& d = desc[t % kSlots];
    if (d.flags & kBegin) {
      const int g = d.hv / p.head_tiles, ht = d.hv - g * p.head_tiles;
      const int h0 = g * p.group + ht * kMaxRows, hn = min(kMaxRows, p.group - ht * kMaxRows);
      const T* q = static_cast<const T*>(p.q.ptr) + d.b * p.q.sb;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = row0 + (i & 1) * 8, col = k * 16 + col2 + (i >> 1) * 8;
          qf[k][i] = row < hn && (EXACT || col < p.head_dim)
                         ? *reinterpret_cast<const uint32_t*>(q + (h0 + row) * p.q.sh + col)
                         : 0u;
        }
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    cp_wait<S - 2>();
    __syncthreads();  // tile t is there for all; stage of tile t - 1 is free

    if (t + S - 1 < n_tiles) fetch(t + S - 1);
    cp_commit();
    if (warp < 2 && t + S < n_tiles) {
      store_plan((t + S) % kSlots);
      plan();
    }

    // ---- logits of this warp's 16 keys
    const uint32_t kst = ring_u + (t % S) * C::kStageBytes;
    float s[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
    {
      const uint32_t a = kst + (warp * 16 + ((lane >> 4) << 3) + (lane & 7)) * kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t kf[4];
        ldsm4(a + k * 32, kf);
        mma16816<T>(s[0], qf[k], kf[0], kf[1]);
        mma16816<T>(s[1], qf[k], kf[2], kf[3]);
      }
    }
    const uint32_t valid = d.valid[warp >> 1] >> ((warp & 1) * 16);
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool ok = (valid >> (n * 8 + col2 + (i & 1))) & 1u;
        float x = p.softcap > 0.f ? p.cap_out * tanh_exp(s[n][i] * p.cap_in) : s[n][i] * p.scale_log2;
        x = ok ? x : -INFINITY;
        s[n][i] = x;
        top[i >> 1] = fmaxf(top[i >> 1], x);
      }
    if (p.logits != nullptr) {
      const int g = d.hv / p.head_tiles, ht = d.hv - g * p.head_tiles;
      const int hn = min(kMaxRows, p.group - ht * kMaxRows);
      const int64_t h0 = static_cast<int64_t>(d.b) * p.h_q + g * p.group + ht * kMaxRows;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (row0 + r * 8 < hn) {
          float* out = p.logits + (h0 + row0 + r * 8) * p.logit_stride + d.rel + warp * 16 + col2;
#pragma unroll
          for (int n = 0; n < 2; ++n)
            *reinterpret_cast<float2*>(out + n * 8) = make_float2(s[n][r * 2], s[n][r * 2 + 1]);
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      if ((lane & 3) == 0) smax[warp * kMaxRows + row0 + r * 8] = top[r];
    }
    __syncthreads();

    // ---- P under the common maximum
    float scale_o[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = m[r];
#pragma unroll
      for (int w = 0; w < 4; ++w) mx = fmaxf(mx, smax[w * kMaxRows + row0 + r * 8]);
      const float base = mx == -INFINITY ? 0.f : mx;
      scale_o[r] = ex2(m[r] - base);
      m[r] = mx;
      float sum = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float p0 = ex2(s[n][r * 2] - base), p1 = ex2(s[n][r * 2 + 1] - base);
        sum += p0 + p1;
        *reinterpret_cast<uint32_t*>(pbuf + (row0 + r * 8) * kPPitch +
                                     (warp * 16 + n * 8 + col2) * 2) = Pack<T>::two(p0, p1);
      }
      l[r] = l[r] * scale_o[r] + sum;
    }
    __syncthreads();

    // ---- O += P V for this warp's columns
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      o[n][0] *= scale_o[0];
      o[n][1] *= scale_o[0];
      o[n][2] *= scale_o[1];
      o[n][3] *= scale_o[1];
    }
    {
      const uint32_t pa = smem_u32(pbuf) + ((lane & 7) + ((lane >> 3) & 1) * 8) * kPPitch + (lane >> 4) * 16;
      const uint32_t va = kst + (kTile + (lane & 7) + ((lane >> 3) & 1) * 8) * kPitch +
                          (warp * kCols + (lane >> 4) * 8) * 2;
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k) {
        uint32_t pf[4];
        ldsm4(pa + k * 32, pf);
#pragma unroll
        for (int n = 0; n < kNt; n += 2) {
          uint32_t vf[4];
          ldsm4_t(va + k * 16 * kPitch + n * 16, vf);
          mma16816<T>(o[n], pf, vf[0], vf[1]);
          mma16816<T>(o[n + 1], pf, vf[2], vf[3]);
        }
      }
    }

    if (d.flags & kEnd) {
      // ---- this run's part of the segment is complete
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = l[r];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if ((lane & 3) == 0) ssum[warp * kMaxRows + row0 + r * 8] = x;
      }
      __syncthreads();
      const int g = d.hv / p.head_tiles, ht = d.hv - g * p.head_tiles;
      const int h0 = g * p.group + ht * kMaxRows, hn = min(kMaxRows, p.group - ht * kMaxRows);
      const bool whole = (d.flags & kWhole) != 0;
      float* part = partial(p, blockIdx.x, (d.flags & kSecond) ? 1 : 0);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + r * 8;
        if (row >= hn) continue;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += ssum[w * kMaxRows + row];
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        if (whole) {
          T* out = static_cast<T*>(const_cast<void*>(p.o.ptr)) + d.b * p.o.sb + (h0 + row) * p.o.sh;
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            const int col = warp * kCols + n * 8 + col2;
            if (EXACT || col < p.head_dim)
              *reinterpret_cast<uint32_t*>(out + col) =
                  Pack<T>::two(none ? 0.f : o[n][r * 2] * inv, none ? 0.f : o[n][r * 2 + 1] * inv);
          }
          if (warp == 0 && (lane & 3) == 0) {
            const float lse2 = none ? INFINITY : m[r] + log2f(sum);
            const int64_t at = static_cast<int64_t>(d.b) * p.h_q + h0 + row;
            if (p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
            p.lse2[at] = lse2;
          }
        } else {
#pragma unroll
          for (int n = 0; n < kNt; ++n)
            *reinterpret_cast<float2*>(part + row * DP + warp * kCols + n * 8 + col2) =
                make_float2(o[n][r * 2], o[n][r * 2 + 1]);
          if (warp == 0 && (lane & 3) == 0) {
            part[p.part_rows * DP + row] = m[r];
            part[p.part_rows * DP + kMaxRows + row] = sum;
          }
        }
      }
    }
  }
  cp_wait<0>();
}

// Joins the partials of cut segments, writes the rows of empty sequences, and adds the
// attention weights.  Blocks [0, batch * h_q): one row of O each; then `chunks` blocks of
// kKeys keys for every (sequence, key/value head) when weights are asked for.
constexpr int kKeys = 1024;

template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(DecodeParams p, int runs, int dp, int chunks) {
  __shared__ long long s_sums[kThreads / 32];
  __shared__ long long s_before;
  __shared__ float4 s_part[kThreads];
  __shared__ float s_lse[256];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t rows = static_cast<int64_t>(p.batch) * p.h_q;
  const bool is_row = blockIdx.x < rows;
  int b, h, j0 = 0;
  if (is_row) {
    b = blockIdx.x / p.h_q;
    h = blockIdx.x - b * p.h_q;
  } else {
    const int64_t u = blockIdx.x - rows;
    const int bh = static_cast<int>(u / chunks);
    j0 = static_cast<int>(u - static_cast<int64_t>(bh) * chunks) * kKeys;
    b = bh / p.h_k;
    h = (bh - b * p.h_k) * p.group;
  }
  const int n = clean_len(p, p.seqlens[b], false);
  const int first = first_key(p, n), t_b = tiles_of(p, n);
  const int hv_n = p.h_k * p.head_tiles;
  const int per = (p.batch + kThreads - 1) / kThreads;
  if (!is_row && j0 >= n) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // no block may end before the first kernel
    return;
  }
  long long mine, total;
  const long long before = scan_tiles(p, blockIdx.x == 0, nullptr, s_sums, per, mine, total);
  if (b / per == tid) {
    long long at = before;
    for (int i = tid * per; i < b; ++i) at += tiles_of(p, clean_len(p, p.seqlens[i], false));
    s_before = at;
  }
  __syncthreads();
  Cut cut;
  cut.total = total * hv_n;
  cut.runs = static_cast<int>(min(static_cast<long long>(runs), cut.total));
  const int part_m = p.part_rows * dp;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (is_row) {
    T* out = static_cast<T*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + h * p.o.sh;
    const int64_t at = static_cast<int64_t>(b) * p.h_q + h;
    if (t_b == 0) {  // no keys
      for (int d = tid; d < p.head_dim; d += kThreads) out[d] = static_cast<T>(0.f);
      if (tid == 0 && p.lse != nullptr) p.lse[at] = INFINITY;
      return;
    }
    const int g = h / p.group, hg = h - g * p.group, ht = hg / kMaxRows, row = hg - ht * kMaxRows;
    const long long s0 = s_before * hv_n + static_cast<long long>(g * p.head_tiles + ht) * t_b;
    const int c0 = cut.run_of(s0), c1 = cut.run_of(s0 + t_b - 1);
    if (c0 == c1) return;  // finished by its run
    float top = -INFINITY, sum = 0.f;
    for (int c = c0; c <= c1; ++c)
      top = fmaxf(top, partial(p, c, cut.start(c) >= s0 ? 0 : 1)[part_m + row]);
    const float base = top == -INFINITY ? 0.f : top;
    // threads: 16-byte column group, and every stripe-th run
    const int groups = dp / 4, stripes = kThreads / groups > 0 ? kThreads / groups : 1;
    const int cg = tid % groups, st = tid / groups;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (st < stripes)
      for (int c = c0 + st; c <= c1; c += stripes) {
        const float* part = partial(p, c, cut.start(c) >= s0 ? 0 : 1);
        const float w = ex2(part[part_m + row] - base);
        const float4 x = *reinterpret_cast<const float4*>(part + row * dp + cg * 4);
        sum += w * part[part_m + kMaxRows + row];
        acc.x += w * x.x;
        acc.y += w * x.y;
        acc.z += w * x.z;
        acc.w += w * x.w;
      }
    s_part[tid] = acc;
    s_lse[tid] = sum;
    __syncthreads();
    if (st == 0 && tid < groups) {
      for (int i = 1; i < stripes; ++i) {
        const float4 x = s_part[tid + i * groups];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
        sum += s_lse[i * groups];
      }
      const bool none = sum == 0.f;
      const float inv = none ? 0.f : 1.f / sum;
      if (cg * 4 < p.head_dim) {
        uint2 v;
        v.x = Pack<T>::two(none ? 0.f : acc.x * inv, none ? 0.f : acc.y * inv);
        v.y = Pack<T>::two(none ? 0.f : acc.z * inv, none ? 0.f : acc.w * inv);
        *reinterpret_cast<uint2*>(out + cg * 4) = v;
      }
      if (tid == 0 && p.lse != nullptr)
        p.lse[at] = none ? INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
    }
    return;
  }

  // ---- weights of keys [j0, j0 + kKeys) of one key/value head
  const int g = h / p.group;
  const float* logits = p.logits + (static_cast<int64_t>(b) * p.h_q + h) * p.logit_stride;
  float w[kKeys / kThreads];
#pragma unroll
  for (int i = 0; i < kKeys / kThreads; ++i) w[i] = 0.f;
  for (int g0 = 0; g0 < p.group; g0 += 256) {
    const int gn = min(256, p.group - g0);
    __syncthreads();
    if (t_b > 0)
      for (int i = warp; i < gn; i += kThreads / 32) {  // the row's LSE, a warp each
        const int hg = g0 + i, ht = hg / kMaxRows, row = hg - ht * kMaxRows;
        const long long s0 = s_before * hv_n + static_cast<long long>(g * p.head_tiles + ht) * t_b;
        const int c0 = cut.run_of(s0), c1 = cut.run_of(s0 + t_b - 1);
        float lse2;
        if (c0 == c1) {
          lse2 = p.lse2[static_cast<int64_t>(b) * p.h_q + h + hg];
        } else {
          float top = -INFINITY, sum = 0.f;
          for (int c = c0 + lane; c <= c1; c += 32)
            top = fmaxf(top, partial(p, c, cut.start(c) >= s0 ? 0 : 1)[part_m + row]);
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float base = top == -INFINITY ? 0.f : top;
          for (int c = c0 + lane; c <= c1; c += 32) {
            const float* part = partial(p, c, cut.start(c) >= s0 ? 0 : 1);
            sum += ex2(part[part_m + row] - base) * part[part_m + kMaxRows + row];
          }
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          lse2 = sum == 0.f ? INFINITY : base + log2f(sum);
        }
        if (lane == 0) s_lse[i] = lse2;
      }
    __syncthreads();
    for (int i = 0; i < gn; ++i) {
      const float lse2 = s_lse[i];
      const float* x = logits + (g0 + i) * p.logit_stride;
#pragma unroll
      for (int k = 0; k < kKeys / kThreads; ++k) {
        const int j = j0 + k * kThreads + tid;
        if (j >= first && j < n) w[k] += ex2(x[j - first] - lse2);
      }
    }
  }
  const int64_t at = (static_cast<int64_t>(b) * p.h_k + g) * p.w_stride;
#pragma unroll
  for (int k = 0; k < kKeys / kThreads; ++k) {
    const int j = j0 + k * kThreads + tid;
    if (j < n) p.w_out[at + j] = p.w_in[at + j] + w[k];
  }
}

int pad_dim(int d) { return d <= 64 ? 64 : (d <= 128 ? 128 : (d <= 192 ? 192 : 256)); }
// Resident blocks of the device at most: sizes the partials without asking a device.
constexpr int kMaxRuns = 384;

template <typename T, int DP, bool EXACT>
cudaError_t launch_main(const DecodeParams& p, int runs, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};  // devices with the attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit) || bit == 0) {
    e = cudaFuncSetAttribute(decode_kernel<T, DP, EXACT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<DP>::kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  decode_kernel<T, DP, EXACT><<<runs, kThreads, Cfg<DP>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(DecodeParams p, cudaStream_t stream) {
  const int dp = pad_dim(p.head_dim);
  p.head_tiles = ceil_div(p.group, kMaxRows);
  p.part_rows = p.group < kMaxRows ? p.group : kMaxRows;
  p.part_stride = static_cast<int64_t>(p.part_rows) * dp + 2 * kMaxRows;
  p.chunks.set(static_cast<uint32_t>(p.head_dim / 8));
  const int64_t most = static_cast<int64_t>(p.batch) * p.h_k * p.head_tiles * ceil_div(p.max_seqlen, kTile);
  int64_t runs = static_cast<int64_t>(num_sms()) * (dp <= 128 ? 2 : 1);
  if (runs > kMaxRuns) runs = kMaxRuns;
  if (runs > most) runs = most;
  cudaError_t e = cudaSuccess;
  const bool exact = dp == p.head_dim;
  if (runs > 0) {
    const int r = static_cast<int>(runs);
    if (dp == 64) e = exact ? launch_main<T, 64, true>(p, r, stream) : launch_main<T, 64, false>(p, r, stream);
    else if (dp == 128) e = exact ? launch_main<T, 128, true>(p, r, stream) : launch_main<T, 128, false>(p, r, stream);
    else if (dp == 192) e = exact ? launch_main<T, 192, true>(p, r, stream) : launch_main<T, 192, false>(p, r, stream);
    else e = exact ? launch_main<T, 256, true>(p, r, stream) : launch_main<T, 256, false>(p, r, stream);
    if (e != cudaSuccess) return e;
  }
  const int chunks = p.w_in != nullptr ? ceil_div(p.max_seqlen, kKeys) : 0;
  const int64_t blocks = static_cast<int64_t>(p.batch) * (p.h_q + static_cast<int64_t>(p.h_k) * chunks);
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = runs > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<T>, p, static_cast<int>(runs), dp, chunks);
}

}  // namespace

DecodeWs decode_ws(int batch, int h_q, int h_k, int head_dim, int max_seqlen, bool weights) {
  DecodeWs w;
  const size_t rows = static_cast<size_t>(batch) * h_q;
  const int group = h_q / h_k, part_rows = group < kMaxRows ? group : kMaxRows;
  w.logit_stride = round_up(max_seqlen, kTile);
  w.off_lse2 = 0;
  w.off_parts = align256(rows * 4);
  w.off_logits = w.off_parts + align256(static_cast<size_t>(kMaxRuns) * 2 *
                                        (static_cast<size_t>(part_rows) * pad_dim(head_dim) + 2 * kMaxRows) * 4);
  w.total = w.off_logits + (weights ? align256(rows * static_cast<size_t>(w.logit_stride) * 4) : 0);
  return w;
}

cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t stream) {
  return dtype == ATTN_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<__half>(p, stream);
}

}  // namespace attn
