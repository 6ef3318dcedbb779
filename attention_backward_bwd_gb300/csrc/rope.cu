// Rotary positions of q and k (attn_rope) and the append to the paged
// key/value cache (attn_cache_append): one kernel, since the append is the
// rotation with k going to pages instead of ok and v copied beside it.
//
// Pair i of a token's head row is turned by angle = position * inv_freq[i]:
//   (x, y) -> (x cos - y sin, x sin + y cos);
// the gradient is the same with -sin.  A warp takes a token (or a part of its heads, when
// there are few tokens): it computes the token's n_freq sines and cosines once, and its
// lanes hold those of their chunk in registers while they pass over the heads, so a head
// costs two FMAs and a rounding an element and the kernel is bound by the memory it
// streams: every row is read once and written once, 16 bytes a lane, four rows in flight.
//
// The angle is reduced before it is rounded: inv_freq / 2 pi is held as a 64-bit
// fraction of a turn F, and position * F modulo 2^64 is exactly the fraction of
// a turn, for any int32 position, in one integer product.  Its top 32 bits go to
// fp32 and sincospif.
#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 4;   // row groups of a warp in flight
// Blocks resident on an SM: halves hold two chunks a row group and eight turns, 128
// registers; pairs and copies less (16384 tokens of 40 heads of 128, halves: 54.6 us with
// two blocks, 60.1 with three; pairs, 19014 appended tokens of 32 heads: 84.1 and 79.1).
template <int MODE>
constexpr int kBlocks = MODE == 1 ? 3 : 2;

// kHalves: a lane takes a chunk of 8 first elements and the chunk of their second ones
// (n_freq a multiple of 8).  kPairs: neighbouring elements, any n_freq.  kMixed: halves
// whose second elements start inside a chunk; a lane takes one chunk and reads the other
// elements of its pairs beside it, all of a row before the row is written.
enum RopeMode { kHalves = 0, kPairs = 1, kMixed = 2 };

// How a warp's lanes share the rows: 1 << lanes_log2 lanes take one rotated row (its
// units: chunks or chunk pairs that turn, then chunks that are copied), 1 << v_lanes_log2
// lanes one row of v (its chunks).
struct RopeGrid {
  int lanes_log2, v_lanes_log2;
  int units, rot_units, chunks;
  int q_groups, k_groups, v_groups;  // groups of rows that a warp takes at once
  int parts;             // warps that share a token's groups
  FastDiv part, seq;
};

template <typename T>
__device__ __forceinline__ void turn8(uint4& lo, uint4& hi, const float2* cs) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Pack<T>::unpack(a[i]), y = Pack<T>::unpack(b[i]);
    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    const float s0 = c0.y, s1 = c1.y;
    a[i] = Pack<T>::two(x.x * c0.x - y.x * s0, x.y * c1.x - y.y * s1);
    b[i] = Pack<T>::two(x.x * s0 + y.x * c0.x, x.y * s1 + y.y * c1.x);
  }
}

// The first `n` of a chunk's four pairs turn.
template <typename T>
__device__ __forceinline__ void turn_pairs(uint4& v, const float2* cs, int n) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= n) break;
    const float2 x = Pack<T>::unpack(a[i]);
    const float2 c = cs[i];
    const float s = c.y;
    a[i] = Pack<T>::two(x.x * c.x - x.y * s, x.x * s + x.y * c.x);
  }
}

// Element i of a chunk becomes x cs.x + y cs.y with its pair's other element y (cs.y is
// -sin in the first half of the pairs, sin in the second); the first `n` (even) turn.
template <typename T>
__device__ __forceinline__ void turn_mixed(uint4& v, const uint32_t (&other)[4], const float2* cs, int n) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Pack<T>::unpack(a[i]);
    const float2 y = Pack<T>::unpack(other[i]);
    if (2 * i < n)
      a[i] = Pack<T>::two(x.x * cs[2 * i].x + y.x * cs[2 * i].y,
                          x.y * cs[2 * i + 1].x + y.y * cs[2 * i + 1].y);
  }
}

struct TokenInfo {
  int64_t k_off, v_off;  // element offsets of the token's slot (head 0) in the cache
  int slot;              // < 0: not stored
  bool live;             // belongs to a sequence
};

// Sequence and slot of new token t, with every device-side check, by a whole warp; its
// first part also writes the token's number into slot_positions.
__device__ __forceinline__ TokenInfo locate(const RopeParams& p, int t, bool first_part) {
  const int lane = lane_id();
  TokenInfo info{0, 0, -1, false};
  int b = t, i = 0;
  if (p.cu != nullptr) {
    int lo = 0, hi = p.batch;  // the last sequence that starts at or before t, 32 probes a step
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = min(lo + lane * step, hi - 1);
      const int n = __popc(__ballot_sync(0xffffffffu, p.cu[at] <= t));
      lo = min(lo + max(n - 1, 0) * step, hi - 1);
      hi = min(lo + step, hi);
    }
    b = lo;
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    if (t >= p.cu[p.batch]) return info;  // behind the last sequence
    if (c0 < 0 || t < c0 || t >= c1) {
      if (lane == 0) report(p.status, kBadOffsets);
      return info;
    }
    i = t - c0;
  }
  info.live = true;
  const int n = p.seqlens[b];
  const int64_t slot = static_cast<int64_t>(n) + i;
  const int64_t cap = static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d;
  if (n < 0 || slot >= cap || (p.slot_positions != nullptr && slot >= p.slots_stride)) {
    if (lane == 0) report(p.status, kBadLength);
    return info;
  }
  int page, within;
  if (!page_of(p.cache, p.cache.table + b * p.cache.table_stride, static_cast<int>(slot), page,
               within, p.status))
    return info;
  info.slot = static_cast<int>(slot);
  info.k_off = page * p.cache.k.sb + within * p.cache.k.ss;
  info.v_off = page * p.cache.v.sb + within * p.cache.v.ss;
  if (first_part && p.slot_positions != nullptr) {
    const int number = p.seen[b] + i;
    for (int h = lane; h < p.h_k; h += 32)
      p.slot_positions[(static_cast<int64_t>(b) * p.h_k + h) * p.slots_stride + slot] = number;
  }
  return info;
}

template <typename T, int MODE, bool APPEND>
__global__ void __launch_bounds__(kThreads, kBlocks<MODE>) rope_kernel(RopeParams p, RopeGrid g) {
  extern __shared__ float2 cs_all[];  // [warp][n_freq] (cos, sin)
  __shared__ unsigned long long turns[128];
  const int nf = p.rot.n_freq, lane = lane_id(), warp = threadIdx.x >> 5;
  float2* cs = cs_all + warp * nf;

  // fraction of a turn that one position adds at each frequency, times 2^64
  for (int i = threadIdx.x; i < nf; i += kThreads) {
    const double x = static_cast<double>(p.rot.inv_freq[i]) * 0.15915494309189535;
    turns[i] = static_cast<unsigned long long>((x - floor(x)) * 18446744073709551616.0);
  }
  if (APPEND && blockIdx.x == 0 && p.cu != nullptr)
    for (int i = threadIdx.x; i < p.batch; i += kThreads)
      if (p.cu[i] < 0 || p.cu[i] > p.cu[i + 1]) report(p.status, kBadOffsets);
  __syncthreads();

  const int c = lane & ((1 << g.lanes_log2) - 1), rl = lane >> g.lanes_log2;
  const bool turns_here = c < g.rot_units;
  const int total = g.q_groups + g.k_groups + g.v_groups;
  const int64_t items = p.tokens * g.parts, step = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items; item += step) {
    int64_t token = item;
    int begin = 0, end = total;
    bool first_part = true;
    if (g.parts > 1) {
      token = item / g.parts;
      const int part = static_cast<int>(item - token * g.parts);
      first_part = part == 0;
      begin = static_cast<int>(g.part.div(part * total));
      end = static_cast<int>(g.part.div((part + 1) * total));
    }
    int64_t b = 0, s = token;
    if (!APPEND) {
      b = g.seq.div(static_cast<uint32_t>(token));
      s = token - b * g.seq.d;
    }
    TokenInfo info{0, 0, -1, false};
    bool ready = false;
    // what the stores need, worked out while the first rows are on their way
    auto prepare = [&]() {
      if (APPEND) info = locate(p, static_cast<int>(token), first_part);
      __syncwarp();  // the last token's values have been read
      for (int i = lane; i < nf; i += 32) {
        int axis = 0;
#pragma unroll
        for (int a = 0; a < 3; ++a) axis += i >= p.rot.end[a] ? 1 : 0;
        const long long pos = p.rot.positions[axis * p.rot.axis_stride + token];
        const unsigned long long phase = static_cast<unsigned long long>(pos) * turns[i];
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &sn, &cn);
        cs[i] = make_float2(cn, sn * p.rot.sign);
      }
      __syncwarp();
      ready = true;
    };
    // The rows of q, of k, and of v (copied).  Head strides stay below 2^31 elements.
    int g0 = 0;
#pragma unroll 1
    for (int kind = 0; kind < (APPEND ? 3 : 2); ++kind) {
      const int n = kind == 0 ? p.h_q : p.h_k;
      const int groups = kind == 0 ? g.q_groups : (kind == 1 ? g.k_groups : g.v_groups);
      const int lanes_log2 = kind == 2 ? g.v_lanes_log2 : g.lanes_log2, rpw = 32 >> lanes_log2;
      const int it_begin = max(begin - g0, 0), it_end = min(end - g0, groups);
      g0 += groups;
      if (it_begin >= it_end) continue;
      const TensorArg& in = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
      const uint32_t ss = static_cast<uint32_t>(in.sh);
      const T* src = static_cast<const T*>(in.ptr) + b * in.sb + s * in.ss;
      auto target = [&](uint32_t& ds) -> T* {  // nullptr: not stored
        if (!APPEND || kind == 0) {
          const TensorArg& out = kind == 0 ? p.oq : p.ok;
          ds = static_cast<uint32_t>(out.sh);
          if (APPEND && !info.live) return nullptr;
          return static_cast<T*>(const_cast<void*>(out.ptr)) + b * out.sb + s * out.ss;
        }
        const TensorArg& out = kind == 1 ? p.cache.k : p.cache.v;
        ds = static_cast<uint32_t>(out.sh);
        if (info.slot < 0) return nullptr;
        return static_cast<T*>(const_cast<void*>(out.ptr)) + (kind == 1 ? info.k_off : info.v_off);
      };

      const int cc = kind == 2 ? lane & ((1 << lanes_log2) - 1) : c, r0 = kind == 2 ? lane >> lanes_log2 : rl;
      const bool lane_on = cc < (kind == 2 ? g.chunks : g.units), turn = kind < 2 && turns_here;
      // elements of this lane's chunk in a row (halves: the pairs' second chunk is nf behind)
      const int at = MODE != kHalves || turn || kind == 2 ? 8 * cc : 2 * nf + 8 * (cc - g.rot_units);
      constexpr int kTurns = MODE == kPairs ? 4 : 8;
      // of this lane's pairs (or elements, kMixed) the first ones that turn
      const int n_turn = min(kTurns, MODE == kPairs ? nf - 4 * cc : (MODE == kMixed ? 2 * nf - 8 * cc : 8));
      float2 mine[kTurns];
      bool have = false;
#pragma unroll 1
      for (int it = it_begin; it < it_end; it += kBatch) {
        uint4 lo[kBatch], hi[kBatch];
        uint32_t other[MODE == kMixed ? kBatch : 1][4];
        const int row = it * rpw + r0;
        const int rows_on = lane_on ? min(n, it_end * rpw) - row : 0;  // of this lane, from `row` on
        const T* x = src + static_cast<uint64_t>(ss) * static_cast<uint32_t>(row) + at;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i * rpw < rows_on) {
            const T* xi = x + static_cast<uint64_t>(ss) * static_cast<uint32_t>(i * rpw);
            lo[i] = *reinterpret_cast<const uint4*>(xi);
            if (MODE == kHalves && turn) hi[i] = *reinterpret_cast<const uint4*>(xi + nf);
            if (MODE == kMixed && turn) {
              if (nf % 2 == 0) {  // two elements at a time: both lie in one half
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int e = at + 2 * k;
                  other[i][k] = e < 2 * nf ? *reinterpret_cast<const uint32_t*>(xi + 2 * k + (e < nf ? nf : -nf)) : 0u;
                }
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int e = at + k;
                  const uint32_t y =
                      e < 2 * nf ? *reinterpret_cast<const unsigned short*>(xi + k + (e < nf ? nf : -nf)) : 0u;
                  other[i][k / 2] = k % 2 == 0 ? y : other[i][k / 2] | (y << 16);
                }
              }
            }
          }
        if (!ready) prepare();
        if (!have && turn)
#pragma unroll
          for (int i = 0; i < kTurns; ++i)
            if (i < n_turn) {
              const int f = kTurns * cc + i;
              mine[i] = cs[MODE == kMixed && f >= nf ? f - nf : f];
              if (MODE == kMixed && f < nf) mine[i].y = -mine[i].y;
            } else {
              mine[i] = make_float2(0.f, 0.f);  // not used
            }
        have = true;
        if (MODE == kMixed) __syncwarp();  // every lane has read its pairs' other elements
        uint32_t ds;
        T* y = target(ds);
        if (y == nullptr) break;
        y += static_cast<uint64_t>(ds) * static_cast<uint32_t>(row) + at;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (i * rpw < rows_on) {
            T* yi = y + static_cast<uint64_t>(ds) * static_cast<uint32_t>(i * rpw);
            if (turn) {
              if (MODE == kHalves) {
                turn8<T>(lo[i], hi[i], mine);
                *reinterpret_cast<uint4*>(yi + nf) = hi[i];
              } else if (MODE == kPairs) {
                turn_pairs<T>(lo[i], mine, n_turn);
              } else {
                turn_mixed<T>(lo[i], other[i], mine, n_turn);
              }
            }
            *reinterpret_cast<uint4*>(yi) = lo[i];
          }
      }
    }
  }
}

int log2_at_least(int n) {  // of the power of two that is at least n, at most 32
  int l = 0;
  while (l < 5 && (1 << l) < n) ++l;
  return l;
}

template <typename T, bool APPEND>
cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
  const int nf = p.rot.n_freq, d = p.head_dim;
  const int mode = p.rot.interleaved ? kPairs : (nf % 8 == 0 ? kHalves : kMixed);
  RopeGrid g;
  g.chunks = d / 8;
  g.rot_units = mode == kHalves ? nf / 8 : (2 * nf + 7) / 8;
  g.units = mode == kHalves ? g.rot_units + (d - 2 * nf) / 8 : d / 8;
  g.lanes_log2 = log2_at_least(g.units);
  g.v_lanes_log2 = log2_at_least(g.chunks);
  g.q_groups = ceil_div(p.h_q, 32 >> g.lanes_log2);
  g.k_groups = ceil_div(p.h_k, 32 >> g.lanes_log2);
  g.v_groups = APPEND ? ceil_div(p.h_k, 32 >> g.v_lanes_log2) : 0;
  // few tokens: a token's groups are shared by several warps, down to a batch each, so
  // that every resident warp has about four items and none waits long for the others
  const int64_t most = static_cast<int64_t>(num_sms()) * (mode == kPairs ? kBlocks<kPairs> : kBlocks<kHalves>);
  const int64_t groups = static_cast<int64_t>(g.q_groups) + g.k_groups + g.v_groups;
  const int64_t batches = (groups + kBatch - 1) / kBatch;
  int64_t parts = 4 * most * kWarps / p.tokens;
  parts = parts < 1 ? 1 : (parts > batches ? batches : parts);
  g.parts = static_cast<int>(parts);
  if (groups * (parts + 1) > INT32_MAX) return cudaErrorInvalidValue;
  g.part.set(static_cast<uint32_t>(parts));
  g.seq.set(static_cast<uint32_t>(p.seqlen));
  int64_t grid = (p.tokens * parts + kWarps - 1) / kWarps;
  const unsigned blocks = static_cast<unsigned>(grid < most ? grid : most);
  const size_t smem = static_cast<size_t>(kWarps) * nf * sizeof(float2);
  if (mode == kHalves)
    rope_kernel<T, kHalves, APPEND><<<blocks, kThreads, smem, stream>>>(p, g);
  else if (mode == kPairs)
    rope_kernel<T, kPairs, APPEND><<<blocks, kThreads, smem, stream>>>(p, g);
  else
    rope_kernel<T, kMixed, APPEND><<<blocks, kThreads, smem, stream>>>(p, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, bool append, cudaStream_t stream) {
  if (append)
    return dtype == ATTN_BF16 ? launch_t<__nv_bfloat16, true>(p, stream)
                              : launch_t<__half, true>(p, stream);
  return dtype == ATTN_BF16 ? launch_t<__nv_bfloat16, false>(p, stream)
                            : launch_t<__half, false>(p, stream);
}

}  // namespace attn
