// The append to a cache in 8 bits (attn_cache_append8) and its read-back (attn_cache_load8).
//
// A block of tokens of a page has, for each head, one factor s, a power of two; its codes c stand
// for c s.  An append takes the smallest s with |x| <= top s for every new value x of the block
// (top = 448 for e4m3, 127 for int8), but not less than the factor of the block's earlier tokens;
// where s grows, their codes are rounded to it again.  With powers of two a value of e4m3 only
// changes then where it leaves the normal range, and x / s is exact, so that a code is off by one
// rounding of x.
//
// Append.  A block of threads takes the new tokens of one block of the cache: they lie in one page
// (its tokens' block divides the page).  It computes the turns of a few rows at a time once for
// all heads; its warps take a head of q, of k or of v each, a lane eight neighbouring elements of a
// row.  Up to kHeld rows a lane stay in registers between the maximum and the rounding, so that
// k and v are read once; blocks with more new tokens are read a second time, from the L2.
// Read-back.  A warp takes a token: 16 codes a lane, 32 bytes out.
#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 8;       // rows of a lane in registers
constexpr int kTurns = 1024;   // turns of the rows that a block takes at once
constexpr int kBlocks = 2;     // of an SM
constexpr float kLargest = 1.152921504606847e18f;    // 2^60

// The order in which a lane finds the other element of a pair: kHalves in the chunk n_freq
// elements away (n_freq a multiple of 8), kPairs in its own chunk, kMixed element by element.
enum RopeMode { kNoTurn = 0, kHalves = 1, kPairs = 2, kMixed = 3 };

struct Append8Grid {
  int lanes_log2;        // lanes of a row
  int mode;
  int parts;             // blocks that share the heads of a block of tokens
};

// Smallest power of two that `top` is at most 448 (127) times, within the bounds; exact.
template <bool INT8>
__device__ __forceinline__ float factor_of(float top) {
  const uint32_t u = __float_as_uint(top);
  // top = m 2^E: the factor is 2^(E - 8) up to m = 1.75, or 2^(E - 6) up to m = 127 / 64
  const uint32_t edge = INT8 ? 0x7e0000u : 0x600000u;
  const int e = static_cast<int>(u >> 23) - 127 - (INT8 ? 6 : 8) + ((u & 0x7fffffu) > edge ? 1 : 0);
  return __int_as_float((min(max(e, -60), 60) + 127) << 23);
}

template <bool INT8>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  if (INT8) {
    auto one = [](float x) { return static_cast<uint32_t>(min(max(__float2int_rn(x), -127), 127)) & 0xffu; };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

template <bool INT8>
__device__ __forceinline__ float4 value4(uint32_t x) {
  if (INT8)
    return make_float4(static_cast<float>(static_cast<int8_t>(x)), static_cast<float>(static_cast<int8_t>(x >> 8)),
                       static_cast<float>(static_cast<int8_t>(x >> 16)), static_cast<float>(static_cast<int8_t>(x >> 24)));
  uint32_t lo, hi;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
  const float2 a = Pack<__half>::unpack(lo), b = Pack<__half>::unpack(hi);
  return make_float4(a.x, a.y, b.x, b.y);
}

// New tokens of sequence b: the first one (packed) and their number; the sequence's length (0 and
// bad where it is negative).
struct Fresh {
  int first, n;
  int len;
  bool bad;
};
__device__ __forceinline__ Fresh fresh_of(const Append8Params& p, int b, bool tell) {
  Fresh f{b, 1, p.seqlens[b], false};
  if (p.cu != nullptr) {
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    f.first = c0;
    f.n = c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > p.tokens) {
      if (tell) report(p.status, kBadOffsets);
      f.n = 0;
    }
  }
  if (f.len < 0) {
    f.bad = true;
    f.len = 0;
    if (tell && f.n > 0) report(p.status, kBadLength);
  }
  return f;
}
// Blocks of the cache that they touch.
__device__ __forceinline__ int blocks_of(const Append8Params& p, const Fresh& f) {
  if (f.n <= 0) return 0;
  const uint32_t size = p.cache.block.d;
  const uint32_t off = static_cast<uint32_t>(f.len) - p.cache.block.div(static_cast<uint32_t>(f.len)) * size;
  const uint32_t n = static_cast<uint32_t>(f.n), rest = size - off;  // new tokens, room of the first block
  return n <= rest ? 1 : 2 + static_cast<int>(p.cache.block.div(n - rest - 1));
}

template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads, kBlocks) append8_kernel(Append8Params p, Append8Grid g) {
  __shared__ float2 cs[kTurns];                  // (cos, sin) of [row][frequency]
  __shared__ unsigned long long turns[128];
  __shared__ int64_t s_pre[kThreads];            // (offsets that do not ascend may name a token often)
  __shared__ int64_t s_sums[kWarps];
  extern __shared__ float s_top[];               // largest values of the heads of k and of v
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nf = g.mode == kNoTurn ? 0 : p.rot.n_freq;

  // fraction of a turn that one position adds at each frequency, times 2^64
  for (int i = tid; i < nf; i += kThreads) {
    const double x = static_cast<double>(p.rot.inv_freq[i]) * 0.15915494309189535;
    turns[i] = static_cast<unsigned long long>((x - floor(x)) * 18446744073709551616.0);
  }
  // ---- blocks of the sequences before this thread's
  const int per = (p.batch + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int i = 0; i < per && tid * per + i < p.batch; ++i)
    mine += blocks_of(p, fresh_of(p, tid * per + i, blockIdx.x == 0));
  int64_t x = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  if (lane == 31) s_sums[warp] = x;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? s_sums[w] : 0;
    total += s_sums[w];
  }
  s_pre[tid] = before + x - mine;
  __syncthreads();

  const int lanes = 1 << g.lanes_log2, rpw = 32 >> g.lanes_log2, chunk_rows = kHeld * rpw;
  const int c = lane & (lanes - 1), r0 = lane >> g.lanes_log2, at = 8 * c;
  const bool on = at < p.head_dim;
  const int jobs = p.h_q + 2 * p.h_k;
  const int64_t items = total * g.parts;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t u = item / g.parts;
    const int part = static_cast<int>(item - u * g.parts);
    const int j0 = static_cast<int>(static_cast<int64_t>(jobs) * part / g.parts);
    const int j1 = static_cast<int>(static_cast<int64_t>(jobs) * (part + 1) / g.parts);
    // ---- the sequence and the block of tokens
    int lo = 0, hi = kThreads - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    int b = lo * per, at_block = static_cast<int>(u - s_pre[lo]);
    Fresh f = fresh_of(p, b, false);
    for (int n = blocks_of(p, f); at_block >= n; n = blocks_of(p, f)) {
      at_block -= n;
      f = fresh_of(p, ++b, false);
    }
    const uint32_t size = p.cache.block.d;
    const int64_t base = static_cast<int64_t>(p.cache.block.div(static_cast<uint32_t>(f.len)) + at_block) * size;
    const int64_t from = base > f.len ? base : f.len, end = min(base + size, static_cast<int64_t>(f.len) + f.n);
    const int token0 = f.first + static_cast<int>(from - f.len), n = static_cast<int>(end - from);
    const int old = static_cast<int>(from - base);  // earlier tokens of the block
    const int64_t cap = static_cast<int64_t>(p.cache.pages.max_pages) * p.cache.pages.page.d;
    bool stored = !f.bad;
    int page = 0, within = 0;
    if (stored && base >= cap) {
      if (tid == 0 && part == 0) report(p.status, kBadLength);
      stored = false;
    }
    if (stored) {
      const int pg = static_cast<int>(p.cache.pages.page.div(static_cast<uint32_t>(base)));
      within = static_cast<int>(base) - pg * static_cast<int>(p.cache.pages.page.d);
      page = p.cache.pages.table[b * p.cache.pages.table_stride + pg];
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.cache.pages.num_pages)) {
        if (tid == 0 && part == 0) report(p.status, kBadPage);
        stored = false;
      }
    }
    const int64_t blk = p.cache.block.div(static_cast<uint32_t>(within));

    // The rows [t0, t0 + chunk_rows) of the block's new tokens: their turns.
    auto turn_rows = [&](int t0) {
      __syncthreads();
      const int rows = min(chunk_rows, n - t0);
      for (int i = tid; i < rows * nf; i += kThreads) {
        const int r = i / nf, fr = i - r * nf;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < 3; ++a) axis += fr >= p.rot.end[a] ? 1 : 0;
        const long long pos = p.rot.positions[axis * p.rot.axis_stride + token0 + t0 + r];
        const unsigned long long phase = static_cast<unsigned long long>(pos) * turns[fr];
        float sn, cn;
        sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &sn, &cn);
        cs[i] = make_float2(cn, sn);
      }
      __syncthreads();
    };
    // This lane's elements of row r (of the chunk from t0 on), turned.
    auto take = [&](const TensorArg& in, int head, bool turn, int t0, int r, float (&v)[8]) {
      const T* row = static_cast<const T*>(in.ptr) + static_cast<int64_t>(token0 + t0 + r) * in.ss + head * in.sh;
      uint4 raw = *reinterpret_cast<const uint4*>(row + at);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = Pack<T>::unpack(w[i]);
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
      }
      if (!turn || at >= 2 * nf) return;
      const float2* t = cs + r * nf;
      if (g.mode == kPairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at / 2 + i < nf) {
            const float2 a = t[at / 2 + i];
            const float x0 = v[2 * i], x1 = v[2 * i + 1];
            v[2 * i] = x0 * a.x - x1 * a.y;
            v[2 * i + 1] = x0 * a.y + x1 * a.x;
          }
      } else if (g.mode == kHalves) {
        const bool second = at >= nf;
        const uint4 other = *reinterpret_cast<const uint4*>(row + at + (second ? -nf : nf));
        const uint32_t* ow = reinterpret_cast<const uint32_t*>(&other);
        const int f0 = second ? at - nf : at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 y = Pack<T>::unpack(ow[i]);
          const float2 a = t[f0 + 2 * i], bb = t[f0 + 2 * i + 1];
          v[2 * i] = v[2 * i] * a.x + y.x * (second ? a.y : -a.y);
          v[2 * i + 1] = v[2 * i + 1] * bb.x + y.y * (second ? bb.y : -bb.y);
        }
      } else {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = at + i;
          const uint16_t y = e < 2 * nf ? reinterpret_cast<const uint16_t*>(row)[e < nf ? e + nf : e - nf] : 0;
          o[i] = Pack<T>::unpack(y).x;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = at + i;
          if (e < 2 * nf) {
            const float2 a = t[e < nf ? e : e - nf];
            v[i] = v[i] * a.x + o[i] * (e < nf ? -a.y : a.y);
          }
        }
      }
    };
    auto largest = [&](const float (&v)[8], float top) {  // of the finite ones
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = fabsf(v[i]);
        top = y < INFINITY ? fmaxf(top, y) : top;
      }
      return top;
    };
    // A head's factor, from its new tokens' largest value; its earlier codes follow it.
    auto settle = [&](const TensorArg& pages, float* scales, const int64_t (&st)[3], int head, float top) {
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      float* s = scales + page * st[0] + blk * st[1] + head * st[2];
      float now = factor_of<INT8>(top);
      if (old > 0) {
        float was = *s;
        was = was > 0.f ? fminf(was, kLargest) : 0.f;
        __syncwarp();
        if (now > was) {
          const float ratio = was / now;
          const int per_row = p.head_dim / 16;
          char* rows = static_cast<char*>(const_cast<void*>(pages.ptr)) + page * pages.sb + within * pages.ss + head * pages.sh;
          for (int i = lane; i < old * per_row; i += 32) {
            const int r = i / per_row;
            uint4* to = reinterpret_cast<uint4*>(rows + r * pages.ss) + (i - r * per_row);
            uint4 codes = *to;
            uint32_t* w = reinterpret_cast<uint32_t*>(&codes);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 y = value4<INT8>(w[k]);
              w[k] = code4<INT8>(y.x * ratio, y.y * ratio, y.z * ratio, y.w * ratio);
            }
            *to = codes;
          }
        } else {
          now = was;
        }
      }
      if (lane == 0) *s = now;
      return 1.f / now;
    };
    auto put8 = [&](const TensorArg& pages, int head, int r, const float (&v)[8], float inv) {
      char* to = static_cast<char*>(const_cast<void*>(pages.ptr)) + page * pages.sb +
                 static_cast<int64_t>(within + old + r) * pages.ss + head * pages.sh + at;
      *reinterpret_cast<uint2*>(to) = make_uint2(code4<INT8>(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                                 code4<INT8>(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    };
    auto put16 = [&](int head, int r, const float (&v)[8]) {
      T* to = static_cast<T*>(const_cast<void*>(p.oq.ptr)) + static_cast<int64_t>(token0 + r) * p.oq.ss + head * p.oq.sh + at;
      *reinterpret_cast<uint4*>(to) = make_uint4(Pack<T>::two(v[0], v[1]), Pack<T>::two(v[2], v[3]),
                                                 Pack<T>::two(v[4], v[5]), Pack<T>::two(v[6], v[7]));
    };

    const bool turns_any = nf > 0 && j0 < p.h_q + p.h_k;
    const bool held = n <= chunk_rows;
    if (!held && j1 > p.h_q && stored) {
      // ---- more rows than the registers hold: their largest values first
      for (int j = j0 + warp; j < j1; j += kWarps)
        if (lane == 0 && j >= p.h_q) s_top[j - p.h_q] = 0.f;
      for (int t0 = 0; t0 < n; t0 += chunk_rows) {
        if (turns_any) turn_rows(t0);
        for (int j = j0 + warp; j < j1; j += kWarps) {
          if (j < p.h_q) continue;
          const bool is_v = j >= p.h_q + p.h_k;
          const int head = j - p.h_q - (is_v ? p.h_k : 0);
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < kHeld; ++i) {
            const int r = r0 + i * rpw;
            float v[8];
            if (on && t0 + r < n) {
              take(is_v ? p.v : p.k, head, !is_v && nf > 0, t0, r, v);
              top = largest(v, top);
            }
          }
#pragma unroll
          for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
          if (lane == 0) s_top[j - p.h_q] = fmaxf(s_top[j - p.h_q], top);
          __syncwarp();
        }
      }
    }
    for (int t0 = 0; t0 < n; t0 += chunk_rows) {
      if (turns_any) turn_rows(t0);
      for (int j = j0 + warp; j < j1; j += kWarps) {
        const bool is_q = j < p.h_q, is_v = j >= p.h_q + p.h_k;
        const int head = is_q ? j : j - p.h_q - (is_v ? p.h_k : 0);
        if (!is_q && !stored) continue;
        const TensorArg& in = is_q ? p.q : (is_v ? p.v : p.k);
        float v[kHeld][8];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int r = r0 + i * rpw;
          if (on && t0 + r < n) {
            take(in, head, !is_v && nf > 0, t0, r, v[i]);
            top = largest(v[i], top);
          }
        }
        if (is_q) {
          __syncwarp();  // every lane has read its pairs' other elements: oq may be q
#pragma unroll
          for (int i = 0; i < kHeld; ++i)
            if (on && t0 + r0 + i * rpw < n) put16(head, t0 + r0 + i * rpw, v[i]);
          continue;
        }
        const TensorArg& pages = is_v ? p.cache.pages.v : p.cache.pages.k;
        float* scales = is_v ? p.cache.v_scale : p.cache.k_scale;
        float inv;
        if (t0 == 0) {
          inv = settle(pages, scales, is_v ? p.cache.vs : p.cache.ks, head, held ? top : s_top[j - p.h_q]);
          if (!held) {
            __syncwarp();
            if (lane == 0) s_top[j - p.h_q] = inv;
            __syncwarp();
          }
        } else {
          inv = s_top[j - p.h_q];
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (on && t0 + r0 + i * rpw < n) put8(pages, head, t0 + r0 + i * rpw, v[i], inv);
      }
    }
  }
}

// A warp a token: rows of k and v of all heads, 16 codes a lane.
template <typename T, bool INT8>
__global__ void __launch_bounds__(kThreads) load8_kernel(Load8Params p, FastDiv per_row) {
  const int lane = threadIdx.x & 31;
  const int chunks = p.h_k * static_cast<int>(per_row.d);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.batch; i += kThreads)
      if (p.cu[i] < 0 || p.cu[i] > p.cu[i + 1]) report(p.status, kBadOffsets);
  for (int t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < p.tokens; t += gridDim.x * kWarps) {
    int lo = 0, hi = p.batch;  // the last sequence that starts at or before t, 32 probes a step
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, probe = min(lo + lane * step, hi - 1);
      const int n = __popc(__ballot_sync(0xffffffffu, p.cu[probe] <= t));
      lo = min(lo + max(n - 1, 0) * step, hi - 1);
      hi = min(lo + step, hi);
    }
    const int b = lo, c0 = p.cu[b], c1 = p.cu[b + 1];
    if (t >= p.cu[p.batch]) continue;  // behind the last sequence
    if (c0 < 0 || t < c0 || t >= c1) {
      if (lane == 0) report(p.status, kBadOffsets);
      continue;
    }
    const int start = p.starts[b];
    const int64_t slot = static_cast<int64_t>(start) + (t - c0);
    const int64_t cap = static_cast<int64_t>(p.cache.pages.max_pages) * p.cache.pages.page.d;
    int page = -1, within = 0;
    if (start < 0 || slot >= cap) {
      if (lane == 0) report(p.status, kBadLength);
    } else if (!page_of(p.cache.pages, p.cache.pages.table + b * p.cache.pages.table_stride, static_cast<int>(slot),
                        page, within, p.status)) {
      page = -1;
    }
    const int64_t blk = p.cache.block.div(static_cast<uint32_t>(within));
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const TensorArg& in = kind ? p.cache.pages.v : p.cache.pages.k;
      const TensorArg& out = kind ? p.v : p.k;
      const int64_t* st = kind ? p.cache.vs : p.cache.ks;
      const float* scales = (kind ? p.cache.v_scale : p.cache.k_scale) + page * st[0] + blk * st[1];
      const char* rows = static_cast<const char*>(in.ptr) + page * in.sb + within * in.ss;
      T* to = static_cast<T*>(const_cast<void*>(out.ptr)) + t * out.ss;
      for (int i = lane; i < chunks; i += 32) {
        const int head = static_cast<int>(per_row.div(i)), c = i - head * static_cast<int>(per_row.d);
        uint4 codes = make_uint4(0, 0, 0, 0);
        float s = 0.f;
        if (page >= 0) {
          codes = *reinterpret_cast<const uint4*>(rows + head * in.sh + c * 16);
          s = scales[head * st[2]];
        }
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&codes);
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 y = value4<INT8>(w[k]);
          o[2 * k] = Pack<T>::two(y.x * s, y.y * s);
          o[2 * k + 1] = Pack<T>::two(y.z * s, y.w * s);
        }
        uint4* dst = reinterpret_cast<uint4*>(to + head * out.sh + c * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

template <typename T, bool INT8>
cudaError_t launch_append(const Append8Params& p, cudaStream_t stream) {
  Append8Grid g;
  const int chunks = p.head_dim / 8, nf = p.rot.n_freq;
  g.lanes_log2 = 0;
  while ((1 << g.lanes_log2) < chunks) ++g.lanes_log2;
  g.mode = p.rot.positions == nullptr ? kNoTurn : (p.rot.interleaved ? kPairs : (nf % 8 == 0 ? kHalves : kMixed));
  const int64_t most = static_cast<int64_t>(num_sms()) * kBlocks;
  const int64_t seqs = p.batch < p.tokens ? p.batch : p.tokens;
  int64_t units = p.tokens / static_cast<int64_t>(p.cache.block.d) + 2 * seqs;
  if (units > p.tokens) units = p.tokens;
  // few blocks of tokens: several blocks share the heads of each, down to one for each warp
  const int64_t jobs = static_cast<int64_t>(p.h_q) + 2 * static_cast<int64_t>(p.h_k);
  const int64_t fit = (jobs + kWarps - 1) / kWarps;
  int64_t parts = most / units;
  parts = parts < 1 ? 1 : (parts > fit ? fit : parts);
  g.parts = static_cast<int>(parts);
  const int64_t grid = units * parts;
  const size_t smem = static_cast<size_t>(p.h_k) * 2 * sizeof(float);
  append8_kernel<T, INT8><<<static_cast<unsigned>(grid < most ? grid : most), kThreads, smem, stream>>>(p, g);
  return cudaGetLastError();
}

template <typename T, bool INT8>
cudaError_t launch_load(const Load8Params& p, cudaStream_t stream) {
  FastDiv per_row;
  per_row.set(static_cast<uint32_t>(p.head_dim / 16));
  const int64_t grid = (static_cast<int64_t>(p.tokens) + kWarps - 1) / kWarps, most = static_cast<int64_t>(num_sms()) * 8;
  load8_kernel<T, INT8><<<static_cast<unsigned>(grid < most ? grid : most), kThreads, 0, stream>>>(p, per_row);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append8(const Append8Params& p, cudaStream_t stream) {
  if (p.cache.int8)
    return p.bf16 ? launch_append<__nv_bfloat16, true>(p, stream) : launch_append<__half, true>(p, stream);
  return p.bf16 ? launch_append<__nv_bfloat16, false>(p, stream) : launch_append<__half, false>(p, stream);
}

cudaError_t launch_load8(const Load8Params& p, cudaStream_t stream) {
  if (p.cache.int8) return p.bf16 ? launch_load<__nv_bfloat16, true>(p, stream) : launch_load<__half, true>(p, stream);
  return p.bf16 ? launch_load<__nv_bfloat16, false>(p, stream) : launch_load<__half, false>(p, stream);
}

}  // namespace attn
