// The append to a cache in 8 bits (attn_cache_append8) and its read-back (attn_cache_load8).
//
// A block of tokens of a page has, for each head, one factor s, a power of two; its codes c stand
// for c s.  An append takes the smallest s with |x| <= top s for every new value x of the block
// (top = 448 for e4m3, 127 for int8), but not less than the factor of the block's earlier tokens;
// where s grows, their codes are rounded to it again.  With powers of two a value of e4m3 only
// changes then where it leaves the normal range, and x / s is exact, so that a code is off by one
// rounding of x.
//
// Append.  A block of threads takes the new tokens of one block of the cache, which lie in one page
// (its tokens' block divides the page), and eight rows of heads of q, k or v, one a warp.  A warp
// asks for its rows first (up to kHeld 16-byte chunks of a lane), then the block's threads compute
// the turns of the tokens, and the rows stay in registers as they came: they are turned once for
// their largest value and once more when they are rounded, so that k and v are read once.
// Warps share the tokens of a row of heads where they are more; what is beyond that, too, is read a
// second time, from the L2.  Of 19014 tokens of 16 + 16 heads of 96 (85 us for a floor of 43) issue slots
// are busy for 58 % of the time, which leaves latencies that 16 warps an SM do not cover, as many as
// 128 registers leave.  (Eight chunks a lane and three blocks an SM: 110 us; rows behind the last
// one read again in place of zeros: 93; a row of heads for every warp of every block, without the loop
// over heads: 157.)
// Read-back.  A warp takes a token: 8 codes a lane, 16 bytes out, so that a warp's stores are whole
// lines: bound by the memory (8 sequences up to 8192 tokens of 8 heads of 128 43.5 us, 87 % of the copy
// bandwidth; with 16 codes a lane, two half-written sectors of 32 bytes at a time, 50).
#include <atomic>
#include <type_traits>

#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 16;      // chunks of a lane in registers
constexpr int kTurns = 2048;   // turns of the rows that a warp takes at once
constexpr int kBlocks = 2;     // of an SM
constexpr int kMostShares = 2; // log2 of the warps that share tokens
constexpr int kLoads = 4;      // of a lane and of each of k and v, in a read-back
constexpr float kLargest = 1.152921504606847e18f;    // 2^60

// Chunks before which a lane looks whether there are more: the work of those between is mixed.
__device__ constexpr bool looks(int i) { return i == 1 || i == 2 || i % 4 == 0; }

// Where the other element of a pair is: kHalves in the lane n_freq / 8 further (n_freq a multiple
// of 8), kPairs in the lane's own chunk, kMixed anywhere, read once more.  kCutPairs: kPairs where n_freq is
// no multiple of 4, so that a chunk holds pairs that turn and others (a form of its own: that case in
// kPairs takes 10 to 12 % more time of interleaved prompts, 87 -> 97 us).
enum RopeMode { kNoTurn = 0, kHalves = 1, kPairs = 2, kMixed = 3, kCutPairs = 4 };

struct Append8Grid {
  int lanes_log2;        // lanes of a row
  int share_log2;        // warps that share the tokens of a row of heads
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

// The codes of x inv.  kClean: of int8, all x are finite and none is beyond the largest code.
template <bool INT8, bool kClean = false>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float inv) {
  if (INT8) {
    // 1.5 2^23 more: the sum's last bits are the rounded number
    auto one = [&](float x) {
      if (kClean) return __float_as_uint(fmaf(x, inv, 12582912.f));
      return static_cast<uint32_t>(min(max(__float2int_rn(x * inv), -127), 127));
    };
    return __byte_perm(__byte_perm(one(a), one(b), 0x0040), __byte_perm(one(c), one(d), 0x0040), 0x5410);
  }
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// A result y that was rounded to 24 bits, given what is left of it (only the sign counts): the number
// with an odd last bit next to it.  That rounds on to the few bits of a code or a 16-bit type, and at
// their ties, as the exact result does.
__device__ __forceinline__ float odd_of(float y, float left) {
  const uint32_t u = __float_as_uint(y);
  if (!(left < 0.f || left > 0.f) || y == 0.f) return y;
  return __uint_as_float(((u ^ __float_as_uint(left)) >> 31) == 0 ? u | 1u : (u - 1u) | 1u);
}
__device__ __forceinline__ float times(float x, float f) {
  const float y = x * f;
  return odd_of(y, fmaf(x, f, -y));
}
// x / f, given 1 / f: the quotient is put right by what is left, so that it is next to the exact one.
__device__ __forceinline__ float over(float x, float f, float inv) {
  const float y = x * inv;
  if (!(fabsf(y) < INFINITY)) return y;
  const float z = fmaf(fmaf(-y, f, x), inv, y);
  return odd_of(z, fmaf(-z, f, x));
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

// The largest of three magnitudes, NaN where one is.
__device__ __forceinline__ float most_of(float top, float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(top));
  return y;
}
__device__ __forceinline__ uint32_t most_of(uint32_t top, uint32_t w, __nv_bfloat16) {
  const __nv_bfloat162 y = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&top), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t most_of(uint32_t top, uint32_t w, __half) {
  const __half2 y = __hmax2_nan(*reinterpret_cast<const __half2*>(&top), __habs2(*reinterpret_cast<const __half2*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Barrier of the warps that share a row of heads.
__device__ __forceinline__ void share_barrier(int which, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(which + 1), "r"(threads) : "memory");
}

template <typename T, bool INT8, int MODE>
__global__ void __launch_bounds__(kThreads, kBlocks) append8_kernel(Append8Params p, Append8Grid g) {
  extern __shared__ __align__(16) float2 cs[];  // (cos, sin) of [row][frequency]
  __shared__ unsigned long long turns[128];
  __shared__ int64_t s_pre[kThreads];  // (offsets that do not ascend may name a token often)
  __shared__ int64_t s_sums[kWarps];
  __shared__ int4 s_fresh[kThreads];   // of the first sequence of each thread: first, n, len, bad
  __shared__ float2 s_top[2][kWarps];  // largest value and whether all are finite, of every other row of heads
  const int tid = threadIdx.x, lane = tid & 31, warp = static_cast<int>(warp_id());  // (uniform to the compiler)
  // turns of a row: up to a multiple of 4, the last ones by nothing
  const int nf = MODE == kNoTurn ? 0 : p.rot.n_freq, pitch = MODE == kNoTurn ? 4 : (nf + 3) / 4 * 4;

  const float inv_freq = tid < nf ? p.rot.inv_freq[tid] : 0.f;  // (at most 128)
  // ---- blocks of the sequences before this thread's
  const int per = (p.batch + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int i = 0; i < per && tid * per + i < p.batch; ++i) {
    const Fresh f = fresh_of(p, tid * per + i, blockIdx.x == 0);
    if (i == 0) s_fresh[tid] = make_int4(f.first, f.n, f.len, f.bad);
    mine += blocks_of(p, f);
  }
  int64_t x = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  if (lane == 31) s_sums[warp] = x;
  if (tid < nf) {  // fraction of a turn that one position adds at each frequency, times 2^64
    const double y = static_cast<double>(inv_freq) * 0.15915494309189535;
    turns[tid] = static_cast<unsigned long long>((y - floor(y)) * 18446744073709551616.0);
  }
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? s_sums[w] : 0;
    total += s_sums[w];
  }
  s_pre[tid] = before + x - mine;
  __syncthreads();

  const int lanes = 1 << g.lanes_log2, rpw = 32 >> g.lanes_log2, chunk_rows = (kHeld * rpw) << g.share_log2;
  // this warp's first row of a chunk, and this lane's
  const int member = warp & ((1 << g.share_log2) - 1), w0 = member * kHeld * rpw;
  const int c = lane & (lanes - 1), r0 = w0 + (lane >> g.lanes_log2), at = 8 * c;
  int parity = 0;
  const bool on = at < p.head_dim;
  const int jobs = p.h_q + 2 * p.h_k, at_once = kWarps >> g.share_log2;
  const int64_t items = total * g.parts;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t u = g.parts == 1 ? item : item / g.parts;
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
    const int4 held_fresh = s_fresh[lo];
    Fresh f{held_fresh.x, held_fresh.y, held_fresh.z, held_fresh.w != 0};
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
    bool stored = !f.bad && base < cap;
    int page = 0, within = 0;
    if (stored) {
      const int pg = static_cast<int>(p.cache.pages.page.div(static_cast<uint32_t>(base)));
      within = static_cast<int>(base) - pg * static_cast<int>(p.cache.pages.page.d);
      page = p.cache.pages.table[b * p.cache.pages.table_stride + pg];
    }
    const bool held = n <= chunk_rows;

    // ---- rows of heads, one a warp (or a part of it) at a time
    int j = j0 + (warp >> g.share_log2), head;
    bool is_q, is_v, turned;
    const T* src;      // this lane's element of the row of heads, of its first token
    int64_t row_step;
    uint4 raw[kHeld];
    auto ask = [&](int t0) {
      const int rows = on && j < j1 ? n - t0 - r0 : 0;
      const T* s = src + t0 * (row_step >> (5 - g.lanes_log2));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        raw[i] = i * rpw < rows ? *reinterpret_cast<const uint4*>(s) : make_uint4(0, 0, 0, 0);
        s += row_step;
      }
    };
    auto begin = [&]() {
      is_q = j < p.h_q;
      is_v = j >= p.h_q + p.h_k;
      turned = MODE != kNoTurn && !is_v;
      head = is_q ? j : j - p.h_q - (is_v ? p.h_k : 0);
      const TensorArg& in = is_q ? p.q : (is_v ? p.v : p.k);
      row_step = in.ss * rpw;
      src = static_cast<const T*>(in.ptr) + static_cast<int64_t>(token0 + r0) * in.ss + head * in.sh + at;
      ask(0);
    };
    begin();

    // The turns of the rows [t0, t0 + chunk_rows), where the block has rows that turn.
    const bool any_turns = MODE != kNoTurn && j0 < p.h_q + p.h_k;
    auto turn_rows = [&](int t0) {
      if (MODE == kNoTurn || !any_turns) return;
      __syncthreads();
      const int rows = min(chunk_rows, n - t0);
      for (int i = tid; i < rows * pitch; i += kThreads) {
        const int r = i / pitch, fr = i - r * pitch;
        float sn = 0.f, cn = 1.f;
        if (fr < nf) {
          int axis = 0;
#pragma unroll
          for (int a = 0; a < 3; ++a) axis += fr >= p.rot.end[a] ? 1 : 0;
          const long long pos = p.rot.positions[axis * p.rot.axis_stride + token0 + t0 + r];
          const unsigned long long phase = static_cast<unsigned long long>(pos) * turns[fr];
          sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &sn, &cn);
        }
        cs[i] = make_float2(cn, sn);
      }
      __syncthreads();
    };
    if (held) turn_rows(0);
    if (stored && static_cast<unsigned>(page) >= static_cast<unsigned>(p.cache.pages.num_pages)) {
      if (tid == 0 && part == 0) report(p.status, kBadPage);
      stored = false;
    } else if (!stored && !f.bad) {
      if (tid == 0 && part == 0) report(p.status, kBadLength);
    }
    const int64_t blk = p.cache.block.div(static_cast<uint32_t>(within));

    // The elements of chunk i of this lane (of the rows from t0 on), turned.
    constexpr bool kInPairs = MODE == kPairs || MODE == kCutPairs;
    const int f0 = kInPairs ? at / 2 : (at >= nf ? at - nf : at);
    const float side = at >= nf ? 1.f : -1.f;
    const bool in_turns = at < 2 * nf;
    const int other_lane = MODE != kHalves || !in_turns ? lane : (at >= nf ? lane - nf / 8 : lane + nf / 8);
    auto take = [&](int i, int t0, float (&v)[8]) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 y = Pack<T>::unpack(w[k]);
        v[2 * k] = y.x;
        v[2 * k + 1] = y.y;
      }
      if (MODE == kNoTurn || !turned) return;
      const int r = min(r0 + i * rpw, n - t0 - 1);  // (what is not a row is zeros)
      const float2* t = cs + r * pitch;
      if (MODE == kHalves) {
        uint32_t ow[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) ow[k] = __shfl_sync(0xffffffffu, w[k], other_lane);
        if (in_turns) {
          const float4* t4 = reinterpret_cast<const float4*>(t + f0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 y = Pack<T>::unpack(ow[k]);
            const float4 a = t4[k];
            v[2 * k] = v[2 * k] * a.x + y.x * (side * a.y);
            v[2 * k + 1] = v[2 * k + 1] * a.z + y.y * (side * a.w);
          }
        }
      } else if (kInPairs) {
        if (in_turns) {
          const float4* t4 = reinterpret_cast<const float4*>(t + f0);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 a = t4[k];
            const float x0 = v[4 * k], x1 = v[4 * k + 1], x2 = v[4 * k + 2], x3 = v[4 * k + 3];
            v[4 * k] = x0 * a.x - x1 * a.y;
            v[4 * k + 1] = x0 * a.y + x1 * a.x;
            v[4 * k + 2] = x2 * a.z - x3 * a.w;
            v[4 * k + 3] = x2 * a.w + x3 * a.z;
            if (MODE == kCutPairs) {  // pairs behind the last that turns stay: not even 0 x infinity is added
              if (f0 + 2 * k >= nf) v[4 * k] = x0, v[4 * k + 1] = x1;
              if (f0 + 2 * k + 1 >= nf) v[4 * k + 2] = x2, v[4 * k + 3] = x3;
            }
          }
        }
      } else if (in_turns && t0 + r0 + i * rpw < n) {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(src + t0 * (row_step >> (5 - g.lanes_log2)) + i * row_step) - at;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int e = at + k;
          if (e < 2 * nf) {
            const float y = Pack<T>::unpack(static_cast<uint32_t>(row[e < nf ? e + nf : e - nf])).x;
            const float2 a = t[e < nf ? e : e - nf];
            v[k] = v[k] * a.x + y * (e < nf ? -a.y : a.y);
          }
        }
      }
    };
    auto pack16 = [&](const float (&v)[8]) {
      return make_uint4(Pack<T>::two(v[0], v[1]), Pack<T>::two(v[2], v[3]), Pack<T>::two(v[4], v[5]), Pack<T>::two(v[6], v[7]));
    };

    const int rounds = (j1 - j0 + at_once - 1) / at_once;  // the same for all warps: some steps are block-wide
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
      if (round > 0) {
        j += at_once;
        begin();
      }
      // of k and v: the factor of the block's earlier tokens
      float* factor = nullptr;
      float was = 0.f;
      if (stored && !is_q && j < j1) {
        const int64_t* st = is_v ? p.cache.vs : p.cache.ks;
        factor = (is_v ? p.cache.v_scale : p.cache.k_scale) + page * st[0] + blk * st[1] + head * st[2];
        if (old > 0) was = *factor;
      }
      float top = 0.f, now = 0.f, inv = 0.f;
      bool clean = true;  // all are finite
      char* to = nullptr;
      int64_t step = 0;
      // Tokens that are not held pass twice: for their largest value, and to be rounded.
      const int passes = held ? 1 : 2;
#pragma unroll 1
      for (int pass = 0; pass < passes; ++pass) {
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += chunk_rows) {
          if (!held) {
            if (pass > 0 || t0 > 0) ask(t0);
            turn_rows(t0);
          }
          // chunks of this warp's lanes that hold a row, and of this lane
          const int left = max(n - t0 - w0 + rpw - 1, 0) >> (5 - g.lanes_log2);
          const int rows = on && j < j1 ? max(n - t0 - r0 + rpw - 1, 0) >> (5 - g.lanes_log2) : 0;
          if (is_q) {
            if (pass > 0) continue;
            T* out = static_cast<T*>(const_cast<void*>(p.oq.ptr)) + static_cast<int64_t>(token0 + t0 + r0) * p.oq.ss +
                     head * p.oq.sh + at;
            const int64_t out_step = p.oq.ss * rpw;
            if (MODE == kMixed) {  // every lane reads its pairs' other elements before one is written: oq may be q
#pragma unroll
              for (int i = 0; i < kHeld; ++i) {
                float v[8];
                take(i, t0, v);
                raw[i] = pack16(v);
              }
              __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
              if (looks(i) && i >= left) break;
              if (MODE != kMixed) {
                float v[8];
                take(i, t0, v);
                raw[i] = pack16(v);
              }
              if (i < rows) *reinterpret_cast<uint4*>(out) = raw[i];
              out += out_step;
            }
            continue;
          }
          if (pass == 0) {
            // ---- the largest value of the new tokens (rows that are none are zeros)
            float most = 0.f;  // NaN where one is
            if (!turned) {
              uint32_t two = 0;
#pragma unroll
              for (int i = 0; i < kHeld; ++i) {
                if (looks(i) && i >= left) break;
                two = most_of(most_of(most_of(most_of(two, raw[i].x, T()), raw[i].y, T()), raw[i].z, T()), raw[i].w, T());
              }
              const float2 y = Pack<T>::unpack(two);
              most = most_of(0.f, y.x, y.y);
            } else {
#pragma unroll
              for (int i = 0; i < kHeld; ++i) {
                if (looks(i) && i >= left) break;
                float v[8];
                take(i, t0, v);
#pragma unroll
                for (int k = 0; k < 8; k += 2) most = most_of(most, v[k], v[k + 1]);
              }
            }
            const bool fine = most < INFINITY;
            if (fine) top = fmaxf(top, most);
            if (__any_sync(0xffffffffu, !fine)) {  // the finite ones, one by one
              clean = false;
#pragma unroll
              for (int i = 0; i < kHeld; ++i) {
                if (looks(i) && i >= left) break;
                float v[8];
                take(i, t0, v);
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fabsf(v[k]) < INFINITY ? fmaxf(top, fabsf(v[k])) : top;
              }
            }
            if (!held) continue;
          }
          if (held || t0 == 0) {
            // ---- the head's factor; its earlier codes follow it
            top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
            if (g.share_log2 > 0) {
              if (lane == 0) s_top[parity][warp] = make_float2(top, clean ? 1.f : 0.f);
              share_barrier(warp >> g.share_log2, 32 << g.share_log2);
              for (int i = 0; i < 1 << g.share_log2; ++i) {
                const float2 other = s_top[parity][warp - member + i];
                top = fmaxf(top, other.x);
                clean = clean && other.y != 0.f;
              }
              parity ^= 1;
            }
            const TensorArg& pages = is_v ? p.cache.pages.v : p.cache.pages.k;
            to = static_cast<char*>(const_cast<void*>(pages.ptr)) + page * pages.sb + within * pages.ss + head * pages.sh;
            was = was > 0.f ? fminf(was, kLargest) : 0.f;
            now = factor_of<INT8>(top);
            if (factor != nullptr && now > was && old > 0) {
              const float ratio = was / now;  // (0 where they stood for zeros)
              const int per_row = p.head_dim / 16;
              for (int i = lane + 32 * member; i < old * per_row; i += 32 << g.share_log2) {
                const int r = i / per_row;
                uint4* at16 = reinterpret_cast<uint4*>(to + r * pages.ss) + (i - r * per_row);
                uint4 codes = *at16;
                uint32_t* w = reinterpret_cast<uint32_t*>(&codes);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float4 y = value4<INT8>(w[k]);
                  w[k] = code4<INT8>(times(y.x, ratio), times(y.y, ratio), times(y.z, ratio), times(y.w, ratio), 1.f);
                }
                *at16 = codes;
              }
            }
            now = fmaxf(now, was);
            if (factor != nullptr && lane == 0 && member == 0) *factor = now;
            inv = 1.f / now;
            clean = clean && now < kLargest;  // a factor at its upper bound leaves values beyond the largest code
            to += (old + r0) * pages.ss + at;
            step = pages.ss * rpw;
          }
          // ---- codes
          char* out = to + t0 * (step >> (5 - g.lanes_log2));
          const int stores = factor != nullptr ? rows : 0;
          // x / s is a product where s is a power of two, which an earlier factor need not be
          const bool power = (__float_as_uint(now) & 0x7fffffu) == 0;
          auto put = [&](auto fits) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
              if (looks(i) && i >= left) break;
              float v[8];
              take(i, t0, v);
              if (!fits.value && !power)
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = over(v[k], now, inv);
              const float mul = !fits.value && !power ? 1.f : inv;
              if (i < stores)
                *reinterpret_cast<uint2*>(out) = make_uint2(code4<INT8, fits.value>(v[0], v[1], v[2], v[3], mul),
                                                            code4<INT8, fits.value>(v[4], v[5], v[6], v[7], mul));
              out += step;
            }
          };
          if (power && (!INT8 || clean)) put(std::true_type());
          else put(std::false_type());
        }
      }
    }
  }
}

// A warp a token: rows of k and v of all heads, 8 codes a lane and kLoads of these on their way.
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
    const char* rows[2];
    const float* scales[2];
    T* to[2];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const TensorArg& in = kind ? p.cache.pages.v : p.cache.pages.k;
      const TensorArg& out = kind ? p.v : p.k;
      const int64_t* st = kind ? p.cache.vs : p.cache.ks;
      scales[kind] = (kind ? p.cache.v_scale : p.cache.k_scale) + page * st[0] + blk * st[1];
      rows[kind] = static_cast<const char*>(in.ptr) + page * in.sb + within * in.ss;
      to[kind] = static_cast<T*>(const_cast<void*>(out.ptr)) + t * out.ss;
    }
    for (int i0 = lane; i0 < chunks; i0 += 32 * kLoads) {
      uint2 codes[kLoads][2];
      float s[kLoads][2];
      bool twice = false;  // a factor is no power of two: fp32 may round its products, and the type once more
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = i0 + 32 * k, head = static_cast<int>(per_row.div(i)), c = i - head * static_cast<int>(per_row.d);
        codes[k][0] = codes[k][1] = make_uint2(0, 0);
        s[k][0] = s[k][1] = 0.f;
        if (i < chunks && page >= 0) {
          codes[k][0] = __ldcs(reinterpret_cast<const uint2*>(rows[0] + head * p.cache.pages.k.sh + c * 8));
          codes[k][1] = __ldcs(reinterpret_cast<const uint2*>(rows[1] + head * p.cache.pages.v.sh + c * 8));
          s[k][0] = scales[0][head * p.cache.ks[2]];
          s[k][1] = scales[1][head * p.cache.vs[2]];
        }
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = i0 + 32 * k, head = static_cast<int>(per_row.div(i)), c = i - head * static_cast<int>(per_row.d);
        if (i >= chunks) break;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          const float f = s[k][kind];
          const float4 x = value4<INT8>(codes[k][kind].x), y = value4<INT8>(codes[k][kind].y);
          *reinterpret_cast<uint4*>(to[kind] + head * (kind ? p.v.sh : p.k.sh) + c * 8) =
              make_uint4(Pack<T>::two(x.x * f, x.y * f), Pack<T>::two(x.z * f, x.w * f), Pack<T>::two(y.x * f, y.y * f),
                         Pack<T>::two(y.z * f, y.w * f));
          twice = twice || (__float_as_uint(f) & 0x7fffffu) != 0;
        }
      }
      // (done again here: in place it takes registers, 64 -> 70, and time of all factors, 46.1 -> 46.9 us for 41800 tokens)
      if (!twice) continue;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind)
#pragma unroll 1
        for (int i = i0; i < min(chunks, i0 + 32 * kLoads); i += 32) {
          const int head = static_cast<int>(per_row.div(i)), c = i - head * static_cast<int>(per_row.d);
          const uint2 z = *reinterpret_cast<const uint2*>(rows[kind] + head * (kind ? p.cache.pages.v.sh : p.cache.pages.k.sh) + c * 8);
          const float f = scales[kind][head * (kind ? p.cache.vs[2] : p.cache.ks[2])];
          const float4 x = value4<INT8>(z.x), y = value4<INT8>(z.y);
          *reinterpret_cast<uint4*>(to[kind] + head * (kind ? p.v.sh : p.k.sh) + c * 8) =
              make_uint4(Pack<T>::two(times(x.x, f), times(x.y, f)), Pack<T>::two(times(x.z, f), times(x.w, f)),
                         Pack<T>::two(times(y.x, f), times(y.y, f)), Pack<T>::two(times(y.z, f), times(y.w, f)));
        }
    }
  }
}

template <typename T, bool INT8, int MODE>
cudaError_t launch_mode(const Append8Params& p, const Append8Grid& g, unsigned grid, size_t smem, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};  // devices with the attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (MODE != kNoTurn && (!(done.load(std::memory_order_relaxed) & bit) || bit == 0)) {
    e = cudaFuncSetAttribute(append8_kernel<T, INT8, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kTurns * static_cast<int>(sizeof(float2)) << kMostShares);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  append8_kernel<T, INT8, MODE><<<grid, kThreads, smem, stream>>>(p, g);
  return cudaGetLastError();
}

template <typename T, bool INT8>
cudaError_t launch_append(const Append8Params& p, cudaStream_t stream) {
  Append8Grid g;
  const int chunks = p.head_dim / 8, nf = p.rot.n_freq;
  g.lanes_log2 = 0;
  while ((1 << g.lanes_log2) < chunks) ++g.lanes_log2;
  const int mode = p.rot.positions == nullptr ? kNoTurn : (p.rot.interleaved ? (nf % 4 == 0 ? kPairs : kCutPairs) : (nf % 8 == 0 ? kHalves : kMixed));
  const int64_t most = static_cast<int64_t>(num_sms()) * kBlocks;
  const int64_t seqs = p.batch < p.tokens ? p.batch : p.tokens;
  int64_t units = p.tokens / static_cast<int64_t>(p.cache.block.d) + 2 * seqs;
  if (units > p.tokens) units = p.tokens;
  // Warps share the tokens of a row of heads where a block of the cache gets more of them than one
  // holds (as many as a sequence has on average).
  const int64_t rows = p.tokens / seqs < p.cache.block.d ? (p.tokens + seqs - 1) / seqs : p.cache.block.d;
  g.share_log2 = 0;
  while (g.share_log2 < kMostShares && ((kHeld << 5 >> g.lanes_log2) << g.share_log2) < rows) ++g.share_log2;
  // few blocks of tokens: several blocks share the heads of each, down to one for each warp; many:
  // a block of tokens is cut so that about four pieces come to each block
  const int64_t jobs = static_cast<int64_t>(p.h_q) + 2 * static_cast<int64_t>(p.h_k);
  const int at_once = kWarps >> g.share_log2;
  const int64_t fit = (jobs + at_once - 1) / at_once;
  int64_t parts = units < most ? most / units : 4 * most / units;
  parts = parts < 1 ? 1 : (parts > fit ? fit : parts);
  g.parts = static_cast<int>(parts);
  const int64_t items = units * parts;
  const unsigned grid = static_cast<unsigned>(items < most ? items : most);
  const size_t smem = mode == kNoTurn ? 0 : (kTurns * sizeof(float2)) << g.share_log2;
  switch (mode) {
    case kNoTurn: return launch_mode<T, INT8, kNoTurn>(p, g, grid, smem, stream);
    case kHalves: return launch_mode<T, INT8, kHalves>(p, g, grid, smem, stream);
    case kPairs: return launch_mode<T, INT8, kPairs>(p, g, grid, smem, stream);
    case kCutPairs: return launch_mode<T, INT8, kCutPairs>(p, g, grid, smem, stream);
    default: return launch_mode<T, INT8, kMixed>(p, g, grid, smem, stream);
  }
}

template <typename T, bool INT8>
cudaError_t launch_load(const Load8Params& p, cudaStream_t stream) {
  FastDiv per_row;
  per_row.set(static_cast<uint32_t>(p.head_dim / 8));
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
