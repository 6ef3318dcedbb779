// Rotary positions of q and k (attn_rope) and the append to the paged
// key/value cache (attn_cache_append): one kernel, since the append is the
// rotation with k going to pages instead of ok and v copied beside it.
//
// Pair i of a token's head row is turned by angle = position * inv_freq[i]:
//   (x, y) -> (x cos - y sin, x sin + y cos);
// the gradient is the same with -sin.  A block takes a few tokens with all their
// heads and computes each token's n_freq sines and cosines once, into shared
// memory, so the heads cost two FMAs and a rounding an element and the kernel is
// bound by the memory it streams: every row is read once and written once, 16
// bytes a thread.
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
constexpr int kMaxTile = 16;  // tokens of a block

enum RopeMode { kHalves = 0, kPairs = 1, kScalar = 2 };

struct RopeGrid {
  int tile;          // tokens of a block
  FastDiv per_token; // units of a token: (h_q + h_k) * per_row + (append) h_k * chunks
  FastDiv per_row;   // units of a rotated row
  FastDiv chunks;    // 16-byte chunks of a row
  int rot_units;     // units of a row that turn pairs (the rest copies)
  FastDiv seq;       // seqlen (padded tensors)
};

template <typename T>
__device__ __forceinline__ void turn8(uint4& lo, uint4& hi, const float2* cs, float sign) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
  uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Pack<T>::unpack(a[i]), y = Pack<T>::unpack(b[i]);
    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
    const float s0 = c0.y * sign, s1 = c1.y * sign;
    a[i] = Pack<T>::two(x.x * c0.x - y.x * s0, x.y * c1.x - y.y * s1);
    b[i] = Pack<T>::two(x.x * s0 + y.x * c0.x, x.y * s1 + y.y * c1.x);
  }
}

template <typename T>
__device__ __forceinline__ void turn_pairs(uint4& v, const float2* cs, float sign) {
  uint32_t* a = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = Pack<T>::unpack(a[i]);
    const float2 c = cs[i];
    const float s = c.y * sign;
    a[i] = Pack<T>::two(x.x * c.x - x.y * s, x.x * s + x.y * c.x);
  }
}

struct TokenInfo {
  int64_t k_off, v_off;  // element offsets of the token's slot (head 0) in the cache
  int seq, slot;         // slot < 0: not stored
  int live;              // belongs to a sequence
};

// Sequence and slot of new token t, with every device-side check.
__device__ void locate(const RopeParams& p, int64_t t, TokenInfo& out) {
  out.live = 0;
  out.slot = -1;
  int b = static_cast<int>(t), i = 0;
  if (p.cu != nullptr) {
    b = seq_of_row(p.cu, p.batch, static_cast<int>(t));
    const int c0 = p.cu[b], c1 = p.cu[b + 1];
    if (t >= p.cu[p.batch]) return;  // behind the last sequence
    if (t < c0 || t >= c1) {
      report(p.status, kBadOffsets);
      return;
    }
    i = static_cast<int>(t) - c0;
  }
  out.live = 1;
  out.seq = b;
  const int n = p.seqlens[b];
  const int64_t slot = static_cast<int64_t>(n) + i;
  const int64_t cap = static_cast<int64_t>(p.cache.max_pages) * p.cache.page.d;
  if (n < 0 || slot >= cap || (p.slot_positions != nullptr && slot >= p.slots_stride)) {
    report(p.status, kBadLength);
    return;
  }
  int page, within;
  if (!page_of(p.cache, p.cache.table + b * p.cache.table_stride, static_cast<int>(slot), page,
               within, p.status))
    return;
  out.slot = static_cast<int>(slot);
  out.k_off = page * p.cache.k.sb + within * p.cache.k.ss;
  out.v_off = page * p.cache.v.sb + within * p.cache.v.ss;
  if (p.slot_positions != nullptr) {
    const int number = p.seen[b] + i;
    for (int h = 0; h < p.h_k; ++h)
      p.slot_positions[(static_cast<int64_t>(b) * p.h_k + h) * p.slots_stride + slot] = number;
  }
}

template <typename T, int MODE, bool APPEND>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p, RopeGrid g) {
  extern __shared__ float2 cs_all[];  // [tile][n_freq] (cos, sin)
  __shared__ unsigned long long turns[128];
  __shared__ TokenInfo info[kMaxTile];
  const int nf = p.rot.n_freq;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * g.tile;
  const int nt = static_cast<int>(min(static_cast<int64_t>(g.tile), p.tokens - t0));

  // fraction of a turn that one position adds at each frequency, times 2^64
  for (int i = threadIdx.x; i < nf; i += kThreads) {
    const double x = static_cast<double>(p.rot.inv_freq[i]) * 0.15915494309189535;
    turns[i] = static_cast<unsigned long long>((x - floor(x)) * 18446744073709551616.0);
  }
  if (APPEND) {
    for (int i = threadIdx.x; i < nt; i += kThreads) locate(p, t0 + i, info[i]);
    if (blockIdx.x == 0 && p.cu != nullptr)
      for (int i = threadIdx.x; i < p.batch; i += kThreads)
        if (p.cu[i] < 0 || p.cu[i] > p.cu[i + 1]) report(p.status, kBadOffsets);
  }
  __syncthreads();
  for (int u = threadIdx.x; u < nt * nf; u += kThreads) {
    const int t = u / nf, i = u - t * nf;
    int axis = 0;
#pragma unroll
    for (int a = 0; a < 3; ++a) axis += i >= p.rot.end[a] ? 1 : 0;
    const long long pos = p.rot.positions[axis * p.rot.axis_stride + t0 + t];
    const unsigned long long phase = static_cast<unsigned long long>(pos) * turns[i];
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);
    cs_all[u] = make_float2(c, s);
  }
  __syncthreads();

  const int total = nt * static_cast<int>(g.per_token.d);
  const int rotated = (p.h_q + p.h_k) * static_cast<int>(g.per_row.d);
  for (int w = threadIdx.x; w < total; w += kThreads) {
    const int t = static_cast<int>(g.per_token.div(w));
    int u = w - t * static_cast<int>(g.per_token.d);
    const int64_t token = t0 + t;
    if (APPEND && u >= rotated) {  // v: copied into its slot
      u -= rotated;
      const int h = static_cast<int>(g.chunks.div(u));
      const int c = u - h * static_cast<int>(g.chunks.d);
      if (info[t].slot < 0) continue;
      const T* src = static_cast<const T*>(p.v.ptr) + token * p.v.ss + h * p.v.sh;
      T* dst = static_cast<T*>(const_cast<void*>(p.cache.v.ptr)) + info[t].v_off + h * p.cache.v.sh;
      *reinterpret_cast<uint4*>(dst + 8 * c) = *reinterpret_cast<const uint4*>(src + 8 * c);
      continue;
    }
    int h = static_cast<int>(g.per_row.div(u));
    u -= h * static_cast<int>(g.per_row.d);
    const T* src;
    T* dst;
    int64_t b = 0, s = token;
    if (!APPEND) {
      b = g.seq.div(static_cast<uint32_t>(token));
      s = token - b * g.seq.d;
    }
    if (h < p.h_q) {
      if (APPEND && !info[t].live) continue;
      src = static_cast<const T*>(p.q.ptr) + b * p.q.sb + s * p.q.ss + h * p.q.sh;
      dst = static_cast<T*>(const_cast<void*>(p.oq.ptr)) + b * p.oq.sb + s * p.oq.ss + h * p.oq.sh;
    } else {
      h -= p.h_q;
      src = static_cast<const T*>(p.k.ptr) + b * p.k.sb + s * p.k.ss + h * p.k.sh;
      if (APPEND) {
        if (info[t].slot < 0) continue;
        dst = static_cast<T*>(const_cast<void*>(p.cache.k.ptr)) + info[t].k_off + h * p.cache.k.sh;
      } else {
        dst = static_cast<T*>(const_cast<void*>(p.ok.ptr)) + b * p.ok.sb + s * p.ok.ss + h * p.ok.sh;
      }
    }
    const float2* cs = cs_all + t * nf;
    if (MODE == kScalar) {  // sizes that are not whole chunks: one pair of elements
      int i0 = 2 * u, i1 = 2 * u + 1;
      if (u < nf && !p.rot.interleaved) {
        i0 = u;
        i1 = u + nf;
      }
      float x = static_cast<float>(src[i0]), y = static_cast<float>(src[i1]);
      if (u < nf) {
        const float c = cs[u].x, sn = cs[u].y * p.rot.sign;
        const float a = x * c - y * sn;
        y = x * sn + y * c;
        x = a;
      }
      dst[i0] = static_cast<T>(x);
      dst[i1] = static_cast<T>(y);
    } else if (u < g.rot_units) {
      if (MODE == kHalves) {
        uint4 lo = *reinterpret_cast<const uint4*>(src + 8 * u);
        uint4 hi = *reinterpret_cast<const uint4*>(src + nf + 8 * u);
        turn8<T>(lo, hi, cs + 8 * u, p.rot.sign);
        *reinterpret_cast<uint4*>(dst + 8 * u) = lo;
        *reinterpret_cast<uint4*>(dst + nf + 8 * u) = hi;
      } else {
        uint4 v = *reinterpret_cast<const uint4*>(src + 8 * u);
        turn_pairs<T>(v, cs + 4 * u, p.rot.sign);
        *reinterpret_cast<uint4*>(dst + 8 * u) = v;
      }
    } else if (src != dst) {
      const int at = 2 * nf + 8 * (u - g.rot_units);
      *reinterpret_cast<uint4*>(dst + at) = *reinterpret_cast<const uint4*>(src + at);
    }
  }
}

template <typename T, bool APPEND>
cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
  const int nf = p.rot.n_freq, d = p.head_dim;
  // 16-byte chunks need whole chunks of pairs: 8 frequencies (halves) or 4 (pairs)
  const int mode = p.rot.interleaved ? (nf % 4 == 0 ? kPairs : kScalar)
                                     : (nf % 8 == 0 ? kHalves : kScalar);
  RopeGrid g;
  g.rot_units = mode == kHalves ? nf / 8 : (mode == kPairs ? nf / 4 : nf);
  const int copies = mode == kScalar ? (d - 2 * nf) / 2 : (d - 2 * nf) / 8;
  g.per_row.set(static_cast<uint32_t>(g.rot_units + copies));
  g.chunks.set(static_cast<uint32_t>(d / 8));
  const int64_t units = static_cast<int64_t>(p.h_q + p.h_k) * g.per_row.d +
                        (APPEND ? static_cast<int64_t>(p.h_k) * g.chunks.d : 0);
  if (units * kMaxTile > INT32_MAX) return cudaErrorInvalidValue;
  g.per_token.set(static_cast<uint32_t>(units));
  g.seq.set(static_cast<uint32_t>(p.seqlen));
  const int64_t tile = p.tokens / (4 * static_cast<int64_t>(num_sms()));
  g.tile = static_cast<int>(tile < 1 ? 1 : (tile > kMaxTile ? kMaxTile : tile));
  const unsigned blocks = static_cast<unsigned>((p.tokens + g.tile - 1) / g.tile);
  const size_t smem = static_cast<size_t>(g.tile) * nf * sizeof(float2);
  if (mode == kHalves)
    rope_kernel<T, kHalves, APPEND><<<blocks, kThreads, smem, stream>>>(p, g);
  else if (mode == kPairs)
    rope_kernel<T, kPairs, APPEND><<<blocks, kThreads, smem, stream>>>(p, g);
  else
    rope_kernel<T, kScalar, APPEND><<<blocks, kThreads, smem, stream>>>(p, g);
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
