// Attention of one new token a sequence over the paged cache (attn_decode).
//
// First form: one block per (sequence, query head); its warps take the keys in
// turn, each lane holding head_dim / 32 elements, with a running maximum and sum
// per warp that are joined at the end.
#include "cache.h"
#include "common.cuh"

namespace attn {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxPer = 8;  // elements of a lane (head_dim <= 256)

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(DecodeParams p) {
  __shared__ float sm[kWarps], sl[kWarps];
  __shared__ float so[kWarps][256];
  const int h = blockIdx.x, b = blockIdx.y, g = h / p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = p.seqlens[b];
  if (n < 0 || n > p.max_seqlen) {
    if (threadIdx.x == 0) report(p.status, kBadLength);
    n = 0;
  }
  const int first = p.win_left >= 0 ? max(0, n - 1 - p.win_left) : 0;
  const int* row = p.cache.table + b * p.cache.table_stride;
  const T* kp = static_cast<const T*>(p.cache.k.ptr) + g * p.cache.k.sh;
  const T* vp = static_cast<const T*>(p.cache.v.ptr) + g * p.cache.v.sh;
  const T* qp = static_cast<const T*>(p.q.ptr) + b * p.q.sb + h * p.q.sh;
  float q[kMaxPer], o[kMaxPer];
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.head_dim ? static_cast<float>(qp[d]) : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  float* logits = p.logits + (static_cast<int64_t>(b) * p.h_q + h) * p.max_seqlen;
  for (int j = warp; j < n; j += kWarps) {
    int page, within;
    float s = -INFINITY;
    const bool live = j >= first && page_of(p.cache, row, j, page, within, p.status);
    if (live) {
      const T* k = kp + page * p.cache.k.sb + within * p.cache.k.ss;
      const T* v = vp + page * p.cache.v.sb + within * p.cache.v.ss;
      s = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxPer; ++i) {
        const int d = lane + 32 * i;
        if (d < p.head_dim) s += q[i] * static_cast<float>(k[d]);
      }
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s = p.softcap > 0.f ? p.cap_out * tanh_exp(s * p.cap_in) : s * p.scale_log2;
      const float top = fmaxf(m, s);
      const float base = top == -INFINITY ? 0.f : top;
      const float old = ex2(m - base), e = ex2(s - base);
      l = l * old + e;
#pragma unroll
      for (int i = 0; i < kMaxPer; ++i) {
        const int d = lane + 32 * i;
        if (d < p.head_dim) o[i] = o[i] * old + e * static_cast<float>(v[d]);
      }
      m = top;
    }
    if (p.w_in != nullptr && lane == 0) logits[j] = s;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kMaxPer; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  const float base = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) total += sl[w] * ex2(sm[w] - base);
  const bool some = !(total == 0.f);
  T* op = static_cast<T*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + h * p.o.sh;
  for (int d = threadIdx.x; d < p.head_dim; d += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += so[w][d] * ex2(sm[w] - base);
    op[d] = static_cast<T>(some ? x / total : 0.f);
  }
  if (threadIdx.x == 0) {
    const float lse2 = some ? base + log2f(total) : INFINITY;
    const int64_t at = static_cast<int64_t>(b) * p.h_q + h;
    if (p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
    p.lse2[at] = lse2;
  }
}

// weights_out = weights_in + the group's sum of exp2(logit - LSE2)
__global__ void __launch_bounds__(256) weights_kernel(DecodeParams p) {
  const int g = blockIdx.y, b = blockIdx.z;
  int n = p.seqlens[b];
  if (n < 0 || n > p.max_seqlen) n = 0;
  for (int j = blockIdx.x * 256 + threadIdx.x; j < n; j += gridDim.x * 256) {
    float w = 0.f;
    for (int i = 0; i < p.group; ++i) {
      const int64_t h = static_cast<int64_t>(b) * p.h_q + g * p.group + i;
      w += ex2(p.logits[h * p.max_seqlen + j] - p.lse2[h]);
    }
    const int64_t at = (static_cast<int64_t>(b) * p.h_k + g) * p.w_stride + j;
    p.w_out[at] = p.w_in[at] + w;
  }
}

}  // namespace

DecodeWs decode_ws(int batch, int h_q, int h_k, int head_dim, int max_seqlen, bool weights) {
  DecodeWs w;
  const size_t rows = static_cast<size_t>(batch) * h_q;
  w.off_lse2 = 0;
  w.off_logits = align256(rows * 4);
  w.total = w.off_logits + (weights ? align256(rows * max_seqlen * 4) : 0);
  return w;
}

cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t stream) {
  const dim3 grid(p.h_q, p.batch);
  if (dtype == ATTN_BF16)
    decode_kernel<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(p);
  else
    decode_kernel<__half><<<grid, kWarps * 32, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.w_in == nullptr || p.max_seqlen == 0) return e;
  weights_kernel<<<dim3(ceil_div(p.max_seqlen, 1024), p.h_k, p.batch), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace attn
