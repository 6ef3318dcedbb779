// Attention of one new token a sequence over a paged cache in 8 bits (attn_decode8).
//
// With codes k8, v8 (e4m3 or int8) and a factor for each block of tokens and head,
//   s_j = scale ks_j (q . k8_j),  o = sum_j p_j vs_j v8_j / sum_j p_j,  p_j = exp(s_j - max).
// Every key is read once for all query heads that share it: bound by the memory it lies in, at
// half the bytes of a 16-bit key, so that the work a byte is twice that of attn_decode.  What
// keeps it small:
//
// Keys are the rows.  The products are m16n8k16 with 16 keys (then 16 columns of V) as M and 8
// query heads as N, S^T = K Q^T and O^T = V^T P^T, so that groups of up to 8 heads fill them.
// Codes are exact in fp16 and are turned into it in registers (e4m3: one conversion for two
// codes; int8: a byte permutation below 0x64 bytes and a subtraction of 1152).  ldmatrix moves
// pairs of bytes; the order in which they then lie along D is undone by reading q in the same
// order, and the order of O's columns by writing them so.
// P^T's fragments are S^T's, transposed in registers by movmatrix.
//
// Warps are on their own.  Each of the eight warps of a block keeps a ring of its own 16 (or 32)
// keys of every tile, which its lanes look up and copy asynchronously, and its own softmax and O
// over all columns: no barrier inside a segment.  Where a run of tiles or a segment ends the
// warps' O are added up through shared memory.  Runs of tiles, lines and partials are those of
// attn_decode, and so is the kernel that joins them.
//
// Numbers.  q enters as fp16: bf16 rows are divided by the power of two of their largest element,
// which is exact down to 2^-17 of it and off by 2^-25 of it below.  The weights of a key in O are
// p_j vs_j.  vs_j = 2^e r with 1 <= r < 2, and the running maximum is that of s_j log2(e) + e, so
// that the weight 2^(s + e - max) r stays within [0, 2] whatever the factors of the blocks are;
// it enters the product as two fp16 numbers, its rounded value and the rounded remainder, times
// 2^14, so that it is right to 2^-22 or 2^-39 of the largest.  The sum of the p_j has the same
// maximum (its terms are 2^-e times as large: e is kept within +-60).  All sums are fp32.
#include <atomic>

#include "decode.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kWeight = 16384.f;  // factor of the weights and of O until it is written
constexpr int kExp = 60;            // exponents of V's factors lie within +-kExp

template <int DP, int HN>
struct Cfg {
  static constexpr int kBlocks = DP <= 128 && HN == 1 ? 2 : (DP == 64 ? 2 : 1);  // of an SM
  static constexpr int kGroups = DP == 64 ? 2 : 1;       // groups of 16 keys of a warp and tile
  static constexpr int kKeys = 16 * kGroups;
  static constexpr int kTileLog2 = kGroups == 2 ? 8 : 7;
  static constexpr int kTile = 1 << kTileLog2;
  static constexpr int kHeads = 8 * HN;
  static constexpr int kStageBytes = 2 * kKeys * DP;     // of a warp
  static constexpr int kMergeCols = 32 / HN;             // columns of O that the warps add up at a time
  static constexpr int kMerge = kWarps * kHeads * (kMergeCols + 4) * 4;
  // stages that fit beside the rest, at most six
  static constexpr int kRest = 1024 + kWarps * (kHeads * 8 + 4) + kMerge + kLens * 4;
  static constexpr int kFit = ((228 * 1024 / kBlocks - kRest) / kWarps - kKeys * 16 - 32) / (kStageBytes + kKeys * 8 + 16);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static constexpr int kSlots = kStages + 2;             // descriptors
  static constexpr int kWarpBytes = kStages * (kStageBytes + kKeys * 8) + kKeys * 16 + kSlots * 16;
  static constexpr int kSmem = kWarps * kWarpBytes + kMerge + kLens * 4;
  static_assert(kWarpBytes % 16 == 0 && kStages >= 2, "");
  static_assert((kSmem + kRest - kMerge - kLens * 4) * kBlocks <= 228 * 1024, "shared memory of an SM");
};

// What a row's 16-byte chunk numbers are permuted by (exclusive or), so that eight neighbouring
// rows' chunks lie in different banks.
template <int DP>
__host__ __device__ constexpr int perm8(int row) {
  return DP % 128 == 0 ? row & 7 : (DP == 96 ? (row >> 2) & 1 : (row >> 1) & 3);
}

__device__ __forceinline__ void cp_async4_or_zero(uint32_t dst, const float* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t sub_h2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// Bytes 0, 1 and bytes 2, 3 of x as fp16 pairs.
template <bool INT8>
__device__ __forceinline__ void halves(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if (INT8) {
    x ^= 0x80808080u;  // + 128: under 0x64 as the upper byte the value 1024 + 128 + code
    lo = sub_h2(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
    hi = sub_h2(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  }
}
// Bytes 0, 2 and bytes 1, 3.
template <bool INT8>
__device__ __forceinline__ void halves_across(uint32_t x, uint32_t& even, uint32_t& odd) {
  if (INT8) {
    x ^= 0x80808080u;
    even = sub_h2(__byte_perm(x, 0x64646464u, 0x4240), 0x64806480u);
    odd = sub_h2(__byte_perm(x, 0x64646464u, 0x4341), 0x64806480u);
  } else {
    halves<false>(__byte_perm(x, 0, 0x3120), even, odd);
  }
}

template <int DP, int HN, bool INT8>
__global__ void __launch_bounds__(kThreads, Cfg<DP, HN>::kBlocks) decode8_kernel(Decode8Params p) {
  using C = Cfg<DP, HN>;
  constexpr int S = C::kStages, kSlots = C::kSlots, kKeys = C::kKeys, kGroups = C::kGroups, kTile = C::kTile;
  constexpr int kSteps = DP / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_sums[kWarps];
  __shared__ float s_max[kWarps][C::kHeads], s_sum[kWarps][C::kHeads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* mine = smem + warp * C::kWarpBytes;  // ring, factors, addresses, descriptors
  float2* factors = reinterpret_cast<float2*>(mine + S * C::kStageBytes);
  longlong2* rows = reinterpret_cast<longlong2*>(factors + S * kKeys);
  int4* desc = reinterpret_cast<int4*>(rows + kKeys);  // sequence, head tile, flags, valid keys
  float* merge = reinterpret_cast<float*>(smem + kWarps * C::kWarpBytes);
  int* s_pre = reinterpret_cast<int*>(merge);  // until the first O is added up
  int* lens = reinterpret_cast<int*>(smem + kWarps * C::kWarpBytes + C::kMerge);
  const int hv_n = p.h_k * p.head_tiles;
  const int line_heads = p.lines > 1 ? 1 : hv_n;
  const int run = blockIdx.x / p.lines, line = blockIdx.x - run * p.lines;
  const uint32_t ring_u = smem_u32(mine), factors_u = smem_u32(factors);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this block's run of tiles
  const int per = (p.batch + kThreads - 1) / kThreads;
  Cut cut;
  if (p.whole) {
    const int b = blockIdx.x / hv_n, n = clean_len(p, p.seqlens[b], true);
    if (n == 0) {
      if (p.bf16) no_keys<__nv_bfloat16>(p, b, blockIdx.x - b * hv_n);
      else no_keys<__half>(p, b, blockIdx.x - b * hv_n);
      return;
    }
    if (tid == 0) lens[0] = n;
  } else {
    int total;
    s_pre[tid] = scan_tiles<kThreads>(p, true, lens, s_sums, per, total);
    cut.total = static_cast<long long>(total) * line_heads;
    cut.runs = static_cast<int>(min(static_cast<long long>(gridDim.x / p.lines), cut.total));
    if (run >= cut.runs) return;
  }
  // columns that no copy writes stay zero
  if (p.chunks < DP / 16) {
    const int nc = DP / 16 - p.chunks;
    for (int i = lane; i < S * 2 * kKeys * nc; i += 32)
      *reinterpret_cast<uint4*>(mine + (i / nc) * DP + (((p.chunks + i % nc) ^ perm8<DP>(i / nc)) << 4)) =
          make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  // ================================================== tiles: looked up, copied
  int left = 0;
  int cb = 0, ch = 0, ct = 0, cn = 0, cfirst = 0, cnt = 0;
  bool seg_from_start = true;
  int nth = 0, begin = 1;
  const int* table = nullptr;
  const char *khead = nullptr, *vhead = nullptr;
  const float *ksh = nullptr, *vsh = nullptr;
  auto load_seq = [&](int n) {
    cn = n;
    cfirst = first_key(p, cn);
    cnt = (cn - cfirst + kTile - 1) >> C::kTileLog2;
    table = p.cache.table + cb * p.cache.table_stride;
  };
  auto load_head = [&]() {
    const int hv = line + ch, g = hv / p.head_tiles, ht = hv - g * p.head_tiles;
    khead = static_cast<const char*>(p.cache.k.ptr) + g * p.cache.k.sh;
    vhead = static_cast<const char*>(p.cache.v.ptr) + g * p.cache.v.sh;
    ksh = p.k_scale + g * p.ks[2];
    vsh = p.v_scale + g * p.vs[2];
    // its queries are asked for a few tiles ahead
    const int h = g * p.group + ht * kMaxRows + (lane & 15);
    if (warp == 0 && h < (g + 1) * p.group)
      for (int i = (lane >> 4) * 64; i < p.head_dim; i += 128)
        prefetch_l2(static_cast<const uint16_t*>(p.q.ptr) + cb * p.q.sb + h * p.q.sh + i);
  };
  auto len_of = [&](int b) { return b < kLens ? lens[b] : clean_len(p, p.seqlens[b], false); };
  if (p.whole) {
    cb = blockIdx.x / hv_n;
    ch = blockIdx.x - cb * hv_n;  // one line
    load_seq(lens[0]);
    left = cnt;
  } else {
    const long long r0 = cut.start(run);
    left = static_cast<int>(cut.start(run + 1) - r0);
    int before;
    cb = find_sequence<kThreads>(p, s_pre, per, line_heads, r0, len_of, before);
    load_seq(len_of(cb));
    const long long in = r0 - static_cast<long long>(before) * line_heads;
    ch = static_cast<int>(in / cnt);
    ct = static_cast<int>(in - static_cast<long long>(ch) * cnt);
    seg_from_start = ct == 0;
  }
  load_head();
  // strides in 16-byte units: a page's offset is one 32 x 32 bit product
  const uint32_t kp = static_cast<uint32_t>(p.cache.k.sb / 16), kslot = static_cast<uint32_t>(p.cache.k.ss / 16);
  const uint32_t vp = static_cast<uint32_t>(p.cache.v.sb / 16), vslot = static_cast<uint32_t>(p.cache.v.ss / 16);
  const int key = lane & (kKeys - 1);  // of this warp's keys the one that the lane looks up
  int pend_page = 0, pend_within = 0, pend_flags = 0, pend_b = 0, pend_hv = 0;
  bool pend_live = false;
  const char *pend_k = nullptr, *pend_v = nullptr;
  const float *pend_ks = nullptr, *pend_vs = nullptr;
  auto plan = [&]() {  // looks one tile up and moves on
    pend_live = false;
    if (left == 0) {
      pend_flags = kNone;
      return;
    }
    pend_k = khead;
    pend_v = vhead;
    pend_ks = ksh;
    pend_vs = vsh;
    const int j = cfirst + ct * kTile + warp * kKeys + key;
    pend_live = j < cn;
    if (pend_live) {
      const int n = static_cast<int>(p.cache.page.div(static_cast<uint32_t>(j)));
      pend_within = j - n * static_cast<int>(p.cache.page.d);
      pend_page = table[n];
    }
    const bool at_end = ct == cnt - 1;
    pend_b = cb;
    pend_hv = line + ch;
    pend_flags = (begin ? kBegin : 0) | (at_end || left == 1 ? kEnd : 0) | (at_end && seg_from_start ? kFull : 0) |
                 (nth ? kSecond : 0);
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
    if (++ch == line_heads) {
      ch = 0;
      do {
        ++cb;
        load_seq(len_of(cb));
      } while (cnt == 0 && cb + 1 < p.batch);
    }
    load_head();
  };
  // Keys and values are read once, unless a group has several head tiles: they leave the L2 first.
  const uint64_t policy = p.head_tiles > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
  // Writes a tile's addresses and descriptor down and asks for its factors.
  auto store_plan = [&](int slot, int stage) {
    bool ok = pend_live;
    if (ok && static_cast<unsigned>(pend_page) >= static_cast<unsigned>(p.cache.num_pages)) {
      report(p.status, kBadPage);
      ok = false;
    }
    longlong2 o = make_longlong2(0, 0);  // addresses of the key's row of k and of v
    const float *fk = p.k_scale, *fv = p.v_scale;
    if (ok) {
      const uint64_t page = static_cast<uint32_t>(pend_page), in = static_cast<uint32_t>(pend_within);
      o.x = reinterpret_cast<long long>(pend_k + ((page * kp + in * kslot) << 4));
      o.y = reinterpret_cast<long long>(pend_v + ((page * vp + in * vslot) << 4));
      const int64_t blk = p.block.div(static_cast<uint32_t>(pend_within));
      fk = pend_ks + static_cast<int64_t>(pend_page) * p.ks[0] + blk * p.ks[1];
      fv = pend_vs + static_cast<int64_t>(pend_page) * p.vs[0] + blk * p.vs[1];
    }
    const uint32_t at = factors_u + (stage * kKeys + key) * 8;
    if (kKeys == 32) {
      cp_async4_or_zero(at, fk, ok);
      cp_async4_or_zero(at + 4, fv, ok);
    } else {
      cp_async4_or_zero(at + (lane >> 4) * 4, lane < 16 ? fk : fv, ok);
    }
    if (lane < kKeys) rows[key] = o;
    const uint32_t bits = __ballot_sync(0xffffffffu, ok);
    if (lane == 0)
      desc[slot] = make_int4(pend_b, pend_hv, pend_flags, static_cast<int>(kKeys == 32 ? bits : bits & 0xffffu));
  };
  // Issues the copies of the tile whose plan was stored last, if there is one.
  auto fetch = [&](int slot, int stage) {
    constexpr int kLanes = DP == 64 ? 4 : (DP <= 128 ? 8 : 16), kStep = 32 / kLanes, kIter = kKeys / kStep;
    const int4 d = desc[slot];
    const int c = lane % kLanes, r0 = lane / kLanes;
    if (!(d.z & kNone) && d.w != 0 && c < p.chunks) {
      const uint32_t dst = ring_u + stage * C::kStageBytes;
#pragma unroll
      for (int i = 0; i < kIter; ++i) {
        const int r = r0 + i * kStep;
        const longlong2 a = rows[r];
        const bool ok = a.x != 0;
        const uint32_t to = dst + r * DP + ((c ^ perm8<DP>(r)) << 4);
        cp_async16_or_zero(to, ok ? a.x + c * 16 : reinterpret_cast<long long>(p.cache.k.ptr), ok, policy);
        cp_async16_or_zero(to + kKeys * DP, ok ? a.y + c * 16 : reinterpret_cast<long long>(p.cache.v.ptr), ok, policy);
      }
    }
    cp_commit();
  };
  plan();
  int slot_w = 0, stage_w = 0;  // of the next tile to store and fetch
  auto next_w = [&]() {
    slot_w = slot_w + 1 == kSlots ? 0 : slot_w + 1;
    stage_w = stage_w + 1 == S ? 0 : stage_w + 1;
  };
  for (int t = 0; t < S - 1; ++t) {
    store_plan(slot_w, stage_w);
    plan();
    __syncwarp();
    fetch(slot_w, stage_w);
    next_w();
    __syncwarp();
  }

  // ================================================== attention
  uint32_t qf[HN][kSteps][2];
  float qscale[HN][2];  // of heads 2 (lane % 4) and the next: times s_j ks_j the base-2 logit
  float o[kSteps][HN][4];
  float m[HN][2], l[HN][2];
  const int g8 = lane >> 2, q4 = lane & 3;
  int b = 0, h0 = 0, hn = 0;
  const uint32_t lrow = (lane & 7) + ((lane >> 3) & 1) * 8;  // of ldmatrix: key and chunk
  const int lchunk = lane >> 4;
  int slot = 0, stage = 0;
  for (;;) {
    cp_wait<S - 2>();
    __syncwarp();  // the copies of all lanes are there, and the last tile's stage is free
    const int4 d = desc[slot];
    if (d.z & kNone) break;
    const int stage_now = stage;
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    stage = stage + 1 == S ? 0 : stage + 1;
    // the tile S - 1 ahead
    store_plan(slot_w, stage_w);
    plan();
    __syncwarp();
    fetch(slot_w, stage_w);
    next_w();

    if (d.z & kBegin) {
      const int g = d.y / p.head_tiles, ht = d.y - g * p.head_tiles;
      b = d.x;
      h0 = g * p.group + ht * kMaxRows;
      hn = min(kMaxRows, p.group - ht * kMaxRows);
      float mul[HN];
#pragma unroll
      for (int n = 0; n < HN; ++n) {
        const int head = g8 + n * 8;
        const uint16_t* q = static_cast<const uint16_t*>(p.q.ptr) + b * p.q.sb + (h0 + head) * p.q.sh + q4 * 4;
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint2 x = head < hn && k < p.chunks ? *reinterpret_cast<const uint2*>(q + k * 16) : make_uint2(0, 0);
          qf[n][k][0] = x.x;
          qf[n][k][1] = x.y;
          top = max(top, max(max((x.x & 0x7fffu) << 16, x.x & 0x7fff0000u),
                             max((x.y & 0x7fffu) << 16, x.y & 0x7fff0000u)));
        }
        mul[n] = 1.f;
        if (p.bf16) {  // divided by the power of two of the row's largest element
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = min(max(static_cast<int>(top >> 23) - 127, -126), 126);
          const float down = __int_as_float((127 - e) << 23);
          mul[n] = __int_as_float((127 + e) << 23);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 x = Pack<__nv_bfloat16>::unpack(qf[n][k][i]);
              qf[n][k][i] = Pack<__half>::two(x.x * down, x.y * down);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) qscale[n][i] = __shfl_sync(0xffffffffu, mul[n], (2 * q4 + i) * 4);
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
      }
    }

    if (d.w != 0) {
      const uint32_t kst = ring_u + stage_now * C::kStageBytes + lrow * DP;
      // ---- base-2 logits of this warp's keys, plus the exponents of V's factors
      float z[kGroups][HN][4], r[kGroups][2], down[kGroups][2];
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        float s[HN][2][4];
#pragma unroll
        for (int n = 0; n < HN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][0][i] = s[n][1][i] = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t x[4], a[8];
          ldsm4(kst + gr * 16 * DP + (((k + lchunk) ^ perm8<DP>(lrow)) << 4), x);
          halves<INT8>(x[0], a[0], a[2]);
          halves<INT8>(x[1], a[1], a[3]);
          halves<INT8>(x[2], a[4], a[6]);
          halves<INT8>(x[3], a[5], a[7]);
#pragma unroll
          for (int n = 0; n < HN; ++n) {
            mma_f16(s[n][0], a[0], a[1], a[2], a[3], qf[n][k][0], qf[n][k][1]);
            mma_f16(s[n][1], a[4], a[5], a[6], a[7], qf[n][k + 1][0], qf[n][k + 1][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = gr * 16 + g8 + i * 8;
          const float2 f = factors[stage_now * kKeys + kk];
          const int e = min(max(static_cast<int>(__float_as_uint(f.y) >> 23) - 127, -kExp), kExp);
          r[gr][i] = f.y * __int_as_float((127 - e) << 23);
          down[gr][i] = __int_as_float((127 - e) << 23);
          const bool valid = (static_cast<uint32_t>(d.w) >> kk) & 1u;
#pragma unroll
          for (int n = 0; n < HN; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float x = (s[n][0][i * 2 + c] + s[n][1][i * 2 + c]) * (f.x * qscale[n][c]);
              const float y = p.softcap > 0.f ? p.cap_out * tanh_exp(x * p.cap_in) : x * p.scale_log2;
              z[gr][n][i * 2 + c] = valid ? y + static_cast<float>(e) : -INFINITY;
            }
        }
      }
      // ---- the running maximum
      float f[HN][2];
      bool moved = false;
#pragma unroll
      for (int n = 0; n < HN; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(z[0][n][c], z[0][n][c + 2]);
          if (kGroups == 2) top = fmaxf(top, fmaxf(z[kGroups - 1][n][c], z[kGroups - 1][n][c + 2]));
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
          const float mx = fmaxf(m[n][c], top);
          f[n][c] = mx == m[n][c] ? 1.f : ex2(m[n][c] - mx);
          moved |= mx != m[n][c];
          m[n][c] = mx;
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < HN; ++n) {
          l[n][0] *= f[n][0];
          l[n][1] *= f[n][1];
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][n][i] *= f[n][i & 1];
        }
      }
      // ---- weights, and O^T += V^T (weights)
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr) {
        uint32_t hi[HN][2], lo[HN][2];
#pragma unroll
        for (int n = 0; n < HN; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float b0 = m[n][0] == -INFINITY ? 0.f : m[n][0], b1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
            const float e0 = ex2(z[gr][n][i * 2] - b0), e1 = ex2(z[gr][n][i * 2 + 1] - b1);
            l[n][0] += e0 * down[gr][i];
            l[n][1] += e1 * down[gr][i];
            const float w0 = e0 * (r[gr][i] * kWeight), w1 = e1 * (r[gr][i] * kWeight);
            const uint32_t h = Pack<__half>::two(w0, w1);
            const float2 back = Pack<__half>::unpack(h);
            hi[n][i] = transposed(h);
            lo[n][i] = transposed(Pack<__half>::two(w0 - back.x, w1 - back.y));
          }
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t x[4], a[8];
          ldsm4_t(kst + (kKeys + gr * 16) * DP + (((k + lchunk) ^ perm8<DP>(lrow)) << 4), x);
          halves_across<INT8>(x[0], a[0], a[1]);
          halves_across<INT8>(x[1], a[2], a[3]);
          halves_across<INT8>(x[2], a[4], a[5]);
          halves_across<INT8>(x[3], a[6], a[7]);
#pragma unroll
          for (int n = 0; n < HN; ++n) {
            mma_f16(o[k][n], a[0], a[1], a[2], a[3], hi[n][0], hi[n][1]);
            mma_f16(o[k + 1][n], a[4], a[5], a[6], a[7], hi[n][0], hi[n][1]);
            mma_f16(o[k][n], a[0], a[1], a[2], a[3], lo[n][0], lo[n][1]);
            mma_f16(o[k + 1][n], a[4], a[5], a[6], a[7], lo[n][0], lo[n][1]);
          }
        }
      }
    }

    if (d.z & kEnd) {
      // ---- this run's part of the segment is complete: the warps' O are added up
      __syncthreads();  // what the last segment left has been read
#pragma unroll
      for (int n = 0; n < HN; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], i);
          if (lane < 4) {
            s_max[warp][n * 8 + 2 * q4 + c] = m[n][c];
            s_sum[warp][n * 8 + 2 * q4 + c] = l[n][c];
          }
        }
      __syncthreads();
      float mul[HN][2];
#pragma unroll
      for (int n = 0; n < HN; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_max[w][n * 8 + 2 * q4 + c]);
          mul[n][c] = ex2(m[n][c] - (top == -INFINITY ? 0.f : top));
        }
      const bool whole = (d.z & kFull) != 0;
      float* part = partial(p, blockIdx.x, (d.z & kSecond) ? 1 : 0);
      constexpr int kCols = C::kMergeCols, kPitch = kCols + 4, kRow = C::kHeads * kPitch;  // of a head, of a warp
#pragma unroll
      for (int k0 = 0; k0 < kSteps; k0 += kCols / 16) {
        float* to = merge + warp * kRow;
#pragma unroll
        for (int n = 0; n < HN; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = n * 8 + 2 * q4 + c;
#pragma unroll
            for (int k = 0; k < kCols / 16; ++k)
              *reinterpret_cast<float2*>(to + row * kPitch + k * 16 + 2 * g8) =
                  make_float2(o[k0 + k][n][c] * mul[n][c], o[k0 + k][n][c + 2] * mul[n][c]);
          }
        __syncthreads();
        for (int i = tid; i < hn * (kCols / 2); i += kThreads) {
          const int row = i / (kCols / 2), col = i % (kCols / 2) * 2;
          float2 x = make_float2(0.f, 0.f);
          float top = -INFINITY, sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 y = *reinterpret_cast<const float2*>(merge + w * kRow + row * kPitch + col);
            x.x += y.x;
            x.y += y.y;
            top = fmaxf(top, s_max[w][row]);
          }
          const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) sum += s_sum[w][row] * ex2(s_max[w][row] - base);
          const int at = k0 * 16 + col;
          if (whole) {
            const bool none = sum == 0.f;
            const float inv = none ? 0.f : 1.f / kWeight / sum;
            const float a = none ? 0.f : x.x * inv, bb = none ? 0.f : x.y * inv;
            uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + (h0 + row) * p.o.sh;
            if (at < p.head_dim)
              *reinterpret_cast<uint32_t*>(out + at) =
                  p.bf16 ? Pack<__nv_bfloat16>::two(a, bb) : Pack<__half>::two(a, bb);
            if (k0 == 0 && col == 0 && p.lse != nullptr)
              p.lse[static_cast<int64_t>(b) * p.h_q + h0 + row] =
                  none ? INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
          } else {
            *reinterpret_cast<float2*>(part + row * DP + at) = make_float2(x.x * (1.f / kWeight), x.y * (1.f / kWeight));
            if (k0 == 0 && col == 0) {
              part[p.part_rows * DP + row] = top;
              part[p.part_rows * DP + kMaxRows + row] = sum;
            }
          }
        }
        if (k0 + kCols / 16 < kSteps) __syncthreads();
      }
    }
  }
  cp_wait<0>();
}

template <int DP, int HN, bool INT8>
cudaError_t launch_main(Decode8Params p, cudaStream_t stream) {
  using C = Cfg<DP, HN>;
  static std::atomic<unsigned long long> done{0};  // devices with the attribute set
  int runs;
  cudaError_t e = shape_decode(p, C::kTileLog2, C::kBlocks, &runs);
  if (e != cudaSuccess) return e;
  if (runs > 0) {
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (!(done.load(std::memory_order_relaxed) & bit) || bit == 0) {
      e = cudaFuncSetAttribute(decode8_kernel<DP, HN, INT8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
      if (e != cudaSuccess) return e;
      done.fetch_or(bit, std::memory_order_relaxed);
    }
    decode8_kernel<DP, HN, INT8><<<runs, kThreads, C::kSmem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return p.whole ? cudaSuccess : launch_join(p, p.bf16 ? ATTN_BF16 : ATTN_FP16, runs, stream);
}

template <int DP>
cudaError_t launch_dim(const Decode8Params& p, int int8, cudaStream_t stream) {
  if (p.group > 8) return int8 ? launch_main<DP, 2, true>(p, stream) : launch_main<DP, 2, false>(p, stream);
  return int8 ? launch_main<DP, 1, true>(p, stream) : launch_main<DP, 1, false>(p, stream);
}

}  // namespace

cudaError_t launch_decode8(const Decode8Params& in, int int8, cudaStream_t stream) {
  Decode8Params p = in;
  p.chunks = p.head_dim / 16;
  switch (pad_dim(p.head_dim)) {
    case 64: return launch_dim<64>(p, int8, stream);
    case 96: return launch_dim<96>(p, int8, stream);
    case 128: return launch_dim<128>(p, int8, stream);
    case 192: return launch_dim<192>(p, int8, stream);
    default: return launch_dim<256>(p, int8, stream);
  }
}

}  // namespace attn
