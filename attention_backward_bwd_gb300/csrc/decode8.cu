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
// warps' O are added up through the stages that they worked on last.  Runs, lines and partials are
// those of attn_decode, and so is the kernel that joins them.  The line is cut in units of 128 keys,
// of which a tile takes two where it can: a look-up for 32 keys costs what one for 16 does (with
// tiles of 128 keys throughout 64 sequences up to 16384 keys took 243 us where 210 with 256).
//
// Measured: 64 sequences of 4096 to 16384 keys, 32 query heads on 8 of 128, e4m3 202 to 210 us, 95 to
// 98 % of the copy bandwidth; one of 131071 keys in int8 53 us (75 %) and e4m3 50.  Beside the bytes there
// are about 8.5 us of first reads (lengths, table, rows) and of the join.  What it was made faster by,
// from 285 us: 32 keys looked up at once, the maximum compared by vote and moved only where it
// grows, weights without a second exponent, O added up in one round (in eight it cost 3 us a segment).
//
// Numbers.  q enters as fp16: bf16 rows are scaled by a power of two, their largest element to
// [2^15, 2^16), which is exact down to 2^-32 of it and off by 2^-40 of it below.  The weight of a code in O is
// p_j vs_j, and the running maximum M is that of s_j log2(e) + floor(log2 vs_j), so that the weight
// 2^(s - M) vs stays below 2 whatever the factors of the blocks are.  It enters the product as two
// fp16 numbers, its rounded value and the rounded remainder, times 2^14, so that it is right to
// 2^-22 of itself or 2^-38 of the largest.  V's factors are kept within 2^+-60, so that the
// 2^(s - M) of the sum, up to 2^60, have room in fp32; where M steps by more than fp32's exponents
// they are scaled in halves, and partials leave with a sum in [1, 2).  Their maximum is that of the
// sum alone, so the join scales a far partial's O in halves, too.  All sums are fp32.
#include <atomic>

#include "decode.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kWeight = 16384.f;  // factor of the weights and of O until it is written
constexpr int kKeys = 32;           // of a warp and tile
constexpr int kUnitLog2 = 7, kUnit = 1 << kUnitLog2;  // keys of a unit of the line: half a tile
constexpr float kLeast = 8.673617379884035e-19f, kMost = 1.152921504606847e18f;  // factors of V: 2^-60, 2^60

template <int DP, int HN>
struct Cfg {
  static constexpr int kBlocks = DP <= 128 && HN == 1 ? 2 : (DP == 64 ? 2 : 1);  // of an SM
  // A warp's 32 keys of a tile are copied and worked on in kSubs parts of kGroups times 16: at once
  // where registers and shared memory have room for that (64 sequences up to 16384 keys of 8 heads,
  // 16 query heads each: of 96 columns 246 us at once, 263 in two parts, of 64 columns 228 and 195).
  static constexpr int kGroups = (DP == 64) == (HN == 1) && DP <= 128 ? 2 : 1, kSubs = 2 / kGroups, kSubKeys = 16 * kGroups;
  static constexpr int kStageBytes = 2 * kSubKeys * DP;  // of a part, of a warp
  static constexpr int kHeads = 8 * HN;
  // tiles that are copied ahead: as fit beside the rest, at most three
  static constexpr int kRest = 1024 + kWarps * (kHeads * 8 + 4) + kThreads * 4 + kLens * 4;
  static constexpr int kFit = (228 * 1024 / kBlocks - kRest) / kWarps;
  static constexpr int warp_bytes(int ahead) {  // stages, addresses, descriptors, factors
    return (ahead * kSubs + 1) * kStageBytes + (ahead + 1) * kKeys * 8 + kKeys * 16 + 128;
  }
  static constexpr int kAhead = warp_bytes(3) <= kFit ? 3 : (warp_bytes(2) <= kFit ? 2 : 1);
  static constexpr int kStages = kAhead * kSubs + 1, kSlots = kAhead + 1;
  static constexpr int kWarpBytes = warp_bytes(kAhead);
  static constexpr int kSmem = kWarps * kWarpBytes + kThreads * 4 + kLens * 4;
  static_assert(kWarpBytes % 128 == 0 && kSlots * 16 <= 128, "");
  static_assert((kWarps * kWarpBytes + kRest) * kBlocks <= 228 * 1024, "shared memory of an SM");
};

// What a row's 16-byte chunk numbers are permuted by (exclusive or), so that eight neighbouring
// rows' chunks lie in different banks.
template <int DP>
__host__ __device__ constexpr int perm8(int row) {
  return DP % 128 == 0 ? row & 7 : (DP == 96 ? (row >> 2) & 1 : (row >> 1) & 3);
}

// The address of chunks k and k + 1 (k even) in a row, from that of chunks 0 and 1: rows start at
// multiples of 32 bytes and more, so that the permutation acts on the address.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(uint32_t row, int k) {
  constexpr int kMask = DP % 128 == 0 ? 6 : (DP == 96 ? 0 : 2);
  return (row ^ ((k & kMask) << 4)) + (k & ~(kMask | 1)) * 16;
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
  constexpr int S = C::kStages, kSlots = C::kSlots, kSubs = C::kSubs, kSubKeys = C::kSubKeys, kGroups = C::kGroups;
  constexpr int kSteps = DP / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_sums[kWarps];
  __shared__ float s_max[kWarps][C::kHeads], s_sum[kWarps][C::kHeads];
  const int tid = threadIdx.x, lane = tid & 31, warp = static_cast<int>(warp_id());
  unsigned char* mine = smem + warp * C::kWarpBytes;  // stages, addresses, descriptors, factors
  longlong2* rows = reinterpret_cast<longlong2*>(mine + S * C::kStageBytes);
  int4* desc = reinterpret_cast<int4*>(rows + kKeys);  // sequence, head tile, flags, valid keys
  float2* factors = reinterpret_cast<float2*>(desc + 8);
  int* s_pre = reinterpret_cast<int*>(smem + kWarps * C::kWarpBytes);
  int* lens = s_pre + kThreads;
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
  auto zero_columns = [&](int first_stage, int stages) {
    const int nc = DP / 16 - p.chunks;
    for (int i = lane; i < stages * 2 * kSubKeys * nc; i += 32)
      *reinterpret_cast<uint4*>(mine + first_stage * C::kStageBytes + (i / nc) * DP +
                                (((p.chunks + i % nc) ^ perm8<DP>(i / nc)) << 4)) = make_uint4(0, 0, 0, 0);
  };
  zero_columns(0, S);
  __syncthreads();

  // ================================================== tiles: looked up, copied
  int left = 0;
  int cb = 0, ch = 0, ct = 0, cn = 0, cfirst = 0, cnt = 0;
  bool seg_from_start = true;
  const int* table = nullptr;
  const char *khead = nullptr, *vhead = nullptr;
  const float *ksh = nullptr, *vsh = nullptr;
  auto load_seq = [&](int n) {
    cn = n;
    cfirst = first_key(p, cn);
    cnt = tiles_of(p, cn);
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
  // strides in 16-byte units: a page's offset is one 32 x 32 bit product; of factors, 32 bits
  const uint32_t kp = static_cast<uint32_t>(p.cache.k.sb / 16), kslot = static_cast<uint32_t>(p.cache.k.ss / 16);
  const uint32_t vp = static_cast<uint32_t>(p.cache.v.sb / 16), vslot = static_cast<uint32_t>(p.cache.v.ss / 16);
  const uint32_t fkp = static_cast<uint32_t>(p.ks[0]), fkb = static_cast<uint32_t>(p.ks[1]);
  const uint32_t fvp = static_cast<uint32_t>(p.vs[0]), fvb = static_cast<uint32_t>(p.vs[1]);
  // The walk stands at the tile that is planned: it moves on when the next one is.
  uint32_t pend_page = 0, pend_within = 0;
  int flags = kBegin;
  bool pend_live = false;
  int units = 0;  // of the line that the planned tile takes: two, or the one that is left
  auto plan = [&]() {  // moves on and looks the tile up
    pend_live = false;
    if (left == 0) {
      flags = kNone;
      return;
    }
    if (units > 0) {
      flags &= kSecond;
      ct += units;
      if (ct == cnt) {
        ct = 0;
        flags = kBegin | kSecond;
        seg_from_start = true;
        if (++ch == line_heads) {
          ch = 0;
          do {
            ++cb;
            load_seq(len_of(cb));
          } while (cnt == 0 && cb + 1 < p.batch);
        }
        load_head();
      }
    }
    units = left > 1 && ct + 1 < cnt ? 2 : 1;
    left -= units;
    if (ct + units == cnt) flags |= seg_from_start ? kEnd | kFull : kEnd;
    if (left == 0) flags |= kEnd;
    // a warp has 32 keys of two units, 16 of one
    const int j = cfirst + ct * kUnit + warp * (units * kUnit / kWarps) + lane;
    pend_live = lane < units * kUnit / kWarps && j < cn;
    if (pend_live) {
      const uint32_t n = p.cache.page.div(static_cast<uint32_t>(j));
      pend_within = static_cast<uint32_t>(j) - n * p.cache.page.d;
      pend_page = static_cast<uint32_t>(table[n]);
    }
  };
  // Writes the tile's addresses and descriptor down and asks for its factors.
  uint32_t live_w = 0;  // its keys
  auto store_plan = [&](int slot) {
    bool ok = pend_live;
    if (ok && pend_page >= static_cast<uint32_t>(p.cache.num_pages)) {
      report(p.status, kBadPage);
      ok = false;
    }
    longlong2 o = make_longlong2(0, 0);  // addresses of the key's row of k and of v
    const float *fk = p.k_scale, *fv = p.v_scale;
    if (ok) {
      const uint64_t page = pend_page, in = pend_within;
      o.x = reinterpret_cast<long long>(khead + ((page * kp + in * kslot) << 4));
      o.y = reinterpret_cast<long long>(vhead + ((page * vp + in * vslot) << 4));
      const uint64_t blk = p.block.div(pend_within);
      fk = ksh + (page * fkp + blk * fkb);
      fv = vsh + (page * fvp + blk * fvb);
    }
    const uint32_t at = factors_u + (slot * kKeys + lane) * 8;
    cp_async4_or_zero(at, fk, ok);
    cp_async4_or_zero(at + 4, fv, ok);
    rows[lane] = o;
    live_w = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) desc[slot] = make_int4(cb, line + ch, flags, static_cast<int>(live_w));
  };
  // Issues the copies of part `sub` of the tile whose plan was stored last, if there is one.
  constexpr int kLanes = DP == 64 ? 4 : (DP <= 128 ? 8 : 16), kStep = 32 / kLanes, kIter = kSubKeys / kStep;
  const int cc = lane % kLanes, cr = lane / kLanes;
  const uint32_t copy_u = ring_u + cr * DP + ((cc ^ perm8<DP>(cr)) << 4);
  auto fetch = [&](int sub, int stage) {
    const uint32_t live = live_w >> (sub * kSubKeys);
    constexpr uint32_t kAll = kSubKeys == 32 ? 0xffffffffu : 0xffffu;
    if ((live & kAll) != 0 && cc < p.chunks) {
      const uint32_t dst = copy_u + stage * C::kStageBytes;
      const longlong2* from = rows + sub * kSubKeys + cr;
      auto to = [&](int i) { return (dst ^ (perm8<DP>(i * kStep) << 4)) + i * kStep * DP; };
      if ((live & kAll) == kAll) {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const longlong2 a = from[i * kStep];
          cp_async16(to(i), a.x + cc * 16);
          cp_async16(to(i) + kSubKeys * DP, a.y + cc * 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const longlong2 a = from[i * kStep];
          const bool ok = a.x != 0;
          cp_async16_or_zero(to(i), ok ? a.x + cc * 16 : reinterpret_cast<long long>(p.cache.k.ptr), ok);
          cp_async16_or_zero(to(i) + kSubKeys * DP, ok ? a.y + cc * 16 : reinterpret_cast<long long>(p.cache.v.ptr), ok);
        }
      }
    }
    cp_commit();
  };
  plan();
  int slot_w = 0, stage_w = 0;  // of the next tile to store, of the next part to fetch
  auto next_stage = [&]() { stage_w = stage_w + 1 == S ? 0 : stage_w + 1; };
  for (int t = 0; t < C::kAhead; ++t) {
    store_plan(slot_w);
    plan();
    __syncwarp();
#pragma unroll
    for (int sub = 0; sub < kSubs; ++sub) {
      fetch(sub, stage_w);
      next_stage();
    }
    ++slot_w;  // kAhead < kSlots
    __syncwarp();
  }

  // ================================================== attention
  uint32_t qf[HN][kSteps][2];
  float qscale[HN][2];  // of heads 2 (lane % 4) and the next: times s_j ks_j the logit (base 2, or under the cap)
  float o[kSteps][HN][4];
  float m[HN][2], base[HN][2], l[HN][2];  // base: m, or 0 without keys so far
  const int g8 = lane >> 2, q4 = lane & 3;
  int b = 0, h0 = 0, hn = 0;
  // ldmatrix: this lane's key and chunk 0 or 1
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t load_u = ring_u + lrow * DP + (((lane >> 4) ^ perm8<DP>(lrow)) << 4);
  int slot = 0, stage = 0;
  for (;;) {
    cp_wait<S - 2>();
    __syncwarp();  // the copies of all lanes are there, and the last part's stage is free
    const int4 d = desc[slot];
    if (d.z & kNone) break;
    const float2* factor = factors + slot * kKeys + g8;
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    // the tile kAhead ahead
    store_plan(slot_w);
    plan();
    __syncwarp();
    fetch(0, stage_w);
    next_stage();

    if (d.z & kBegin) {
      const int g = d.y / p.head_tiles, ht = d.y - g * p.head_tiles;
      b = d.x;
      h0 = g * p.group + ht * kMaxRows;
      hn = min(kMaxRows, p.group - ht * kMaxRows);
      const float unit = p.softcap > 0.f ? p.cap_in : p.scale_log2;
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
        float mul = 1.f;
        if (p.bf16) {  // the row's largest element to [2^15, 2^16): of bf16 at most 65280, which fp16 holds
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = max(static_cast<int>(top >> 23) - 127 - 15, -126);
          const float down = __int_as_float((127 - e) << 23);
          mul = __int_as_float((127 + e) << 23);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 x = Pack<__nv_bfloat16>::unpack(qf[n][k][i]);
              qf[n][k][i] = Pack<__half>::two(x.x * down, x.y * down);
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          qscale[n][c] = __shfl_sync(0xffffffffu, mul, (2 * q4 + c) * 4) * unit;
          m[n][c] = -INFINITY;
          base[n][c] = l[n][c] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
      }
    }

#pragma unroll 1
    for (int sub = 0; sub < kSubs; ++sub) {
      if (sub > 0) {
        cp_wait<S - 2>();
        __syncwarp();
        fetch(sub, stage_w);
        next_stage();
      }
      const uint32_t kst = load_u + stage * C::kStageBytes;
      stage = stage + 1 == S ? 0 : stage + 1;
      constexpr uint32_t kAllKeys = kSubKeys == 32 ? 0xffffffffu : 0xffffu;
      const uint32_t live = (static_cast<uint32_t>(d.w) >> (sub * kSubKeys)) & kAllKeys;
      if (live == 0) continue;

      // ---- base-2 logits of this warp's keys; V's factors and their exponents
      float y[kGroups][HN][4], e[kGroups][2], fv[kGroups][2];
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
          ldsm4(chunk_at<DP>(kst, k) + gr * 16 * DP, x);
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
          const int kk = gr * 16 + i * 8;
          const float2 f = factor[sub * kSubKeys + kk];
          const float v = fminf(fmaxf(f.y, kLeast), kMost);
          e[gr][i] = __uint_as_float(0x4b000000u | (__float_as_uint(v) >> 23)) - 8388735.f;  // 2^23 + 127
          fv[gr][i] = f.y == 0.f ? 0.f : v * kWeight;
#pragma unroll
          for (int n = 0; n < HN; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)  // (ks times q's scale may be beyond fp32, beside a sum of 0)
              y[gr][n][i * 2 + c] = (s[n][0][i * 2 + c] + s[n][1][i * 2 + c]) * f.x * qscale[n][c];
        }
      }
      if (p.softcap > 0.f) {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
          for (int n = 0; n < HN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[gr][n][i] = p.cap_out * tanh_exp(y[gr][n][i]);
      }
      if (live != kAllKeys) {
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!((live >> (gr * 16 + i * 8 + g8)) & 1u))
#pragma unroll
              for (int n = 0; n < HN; ++n) y[gr][n][i * 2] = y[gr][n][i * 2 + 1] = -INFINITY;
      }
      bool moved = false;
#pragma unroll
      for (int gr = 0; gr < kGroups; ++gr)
#pragma unroll
        for (int n = 0; n < HN; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) moved |= y[gr][n][i] + e[gr][i >> 1] > m[n][i & 1];
      // ---- the running maximum
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < HN; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = -INFINITY;
#pragma unroll
            for (int gr = 0; gr < kGroups; ++gr)
              top = fmaxf(top, fmaxf(y[gr][n][c] + e[gr][0], y[gr][n][c + 2] + e[gr][1]));
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
            const float mx = fmaxf(m[n][c], top);
            // (in halves: a step may be larger than fp32's exponents, where the sum starts at 2^60)
            const float h = mx == m[n][c] ? 1.f : ex2(0.5f * (m[n][c] - mx)), f = h * h;
            m[n][c] = mx;
            base[n][c] = mx == -INFINITY ? 0.f : mx;
            l[n][c] = l[n][c] * h * h;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              o[k][n][c] *= f;
              o[k][n][c + 2] *= f;
            }
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
            const float p0 = ex2(y[gr][n][i * 2] - base[n][0]), p1 = ex2(y[gr][n][i * 2 + 1] - base[n][1]);
            l[n][0] += p0;
            l[n][1] += p1;
            const float w0 = p0 * fv[gr][i], w1 = p1 * fv[gr][i];
            const uint32_t h = Pack<__half>::two(w0, w1);
            const float2 back = Pack<__half>::unpack(h);
            hi[n][i] = transposed(h);
            lo[n][i] = transposed(Pack<__half>::two(w0 - back.x, w1 - back.y));
          }
#pragma unroll
        for (int k = 0; k < kSteps; k += 2) {
          uint32_t x[4], a[8];
          ldsm4_t(chunk_at<DP>(kst, k) + (kSubKeys + gr * 16) * DP, x);
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
    slot_w = slot_w + 1 == kSlots ? 0 : slot_w + 1;

    if (d.z & kEnd) {
      // ---- this run's part of the segment is complete: the warps' O are added up
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
      const bool whole = (d.z & kFull) != 0;
      float* part = partial(p, blockIdx.x, (d.z & kSecond) ? 1 : 0);
      // Eight heads at a time each warp leaves its O in the stage that it worked on last, which
      // the next copy will take: [head][column], columns permuted by the head.
      const int done = stage == 0 ? S - 1 : stage - 1;
#pragma unroll
      for (int n = 0; n < HN; ++n) {
        const int heads = min(8, hn - n * 8);
        if (heads <= 0) break;
        float* to = reinterpret_cast<float*>(mine + done * C::kStageBytes);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (2 * q4 + c < heads)
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
              *reinterpret_cast<float2*>(to + (2 * q4 + c) * DP + ((k * 16 + 2 * g8) ^ (q4 * 8))) =
                  make_float2(o[k][n][c], o[k][n][c + 2]);
        __syncthreads();
        for (int i = tid; i < heads * (DP / 2); i += kThreads) {
          const int in = i / (DP / 2), col = (i - in * (DP / 2)) * 2, row = n * 8 + in;
          const unsigned char* from = smem + done * C::kStageBytes + (in * DP + (col ^ ((in >> 1) * 8))) * 4;
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_max[w][row]);
          const float low = top == -INFINITY ? 0.f : top;
          float2 x = make_float2(0.f, 0.f);
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 y = *reinterpret_cast<const float2*>(from + w * C::kWarpBytes);
            const float h = ex2(0.5f * (s_max[w][row] - low)), f = h * h;
            x.x = fmaf(y.x, f, x.x);
            x.y = fmaf(y.y, f, x.y);
            sum = fmaf(s_sum[w][row] * h, h, sum);
          }
          if (whole) {
            const bool none = sum == 0.f;
            const float inv = none ? 0.f : 1.f / kWeight / sum;
            const float u = none ? 0.f : x.x * inv, v = none ? 0.f : x.y * inv;
            uint16_t* out = static_cast<uint16_t*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + (h0 + row) * p.o.sh;
            if (col < p.head_dim)
              *reinterpret_cast<uint32_t*>(out + col) = p.bf16 ? Pack<__nv_bfloat16>::two(u, v) : Pack<__half>::two(u, v);
            if (col == 0 && p.lse != nullptr)
              p.lse[static_cast<int64_t>(b) * p.h_q + h0 + row] =
                  none ? INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
          } else {
            // the maximum without V's exponents, as the kernel that joins takes it: the sum lies in [1, 2)
            const int e = sum > 0.f ? min(max(static_cast<int>(__float_as_uint(sum) >> 23) - 127, -126), 126) : 0;
            const float down = __int_as_float((127 - e) << 23);
            *reinterpret_cast<float2*>(part + row * DP + col) =
                make_float2(x.x * (1.f / kWeight) * down, x.y * (1.f / kWeight) * down);
            if (col == 0) {
              part[p.part_rows * DP + row] = top + static_cast<float>(e);
              part[p.part_rows * DP + kMaxRows + row] = sum * down;
            }
          }
        }
        __syncthreads();  // all of it has been read
      }
      zero_columns(done, 1);
    }
  }
  cp_wait<0>();
}

template <int DP, int HN, bool INT8>
cudaError_t launch_main(Decode8Params p, cudaStream_t stream) {
  using C = Cfg<DP, HN>;
  static std::atomic<unsigned long long> done{0};  // devices with the attribute set
  int runs;
  cudaError_t e = shape_decode(p, kUnitLog2, C::kBlocks, &runs);
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
  return p.whole ? cudaSuccess : launch_join(p, p.bf16 ? ATTN_BF16 : ATTN_FP16, runs, true, stream);
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
