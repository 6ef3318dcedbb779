// Attention of one new token a sequence over the paged cache (attn_decode).
//
// For each (sequence, key/value head) the query heads of the group share every key and
// value, so the work is one pass over the cached rows: bound by the memory they lie in.
// With up to 16 query heads as the M rows of an m16n8k16 product, S = Q K^T and O += P V
// keep the tensor pipe busy for a fifth of the time at full memory speed (heads of 128; groups
// above 8 half as long again), so the products are kept small and synchronous and the design
// goes into the loads.
//
// Split.  Keys come in tiles of about 32 KB (128 keys of 64 columns, 64 of
// up to 128, 32 above; rows of 65 to 96 columns take 192 bytes and four stages: 64 sequences
// of 4000 keys, 8 heads of 96, 129 us against 138 with 256 bytes and three, of 80 119 and 127,
// of 72 139 and 148; but 16 heads without groups of 72 291 both ways, of 88 337 and 329).
// All tiles of all (sequence, head) segments form one line, cut into equal runs, one per
// resident block: ragged lengths balance by themselves, and one long sequence uses every
// SM.  Where the blocks divide among the heads, every head has a line of its own instead,
// all cut alike, and neighbouring blocks walk the same keys of different heads in step: a
// token's heads lie side by side in memory, and rows that are not whole 128-byte lines
// would otherwise be fetched again for the next head (heads of 112, 32 sequences up to
// 8192 keys: 630 MB read for 491, 105 us; in step 86 us).  A segment that lies inside one run
// is finished there; one that is cut leaves (O, maximum, sum) partials which a second small
// kernel joins (it is launched early and waits for the first).  The cut depends on the lengths
// alone, so results do not depend on timing.  (More and shorter runs, taken over by blocks as
// they finish, were slower: when 64 sequences of 4096 to 16384 keys took 425 us, 380 since, two
// runs a block took 428 and four 432.)  Where no sequence passes kWholeKeys a block takes one
// segment and nothing is joined.
//
// Block.  Two warps look the pages up and keep a ring of shared-memory stages filled with
// 16-byte asynchronous copies, several tiles ahead; eight warps compute; two blocks share
// an SM.  The 16-byte chunks of row r lie permuted by r % 8 inside each 128 bytes, so that
// neither the copies nor ldmatrix meet a bank conflict (with padded rows the copies alone
// were 4 % slower).  Of a tile the compute warps first take the logits of 8 keys each (16
// of 128; of 32 keys, 8 keys over half of the columns), then the softmax of one or two rows
// each, a lane a key or two, then an eighth of the columns of O over all keys (larger groups:
// below).
// (With four warps that also did the copies, the chain of dependent steps of a tile took
// 3100 cycles against 2600 for its loads.)
//
// P enters the P V product as two numbers of the inputs' type, its rounded value and the rounded
// remainder, so that the weights are right to 2^-16 in bf16 and 2^-22 in fp16 and O's error is
// that of its own rounding.  (With the rounded value alone it was 1.3 to 1.4 times that.)  Groups
// of up to 8 query heads have the remainders in the product's rows 8 to 15, which are empty
// there, at no cost (64 sequences of 4000 keys, 8 heads of 128: 152 us with and without).  Larger
// groups (kLarge) take a second product: 4 heads of 64 with 16 query heads each 61.5 us against
// 57.3, 64 heads on one of 128 95.7 against 83.9.  There the warps read P from shared memory at
// a rate near its limit (eight warps all of it, for their columns), so that two or four of them
// share columns and take a part of the tile's keys each; with all keys a warp the same took
// 68.4 and 99.7.  (Parts for the smaller groups too made heads of 80 6 % slower.)  In fp16 P is
// taken times 2^15 (kPScale), so that its finest step is 2^-39 of the largest weight.
// (Unscaled, weights vanished below 2^-25: 16383 keys beside one of 2^30 times their weight and
// of value 0 gave O = 0 in place of 1.5e-5.)  The sum itself, maxima and logits stay fp32,
// without the factor.
#include <atomic>

#include "decode.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;       // compute warps
constexpr int kCompute = kWarps * 32;
constexpr int kCopy = 64;       // copying threads
constexpr int kThreads = kCompute + kCopy;
constexpr int kJoin = 128;      // threads of a join block
constexpr int kAhead = 8;       // partials of a lane in flight there
constexpr int kBlocks = 2;      // of an SM

// Factor of P in shared memory and of O until it is written (a power of two: exact).
template <typename T>
constexpr float kPScale = Pack<T>::kIsBf16 ? 1.f : 32768.f;

constexpr int tile_log2(int dp) { return dp == 64 ? 7 : (dp <= 128 ? 6 : 5); }

template <int DP, bool kLarge>
struct Cfg {
  static constexpr int kTile = 1 << tile_log2(DP);       // keys of a tile
  static constexpr int kPitch = DP * 2;
  static constexpr int kStageBytes = 2 * kTile * kPitch;
  static constexpr int kStages = DP == 96 || DP == 192 ? 4 : 3;  // 96 KB
  static constexpr int kSlots = kStages + 2;             // descriptors
  static constexpr int kPlan = kTile > kCopy ? kTile / kCopy : 1;  // keys a copying thread looks up
  static constexpr int kSplits = kTile == 32 ? 2 : 1;    // warps that share a key's logits
  static constexpr int kSPitch = kTile * 4 + 16;         // bytes of a row of logits, then of P
  // warps that share columns of O, each over its part of the tile's keys
  static constexpr int kParts = !kLarge || kTile == 32 ? 1 : kTile / 32;
  static constexpr int kSBytes = kSplits * kMaxRows * kSPitch;
  static constexpr int kXBytes = kParts / 2 * kMaxRows * DP * 4;  // O of half of them, in the same place
  static constexpr int kSBuf = kSBytes > kXBytes ? kSBytes : kXBytes;
  static constexpr int kSmem = kStages * kStageBytes + 2 * kTile * 16 + kSlots * 48 + kSBuf + kLens * 4;
};

struct __align__(16) TileDesc {
  int b, hv, rel;  // sequence, head tile, first key of the tile (from the first seen)
  int flags;
  uint32_t valid[4];  // bit per key of the tile
  int pad[4];
};

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

// What a row's chunk numbers are permuted by (exclusive or): eight rows, four of them where a
// row is one and a half times 128 bytes and its neighbours start 64 bytes apart.
template <int DP>
__host__ __device__ constexpr int perm(int row) {
  return DP % 64 == 0 ? row & 7 : (row >> 1) & 3;
}

// Copies the rows of a tile, kLanes of the copying threads to a row.  `rows`: the addresses
// of each key's rows of k and of v.
// Addresses are read eight at a time before their copies are issued: a copy writes shared
// memory, so a read behind it in program order waits until it has been issued.
template <int DP>
__device__ __forceinline__ void copy_rows(const longlong2* rows, const uint32_t* valid, uint32_t dst,
                                          int idx, const DecodeParams& p) {
  constexpr int kLanes = DP == 64 ? 8 : (DP <= 128 ? 16 : 32), kStep = kCopy / kLanes;
  constexpr int kTile = Cfg<DP, false>::kTile, kIter = kTile / kStep, kPitch = Cfg<DP, false>::kPitch;
  const int c = idx % kLanes, r0 = idx / kLanes;
  if (c >= p.chunks) return;
  rows += r0;
  dst += r0 * kPitch + ((c ^ perm<DP>(r0)) << 4);  // r0 < kStep, and kStep divides 8
  auto at = [&](int i) { return (dst ^ (perm<DP>(i * kStep) << 4)) + i * kStep * kPitch; };
  uint32_t all = valid[0];
#pragma unroll
  for (int i = 1; i < kTile / 32; ++i) all &= valid[i];
  if (all == 0xffffffffu) {
    static_assert(kIter % 8 == 0, "groups of eight rows");
#pragma unroll
    for (int i0 = 0; i0 < kIter; i0 += 8) {
      longlong2 a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = rows[(i0 + i) * kStep];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cp_async16(at(i0 + i), a[i].x + c * 16);
        cp_async16(at(i0 + i) + kTile * kPitch, a[i].y + c * 16);
      }
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < kIter; ++i) {
      const longlong2 a = rows[i * kStep];
      const bool ok = a.x != 0;
      const long long k = ok ? a.x + c * 16 : reinterpret_cast<long long>(p.cache.k.ptr);
      const long long v = ok ? a.y + c * 16 : reinterpret_cast<long long>(p.cache.v.ptr);
      cp_async16_or_zero(at(i), k, ok);
      cp_async16_or_zero(at(i) + kTile * kPitch, v, ok);
    }
  }
}

// O and what P's remainders add to it.  Of an infinite value a remainder of 0 or below makes
// a NaN, where the weight itself has made the infinity that O is.
__device__ __forceinline__ float with_rest(float o, float rest) {
  return fabsf(rest) < INFINITY ? o + rest : o;
}

// Barrier of the compute warps.
__device__ __forceinline__ void compute_barrier() {
  asm volatile("bar.sync 2, %0;" ::"n"(kCompute) : "memory");
}

template <typename T, int DP, bool kLarge>
__global__ void __launch_bounds__(kThreads, kBlocks)
    decode_kernel(DecodeParams p) {
  using C = Cfg<DP, kLarge>;
  constexpr int S = C::kStages, kPitch = C::kPitch, kSlots = C::kSlots, kTile = C::kTile;
  constexpr int kSteps = DP / 16 / C::kSplits;  // k-steps of Q K^T of a warp
  constexpr int kGroups = kTile == 128 ? 2 : 1; // groups of 8 keys of a warp
  constexpr int kPer = kTile / 32;      // keys of a lane in the softmax
  constexpr int kPair = kPer > 1 ? 2 : 1;  // of them neighbours
  constexpr int kSets = kLarge ? 2 : 1; // of 8 query heads
  constexpr int kParts = C::kParts, kColWarps = kWarps / kParts;
  // columns of O of a warp (of 96 two warps have none, but with parts)
  constexpr int kCols = DP == 96 && kParts == 1 ? 16 : DP / kColWarps;
  constexpr int kNt = kCols / 8;        // their n-tiles
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int s_sums[kThreads / 32];
  __shared__ int s_pre[kThreads];
  __shared__ float s_scale[kMaxRows], s_max[kMaxRows], s_sum[kMaxRows];
  unsigned char* ring = smem;
  longlong2* rows = reinterpret_cast<longlong2*>(ring + S * C::kStageBytes);  // of two tiles
  TileDesc* desc = reinterpret_cast<TileDesc*>(rows + 2 * kTile);
  unsigned char* sbuf = reinterpret_cast<unsigned char*>(desc + kSlots);      // logits, then P
  int* lens = reinterpret_cast<int*>(sbuf + C::kSBuf);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hv_n = p.h_k * p.head_tiles;
  // lines: one of all heads, or one of each; this block's line and its run of it
  const int line_heads = p.lines > 1 ? 1 : hv_n;
  const int run = blockIdx.x / p.lines, line = blockIdx.x - run * p.lines;
  const uint32_t ring_u = smem_u32(ring);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this block's run of tiles
  const int per = (p.batch + kThreads - 1) / kThreads;
  Cut cut;
  if (p.whole) {
    const int b = blockIdx.x / hv_n, n = clean_len(p, p.seqlens[b], true);
    if (n == 0) {
      no_keys<T>(p, b, blockIdx.x - b * hv_n);
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
  if (p.head_dim < DP) {
    const int c0 = p.head_dim / 8, nc = DP / 8 - c0;
    for (int i = tid; i < S * 2 * kTile * nc; i += kThreads)
      *reinterpret_cast<uint4*>(ring + (i / nc) * kPitch + (((c0 + i % nc) ^ perm<DP>(i / nc)) << 4)) =
          make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  if (warp >= kWarps) {
    // ================================================== copies, one thread a key
    const int key = tid - kCompute;
    int left = 0;
    int cb = 0, ch = 0, ct = 0, cn = 0, cfirst = 0, cnt = 0;
    bool seg_from_start = true;
    int nth = 0;  // segment of the run: 0 first, then 1
    int begin = 1;
    // of the sequence: its keys and its table row; of the segment: the head's rows of slot 0
    const int* table = nullptr;
    const char *khead = nullptr, *vhead = nullptr;
    auto load_seq = [&](int n) {
      cn = n;
      cfirst = first_key(p, cn);
      cnt = (cn - cfirst + kTile - 1) / kTile;
      table = p.cache.table + cb * p.cache.table_stride;
    };
    auto load_head = [&]() {
      const int hv = line + ch, g = hv / p.head_tiles, ht = hv - g * p.head_tiles;
      khead = reinterpret_cast<const char*>(static_cast<const T*>(p.cache.k.ptr) + g * p.cache.k.sh);
      vhead = reinterpret_cast<const char*>(static_cast<const T*>(p.cache.v.ptr) + g * p.cache.v.sh);
      // its queries are asked for a few tiles ahead
      const int h = g * p.group + ht * kMaxRows + (key & 15);
      if (h < (g + 1) * p.group)
        for (int i = (key >> 4) * 64; i < p.head_dim; i += 256)
          prefetch_l2(static_cast<const T*>(p.q.ptr) + cb * p.q.sb + h * p.q.sh + i);
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
    const uint32_t kp = static_cast<uint32_t>(p.cache.k.sb / 8), ks = static_cast<uint32_t>(p.cache.k.ss / 8);
    const uint32_t vp = static_cast<uint32_t>(p.cache.v.sb / 8), vs = static_cast<uint32_t>(p.cache.v.ss / 8);
    // what plan() saw, for store_plan()
    int pend_page[C::kPlan], pend_within[C::kPlan];
    bool pend_live[C::kPlan];
    const char *pend_k = nullptr, *pend_v = nullptr;
    int4 pend = make_int4(0, 0, 0, 0);
    auto plan = [&]() {  // looks one tile up and moves on
#pragma unroll
      for (int i = 0; i < C::kPlan; ++i) pend_live[i] = false;
      if (left == 0) {
        pend.w = kNone;
        return;
      }
      pend_k = khead;
      pend_v = vhead;
#pragma unroll
      for (int i = 0; i < C::kPlan; ++i) {
        const int k = key + i * kCopy, j = cfirst + ct * kTile + k;
        pend_live[i] = j < cn && k < kTile;
        if (pend_live[i]) {
          const int n = static_cast<int>(p.cache.page.div(static_cast<uint32_t>(j)));
          pend_within[i] = j - n * static_cast<int>(p.cache.page.d);
          pend_page[i] = table[n];
        }
      }
      const bool at_end = ct == cnt - 1;
      pend = make_int4(cb, line + ch, ct * kTile,
                       (begin ? kBegin : 0) | (at_end || left == 1 ? kEnd : 0) |
                           (at_end && seg_from_start ? kFull : 0) | (nth ? kSecond : 0));
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
    auto store_plan = [&](int tile) {
      TileDesc& d = desc[tile % kSlots];
#pragma unroll
      for (int i = 0; i < C::kPlan; ++i) {
        bool ok = pend_live[i];
        if (ok && static_cast<unsigned>(pend_page[i]) >= static_cast<unsigned>(p.cache.num_pages)) {
          report(p.status, kBadPage);
          ok = false;
        }
        longlong2 o = make_longlong2(0, 0);  // addresses of the key's row of k and of v
        if (ok) {
          const uint64_t page = static_cast<uint32_t>(pend_page[i]), in = static_cast<uint32_t>(pend_within[i]);
          o.x = reinterpret_cast<long long>(pend_k + ((page * kp + in * ks) << 4));
          o.y = reinterpret_cast<long long>(pend_v + ((page * vp + in * vs) << 4));
        }
        const int k = key + i * kCopy;
        if (k < kTile) rows[(tile & 1) * kTile + k] = o;
        const uint32_t bits = __ballot_sync(0xffffffffu, ok);
        if (lane == 0 && k < kTile) d.valid[k >> 5] = bits;
      }
      if (key == 0) *reinterpret_cast<int4*>(&d) = pend;
    };
    auto fetch = [&](int tile) {  // issues the copies of one tile, if there is one
      const TileDesc& d = desc[tile % kSlots];
      if (!(d.flags & kNone))
        copy_rows<DP>(rows + (tile & 1) * kTile, d.valid, ring_u + (tile % S) * C::kStageBytes, key, p);
      cp_commit();
    };
    // the first copies leave as soon as their rows are known
    plan();
    for (int t = 0; t < S - 1; ++t) {
      store_plan(t);
      plan();
      asm volatile("bar.sync 1, %0;" ::"n"(kCopy) : "memory");  // rows and descriptor of tile t
      fetch(t);
    }
    store_plan(S - 1);
    plan();  // tile S waits in the registers
    __syncthreads();
    for (int t = 0; !(desc[t % kSlots].flags & kNone); ++t) {
      cp_wait<S - 2>();
      __syncthreads();  // tile t is there for all; the stage of tile t - 1 is free
      fetch(t + S - 1);
      store_plan(t + S);
      plan();
    }
    cp_wait<0>();
    return;
  }

  // ==================================================== attention
  uint32_t qf[kSteps][4];
  float o[kNt][4];
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // softmax of rows `warp` and `warp` + 8
  const int row0 = lane >> 2, col2 = (lane & 3) * 2;
  const int cw = warp % kColWarps, part_of = warp / kColWarps;
  const bool has_columns = DP % (kCols * kColWarps) == 0 || cw * kCols < DP;
  const int group8 = C::kSplits == 2 ? warp & 3 : warp, split = C::kSplits == 2 ? warp >> 2 : 0;
  int b = 0, h0 = 0, hn = 0;  // of the segment: sequence, first query head and their number
  __syncthreads();
  for (int t = 0;; ++t) {
    const TileDesc& d = desc[t % kSlots];
    if (d.flags & kNone) break;
    if (d.flags & kBegin) {
      const int g = d.hv / p.head_tiles, ht = d.hv - g * p.head_tiles;
      b = d.b;
      h0 = g * p.group + ht * kMaxRows;
      hn = min(kMaxRows, p.group - ht * kMaxRows);
      const T* q = static_cast<const T*>(p.q.ptr) + b * p.q.sb;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = row0 + (i & 1) * 8, col = (split * kSteps + k) * 16 + col2 + (i >> 1) * 8;
          qf[k][i] = row < hn && col < p.head_dim
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
    __syncthreads();  // tile t is there for all

    // ---- products of q with this warp's keys
    const uint32_t kst = ring_u + (t % S) * C::kStageBytes;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) {
      float s[4], s1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = s1[i] = 0.f;
      const int k0 = (group8 + gr * kWarps) * 8;
      const uint32_t a = kst + (k0 + (lane & 7)) * kPitch;
#pragma unroll
      for (int k = 0; k < kSteps; k += 2) {
        uint32_t kf[4];
        ldsm4(a + (((split * kSteps * 2 + k * 2 + (lane >> 3)) ^ perm<DP>(lane & 7)) << 4), kf);
        mma16816<T>(s, qf[k], kf[0], kf[1]);
        mma16816<T>(s1, qf[k + 1], kf[2], kf[3]);
      }
#pragma unroll
      for (int r = 0; r < kSets; ++r)
        *reinterpret_cast<float2*>(sbuf + (split * kMaxRows + row0 + r * 8) * C::kSPitch + (k0 + col2) * 4) =
            make_float2(s[r * 2] + s1[r * 2], s[r * 2 + 1] + s1[r * 2 + 1]);
    }
    compute_barrier();

    // ---- softmax of this warp's rows; P takes the place of the logits.  A lane takes kPair
    // neighbouring keys of every 32 * kPair.
#pragma unroll
    for (int r = 0; r < kSets; ++r) {
      const int row = warp + r * 8;
      if (row >= hn) break;
      float* srow = reinterpret_cast<float*>(sbuf + row * C::kSPitch);
      float x[kPer], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; i += kPair) {
        const int key = kPair * lane + 32 * i;
        if (kPair == 2) {
          const float2 v = *reinterpret_cast<const float2*>(srow + key);
          x[i] = v.x;
          x[i + kPair - 1] = v.y;
        } else {
          x[i] = srow[key];
        }
        const uint32_t valid = d.valid[key >> 5] >> (key & 31);
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          float& y = x[i + k];
          if (C::kSplits == 2)
            y += reinterpret_cast<const float*>(sbuf + (kMaxRows + row) * C::kSPitch)[key + k];
          y = p.softcap > 0.f ? p.cap_out * tanh_exp(y * p.cap_in) : y * p.scale_log2;
          if (!((valid >> k) & 1u)) y = -INFINITY;
          top = fmaxf(top, y);
        }
      }
      if (p.logits != nullptr) {
        float* out = p.logits + (static_cast<int64_t>(b) * p.h_q + h0 + row) * p.logit_stride + d.rel +
                     kPair * lane;
#pragma unroll
        for (int i = 0; i < kPer; i += kPair)
          if (kPair == 2)
            *reinterpret_cast<float2*>(out + 32 * i) = make_float2(x[i], x[i + kPair - 1]);
          else
            out[32 * i] = x[i];
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      const float mx = fmaxf(m[r], top), base = mx == -INFINITY ? 0.f : mx;
      const float scale = ex2(m[r] - base);
      float sum = 0.f;
      T* prow = reinterpret_cast<T*>(srow);
      T* rest = kLarge ? prow + kTile : reinterpret_cast<T*>(sbuf + (row + 8) * C::kSPitch);
#pragma unroll
      for (int i = 0; i < kPer; i += kPair) {
        const int key = kPair * lane + 32 * i;
        const float e0 = ex2(x[i] - base), e1 = kPair == 2 ? ex2(x[i + kPair - 1] - base) : 0.f;
        sum += e0 + e1;
        const uint32_t hi = Pack<T>::two(e0 * kPScale<T>, e1 * kPScale<T>);
        const float2 h = Pack<T>::unpack(hi);
        const uint32_t lo = Pack<T>::two(e0 * kPScale<T> - h.x, e1 * kPScale<T> - h.y);
        if (kPair == 2) {
          *reinterpret_cast<uint32_t*>(prow + key) = hi;
          *reinterpret_cast<uint32_t*>(rest + key) = lo;
        } else {
          reinterpret_cast<unsigned short*>(prow)[key] = static_cast<unsigned short>(hi);
          reinterpret_cast<unsigned short*>(rest)[key] = static_cast<unsigned short>(lo);
        }
      }
      m[r] = mx;
      l[r] = l[r] * scale + sum;
      if (lane == 0) {
        s_scale[row] = scale;
        if (!kLarge) s_scale[row + 8] = scale;
      }
    }
    compute_barrier();

    // ---- O += P V for this warp's columns
    if (has_columns) {
      const float c0 = s_scale[row0], c1 = s_scale[row0 + 8];
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
        o[n][0] *= c0;
        o[n][1] *= c0;
        o[n][2] *= c1;
        o[n][3] *= c1;
      }
      const int first = part_of * (kTile / kParts);  // key of this warp's part
      const uint32_t pa = smem_u32(sbuf) + (lane & 15) * C::kSPitch + (lane >> 4) * 16 + first * 2;
      const uint32_t va = kst + (kTile + first + lane) * kPitch;
      float rest[kNt][4];
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) rest[n][i] = 0.f;
#pragma unroll
      for (int k = 0; k < kTile / 32 / kParts; ++k) {
        uint32_t p0[4], p1[4], r0[4], r1[4];
        ldsm4(pa + k * 64, p0);
        ldsm4(pa + k * 64 + 32, p1);
        if (kLarge) {
          ldsm4(pa + kTile * 2 + k * 64, r0);
          ldsm4(pa + kTile * 2 + k * 64 + 32, r1);
        }
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          uint32_t vf[4];
          ldsm4_t(va + k * 32 * kPitch + (((cw * kNt + n) ^ perm<DP>(lane)) << 4), vf);
          mma16816<T>(o[n], p0, vf[0], vf[1]);
          if (kLarge) mma16816<T>(rest[n], r0, vf[0], vf[1]);
          mma16816<T>(o[n], p1, vf[2], vf[3]);
          if (kLarge) mma16816<T>(rest[n], r1, vf[2], vf[3]);
        }
      }
      if (kLarge)
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[n][i] = with_rest(o[n][i], rest[n][i]);
    }

    if (d.flags & kEnd) {
      // ---- this run's part of the segment is complete
      if (!kLarge)
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
          o[n][0] = with_rest(o[n][0], o[n][2]);
          o[n][1] = with_rest(o[n][1], o[n][3]);
        }
#pragma unroll
      for (int r = 0; r < kSets; ++r) {
        float x = l[r];
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) x += __shfl_xor_sync(0xffffffffu, x, i);
        if (lane == 0) {
          s_sum[warp + r * 8] = x;
          s_max[warp + r * 8] = m[r];
        }
      }
      compute_barrier();
      // the warps' parts of O are added up, half of them to the others at a time
#pragma unroll
      for (int h = kParts / 2; h > 0; h /= 2) {
        float* x = reinterpret_cast<float*>(sbuf) + ((part_of % h) * kColWarps + cw) * (kNt * 128) + lane;
        if (part_of >= h && part_of < 2 * h)
#pragma unroll
          for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[(n * 4 + i) * 32] = o[n][i];
        compute_barrier();
        if (part_of < h)
#pragma unroll
          for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] += x[(n * 4 + i) * 32];
        if (h > 1) compute_barrier();
      }
      const bool whole = (d.flags & kFull) != 0;
      float* part = partial(p, blockIdx.x, (d.flags & kSecond) ? 1 : 0);
#pragma unroll
      for (int r = 0; r < kSets; ++r) {
        const int row = row0 + r * 8;
        if (row >= hn || part_of > 0) continue;
        const float sum = s_sum[row];
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : 1.f / kPScale<T> / sum;
        if (whole) {
          T* out = static_cast<T*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + (h0 + row) * p.o.sh;
#pragma unroll
          for (int n = 0; n < kNt; ++n) {
            const int col = cw * kCols + n * 8 + col2;
            if (col < p.head_dim)
              *reinterpret_cast<uint32_t*>(out + col) =
                  Pack<T>::two(none ? 0.f : o[n][r * 2] * inv, none ? 0.f : o[n][r * 2 + 1] * inv);
          }
          if (warp == 0 && (lane & 3) == 0) {
            const float lse2 = none ? INFINITY : s_max[row] + log2f(sum);
            const int64_t at = static_cast<int64_t>(b) * p.h_q + h0 + row;
            if (p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
            if (p.lse2 != nullptr) p.lse2[at] = lse2;
          }
        } else {
#pragma unroll
          for (int n = 0; n < kNt; ++n)
            if (has_columns)
              *reinterpret_cast<float2*>(part + row * DP + cw * kCols + n * 8 + col2) =
                  make_float2(o[n][r * 2] * (1.f / kPScale<T>), o[n][r * 2 + 1] * (1.f / kPScale<T>));
          if (warp == 0 && (lane & 3) == 0) {
            part[p.part_rows * DP + row] = s_max[row];
            part[p.part_rows * DP + kMaxRows + row] = sum;
          }
        }
      }
    }
  }
}

// Joins the partials of cut segments and writes the rows of empty sequences.  A block takes
// rows_per rows of one segment, a warp a row or several that share its partials.  Where
// there are more segments than blocks of the first kernel (`blocks`), its segment is the
// one that starts in the run of such a block and is cut at its end, if there is one; else
// (by_segment) it is counted off.
//
// FAR: partials whose values are 2^+-60 apart beside their weights (V's factors).  Where a weight is
// below fp32's normal range its values may still count: they are scaled by its root twice, which w
// holds below 0 for them.
template <typename T, bool FAR>
__global__ void __launch_bounds__(kJoin) join_kernel(DecodeParams p, int blocks, int by_segment, int rows_per,
                                                     int dp) {
  __shared__ int s_sums[kJoin / 32];
  __shared__ int s_pre[kJoin];
  __shared__ float s_w[kJoin / 32][kMaxRuns];
  __shared__ float4 s_part[kJoin / 32][64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hv_n = p.h_k * p.head_tiles;
  const int per = (p.batch + kJoin - 1) / kJoin;
  const int part_m = p.part_rows * dp;
  auto len_of = [&](int b) { return clean_len(p, p.seqlens[b], false); };
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  for (int b = blockIdx.x; b < p.batch; b += gridDim.x)
    if (clean_len(p, p.seqlens[b], blocks == 0) == 0)
      for (int hv = 0; hv < hv_n; ++hv) no_keys<T>(p, b, hv);
  int total;
  s_pre[tid] = scan_tiles<kJoin>(p, false, nullptr, s_sums, per, total);
  const int line_heads = p.lines > 1 ? 1 : hv_n;
  Cut cut;
  cut.total = static_cast<long long>(total) * line_heads;
  cut.runs = static_cast<int>(min(static_cast<long long>(blocks / p.lines), cut.total));
  __syncthreads();
  const int row_blocks = (p.part_rows + rows_per - 1) / rows_per, shares = kJoin / 32 / rows_per;
  const int at = blockIdx.x / row_blocks;
  const int row = (blockIdx.x - at * row_blocks) * rows_per + warp / shares, share = warp % shares;
  bool mine = false;
  int b = 0, hv = 0, nc = 0, lead = 0, block = at;
  if (by_segment) {
    b = at / hv_n;
    hv = at - b * hv_n;
    const int t_b = tiles_of(p, len_of(b));
    if (t_b > 0) {
      int before = s_pre[b / per];
      for (int i = b / per * per; i < b; ++i) before += tiles_of(p, len_of(i));
      const int line = p.lines > 1 ? hv : 0;
      const long long s0 = static_cast<long long>(before) * line_heads +
                           static_cast<long long>(hv - line) * t_b;
      const int run = cut.run_of(s0);
      nc = cut.run_of(s0 + t_b - 1) - run + 1;
      lead = cut.start(run) == s0 ? 0 : 1;
      block = run * p.lines + line;
      mine = nc > 1;
    }
  } else {
    const int run = block / p.lines, line = block - run * p.lines;
    if (run + 1 < cut.runs) {  // a run with an end inside the line
      const long long r0 = cut.start(run), e = cut.start(run + 1);
      int before;
      b = find_sequence<kJoin>(p, s_pre, per, line_heads, e - 1, len_of, before);
      const int t_b = tiles_of(p, len_of(b));
      const long long line0 = static_cast<long long>(before) * line_heads;
      const int ch = static_cast<int>((e - 1 - line0) / t_b);
      const long long s0 = line0 + static_cast<long long>(ch) * t_b;
      hv = line + ch;
      mine = s0 >= r0 && s0 + t_b > e;  // starts here and goes on
      if (mine) {
        nc = cut.run_of(s0 + t_b - 1) - run + 1;
        lead = r0 == s0 ? 0 : 1;  // only in its first run can the segment be the second
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const bool on = row < min(kMaxRows, p.group - (hv % p.head_tiles) * kMaxRows);
  const int64_t stride = 2 * p.part_stride * p.lines;
  const float* first = partial(p, block, lead);
  const float* rest = partial(p, block, 0);
  auto part = [&](int i) { return i == 0 ? first : rest + i * stride; };
  float top = -INFINITY, sum = 0.f;
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  if (on) {
    float* w = s_w[warp];
    // rows of the first partials are on their way while the maxima are compared
    float4 x[2][kAhead];
    auto load = [&](int c, int i0) {
      const int col = row * dp + (lane + 32 * c) * 4;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k * shares < nc) x[c][k] = *reinterpret_cast<const float4*>(part(i0 + k * shares) + col);
    };
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (lane + 32 * c < dp / 4) load(c, share);
    float sums = 0.f;  // of partial `lane`
    for (int i = lane; i < nc; i += 32) {
      w[i] = part(i)[part_m + row];
      if (i == lane) sums = part(i)[part_m + kMaxRows + row];
      top = fmaxf(top, w[i]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float base = top == -INFINITY ? 0.f : top;
    for (int i = lane; i < nc; i += 32) {
      const float d = w[i] - base, f = ex2(d);
      w[i] = FAR && d < -126.f ? -ex2(0.5f * d) : f;
      sum += f * (i == lane ? sums : part(i)[part_m + kMaxRows + row]);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (lane + 32 * c < dp / 4)
        for (int i0 = share; i0 < nc; i0 += kAhead * shares) {
          if (i0 != share) load(c, i0);
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (i0 + k * shares < nc) {
              float f = w[i0 + k * shares];
              if (FAR && f < 0.f) {
                f = -f;
                x[c][k] = make_float4(x[c][k].x * f, x[c][k].y * f, x[c][k].z * f, x[c][k].w * f);
              }
              acc[c].x += f * x[c][k].x;
              acc[c].y += f * x[c][k].y;
              acc[c].z += f * x[c][k].z;
              acc[c].w += f * x[c][k].w;
            }
        }
  }
  if (shares > 1) {
    s_part[warp][lane] = acc[0];
    s_part[warp][lane + 32] = acc[1];
    __syncthreads();
    if (share == 0)
      for (int i = 1; i < shares; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float4 x = s_part[warp + i][lane + 32 * c];
          acc[c].x += x.x;
          acc[c].y += x.y;
          acc[c].z += x.z;
          acc[c].w += x.w;
        }
  }
  if (!on || share != 0) return;
  const int h = (hv / p.head_tiles) * p.group + (hv % p.head_tiles) * kMaxRows + row;
  const bool none = sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  T* out = static_cast<T*>(const_cast<void*>(p.o.ptr)) + b * p.o.sb + h * p.o.sh;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int col = (lane + 32 * c) * 4;
    if (col >= p.head_dim) continue;
    uint2 v;
    v.x = Pack<T>::two(none ? 0.f : acc[c].x * inv, none ? 0.f : acc[c].y * inv);
    v.y = Pack<T>::two(none ? 0.f : acc[c].z * inv, none ? 0.f : acc[c].w * inv);
    *reinterpret_cast<uint2*>(out + col) = v;
  }
  if (lane == 0) {
    const float lse2 = none ? INFINITY : (top == -INFINITY ? 0.f : top) + log2f(sum);
    const int64_t at = static_cast<int64_t>(b) * p.h_q + h;
    if (p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
    if (p.lse2 != nullptr) p.lse2[at] = lse2;
  }
}

// weights_out = weights_in + the group's sum of exp2(logit - LSE2).  A block takes every
// `blocks`-th kKeys keys, from the first one seen, of one (sequence, key/value head), a thread
// four of them.  (With a block for each kKeys keys of max_seqlen a loose bound cost more than
// the rest: 64 sequences of 500 keys 33 us with a bound of 512, 98 with 131072.)
constexpr int kKeys = 512;

__global__ void __launch_bounds__(kJoin) weights_kernel(DecodeParams p, int blocks) {
  const int tid = threadIdx.x;
  const int bg = blockIdx.x / blocks, b = bg / p.h_k, g = bg - b * p.h_k, h = g * p.group;
  const int n = clean_len(p, p.seqlens[b], false), first = first_key(p, n), seen = n - first;
  const int from = (blockIdx.x - bg * blocks) * kKeys;
  const int64_t at = (static_cast<int64_t>(b) * p.h_k + g) * p.w_stride, step = static_cast<int64_t>(blocks) * kKeys;
  const float* in = p.w_in + at;
  float* out = p.w_out + at;
  // keys before the window keep their weights
  if (out != in)
    for (int64_t j0 = from; j0 < first; j0 += step)
      for (int64_t j = j0 + tid; j < min(static_cast<int64_t>(first), j0 + kKeys); j += kJoin) out[j] = in[j];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float* logits = p.logits + (static_cast<int64_t>(b) * p.h_q + h) * p.logit_stride;
  const float* lse2 = p.lse2 + static_cast<int64_t>(b) * p.h_q + h;
#pragma unroll 1
  for (int64_t rel = from + tid * 4; rel < seen; rel += step) {
    float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < p.group; ++i) {
      const float l = lse2[i];
      const float4 v = *reinterpret_cast<const float4*>(logits + i * p.logit_stride + rel);
      w[0] += ex2(v.x - l);
      w[1] += ex2(v.y - l);
      w[2] += ex2(v.z - l);
      w[3] += ex2(v.w - l);
    }
    const int64_t j = first + rel;
    if (rel + 3 < seen && ((reinterpret_cast<uintptr_t>(in + j) | reinterpret_cast<uintptr_t>(out + j)) & 15) == 0) {
      float4 x = *reinterpret_cast<const float4*>(in + j);
      x.x += w[0];
      x.y += w[1];
      x.z += w[2];
      x.w += w[3];
      *reinterpret_cast<float4*>(out + j) = x;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (rel + i < seen) out[j + i] = in[j + i] + w[i];
    }
  }
}

// One block a segment, without partials.
bool takes_whole(int batch, int h_k, int group, int max_seqlen, bool weights) {
  return !weights && max_seqlen <= kWholeKeys &&
         static_cast<int64_t>(batch) * h_k * ceil_div(group, kMaxRows) <= kMaxRuns;
}

template <typename T, int DP, bool kLarge>
cudaError_t launch_main(const DecodeParams& p, int runs, cudaStream_t stream) {
  static std::atomic<unsigned long long> done{0};  // devices with the attribute set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit) || bit == 0) {
    e = cudaFuncSetAttribute(decode_kernel<T, DP, kLarge>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<DP, kLarge>::kSmem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  decode_kernel<T, DP, kLarge><<<runs, kThreads, Cfg<DP, kLarge>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t launch_main(const DecodeParams& p, int runs, cudaStream_t stream) {
  return p.group > kMaxRows / 2 ? launch_main<T, DP, true>(p, runs, stream)
                                : launch_main<T, DP, false>(p, runs, stream);
}

template <typename T>
cudaError_t launch_t(DecodeParams p, cudaStream_t stream) {
  const int dp = pad_dim(p.head_dim);
  p.chunks = p.head_dim / 8;
  int r;
  cudaError_t e = shape_decode(p, tile_log2(dp), kBlocks, &r);
  if (e != cudaSuccess) return e;
  if (r > 0) {
    if (dp == 64) e = launch_main<T, 64>(p, r, stream);
    else if (dp == 96) e = launch_main<T, 96>(p, r, stream);
    else if (dp == 128) e = launch_main<T, 128>(p, r, stream);
    else if (dp == 192) e = launch_main<T, 192>(p, r, stream);
    else e = launch_main<T, 256>(p, r, stream);
    if (e != cudaSuccess) return e;
  }
  if (p.whole) return cudaSuccess;
  e = launch_join(p, Pack<T>::kIsBf16 ? ATTN_BF16 : ATTN_FP16, r, false, stream);
  if (e != cudaSuccess || p.w_in == nullptr || p.max_seqlen == 0) return e;
  // 16 blocks fit an SM
  const int64_t bg = static_cast<int64_t>(p.batch) * p.h_k, fit = (16 * static_cast<int64_t>(num_sms()) + bg - 1) / bg;
  const int chunks = ceil_div(p.max_seqlen, kKeys), blocks = chunks < fit ? chunks : static_cast<int>(fit);
  if (bg * blocks > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchAttribute early;  // starts while the kernel before it drains, and waits for it
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(bg * blocks));
  cfg.blockDim = dim3(kJoin);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_kernel, p, blocks);
}

}  // namespace

cudaError_t shape_decode(DecodeParams& p, int tile_log2, int blocks_per_sm, int* runs_out) {
  p.head_tiles = ceil_div(p.group, kMaxRows);
  p.part_rows = p.group < kMaxRows ? p.group : kMaxRows;
  p.part_stride = static_cast<int64_t>(p.part_rows) * pad_dim(p.head_dim) + 2 * kMaxRows;
  p.tile_log2 = tile_log2;
  const int most_tiles = ceil_div(p.max_seqlen, 1 << p.tile_log2);
  if (static_cast<int64_t>(p.batch) * most_tiles > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t most = static_cast<int64_t>(p.batch) * p.h_k * p.head_tiles * most_tiles;
  int64_t runs = static_cast<int64_t>(num_sms()) * blocks_per_sm;
  if (runs > kMaxRuns) runs = kMaxRuns;
  const int64_t heads = static_cast<int64_t>(p.h_k) * p.head_tiles;
  // A line a head when that leaves at most a quarter of the blocks idle (64 heads of 64, 256
  // of 304 blocks: 338 us against 371; 32 heads of 128, 288 blocks: 310 against 329).
  p.lines = 1;
  if (heads <= runs && runs % heads * 4 <= runs) {
    p.lines = static_cast<int>(heads);
    runs -= runs % heads;
  }
  if (runs > most) runs = most;  // a multiple of the heads, too
  p.whole = takes_whole(p.batch, p.h_k, p.group, p.max_seqlen, p.w_in != nullptr) && runs > 0;
  if (p.whole) {
    runs = p.batch * heads;
    p.lines = 1;
  }
  *runs_out = static_cast<int>(runs);
  return cudaSuccess;
}

cudaError_t launch_join(const DecodeParams& p, int dtype, int runs, bool far, cudaStream_t stream) {
  cudaLaunchAttribute early;  // starts while the kernel before it drains, and waits for it
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // few segments have many partials each: then four warps share a row's
  const int64_t segments = static_cast<int64_t>(p.batch) * p.h_k * p.head_tiles;
  const int by_segment = segments <= runs;
  const int rows_per = segments * p.part_rows <= 2 * static_cast<int64_t>(runs) ? 1 : (p.part_rows > 2 ? 4 : p.part_rows);
  cfg.gridDim = dim3(static_cast<unsigned>(
      runs > 0 ? (by_segment ? segments : runs) * ceil_div(p.part_rows, rows_per) : 1));
  cfg.blockDim = dim3(kJoin);
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = runs > 0 ? 1 : 0;
  const int dp = pad_dim(p.head_dim);
  auto* kernel = dtype == ATTN_BF16 ? (far ? join_kernel<__nv_bfloat16, true> : join_kernel<__nv_bfloat16, false>)
                                    : (far ? join_kernel<__half, true> : join_kernel<__half, false>);
  return cudaLaunchKernelEx(&cfg, kernel, p, runs, by_segment, rows_per, dp);
}

DecodeWs decode_ws(int batch, int h_q, int h_k, int head_dim, int max_seqlen, bool weights) {
  DecodeWs w = {};
  if (takes_whole(batch, h_k, h_q / h_k, max_seqlen, weights)) return w;  // nothing is joined
  const size_t rows = static_cast<size_t>(batch) * h_q;
  const int group = h_q / h_k, part_rows = group < kMaxRows ? group : kMaxRows;
  w.logit_stride = round_up(max_seqlen, 1 << tile_log2(64));  // whole tiles of any width
  w.off_lse2 = 0;  // with weights only
  w.off_parts = weights ? align256(rows * 4) : 0;
  w.off_logits = w.off_parts + align256(static_cast<size_t>(kMaxRuns) * 2 *
                                        (static_cast<size_t>(part_rows) * pad_dim(head_dim) + 2 * kMaxRows) * 4);
  w.total = w.off_logits + (weights ? align256(rows * static_cast<size_t>(w.logit_stride) * 4) : 0);
  return w;
}

cudaError_t launch_decode(const DecodeParams& p, int dtype, cudaStream_t stream) {
  return dtype == ATTN_BF16 ? launch_t<__nv_bfloat16>(p, stream) : launch_t<__half>(p, stream);
}

}  // namespace attn
