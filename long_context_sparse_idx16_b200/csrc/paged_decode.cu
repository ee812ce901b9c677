// paged_decode.cu -- attention of new tokens over the pages of their sequences.
//
//   out = softmax_j(scale q . k_j) v_j  per query head, over all of a row's slots, a window with
//   sinks, or a list of pages.
//
// A row reads 2 D elements of cache per key and KV head and does 4 D G flops with them (G query
// heads per KV head, at most 16 in one pass), so HBM bounds it; the split follows from that:
//   * The keys of all problems (row, KV head, block of 8 or 16 query heads) are cut into tiles of 64
//     and numbered through, each problem counting kOverhead tiles more than it has (what starting
//     and ending it costs).  CTA c of a grid of two to four per SM takes the numbers [c T / G, (c + 1)
//     T / G), so every SM has the same work whatever the lengths are, and the host need not know
//     them.  A problem that crosses CTAs leaves partial results (running max, sum, unnormalised
//     output), at most two per CTA, which join_kernel adds up in CTA order.
//   * One warp of a CTA feeds a ring of shared-memory stages with TMA boxes of one page each (the
//     page table is looked up by the lane that issues the box), with the swizzle that ldmatrix
//     reads without bank conflicts.  Boxes without a slot to attend are not loaded.  It also sends
//     the next problem's queries ahead, so that nobody waits for a problem to begin.
//   * Four warps take 16 of the 64 keys each, with running maxima and sums of their own, so the
//     stream needs no barrier between them; their states meet when the problem (or the CTA's part
//     of it) ends.  The products run on mma.sync, keys (then dims) as the 16 rows and eight query
//     heads as the columns: S^T = K Q^T, O^T = V^T P^T, the weights transposed by movmatrix.  A
//     tcgen05 tile (64 or 128 rows) would be mostly padding, and the tensor pipe is not the bound.
//   * Scores, maxima, sums and outputs are fp32.  The weights are rounded once to 16 bits for the
//     product with the values, to the type of these (mma.sync takes both operands in one): by at most
//     half a step each, and independently, so that over many keys the output's own rounding is the
//     larger (the error against 64 bits grows by up to 11%).  Keeping more bits would take a second
//     product with the remainders.  In fp16 the weights carry a factor 2^15, so that those down to
//     2^-29 of the largest keep all their bits and sums of many small ones are not lost.
//   * e4m3 pages are read as 16-bit pairs and widened to fp16 (exactly): ldmatrix gives a lane four
//     successive dims of a key, which the query fragments match by the same permutation of the
//     contraction, and (transposed) two dims of two keys, which a byte permute splits over two
//     output rows.  Their queries are scaled per head by a power of two into fp16's range, which is
//     exact for values down to 2^-29 of the head's largest and off by 2^-40 of that below.
// Measured (one B200, 32 / 4 heads of 128; a copy reaches 6.55 TB/s): 8 x 128K fp16 keys, 2.15 GB, in
// 326 us (6.6 TB/s); 1M e4m3 keys, 1.07 GB, in 188 us (5.7 TB/s; the widening keeps the issue slots
// half busy; 178 us on the same cache again and again, where L2 holds a part); 48 sequences of 1 to 32K
// keys, 363 MB, in 69 us (5.2 TB/s, of which 10 us are starts, ends and the join); 777 keys in 9 us,
// latency.  A window of 8192 and 4 sinks of 8 x 128K keys, 134 MB, in 32 us.  Sixteen query rows to a
// tile (queries as the rows) took 254 us at 1M e4m3 keys; unweighted problems took 132 us for the 48
// sequences.
// Accumulated weights need the final sums: the scores go through the workspace in fp32 and
// weights_kernel adds exp2((s - M) - log2 L) over the query heads, beside the join.
#include <type_traits>

#include "paged.cuh"
#include "tc_umma.cuh"

namespace rtp {

namespace {

constexpr int kTile = 64;         // keys per stage
constexpr int kConsumers = 4;     // warps, 16 keys of a tile each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kInline = 256;      // entries whose tile prefix every CTA forms by itself
constexpr int kNoSlot = 0x7fff8000;  // beyond every length: a box none of whose slots is attended
constexpr int kOverhead = 2;      // tiles' worth of time that a problem costs besides its tiles: about
                                  // 1.5 us for the queries, the first look-up and the exchange of states
constexpr int kMaxPerSm = 4;
constexpr int kMaxSms = 160;      // what the workspace is sized for; a grid is at most kMaxPerSm times it

// Eight query heads need half the registers of sixteen: three CTAs per SM instead of two, with
// rings of 64 KB instead of 96 KB.  Four with rows of 64 values, whose stages are small and whose tiles
// cost more in steps than in bytes: 8 x 128K keys of 64 values 176 -> 165 us (e4m3 126 -> 114 us).
constexpr int per_sm(int octets, int D) { return octets == 1 ? (D == 64 ? 4 : 3) : 2; }
constexpr int ring_bytes(int octets, int D) { return octets == 1 ? (D == 64 ? 40 : 64) * 1024 : 96 * 1024; }

struct AttnArgs {
  DecodeArgs d;
  int octets;            // 8 * octets query heads per problem: 1 or 2
  int blocks;            // problems per KV head
  int box;               // slots per TMA box: min(page_size, 64)
  int whole;             // problems are never split (short caches)
  int n_entries, mult;   // dense: rows, Hkv * blocks; page lists: rows * Hkv, blocks
  int64_t* prefix;       // [n_entries + 1] tiles (with overhead) of the entries before, one problem each
  float2* sums;          // [rows][Hq] largest base-2 score and log2 of the sum of weights beside it, or NULL
  float* logits;         // [rows][Hq][cap] base-2 scores, or NULL
  int64_t cap;
  int4* split;           // [CTAs] problem that the CTA begins and others go on with: (row, query head,
                         // heads, last CTA), or row -1
  int2* span;            // [rows][Hkv * blocks] first and last CTA of a split problem, or -1 (with logits)
  float2* part_ml;       // [CTAs][continued, begun][16]
  float* part_o;         // [CTAs][continued, begun][16][D]
};

// What an entry (a row, or a row's KV head with a page list) attends to.
struct Entry {
  int row, seq, len, lo, sinks;  // dense: slots [0, sinks) and [lo, len)
  int t_sink, t_skip;            // tiles of the sinks; tiles left out behind them
  const int32_t* list;
  int n_list, tiles;
};

__device__ __forceinline__ Entry entry_of(const AttnArgs& a, int e) {
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  Entry n;
  n.row = d.sel ? e / kv.Hkv : e;
  const int listed = d.sel ? d.sel_count[e] : 0;  // in flight together with the length
  n.len = paged_row(kv, d.row_seq, d.row_len, n.row, &n.seq);
  n.lo = n.sinks = n.t_sink = n.t_skip = n.n_list = 0;
  n.list = nullptr;
  if (d.sel) {
    n.list = d.sel + (int64_t)e * d.sel_stride;
    n.n_list = n.len == 0 || listed < 0 ? 0 : listed > d.sel_stride ? (int)d.sel_stride : listed;
    n.tiles = (int)((((int64_t)n.n_list << kv.page_shift) + kTile - 1) / kTile);
    return n;
  }
  if (d.window && n.len > d.window) {
    n.lo = n.len - d.window;
    n.sinks = min(d.n_sink, n.lo);
    n.t_sink = (n.sinks + kTile - 1) / kTile;
    n.t_skip = max(n.lo / kTile - n.t_sink, 0);
  }
  n.tiles = (n.len + kTile - 1) / kTile - n.t_skip;
  return n;
}

// From the largest base-2 score M and the sum L of 2^(score - M + bias): the natural log-sum-exp; and M
// with log2 of the sum beside it, which a weight is formed from.  The two stay apart there: their sum
// would lose the logarithm where M is large.
__device__ __forceinline__ float lse_of(float M, float L, float bias) {
  return (L == 0.f ? -INFINITY : M + (log2f(L) - bias)) * 0.6931471805599453f;
}
__device__ __forceinline__ float2 sums_of(float M, float L, float bias) {
  return L == 0.f ? make_float2(0.f, INFINITY) : make_float2(M, log2f(L) - bias);
}

// Length of an entry's problem in the numbering: its tiles and the overhead (1 if it is not to be split).
__device__ __forceinline__ int64_t units_of(const AttnArgs& a, const Entry& n) {
  return !n.tiles ? 0 : a.whole ? 1 : n.tiles + kOverhead;
}

// x / y for x >= 0, y > 0: in 32 bits where both fit, which is nearly always and much faster.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return (int64_t)((uint32_t)x / (uint32_t)y);
  return x / y;
}

// The numbers [0, total) shared out over CTAs: the first `more` of them take one more than the others.
struct Ranges {
  int64_t total, each, more;
  int ctas;
  __device__ Ranges(int64_t total_, int grid) : total(total_), ctas((int)min((int64_t)grid, total_)) {
    each = ctas ? quotient(total, ctas) : 0;
    more = total - each * ctas;
  }
  __device__ int64_t start(int c) const { return each * c + min((int64_t)c, more); }
  __device__ int owner(int64_t t) const {
    const int64_t big = more * (each + 1);
    return (int)(t < big ? quotient(t, each + 1) : more + quotient(t - big, each));
  }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];"
      :
      : "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(mbar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t mbar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(mbar) : "memory");
}

// Layout of a stage: K then V; each as blocks of kTile rows of kRow bytes (128, or 64 where a whole
// row is 64), swizzled by TMA.
template <typename K, int D>
struct Stage {
  static constexpr int kBytes = D * (int)sizeof(K);           // bytes of a row
  static constexpr int kRow = kBytes < 128 ? kBytes : 128;    // of it per block
  static constexpr int kBlocks = kBytes / kRow;
  static constexpr int kHalf = kTile * kBytes;                // K, and V
  static constexpr int stages(int octets) {
    return ring_bytes(octets, D) / (2 * kHalf) > 8 ? 8 : ring_bytes(octets, D) / (2 * kHalf);
  }
  // byte offset of 16-byte chunk ch of row r
  static __device__ __forceinline__ uint32_t at(int r, int ch) {
    if constexpr (kRow == 128)
      return (uint32_t)((ch >> 3) * (kTile * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
    else
      return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
  }
};

// The tile prefix of all entries, by one warp.
__device__ __forceinline__ void tile_prefix(const AttnArgs& a, int64_t* out, int lane) {
  int64_t run = 0;
  for (int e0 = 0; e0 < a.n_entries; e0 += 32) {
    const int e = e0 + lane;
    const int64_t t = e < a.n_entries ? units_of(a, entry_of(a, e)) : 0;
    int64_t y = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (e < a.n_entries) out[e] = run + y - t;
    run += __shfl_sync(0xffffffffu, y, 31);
  }
  if (lane == 0) out[a.n_entries] = run;
}

// More entries than kInline: one CTA writes the prefix for everybody, kPlan entries a thread at a time.
constexpr int kPlan = 4;
__global__ void __launch_bounds__(1024) plan_kernel(const AttnArgs a) {
  __shared__ int64_t sums[33];
  after_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t run = 0;
  for (int e0 = 0; e0 < a.n_entries; e0 += 1024 * kPlan) {
    const int e = e0 + tid * kPlan;
    int64_t t[kPlan], own = 0;
#pragma unroll
    for (int u = 0; u < kPlan; ++u) t[u] = e + u < a.n_entries ? units_of(a, entry_of(a, e + u)) : 0;
#pragma unroll
    for (int u = 0; u < kPlan; ++u) own += t[u];
    int64_t y = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    if (warp == 0) {
      const int64_t w = sums[lane];
      int64_t x = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += z;
      }
      sums[lane] = x - w;
      if (lane == 31) sums[32] = x;
    }
    __syncthreads();
    int64_t at = run + sums[warp] + y - own;
#pragma unroll
    for (int u = 0; u < kPlan; ++u) {
      if (e + u < a.n_entries) a.prefix[e + u] = at;
      at += t[u];
    }
    run += sums[32];
    __syncthreads();
  }
  if (tid == 0) a.prefix[a.n_entries] = run;
}

// Part of the CTA's range inside one problem.
struct Segment {
  Entry n;
  int e, prob, first, count;  // entry, its problem, first tile of the problem, tiles (perhaps none)
  int64_t units;              // of the CTA's range
};

__device__ __forceinline__ Segment segment_at(const AttnArgs& a, const int64_t* prefix, int64_t t, int64_t t1) {
  Segment s;
  int lo = 0, hi = a.n_entries - 1;
  while (lo < hi) {  // the last entry that starts at or before t (entries without tiles are passed)
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] * a.mult <= t) lo = mid;
    else hi = mid - 1;
  }
  s.e = lo;
  s.n = entry_of(a, lo);
  const int64_t x = t - prefix[lo] * a.mult, u = units_of(a, s.n);
  s.prob = (int)quotient(x, u);
  const int64_t at = x - s.prob * u;
  s.units = min(u - at, t1 - t);
  if (a.whole) {
    s.first = 0;
    s.count = s.n.tiles;
    return s;
  }
  // the overhead comes first
  s.first = (int)max(at - kOverhead, (int64_t)0);
  s.count = (int)max(at + s.units - kOverhead - s.first, (int64_t)0);
  return s;
}

// What the consumers need of a segment.
struct Job {
  int row, len, lo, sinks;
  int g, h0, nh;      // KV head, first query head of the group, query heads
  int first, count;
  bool whole, last;   // the problem lies in this CTA alone; nothing follows
};

template <int NB, int D>
struct Shared {
  static constexpr int H = 8 * NB;       // query heads
  static constexpr int R = 32;           // dims of the output exchanged at a time
  static constexpr int kQRow = 2 * D + 16;  // bytes: rows shifted by 16 bytes, ldmatrix without conflicts
  uint8_t q[H][kQRow];
  float x[kConsumers][H][R + 4];
  float m[kConsumers][H], l[kConsumers][H];
  unsigned long long full[8], empty[8], job_full, job_empty, meet;
  int base[8][4];                        // first slot of each box of a stage
  int stop;                              // a wait gave up
  int verdict;                           // of the consumers, on the job that begins
  Job job;
  int64_t prefix[kInline + 1];
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename QT, typename K, int D, int NB>
__global__ void __launch_bounds__(kThreads, per_sm(NB, D)) attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap km,
                                                                    const __grid_constant__ CUtensorMap vm) {
  using S = Stage<K, D>;
  using Sh = Shared<NB, D>;
  constexpr bool k8 = sizeof(K) == 1;
  using MT = std::conditional_t<k8, __half, K>;  // operands of the products
  constexpr float kBias = std::is_same_v<MT, __half> ? 15.f : 0.f;
  constexpr int ST = S::stages(NB);
  constexpr int KS = D / 16;  // contraction steps of the scores; row tiles of the output
  extern __shared__ __align__(1024) uint8_t smem[];
  Sh& sh = *reinterpret_cast<Sh*>(smem + ST * 2 * S::kHalf);
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = smem_u32(smem);
  const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty);
  const uint32_t job_full = smem_u32(&sh.job_full), job_empty = smem_u32(&sh.job_empty), meet = smem_u32(&sh.meet);
  volatile int* stop = &sh.stop;
  const bool inl = a.n_entries <= kInline;
  if (tid == 32 * kConsumers) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&km) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&vm) : "memory");
    for (int i = 0; i < ST; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, kConsumers);
    }
    mbar_init(job_full, 1);
    mbar_init(job_empty, kConsumers);
    mbar_init(meet, kConsumers);
    fence_mbar_init();
    sh.stop = sh.verdict = 0;
  }
  after_wait();
  if (warp == 0 && inl) tile_prefix(a, sh.prefix, lane);
  __syncthreads();
  const int64_t* prefix = inl ? sh.prefix : a.prefix;
  const Ranges ranges(prefix[a.n_entries] * a.mult, gridDim.x);
  if (tid == 32 * kConsumers) a.split[blockIdx.x] = make_int4(-1, 0, 0, 0);  // the thread that may overwrite it
  // entries without a tile: zeros
  for (int e = blockIdx.x; e < a.n_entries; e += gridDim.x) {
    const int r = d.sel ? e / kv.Hkv : e;
    if (tid == 0 && paged_row_bad(kv, d.row_seq, d.row_len, r)) paged_err(kv, RTP_PAGED_ERANGE);
    if (prefix[e + 1] != prefix[e]) continue;
    const int h = d.sel ? e % kv.Hkv * d.group : 0, nh = d.sel ? d.group : d.Hq;
    uint16_t* out = (uint16_t*)d.out + r * d.out_stride + (int64_t)h * D;
    for (int x = tid; x < nh * D / 8; x += kThreads) ((uint4*)out)[x] = make_uint4(0u, 0u, 0u, 0u);
    for (int x = tid; x < nh; x += kThreads) {
      if (d.lse) d.lse[(int64_t)r * d.Hq + h + x] = -INFINITY;
      if (a.sums) a.sums[(int64_t)r * d.Hq + h + x] = make_float2(0.f, INFINITY);
    }
  }
  if ((int)blockIdx.x >= ranges.ctas) return;
  const int64_t t0 = ranges.start(blockIdx.x), t1 = ranges.start(blockIdx.x + 1);

  if (warp == kConsumers) {
    // ---- producer: lane (half, block, box) issues one TMA box of a tile
    const int boxes = kTile / a.box;
    const int bi = lane % boxes, blk = (lane / boxes) % S::kBlocks, is_v = lane / (boxes * S::kBlocks);
    const bool mine = is_v < 2;
    const CUtensorMap* map = is_v ? &vm : &km;
    const uint32_t dst0 = ring + is_v * S::kHalf + blk * (kTile * 128) + bi * a.box * S::kRow;
    const int sub_shift = kv.page_size > kTile ? 1 : 0;  // boxes per page: 1 or 2
    bool dead = false;
    int st = 0;
    uint32_t phase = 0, jphase = 0;
    for (int64_t t = t0; t < t1 && !dead;) {
      const Segment s = segment_at(a, prefix, t, t1);
      t += s.units;
      if (s.count == 0 && t < t1) continue;
      const int g = d.sel ? s.e % kv.Hkv : s.prob / a.blocks;
      const int h0 = (d.sel ? s.prob : s.prob % a.blocks) * Sh::H;
      const int nh = min(Sh::H, d.group - h0);
      dead = !mbar_wait(job_empty, jphase ^ 1u) || *stop;
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      if (lane == 0) {
        Job& j = sh.job;
        j.row = s.n.row;
        j.len = s.n.len;
        j.lo = s.n.lo;
        j.sinks = s.n.sinks;
        j.g = g;
        j.h0 = h0;
        j.nh = nh;
        j.first = s.first;
        j.count = s.count;
        j.whole = s.count == s.n.tiles;
        j.last = t >= t1;
        mbar_expect_tx(job_full, s.count ? nh * 2 * D : 0);
      }
      __syncwarp();
      if (lane < nh && s.count)
        bulk_load(smem_u32(sh.q[lane]),
                  (const uint16_t*)d.q + s.n.row * d.q_stride + (int64_t)(g * d.group + h0 + lane) * D, 2 * D, job_full);
      if (lane == 0 && s.count && s.first == 0) {  // a problem begins here
        int c1 = -1;
        if (s.count < s.n.tiles) {
          c1 = ranges.owner(t + (s.n.tiles - s.count) - 1);  // the CTA with its last tile
          a.split[blockIdx.x] = make_int4(s.n.row, g * d.group + h0, nh, c1);
        }
        if (a.logits) a.span[(int64_t)s.n.row * a.mult + s.prob] = make_int2(c1 < 0 ? -1 : (int)blockIdx.x, c1);
      }
      jphase ^= 1u;
      // One tile ahead in the page table, two in the list: the look-ups' latency passes while the
      // ring is full.
      const int end = s.first + s.count;
      const auto listed = [&](int i) -> int {  // the list's entry for this lane's box of tile i
        const int64_t li = ((int64_t)i * boxes + bi) >> sub_shift;
        return mine && i < end && li < s.n.n_list ? s.n.list[li] : -1;
      };
      const auto slot_of = [&](int i, int p) -> int {  // the box's first slot
        if (!mine || i >= end) return kNoSlot;
        int base;
        if (d.sel) {
          if (p < 0 || p >= kv.max_pages) return kNoSlot;
          base = (p << kv.page_shift) + (((i * boxes + bi) & sub_shift) ? a.box : 0);
        } else {
          base = (i < s.n.t_sink ? i : i + s.n.t_skip) * kTile + bi * a.box;
        }
        return base >= s.n.len || (base + a.box <= s.n.lo && base >= s.n.sinks) ? kNoSlot : base;
      };
      const auto page_of = [&](int base) -> int {
        return base == kNoSlot ? 0 : kv.table[(int64_t)s.n.seq * kv.table_stride + (base >> kv.page_shift)];
      };
      int next_base = slot_of(s.first, d.sel ? listed(s.first) : 0);
      int next_page = page_of(next_base);
      int next_list = d.sel ? listed(s.first + 1) : 0;
      for (int i = s.first; i < end; ++i) {
        int base = next_base;
        const int page = next_page;
        next_base = slot_of(i + 1, next_list);
        next_page = page_of(next_base);
        if (d.sel) next_list = listed(i + 2);
        if (base != kNoSlot && (uint32_t)page >= (uint64_t)kv.n_pages) {
          paged_err(kv, RTP_PAGED_ERANGE);
          base = kNoSlot;
        }
        const bool load = base != kNoSlot;
        dead = !mbar_wait(empty + 8 * st, phase ^ 1u) || *stop;
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        const int n_load = __popc(__ballot_sync(0xffffffffu, load));
        if (lane < boxes) sh.base[st][lane] = base;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(full + 8 * st, (uint32_t)(n_load * a.box * S::kRow));
        __syncwarp();
        if (load)
          tma_load_4d(dst0 + st * 2 * S::kHalf, map, blk * (128 / (int)sizeof(K)), base & (kv.page_size - 1), g, page,
                      full + 8 * st);
        if (++st == ST) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    if (dead) {  // the consumers may have left: wait (to a limit) for the copies still in flight
      if (lane == 0) paged_err(kv, RTP_PAGED_ETIMEOUT);
      *stop = 1;
      if (lane < ST) mbar_wait(full + 8 * lane, lane < st ? phase : phase ^ 1u);
      if (lane == ST) mbar_wait(job_full, jphase ^ 1u);
    }
    return;
  }

  // ---- consumers
  const int r0 = warp * 16, row = lane >> 2, c2 = (lane & 3) * 2;
  // A warp that gives up a wait sets `stop` and goes on without computing.  When a job begins the four
  // warps meet (with a bounded wait) and the first to come out says whether all go on or all leave.
  // Inside a job they all take the same steps, so that the barriers there cannot be left waiting.
  bool dead = false;
  const auto give_up = [&]() {
    dead = true;
    *stop = 1;
    if (lane == 0) paged_err(kv, RTP_PAGED_ETIMEOUT);
  };
  const auto consumers_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); };
  int st = 0;
  uint32_t phase = 0, jphase = 0, mphase = 0;
  int verdict = 0;  // 2 per job, odd: leave
  for (bool last = false; !last;) {
    if (!mbar_wait(job_full, jphase)) give_up();
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    if (!mbar_wait(meet, mphase)) give_up();
    mphase ^= 1u;
    int said = 0;
    if (lane == 0) {
      const int say = verdict + 2 + (dead || *stop ? 1 : 0);
      said = atomicCAS(&sh.verdict, verdict, say);
      if (said == verdict) said = say;
    }
    verdict = __shfl_sync(0xffffffffu, said, 0);
    if (verdict & 1) return;
    jphase ^= 1u;
    const Job j = sh.job;
    last = j.last;
    if (j.count == 0) return;  // only ever the last
    // query fragments (B operands): columns are heads; for e4m3 the contraction slots of a step are
    // permuted as ldmatrix delivers the keys' bytes
    uint32_t q[NB][KS][2];
    float scale[NB][2];  // of this lane's score columns, heads c2 and c2 + 1 of each octet
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if constexpr (!k8) {
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2)
          ldsm_x4(smem_u32(sh.q[n * 8 + (lane & 7)]) + (ks * 2 + (lane >> 3)) * 16, q[n][ks][0], q[n][ks][1],
                  q[n][ks + 1][0], q[n][ks + 1][1]);
        scale[n][0] = scale[n][1] = d.scale_log2;
      } else {
        // head `row` of the octet: dims 16 ks + 2 c2 ... + 3; scaled by a power of two so that the
        // largest lies in [2^14, 2^15)
        const uint8_t* qp = sh.q[n * 8 + row];
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 u = *(const uint2*)(qp + (ks * 16 + 2 * c2) * 2);
          const QT* h = reinterpret_cast<const QT*>(&u);
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(to_f32(h[e])));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (int)(__float_as_uint(top) >> 23);  // biased exponent
        // 2^(14 - e) and its inverse, both normal numbers: 2^126 at most, which brings bf16's least values
        // (2^-133) to 2^-7; 1 for infinities
        const bool odd = ex > 254;
        const float up = odd ? 1.f : __uint_as_float((uint32_t)min(254 + 14 - ex, 253) << 23);
        const float down = odd ? 1.f : __uint_as_float((uint32_t)max(ex - 14, 1) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 u = *(const uint2*)(qp + (ks * 16 + 2 * c2) * 2);
          const QT* h = reinterpret_cast<const QT*>(&u);
          q[n][ks][0] = pack2<__half>(to_f32(h[0]) * up, to_f32(h[1]) * up);
          q[n][ks][1] = pack2<__half>(to_f32(h[2]) * up, to_f32(h[3]) * up);
        }
        // lane 4 h holds head h's factor; the score columns are heads c2 and c2 + 1
        scale[n][0] = d.scale_log2 * __shfl_sync(0xffffffffu, down, c2 * 4);
        scale[n][1] = d.scale_log2 * __shfl_sync(0xffffffffu, down, c2 * 4 + 4);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(job_empty);
    float m[NB][2], l[NB][2];
    float o[NB][KS][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) o[n][k][0] = o[n][k][1] = o[n][k][2] = o[n][k][3] = 0.f;
    }
    float* logit = nullptr;
    if (a.logits) logit = a.logits + ((int64_t)j.row * d.Hq + j.g * d.group + j.h0) * a.cap;

    for (int i = 0; i < j.count; ++i) {
      if (!dead && !mbar_wait(full + 8 * st, phase)) give_up();
      const int base = sh.base[st][r0 / a.box] + (r0 & (a.box - 1));
      if (!dead && base < j.len && (base + 16 > j.lo || base < j.sinks)) {
        const uint32_t kb = ring + st * 2 * S::kHalf, vb = kb + S::kHalf;
        float z[NB][4] = {};
        if constexpr (!k8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t f[4];
            ldsm_x4(kb + S::at(r0 + (lane & 15), 2 * ks + (lane >> 4)), f[0], f[1], f[2], f[3]);
#pragma unroll
            for (int n = 0; n < NB; ++n) mma<MT>(z[n], f, q[n][ks][0], q[n][ks][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            uint32_t b[4];
            ldsm_x4(kb + S::at(r0 + (lane & 15), ks + (lane >> 4)), b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t f[4] = {widen2<MT>(b[2 * u]), widen2<MT>(b[2 * u + 1]), widen2<MT>(b[2 * u] >> 16),
                                     widen2<MT>(b[2 * u + 1] >> 16)};
#pragma unroll
              for (int n = 0; n < NB; ++n) mma<MT>(z[n], f, q[n][ks + u][0], q[n][ks + u][1]);
            }
          }
        }
        // z: keys base + row (first two) and base + row + 8, heads c2 and c2 + 1
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[n][e] *= scale[n][e & 1];
        const bool part = base + 15 >= j.len || !(base >= j.lo || base + 15 < j.sinks);
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // of the values of slots base + c2 + {0, 1, 8, 9}
        bool ok0 = true, ok1 = true;                        // of this lane's two keys
        if (part) {
          const auto ok = [&](int x) { return x < j.len && (x >= j.lo || x < j.sinks); };
          ok0 = ok(base + row);
          ok1 = ok(base + row + 8);
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            if (!ok0) z[n][0] = z[n][1] = -INFINITY;
            if (!ok1) z[n][2] = z[n][3] = -INFINITY;
          }
          keep0 = (ok(base + c2) ? 0xffffu : 0u) | (ok(base + c2 + 1) ? 0xffff0000u : 0u);
          keep1 = (ok(base + c2 + 8) ? 0xffffu : 0u) | (ok(base + c2 + 9) ? 0xffff0000u : 0u);
        }
        if (logit) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = n * 8 + c2 + (e & 1);
              if (h < j.nh && (e < 2 ? ok0 : ok1)) logit[h * a.cap + base + row + (e >> 1) * 8] = z[n][e];
            }
        }
        float mx[NB][2];
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float x = fmaxf(z[n][u], z[n][2 + u]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            mx[n][u] = fmaxf(m[n][u], x);
            grew |= mx[n][u] > m[n][u];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            float f[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              f[u] = mx[n][u] == m[n][u] ? 1.f : fast_exp2(m[n][u] - mx[n][u]);
              m[n][u] = mx[n][u];
              l[n][u] *= f[u];
            }
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][k][e] *= f[e & 1];
          }
        }
        // Weights as the B operand: keys (contraction) by heads.  The difference to the maximum comes
        // first: it is 0 for the largest score, whatever its size, so no weight passes 2^kBias and the sums
        // carry exactly this factor.  (m - kBias would be rounded from 2^24 on, up to a weight of 2^16.)
        uint32_t p[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = fast_exp2((z[n][e] - (m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1])) + kBias);
          l[n][0] += w[0] + w[2];
          l[n][1] += w[1] + w[3];
          p[n][0] = movmatrix(pack2<MT>(w[0], w[1]));
          p[n][1] = movmatrix(pack2<MT>(w[2], w[3]));
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          // 16 dims by 16 keys of V^T
          uint32_t f[4];
          if constexpr (!k8) {
            ldsm_x4_t(vb + S::at(r0 + (lane >> 4) * 8 + (lane & 7), 2 * k + ((lane >> 3) & 1)), f[0], f[1], f[2], f[3]);
            if (part) {  // what lies in slots left out may be infinite or NaN
              f[0] &= keep0;
              f[1] &= keep0;
              f[2] &= keep1;
              f[3] &= keep1;
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) mma<MT>(o[n][k], f, p[n][0], p[n][1]);
          } else if ((k & 1) == 0) {
            uint32_t b[4];
            ldsm_x4_t(vb + S::at(r0 + (lane & 15), k + (lane >> 4)), b[0], b[1], b[2], b[3]);
            if (part) {
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t x = __byte_perm(b[2 * u], 0, 0x3120), y = __byte_perm(b[2 * u + 1], 0, 0x3120);
              const uint32_t f8[4] = {widen2<MT>(x), widen2<MT>(x >> 16), widen2<MT>(y), widen2<MT>(y >> 16)};
#pragma unroll
              for (int n = 0; n < NB; ++n) mma<MT>(o[n][k + u], f8, p[n][0], p[n][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
      if (++st == ST) {
        st = 0;
        phase ^= 1u;
      }
    }

    // ---- the four warps' states joined; the whole result, or a partial one
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x = l[n][u];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (row == 0) {
          sh.m[warp][n * 8 + c2 + u] = m[n][u];
          sh.l[warp][n * 8 + c2 + u] = x;
        }
      }
    consumers_sync();
    constexpr int R = Sh::R;
    const int oh = tid / (R / 4), od = (tid % (R / 4)) * 4;  // this thread's head and dims in the exchange
    float f[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, sh.m[w][n * 8 + c2 + u]);
        f[n][u] = fast_exp2(m[n][u] - (M == -INFINITY ? 0.f : M));
      }
    float M = -INFINITY, L = 0.f;
    if (oh < Sh::H) {
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, sh.m[w][oh]);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) L += sh.l[w][oh] * fast_exp2(sh.m[w][oh] - (M == -INFINITY ? 0.f : M));
    }
    const int64_t pslot = 2 * (int64_t)blockIdx.x + (j.first > 0 ? 0 : 1);
#pragma unroll
    for (int rd = 0; rd < D / R; ++rd) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int k = 0; k < R / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sh.x[warp][n * 8 + c2 + (e & 1)][k * 16 + (k8 ? 2 * row + (e >> 1) : row + (e >> 1) * 8)] =
                o[n][rd * (R / 16) + k][e] * f[n][e & 1];
      consumers_sync();
      if (oh < j.nh) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
          const float4 y = *(const float4*)&sh.x[w][oh][od];
          x.x += y.x;
          x.y += y.y;
          x.z += y.z;
          x.w += y.w;
        }
        if (j.whole) {
          const float inv = kv.v_scale / L;
          uint2 r;
          r.x = pack2<QT>(x.x * inv, x.y * inv);
          r.y = pack2<QT>(x.z * inv, x.w * inv);
          if (L == 0.f) r = make_uint2(0u, 0u);
          *(uint2*)((uint16_t*)d.out + j.row * d.out_stride + (int64_t)(j.g * d.group + j.h0 + oh) * D + rd * R + od) = r;
        } else {
          *(float4*)(a.part_o + (pslot * 16 + oh) * D + rd * R + od) = x;
        }
      }
      consumers_sync();
    }
    if (od == 0 && oh < j.nh) {
      if (j.whole) {
        const int64_t at = (int64_t)j.row * d.Hq + j.g * d.group + j.h0 + oh;
        if (d.lse) d.lse[at] = lse_of(M, L, kBias);
        if (a.sums) a.sums[at] = sums_of(M, L, kBias);
      } else {
        a.part_ml[pslot * 16 + oh] = make_float2(M, L);
      }
    }
  }
}

// One CTA per (CTA of attn_kernel, query head of a problem): the partial results of the problem that
// the CTA begins and others go on with, in CTA order.
constexpr int kJoinWarps = 8;

template <typename QT, int D>
__device__ void join_part(const AttnArgs& a, float bias, int c0, int hrow) {
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ float weight[kMaxPerSm * kMaxSms];
  __shared__ float red[2][kJoinWarps];
  __shared__ float so[kJoinWarps][D];
  const int4 s = a.split[c0];
  if (s.x < 0 || hrow >= s.z) return;
  const int r = s.x, h = s.y + hrow, n = s.w - c0 + 1;
  uint16_t* out = (uint16_t*)d.out + r * d.out_stride + (int64_t)h * D;
  const int64_t at = (int64_t)r * d.Hq + h;
  const auto part = [&](int i) { return (2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0)) * 16 + hrow; };
  // the first parts' outputs, in flight while their weights are formed: a warp takes every
  // kJoinWarps-th part
  constexpr int V = D / 32, kAhead = 4;
  const auto load = [&](int i, float* y) {
    const float* p = a.part_o + part(i) * D + lane * V;
    if constexpr (V == 4) *(float4*)y = *(const float4*)p;
    else *(float2*)y = *(const float2*)p;
  };
  float first[kAhead][V];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (warp + u * kJoinWarps < n) load(warp + u * kJoinWarps, first[u]);
  // the parts' weights exp2(m - M), their sum of sums
  float m = -INFINITY;
  for (int i = tid; i < n; i += kJoinWarps * 32) {
    const float y = a.part_ml[part(i)].x;
    weight[i] = y;
    m = fmaxf(m, y);
  }
  m = warp_max(m);
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  float M = red[0][0];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, red[0][w]);
  const float base = M == -INFINITY ? 0.f : M;
  float l = 0.f;
  for (int i = tid; i < n; i += kJoinWarps * 32) {
    const float f = exp2f(weight[i] - base);
    l += a.part_ml[part(i)].y * f;
    weight[i] = f;
  }
  l = warp_sum(l);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  float L = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) L += red[1][w];
  float o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = 0.f;
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int i = warp + u * kJoinWarps;
    if (i < n) {
      const float f = weight[i];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = fmaf(first[u][v], f, o[v]);
    }
  }
#pragma unroll 4
  for (int i = warp + kAhead * kJoinWarps; i < n; i += kJoinWarps) {
    float y[V];
    load(i, y);
    const float f = weight[i];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = fmaf(y[v], f, o[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) so[warp][lane * V + v] = o[v];
  __syncthreads();
  if (tid < D / 2) {
    const int x = 2 * tid;
    float y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      y0 += so[w][x];
      y1 += so[w][x + 1];
    }
    const float inv = kv.v_scale / L;
    *(uint32_t*)(out + x) = L == 0.f ? 0u : pack2<QT>(y0 * inv, y1 * inv);
  }
  if (tid == 0 && d.lse) d.lse[at] = lse_of(M, L, bias);
}

// scores[row][g][j] += sum over g's heads of exp2((logit - M) - log2 L), for the slots attended.  M and
// log2 L of a split problem are joined here again, a warp per head.
__device__ void add_weights(const AttnArgs& a, float bias, int chunk, int chunks) {
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  const int g = blockIdx.y, r = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float2 sums[64];
  const Entry n = entry_of(a, r);
  const int slots = n.sinks + n.len - n.lo;
  if (chunk * (kJoinWarps * 32) >= slots) return;
  const int heads = 8 * a.octets;
  for (int u = warp; u < d.group; u += kJoinWarps) {
    const int2 c = a.span[(int64_t)r * a.mult + g * a.blocks + u / heads];
    float2 y;
    if (c.x < 0) {
      y = a.sums[(int64_t)r * d.Hq + g * d.group + u];
    } else {
      float m = -INFINITY, l = 0.f;
      for (int i = c.x + lane; i <= c.y; i += 32) {
        const float2 p = a.part_ml[(2 * (int64_t)i + (i == c.x ? 1 : 0)) * 16 + u % heads];
        const float mn = fmaxf(m, p.x), base = mn == -INFINITY ? 0.f : mn;
        l = l * exp2f(m - base) + p.y * exp2f(p.x - base);
        m = mn;
      }
      const float M = warp_max(m);
      const float L = warp_sum(l * exp2f(m - (M == -INFINITY ? 0.f : M)));
      y = sums_of(M, L, bias);
    }
    if (lane == 0) sums[u] = y;
  }
  __syncthreads();
  const float* lg = a.logits + ((int64_t)r * d.Hq + g * d.group) * a.cap;
  float* sc = d.scores + ((int64_t)r * kv.Hkv + g) * d.scores_stride;
  for (int i = chunk * (kJoinWarps * 32) + threadIdx.x; i < slots; i += chunks * (kJoinWarps * 32)) {
    const int j = i < n.sinks ? i : n.lo + i - n.sinks;
    if (paged_page(kv, n.seq, j >> kv.page_shift) < 0) continue;
    float w = 0.f;
#pragma unroll 8
    for (int u = 0; u < d.group; ++u) w += fast_exp2((lg[u * a.cap + j] - sums[u].x) - sums[u].y);
    sc[j] += w;
  }
}

// The join, and with accumulated weights also these: both need only what attn_kernel left.
template <typename QT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttnArgs a, float bias, int heads) {
  after_wait();
  join_part<QT, D>(a, bias, blockIdx.x / heads, blockIdx.x % heads);
}
template <typename QT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) weights_kernel(const AttnArgs a, float bias, int heads, int joins,
                                                                  int chunks) {
  after_wait();
  if ((int)blockIdx.x < chunks) return add_weights(a, bias, blockIdx.x, chunks);
  const int64_t i = ((int64_t)(blockIdx.x - chunks) * gridDim.z + blockIdx.z) * gridDim.y + blockIdx.y;
  if (i < joins) join_part<QT, D>(a, bias, (int)i / heads, (int)i % heads);
}

// ---- host

int device_sms() {
  static std::atomic<int> known[64];
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return sms;
  if (const int k = known[dev & 63].load()) return k;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  known[dev & 63].store(sms);
  return sms;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t prefix, split, span, sums, ml, o, logits, total;
};
Layout layout_of(const rtp_paged_kv* kv, int n_rows, int n_q_heads, bool scores) {
  Layout l;
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t x = at;
    at += align256(n);
    return x;
  };
  const size_t parts = (size_t)2 * kMaxPerSm * kMaxSms * 16;
  l.prefix = take(((size_t)n_rows * kv->n_kv_heads + 1) * sizeof(int64_t));
  l.split = take((size_t)kMaxPerSm * kMaxSms * sizeof(int4));
  l.ml = take(parts * sizeof(float2));
  l.o = take(parts * kv->head_dim * sizeof(float));
  const int group = n_q_heads / kv->n_kv_heads, blocks = group <= 8 ? 1 : (group + 15) / 16;
  l.span = take(scores ? (size_t)n_rows * kv->n_kv_heads * blocks * sizeof(int2) : 0);
  l.sums = take(scores ? (size_t)n_rows * n_q_heads * sizeof(float2) : 0);
  l.logits = take(scores ? (size_t)n_rows * n_q_heads * kv->max_pages * kv->page_size * sizeof(float) : 0);
  l.total = at;
  return l;
}

bool map_pages(CUtensorMap* m, void* base, const int64_t* stride, const rtp_paged_kv* kv, int box) {
  const int es = kv->dtype == RTP_E4M3 ? 1 : 2, bytes = kv->head_dim * es;
  const uint64_t dims[4] = {(uint64_t)kv->head_dim, (uint64_t)kv->page_size, (uint64_t)kv->n_kv_heads,
                            (uint64_t)kv->n_pages};
  const uint64_t strides[3] = {(uint64_t)stride[2] * es, (uint64_t)stride[1] * es, (uint64_t)stride[0] * es};
  const uint32_t bx[4] = {(uint32_t)((bytes < 128 ? bytes : 128) / es), (uint32_t)box, 1, 1};
  return tma_encode(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, base, dims, strides,
                    bx, bytes < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Slots that a problem can have.
int64_t slots_of(const AttnArgs& a) { return a.d.sel ? a.d.sel_stride * a.d.kv.page_size : a.cap; }

template <typename QT, typename K, int D, int NB>
cudaError_t run(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  using S = Stage<K, D>;
  constexpr size_t smem = (size_t)S::stages(NB) * 2 * S::kHalf + sizeof(Shared<NB, D>);
  static_assert((smem + 1024) * per_sm(NB, D) <= 228 * 1024, "the CTAs of an SM share 228 KB");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(attn_kernel<QT, K, D, NB>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)a.n_entries * a.mult * (a.whole ? 1 : slots_of(a) / kTile + 1 + kOverhead);
  const int sms = device_sms();
  int64_t grid = (int64_t)per_sm(NB, D) * (sms < kMaxSms ? sms : kMaxSms);
  if (grid > most) grid = most;
  if (a.n_entries > kInline && (e = launch_after(plan_kernel, dim3(1), 1024, 0, st, a)) != cudaSuccess) return e;
  e = launch_after(attn_kernel<QT, K, D, NB>, dim3((unsigned)grid), kThreads, smem, st, a, km, vm);
  if (e != cudaSuccess) return e;
  const float bias = std::is_same_v<K, __nv_bfloat16> ? 0.f : 15.f;
  const int joins = a.whole ? 0 : (int)grid * 8 * NB;
  if (!a.logits)
    return joins ? launch_after(join_kernel<QT, D>, dim3(joins), kJoinWarps * 32, 0, st, a, bias, 8 * NB) : cudaSuccess;
  const int64_t chunks = (a.cap + 1023) / 1024, lists = (int64_t)a.d.kv.Hkv * a.d.n_rows;
  const int blocks = (int)(chunks < 1024 ? chunks : 1024);
  return launch_after(weights_kernel<QT, D>, dim3((unsigned)(blocks + (joins + lists - 1) / lists), a.d.kv.Hkv, a.d.n_rows),
                      kJoinWarps * 32, 0, st, a, bias, 8 * NB, joins, blocks);
}

template <typename QT, typename K>
cudaError_t run_d(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  if (a.octets == 1)
    return a.d.kv.D == 64 ? run<QT, K, 64, 1>(a, km, vm, st) : run<QT, K, 128, 1>(a, km, vm, st);
  return a.d.kv.D == 64 ? run<QT, K, 64, 2>(a, km, vm, st) : run<QT, K, 128, 2>(a, km, vm, st);
}

}  // namespace

size_t paged_decode_workspace(const rtp_paged_kv* kv, int n_rows, int n_q_heads, bool scores) {
  return layout_of(kv, n_rows, n_q_heads, scores).total;
}

cudaError_t launch_paged_decode(const DecodeArgs& d, const rtp_paged_kv* kv, int qt, cudaStream_t st) {
  AttnArgs a{};
  a.d = d;
  a.octets = d.group <= 8 ? 1 : 2;
  a.blocks = (d.group + 8 * a.octets - 1) / (8 * a.octets);
  a.box = kv->page_size < kTile ? kv->page_size : kTile;
  a.n_entries = d.sel ? d.n_rows * kv->n_kv_heads : d.n_rows;
  a.mult = d.sel ? a.blocks : kv->n_kv_heads * a.blocks;
  a.cap = (int64_t)kv->max_pages * kv->page_size;
  // Four tiles take less time in one CTA than a second launch to join them does.
  a.whole = slots_of(a) <= 4 * kTile;
  const Layout l = layout_of(kv, d.n_rows, d.Hq, d.scores != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(d.workspace);
  a.prefix = reinterpret_cast<int64_t*>(ws + l.prefix);
  a.split = reinterpret_cast<int4*>(ws + l.split);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  if (d.scores) {
    a.span = reinterpret_cast<int2*>(ws + l.span);
    a.sums = reinterpret_cast<float2*>(ws + l.sums);
    a.logits = reinterpret_cast<float*>(ws + l.logits);
  }
  CUtensorMap km, vm;
  if (!map_pages(&km, kv->k, kv->k_stride, kv, a.box) || !map_pages(&vm, kv->v, kv->v_stride, kv, a.box))
    return cudaErrorInvalidValue;
  const int kt = kv->dtype;
  if (qt == RTP_FP16 && kt == RTP_FP16) return run_d<__half, __half>(a, km, vm, st);
  if (qt == RTP_BF16 && kt == RTP_BF16) return run_d<__nv_bfloat16, __nv_bfloat16>(a, km, vm, st);
  if (qt == RTP_FP16) return run_d<__half, __nv_fp8_e4m3>(a, km, vm, st);
  return run_d<__nv_bfloat16, __nv_fp8_e4m3>(a, km, vm, st);
}

}  // namespace rtp
