// paged_decode.cu -- attention of new tokens over the pages of their sequences.
//
//   out = softmax_j(scale q . k_j) v_j  per query head, over all of a row's slots, a window with
//   sinks, or a list of pages.
//
// A row reads 2 D elements of cache per key and KV head and does 4 D G flops with them (G query
// heads per KV head, at most 16 in one pass), so HBM bounds it; the split follows from that:
//   * The keys of all problems (row, KV head, block of 16 query heads) are cut into tiles of 64
//     and numbered through.  CTA c of a grid of two per SM takes tiles [c T / G, (c + 1) T / G), so
//     every SM streams the same bytes whatever the lengths are, and the host need not know them.
//     A problem that crosses CTAs leaves partial results (running max, sum, unnormalised output),
//     at most two per CTA, which join_kernel adds up in CTA order.
//   * One warp of a CTA feeds a ring of shared-memory stages with TMA boxes of one page each (the
//     page table is looked up by the lane that issues the box), with the swizzle that ldmatrix
//     reads without bank conflicts.  Boxes without a slot to attend are not loaded.
//   * Four warps take 16 of the 64 keys each, with running maxima and sums of their own, so the
//     stream needs no barrier between them; their states meet when the problem (or the CTA's part
//     of it) ends.  The products run on mma.sync: with at most 16 rows a tcgen05 tile (64 or 128
//     rows) would be mostly padding, and the tensor pipe is not the bound.
//   * Scores, maxima, sums and outputs are fp32.  The weights are rounded once to 16 bits for the
//     product with the values; in fp16 they carry a factor 2^15, so that weights down to 2^-29 of
//     the largest keep all their bits and sums of many small ones are not lost.
//   * e4m3 pages are read as 16-bit pairs: ldmatrix gives a lane four successive dims of a key,
//     which the query fragments match by the same permutation of the contraction, and (transposed)
//     two dims of two keys, which a byte permute splits over two output tiles.
// Accumulated weights need the final log-sum-exp: the scores go through the workspace in fp32 and
// weights_kernel adds exp(s - lse) over the query heads.
#include <type_traits>

#include "paged.cuh"
#include "tc_umma.cuh"

namespace rtp {

namespace {

constexpr int kTile = 64;         // keys per stage
constexpr int kConsumers = 4;     // warps, 16 keys of a tile each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kHeads = 16;        // query heads of a problem
constexpr int kPerSm = 2;         // CTAs per SM
constexpr int kRingBytes = 96 * 1024;
constexpr int kInline = 256;      // entries whose tile prefix every CTA forms by itself
constexpr int kPad = 36;          // floats per row of the exchange buffer (32 used)
constexpr int kNoSlot = 0x7fff8000;  // beyond every length: a box none of whose slots is attended

constexpr int stages_of(int stage_bytes) { return kRingBytes / stage_bytes > 8 ? 8 : kRingBytes / stage_bytes; }

struct Shared {
  unsigned long long full[8], empty[8];
  int base[8][4];                      // first slot of each box of a stage
  float m[kConsumers][kHeads], l[kConsumers][kHeads];
  int stop;                            // a wait gave up: no more copies
  int64_t prefix[kInline + 1];
  float x[kConsumers][kHeads][kPad];
};

struct AttnArgs {
  DecodeArgs d;
  int blocks;            // blocks of 16 query heads per KV head
  int box;               // slots per TMA box: min(page_size, 64)
  int n_entries, mult;   // dense: rows, Hkv * blocks; page lists: rows * Hkv, blocks
  int64_t* prefix;       // [n_entries + 1] tiles of the entries before (one problem each)
  float* lse2;           // [rows][Hq] base-2 log-sum-exp, or NULL
  float* logits;         // [rows][Hq][cap] base-2 scores, or NULL
  int64_t cap;
  float2* part_ml;       // [2 CTAs][16]
  float* part_o;         // [2 CTAs][16][D]
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
  n.len = paged_row(kv, d.row_seq, d.row_len, n.row, &n.seq);
  n.lo = n.sinks = n.t_sink = n.t_skip = n.n_list = 0;
  n.list = nullptr;
  if (d.sel) {
    const int c = d.sel_count[e];
    n.list = d.sel + (int64_t)e * d.sel_stride;
    n.n_list = n.len == 0 || c < 0 ? 0 : c > d.sel_stride ? (int)d.sel_stride : c;
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

// First tile of CTA c's range.
__device__ __forceinline__ int64_t range_start(int64_t total, int c, int ctas) { return total * c / ctas; }

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
  static constexpr int kStages = stages_of(2 * kHalf);
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
    const int64_t t = e < a.n_entries ? entry_of(a, e).tiles : 0;
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

// More entries than kInline: one CTA writes the prefix for everybody.
__global__ void __launch_bounds__(1024) plan_kernel(const AttnArgs a) {
  __shared__ int64_t sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t run = 0;
  for (int e0 = 0; e0 < a.n_entries; e0 += 1024) {
    const int e = e0 + tid;
    const int64_t t = e < a.n_entries ? entry_of(a, e).tiles : 0;
    int64_t y = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    if (e < a.n_entries) a.prefix[e] = run + before + y - t;
    run += all;
    __syncthreads();
  }
  if (tid == 0) a.prefix[a.n_entries] = run;
}

// Part of the CTA's range inside one problem.
struct Segment {
  Entry n;
  int e, prob, first, count;  // entry, its problem, first tile of the problem, tiles
  bool whole;                 // the problem lies in this CTA alone
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
  const int64_t x = t - prefix[lo] * a.mult;
  s.prob = (int)(x / s.n.tiles);
  s.first = (int)(x - (int64_t)s.prob * s.n.tiles);
  s.count = (int)min((int64_t)(s.n.tiles - s.first), t1 - t);
  s.whole = s.count == s.n.tiles;
  return s;
}

template <typename QT, typename K, int D>
__global__ void __launch_bounds__(kThreads, kPerSm) attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap km,
                                                                const __grid_constant__ CUtensorMap vm) {
  using S = Stage<K, D>;
  using PT = std::conditional_t<std::is_same_v<K, __nv_bfloat16>, __nv_bfloat16, __half>;  // weights, values
  constexpr bool k8 = sizeof(K) == 1;
  constexpr float kBias = std::is_same_v<PT, __half> ? 15.f : 0.f;
  constexpr int NT = D / 8;   // output tiles of 8 dims
  constexpr int KS = D / 16;  // contraction steps of the scores
  extern __shared__ __align__(1024) uint8_t ring_[];
  __shared__ Shared sh;
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = (smem_u32(ring_) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(sh.full), empty = smem_u32(sh.empty);
  const bool inl = a.n_entries <= kInline;
  if (warp == kConsumers) {
    if (lane == 0) {
      for (int i = 0; i < S::kStages; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, kConsumers);
      }
      fence_mbar_init();
      sh.stop = 0;
    }
  } else if (warp == 0) {
    if (inl) tile_prefix(a, sh.prefix, lane);
  }
  asm volatile("griddepcontrol.launch_dependents;");
  if (!inl) asm volatile("griddepcontrol.wait;" ::: "memory");  // plan_kernel's prefix
  __syncthreads();
  const int64_t* prefix = inl ? sh.prefix : a.prefix;
  if (inl && blockIdx.x == 0)
    for (int e = tid; e <= a.n_entries; e += kThreads) a.prefix[e] = sh.prefix[e];
  const int64_t total = prefix[a.n_entries] * a.mult;
  const int ctas = (int)min((int64_t)gridDim.x, total);
  if ((int)blockIdx.x >= ctas) return;
  const int64_t t0 = range_start(total, blockIdx.x, ctas), t1 = range_start(total, blockIdx.x + 1, ctas);

  if (warp == kConsumers) {
    // ---- producer: lane (half, block, box) issues one TMA box of a tile
    const int boxes = kTile / a.box;
    const int bi = lane % boxes, blk = (lane / boxes) % S::kBlocks, is_v = lane / (boxes * S::kBlocks);
    const bool mine = is_v < 2;
    const CUtensorMap* map = is_v ? &vm : &km;
    const uint32_t dst0 = ring + is_v * S::kHalf + blk * (kTile * 128) + bi * a.box * S::kRow;
    const int subs = kv.page_size / a.box;
    bool dead = false;
    int st = 0;
    uint32_t phase = 0;
    int64_t t = t0;
    while (t < t1) {
      const Segment s = segment_at(a, prefix, t, t1);
      const int g = d.sel ? s.e % kv.Hkv : s.prob / a.blocks;
      for (int i = s.first; i < s.first + s.count; ++i) {
        int base = kNoSlot, page = 0;
        if (mine) {
          if (d.sel) {
            const int64_t b = (int64_t)i * boxes + bi;
            const int64_t li = b / subs;
            if (li < s.n.n_list) {
              const int p = s.n.list[li];
              if (p >= 0 && p < kv.max_pages) base = (p << kv.page_shift) + (int)(b % subs) * a.box;
            }
          } else {
            base = (i < s.n.t_sink ? i : i + s.n.t_skip) * kTile + bi * a.box;
          }
          if (base >= s.n.len || (base + a.box <= s.n.lo && base >= s.n.sinks)) {
            base = kNoSlot;
          } else {
            page = (int)paged_page(kv, s.n.seq, base >> kv.page_shift);
            if (page < 0) {
              paged_err(kv, RTP_PAGED_ERANGE);
              base = kNoSlot;
            }
          }
        }
        const bool load = base != kNoSlot;
        if (!dead && !mbar_wait(empty + 8 * st, phase ^ 1u)) {
          dead = true;
          paged_err(kv, RTP_PAGED_ETIMEOUT);
        }
        dead = __any_sync(0xffffffffu, dead || *(volatile int*)&sh.stop != 0);
        const int n_load = __popc(__ballot_sync(0xffffffffu, load));
        if (lane < boxes) sh.base[st][lane] = base;
        __syncwarp();
        if (lane == 0) mbar_expect_tx(full + 8 * st, dead ? 0u : (uint32_t)(n_load * a.box * S::kRow));
        __syncwarp();
        if (load && !dead)
          tma_load_4d(dst0 + st * 2 * S::kHalf, map, blk * (128 / (int)sizeof(K)), base & (kv.page_size - 1), g, page,
                      full + 8 * st);
        if (++st == S::kStages) {
          st = 0;
          phase ^= 1u;
        }
      }
      t += s.count;
    }
    // the consumers have waited for every copy, unless a wait gave up
    if (dead && lane < S::kStages) mbar_wait(full + 8 * lane, lane < st ? phase : phase ^ 1u);
    return;
  }

  // ---- consumers
  const int r0 = warp * 16, row = lane >> 2, c2 = (lane & 3) * 2;
  bool dead = false;
  int st = 0;
  uint32_t phase = 0;
  int64_t t = t0;
  while (t < t1) {
    const Segment s = segment_at(a, prefix, t, t1);
    const int g = d.sel ? s.e % kv.Hkv : s.prob / a.blocks;
    const int h0 = (d.sel ? s.prob : s.prob % a.blocks) * kHeads;  // first head of the group
    const int nh = min(kHeads, d.group - h0);
    // query fragments (A operands): rows are heads; for e4m3 the contraction slots of a step are
    // permuted as ldmatrix delivers the keys' bytes
    uint32_t q[KS][4];
    {
      const uint16_t* qp = (const uint16_t*)d.q + s.n.row * d.q_stride + (int64_t)(g * d.group + h0) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = row + (e & 1) * 8;
          const int dim = ks * 16 + (k8 ? 2 * c2 + (e >> 1) * 2 : c2 + (e >> 1) * 8);
          q[ks][e] = h < nh ? *(const uint32_t*)(qp + h * D + dim) : 0u;
        }
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float* logit = nullptr;
    if (a.logits) logit = a.logits + ((int64_t)s.n.row * d.Hq + g * d.group + h0) * a.cap;

    for (int i = 0; i < s.count; ++i) {
      if (!dead && !mbar_wait(full + 8 * st, phase)) {
        dead = true;
        *(volatile int*)&sh.stop = 1;
        if (lane == 0) paged_err(kv, RTP_PAGED_ETIMEOUT);
      }
      const int base = sh.base[st][r0 / a.box] + (r0 & (a.box - 1));
      const bool any = base < s.n.len && (base + 16 > s.n.lo || base < s.n.sinks) && !dead;
      if (any) {
        const uint32_t kb = ring + st * 2 * S::kHalf, vb = kb + S::kHalf;
        float z[2][4] = {};
        if constexpr (!k8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t b[4];
            ldsm_x4(kb + S::at(r0 + (lane >> 4) * 8 + (lane & 7), 2 * ks + ((lane >> 3) & 1)), b[0], b[1], b[2], b[3]);
            mma<QT>(z[0], q[ks], b[0], b[1]);
            mma<QT>(z[1], q[ks], b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ks += 2) {
            uint32_t b[4];
            ldsm_x4(kb + S::at(r0 + ((lane >> 3) & 1) * 8 + (lane & 7), ks + (lane >> 4)), b[0], b[1], b[2], b[3]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              mma<QT>(z[0], q[ks + u], widen2<QT>(b[2 * u]), widen2<QT>(b[2 * u] >> 16));
              mma<QT>(z[1], q[ks + u], widen2<QT>(b[2 * u + 1]), widen2<QT>(b[2 * u + 1] >> 16));
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u >> 2][u & 3] *= d.scale_log2;
        // slots of this lane: base + c2 + {0, 1, 8, 9}
        const bool part = base + 15 >= s.n.len || !(base >= s.n.lo || base + 15 < s.n.sinks);
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (part) {
          bool ok[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = base + c2 + (u & 1) + (u >> 1) * 8;
            ok[u] = j < s.n.len && (j >= s.n.lo || j < s.n.sinks);
            if (!ok[u]) z[u >> 1][u & 1] = z[u >> 1][2 + (u & 1)] = -INFINITY;
          }
          keep0 = (ok[0] ? 0xffffu : 0u) | (ok[1] ? 0xffff0000u : 0u);
          keep1 = (ok[2] ? 0xffffu : 0u) | (ok[3] ? 0xffff0000u : 0u);
        }
        if (logit) {
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int j = base + c2 + (u & 1) + (u >> 2) * 8, h = row + ((u >> 1) & 1) * 8;
            const uint32_t k = u >> 2 ? keep1 : keep0;
            if (h < nh && ((u & 1) ? k >> 31 : k & 1u)) logit[h * a.cap + j] = z[u >> 2][u & 3];
          }
        }
        float mx[2];
        bool grew = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float x = fmaxf(fmaxf(z[0][2 * u], z[0][2 * u + 1]), fmaxf(z[1][2 * u], z[1][2 * u + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          mx[u] = fmaxf(m[u], x);
          grew |= mx[u] > m[u];
        }
        if (__any_sync(0xffffffffu, grew)) {
          float f[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            f[u] = mx[u] == m[u] ? 1.f : fast_exp2(m[u] - mx[u]);
            m[u] = mx[u];
            l[u] *= f[u];
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][0] *= f[0];
            o[n][1] *= f[0];
            o[n][2] *= f[1];
            o[n][3] *= f[1];
          }
        }
        uint32_t p[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float off = (m[u] == -INFINITY ? 0.f : m[u]) - kBias;
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = fast_exp2(z[e >> 1][2 * u + (e & 1)] - off);
          }
          l[u] += (w[0] + w[1]) + (w[2] + w[3]);
          p[u] = pack2<PT>(w[0], w[1]);
          p[2 + u] = pack2<PT>(w[2], w[3]);
        }
        if constexpr (!k8) {
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            uint32_t b[4];
            ldsm_x4_t(vb + S::at(r0 + ((lane >> 3) & 1) * 8 + (lane & 7), n + (lane >> 4)), b[0], b[1], b[2], b[3]);
            if (part) {  // what lies in slots left out may be infinite or NaN
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
            mma<PT>(o[n], p, b[0], b[1]);
            mma<PT>(o[n + 1], p, b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; n += 4) {
            uint32_t b[4];
            ldsm_x4_t(vb + S::at(r0 + ((lane >> 3) & 1) * 8 + (lane & 7), n / 2 + (lane >> 4)), b[0], b[1], b[2], b[3]);
            if (part) {
              b[0] &= keep0;
              b[1] &= keep1;
              b[2] &= keep0;
              b[3] &= keep1;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t x = __byte_perm(b[2 * u], 0, 0x3120), y = __byte_perm(b[2 * u + 1], 0, 0x3120);
              mma<PT>(o[n + 2 * u], p, widen2<PT>(x), widen2<PT>(y));
              mma<PT>(o[n + 2 * u + 1], p, widen2<PT>(x >> 16), widen2<PT>(y >> 16));
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * st);
      if (++st == S::kStages) {
        st = 0;
        phase ^= 1u;
      }
    }

    // ---- the four warps' states joined; the whole result, or a partial one
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
      if ((lane & 3) == 0) {
        sh.m[warp][row + 8 * u] = m[u];
        sh.l[warp][row + 8 * u] = l[u];
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
    float f[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, sh.m[w][row + 8 * u]);
      f[u] = fast_exp2(m[u] - (M == -INFINITY ? 0.f : M));
    }
    const int oh = tid >> 3, od = (tid & 7) * 4;  // this thread's head and dims (of 32) in the exchange
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, sh.m[w][oh]);
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) L += sh.l[w][oh] * fast_exp2(sh.m[w][oh] - (M == -INFINITY ? 0.f : M));
    const int64_t pslot = 2 * (int64_t)blockIdx.x + (t == t0 ? 0 : 1);
#pragma unroll
    for (int rd = 0; rd < D / 32; ++rd) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int dim = k8 ? (n >> 1) * 16 + 2 * c2 + 2 * (e & 1) + (n & 1) : n * 8 + c2 + (e & 1);
          sh.x[warp][row + (e >> 1) * 8][dim] = o[rd * 4 + n][e] * f[e >> 1];
        }
      asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float4 y = *(const float4*)&sh.x[w][oh][od];
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      if (oh < nh) {
        if (s.whole) {
          const float inv = L == 0.f ? 0.f : kv.v_scale / L;
          uint2 r;
          r.x = pack2<QT>(x.x * inv, x.y * inv);
          r.y = pack2<QT>(x.z * inv, x.w * inv);
          if (L == 0.f) r = make_uint2(0u, 0u);
          *(uint2*)((uint16_t*)d.out + s.n.row * d.out_stride + (int64_t)(g * d.group + h0 + oh) * D + rd * 32 + od) = r;
        } else {
          *(float4*)(a.part_o + (pslot * kHeads + oh) * D + rd * 32 + od) = x;
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
    }
    if ((tid & 7) == 0 && oh < nh) {
      if (s.whole) {
        const float y = L == 0.f ? -INFINITY : M + (log2f(L) - kBias);
        const int64_t at = (int64_t)s.n.row * d.Hq + g * d.group + h0 + oh;
        if (d.lse) d.lse[at] = y * 0.6931471805599453f;
        if (a.lse2) a.lse2[at] = y;
      } else {
        a.part_ml[pslot * kHeads + oh] = make_float2(M, L);
      }
    }
    t += s.count;
  }
}

// One CTA per (query head, row): the partial results of a problem that crosses CTAs, in CTA order;
// zeros for a row without slots.
constexpr int kJoinWarps = 4;

template <typename QT, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const AttnArgs a, int grid, float bias) {
  asm volatile("griddepcontrol.launch_dependents;");
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  const int h = blockIdx.x, r = blockIdx.y, g = h / d.group, hh = h % d.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = d.sel ? r * kv.Hkv + g : r;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (h == 0 && threadIdx.x == 0 && paged_row_bad(kv, d.row_seq, d.row_len, r)) paged_err(kv, RTP_PAGED_ERANGE);
  const int64_t tiles = a.prefix[e + 1] - a.prefix[e];
  uint16_t* out = (uint16_t*)d.out + r * d.out_stride + (int64_t)h * D;
  const int64_t at = (int64_t)r * d.Hq + h;
  if (tiles == 0) {
    if (threadIdx.x < D / 2) *(uint32_t*)(out + 2 * threadIdx.x) = 0u;
    if (threadIdx.x == 0) {
      if (d.lse) d.lse[at] = -INFINITY;
      if (a.lse2) a.lse2[at] = -INFINITY;
    }
    return;
  }
  const int64_t total = a.prefix[a.n_entries] * a.mult;
  const int ctas = (int)min((int64_t)grid, total);
  const int prob = d.sel ? hh / kHeads : g * a.blocks + hh / kHeads;
  const int64_t s0 = a.prefix[e] * a.mult + prob * tiles, s1 = s0 + tiles - 1;
  int c0 = (int)(s0 * ctas / total), c1 = (int)(s1 * ctas / total);
  while (c0 + 1 < ctas && range_start(total, c0 + 1, ctas) <= s0) ++c0;
  while (c1 + 1 < ctas && range_start(total, c1 + 1, ctas) <= s1) ++c1;
  if (c0 == c1) return;  // written by its CTA
  const int hrow = hh % kHeads;
  const int64_t slot0 = 2 * (int64_t)c0 + (range_start(total, c0, ctas) == s0 ? 0 : 1);
  __shared__ float sm[kJoinWarps], sl[kJoinWarps];
  __shared__ float so[kJoinWarps][D];
  constexpr int V = D / 32;
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = 0.f;
  for (int c = c0 + warp; c <= c1; c += kJoinWarps) {
    const int64_t p = (c == c0 ? slot0 : 2 * (int64_t)c) * kHeads + hrow;
    const float2 ml = a.part_ml[p];
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = a.part_o[p * D + lane * V + v];
    const float mn = fmaxf(m, ml.x), base = mn == -INFINITY ? 0.f : mn;
    const float f0 = exp2f(m - base), f1 = exp2f(ml.x - base);
    m = mn;
    l = l * f0 + ml.y * f1;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = o[v] * f0 + x[v] * f1;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) so[warp][lane * V + v] = o[v];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, sm[w]);
  float f[kJoinWarps];
  for (int w = 0; w < kJoinWarps; ++w) {
    f[w] = exp2f(sm[w] - (M == -INFINITY ? 0.f : M));
    L += sl[w] * f[w];
  }
  if (threadIdx.x < D / 2) {
    const int x = 2 * threadIdx.x;
    float y0 = 0.f, y1 = 0.f;
    for (int w = 0; w < kJoinWarps; ++w) {
      y0 += so[w][x] * f[w];
      y1 += so[w][x + 1] * f[w];
    }
    const float inv = kv.v_scale / L;
    *(uint32_t*)(out + x) = L == 0.f ? 0u : pack2<QT>(y0 * inv, y1 * inv);
  }
  if (threadIdx.x == 0) {
    const float y = L == 0.f ? -INFINITY : M + (log2f(L) - bias);
    if (d.lse) d.lse[at] = y * 0.6931471805599453f;
    if (a.lse2) a.lse2[at] = y;
  }
}

// scores[row][g][j] += sum over g's heads of exp2(logit - lse2), for the slots attended.
__global__ void __launch_bounds__(256) weights_kernel(const AttnArgs a) {
  const DecodeArgs& d = a.d;
  const PagedView& kv = d.kv;
  const int g = blockIdx.y, r = blockIdx.z;
  __shared__ float lse[64];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Entry n = entry_of(a, r);
  if (threadIdx.x < d.group) {
    const float y = a.lse2[(int64_t)r * d.Hq + g * d.group + threadIdx.x];
    lse[threadIdx.x] = y == -INFINITY ? INFINITY : y;
  }
  __syncthreads();
  const float* lg = a.logits + ((int64_t)r * d.Hq + g * d.group) * a.cap;
  float* sc = d.scores + ((int64_t)r * kv.Hkv + g) * d.scores_stride;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n.sinks + n.len - n.lo; i += gridDim.x * 256) {
    const int j = i < n.sinks ? i : n.lo + i - n.sinks;
    if (paged_page(kv, n.seq, j >> kv.page_shift) < 0) continue;
    float w = 0.f;
    for (int u = 0; u < d.group; ++u) w += fast_exp2(lg[u * a.cap + j] - lse[u]);
    sc[j] += w;
  }
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

constexpr int kMaxSms = 160;  // what the workspace is sized for; a grid is at most kPerSm times it

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t prefix, lse2, ml, o, logits, total;
};
Layout layout_of(const rtp_paged_kv* kv, int n_rows, int n_q_heads, bool scores) {
  Layout l;
  size_t at = 0;
  const auto take = [&](size_t n) {
    const size_t x = at;
    at += align256(n);
    return x;
  };
  const size_t parts = (size_t)2 * kPerSm * kMaxSms * kHeads;
  l.prefix = take(((size_t)n_rows * kv->n_kv_heads + 1) * sizeof(int64_t));
  l.ml = take(parts * sizeof(float2));
  l.o = take(parts * kv->head_dim * sizeof(float));
  l.lse2 = take(scores ? (size_t)n_rows * n_q_heads * sizeof(float) : 0);
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

template <typename QT, typename K, int D>
cudaError_t run(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int grid, cudaStream_t st) {
  using S = Stage<K, D>;
  constexpr size_t smem = (size_t)S::kStages * 2 * S::kHalf + 1024;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(attn_kernel<QT, K, D>, smem, done);
  if (e != cudaSuccess) return e;
  if (a.n_entries > kInline) {
    plan_kernel<<<1, 1024, 0, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_after(attn_kernel<QT, K, D>, dim3(grid), kThreads, smem, st, a, km, vm);
  } else {
    attn_kernel<QT, K, D><<<grid, kThreads, smem, st>>>(a, km, vm);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const float bias = std::is_same_v<K, __nv_bfloat16> ? 0.f : 15.f;
  e = launch_after(join_kernel<QT, D>, dim3(a.d.Hq, a.d.n_rows), kJoinWarps * 32, 0, st, a, grid, bias);
  if (e != cudaSuccess || !a.logits) return e;
  const int64_t blocks = (a.cap + 1023) / 1024;
  return launch_after(weights_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024), a.d.kv.Hkv, a.d.n_rows), 256, 0,
                      st, a);
}

template <typename QT, typename K>
cudaError_t run_d(const AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, int grid, cudaStream_t st) {
  return a.d.kv.D == 64 ? run<QT, K, 64>(a, km, vm, grid, st) : run<QT, K, 128>(a, km, vm, grid, st);
}

}  // namespace

size_t paged_decode_workspace(const rtp_paged_kv* kv, int n_rows, int n_q_heads, bool scores) {
  return layout_of(kv, n_rows, n_q_heads, scores).total;
}

cudaError_t launch_paged_decode(const DecodeArgs& d, const rtp_paged_kv* kv, int qt, cudaStream_t st) {
  AttnArgs a{};
  a.d = d;
  a.blocks = (d.group + kHeads - 1) / kHeads;
  a.box = kv->page_size < kTile ? kv->page_size : kTile;
  a.n_entries = d.sel ? d.n_rows * kv->n_kv_heads : d.n_rows;
  a.mult = d.sel ? a.blocks : kv->n_kv_heads * a.blocks;
  a.cap = (int64_t)kv->max_pages * kv->page_size;
  const Layout l = layout_of(kv, d.n_rows, d.Hq, d.scores != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(d.workspace);
  a.prefix = reinterpret_cast<int64_t*>(ws + l.prefix);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  if (d.scores) {
    a.lse2 = reinterpret_cast<float*>(ws + l.lse2);
    a.logits = reinterpret_cast<float*>(ws + l.logits);
  }
  CUtensorMap km, vm;
  if (!map_pages(&km, kv->k, kv->k_stride, kv, a.box) || !map_pages(&vm, kv->v, kv->v_stride, kv, a.box))
    return cudaErrorInvalidValue;
  const int64_t slots = d.sel ? (int64_t)d.sel_stride * kv->page_size : a.cap;
  const int64_t most = (int64_t)a.n_entries * a.mult * ((slots + kTile - 1) / kTile);
  const int sms = device_sms();
  int64_t grid = (int64_t)kPerSm * (sms < kMaxSms ? sms : kMaxSms);
  if (grid > most) grid = most;
  const int kt = kv->dtype;
  if (qt == RTP_FP16 && kt == RTP_FP16) return run_d<__half, __half>(a, km, vm, (int)grid, st);
  if (qt == RTP_BF16 && kt == RTP_BF16) return run_d<__nv_bfloat16, __nv_bfloat16>(a, km, vm, (int)grid, st);
  if (qt == RTP_FP16) return run_d<__half, __nv_fp8_e4m3>(a, km, vm, (int)grid, st);
  return run_d<__nv_bfloat16, __nv_fp8_e4m3>(a, km, vm, (int)grid, st);
}

}  // namespace rtp
