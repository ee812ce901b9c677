// paged_select.cu -- the pages a query attends to, by an upper bound of its scores in each page.
//
// For KV head g: score(page) = max_h sum_d max(q_hd lo_d, q_hd hi_d) over g's query heads h, which is
// [max(q, 0), min(q, 0)] . [hi, lo]: a product with 2 D terms.  The top pages by the exact (fp64)
// scores are wanted, ties to the lower page; that takes two steps:
//   * page_score_kernel forms all scores on the tensor cores (mma.sync, fp32 sums) and takes them to be
//     off by at most eps = 2^-14 |q|_1 max|bound|.  How these instructions add is not documented.  The
//     assumption is: products of 16-bit values exact; 2 D / 16 steps that each add 16 products and
//     the running sum, every term cut at 2^-23 of the largest, which make at most 16 * 17 * 2^-23 <
//     2^-14.9 of the sum of all magnitudes; 2^-14 leaves a factor 1.9.  Tests of scores nearer to one
//     another than fp32 tells check the choice.
//   * page_pick_kernel finds the bin of the last page taken in a linear histogram of these scores.
//     Pages above the bin by 2 eps are in, pages below it by 2 eps are out; the few between get
//     their exact fp64 scores and are ranked by them.  Where too many are between (equal scores,
//     infinities, NaN) all of them are scored exactly and a radix select over their 64-bit keys
//     decides.
// The bounds are read once per row (once per eight rows of a sequence that follow one another),
// 4 D bytes a page in 16 bits: HBM bounds the scoring of decode rows, the tensor cores and the issue
// slots that of chunks.  Measured (one B200, 32 / 4 heads of 128): 8 rows of 2048 pages (33.5 MB) are
// scored in 10 us and chosen from in 8 us; four lists of 16384 pages in 10 and 13 us; 1000 chunk rows
// of 1022 pages (a third of the tensor pipe's rate) in 105 and 62 us.  All scores in fp64, a warp per
// page, took 98 us, 94 us and 4.2 ms.  A cluster per list with the histogram in distributed shared
// memory was slower than one CTA (59 against 47 us for the 2048-page case as a whole).
#include "paged.cuh"
#include "tc_umma.cuh"

namespace rtp {

namespace {

// ---- scores

constexpr int kScoreWarps = 8;
constexpr int kRowBlock = 8;  // rows of a chunk that share one read of the bounds, at most
constexpr int kMaxM = 192;    // heads of these rows, at most
constexpr int kCtaPages = kScoreWarps * kPageChunk;

template <typename T>
using pair_t = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
template <typename T>
__device__ __forceinline__ pair_t<T> as_pair(uint32_t x) {
  return *reinterpret_cast<pair_t<T>*>(&x);
}
template <typename P>
__device__ __forceinline__ uint32_t as_bits(P x) {
  return *reinterpret_cast<uint32_t*>(&x);
}
// max(x, 0) and min(x, 0) of a pair; a NaN gives NaN
template <typename T>
__device__ __forceinline__ uint32_t pos_part(uint32_t x) {
  return as_bits(__hmax2_nan(as_pair<T>(x), as_pair<T>(0u)));
}
template <typename T>
__device__ __forceinline__ uint32_t neg_part(uint32_t x) {
  return as_bits(__hmin2_nan(as_pair<T>(x), as_pair<T>(0u)));
}
// running maximum of magnitudes, in T pairs (NaN shows in the scores themselves)
template <typename T>
__device__ __forceinline__ uint32_t abs_max(uint32_t m, uint32_t x) {
  return as_bits(__hmax2(as_pair<T>(m), as_pair<T>(x & 0x7fff7fffu)));
}

// A run of rows of one sequence inside a block of kRowBlock rows.
struct Run {
  int first, count, seq, pages;  // pages: of its longest row
};
__device__ __forceinline__ Run run_at(const SelectPagesArgs& a, int r, int end) {
  Run u;
  u.first = r;
  int len = paged_row(a.kv, a.row_seq, a.row_len, r, &u.seq);
  u.count = 1;
  while (r + u.count < end && a.row_seq[r + u.count] == a.row_seq[r]) {
    int s;
    len = max(len, paged_row(a.kv, a.row_seq, a.row_len, r + u.count, &s));
    ++u.count;
  }
  u.pages = (int)(((int64_t)len + a.kv.page_size - 1) >> a.kv.page_shift);
  return u;
}

// One CTA: a KV head, a block of rows, `rounds` times 128 pages.  The rows' queries are laid out in
// shared memory in the order of the contraction, max(q, 0) and min(q, 0) apart; from there on the warps
// work by themselves, 16 pages at a time.  A lane copies half of one page's bounds (its lo or its hi
// row) to the warp's piece of shared memory, so that 16 pages are in flight at once; rows there are 16
// bytes off a multiple of 128, which ldmatrix reads without conflicts.  The bounds go to registers for
// all of the heads, and the next 16 pages are on their way meanwhile.
template <typename T, typename K, int D>
struct Score {
  static constexpr int kB = 2 * D * (int)sizeof(K);  // bytes of a page's bounds
  static constexpr int kBS = kB + 16;
  static constexpr int kQS = 2 * D + 16;             // bytes between query rows
  static size_t smem(int m_pad, int row_block) {
    return (size_t)kCtaPages * kBS + (size_t)2 * m_pad * kQS + (size_t)row_block * kCtaPages * sizeof(uint32_t);
  }
};

template <typename T, typename K, int D>
__global__ void __launch_bounds__(32 * kScoreWarps) page_score_kernel(const SelectPagesArgs a, int row_block, int m_pad,
                                                                      int rounds, int chunks) {
  using S = Score<T, K, D>;
  constexpr bool k8 = sizeof(K) == 1;
  constexpr int KS = D / 16;  // steps of 16 terms per bound
  extern __shared__ __align__(16) uint8_t smem_[];
  uint8_t* sq = smem_ + kCtaPages * S::kBS;                                           // [2][m_pad][kQS]
  __shared__ unsigned long long bar[kScoreWarps];
  const PagedView& kv = a.kv;
  const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* sb = smem_ + warp * kPageChunk * S::kBS;                                   // [kPageChunk][kBS], this warp's
  uint32_t* best = reinterpret_cast<uint32_t*>(sq + (size_t)2 * m_pad * S::kQS) + warp * kPageChunk;  // [row_block][kCtaPages]
  const int r_end = min(a.n_rows, ((int)blockIdx.z + 1) * row_block);
  const uint32_t landed = smem_u32(&bar[warp]);
  if (lane == 0) {
    mbar_init(landed, 1);
    fence_mbar_init();
  }
  __syncwarp();
  uint32_t phase = 0;
  after_wait();
  for (int r = blockIdx.z * row_block; r < r_end;) {
    const Run u = run_at(a, r, r_end);
    r += u.count;
    const int first = blockIdx.x * rounds * kCtaPages;
    if (first >= u.pages) continue;  // the whole CTA alike
    // copies of 16 pages from p on; whether this lane's page (lane % 16) lies outside the pool
    const auto start = [&](int p) -> bool {
      const bool live = p + (lane & 15) < u.pages;
      const int64_t page = live ? paged_page(kv, u.seq, p + (lane & 15)) : -1;
      const int n_load = __popc(__ballot_sync(0xffffffffu, page >= 0));
      uint8_t* to = sb + (lane & 15) * S::kBS + (lane >> 4) * (S::kB / 2);
      if (page < 0)  // pages left out: zeros
        for (int x = 0; x < S::kB / 32; ++x) ((uint4*)to)[x] = make_uint4(0u, 0u, 0u, 0u);
      if (lane == 0) mbar_expect_tx(landed, n_load * (S::kB / 2));
      __syncwarp();
      fence_async_smem();  // zeros of an earlier round lie behind this copy
      if (page >= 0)
        bulk_load(smem_u32(to), (const K*)kv.bounds + ((page * kv.Hkv + g) * 2 + (lane >> 4)) * D, S::kB / 2, landed);
      return live && page < 0;
    };
    int p = first + warp * kPageChunk;
    bool bad = false;
    if (p < u.pages) bad = start(p);
    const int m_rows = u.count * a.group, m_tiles = (m_rows + 15) / 16;
    __syncthreads();  // the last run's queries have been read
    for (int i = tid; i < m_tiles * 16 * (D / 4); i += 32 * kScoreWarps) {
      // four dims: 16-bit bounds in order; for e4m3, lane c's pair of pairs of step k, two slots at
      // 2 c and two at 8 + 2 c, as ldmatrix delivers the bounds' bytes
      const int m = i / (D / 4), d = i % (D / 4) * 4;
      uint2 v = make_uint2(0u, 0u);
      if (m < m_rows)
        v = *(const uint2*)((const T*)a.q + (u.first + m / a.group) * a.q_stride +
                            (int64_t)(g * a.group + m % a.group) * D + d);
      uint8_t* at = sq + m * S::kQS + (k8 ? d / 16 * 32 + d % 16 : d * 2);
      const int second = k8 ? 16 : 4;
      *(uint32_t*)at = pos_part<T>(v.x);
      *(uint32_t*)(at + second) = pos_part<T>(v.y);
      *(uint32_t*)(at + m_pad * S::kQS) = neg_part<T>(v.x);
      *(uint32_t*)(at + m_pad * S::kQS + second) = neg_part<T>(v.y);
    }
    __syncthreads();
    for (int round = 0; round < rounds && p < u.pages; ++round, p += kCtaPages) {
      if (!mbar_wait(landed, phase) && lane == 0) paged_err(kv, RTP_PAGED_ETIMEOUT);
      phase ^= 1u;
      __syncwarp();  // the other lanes' zeros
      uint32_t bb[2][2][KS][2];  // B operands [tile of 8 pages][hi, lo][step][2]
      uint32_t mag = 0u;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        // matrices of 8 pages by 16 bytes, four along the bounds: lo, then hi
        const uint32_t bt = smem_u32(sb + (t * 8 + (lane & 7)) * S::kBS + (lane >> 3) * 16);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int k = 0; k < KS; k += k8 ? 4 : 2) {
            uint32_t w[4];
            ldsm_x4(bt + (1 - x) * D * (int)sizeof(K) + k * 16 * (int)sizeof(K), w[0], w[1], w[2], w[3]);
            if constexpr (k8) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                bb[t][x][k + e][0] = widen2<T>(w[e]);
                bb[t][x][k + e][1] = widen2<T>(w[e] >> 16);
              }
            } else {
              bb[t][x][k][0] = w[0];
              bb[t][x][k][1] = w[1];
              bb[t][x][k + 1][0] = w[2];
              bb[t][x][k + 1][1] = w[3];
            }
          }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int k = 0; k < KS; ++k) mag = abs_max<T>(abs_max<T>(mag, bb[t][x][k][0]), bb[t][x][k][1]);
      }
      // The greatest magnitude of the 16 pages' bounds.  It depends on every value read, so the copy of
      // the next 16 pages behind it cannot overtake the reads.
      {
        const T* h = reinterpret_cast<const T*>(&mag);
        const float x = fmaxf(to_f32(h[0]), to_f32(h[1]));
        const uint32_t y = __reduce_max_sync(0xffffffffu, __float_as_uint(x));  // not negative: bits order alike
        if (lane < u.count)
          a.chunk_max[((int64_t)(u.first + lane) * kv.Hkv + g) * chunks + p / kPageChunk] = __uint_as_float(y);
      }
      const bool bad_now = bad;
      if (round + 1 < rounds && p + kCtaPages < u.pages) bad = start(p + kCtaPages);
      for (int i = lane; i < u.count * kPageChunk; i += 32) best[i / kPageChunk * kCtaPages + i % kPageChunk] = 0u;
      __syncwarp();
#pragma unroll 1
      for (int mt = 0; mt < m_tiles; ++mt) {
        // c[t][e]: head lane / 4 + 8 (e / 2), page 8 t + 2 (lane % 4) + e % 2
        float c[2][4] = {};
        const uint32_t at = smem_u32(sq + (mt * 16 + (lane & 15)) * S::kQS + (lane >> 4) * 16);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t f[4];
            ldsm_x4(at + x * m_pad * S::kQS + k * 32, f[0], f[1], f[2], f[3]);
            mma<T>(c[0], f, bb[0][x][k][0], bb[0][x][k][1]);
            mma<T>(c[1], f, bb[1][x][k][0], bb[1][x][k][1]);
          }
        // the greatest head of each row, as order keys (a NaN of the products is the greatest key)
        if ((a.group & 7) == 0) {
          // eight heads of a row in the eight lanes of a page: halved three times, each lane ends with
          // one of the eight (row half, tile, page parity) combinations
          uint32_t key[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) key[x] = order_key(c[(x >> 1) & 1][(x & 1) + (x >> 2) * 2]);
          const int hi2 = (lane >> 4) & 1, hi1 = (lane >> 3) & 1, hi0 = (lane >> 2) & 1;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t own = hi2 ? key[x + 4] : key[x], other = hi2 ? key[x] : key[x + 4];
            key[x] = max(own, __shfl_xor_sync(0xffffffffu, other, 16));
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t own = hi1 ? key[x + 2] : key[x], other = hi1 ? key[x] : key[x + 2];
            key[x] = max(own, __shfl_xor_sync(0xffffffffu, other, 8));
          }
          const uint32_t own = hi0 ? key[1] : key[0], other = hi0 ? key[0] : key[1];
          const uint32_t top = max(own, __shfl_xor_sync(0xffffffffu, other, 4));
          const int m = mt * 16 + hi2 * 8;
          uint32_t* to = best + hi1 * 8 + (lane & 3) * 2 + hi0;
          if (a.group == 8) {
            if (m < m_rows) to[(m >> 3) * kCtaPages] = top;  // all of the row's heads
          } else if (m < m_rows) {
            atomicMax(to + m / a.group * kCtaPages, top);
          }
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int m = mt * 16 + (lane >> 2) + (e >> 1) * 8;
              if (m < m_rows)
                atomicMax(best + m / a.group * kCtaPages + t * 8 + (lane & 3) * 2 + (e & 1), order_key(c[t][e]));
            }
        }
      }
      __syncwarp();
      // two rows of 16 pages at a time; no number for a page outside the pool: the exact path ranks it last
      for (int i = lane >> 4; i < u.count; i += 2) {
        const uint32_t key = best[i * kCtaPages + (lane & 15)];
        if (p + (lane & 15) < u.pages)
          a.approx[((int64_t)(u.first + i) * kv.Hkv + g) * kv.max_pages + p + (lane & 15)] =
              bad_now || key == 0xffffffffu ? __uint_as_float(0x7fc00000u) : key_to_float(key);
      }
      __syncwarp();
    }
  }
}

// ---- the choice

constexpr int kBins = 1024;
constexpr int kMaxBetween = 256;  // pages ranked by their exact scores in shared memory
constexpr int kPagesInSmem = 40 * 1024;

constexpr int kExactPages = 16;   // pages whose bounds are staged at a time for their exact scores
constexpr int kMaxPer = 64;       // pages a thread keeps its verdicts of

struct PickShared {
  uint32_t hist[kBins];
  uint32_t small[257];
  uint32_t low, high, mag, q1;      // order keys of the scores' range; bits of the magnitudes
  int sums[33];
  int bin, n_in, n_between, got;
  int idx[kMaxBetween], page[kMaxBetween];
  unsigned long long key[kMaxBetween];
};

// Exact order keys of pages [0, m) of `page` (pool numbers, -1: 0, which ranks last): the greatest
// head's, or 0 where one is no number.  Bounds go through shared memory, kExactPages at a time; a warp
// takes a (page, head).
template <typename T, typename K, int kT>
__device__ void exact_keys(const SelectPagesArgs& a, const T* sq, uint4* stage, unsigned long long* head_key,
                           const int* page, int g, int m, unsigned long long* key) {
  const PagedView& kv = a.kv;
  const int D = kv.D, tid = threadIdx.x, lane = tid & 31, units = 2 * D * (int)sizeof(K) / 16;
  for (int j0 = 0; j0 < m; j0 += kExactPages) {
    const int n = min(kExactPages, m - j0);
    __syncthreads();
    for (int i = tid; i < n * units; i += kT) {
      const int64_t p = page[j0 + i / units];
      stage[i] = p < 0 ? make_uint4(0u, 0u, 0u, 0u)
                       : ((const uint4*)((const K*)kv.bounds + ((p * kv.Hkv + g) * 2) * D))[i % units];
    }
    __syncthreads();
    for (int j = tid >> 5; j < n * a.group; j += kT / 32) {
      const K* lim = (const K*)stage + j / a.group * 2 * D;
      const T* q = sq + j % a.group * D;
      double s = 0.0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = e * 32 + lane;
        if (d < D) {
          const float x = to_f32(q[d]), b = to_f32(x < 0.f ? lim[d] : lim[D + d]);
          s += (double)x * (double)b;
        }
      }
      s = warp_sum(s);
      if (lane == 0) head_key[j] = s != s ? ~0ull : order_key64(s);
    }
    __syncthreads();
    for (int i = tid; i < n; i += kT) {
      unsigned long long k = 0ull;
      for (int u = 0; u < a.group; ++u) k = max(k, head_key[i * a.group + u]);
      key[j0 + i] = k == ~0ull || page[j0 + i] < 0 ? 0ull : k;
    }
  }
  __syncthreads();
}

// One CTA of kT threads per (KV head, row); the scores in shared memory, or in the workspace itself.
template <typename T, typename K, int kT, bool kSmem>
__global__ void __launch_bounds__(kT) page_pick_kernel(const SelectPagesArgs a, int chunks) {
  // [kExactPages][2 D] bounds, [kExactPages][group] keys, [group][D] queries, [pages] scores
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ PickShared s;
  const PagedView& kv = a.kv;
  const int g = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint4* stage = reinterpret_cast<uint4*>(dyn);
  unsigned long long* head_key = reinterpret_cast<unsigned long long*>(dyn + kExactPages * 2 * kv.D * sizeof(K));
  T* sq = reinterpret_cast<T*>(head_key + kExactPages * a.group);
  float* list = reinterpret_cast<float*>(sq + a.group * kv.D);
  for (int i = tid; i < kBins; i += kT) s.hist[i] = 0;
  if (tid == 0) {
    s.got = 0;
    s.low = ~0u;
    s.high = s.mag = s.q1 = 0u;
  }
  if (chunks == 0) after_wait();  // no scoring kernel runs ahead of this one
  // the operator's inputs may be read ahead of the scores, its outputs be written
  int seq;
  const int len = paged_row(kv, a.row_seq, a.row_len, r, &seq);
  if (g == 0 && tid == 0 && paged_row_bad(kv, a.row_seq, a.row_len, r)) paged_err(kv, RTP_PAGED_ERANGE);
  const int64_t prob = (int64_t)r * kv.Hkv + g;
  const int pages = (int)(((int64_t)len + kv.page_size - 1) >> kv.page_shift);
  const int take = min(a.top, pages);
  const int c0 = min(a.n_first, pages), c1 = max(c0, pages - a.n_recent);  // the pages to choose from
  const int want = take - (pages - (c1 - c0));
  int32_t* sel = a.sel + prob * a.sel_stride;
  if (tid == 0) a.sel_count[prob] = take;
  for (int i = take + tid; i < a.top; i += kT) sel[i] = -1;
  float* ws = a.approx + prob * kv.max_pages;
  float* x = kSmem ? list : ws;
  // a page is in if its score lies in a bin from `cut` on, or is +inf
  float lo = 0.f, scale = 0.f;
  int cut = kBins;
  bool told = false;  // by the histogram and the exact scores of a few pages
  const auto bin_of = [&](float y) { return min(kBins - 1, (int)((y - lo) * scale)); };
  const bool choose = want > 0 && want < c1 - c0;
  // a thread's own pages for the list at the end: an odd number of successive ones (no bank conflicts)
  const int per = (pages + kT - 1) / kT | 1;
  const int i0 = min(pages, tid * per), i1 = min(pages, i0 + per);
  unsigned long long sure = 0ull, maybe = 0ull;  // of these pages: taken; to be told by their exact scores
  __syncthreads();
  if (choose) {
    // the queries, and the greatest |q|_1 of the heads
    const T* q = (const T*)a.q + r * a.q_stride + (int64_t)g * a.group * kv.D;
    float q1 = 0.f;
    for (int u = warp; u < a.group; u += kT / 32) {
      float y = 0.f;
      for (int d = lane; d < kv.D; d += 32) {
        const T v = q[u * kv.D + d];
        sq[u * kv.D + d] = v;
        y += fabsf(to_f32(v));
      }
      q1 = fmaxf(q1, warp_sum(y));
    }
    if (lane == 0) atomicMax(&s.q1, q1 != q1 ? 0x7f800000u : __float_as_uint(q1));
  }
  after_wait();
  if (choose) {
    // the scores' range; eps
    uint32_t low = ~0u, high = 0u;
    float mag = 0.f;
    bool odd = false;
#pragma unroll 4
    for (int i = c0 + tid; i < c1; i += kT) {
      const float y = ws[i];
      if (kSmem) x[i] = y;
      low = min(low, order_key(y));
      high = max(high, order_key(y));
      odd |= !isfinite(y);
    }
    for (int i = tid; i < chunks && i * kPageChunk < pages; i += kT) mag = fmaxf(mag, a.chunk_max[prob * chunks + i]);
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    const uint32_t mags = __reduce_max_sync(0xffffffffu, __float_as_uint(mag));
    if (lane == 0) {
      atomicMin(&s.low, low);
      atomicMax(&s.high, high);
      atomicMax(&s.mag, mags);
    }
    odd = __syncthreads_or(odd);
    const float least = key_to_float(s.low), range = key_to_float(s.high) - least;
    // 1.01 covers the rounding of |q|_1 and of this product; 2^-110 what underflows in fp32
    const float eps = 1.01f * 6.103515625e-05f * __uint_as_float(s.q1) * __uint_as_float(s.mag) + 7.7e-34f;
    // Bins at least 2.5 eps wide (a bin's place is off by less than 2^-12 of a bin): whatever lies
    // within 2 eps of the last page taken lies in its bin or a neighbouring one.
    bool done = !odd && isfinite(eps) && isfinite(range);
    if (done) {
      lo = least;
      scale = fminf((float)kBins / fmaxf(range, 1e-30f), 0.4f / eps);
#pragma unroll 4
      for (int i = c0 + tid; i < c1; i += kT) atomicAdd(&s.hist[bin_of(x[i])], 1u);
      __syncthreads();
      constexpr int B = kBins / kT;
      int c[B], sum = 0, total;
#pragma unroll
      for (int e = 0; e < B; ++e) sum += c[e] = (int)s.hist[kBins - 1 - (tid * B + e)];
      int before = block_exclusive(sum, s.sums, &total);
#pragma unroll
      for (int e = 0; e < B; ++e) {
        if (before < want && before + c[e] >= want) {
          const int bin = kBins - 1 - (tid * B + e);
          const int up = bin + 1 < kBins ? (int)s.hist[bin + 1] : 0, down = bin > 0 ? (int)s.hist[bin - 1] : 0;
          s.bin = bin;
          s.n_in = before - up;
          s.n_between = up + c[e] + down;
        }
        before += c[e];
      }
      __syncthreads();
      done = s.n_between <= kMaxBetween;
    }
    if (done) {
      told = true;
      const int bin = s.bin, m = s.n_between, need = want - s.n_in;
      cut = bin + 2;
      for (int i = max(i0, c0); i < min(i1, c1); ++i) {
        const int b = bin_of(x[i]);
        if (b >= cut) {
          sure |= 1ull << ((i - i0) & 63);
        } else if (b >= bin - 1) {
          maybe |= 1ull << ((i - i0) & 63);
          const int at = atomicAdd(&s.got, 1);
          s.idx[at] = i;
          s.page[at] = (int)paged_page(kv, seq, i);
        }
      }
      exact_keys<T, K, kT>(a, sq, stage, head_key, s.page, g, m, s.key);
      for (int j = tid; j < m; j += kT) {
        const unsigned long long k = s.key[j];
        const int i = s.idx[j];
        int rank = 0;
        for (int l = 0; l < m; ++l) rank += s.key[l] > k || (s.key[l] == k && s.idx[l] < i);
        x[i] = rank < need ? INFINITY : lo;  // lo lies in bin 0, below the cut
      }
      __syncthreads();
    } else {
      // every page by its exact score
      unsigned long long* keys = a.keys + prob * kv.max_pages;
      for (int i0 = c0; i0 < c1; i0 += kMaxBetween) {
        const int n = min(kMaxBetween, c1 - i0);
        for (int i = tid; i < n; i += kT) {
          s.page[i] = (int)paged_page(kv, seq, i0 + i);
          if (s.page[i] < 0) paged_err(kv, RTP_PAGED_ERANGE);
        }
        exact_keys<T, K, kT>(a, sq, stage, head_key, s.page, g, n, s.key);
        for (int i = tid; i < n; i += kT) keys[i0 + i] = s.key[i];
        __syncthreads();
      }
      int ties;
      const unsigned long long kth = block_kth_largest(c1 - c0, want, s.small, &ties, [&](int i) { return keys[c0 + i]; });
      int tied = 0;
      for (int i0 = c0; i0 < c1; i0 += kT) {
        const int i = i0 + tid;
        const unsigned long long k = i < c1 ? keys[i] : 0ull;
        const bool eq = i < c1 && k == kth;
        int total;
        const int e = block_exclusive(eq, s.sums, &total);
        if (i < c1) x[i] = k > kth || (eq && tied + e < ties) ? INFINITY : 0.f;
        tied += total;
      }
      lo = scale = 0.f;
      cut = kBins;
      __syncthreads();
    }
  }
  // The pages taken, ascending: each thread counts its own and writes behind the threads before it.
  const bool all = want >= c1 - c0;
  const auto taken = [&](int i) {
    if (i < c0 || i >= c1 || all) return true;
    if (want <= 0) return false;
    const float y = x[i];
    return y == INFINITY || bin_of(y) >= cut;
  };
  const bool bits = per <= kMaxPer;
  if (bits) {
    if (told) {
      for (unsigned long long b = maybe; b; b &= b - 1) {
        const int u = __ffsll((long long)b) - 1;
        if (x[i0 + u] == INFINITY) sure |= 1ull << u;
      }
    }
    if (!choose || !told) {
      for (int i = i0; i < i1; ++i)
        if (taken(i)) sure |= 1ull << (i - i0);
    } else {
      for (int i = i0; i < min(i1, c0); ++i) sure |= 1ull << (i - i0);
      for (int i = max(i0, c1); i < i1; ++i) sure |= 1ull << (i - i0);
    }
  }
  int n = 0, total;
  if (bits) n = __popcll(sure);
  else
    for (int i = i0; i < i1; ++i) n += taken(i);
  int at = block_exclusive(n, s.sums, &total);
  if (bits) {
    for (unsigned long long b = sure; b; b &= b - 1) sel[at++] = i0 + __ffsll((long long)b) - 1;
  } else if (n) {
    for (int i = i0; i < i1; ++i)
      if (taken(i)) sel[at++] = i;
  }
}

template <typename T, typename K, int kT>
cudaError_t run_pick(const SelectPagesArgs& a, int chunks, cudaStream_t st) {
  const dim3 grid(a.kv.Hkv, a.n_rows);
  const size_t fixed = (size_t)kExactPages * 2 * a.kv.D * sizeof(K) +
                       (size_t)a.group * (kExactPages * sizeof(unsigned long long) + a.kv.D * sizeof(T));
  constexpr size_t kMost = kExactPages * 2 * kD * sizeof(T) + 64 * (kExactPages * 8 + kD * sizeof(T));  // of `fixed`
  cudaError_t e;
  if constexpr (kT == 1024) {  // (the small CTAs take short lists only)
    if (a.kv.max_pages > kPagesInSmem) {
      static std::atomic<uint64_t> done{0};
      if ((e = allow_smem(page_pick_kernel<T, K, kT, false>, kMost, done)) != cudaSuccess) return e;
      return launch_after(page_pick_kernel<T, K, kT, false>, grid, kT, fixed, st, a, chunks);
    }
  }
  static std::atomic<uint64_t> done{0};
  if ((e = allow_smem(page_pick_kernel<T, K, kT, true>, kMost + kPagesInSmem * sizeof(float), done)) != cudaSuccess) return e;
  return launch_after(page_pick_kernel<T, K, kT, true>, grid, kT, fixed + a.kv.max_pages * sizeof(float), st, a, chunks);
}

template <typename T, typename K, int D>
cudaError_t run_select(const SelectPagesArgs& a, cudaStream_t st) {
  const int chunks = page_chunks(a.kv.max_pages);
  int row_block = a.row_seq ? kRowBlock : 1;
  while (row_block * a.group > kMaxM) row_block /= 2;
  const int m_pad = (row_block * a.group + 15) / 16 * 16;
  // as many pages per CTA as still leaves two CTAs for every SM: the queries are laid out once for them
  const int blocks = (a.n_rows + row_block - 1) / row_block, groups = (chunks + kScoreWarps - 1) / kScoreWarps;
  int rounds = groups;
  while (rounds > 1 && (int64_t)((groups + rounds - 1) / rounds) * a.kv.Hkv * blocks < 2 * 148) rounds = (rounds + 1) / 2;
  using S = Score<T, K, D>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(page_score_kernel<T, K, D>, S::smem(kMaxM, kRowBlock), done);
  if (e != cudaSuccess) return e;
  // where every page is taken anyway no score is read
  if (a.top < a.kv.max_pages)
    e = launch_after(page_score_kernel<T, K, D>, dim3((groups + rounds - 1) / rounds, a.kv.Hkv, blocks), 32 * kScoreWarps,
                     S::smem(m_pad, row_block), st, a, row_block, m_pad, rounds, chunks);
  if (e != cudaSuccess) return e;
  const int scored = a.top < a.kv.max_pages ? chunks : 0;
  // Few lists: as many threads as a CTA has, for the latency; many: small CTAs, many at once.
  const int64_t lists = (int64_t)a.n_rows * a.kv.Hkv;
  if (lists <= 2 * 148 || a.kv.max_pages > 8192) return run_pick<T, K, 1024>(a, scored, st);
  return run_pick<T, K, 128>(a, scored, st);
}

template <typename T, typename K>
cudaError_t run_select_d(const SelectPagesArgs& a, cudaStream_t st) {
  return a.kv.D == 64 ? run_select<T, K, 64>(a, st) : run_select<T, K, 128>(a, st);
}

}  // namespace

cudaError_t launch_paged_select(const SelectPagesArgs& a, int qt, int kvt, cudaStream_t st) {
  if (qt == RTP_FP16 && kvt == RTP_FP16) return run_select_d<__half, __half>(a, st);
  if (qt == RTP_BF16 && kvt == RTP_BF16) return run_select_d<__nv_bfloat16, __nv_bfloat16>(a, st);
  if (qt == RTP_FP16) return run_select_d<__half, __nv_fp8_e4m3>(a, st);
  return run_select_d<__nv_bfloat16, __nv_fp8_e4m3>(a, st);
}

}  // namespace rtp
