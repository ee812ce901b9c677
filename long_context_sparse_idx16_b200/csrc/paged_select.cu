// paged_select.cu -- the pages a query attends to, by an upper bound of its scores in each page.
//
// For KV head g: score(page) = max_h sum_d max(q_hd lo_d, q_hd hi_d) over g's query heads h, which is
// [max(q, 0), min(q, 0)] . [hi, lo]: a product with 2 D terms.  The top pages by the exact (fp64)
// scores are wanted, ties to the lower page; that takes two steps:
//   * page_score_kernel forms all scores on the tensor cores (mma.sync, fp32 sums).  Products of
//     16-bit values are exact, so a score is off by at most eps = 2^-14 |q|_1 max|bound|: 2 D / 16
//     steps that each add 16 products and the running sum, every term cut at 2^-23 of the largest,
//     make at most 16 * 17 * 2^-23 < 2^-14.9 of the sum of all magnitudes.
//   * page_pick_kernel finds the bin of the last page taken in a linear histogram of these scores.
//     Pages above the bin by 2 eps are in, pages below it by 2 eps are out; the few between get
//     their exact fp64 scores and are ranked by them.  Where too many are between (equal scores,
//     infinities, NaN) all of them are scored exactly and a radix select over their 64-bit keys
//     decides.
// The bounds are read once per row (once per eight rows of a sequence that follow one another),
// 4 D bytes a page in 16 bits: HBM bounds the scoring of decode rows, the tensor cores that of chunks.
#include "paged.cuh"

namespace rtp {

namespace {

// ---- scores

constexpr int kScoreWarps = 8;
constexpr int kPagesPerWarp = kPageChunk / kScoreWarps;  // 32
constexpr int kRowBlock = 8;  // rows of a chunk that share one read of the bounds
constexpr int kMaxM = 64 + 16 * kRowBlock;  // heads of a run of rows that are kept at once

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

// One CTA: a chunk of pages, a KV head, a block of rows.  A warp takes 32 pages, 16 at a time: a lane
// holds E = 16 bytes' worth of successive dims of page (lane / 4) of an 8-page tile, dims
// (4 j + lane % 4) E ... of load j.  The queries lie in shared memory in the order of the
// contraction that this gives, max(q, 0) and min(q, 0) apart, rows 16 bytes off a multiple of 128.
template <typename T, typename K, int D>
__global__ void __launch_bounds__(32 * kScoreWarps) page_score_kernel(const SelectPagesArgs a, int row_block, int m_pad) {
  constexpr int E = 16 / (int)sizeof(K);
  constexpr int J = D / (4 * E);  // loads per bound
  constexpr int KS = D / 16;      // steps of 16 terms per bound
  constexpr int QS = 2 * D + 16;  // bytes between query rows
  extern __shared__ __align__(16) uint8_t smem_[];
  uint8_t* sq = smem_;                                                            // [2][m_pad][QS]
  uint32_t* best = reinterpret_cast<uint32_t*>(smem_ + (size_t)2 * m_pad * QS);   // [row_block][kPageChunk]
  __shared__ uint32_t s_max;
  const PagedView& kv = a.kv;
  const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r_end = min(a.n_rows, ((int)blockIdx.z + 1) * row_block);
  after_wait();
  for (int r = blockIdx.z * row_block; r < r_end;) {
    const Run u = run_at(a, r, r_end);
    r += u.count;
    const int p0 = blockIdx.x * kPageChunk;
    if (p0 >= u.pages) continue;  // the whole CTA alike
    const int m_rows = u.count * a.group;
    __syncthreads();
    for (int i = tid; i < u.count * kPageChunk; i += 32 * kScoreWarps) best[i] = 0u;
    if (tid == 0) s_max = 0u;
    uint32_t mag = 0u;
    // the bounds of two tiles of 8 pages: B operands [tile][hi, lo][step][2]
    uint32_t bb[2][2][KS][2];
    const auto load_bounds = [&](int n0) {
      const int pw = p0 + warp * kPagesPerWarp + n0;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int p = pw + t * 8 + (lane >> 2);
        const int64_t page = p < u.pages ? paged_page(kv, u.seq, p) : -1;
        const K* lim = (const K*)kv.bounds + ((page * kv.Hkv + g) * 2) * D + (lane & 3) * E;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const uint4 v = page < 0 ? make_uint4(0u, 0u, 0u, 0u) : ld_nc_u4(lim + (x ? 0 : D) + j * 4 * E);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (sizeof(K) == 1) {
                bb[t][x][4 * j + e][0] = widen2<T>(w[e]);
                bb[t][x][4 * j + e][1] = widen2<T>(w[e] >> 16);
              } else {
                bb[t][x][2 * j + (e >> 1)][e & 1] = w[e];
              }
            }
          }
      }
    };
    const int n_mine = min(kPagesPerWarp, u.pages - (p0 + warp * kPagesPerWarp));  // pages of this warp
    if (n_mine > 0) load_bounds(0);  // in flight while the queries are laid out
    // the run's heads, m_pad at a time (all of them, unless groups are large)
    for (int m0 = 0; m0 < m_rows; m0 += m_pad) {
      const int m_n = min(m_rows - m0, m_pad), m_tiles = (m_n + 15) / 16;
      __syncthreads();
      for (int i = tid; i < m_tiles * 16 * (D / 4); i += 32 * kScoreWarps) {
        // four dims: lane c's share of step k, two slots at 2 c and two at 8 + 2 c
        const int m = i / (D / 4), d = i % (D / 4) * 4, c = d / E % 4, k = d / (4 * E) * (E / 4) + d % E / 4;
        uint2 v = make_uint2(0u, 0u);
        if (m < m_n)
          v = *(const uint2*)((const T*)a.q + (u.first + (m0 + m) / a.group) * a.q_stride +
                              (int64_t)(g * a.group + (m0 + m) % a.group) * D + d);
        uint8_t* at = sq + m * QS + k * 32 + c * 4;
        *(uint32_t*)at = pos_part<T>(v.x);
        *(uint32_t*)(at + 16) = pos_part<T>(v.y);
        *(uint32_t*)(at + m_pad * QS) = neg_part<T>(v.x);
        *(uint32_t*)(at + m_pad * QS + 16) = neg_part<T>(v.y);
      }
      __syncthreads();
      for (int n0 = 0; n0 < n_mine; n0 += 16) {
        if (n0 > 0 || m0 > 0) load_bounds(n0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // pages outside the pool: no number, which the exact path ranks last
          const int p = n0 + t * 8 + (lane >> 2);
          if (p < n_mine && (lane & 3) == 0 && paged_page(kv, u.seq, p0 + warp * kPagesPerWarp + p) < 0)
            for (int i = 0; i < u.count; ++i) atomicMax(&best[i * kPageChunk + warp * kPagesPerWarp + p], 0xffffffffu);
        }
        if (m0 == 0) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int k = 0; k < KS; ++k) mag = abs_max<T>(abs_max<T>(mag, bb[t][x][k][0]), bb[t][x][k][1]);
        }
        __syncwarp();
        uint32_t* out = best + warp * kPagesPerWarp + n0;  // [row][page of this warp's 16]
#pragma unroll 1
        for (int mt = 0; mt < m_tiles; ++mt) {
          float c[2][4] = {};
          const uint32_t at = smem_u32(sq + (mt * 16 + (lane & 15)) * QS + (lane >> 4) * 16);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t f[4];
            ldsm_x4(at + k * 32, f[0], f[1], f[2], f[3]);
            mma<T>(c[0], f, bb[0][0][k][0], bb[0][0][k][1]);
            mma<T>(c[1], f, bb[1][0][k][0], bb[1][0][k][1]);
            ldsm_x4(at + m_pad * QS + k * 32, f[0], f[1], f[2], f[3]);
            mma<T>(c[0], f, bb[0][1][k][0], bb[0][1][k][1]);
            mma<T>(c[1], f, bb[1][1][k][0], bb[1][1][k][1]);
          }
          // the greatest head of each row, as order keys (a NaN of the products is the greatest key).
          // c[t][e]: head lane / 4 + 8 (e / 2), page 8 t + 2 (lane % 4) + e % 2
          const int m = m0 + mt * 16 + (lane >> 2);
          if ((a.group & 7) == 0) {
            // eight heads of a row in the eight lanes of a page: halved three times, each lane ends
            // with one of the eight (row half, tile, page parity) combinations
            uint32_t key[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) key[x] = order_key(c[(x >> 1) & 1][(x & 1) + (x >> 2) * 2]);
            const int hi2 = (lane >> 4) & 1, hi1 = (lane >> 3) & 1, hi0 = (lane >> 2) & 1;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t mine = hi2 ? key[x + 4] : key[x], other = hi2 ? key[x] : key[x + 4];
              key[x] = max(mine, __shfl_xor_sync(0xffffffffu, other, 16));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t mine = hi1 ? key[x + 2] : key[x], other = hi1 ? key[x] : key[x + 2];
              key[x] = max(mine, __shfl_xor_sync(0xffffffffu, other, 8));
            }
            const uint32_t mine = hi0 ? key[1] : key[0], other = hi0 ? key[0] : key[1];
            const uint32_t top = max(mine, __shfl_xor_sync(0xffffffffu, other, 4));
            const int row = m0 + mt * 16 + hi2 * 8;
            if (row < m_rows) {
              uint32_t* to = out + row / a.group * kPageChunk + hi1 * 8 + (lane & 3) * 2 + hi0;
              if (a.group == 8) *to = max(*to, top);  // nobody else writes it now
              else atomicMax(to, top);
            }
          } else {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int x = m + (e >> 1) * 8;
                if (x < m_rows)
                  atomicMax(out + x / a.group * kPageChunk + t * 8 + (lane & 3) * 2 + (e & 1), order_key(c[t][e]));
              }
          }
        }
      }
    }
    // magnitude of the bounds seen
    {
      const T* h = reinterpret_cast<const T*>(&mag);
      const float x = fmaxf(to_f32(h[0]), to_f32(h[1]));
      const uint32_t y = __reduce_max_sync(0xffffffffu, __float_as_uint(x));  // not negative: bits order alike
      if (lane == 0) atomicMax(&s_max, y);
    }
    __syncthreads();
    for (int i = tid; i < u.count * kPageChunk; i += 32 * kScoreWarps) {
      const int row = u.first + i / kPageChunk, p = p0 + i % kPageChunk;
      if (p < u.pages) {
        const uint32_t key = best[i];
        a.approx[((int64_t)row * kv.Hkv + g) * kv.max_pages + p] =
            key == 0xffffffffu ? __uint_as_float(0x7fc00000u) : key_to_float(key);
      }
    }
    for (int i = tid; i < u.count; i += 32 * kScoreWarps)
      a.chunk_max[((int64_t)(u.first + i) * kv.Hkv + g) * gridDim.x + blockIdx.x] = __uint_as_float(s_max);
  }
}

// ---- the choice

constexpr int kBins = 1024;
constexpr int kMaxBetween = 256;  // pages ranked by their exact scores in shared memory
constexpr int kPagesInSmem = 48 * 1024;

struct PickShared {
  uint32_t hist[kBins];
  uint32_t small[257];
  float f[4][32];
  int sums[33];
  int bin, n_in, n_between, got;
  int idx[kMaxBetween];
  unsigned long long key[kMaxBetween];
};

// Exact order key of one head's score in a page, by one warp; 0 (last) for a page outside the pool,
// ~0 for a score that is no number (one such head makes the page rank last).
template <typename T, typename K>
__device__ __forceinline__ unsigned long long exact_key(const SelectPagesArgs& a, const T* q, int seq, int g, int p) {
  const PagedView& kv = a.kv;
  const int lane = threadIdx.x & 31;
  const int64_t page = paged_page(kv, seq, p);
  if (page < 0) {
    if (lane == 0) paged_err(kv, RTP_PAGED_ERANGE);
    return 0ull;
  }
  const K* lim = (const K*)kv.bounds + ((page * kv.Hkv + g) * 2) * kv.D;
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = e * 32 + lane;
    const double x = d < kv.D ? to_f32(q[d]) : 0.f;
    const double lo = d < kv.D ? to_f32(lim[d]) : 0.f, hi = d < kv.D ? to_f32(lim[kv.D + d]) : 0.f;
    s += x * (x < 0.0 ? lo : hi);
  }
  s = warp_sum(s);
  return s != s ? ~0ull : order_key64(s);
}

// One CTA of kT threads per (KV head, row); the scores in shared memory, or in the workspace itself.
template <typename T, typename K, int kT, bool kSmem>
__global__ void __launch_bounds__(kT) page_pick_kernel(const SelectPagesArgs a, int chunks) {
  extern __shared__ float list_[];
  __shared__ PickShared s;
  const PagedView& kv = a.kv;
  const int g = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins; i += kT) s.hist[i] = 0;
  for (int i = tid; i < kMaxBetween; i += kT) s.key[i] = 0ull;
  if (tid == 0) s.got = 0;
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
  float* x = kSmem ? list_ : ws;
  const T* q = (const T*)a.q + r * a.q_stride + (int64_t)g * a.group * kv.D;
  // a page is in if its score lies in a bin from `cut` on, or is +inf
  float lo = 0.f, scale = 0.f;
  int cut = kBins;
  const auto bin_of = [&](float y) { return min(kBins - 1, (int)((y - lo) * scale)); };
  const bool choose = want > 0 && want < c1 - c0;
  float q1 = 0.f;  // the greatest |q|_1 of the heads
  if (choose)
    for (int u = warp; u < a.group; u += kT / 32) {
      float y = 0.f;
      for (int d = lane; d < kv.D; d += 32) y += fabsf(to_f32(q[u * kv.D + d]));
      q1 = fmaxf(q1, warp_sum(y));
    }
  after_wait();
  if (choose) {
    // the scores' range; eps
    float low = INFINITY, high = -INFINITY, mag = 0.f;
    bool odd = false;
#pragma unroll 4
    for (int i = c0 + tid; i < c1; i += kT) {
      const float y = ws[i];
      if (kSmem) x[i] = y;
      low = fminf(low, y);
      high = fmaxf(high, y);
      odd |= !isfinite(y);
    }
    for (int i = tid; i < chunks && i * kPageChunk < pages; i += kT) mag = fmaxf(mag, a.chunk_max[prob * chunks + i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
      mag = fmaxf(mag, __shfl_xor_sync(0xffffffffu, mag, o));
    }
    if (lane == 0) {
      s.f[0][warp] = low;
      s.f[1][warp] = high;
      s.f[2][warp] = mag;
      s.f[3][warp] = q1;
    }
    odd = __syncthreads_or(odd);
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) {
      low = fminf(low, s.f[0][w]);
      high = fmaxf(high, s.f[1][w]);
      mag = fmaxf(mag, s.f[2][w]);
      q1 = fmaxf(q1, s.f[3][w]);
    }
    // 1.01 covers the rounding of |q|_1 and of this product; 2^-110 what underflows in fp32
    const float eps = 1.01f * 6.103515625e-05f * q1 * mag + 7.7e-34f;
    // Bins at least 2.5 eps wide (a bin's place is off by less than 2^-12 of a bin): whatever lies
    // within 2 eps of the last page taken lies in its bin or a neighbouring one.
    const float range = high - low;
    bool done = !odd && isfinite(eps) && isfinite(range);
    if (done) {
      lo = low;
      scale = fminf((float)kBins / fmaxf(range, 1e-30f), 0.4f / eps);
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
      const int bin = s.bin, m = s.n_between, need = want - s.n_in;
      cut = bin + 2;
      for (int i = c0 + tid; i < c1; i += kT) {
        const int b = bin_of(x[i]);
        if (b >= bin - 1 && b <= bin + 1) s.idx[atomicAdd(&s.got, 1)] = i;
      }
      __syncthreads();
      // a warp per page and head; the greatest head's key
      for (int j = warp; j < m * a.group; j += kT / 32) {
        const unsigned long long k = exact_key<T, K>(a, q + j % a.group * kv.D, seq, g, s.idx[j / a.group]);
        if (lane == 0) atomicMax(&s.key[j / a.group], k);
      }
      __syncthreads();
      for (int j = tid; j < m; j += kT)
        if (s.key[j] == ~0ull) s.key[j] = 0ull;
      __syncthreads();
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
      for (int i = c0 + warp; i < c1; i += kT / 32) {
        unsigned long long k = 0ull;
        for (int u = 0; u < a.group; ++u) k = max(k, exact_key<T, K>(a, q + u * kv.D, seq, g, i));
        if (lane == 0) keys[i] = k == ~0ull ? 0ull : k;
      }
      __syncthreads();
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
  // the pages taken, ascending: a warp takes a contiguous piece
  const bool all = want >= c1 - c0;
  const int per = (pages + kT - 1) / kT * 32;
  const int i0 = warp * per, i1 = min(pages, i0 + per);
  const auto taken = [&](int i) {
    if (i < c0 || i >= c1 || all) return true;
    if (want <= 0) return false;
    const float y = x[i];
    return y == INFINITY || bin_of(y) >= cut;
  };
  int n = 0;
  for (int i = i0 + lane; i - lane < i1; i += 32) n += __popc(__ballot_sync(0xffffffffu, i < i1 && taken(i)));
  int total;
  int at = block_exclusive(lane == 0 ? n : 0, s.sums, &total);
  at = __shfl_sync(0xffffffffu, at, 0);
  for (int i = i0 + lane; i - lane < i1; i += 32) {
    const bool in = i < i1 && taken(i);
    const uint32_t bits = __ballot_sync(0xffffffffu, in);
    if (in) sel[at + __popc(bits & ((1u << lane) - 1u))] = i;
    at += __popc(bits);
  }
}

template <typename T, typename K, int kT>
cudaError_t run_pick(const SelectPagesArgs& a, int chunks, cudaStream_t st) {
  const dim3 grid(a.kv.Hkv, a.n_rows);
  if (a.kv.max_pages > kPagesInSmem) return launch_after(page_pick_kernel<T, K, kT, false>, grid, kT, 0, st, a, chunks);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(page_pick_kernel<T, K, kT, true>, kPagesInSmem * sizeof(float), done);
  if (e != cudaSuccess) return e;
  return launch_after(page_pick_kernel<T, K, kT, true>, grid, kT, a.kv.max_pages * sizeof(float), st, a, chunks);
}

template <typename T, typename K, int D>
cudaError_t run_select(const SelectPagesArgs& a, cudaStream_t st) {
  const int chunks = page_chunks(a.kv.max_pages);
  const int row_block = a.row_seq ? kRowBlock : 1;
  int m_pad = (row_block * a.group + 15) / 16 * 16;
  if (m_pad > kMaxM) m_pad = kMaxM;
  constexpr int QS = 2 * D + 16;
  const size_t smem = (size_t)2 * m_pad * QS + (size_t)row_block * kPageChunk * sizeof(uint32_t);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(page_score_kernel<T, K, D>, (size_t)2 * kMaxM * QS + kRowBlock * kPageChunk * sizeof(uint32_t),
                             done);
  if (e != cudaSuccess) return e;
  e = launch_after(page_score_kernel<T, K, D>, dim3(chunks, a.kv.Hkv, (a.n_rows + row_block - 1) / row_block),
                   32 * kScoreWarps, smem, st, a, row_block, m_pad);
  if (e != cudaSuccess) return e;
  // Few lists: as many threads as a CTA has, for the latency; many: small CTAs, many at once.
  const int64_t lists = (int64_t)a.n_rows * a.kv.Hkv;
  if (lists <= 2 * 148 || a.kv.max_pages > 8192) return run_pick<T, K, 1024>(a, chunks, st);
  return run_pick<T, K, 128>(a, chunks, st);
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
