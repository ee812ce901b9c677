// paged_evict.cu -- a cache brought back to a budget by the attention weight its slots drew.
//
// Slots are ranked by the 32-bit order key of their score, all ones for the slots that always stay
// (sinks and the newest); the budget-th largest key is the cut, equal keys take the lower position,
// then the lower slot.  Survivors behind the budget fill the freed slots below it, both in slot
// order, so exactly as many rows move as slots below the budget are freed, and no row moves that
// can stay.
//
// pick_kernel: one CTA per (sequence, KV head) reads scores and positions, keeps the keys in shared
// memory (beyond 24K slots it reads them again in each pass), finds the cut in three radix passes
// and writes the two lists.  move_kernel: the rows, 16 bytes a lane, over the whole GPU; HBM bounds
// it (each moved row is read and written once).
//
// Measured (one B200, 16 sequences of 8 KV heads, 8K to 16K slots brought to 8K, fp16, D = 128): 86 us,
// of which the move takes 53 us at the rate of a copy and the pick 32 us (latency: one CTA per list, on
// 128 of the SMs).  With the arrays read anew in every pass the pick took 320 us.
#include "paged.cuh"

namespace rtp {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kKeysInSmem = 24 * 1024;

struct PickShared {
  uint32_t hist[kBins];
  uint32_t small[257];
  int a[33], b[33];
  int newest, bin, above, exact;
};

// Finds the bin of the `want`-th largest key in hist: its number and the keys in the bins above it.
__device__ void find_bin(PickShared& s, int want) {
  // thread t holds bins kBins - 1 - 2 t and the one below it
  const int t = threadIdx.x;
  const int c0 = (int)s.hist[kBins - 1 - 2 * t], c1 = (int)s.hist[kBins - 2 - 2 * t];
  int total;
  const int before = block_exclusive(c0 + c1, s.a, &total);
  if (before < want && before + c0 >= want) {
    s.bin = kBins - 1 - 2 * t;
    s.above = before;
    s.exact = before + c0 == want;
  } else if (before + c0 < want && before + c0 + c1 >= want) {
    s.bin = kBins - 2 - 2 * t;
    s.above = before + c0;
    s.exact = before + c0 + c1 == want;
  }
  __syncthreads();  // (the caller's next write of hist lies behind another one)
}

template <bool kSmem>
__global__ void __launch_bounds__(kThreads) pick_kernel(const EvictArgs a) {
  extern __shared__ uint32_t keys[];  // [n] keys, then [n] positions
  __shared__ PickShared s;
  const PagedView& kv = a.kv;
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) s.newest = INT32_MIN;
  for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
  __syncthreads();
  after_wait();
  const int64_t prob = (int64_t)b * kv.Hkv + g, base = prob * a.stride;
  const float* sc = a.scores + base;
  const int32_t* pos = a.positions + base;
  int seq;
  const int n = paged_row(kv, nullptr, a.seq_len, b, &seq);
  if (g == 0 && tid == 0 && paged_row_bad(kv, nullptr, a.seq_len, b)) paged_err(kv, RTP_PAGED_ERANGE);
  const int keep = min(n, a.budget);
  if (g == 0 && tid == 0) a.out_len[b] = keep;
  const bool apart = a.out_scores != a.scores || a.out_positions != a.positions;
  int moved = 0;
  int32_t* pos_s = reinterpret_cast<int32_t*>(keys + n);
  // One pass over the arrays, in batches that are in flight together: the newest position; what stays
  // is copied (slots that are freed are written again below); scores and positions are kept.
  {
    constexpr int kBatch = 8;
    int newest = INT32_MIN;
    const int end = keep < n ? n : apart ? keep : 0;
    for (int i0 = tid; i0 < end; i0 += kThreads * kBatch) {
      float x[kBatch];
      int p[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads;
        x[u] = i < end ? sc[i] : 0.f;
        p[u] = i < end ? pos[i] : INT32_MIN;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kThreads;
        newest = max(newest, p[u]);
        if (i < end && kSmem && keep < n) {
          keys[i] = __float_as_uint(x[u]);
          pos_s[i] = p[u];
        }
        if (apart && i < keep) {
          a.out_scores[base + i] = x[u];
          a.out_positions[base + i] = p[u];
        }
      }
    }
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) atomicMax(&s.newest, newest);
  }
  if (keep < n) {
    __syncthreads();
    const int64_t recent = (int64_t)s.newest - a.n_recent;
    const auto position = [&](int i) -> int { return kSmem ? pos_s[i] : pos[i]; };
    const auto form = [&](int i) -> uint32_t {
      const int p = position(i);
      const float x = kSmem ? __uint_as_float(keys[i]) : sc[i];
      return p < a.n_sink || p > recent ? 0xffffffffu : x != x ? 0u : order_key(x + 0.f);
    };
    bool formed = false;  // each thread forms the keys of its own slots in its first pass over them
    const auto key = [&](int i) -> uint32_t { return kSmem && formed ? keys[i] : form(i); };

    // the cut: digits of 11, 11 and 10 bits; done early when a bin is taken whole
    uint32_t cut = 0;
    int want = keep;
    bool whole = false;
#pragma unroll 1
    for (int d = 0; d < 3 && !whole; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      if (d > 0) {
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
        __syncthreads();
      }
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads) {
        const uint32_t x = key(i);
        if (kSmem && d == 0) keys[i] = x;
        if (d == 0 || (x >> (d == 1 ? 21 : 10)) == (cut >> (d == 1 ? 21 : 10)))
          atomicAdd(&s.hist[d == 2 ? x & 1023u : (x >> shift) & 2047u], 1u);
      }
      formed = true;
      __syncthreads();
      find_bin(s, want);
      cut |= (uint32_t)s.bin << shift;
      want -= s.above;
      whole = s.exact != 0;
    }
    // ties: of the slots whose key is the cut, the `want` of lowest (position, slot)
    unsigned long long tie_cut = 0;
    if (!whole) {
      int ties;
      tie_cut = block_kth_largest(n, want, s.small, &ties, [&](int i) -> unsigned long long {
        if (key(i) != cut) return 0ull;
        return (unsigned long long)~((uint32_t)position(i) ^ 0x80000000u) << 32 | ~(uint32_t)i;
      });
    }
    const auto stays = [&](int i) -> bool {
      const uint32_t x = key(i);
      if (x != cut || whole) return x >= cut;
      return ((unsigned long long)~((uint32_t)position(i) ^ 0x80000000u) << 32 | ~(uint32_t)i) >= tie_cut;
    };

    // The lists, in slot order: a thread takes an odd number of successive slots (no bank conflicts),
    // counts its movers and holes, and writes them behind those of the threads before it.
    int32_t* mover = a.moves + base;
    int32_t* hole = mover + (n - keep);
    const int per = (n + kThreads - 1) / kThreads | 1;
    const int i0 = min(n, tid * per), i1 = min(n, i0 + per);
    int nm = 0, nh = 0;
    uint32_t verdict = 0;  // with the keys in shared memory a thread has at most 25 slots
    for (int i = i0; i < i1; ++i) {
      const bool in = stays(i);
      if (kSmem) verdict |= (uint32_t)in << (i - i0);
      nm += in && i >= keep;
      nh += !in && i < keep;
    }
    int holes;
    int om, oh;
    if (kSmem) {  // both counts in one sum: they stay below 2^16
      const int both = block_exclusive(nm | nh << 16, s.a, &holes);
      om = both & 0xffff;
      oh = both >> 16;
      moved = holes & 0xffff;
    } else {
      om = block_exclusive(nm, s.a, &moved);
      oh = block_exclusive(nh, s.b, &holes);
    }
    // the keys have served: their place takes the lists (moved <= n / 2)
    int32_t* movers = kSmem ? reinterpret_cast<int32_t*>(keys) : mover;
    int32_t* freed = kSmem ? movers + moved : hole;
    for (int i = i0; i < i1; ++i) {
      const bool in = kSmem ? (verdict >> (i - i0)) & 1u : stays(i);
      if (in && i >= keep) movers[om++] = i;
      if (!in && i < keep) freed[oh++] = i;
    }
    __syncthreads();
    // what moves in: the sources lie at or behind the budget, where nothing has been written yet
    constexpr int kBatch = 4;
    for (int m0 = tid; m0 < moved; m0 += kThreads * kBatch) {
      int to[kBatch], from[kBatch];
      float x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int m = m0 + u * kThreads;
        to[u] = m < moved ? freed[m] : 0;
        from[u] = m < moved ? movers[m] : 0;
        x[u] = sc[from[u]];
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int m = m0 + u * kThreads;
        if (m < moved) {
          if (kSmem) {
            mover[m] = from[u];
            hole[m] = to[u];
          }
          a.out_scores[base + to[u]] = x[u];
          a.out_positions[base + to[u]] = position(from[u]);
        }
      }
    }
    __syncthreads();
  }
  if (tid == 0) a.n_moves[prob] = moved;
  for (int64_t i = keep + tid; i < a.stride; i += kThreads) {
    a.out_scores[base + i] = 0.f;
    a.out_positions[base + i] = -1;
  }
}

// kMoveRows moves of one (sequence, KV head) per CTA: P = 2 row_bytes / 16 lanes per row (K, then V).
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a) {
  const PagedView& kv = a.kv;
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t prob = (int64_t)b * kv.Hkv + g, base = prob * a.stride;
  after_wait();
  const int moved = a.n_moves[prob];
  if ((int64_t)blockIdx.x * kMoveRows >= moved) return;
  int seq;
  const int n = paged_row(kv, nullptr, a.seq_len, b, &seq);
  const int32_t* mover = a.moves + base;
  const int32_t* hole = mover + (n - min(n, a.budget));
  __shared__ uint8_t* from_to[2][2][kMoveRows];  // [from, to][K, V]
  const int m0 = blockIdx.x * kMoveRows, rows = min(kMoveRows, moved - m0);
  if (threadIdx.x < 2 * rows) {
    const int m = threadIdx.x >> 1, to = threadIdx.x & 1;
    const int slot = to ? hole[m0 + m] : mover[m0 + m];
    const int64_t page = paged_page(kv, b, slot >> kv.page_shift);
    const int off = slot & (kv.page_size - 1);
    if (page < 0) paged_err(kv, RTP_PAGED_ERANGE);
    from_to[to][0][m] = page < 0 ? nullptr : kv.k + page * kv.kp + g * kv.kh + off * kv.ks;
    from_to[to][1][m] = page < 0 ? nullptr : kv.v + page * kv.vp + g * kv.vh + off * kv.vs;
  }
  __syncthreads();
  const int half = a.row_bytes / 16;  // lanes of a K or V row: 4, 8 or 16
  const int x = threadIdx.x % half, which = (threadIdx.x / half) & 1, step = kMoveThreads / (2 * half);
  constexpr int kUnroll = 4;
  for (int m = threadIdx.x / (2 * half); m < rows; m += step * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = m + u * step;
      if (r < rows && from_to[0][which][r] && from_to[1][which][r]) v[u] = ((const uint4*)from_to[0][which][r])[x];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = m + u * step;
      if (r < rows && from_to[0][which][r] && from_to[1][which][r]) ((uint4*)from_to[1][which][r])[x] = v[u];
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(const EvictArgs& a, cudaStream_t st) {
  const int64_t cap = (int64_t)a.kv.max_pages << a.kv.page_shift;
  const dim3 grid(a.kv.Hkv, a.kv.n_seqs);
  cudaError_t e;
  if (cap <= kKeysInSmem) {
    static std::atomic<uint64_t> done{0};
    if ((e = allow_smem(pick_kernel<true>, kKeysInSmem * 2 * sizeof(uint32_t), done)) != cudaSuccess) return e;
    e = launch_after(pick_kernel<true>, grid, kThreads, cap * 2 * sizeof(uint32_t), st, a);
  } else {
    e = launch_after(pick_kernel<false>, grid, kThreads, 0, st, a);
  }
  if (e != cudaSuccess) return e;
  // at most the smaller of the slots kept and the slots dropped move
  const int64_t most = cap - a.budget < a.budget ? cap - a.budget : a.budget;
  if (most <= 0) return cudaSuccess;
  return launch_after(move_kernel, dim3((unsigned)((most + kMoveRows - 1) / kMoveRows), a.kv.Hkv, a.kv.n_seqs),
                      kMoveThreads, 0, st, a);
}

}  // namespace rtp
