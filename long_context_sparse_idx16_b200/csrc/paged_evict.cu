// paged_evict.cu -- a cache brought back to a budget by the attention weight its slots drew.
//
// Slots are ranked by a 64-bit key, larger first: (score order key << 32) | ~position, the upper
// half all ones for the slots that always stay (sinks and the newest).  The budget-th largest key
// is the cut; equal keys take the lower slot.  Survivors behind the budget fill the freed slots
// below it, both in slot order, so exactly as many rows move as slots below the budget are freed.
#include "paged.cuh"

namespace rtp {

namespace {

constexpr int kThreads = 512;

// One CTA per (KV head, sequence).
__global__ void __launch_bounds__(kThreads) evict_kernel(const EvictArgs a) {
  const PagedView& kv = a.kv;
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  __shared__ uint32_t hist[257];
  __shared__ int sums[33];
  __shared__ int s_newest;
  const int64_t base = ((int64_t)b * kv.Hkv + g) * a.stride;
  const float* sc = a.scores + base;
  const int32_t* pos = a.positions + base;
  int seq;
  const int n = paged_row(kv, nullptr, a.seq_len, b, &seq);
  if (g == 0 && tid == 0 && paged_row_bad(kv, nullptr, a.seq_len, b)) paged_err(kv, RTP_PAGED_ERANGE);
  const int keep = min(n, a.budget);
  if (g == 0 && tid == 0) a.out_len[b] = keep;
  int32_t* mover = a.moves + base;
  if (keep < n) {
    if (tid == 0) s_newest = INT32_MIN;
    __syncthreads();
    int newest = INT32_MIN;
    for (int i = tid; i < n; i += kThreads) newest = max(newest, pos[i]);
    for (int o = 16; o > 0; o >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, o));
    if ((tid & 31) == 0) atomicMax(&s_newest, newest);
    __syncthreads();
    const int64_t recent = (int64_t)s_newest - a.n_recent;
    auto key = [&](int i) -> unsigned long long {
      const int p = pos[i];
      const float x = sc[i];
      const uint32_t hi = p < a.n_sink || p > recent ? 0xffffffffu : x != x ? 0u : order_key(x + 0.f);
      return (unsigned long long)hi << 32 | (uint32_t)~((uint32_t)p ^ 0x80000000u);
    };
    int ties;
    const unsigned long long cut = block_kth_largest(n, keep, hist, &ties, key);
    // movers first, in slot order, then the holes they fill (as many)
    int tied = 0, moved = 0, total;
    int32_t* hole = mover + (n - keep);
    int holes = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      const unsigned long long x = i < n ? key(i) : 0;
      const bool eq = i < n && x == cut;
      const int e = block_exclusive(eq, sums, &total);
      const bool in = i < n && (x > cut || (eq && tied + e < ties));
      tied += total;
      const bool mv = in && i >= keep, ho = i < keep && !in;
      const int om = block_exclusive(mv, sums, &total);
      if (mv) mover[moved + om] = i;
      moved += total;
      const int oh = block_exclusive(ho, sums, &total);
      if (ho) hole[holes + oh] = i;
      holes += total;
    }
    __syncthreads();
    // rows: a warp per move
    for (int m = tid >> 5; m < moved; m += kThreads / 32) {
      const int from = mover[m], to = hole[m];
      const int64_t fp = paged_page(kv, b, from >> kv.page_shift), tp = paged_page(kv, b, to >> kv.page_shift);
      if (fp < 0 || tp < 0) {
        if ((tid & 31) == 0) paged_err(kv, RTP_PAGED_ERANGE);
        continue;
      }
      const int fo = from & (kv.page_size - 1), to_ = to & (kv.page_size - 1);
      for (int c = (tid & 31) * 16; c < 2 * a.row_bytes; c += 512) {
        if (c < a.row_bytes)
          *(uint4*)(kv.k + tp * kv.kp + g * kv.kh + to_ * kv.ks + c) =
              *(const uint4*)(kv.k + fp * kv.kp + g * kv.kh + fo * kv.ks + c);
        else
          *(uint4*)(kv.v + tp * kv.vp + g * kv.vh + to_ * kv.vs + c - a.row_bytes) =
              *(const uint4*)(kv.v + fp * kv.vp + g * kv.vh + fo * kv.vs + c - a.row_bytes);
      }
    }
    // scores and positions: what stays, then what moves in (the sources lie at or behind the budget)
    if (a.out_scores != a.scores || a.out_positions != a.positions) {
      for (int i = tid; i < keep; i += kThreads) {
        a.out_scores[base + i] = sc[i];
        a.out_positions[base + i] = pos[i];
      }
      __syncthreads();
    }
    for (int m = tid; m < moved; m += kThreads) {
      a.out_scores[base + hole[m]] = sc[mover[m]];
      a.out_positions[base + hole[m]] = pos[mover[m]];
    }
    __syncthreads();
  } else {
    for (int i = tid; i < keep; i += kThreads) {
      a.out_scores[base + i] = sc[i];
      a.out_positions[base + i] = pos[i];
    }
  }
  for (int i = keep + tid; i < a.stride; i += kThreads) {
    a.out_scores[base + i] = 0.f;
    a.out_positions[base + i] = -1;
  }
}

}  // namespace

cudaError_t launch_paged_evict(const EvictArgs& a, cudaStream_t st) {
  evict_kernel<<<dim3(a.kv.Hkv, a.kv.n_seqs), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace rtp
