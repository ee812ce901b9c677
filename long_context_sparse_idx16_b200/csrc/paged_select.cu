// paged_select.cu -- the pages a query attends to, by an upper bound of its scores in each page.
//
// For KV head g: score(page) = max_h sum_d max(q_hd lo_d, q_hd hi_d) over g's query heads h, in
// fp64 (products of 16-bit values are exact there and sums of 128 nearly always are, so the order
// of summation does not move a page across the cut).  The top pages come from a radix select over
// the order-preserving 64-bit keys of the scores; ties take the lower page.
#include "paged.cuh"

namespace rtp {

namespace {

constexpr int kThreads = 256;

// A warp per page.
template <typename T, typename K>
__global__ void __launch_bounds__(kThreads) page_score_kernel(const SelectPagesArgs a) {
  const PagedView& kv = a.kv;
  const int g = blockIdx.y, r = blockIdx.z, lane = threadIdx.x & 31;
  int b;
  const int len = paged_row(kv, a.row_seq, a.row_len, r, &b);
  const int pages = (len + kv.page_size - 1) >> kv.page_shift;
  const T* q = (const T*)a.q + r * a.q_stride + (int64_t)g * a.group * kv.D;
  unsigned long long* keys = a.keys + ((int64_t)r * kv.Hkv + g) * kv.max_pages;
  for (int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < pages; i += gridDim.x * (kThreads / 32)) {
    unsigned long long key;
    const int64_t page = paged_page(kv, b, i);
    if (i < a.n_first || i >= pages - a.n_recent) {
      key = ~0ull;
    } else if (page < 0) {
      if (lane == 0) paged_err(kv, RTP_PAGED_ERANGE);
      key = 0;
    } else {
      const K* lim = (const K*)kv.bounds + ((page * kv.Hkv + g) * 2) * kv.D;
      double best = -INFINITY;
      bool nan = false;
      for (int u = 0; u < a.group; ++u) {
        double s = 0.0;
        for (int d = lane; d < kv.D; d += 32) {
          const double x = to_f32(q[u * kv.D + d]);
          s += x * to_f32(x < 0.0 ? lim[d] : lim[kv.D + d]);
        }
        s = warp_sum(s);
        nan |= s != s;
        best = fmax(best, s);
      }
      key = nan ? 0ull : order_key64(best);
    }
    if (lane == 0) keys[i] = key;
  }
}

// One CTA per (row, KV head): the threshold, then the pages above it in ascending order.
__global__ void __launch_bounds__(kThreads) page_pick_kernel(const SelectPagesArgs a) {
  const PagedView& kv = a.kv;
  const int g = blockIdx.x, r = blockIdx.y;
  __shared__ uint32_t hist[257];
  __shared__ int sums[33];
  int b;
  const int len = paged_row(kv, a.row_seq, a.row_len, r, &b);
  if (g == 0 && threadIdx.x == 0 && paged_row_bad(kv, a.row_seq, a.row_len, r)) paged_err(kv, RTP_PAGED_ERANGE);
  const int pages = (len + kv.page_size - 1) >> kv.page_shift;
  const int take = min(a.top, pages);
  const unsigned long long* keys = a.keys + ((int64_t)r * kv.Hkv + g) * kv.max_pages;
  int32_t* sel = a.sel + ((int64_t)r * kv.Hkv + g) * a.sel_stride;
  if (threadIdx.x == 0) a.sel_count[(int64_t)r * kv.Hkv + g] = take;
  for (int i = take + threadIdx.x; i < a.top; i += kThreads) sel[i] = -1;
  if (take == 0) return;
  int ties = 0x7fffffff;
  unsigned long long cut = 0;
  if (take < pages) cut = block_kth_largest(pages, take, hist, &ties, [&](int i) { return keys[i]; });
  int at = 0, tied = 0;
  for (int i0 = 0; i0 < pages; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const unsigned long long key = i < pages ? keys[i] : 0;
    const bool eq = i < pages && key == cut;
    int total;
    const int e = block_exclusive(eq, sums, &total);
    const bool in = i < pages && (key > cut || (eq && tied + e < ties));
    tied += total;
    const int o = block_exclusive(in, sums, &total);
    if (in) sel[at + o] = i;
    at += total;
  }
}

template <typename T, typename K>
void run_select(const SelectPagesArgs& a, cudaStream_t st) {
  const int per = kThreads / 32 * 8;
  const int blocks = (a.kv.max_pages + per - 1) / per;
  page_score_kernel<T, K><<<dim3(blocks < 1024 ? blocks : 1024, a.kv.Hkv, a.n_rows), kThreads, 0, st>>>(a);
  page_pick_kernel<<<dim3(a.kv.Hkv, a.n_rows), kThreads, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_paged_select(const SelectPagesArgs& a, int qt, int kvt, cudaStream_t st) {
  if (qt == RTP_FP16 && kvt == RTP_FP16) run_select<__half, __half>(a, st);
  else if (qt == RTP_BF16 && kvt == RTP_BF16) run_select<__nv_bfloat16, __nv_bfloat16>(a, st);
  else if (qt == RTP_FP16) run_select<__half, __nv_fp8_e4m3>(a, st);
  else run_select<__nv_bfloat16, __nv_fp8_e4m3>(a, st);
  return cudaGetLastError();
}

}  // namespace rtp
