// paged_append.cu -- head norms, rotation and the write of K and V rows to their pages.
//
// For each head row x of q and k (fp32, rounded once to the stored type):
//   y = x * rsqrt(mean(x^2) + eps) * weight,
//   z_c = y_c cos - y_{c+D/2} sin, z_{c+D/2} = y_{c+D/2} cos + y_c sin, angle = pos * theta_c.
// The angle is formed and reduced in fp64 (rope_cos_sin); the rest is fp32.
#include "paged.cuh"

namespace rtp {

namespace {

// Sequence of token t: the last b with cu[b] <= t.
__device__ __forceinline__ int token_seq(const int32_t* cu, int n_seqs, int t) {
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One CTA of D/2 threads per token, thread c holding the pair (c, c + D/2) of a row.
template <typename T, typename K>
__global__ void append_kernel(const AppendArgs a) {
  const PagedView& kv = a.kv;
  const int t = blockIdx.x, c = threadIdx.x, H = kv.D / 2;
  __shared__ float red[4];
  if (a.cu_new && t >= a.cu_new[kv.n_seqs]) return;  // rows behind the last sequence stay as they are
  const int b = a.cu_new ? token_seq(a.cu_new, kv.n_seqs, t) : t;
  const int i = a.cu_new ? t - a.cu_new[b] : 0;
  const int64_t slot = (int64_t)a.seq_len[b] + i;
  int64_t page = -1;
  if (slot >= 0 && slot < ((int64_t)kv.max_pages << kv.page_shift)) page = paged_page(kv, b, (int)(slot >> kv.page_shift));
  if (page < 0 && c == 0) paged_err(kv, RTP_PAGED_ERANGE);
  const int off = (int)(slot & (kv.page_size - 1));
  const int pos = a.positions ? a.positions[t] : (int)slot;
  float cs, sn;
  rope_cos_sin(pos, a.theta[c], &cs, &sn);
  for (int h = 0; h < a.Hq + kv.Hkv; ++h) {
    const bool is_q = h < a.Hq;
    const T* x = is_q ? (const T*)a.q + t * a.q_stride + h * kv.D : (const T*)a.k + t * a.k_stride + (h - a.Hq) * kv.D;
    const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
    float x0 = to_f32(x[c]), x1 = to_f32(x[c + H]);
    if (w) {
      const float s = warp_sum(x0 * x0 + x1 * x1);
      __syncthreads();
      if ((c & 31) == 0) red[c >> 5] = s;
      __syncthreads();
      float tot = red[0];
      if (H > 32) tot += red[1];
      const float r = rsqrtf(tot / kv.D + a.eps);
      x0 = x0 * r * to_f32(w[c]);
      x1 = x1 * r * to_f32(w[c + H]);
    }
    const float y0 = x0 * cs - x1 * sn, y1 = x1 * cs + x0 * sn;
    if (is_q) {
      T* o = (T*)a.q_out + t * a.q_out_stride + h * kv.D;
      o[c] = from_f32<T>(y0);
      o[c + H] = from_f32<T>(y1);
    } else if (page >= 0) {
      const int g = h - a.Hq;
      K* o = (K*)(kv.k + page * kv.kp + g * kv.kh + off * kv.ks);
      K* ov = (K*)(kv.v + page * kv.vp + g * kv.vh + off * kv.vs);
      const T* xv = (const T*)a.v + t * a.v_stride + g * kv.D;
      o[c] = from_f32<K>(y0 / kv.k_scale);
      o[c + H] = from_f32<K>(y1 / kv.k_scale);
      ov[c] = from_f32<K>(to_f32(xv[c]) / kv.v_scale);
      ov[c + H] = from_f32<K>(to_f32(xv[c + H]) / kv.v_scale);
      if (c == 0 && a.slot_pos) a.slot_pos[((int64_t)b * kv.Hkv + g) * a.slot_pos_stride + slot] = pos;
    }
  }
}

// Bounds of page blockIdx.x of sequence blockIdx.z for KV head blockIdx.y over slots
// [first, last) of it; `widen`: from the stored bounds on unless slot 0 is among them.
template <typename K>
__device__ void bounds_of(const PagedView& kv, int b, int i, int g, int first, int last, bool widen) {
  const int d = threadIdx.x;
  const int64_t page = paged_page(kv, b, i);
  if (page < 0) {
    if (d == 0) paged_err(kv, RTP_PAGED_ERANGE);
    return;
  }
  K* o = (K*)kv.bounds + ((page * kv.Hkv + g) * 2) * kv.D;
  float lo = INFINITY, hi = -INFINITY;
  if (widen && first > 0) {
    lo = to_f32(o[d]);
    hi = to_f32(o[kv.D + d]);
  }
  const uint8_t* row = kv.k + page * kv.kp + g * kv.kh;
  for (int s = first; s < last; ++s) {
    const float x = to_f32(((const K*)(row + s * kv.ks))[d]);
    lo = fminf(lo, x);
    hi = fmaxf(hi, x);
  }
  o[d] = from_f32<K>(lo);
  o[kv.D + d] = from_f32<K>(hi);
}

template <typename K>
__global__ void append_bounds_kernel(const AppendArgs a) {
  const PagedView& kv = a.kv;
  const int b = blockIdx.z;
  const int n = a.cu_new ? a.cu_new[b + 1] - a.cu_new[b] : 1;
  const int64_t cap = (int64_t)kv.max_pages << kv.page_shift;
  const int64_t s0 = a.seq_len[b], s1 = min(s0 + n, cap);
  if (s0 < 0) return;
  const int64_t i = (s0 >> kv.page_shift) + blockIdx.x;
  const int64_t first = max(s0, i << kv.page_shift), last = min(s1, (i + 1) << kv.page_shift);
  if (first >= last) return;
  const int64_t base = i << kv.page_shift;
  bounds_of<K>(kv, b, (int)i, blockIdx.y, (int)(first - base), (int)(last - base), true);
}

template <typename K>
__global__ void bounds_kernel(const PagedView kv, const int32_t* seq_len) {
  const int b = blockIdx.z;
  int seq;
  const int n = paged_row(kv, nullptr, seq_len, b, &seq);
  if (blockIdx.x == 0 && threadIdx.x == 0 && paged_row_bad(kv, nullptr, seq_len, b)) paged_err(kv, RTP_PAGED_ERANGE);
  for (int i = blockIdx.x; ((int64_t)i << kv.page_shift) < n; i += gridDim.x)
    bounds_of<K>(kv, b, i, blockIdx.y, 0, min(kv.page_size, n - (i << kv.page_shift)), false);
}

template <typename T, typename K>
void run_append(const AppendArgs& a, cudaStream_t st) {
  append_kernel<T, K><<<a.n_tokens, a.kv.D / 2, 0, st>>>(a);
  if (a.kv.bounds) {
    const dim3 grid(a.max_new / a.kv.page_size + 2, a.kv.Hkv, a.kv.n_seqs);
    append_bounds_kernel<K><<<grid, a.kv.D, 0, st>>>(a);
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int io, int kvt, cudaStream_t st) {
  if (io == RTP_FP16 && kvt == RTP_FP16) run_append<__half, __half>(a, st);
  else if (io == RTP_BF16 && kvt == RTP_BF16) run_append<__nv_bfloat16, __nv_bfloat16>(a, st);
  else if (io == RTP_FP16) run_append<__half, __nv_fp8_e4m3>(a, st);
  else run_append<__nv_bfloat16, __nv_fp8_e4m3>(a, st);
  return cudaGetLastError();
}

cudaError_t launch_paged_bounds(const PagedView& kv, int kvt, const int32_t* seq_len, cudaStream_t st) {
  const dim3 grid(kv.max_pages < 1024 ? kv.max_pages : 1024, kv.Hkv, kv.n_seqs);
  if (kvt == RTP_FP16) bounds_kernel<__half><<<grid, kv.D, 0, st>>>(kv, seq_len);
  else if (kvt == RTP_BF16) bounds_kernel<__nv_bfloat16><<<grid, kv.D, 0, st>>>(kv, seq_len);
  else bounds_kernel<__nv_fp8_e4m3><<<grid, kv.D, 0, st>>>(kv, seq_len);
  return cudaGetLastError();
}

}  // namespace rtp
