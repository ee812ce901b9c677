// paged_decode.cu -- attention of new tokens over the pages of their sequences.
//
// One CTA per (row, query head), a warp per key: s = q . k in fp32, a running max and sum per
// warp, joined at the end.  Accumulated weights take a second pass over the keys with the joined
// log-sum-exp.
#include "paged.cuh"

namespace rtp {

namespace {

constexpr int kWarps = 8;

// Logical slot of the j-th attended key of a row, or -1.
struct Keys {
  const PagedView& kv;
  int seq, len, lo, sinks;  // dense: slots [0, sinks) and [lo, len)
  const int32_t* list;
  int n;  // keys to walk
  __device__ Keys(const DecodeArgs& a, int r, int g) : kv(a.kv) {
    len = paged_row(kv, a.row_seq, a.row_len, r, &seq);
    list = nullptr;
    if (a.sel) {
      list = a.sel + ((int64_t)r * kv.Hkv + g) * a.sel_stride;
      const int c = a.sel_count[(int64_t)r * kv.Hkv + g];
      n = (int)(c < 0 ? 0 : c > a.sel_stride ? a.sel_stride : c) << kv.page_shift;
      return;
    }
    lo = a.window && len > a.window ? len - a.window : 0;
    sinks = min(a.n_sink, lo);
    n = sinks + len - lo;
  }
  __device__ int slot(int j) const {
    if (!list) return j < sinks ? j : lo + j - sinks;
    const int i = list[j >> kv.page_shift];
    if (i < 0 || i >= kv.max_pages) return -1;
    const int s = (i << kv.page_shift) + (j & (kv.page_size - 1));
    return s < len ? s : -1;
  }
};

template <typename T, typename K>
__device__ float score(const DecodeArgs& a, const float* q, int64_t page, int g, int off) {
  const K* k = (const K*)(a.kv.k + page * a.kv.kp + g * a.kv.kh + off * a.kv.ks);
  float s = 0.f;
  for (int d = threadIdx.x & 31; d < a.kv.D; d += 32) s = fmaf(q[d], to_f32(k[d]), s);
  return warp_sum(s) * a.scale_log2;
}

template <typename T, typename K>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeArgs a, float* lse2) {
  const PagedView& kv = a.kv;
  const int h = blockIdx.x, r = blockIdx.y, g = h / a.group, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float q[kD], m_s[kWarps], l_s[kWarps], o_s[kWarps][kD];
  if (h == 0 && threadIdx.x == 0 && paged_row_bad(kv, a.row_seq, a.row_len, r)) paged_err(kv, RTP_PAGED_ERANGE);
  for (int d = threadIdx.x; d < kv.D; d += blockDim.x) q[d] = to_f32(((const T*)a.q)[r * a.q_stride + h * kv.D + d]);
  __syncthreads();
  const Keys keys(a, r, g);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = warp; j < keys.n; j += kWarps) {
    const int s = keys.slot(j);
    if (s < 0) continue;
    const int64_t page = paged_page(kv, keys.seq, s >> kv.page_shift);
    if (page < 0) {
      if (lane == 0) paged_err(kv, RTP_PAGED_ERANGE);
      continue;
    }
    const int off = s & (kv.page_size - 1);
    const float z = score<T, K>(a, q, page, g, off);
    const float mn = fmaxf(m, z);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - base), p = exp2f(z - base);
    m = mn;
    l = l * f + p;
    const K* v = (const K*)(kv.v + page * kv.vp + g * kv.vh + off * kv.vs);
    for (int e = 0; e < kv.D / 32; ++e) o[e] = o[e] * f + p * to_f32(v[e * 32 + lane]);
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  for (int e = 0; e < kv.D / 32; ++e) o_s[warp][e * 32 + lane] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w]);
  const float base = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kWarps; ++w) L += l_s[w] * exp2f(m_s[w] - base);
  for (int d = threadIdx.x; d < kv.D; d += blockDim.x) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += o_s[w][d] * exp2f(m_s[w] - base);
    ((T*)a.out)[r * a.out_stride + h * kv.D + d] = from_f32<T>(L == 0.f ? 0.f : x / L * kv.v_scale);
  }
  if (threadIdx.x == 0) {
    const float y = M + log2f(L);
    if (a.lse) a.lse[(int64_t)r * a.Hq + h] = L == 0.f ? -INFINITY : y * 0.6931471805599453f;
    if (lse2) lse2[(int64_t)r * a.Hq + h] = L == 0.f ? INFINITY : y;
  }
}

template <typename T, typename K>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const DecodeArgs a, const float* lse2) {
  const PagedView& kv = a.kv;
  const int g = blockIdx.y, r = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Keys keys(a, r, g);
  __shared__ float q[64 * kD];
  for (int i = threadIdx.x; i < a.group * kv.D; i += blockDim.x)
    q[i] = to_f32(((const T*)a.q)[r * a.q_stride + g * a.group * kv.D + i]);
  __syncthreads();
  for (int j = blockIdx.x * kWarps + warp; j < keys.n; j += gridDim.x * kWarps) {
    const int s = keys.slot(j);
    const int64_t page = paged_page(kv, keys.seq, s >> kv.page_shift);
    if (page < 0) continue;
    float w = 0.f;
    for (int u = 0; u < a.group; ++u)
      w += exp2f(score<T, K>(a, q + u * kv.D, page, g, s & (kv.page_size - 1)) -
                 lse2[(int64_t)r * a.Hq + g * a.group + u]);
    if (lane == 0) a.scores[((int64_t)r * kv.Hkv + g) * a.scores_stride + s] += w;
  }
}

template <typename T, typename K>
void run_decode(const DecodeArgs& a, cudaStream_t st) {
  float* lse2 = a.scores ? static_cast<float*>(a.workspace) : nullptr;
  decode_kernel<T, K><<<dim3(a.Hq, a.n_rows), kWarps * 32, 0, st>>>(a, lse2);
  if (a.scores) weights_kernel<T, K><<<dim3(64, a.kv.Hkv, a.n_rows), kWarps * 32, 0, st>>>(a, lse2);
}

}  // namespace

size_t paged_decode_workspace(const rtp_paged_kv*, int n_rows, int n_q_heads, bool) {
  return (size_t)n_rows * n_q_heads * sizeof(float);
}

cudaError_t launch_paged_decode(const DecodeArgs& a, const rtp_paged_kv* kv, int qt, cudaStream_t st) {
  const int kvt = kv->dtype;
  if (qt == RTP_FP16 && kvt == RTP_FP16) run_decode<__half, __half>(a, st);
  else if (qt == RTP_BF16 && kvt == RTP_BF16) run_decode<__nv_bfloat16, __nv_bfloat16>(a, st);
  else if (qt == RTP_FP16) run_decode<__half, __nv_fp8_e4m3>(a, st);
  else run_decode<__nv_bfloat16, __nv_fp8_e4m3>(a, st);
  return cudaGetLastError();
}

}  // namespace rtp
