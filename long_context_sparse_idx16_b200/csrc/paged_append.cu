// paged_append.cu -- head norms, rotation and the write of K and V rows to their pages.
//
// For each head row x of q and k (fp32, rounded once to the stored type):
//   y = x * rsqrt(mean(x^2) + eps) * weight,
//   z_c = y_c cos - y_{c+D/2} sin, z_{c+D/2} = y_{c+D/2} cos + y_c sin, angle = pos * theta_c.
// The angle is formed and reduced in fp64 (rope_cos_sin); the rest is fp32.
//
// Every row is read once and written once, so HBM bounds a chunk and launch latency a decode step.
// A warp takes one token and a run of its heads: the D/8 lanes of a row hold four dims of each half
// (the two members of four rotation pairs), so norm and rotation need no shared memory, and the
// sines and cosines stay in registers for all heads of the run.  The runs are as long as still
// leaves enough warps (the host picks), since every warp forms the angles again.
// One token per sequence: the K rows' warps also widen the page bounds.  In a chunk a page gets
// several rows: a second kernel takes its bounds from the rows just written (in L2).
#include "paged.cuh"

namespace rtp {

namespace {

constexpr int kWarps = 4;
constexpr int kUnroll = 4;  // row groups in flight per warp

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

template <typename T>
__device__ __forceinline__ void unpack4(uint2 u, float* f) {
  const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = to_f32(h[i]);
}

// Four values to 16 bits (8 bytes) or e4m3 (4 bytes).
template <typename K>
__device__ __forceinline__ void store4(void* at, const float* f) {
  if constexpr (sizeof(K) == 1) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
    *(uint32_t*)at = lo | hi << 16;
  } else {
    K h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = from_f32<K>(f[i]);
    *(uint2*)at = *reinterpret_cast<const uint2*>(h);
  }
}

template <typename K>
__device__ __forceinline__ void load4(const void* at, float* f) {
  if constexpr (sizeof(K) == 1) {
    const uint32_t u = *(const uint32_t*)at;
    const __nv_fp8_e4m3* h = reinterpret_cast<const __nv_fp8_e4m3*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = to_f32(h[i]);
  } else {
    unpack4<K>(*(const uint2*)at, f);
  }
}

// Units: heads 0 .. Hq-1 are q, then Hkv of k, then Hkv of v.  `run` units per warp.
template <typename T, typename K, int D>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendArgs a, int run, int runs, bool widen) {
  constexpr int L = D / 8;        // lanes of a row
  constexpr int R = 32 / L;       // rows a warp holds at once
  constexpr int H = D / 2;
  const PagedView& kv = a.kv;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(task / runs), lane = threadIdx.x & 31, sub = lane / L, c = (lane % L) * 4;
  if (t >= a.n_tokens) return;
  int b = t, i = 0;
  if (a.cu_new) {
    if (t >= a.cu_new[kv.n_seqs]) return;  // rows behind the last sequence stay as they are
    b = token_seq(a.cu_new, kv.n_seqs, t);
    i = t - a.cu_new[b];
  }
  const int u0 = (int)(task % runs) * run, units = a.Hq + 2 * kv.Hkv, u1 = min(u0 + run, units);
  const int64_t slot = (int64_t)a.seq_len[b] + i;
  const int pos = a.positions ? a.positions[t] : (int)slot;
  int64_t page = -1;
  if (u1 > a.Hq) {
    if (slot >= 0 && slot < ((int64_t)kv.max_pages << kv.page_shift))
      page = paged_page(kv, b, (int)(slot >> kv.page_shift));
    if (page < 0 && lane == 0) paged_err(kv, RTP_PAGED_ERANGE);
  }
  const int off = (int)(slot & (kv.page_size - 1));
  float cs[4], sn[4];
  if (u0 < a.Hq + kv.Hkv) {
#pragma unroll
    for (int e = 0; e < 4; ++e) rope_cos_sin(pos, a.theta[c + e], &cs[e], &sn[e]);
  }
  for (int v0 = u0; v0 < u1; v0 += R * kUnroll) {
    uint2 x[kUnroll][2];
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      const int u = v0 + n * R + sub;
      if (u < u1) {
        const T* p = u < a.Hq            ? (const T*)a.q + t * a.q_stride + (int64_t)u * D
                     : u < a.Hq + kv.Hkv ? (const T*)a.k + t * a.k_stride + (int64_t)(u - a.Hq) * D
                                         : (const T*)a.v + t * a.v_stride + (int64_t)(u - a.Hq - kv.Hkv) * D;
        x[n][0] = *(const uint2*)(p + c);
        x[n][1] = *(const uint2*)(p + H + c);
      } else {
        x[n][0] = x[n][1] = make_uint2(0u, 0u);
      }
    }
#pragma unroll
    for (int n = 0; n < kUnroll; ++n) {
      const int u = v0 + n * R + sub;
      const bool is_q = u < a.Hq, is_v = u >= a.Hq + kv.Hkv;
      float y[8];
      unpack4<T>(x[n][0], y);
      unpack4<T>(x[n][1], y + 4);
      const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(y[e], y[e], s);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (u >= u1) continue;
      if (!is_v) {
        if (w) {
          const float r = rsqrtf(s * (1.f / D) + a.eps);
          float g[8];
          unpack4<T>(*(const uint2*)(w + c), g);
          unpack4<T>(*(const uint2*)(w + H + c), g + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = y[e] * r * g[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y0 = y[e], y1 = y[e + 4];
          y[e] = y0 * cs[e] - y1 * sn[e];
          y[e + 4] = y1 * cs[e] + y0 * sn[e];
        }
      }
      if (is_q) {
        T* o = (T*)a.q_out + t * a.q_out_stride + (int64_t)u * D;
        store4<T>(o + c, y);
        store4<T>(o + H + c, y + 4);
      } else if (page >= 0) {
        const int g = u - a.Hq - (is_v ? kv.Hkv : 0);
        K* o = (K*)(is_v ? kv.v + page * kv.vp + g * kv.vh + off * kv.vs : kv.k + page * kv.kp + g * kv.kh + off * kv.ks);
        const float f = is_v ? kv.v_scale : kv.k_scale;
        if (f != 1.f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = y[e] / f;
        }
        store4<K>(o + c, y);
        store4<K>(o + H + c, y + 4);
        if (!is_v) {
          if (c == 0 && a.slot_pos) a.slot_pos[((int64_t)b * kv.Hkv + g) * a.slot_pos_stride + slot] = pos;
          if (widen) {  // the page's only new row
            K* lim = (K*)kv.bounds + ((page * kv.Hkv + g) * 2) * D;
            float lo[8], hi[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = to_f32(from_f32<K>(y[e]));  // the key as it was stored
            if (off > 0) {
              load4<K>(lim + c, lo);
              load4<K>(lim + H + c, lo + 4);
              load4<K>(lim + D + c, hi);
              load4<K>(lim + D + H + c, hi + 4);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              lo[e] = fminf(off > 0 ? lo[e] : INFINITY, y[e]);
              hi[e] = fmaxf(off > 0 ? hi[e] : -INFINITY, y[e]);
            }
            store4<K>(lim + c, lo);
            store4<K>(lim + H + c, lo + 4);
            store4<K>(lim + D + c, hi);
            store4<K>(lim + D + H + c, hi + 4);
          }
        }
      }
    }
  }
}

// Bounds of page `i` of sequence b for KV head g over slots [first, last) of it, by one warp-sized
// group of rows: lanes hold four dims each, the CTA's row groups take every R-th slot.  `widen`:
// from the stored bounds on, unless slot 0 is among them.
constexpr int kBoundThreads = 128;

template <typename K, int D>
__device__ void bounds_of(const PagedView& kv, int b, int i, int g, int first, int last, bool widen,
                          float (*sh)[2][D]) {
  constexpr int L = D / 4;                 // lanes of a row
  constexpr int R = kBoundThreads / L;     // rows at once
  const int c = (threadIdx.x % L) * 4, r = threadIdx.x / L;
  const int64_t page = paged_page(kv, b, i);
  if (page < 0) {
    if (threadIdx.x == 0) paged_err(kv, RTP_PAGED_ERANGE);
    return;
  }
  K* o = (K*)kv.bounds + ((page * kv.Hkv + g) * 2) * D;
  float lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
  if (widen && first > 0 && r == 0) {
    load4<K>(o + c, lo);
    load4<K>(o + D + c, hi);
  }
  const uint8_t* row = kv.k + page * kv.kp + g * kv.kh;
#pragma unroll 4
  for (int s = first + r; s < last; s += R) {
    float x[4];
    load4<K>((const K*)(row + s * kv.ks) + c, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = fminf(lo[e], x[e]);
      hi[e] = fmaxf(hi[e], x[e]);
    }
  }
  __syncthreads();  // the last page's exchange has been read
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    sh[r][0][c + e] = lo[e];
    sh[r][1][c + e] = hi[e];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < 2 * D; x += kBoundThreads) {
    float y = sh[0][x / D][x % D];
#pragma unroll
    for (int n = 1; n < R; ++n) y = x < D ? fminf(y, sh[n][0][x]) : fmaxf(y, sh[n][1][x - D]);
    o[x] = from_f32<K>(y);
  }
}

template <typename K, int D>
__global__ void __launch_bounds__(kBoundThreads) append_bounds_kernel(const AppendArgs a) {
  __shared__ float sh[kBoundThreads * 4 / D][2][D];
  const PagedView& kv = a.kv;
  const int b = blockIdx.z;
  const int n = a.cu_new[b + 1] - a.cu_new[b];
  const int64_t cap = (int64_t)kv.max_pages << kv.page_shift;
  const int64_t s0 = a.seq_len[b], s1 = min(s0 + n, cap);
  if (s0 < 0) return;
  const int64_t i = (s0 >> kv.page_shift) + blockIdx.x;
  const int64_t first = max(s0, i << kv.page_shift), last = min(s1, (i + 1) << kv.page_shift);
  if (first >= last) return;
  const int64_t base = i << kv.page_shift;
  bounds_of<K, D>(kv, b, (int)i, blockIdx.y, (int)(first - base), (int)(last - base), true, sh);
}

template <typename K, int D>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const PagedView kv, const int32_t* seq_len) {
  __shared__ float sh[kBoundThreads * 4 / D][2][D];
  const int b = blockIdx.z;
  int seq;
  const int n = paged_row(kv, nullptr, seq_len, b, &seq);
  if (blockIdx.x == 0 && threadIdx.x == 0 && paged_row_bad(kv, nullptr, seq_len, b)) paged_err(kv, RTP_PAGED_ERANGE);
  for (int i = blockIdx.x; ((int64_t)i << kv.page_shift) < n; i += gridDim.x)
    bounds_of<K, D>(kv, b, i, blockIdx.y, 0, min(kv.page_size, n - (i << kv.page_shift)), false, sh);
}

// Units per warp: all of a token's in a large chunk (one set of angles per token), fewer while the
// warps would not fill the GPU (64 warps on each of 148 SMs), but no less than a warp holds at once.
int units_per_warp(int64_t tokens, int units, int at_once) {
  const int64_t want = 148 * 64;
  int run = units;
  while (run > at_once && tokens * ((units + run - 1) / run) < want) run = (run + 1) / 2;
  return (run + at_once - 1) / at_once * at_once;
}

template <typename T, typename K, int D>
cudaError_t run_append(const AppendArgs& a, cudaStream_t st) {
  const int units = a.Hq + 2 * a.kv.Hkv, run = units_per_warp(a.n_tokens, units, 256 / D);
  const int runs = (units + run - 1) / run;
  const int64_t warps = (int64_t)a.n_tokens * runs;
  const bool one = !a.cu_new && a.kv.bounds;
  append_kernel<T, K, D><<<(unsigned)((warps + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a, run, runs, one);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.kv.bounds || one) return e;
  const dim3 grid(a.max_new / a.kv.page_size + 2, a.kv.Hkv, a.kv.n_seqs);
  append_bounds_kernel<K, D><<<grid, kBoundThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, typename K>
cudaError_t run_append_d(const AppendArgs& a, cudaStream_t st) {
  return a.kv.D == 64 ? run_append<T, K, 64>(a, st) : run_append<T, K, 128>(a, st);
}

template <typename K>
cudaError_t run_bounds(const PagedView& kv, const int32_t* seq_len, cudaStream_t st) {
  const dim3 grid(kv.max_pages < 1024 ? kv.max_pages : 1024, kv.Hkv, kv.n_seqs);
  if (kv.D == 64) bounds_kernel<K, 64><<<grid, kBoundThreads, 0, st>>>(kv, seq_len);
  else bounds_kernel<K, 128><<<grid, kBoundThreads, 0, st>>>(kv, seq_len);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, int io, int kvt, cudaStream_t st) {
  if (io == RTP_FP16 && kvt == RTP_FP16) return run_append_d<__half, __half>(a, st);
  if (io == RTP_BF16 && kvt == RTP_BF16) return run_append_d<__nv_bfloat16, __nv_bfloat16>(a, st);
  if (io == RTP_FP16) return run_append_d<__half, __nv_fp8_e4m3>(a, st);
  return run_append_d<__nv_bfloat16, __nv_fp8_e4m3>(a, st);
}

cudaError_t launch_paged_bounds(const PagedView& kv, int kvt, const int32_t* seq_len, cudaStream_t st) {
  if (kvt == RTP_FP16) return run_bounds<__half>(kv, seq_len, st);
  if (kvt == RTP_BF16) return run_bounds<__nv_bfloat16>(kv, seq_len, st);
  return run_bounds<__nv_fp8_e4m3>(kv, seq_len, st);
}

}  // namespace rtp
