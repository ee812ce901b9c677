// paged_append.cu -- head norms, rotation and the write of K and V rows to their pages.
//
// For each head row x of q and k (fp32, rounded once to the stored type):
//   y = x * rsqrt(mean(x^2) + eps) * weight,
//   z_c = y_c cos - y_{c+D/2} sin, z_{c+D/2} = y_{c+D/2} cos + y_c sin, angle = pos * theta_c.
// The angle is formed and reduced in fp64 (rope_cos_sin); the rest is fp32.
//
// Every row is read once and written once, so HBM bounds a chunk and launch latency a decode step;
// what stands between is instructions.  A warp takes one token and a run of its row groups (as many
// rows as it holds at once, all of q, of k or of v).  A lane holds eight dims of each half of a row,
// the two members of eight rotation pairs: 16-byte loads and stores, norm and rotation without
// shared memory, two fp32 values an instruction (fma.f32x2).  The sines and cosines are formed once
// per warp, shared out over the lanes that need the same ones.  The runs are as long as still leaves
// enough warps to fill the GPU (the host picks), since every warp forms the angles again.
// One token per sequence: the K rows' warps also widen the page bounds.  In a chunk a page gets
// several rows: a second kernel takes its bounds from the rows just written (in L2: the other rows are
// read and written as streams).
//
// Measured (one B200, 32 / 4 heads of 128, bf16, norms, bounds): 16384 tokens, 336 MB, in 70.6 us (4.8
// TB/s); on inputs already in L2 65.6 us, 60.7 us of it this kernel; 64 tokens in 4 us.  Four dims
// a lane instead of eight took 134 us (54.8 M warp instructions instead of 35.8 M).
#include "paged.cuh"

namespace rtp {

namespace {

constexpr int kWarps = 4;

// ---- two fp32 values in one register pair

using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack(f2 r, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 16-bit pair to fp32 pair
template <typename T>
__device__ __forceinline__ f2 widen(uint32_t u) {
  if constexpr (std::is_same_v<T, __half>) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    return pack(f.x, f.y);
  } else {
    return pack(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ void widen8(uint4 u, f2* y) {
  y[0] = widen<T>(u.x);
  y[1] = widen<T>(u.y);
  y[2] = widen<T>(u.z);
  y[3] = widen<T>(u.w);
}

// Eight values to K: 16 bytes of 16-bit values, or 8 of e4m3 (nearest, saturating).
template <typename K>
struct Pack8;
template <>
struct Pack8<__nv_fp8_e4m3> {
  using type = uint2;
  static __device__ __forceinline__ uint2 of(const f2* y) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      unpack(y[i], f.x, f.y);
      w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
};
template <typename T>
struct Pack8 {
  using type = uint4;
  static __device__ __forceinline__ uint4 of(const f2* y) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpack(y[i], a, b);
      w[i] = pack2<T>(a, b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Least and greatest of stored values, eight at a time, as 16-bit pairs (e4m3: as fp16, exactly).
// A NaN yields to the other value.
template <typename K>
struct Range8 {
  using T = std::conditional_t<sizeof(K) == 1, __half, K>;
  using Raw = typename Pack8<K>::type;
  using V2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
  uint32_t lo[4], hi[4];
  static __device__ __forceinline__ V2 v(uint32_t x) { return *reinterpret_cast<V2*>(&x); }
  static __device__ __forceinline__ uint32_t u(V2 x) { return *reinterpret_cast<uint32_t*>(&x); }
  static __device__ __forceinline__ void wide(Raw r, uint32_t* w) {
    if constexpr (sizeof(K) == 1) {
      w[0] = widen2<T>(r.x);
      w[1] = widen2<T>(r.x >> 16);
      w[2] = widen2<T>(r.y);
      w[3] = widen2<T>(r.y >> 16);
    } else {
      w[0] = r.x;
      w[1] = r.y;
      w[2] = r.z;
      w[3] = r.w;
    }
  }
  static __device__ __forceinline__ Raw narrow(const uint32_t* w) {
    if constexpr (sizeof(K) == 1) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2_raw x = *reinterpret_cast<const __half2_raw*>(&w[i]);
        h[i] = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
      }
      return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    } else {
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void none() {
    const uint32_t inf = std::is_same_v<T, __half> ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = inf;
      hi[i] = inf | 0x80008000u;
    }
  }
  __device__ __forceinline__ void add(const uint32_t* l, const uint32_t* h) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = u(__hmin2(v(lo[i]), v(l[i])));
      hi[i] = u(__hmax2(v(hi[i]), v(h[i])));
    }
  }
  __device__ __forceinline__ void row(Raw r) {
    uint32_t w[4];
    wide(r, w);
    add(w, w);
  }
  // the stored bounds, D values apart
  __device__ __forceinline__ void stored(const K* p, int D) {
    uint32_t l[4], h[4];
    wide(*(const Raw*)p, l);
    wide(*(const Raw*)(p + D), h);
    add(l, h);
  }
  __device__ __forceinline__ void store(K* p, int D) const {
    *(Raw*)p = narrow(lo);
    *(Raw*)(p + D) = narrow(hi);
  }
};

// Sequence of token t: the last b with cu[b] <= t, or -1 if no sequence names row t.  A warp looks at
// 32 places at a time.  *first: cu[b].
__device__ __forceinline__ int token_seq(const int32_t* cu, int n_seqs, int t, int* first) {
  int lo = 0, n = n_seqs + 1;  // the answer lies in [lo, lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32, at = lo + (threadIdx.x & 31) * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at <= n_seqs && cu[min(at, n_seqs)] <= t);
    const int k = 31 - __clz(le | 1u);
    n = min(step, lo + n - (lo + k * step));
    lo += k * step;
  }
  const int c = cu[min(lo + (int)(threadIdx.x & 31), n_seqs)];
  const uint32_t le = __ballot_sync(0xffffffffu, (threadIdx.x & 31) < n && c <= t);
  const int k = 31 - __clz(le | 1u);
  *first = __shfl_sync(0xffffffffu, c, k);
  return (le & 1u) && lo + k < n_seqs ? lo + k : -1;
}

// Offsets that begin elsewhere than at 0, descend or name more rows than there are; by one CTA.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int n_seqs, int n_tokens, uint32_t* err) {
  bool bad = threadIdx.x == 0 && (cu[0] != 0 || cu[n_seqs] > n_tokens);
#pragma unroll 4
  for (int e = threadIdx.x; e < n_seqs; e += 32 * kWarps) bad |= cu[e] > cu[e + 1];
  if (bad && err) atomicOr(err, RTP_PAGED_ERANGE);
}

// Row groups of a token: ceil(Hq / R) of q, then ceil(Hkv / R) of k, then as many of v; `run` of them
// per warp.  U groups are in flight at once: two where a warp has several (16384 tokens: 72 us, one
// 85 us, four 82 us, for want of registers), one where it has one.
template <typename T, typename K, int D, int U>
__global__ void __launch_bounds__(32 * kWarps, 5) append_kernel(const AppendArgs a, int run, int runs, bool widen_bounds) {
  constexpr int L = D / 16;       // lanes of a row
  constexpr int R = 32 / L;       // rows a warp holds at once
  constexpr int H = D / 2;
  const PagedView& kv = a.kv;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(task / runs), lane = threadIdx.x & 31, sub = lane / L, c = (lane % L) * 8;
  after_wait();
  // (a CTA behind those of the tokens: inside theirs the test costs registers, and 2% of a large chunk)
  if (a.cu_new && blockIdx.x == gridDim.x - 1) return check_offsets(a.cu_new, kv.n_seqs, a.n_tokens, kv.err);
  if (t >= a.n_tokens) return;
  int b = t, i = 0;
  if (a.cu_new) {
    b = token_seq(a.cu_new, kv.n_seqs, t, &i);
    if (b < 0) return;  // rows before the first sequence and behind the last stay as they are
    i = t - i;
  }
  const int gq = (a.Hq + R - 1) / R, gk = (kv.Hkv + R - 1) / R;
  const int u0 = (int)(task % runs) * run, u1 = min(u0 + run, gq + 2 * gk);
  const auto load = [&](int u, uint4* x) {
    const bool is_q = u < gq, is_v = u >= gq + gk;
    const int h = (u - (is_q ? 0 : is_v ? gq + gk : gq)) * R + sub;
    const T* p = (is_q ? (const T*)a.q + t * a.q_stride : is_v ? (const T*)a.v + t * a.v_stride : (const T*)a.k + t * a.k_stride) +
                 (int64_t)h * D + c;
    x[0] = x[1] = make_uint4(0u, 0u, 0u, 0u);
    if (u < u1 && h < (is_q ? a.Hq : kv.Hkv)) {
      x[0] = __ldcs((const uint4*)p);
      x[1] = __ldcs((const uint4*)(p + H));
    }
  };
  uint4 x[U][2];
#pragma unroll
  for (int n = 0; n < U; ++n) load(u0 + n, x[n]);
  const int start = a.seq_len[b];
  const int64_t slot = (int64_t)start + i;
  const int pos = a.positions ? a.positions[t] : (int)slot;
  int64_t page = -1;
  if (u1 > gq) {
    // (a negative length takes out all of its sequence: tokens behind it would land on older ones; i is
    // negative where an offset so far below 0 overflows it)
    if ((start | i) >= 0 && slot < ((int64_t)kv.max_pages << kv.page_shift))
      page = paged_page(kv, b, (int)(slot >> kv.page_shift));
    if (page < 0 && lane == 0) paged_err(kv, RTP_PAGED_ERANGE);
  }
  const int off = (int)(slot & (kv.page_size - 1));
  // this lane's eight angles: the R lanes of equal c form 8 / R of them each
  f2 cs[4], sn[4], wt[2][4];
  if (u0 < gq + gk) {
    constexpr int N = 8 / R > 0 ? 8 / R : 1;
    float cc[N], ss[N];
#pragma unroll
    for (int e = 0; e < N; ++e) rope_cos_sin(pos, a.theta[c + (sub * N + e) % 8], &cc[e], &ss[e]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int s0 = (2 * e) / N, s1 = (2 * e + 1) / N;
      cs[e] = pack(__shfl_sync(0xffffffffu, cc[(2 * e) % N], s0 * L + lane % L),
                   __shfl_sync(0xffffffffu, cc[(2 * e + 1) % N], s1 * L + lane % L));
      sn[e] = pack(__shfl_sync(0xffffffffu, ss[(2 * e) % N], s0 * L + lane % L),
                   __shfl_sync(0xffffffffu, ss[(2 * e + 1) % N], s1 * L + lane % L));
    }
  }
  const void* have = nullptr;  // the weights in wt
#pragma unroll 1
  for (int v0 = u0; v0 < u1; v0 += U) {
    uint4 y[U][2];
#pragma unroll
    for (int n = 0; n < U; ++n) {
      y[n][0] = x[n][0];
      y[n][1] = x[n][1];
    }
    if (v0 + U < u1) {
#pragma unroll
      for (int n = 0; n < U; ++n) load(v0 + U + n, x[n]);
    }
#pragma unroll
    for (int n = 0; n < U; ++n) {
      const int u = v0 + n;
      if (u >= u1) break;  // the whole warp alike
      const bool is_q = u < gq, is_v = u >= gq + gk;
      const int h = (u - (is_q ? 0 : is_v ? gq + gk : gq)) * R + sub;
      f2 z[2][4];
      widen8<T>(y[n][0], z[0]);
      widen8<T>(y[n][1], z[1]);
      if (!is_v) {
        const T* w = (const T*)(is_q ? a.q_weight : a.k_weight);
        if (w) {
          f2 s2 = mul2(z[0][0], z[0][0]);
#pragma unroll
          for (int e = 1; e < 8; ++e) s2 = fma2(z[e >> 2][e & 3], z[e >> 2][e & 3], s2);
          float s, s1;
          unpack(s2, s, s1);
          s += s1;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          const float r = rsqrtf(s * (1.f / D) + a.eps);
          const f2 r2 = pack(r, r);
          if (w != have) {
            widen8<T>(*(const uint4*)(w + c), wt[0]);
            widen8<T>(*(const uint4*)(w + H + c), wt[1]);
            have = w;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e >> 2][e & 3] = mul2(mul2(z[e >> 2][e & 3], r2), wt[e >> 2][e & 3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 z0 = z[0][e], z1 = z[1][e];
          float n0, n1;
          unpack(mul2(z1, sn[e]), n0, n1);
          z[0][e] = fma2(z0, cs[e], pack(-n0, -n1));
          z[1][e] = fma2(z1, cs[e], mul2(z0, sn[e]));
        }
      }
      if (h >= (is_q ? a.Hq : kv.Hkv)) continue;
      if (is_q) {
        T* o = (T*)a.q_out + t * a.q_out_stride + (int64_t)h * D + c;
        __stcs((uint4*)o, Pack8<T>::of(z[0]));
        __stcs((uint4*)(o + H), Pack8<T>::of(z[1]));
      } else if (page >= 0) {
        K* o = (K*)(is_v ? kv.v + page * kv.vp + h * kv.vh + off * kv.vs : kv.k + page * kv.kp + h * kv.kh + off * kv.ks) + c;
        const float f = is_v ? kv.v_scale : kv.k_scale;
        if (f != 1.f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float p, q;
            unpack(z[e >> 2][e & 3], p, q);
            z[e >> 2][e & 3] = pack(p / f, q / f);
          }
        }
        const auto k0 = Pack8<K>::of(z[0]), k1 = Pack8<K>::of(z[1]);
        using Raw = typename Pack8<K>::type;
        *(Raw*)o = k0;
        *(Raw*)(o + H) = k1;
        if (!is_v) {
          if (c == 0 && a.slot_pos) a.slot_pos[((int64_t)b * kv.Hkv + h) * a.slot_pos_stride + slot] = pos;
          if (widen_bounds) {  // the page's only new row
            K* lim = (K*)kv.bounds + ((page * kv.Hkv + h) * 2) * D + c;
            Range8<K> r0, r1;
            r0.none();
            r1.none();
            if (off > 0) {
              r0.stored(lim, D);
              r1.stored(lim + H, D);
            }
            r0.row(k0);
            r1.row(k1);
            r0.store(lim, D);
            r1.store(lim + H, D);
          }
        }
      }
    }
  }
}

// Bounds of page `i` of sequence b for KV head g over slots [first, last) of it: lanes hold eight
// dims each, the CTA's row groups take every R-th slot.  `widen` (behind the append kernel): from the
// stored bounds on, unless slot 0 is among them.
constexpr int kBoundThreads = 128;

template <typename K, int D>
__device__ void bounds_of(const PagedView& kv, int b, int i, int g, int first, int last, bool widen,
                          uint32_t (*sh)[2][D / 2]) {
  constexpr int L = D / 8;                 // lanes of a row
  constexpr int R = kBoundThreads / L;     // rows at once: 8 or 16
  using Raw = typename Pack8<K>::type;
  const int c = (threadIdx.x % L) * 8, r = threadIdx.x / L;
  const int64_t page = paged_page(kv, b, i);
  if (widen) after_wait();
  if (page < 0) {
    if (threadIdx.x == 0) paged_err(kv, RTP_PAGED_ERANGE);
    return;
  }
  K* o = (K*)kv.bounds + ((page * kv.Hkv + g) * 2) * D + c;
  Range8<K> m;
  m.none();
  if (widen && first > 0 && r == 0) m.stored(o, D);
  const uint8_t* row = kv.k + page * kv.kp + g * kv.kh;
#pragma unroll 8
  for (int s = first + r; s < last; s += R) m.row(*(const Raw*)((const K*)(row + s * kv.ks) + c));
  __syncthreads();  // the last page's exchange has been read
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    sh[r][0][c / 2 + e] = m.lo[e];
    sh[r][1][c / 2 + e] = m.hi[e];
  }
  __syncthreads();
  if (r == 0) {
#pragma unroll
    for (int n = 1; n < R; ++n) m.add(&sh[n][0][c / 2], &sh[n][1][c / 2]);
    m.store(o, D);
  }
}

template <typename K, int D>
__global__ void __launch_bounds__(kBoundThreads) append_bounds_kernel(const AppendArgs a) {
  __shared__ uint32_t sh[kBoundThreads * 8 / D][2][D / 2];
  const PagedView& kv = a.kv;
  const int b = blockIdx.z;
  // (the lengths and the table are inputs of the whole operator: read ahead)
  const int64_t cap = (int64_t)kv.max_pages << kv.page_shift, start = a.seq_len[b];
  // the slots of the rows that were given
  const int64_t row0 = a.cu_new[b], row1 = a.cu_new[b + 1];
  const int64_t s0 = start + max(row0, (int64_t)0) - row0, s1 = min(start + min(row1, (int64_t)a.n_tokens) - row0, cap);
  if (start < 0 || s0 >= s1) return after_wait();
  bool waited = false;
  for (int64_t i = (s0 >> kv.page_shift) + blockIdx.x; i << kv.page_shift < s1; i += gridDim.x) {
    const int64_t base = i << kv.page_shift, first = max(s0, base), last = min(s1, base + kv.page_size);
    bounds_of<K, D>(kv, b, (int)i, blockIdx.y, (int)(first - base), (int)(last - base), true, sh);
    waited = true;
  }
  if (!waited) after_wait();
}

template <typename K, int D>
__global__ void __launch_bounds__(kBoundThreads) bounds_kernel(const PagedView kv, const int32_t* seq_len) {
  __shared__ uint32_t sh[kBoundThreads * 8 / D][2][D / 2];
  after_wait();
  const int b = blockIdx.z;
  int seq;
  const int n = paged_row(kv, nullptr, seq_len, b, &seq);
  if (blockIdx.x == 0 && threadIdx.x == 0 && paged_row_bad(kv, nullptr, seq_len, b)) paged_err(kv, RTP_PAGED_ERANGE);
  for (int i = blockIdx.x; ((int64_t)i << kv.page_shift) < n; i += gridDim.x)
    bounds_of<K, D>(kv, b, i, blockIdx.y, 0, min(kv.page_size, n - (i << kv.page_shift)), false, sh);
}

// Row groups per warp: all of a token's in a large chunk (one set of angles per token), fewer while
// the warps would not fill the GPU (16 on each of 148 SMs).
int groups_per_warp(int64_t tokens, int groups) {
  int run = groups;
  while (run > 1 && tokens * ((groups + run - 1) / run) < 148 * 16) run = (run + 1) / 2;
  return run;
}

template <typename T, typename K, int D>
cudaError_t run_append(const AppendArgs& a, cudaStream_t st) {
  constexpr int R = 512 / D;
  const int groups = (a.Hq + R - 1) / R + 2 * ((a.kv.Hkv + R - 1) / R), run = groups_per_warp(a.n_tokens, groups);
  const int runs = (groups + run - 1) / run;
  const int64_t warps = (int64_t)a.n_tokens * runs;
  const bool one = !a.cu_new && a.kv.bounds;
  const dim3 grid((unsigned)((warps + kWarps - 1) / kWarps + (a.cu_new ? 1 : 0)));
  const cudaError_t e = run == 1 ? launch_after(append_kernel<T, K, D, 1>, grid, 32 * kWarps, 0, st, a, run, runs, one)
                                 : launch_after(append_kernel<T, K, D, 2>, grid, 32 * kWarps, 0, st, a, run, runs, one);
  if (e != cudaSuccess || !a.kv.bounds || one) return e;
  const dim3 pages(a.max_new / a.kv.page_size + 2, a.kv.Hkv, a.kv.n_seqs);
  return launch_after(append_bounds_kernel<K, D>, pages, kBoundThreads, 0, st, a);
}

template <typename T, typename K>
cudaError_t run_append_d(const AppendArgs& a, cudaStream_t st) {
  return a.kv.D == 64 ? run_append<T, K, 64>(a, st) : run_append<T, K, 128>(a, st);
}

template <typename K>
cudaError_t run_bounds(const PagedView& kv, const int32_t* seq_len, cudaStream_t st) {
  const dim3 grid(kv.max_pages < 1024 ? kv.max_pages : 1024, kv.Hkv, kv.n_seqs);
  if (kv.D == 64) return launch_after(bounds_kernel<K, 64>, grid, kBoundThreads, 0, st, kv, seq_len);
  return launch_after(bounds_kernel<K, 128>, grid, kBoundThreads, 0, st, kv, seq_len);
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
