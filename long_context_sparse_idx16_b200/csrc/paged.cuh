// paged.cuh -- shared pieces of the paged-cache operators (paged_*.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <string>
#include <type_traits>

#include "mma_tile.cuh"
#include "rtp_device.cuh"
#include "rtp_internal.h"
#include "rtp_paged.h"

namespace rtp {

// What the kernels need of an rtp_paged_kv, by value.  Strides in bytes.
struct PagedView {
  uint8_t* k;
  uint8_t* v;
  int64_t kp, kh, ks;  // page, head, slot strides
  int64_t vp, vh, vs;
  int64_t n_pages;
  int page_size, page_shift, Hkv, D;
  int max_pages, n_seqs;
  const int32_t* table;
  int64_t table_stride;
  float k_scale, v_scale;
  uint8_t* bounds;
  uint32_t* err;
};

// A kernel launched by launch_after may start while the one before it drains, and waits here until
// that one has finished and its writes can be seen.  Only then does it let the next one start: when
// a kernel starts, all work before its predecessor is done, so the second and later kernels of an
// operator may read the operator's inputs before they wait (but nothing that the predecessor
// writes).  The first kernel of an operator waits before it touches global memory.
__device__ __forceinline__ void after_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

__device__ __forceinline__ void paged_err(const PagedView& p, uint32_t bit) {
  if (p.err) atomicOr(p.err, bit);
}

// Length of a row's cache, brought into [0, max_pages * page_size]; 0 for a sequence number
// outside the batch.
__device__ __forceinline__ int paged_row(const PagedView& p, const int32_t* row_seq, const int32_t* row_len, int r,
                                         int* seq) {
  const int b = row_seq ? row_seq[r] : r;
  const int n = row_len[r];
  *seq = b;
  if ((unsigned)b >= (unsigned)p.n_seqs) {
    *seq = 0;
    return 0;
  }
  const int64_t cap = (int64_t)p.max_pages << p.page_shift;
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}

__device__ __forceinline__ bool paged_row_bad(const PagedView& p, const int32_t* row_seq, const int32_t* row_len,
                                              int r) {
  const int b = row_seq ? row_seq[r] : r;
  const int n = row_len[r];
  return (unsigned)b >= (unsigned)p.n_seqs || n < 0 || n > ((int64_t)p.max_pages << p.page_shift);
}

// Pool page of page `i` of sequence b, or -1 if the table holds a number outside the pool.
__device__ __forceinline__ int64_t paged_page(const PagedView& p, int b, int i) {
  const int32_t g = p.table[(int64_t)b * p.table_stride + i];
  return (uint32_t)g < (uint64_t)p.n_pages ? (int64_t)g : -1;
}

__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__nv_fp8_e4m3 x) { return (float)x; }

// ---- products on the tensor cores, fp16 or bf16 operands

template <typename T>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same_v<T, __half>)
    mma16816(c, a, b0, b1);
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (std::is_same_v<T, __half>) return pack_half2(x, y);
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// two e4m3 values (low 16 bits) as two T, exactly
template <typename T>
__device__ __forceinline__ uint32_t widen2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3);
  const __half2 y = *reinterpret_cast<const __half2*>(&h);
  if constexpr (std::is_same_v<T, __half>) return *reinterpret_cast<const uint32_t*>(&y);
  const float2 f = __half22float2(y);
  return pack2<T>(f.x, f.y);
}

// Order-preserving map of a double to 64 bits: equal values (0 and -0 among them) get equal keys,
// NaN gets 0, below -inf.
__device__ __forceinline__ unsigned long long order_key64(double x) {
  if (x != x) return 0ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// The k-th largest (1 <= k <= n) of n 64-bit keys, found by one CTA in 8-bit digits from the top.
// Returns a threshold T and in *ties how many of the keys equal to T belong to the first k: keys
// above T all do.  hist: 257 words of shared memory.  Stops as soon as a digit's bin is taken whole.
template <typename KeyFn>
__device__ unsigned long long block_kth_largest(int n, int k, uint32_t* hist, int* ties, KeyFn key) {
  unsigned long long prefix = 0;
  int want = k;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 257; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const unsigned long long x = key(i);
      if (shift == 56 || (x >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(x >> shift) & 255], 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane l holds bins 255 - 8 l ... 248 - 8 l, in falling order
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - 8 * threadIdx.x - e];
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, before, o);
        if (threadIdx.x >= o) before += y;
      }
      before -= sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (before < (uint32_t)want && before + c[e] >= (uint32_t)want)
          hist[256] = (uint32_t)(255 - 8 * threadIdx.x - e) << 16 | (before + c[e] == (uint32_t)want ? 1u : 0u);
        before += c[e];
      }
    }
    __syncthreads();
    const uint32_t found = hist[256];
    const int bin = (int)(found >> 16);
    for (int e = 255; e > bin; --e) want -= (int)hist[e];
    prefix |= (unsigned long long)bin << shift;
    __syncthreads();
    if (found & 1u) {
      // every key of the bin belongs: all keys >= prefix do
      *ties = 0x7fffffff;
      return prefix;
    }
  }
  *ties = want;
  return prefix;
}

// Exclusive prefix sum over the CTA of one int per thread (blockDim.x a multiple of 32, at most
// 1024).  warp_sums: 33 ints of shared memory; *total receives the sum.
__device__ __forceinline__ int block_exclusive(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < nw ? warp_sums[lane] : 0;
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += z;
    }
    if (lane < nw) warp_sums[lane] = s - w;
    if (lane == 31) warp_sums[32] = s;
  }
  __syncthreads();
  *total = warp_sums[32];
  return warp_sums[warp] + y - x;
}

// ---- host: checked arguments of the launches

struct AppendArgs {
  PagedView kv;
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements
  int n_tokens, Hq, max_new;
  const int32_t* cu_new;
  const int32_t* seq_len;
  const int32_t* positions;
  const void* q_weight;
  const void* k_weight;
  float eps;
  void* q_out;
  int64_t q_out_stride;
  int32_t* slot_pos;
  int64_t slot_pos_stride;
  double theta[kD / 2];  // rope_base^(-2c/D)
};

struct DecodeArgs {
  PagedView kv;
  const void* q;
  int64_t q_stride;  // elements
  int n_rows, Hq, group;
  const int32_t* row_seq;
  const int32_t* row_len;
  int window, n_sink;
  float scale_log2;  // sm_scale * k_scale * log2(e)
  const int32_t* sel;
  const int32_t* sel_count;
  int64_t sel_stride;
  void* out;
  int64_t out_stride;
  float* lse;
  float* scores;
  int64_t scores_stride;
  void* workspace;
};

struct SelectPagesArgs {
  PagedView kv;
  const void* q;
  int64_t q_stride;
  int n_rows, Hq, group;
  const int32_t* row_seq;
  const int32_t* row_len;
  int top, n_first, n_recent;
  int32_t* sel;
  int64_t sel_stride;
  int32_t* sel_count;
  unsigned long long* keys;  // workspace [n_rows][Hkv][max_pages]: exact keys, where many are needed
  float* approx;             // workspace [n_rows][Hkv][max_pages]
  float* chunk_max;          // workspace [n_rows][Hkv][page_chunks(max_pages)]
};
// pages that a warp of the page scoring takes at a time
constexpr int kPageChunk = 16;
inline int page_chunks(int max_pages) { return (max_pages + kPageChunk - 1) / kPageChunk; }

struct EvictArgs {
  PagedView kv;
  int row_bytes;
  const int32_t* seq_len;
  int budget, n_recent, n_sink;
  const float* scores;
  const int32_t* positions;
  int64_t stride;
  float* out_scores;
  int32_t* out_positions;
  int32_t* out_len;
  int32_t* moves;   // workspace [n_seqs][Hkv][stride]: slots that move, then the slots they fill
  int32_t* n_moves; // workspace [n_seqs][Hkv]
};

// Launch that may start while the kernel before it in the stream drains (see after_wait).
template <typename... P, typename... A>
cudaError_t launch_after(void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, fn, args...);
}

// Dynamic shared memory of a kernel raised to `bytes`, once per device.
template <typename Fn>
cudaError_t allow_smem(Fn* fn, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
  return e;
}

cudaError_t launch_paged_append(const AppendArgs& a, int io_dtype, int kv_dtype, cudaStream_t st);
cudaError_t launch_paged_bounds(const PagedView& kv, int kv_dtype, const int32_t* seq_len, cudaStream_t st);
size_t paged_decode_workspace(const rtp_paged_kv* kv, int n_rows, int n_q_heads, bool scores);
cudaError_t launch_paged_decode(const DecodeArgs& a, const rtp_paged_kv* kv, int q_dtype, cudaStream_t st);
cudaError_t launch_paged_select(const SelectPagesArgs& a, int q_dtype, int kv_dtype, cudaStream_t st);
cudaError_t launch_paged_evict(const EvictArgs& a, cudaStream_t st);

}  // namespace rtp
