// paged_api.cu -- the C entry points of the paged-cache operators: host checks and launches.
#include <math.h>

#include "paged.cuh"

using namespace rtp;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
int elem_size(int dtype) { return dtype == RTP_E4M3 ? 1 : 2; }

// Whether two arrays share a byte.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

rtp_status bad(const char* fn, const char* what) { return fail(nullptr, RTP_EINVAL, std::string(fn) + ": " + what); }

// Checks a cache description and fills the kernels' view of it; NULL if it is right, else what is not.
const char* view_of(const rtp_paged_kv* kv, PagedView* p) {
  if (!kv) return "kv is NULL";
  if (!kv->k || !kv->v || !kv->block_table) return "k, v and block_table must not be NULL";
  if (kv->dtype != RTP_FP16 && kv->dtype != RTP_BF16 && kv->dtype != RTP_E4M3) return "unknown page dtype";
  if (kv->page_size != 16 && kv->page_size != 32 && kv->page_size != 64 && kv->page_size != 128)
    return "page_size must be 16, 32, 64 or 128";
  if (kv->head_dim != 64 && kv->head_dim != 128) return "head_dim must be 64 or 128";
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024) return "need 1 <= n_kv_heads <= 1024";
  if (kv->n_pages < 1 || kv->n_pages > 0x7fffffffLL) return "need 1 <= n_pages < 2^31";
  if (kv->n_seqs < 1 || kv->n_seqs > 65535) return "need 1 <= n_seqs <= 65535";
  if (kv->max_pages < 1 || (int64_t)kv->max_pages * kv->page_size > 0x7fff0000LL)
    return "need max_pages >= 1 and at most 2^31 - 2^16 slots in a table row";
  if (kv->table_stride < kv->max_pages) return "table_stride must be at least max_pages";
  if (!(kv->k_scale > 0.f) || !(kv->v_scale > 0.f) || !isfinite(kv->k_scale) || !isfinite(kv->v_scale))
    return "k_scale and v_scale must be positive and finite";
  if (!aligned16(kv->k) || !aligned16(kv->v) || !aligned16(kv->bounds)) return "k, v and bounds must be 16-byte aligned";
  const int es = elem_size(kv->dtype);
  for (int i = 0; i < 3; ++i) {
    // tensor maps describe strides below 2^40 bytes
    for (int64_t s : {kv->k_stride[i], kv->v_stride[i]})
      if (s < 1 || s >= (1LL << 38) || s * es % 16 != 0) return "page strides must be positive multiples of 16 bytes";
    if (i == 2 && (kv->k_stride[i] < kv->head_dim || kv->v_stride[i] < kv->head_dim))
      return "slot strides must be at least head_dim";
  }
  if (p) {
    p->k = static_cast<uint8_t*>(kv->k);
    p->v = static_cast<uint8_t*>(kv->v);
    p->kp = kv->k_stride[0] * es;
    p->kh = kv->k_stride[1] * es;
    p->ks = kv->k_stride[2] * es;
    p->vp = kv->v_stride[0] * es;
    p->vh = kv->v_stride[1] * es;
    p->vs = kv->v_stride[2] * es;
    p->n_pages = kv->n_pages;
    p->page_size = kv->page_size;
    p->page_shift = kv->page_size == 16 ? 4 : kv->page_size == 32 ? 5 : kv->page_size == 64 ? 6 : 7;
    p->Hkv = kv->n_kv_heads;
    p->D = kv->head_dim;
    p->max_pages = kv->max_pages;
    p->n_seqs = kv->n_seqs;
    p->table = kv->block_table;
    p->table_stride = kv->table_stride;
    p->k_scale = kv->k_scale;
    p->v_scale = kv->v_scale;
    p->bounds = static_cast<uint8_t*>(kv->bounds);
    p->err = kv->err;
  }
  return nullptr;
}

// rope_base^(-2c/D) for c < D/2.  64 calls of pow take 2 us, as long as a launch: the last table of a
// thread is kept with the numbers it was made from.
void frequencies(double base, int D, double* theta) {
  thread_local double table[kD / 2];
  thread_local double of_base = 0.0;
  thread_local int of_D = 0;
  if (base != of_base || D != of_D) {
    for (int c = 0; c < D / 2; ++c) table[c] = pow(base, -2.0 * c / D);
    of_base = base;
    of_D = D;
  }
  for (int c = 0; c < D / 2; ++c) theta[c] = table[c];
}

const char* check_io_dtype(const rtp_paged_kv* kv, int dtype) {
  if (dtype != RTP_FP16 && dtype != RTP_BF16) return "activations must be fp16 or bf16";
  if (kv->dtype != RTP_E4M3 && kv->dtype != dtype) return "activations must have the pages' dtype";
  return nullptr;
}

const char* check_rows(const rtp_paged_kv* kv, const void* q, int64_t q_stride, int n_rows, int n_q_heads,
                       const int32_t* row_seq, const int32_t* row_len) {
  if (!q || !row_len) return "q and row_len must not be NULL";
  if (n_rows < 1 || n_rows > 65535) return "need 1 <= n_rows <= 65535";
  if (!row_seq && n_rows > kv->n_seqs) return "more rows than sequences need row_seq";
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads != 0 || n_q_heads / kv->n_kv_heads > 64)
    return "n_q_heads must be a multiple of n_kv_heads, at most 64 times it";
  if (!aligned16(q) || q_stride % 8 != 0 || q_stride < (int64_t)n_q_heads * kv->head_dim)
    return "q must be 16-byte aligned, its row stride a multiple of 8 and at least n_q_heads * head_dim";
  return nullptr;
}

__global__ void take_errors_kernel(uint32_t* err, uint32_t* bits) {
  after_wait();
  *bits = atomicExch(err, 0u);
}

}  // namespace

extern "C" {

rtp_status rtp_paged_take_errors(const rtp_paged_kv* kv, uint32_t* bits, cudaStream_t stream) {
  const char* fn = "rtp_paged_take_errors";
  if (!kv || !kv->err || !bits) return bad(fn, "kv, kv->err and bits must not be NULL");
  const cudaError_t e = launch_after(take_errors_kernel, dim3(1), 1, 0, stream, kv->err, bits);
  return e == cudaSuccess ? RTP_OK : cuda_fail(nullptr, e, fn);
}

rtp_status rtp_paged_append(const rtp_paged_kv* kv, const void* q, const void* k, const void* v, int32_t dtype,
                            int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t n_tokens,
                            int32_t n_q_heads, const int32_t* cu_new, int32_t max_new, const int32_t* seq_len,
                            const int32_t* positions, const void* q_weight, const void* k_weight, float eps,
                            double rope_base, void* q_out, int64_t q_out_stride, int32_t* slot_pos,
                            int64_t slot_pos_stride, cudaStream_t stream) {
  const char* fn = "rtp_paged_append";
  AppendArgs a{};
  if (const char* m = view_of(kv, &a.kv)) return bad(fn, m);
  if (const char* m = check_io_dtype(kv, dtype)) return bad(fn, m);
  const int D = kv->head_dim;
  if (!k || !v || !seq_len) return bad(fn, "k, v and seq_len must not be NULL");
  if ((q == nullptr) != (q_out == nullptr)) return bad(fn, "q and q_out go together");
  if (n_tokens < 1) return bad(fn, "need n_tokens >= 1");
  if (!cu_new && n_tokens != kv->n_seqs) return bad(fn, "without cu_new there is one token per sequence");
  if (max_new < 1 || max_new > n_tokens) return bad(fn, "need 1 <= max_new <= n_tokens");
  if (q && (n_q_heads < 1 || n_q_heads > 65535)) return bad(fn, "need 1 <= n_q_heads <= 65535");
  if (!(eps >= 0.f) || !isfinite(eps)) return bad(fn, "eps must be finite and not negative");
  if (!(rope_base > 1.0) || !isfinite(rope_base)) return bad(fn, "rope_base must be finite and above 1");
  if (!aligned16(k) || !aligned16(v) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
      k_stride < (int64_t)kv->n_kv_heads * D || v_stride < (int64_t)kv->n_kv_heads * D)
    return bad(fn, "k and v must be 16-byte aligned, row strides multiples of 8 and at least n_kv_heads * head_dim");
  if (q && (!aligned16(q) || !aligned16(q_out) || q_stride % 8 != 0 || q_out_stride % 8 != 0 ||
            q_stride < (int64_t)n_q_heads * D || q_out_stride < (int64_t)n_q_heads * D))
    return bad(fn, "q and q_out must be 16-byte aligned, row strides multiples of 8 and at least n_q_heads * head_dim");
  if (q && q == q_out && q_stride != q_out_stride) return bad(fn, "q_out may be q only with q's stride");
  if (!aligned16(q_weight) || !aligned16(k_weight)) return bad(fn, "q_weight and k_weight must be 16-byte aligned");
  if (slot_pos && slot_pos_stride < (int64_t)kv->max_pages * kv->page_size)
    return bad(fn, "slot_pos_stride must cover max_pages * page_size slots");
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_tokens = n_tokens;
  a.Hq = q ? n_q_heads : 0;
  a.max_new = cu_new ? max_new : 1;
  a.cu_new = cu_new;
  a.seq_len = seq_len;
  a.positions = positions;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.slot_pos = slot_pos;
  a.slot_pos_stride = slot_pos_stride;
  frequencies(rope_base, D, a.theta);
  const cudaError_t e = launch_paged_append(a, dtype, kv->dtype, stream);
  return e == cudaSuccess ? RTP_OK : cuda_fail(nullptr, e, fn);
}

rtp_status rtp_paged_bounds(const rtp_paged_kv* kv, const int32_t* seq_len, cudaStream_t stream) {
  const char* fn = "rtp_paged_bounds";
  PagedView p{};
  if (const char* m = view_of(kv, &p)) return bad(fn, m);
  if (!kv->bounds || !seq_len) return bad(fn, "kv->bounds and seq_len must not be NULL");
  const cudaError_t e = launch_paged_bounds(p, kv->dtype, seq_len, stream);
  return e == cudaSuccess ? RTP_OK : cuda_fail(nullptr, e, fn);
}

size_t rtp_paged_decode_workspace(const rtp_paged_kv* kv, int32_t n_rows, int32_t n_q_heads, int with_scores) {
  if (view_of(kv, nullptr) || n_rows < 1 || n_rows > 65535 || n_q_heads < 1 || n_q_heads % kv->n_kv_heads != 0 ||
      n_q_heads / kv->n_kv_heads > 64)
    return 0;
  return paged_decode_workspace(kv, n_rows, n_q_heads, with_scores != 0);
}

rtp_status rtp_paged_decode(const rtp_paged_kv* kv, const void* q, int32_t q_dtype, int64_t q_stride,
                            int32_t n_rows, int32_t n_q_heads, const int32_t* row_seq, const int32_t* row_len,
                            int32_t window, int32_t n_sink, float sm_scale, const int32_t* sel,
                            const int32_t* sel_count, int64_t sel_stride, void* out, int64_t out_stride, float* lse,
                            float* scores, int64_t scores_stride, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  const char* fn = "rtp_paged_decode";
  DecodeArgs a{};
  if (const char* m = view_of(kv, &a.kv)) return bad(fn, m);
  if (const char* m = check_io_dtype(kv, q_dtype)) return bad(fn, m);
  if (const char* m = check_rows(kv, q, q_stride, n_rows, n_q_heads, row_seq, row_len)) return bad(fn, m);
  if (!out || !aligned16(out) || out_stride % 8 != 0 || out_stride < (int64_t)n_q_heads * kv->head_dim)
    return bad(fn, "out must be 16-byte aligned, its row stride a multiple of 8 and at least n_q_heads * head_dim");
  if (window < 0 || n_sink < 0) return bad(fn, "window and n_sink must not be negative");
  if (!(sm_scale >= 0.f) || !isfinite(sm_scale)) return bad(fn, "sm_scale must be finite and not negative");
  if (sel) {
    if (!sel_count || sel_stride < 1) return bad(fn, "sel needs sel_count and sel_stride >= 1");
    if (window) return bad(fn, "window must be 0 with a page list");
    if (scores) return bad(fn, "scores cannot be accumulated over a page list");
    if (sel_stride > 0x7fffffffLL / kv->page_size) return bad(fn, "sel_stride is too large");
  }
  if (scores && row_seq) return bad(fn, "scores need row r to be sequence r (row_seq NULL)");
  if (scores && scores_stride < (int64_t)kv->max_pages * kv->page_size)
    return bad(fn, "scores_stride must cover max_pages * page_size slots");
  const size_t need = paged_decode_workspace(kv, n_rows, n_q_heads, scores != nullptr);
  if (!workspace || !aligned16(workspace) || workspace_bytes < need)
    return bad(fn, "the workspace is missing, misaligned or smaller than rtp_paged_decode_workspace says");
  a.q = q;
  a.q_stride = q_stride;
  a.n_rows = n_rows;
  a.Hq = n_q_heads;
  a.group = n_q_heads / kv->n_kv_heads;
  a.row_seq = row_seq;
  a.row_len = row_len;
  a.window = window;
  a.n_sink = window ? n_sink : 0;
  const float scale = sm_scale > 0.f ? sm_scale : (float)(1.0 / sqrt((double)kv->head_dim));
  a.scale_log2 = (float)((double)scale * kv->k_scale * 1.4426950408889634);
  if (!isfinite(a.scale_log2)) return bad(fn, "sm_scale * k_scale must be below fp32's largest value by log2(e)");
  a.sel = sel;
  a.sel_count = sel_count;
  a.sel_stride = sel_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.lse = lse;
  a.scores = scores;
  a.scores_stride = scores_stride;
  a.workspace = workspace;
  const cudaError_t e = launch_paged_decode(a, kv, q_dtype, stream);
  return e == cudaSuccess ? RTP_OK : cuda_fail(nullptr, e, fn);
}

size_t rtp_paged_select_workspace(const rtp_paged_kv* kv, int32_t n_rows, int32_t n_q_heads) {
  if (view_of(kv, nullptr) || n_rows < 1 || n_rows > 65535 || n_q_heads < 1) return 0;
  return (size_t)n_rows * kv->n_kv_heads *
         ((size_t)kv->max_pages * (sizeof(unsigned long long) + sizeof(float)) +
          (size_t)page_chunks(kv->max_pages) * sizeof(float));
}

rtp_status rtp_paged_select(const rtp_paged_kv* kv, const void* q, int32_t q_dtype, int64_t q_stride,
                            int32_t n_rows, int32_t n_q_heads, const int32_t* row_seq, const int32_t* row_len,
                            int32_t top_pages, int32_t n_first, int32_t n_recent, int32_t* sel, int64_t sel_stride,
                            int32_t* sel_count, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const char* fn = "rtp_paged_select";
  SelectPagesArgs a{};
  if (const char* m = view_of(kv, &a.kv)) return bad(fn, m);
  if (const char* m = check_io_dtype(kv, q_dtype)) return bad(fn, m);
  if (const char* m = check_rows(kv, q, q_stride, n_rows, n_q_heads, row_seq, row_len)) return bad(fn, m);
  if (!kv->bounds) return bad(fn, "the cache keeps no page bounds");
  if (!sel || !sel_count) return bad(fn, "sel and sel_count must not be NULL");
  if (n_first < 0 || n_recent < 0 || top_pages < 1 || (int64_t)n_first + n_recent > top_pages ||
      top_pages > sel_stride)
    return bad(fn, "need 1 <= top_pages <= sel_stride and n_first + n_recent <= top_pages, none negative");
  if (!workspace || !aligned16(workspace) || workspace_bytes < rtp_paged_select_workspace(kv, n_rows, n_q_heads))
    return bad(fn, "the workspace is missing, misaligned or smaller than rtp_paged_select_workspace says");
  a.q = q;
  a.q_stride = q_stride;
  a.n_rows = n_rows;
  a.Hq = n_q_heads;
  a.group = n_q_heads / kv->n_kv_heads;
  a.row_seq = row_seq;
  a.row_len = row_len;
  a.top = top_pages;
  a.n_first = n_first;
  a.n_recent = n_recent;
  a.sel = sel;
  a.sel_stride = sel_stride;
  a.sel_count = sel_count;
  a.keys = static_cast<unsigned long long*>(workspace);
  const size_t lists = (size_t)n_rows * kv->n_kv_heads * kv->max_pages;
  a.approx = reinterpret_cast<float*>(a.keys + lists);
  a.chunk_max = a.approx + lists;
  const cudaError_t e = launch_paged_select(a, q_dtype, kv->dtype, stream);
  return e == cudaSuccess ? RTP_OK : cuda_fail(nullptr, e, fn);
}

size_t rtp_paged_evict_workspace(const rtp_paged_kv* kv, int64_t stride) {
  if (view_of(kv, nullptr) || stride < 1 || stride > (1 << 24)) return 0;
  return (size_t)kv->n_seqs * kv->n_kv_heads * (stride + 1) * sizeof(int32_t);
}

rtp_status rtp_paged_evict(const rtp_paged_kv* kv, const int32_t* seq_len, int32_t budget, int32_t n_recent,
                           int32_t n_sink, const float* scores, const int32_t* positions, int64_t stride,
                           float* out_scores, int32_t* out_positions, int32_t* out_len, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  const char* fn = "rtp_paged_evict";
  EvictArgs a{};
  if (const char* m = view_of(kv, &a.kv)) return bad(fn, m);
  if (!seq_len || !scores || !positions || !out_scores || !out_positions || !out_len)
    return bad(fn, "NULL pointer");
  if (budget < 1 || budget > (1 << 24)) return bad(fn, "need 1 <= budget <= 2^24");
  if (n_recent < 0 || n_sink < 0 || (int64_t)n_recent + n_sink > budget)
    return bad(fn, "need n_sink + n_recent <= budget, none negative");
  if (stride < (int64_t)kv->max_pages * kv->page_size || stride > (1 << 24))
    return bad(fn, "stride must cover max_pages * page_size slots and be at most 2^24");
  // CTAs of all heads read lengths, scores and positions while others have begun to write
  const size_t lens = (size_t)kv->n_seqs * sizeof(int32_t), lists = lens * kv->n_kv_heads * stride;
  if (overlap(out_len, lens, seq_len, lens)) return bad(fn, "out_len must not be seq_len");
  if ((out_scores != scores && overlap(out_scores, lists, scores, lists)) ||
      (out_positions != positions && overlap(out_positions, lists, positions, lists)))
    return bad(fn, "out_scores and out_positions may be scores and positions, but must not overlap them otherwise");
  if (overlap(out_scores, lists, positions, lists) || overlap(out_positions, lists, scores, lists) ||
      overlap(out_scores, lists, out_positions, lists))
    return bad(fn, "scores and positions must not share memory");
  for (const void* p : {(const void*)scores, (const void*)positions, (const void*)out_scores, (const void*)out_positions})
    if (overlap(out_len, lens, p, lists)) return bad(fn, "out_len must not lie in another array");
  if (overlap(seq_len, lens, out_scores, lists) || overlap(seq_len, lens, out_positions, lists))
    return bad(fn, "seq_len must not lie in an output");
  if (!workspace || !aligned16(workspace) || workspace_bytes < rtp_paged_evict_workspace(kv, stride))
    return bad(fn, "the workspace is missing, misaligned or smaller than rtp_paged_evict_workspace says");
  a.row_bytes = kv->head_dim * elem_size(kv->dtype);
  a.seq_len = seq_len;
  a.budget = budget;
  a.n_recent = n_recent;
  a.n_sink = n_sink;
  a.scores = scores;
  a.positions = positions;
  a.stride = stride;
  a.out_scores = out_scores;
  a.out_positions = out_positions;
  a.out_len = out_len;
  a.moves = static_cast<int32_t*>(workspace);
  a.n_moves = a.moves + (size_t)kv->n_seqs * kv->n_kv_heads * stride;
  const cudaError_t e = launch_paged_evict(a, stream);
  return e == cudaSuccess ? RTP_OK : cuda_fail(nullptr, e, fn);
}

}  // extern "C"
