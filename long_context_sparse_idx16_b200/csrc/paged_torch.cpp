// paged_torch.cpp -- torch binding of the paged-cache operators (include/rtp_paged.h).
//
// Checks and marshalling of arguments only; the work is librtp.so's.  It is a compiled module
// because a decode step's kernels take a few microseconds: a decode call, its launches and allocations
// included, took 28 us of host time through ctypes and takes 6.5 here.
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/extension.h>

#include <map>
#include <mutex>
#include <optional>
#include <string>

#include "rtp_paged.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}
template <typename... A>
[[noreturn]] void bad(const A&... a) {
  std::string s;
  ((s += a), ...);
  throw py::value_error(s);
}

int code_of(at::ScalarType t) {
  return t == at::kHalf ? RTP_FP16 : t == at::kBFloat16 ? RTP_BF16 : t == at::kFloat8_e4m3fn ? RTP_E4M3 : -1;
}

void check(rtp_status st) {
  if (st == RTP_OK) return;
  const py::object cls = py::module_::import("long_context_sparse_idx16_b200").attr("RTPError");
  const py::object e = cls((int)st, std::string(rtp_last_error(nullptr)));
  PyErr_SetObject(cls.ptr(), e.ptr());
  throw py::error_already_set();
}

void* ptr(const OptTensor& t) { return t ? t->data_ptr() : nullptr; }

// A CUDA stream given as a torch.cuda.Stream.
c10::Stream stream_of(const py::object& s) {
  return c10::Stream::unpack3(s.attr("stream_id").cast<int64_t>(), (c10::DeviceIndex)s.attr("device_index").cast<int64_t>(),
                              (c10::DeviceType)s.attr("device_type").cast<int64_t>());
}

// A zero in the device's memory for a cache's errors.  It is zero when this returns, whatever the streams
// still have to do (a memset on the current stream would come behind the first errors of another), and
// is never given back: kernels of a cache that was dropped may still write it.  Four bytes a cache.
uint32_t* error_word(int device) {
  constexpr int kWords = 1 << 14;
  struct Slab {
    uint32_t* next = nullptr;
    int left = 0;
  };
  static std::mutex lock;
  static std::map<int, Slab>& slabs = *new std::map<int, Slab>;
  const std::lock_guard<std::mutex> held(lock);
  Slab& s = slabs[device];
  if (!s.left) {
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
    const c10::cuda::CUDAStreamCaptureModeGuard relaxed(cudaStreamCaptureModeRelaxed);  // a capture may be under way
    void* p = nullptr;
    if (cudaMalloc(&p, kWords * sizeof(uint32_t)) != cudaSuccess) {
      cudaGetLastError();
      c10::cuda::CUDACachingAllocator::emptyCache();
      C10_CUDA_CHECK(cudaMalloc(&p, kWords * sizeof(uint32_t)));
    }
    cudaStream_t st;
    C10_CUDA_CHECK(cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking));
    C10_CUDA_CHECK(cudaMemsetAsync(p, 0, kWords * sizeof(uint32_t), st));
    C10_CUDA_CHECK(cudaStreamSynchronize(st));
    C10_CUDA_CHECK(cudaStreamDestroy(st));
    s.next = static_cast<uint32_t*>(p);
    s.left = kWords;
  }
  --s.left;
  return s.next++;
}

class PagedKV {
 public:
  PagedKV(const Tensor& k, const Tensor& v, const Tensor& table, double k_scale, double v_scale, const OptTensor& bounds)
      : k_(k), v_(v), table_(table), bounds_(bounds), device_(k.device()), dtype_(k.scalar_type()) {
    if (k.dim() != 4 || v.sizes() != k.sizes()) bad("k and v: expected [n_pages][Hkv][page_size][D] tensors of one shape");
    if (code_of(dtype_) < 0 || v.scalar_type() != dtype_)
      bad("k and v: expected one of float16, bfloat16, float8_e4m3fn for both");
    if (table.dim() != 2 || table.scalar_type() != at::kInt || (table.size(1) > 1 && table.stride(1) != 1))
      bad("block_table: expected int32 [n_seqs][max_pages] with contiguous rows");
    if (v.device() != device_ || table.device() != device_) bad("k, v and block_table must be on one device");
    if (k.stride(3) != 1 || v.stride(3) != 1) bad("k and v: the last dimension must be contiguous");
    h_.k = k.data_ptr();
    h_.v = v.data_ptr();
    // a dimension of one entry may carry any stride: give it that of a packed tensor
    int64_t packed = k.size(3);
    for (int i = 2; i >= 0; --i) {
      h_.k_stride[i] = k.size(i) == 1 ? packed : k.stride(i);
      h_.v_stride[i] = k.size(i) == 1 ? packed : v.stride(i);
      packed *= k.size(i);
    }
    h_.n_pages = k.size(0);
    h_.n_kv_heads = (int32_t)k.size(1);
    h_.page_size = (int32_t)k.size(2);
    h_.head_dim = (int32_t)k.size(3);
    h_.dtype = code_of(dtype_);
    h_.k_scale = (float)k_scale;
    h_.v_scale = (float)v_scale;
    h_.block_table = table.data_ptr<int32_t>();
    h_.n_seqs = (int32_t)table.size(0);
    h_.max_pages = (int32_t)table.size(1);
    h_.table_stride = table.size(0) > 1 ? table.stride(0) : std::max<int64_t>(1, table.size(1));
    if (bounds) {
      exact(*bounds, "bounds", {k.size(0), k.size(1), 2, k.size(3)}, dtype_);
      h_.bounds = bounds->data_ptr();
    }
    if (device_.is_cuda()) h_.err = error_word(device_.index());
  }

  const Tensor& k() const { return k_; }
  const Tensor& v() const { return v_; }
  const Tensor& table() const { return table_; }
  const OptTensor& bounds() const { return bounds_; }
  py::object device() const { return py::cast(device_); }
  int64_t n_seqs() const { return h_.n_seqs; }
  int64_t n_pages() const { return h_.n_pages; }
  int64_t n_kv_heads() const { return h_.n_kv_heads; }
  int64_t page_size() const { return h_.page_size; }
  int64_t head_dim() const { return h_.head_dim; }
  int64_t max_pages() const { return h_.max_pages; }
  int64_t capacity() const { return (int64_t)h_.max_pages * h_.page_size; }

  OptTensor append(const OptTensor& q, const Tensor& k, const Tensor& v, const Tensor& seq_lens, const OptTensor& cu_new,
                   std::optional<int64_t> max_new, const OptTensor& positions, const OptTensor& q_weight,
                   const OptTensor& k_weight, double eps, double rope_base, OptTensor q_out,
                   const OptTensor& slot_positions, const py::object& stream) {
    const at::ScalarType dt = k.scalar_type();
    const int64_t ks = heads(k, "k", -1, h_.n_kv_heads), T = k.size(0);
    const int64_t vs = heads(v, "v", T, h_.n_kv_heads, &dt);
    exact(seq_lens, "seq_lens", {h_.n_seqs}, at::kInt);
    if (cu_new) exact(*cu_new, "cu_new", {h_.n_seqs + 1}, at::kInt);
    else if (T != h_.n_seqs) bad("k: ", std::to_string(T), " tokens for ", std::to_string(h_.n_seqs), " sequences need cu_new");
    if (positions) exact(*positions, "positions", {T}, at::kInt);
    if (q_weight) exact(*q_weight, "q_weight", {h_.head_dim}, dt);
    if (k_weight) exact(*k_weight, "k_weight", {h_.head_dim}, dt);
    int64_t sps = 0;
    if (slot_positions) sps = slots(*slot_positions, "slot_positions", at::kInt);
    if (q_out && !q) bad("q_out needs q");
    const Guard guard(*this, stream);
    int64_t qs = 0, os = 0, hq = 0;
    if (q) {
      qs = heads(*q, "q", T, -1, &dt);
      hq = q->size(1);
      if (!q_out) q_out = make(guard, {T, hq, h_.head_dim}, dt);
      os = heads(*q_out, "q_out", T, hq, &dt);
    }
    guard.inputs(*this, q, k, v, seq_lens, cu_new, positions, q_weight, k_weight, q_out, slot_positions);
    if (T)
      check(rtp_paged_append(&h_, ptr(q), k.data_ptr(), v.data_ptr(), code_of(dt), qs, ks, vs, num(T), num(hq),
                             static_cast<int32_t*>(ptr(cu_new)), num(max_new.value_or(T)), seq_lens.data_ptr<int32_t>(),
                             static_cast<int32_t*>(ptr(positions)), ptr(q_weight), ptr(k_weight), (float)eps, rope_base,
                             ptr(q_out), os, static_cast<int32_t*>(ptr(slot_positions)), sps, guard.stream));
    return q_out;
  }

  void update_bounds(const Tensor& seq_lens, const py::object& stream) {
    if (!bounds_) bad("the cache keeps no page bounds");
    exact(seq_lens, "seq_lens", {h_.n_seqs}, at::kInt);
    const Guard guard(*this, stream);
    guard.inputs(*this, seq_lens);
    check(rtp_paged_bounds(&h_, seq_lens.data_ptr<int32_t>(), guard.stream));
  }

  py::object decode(const Tensor& q, const Tensor& seq_lens, const OptTensor& row_seq, int64_t window, int64_t n_sink,
                    double sm_scale, const std::optional<std::pair<Tensor, Tensor>>& pages, const OptTensor& scores,
                    OptTensor out, bool return_lse, const py::object& stream) {
    const int64_t qs = queries(q), n = q.size(0), hq = q.size(1);
    rows(n, seq_lens, row_seq);
    if (sm_scale != 0.0 && (float)sm_scale == 0.f) bad("sm_scale is below fp32's least value (0 stands for 1/sqrt(D))");
    const int32_t *sel = nullptr, *cnt = nullptr;
    int64_t ss = 0, st = 0;
    if (pages) {
      const Tensor& p = pages->first;
      is(p, "pages", at::kInt);
      // (an empty list has no address, and without one every slot is attended)
      if (p.dim() != 3 || p.size(0) != n || p.size(1) != h_.n_kv_heads || p.size(2) < 1 || !p.is_contiguous())
        bad("pages: expected contiguous indexes [", std::to_string(n), "][", std::to_string(h_.n_kv_heads),
            "][at least 1], got ", shape_of(p));
      exact(pages->second, "page counts", {n, h_.n_kv_heads}, at::kInt);
      ss = p.size(2);
      sel = p.data_ptr<int32_t>();
      cnt = pages->second.data_ptr<int32_t>();
    }
    if (scores) st = slots(*scores, "scores", at::kFloat);
    const at::ScalarType dt = q.scalar_type();
    const Guard guard(*this, stream);
    if (!out) out = make(guard, {n, hq, h_.head_dim}, dt);
    const int64_t os = heads(*out, "out", n, hq, &dt);
    OptTensor lse;
    if (return_lse) lse = make(guard, {n, hq}, at::kFloat);
    guard.inputs(*this, q, seq_lens, row_seq, scores, out);
    if (pages) guard.inputs(*this, pages->first, pages->second);
    if (n) {
      const size_t need = rtp_paged_decode_workspace(&h_, num(n), num(hq), scores ? 1 : 0);
      const at::DataPtr ws = workspace(need);
      check(rtp_paged_decode(&h_, q.data_ptr(), code_of(dt), qs, num(n), num(hq), static_cast<int32_t*>(ptr(row_seq)),
                             seq_lens.data_ptr<int32_t>(), num(window), num(n_sink), (float)sm_scale, sel, cnt, ss,
                             out->data_ptr(), os, static_cast<float*>(ptr(lse)), static_cast<float*>(ptr(scores)), st,
                             ws.get(), need, guard.stream));
    }
    if (return_lse) return py::make_tuple(*out, *lse);
    return py::cast(*out);
  }

  py::tuple select_pages(const Tensor& q, const Tensor& seq_lens, int64_t top_pages, const OptTensor& row_seq,
                         int64_t n_first, int64_t n_recent, const py::object& stream) {
    const int64_t qs = queries(q), n = q.size(0), hq = q.size(1);
    rows(n, seq_lens, row_seq);
    if (!bounds_) bad("the cache keeps no page bounds");
    if (top_pages < 1) bad("top_pages must be at least 1");
    const Guard guard(*this, stream);
    const Tensor sel = make(guard, {n, h_.n_kv_heads, top_pages}, at::kInt);
    const Tensor cnt = make(guard, {n, h_.n_kv_heads}, at::kInt);
    guard.inputs(*this, q, seq_lens, row_seq);
    if (n) {
      const size_t need = rtp_paged_select_workspace(&h_, num(n), num(hq));
      const at::DataPtr ws = workspace(need);
      check(rtp_paged_select(&h_, q.data_ptr(), code_of(q.scalar_type()), qs, num(n), num(hq),
                             static_cast<int32_t*>(ptr(row_seq)), seq_lens.data_ptr<int32_t>(), num(top_pages),
                             num(n_first), num(n_recent), sel.data_ptr<int32_t>(), top_pages, cnt.data_ptr<int32_t>(),
                             ws.get(), need, guard.stream));
    }
    return py::make_tuple(sel, cnt);
  }

  py::tuple evict(const Tensor& seq_lens, int64_t budget, const Tensor& scores, const Tensor& positions,
                  int64_t n_recent, int64_t n_sink, const OptTensor& out_scores, const OptTensor& out_positions,
                  const py::object& stream) {
    exact(seq_lens, "seq_lens", {h_.n_seqs}, at::kInt);
    const Tensor so = out_scores.value_or(scores), po = out_positions.value_or(positions);
    const int64_t st = slots(scores, "scores", at::kFloat);
    for (const auto& [t, name, dt] : {std::tuple{&positions, "positions", at::kInt}, std::tuple{&so, "out_scores", at::kFloat},
                                      std::tuple{&po, "out_positions", at::kInt}})
      if (slots(*t, name, dt) != st) bad(name, ": expected ", std::to_string(st), " slots, as scores have");
    const Guard guard(*this, stream);
    const Tensor len = make(guard, {h_.n_seqs}, at::kInt);
    guard.inputs(*this, seq_lens, scores, positions, so, po);
    const size_t need = rtp_paged_evict_workspace(&h_, st);
    const at::DataPtr ws = workspace(need);
    check(rtp_paged_evict(&h_, seq_lens.data_ptr<int32_t>(), num(budget), num(n_recent), num(n_sink),
                          scores.data_ptr<float>(), positions.data_ptr<int32_t>(), st, so.data_ptr<float>(),
                          po.data_ptr<int32_t>(), len.data_ptr<int32_t>(), ws.get(), need, guard.stream));
    if (bounds_) check(rtp_paged_bounds(&h_, len.data_ptr<int32_t>(), guard.stream));
    return py::make_tuple(len, so, po);
  }

  // Bits of the error word, taken and cleared in one step; waits for the stream, and lets other Python
  // threads (and host callbacks on the stream that need the interpreter) run meanwhile.
  int64_t errors(const py::object& stream) {
    const Guard guard(*this, stream);
    const at::DataPtr bits = workspace(sizeof(uint32_t));
    check(rtp_paged_take_errors(&h_, static_cast<uint32_t*>(bits.get()), guard.stream));
    uint32_t w = 0;
    const py::gil_scoped_release others;
    c10::cuda::memcpy_and_sync(&w, bits.get(), sizeof(w), cudaMemcpyDeviceToHost, guard.stream);
    return w;
  }

 private:
  // The cache's device, and the stream that the call (and what it allocates) uses.  If that is not the
  // current one, torch's allocator is told of every tensor that crosses: a tensor freed after the call
  // would otherwise go to work of the one stream while the other still reads it.
  struct Guard {
    c10::OptionalDeviceGuard device;
    c10::OptionalStreamGuard other;
    std::optional<c10::Stream> mine, callers;  // with a stream given that is not the current one
    cudaStream_t stream = nullptr;
    Guard(const PagedKV& kv, const py::object& s) {
      if (!kv.device_.is_cuda()) bad("the cache must be on a CUDA device, not ", kv.device_.str());
      device.reset_device(kv.device_);
      const at::cuda::CUDAStream current = at::cuda::getCurrentCUDAStream(kv.device_.index());
      stream = current.stream();
      if (!s.is_none()) {
        const c10::Stream st = stream_of(s);
        if (st.device() != kv.device_) bad("stream: expected a stream of ", kv.device_.str());
        if (st != current.unwrap()) {
          other.reset_stream(st);
          mine = st;
          callers = current.unwrap();
          stream = at::cuda::getCurrentCUDAStream(kv.device_.index()).stream();
        }
      }
    }
    template <typename... T>
    void inputs(const PagedKV& kv, const T&... t) const {
      if (!mine) return;
      (read(t), ...);
      read(kv.k_);
      read(kv.v_);
      read(kv.table_);
      read(kv.bounds_);
    }
    void output(const Tensor& t) const {
      if (mine) t.record_stream(*callers);
    }

   private:
    void read(const Tensor& t) const { t.record_stream(*mine); }
    void read(const OptTensor& t) const {
      if (t) t->record_stream(*mine);
    }
  };

  static int32_t num(int64_t x) {
    if (x > INT32_MAX || x < INT32_MIN) bad("a size or count is beyond 32 bits");
    return (int32_t)x;
  }

  // A new tensor, and a workspace that lives until the call returns (its memory is then torch's to give
  // to later work of the same stream).  Both straight from torch's allocator: through the dispatcher an
  // allocation takes 0.5 us more, and a decode call makes three.
  Tensor make(const Guard& guard, at::IntArrayRef shape, at::ScalarType dt) const {
    const Tensor t = at::detail::empty_cuda(shape, dt, device_, std::nullopt);
    guard.output(t);
    return t;
  }
  static at::DataPtr workspace(size_t n) {
    return c10::cuda::CUDACachingAllocator::get()->allocate(std::max<size_t>(n, 16));
  }

  void is(const Tensor& t, const char* name, at::ScalarType dt) const {
    if (t.device() != device_) bad(name, ": expected a tensor on ", device_.str(), ", got ", t.device().str());
    if (t.scalar_type() != dt)
      bad(name, ": expected dtype ", c10::toString(dt), ", got ", c10::toString(t.scalar_type()));
  }

  // A contiguous tensor of exactly this shape and dtype on the cache's device.
  void exact(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dt) const {
    is(t, name, dt);
    if (t.sizes() != shape) {
      std::string s = "(";
      for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
      bad(name, ": expected shape ", s, "), got ", shape_of(t));
    }
    if (!t.is_contiguous()) bad(name, ": expected a contiguous tensor");
  }

  // [rows][heads][D] activations with contiguous heads (-1: any number); returns the row stride.
  int64_t heads(const Tensor& t, const char* name, int64_t n, int64_t h, const at::ScalarType* dt = nullptr) const {
    if (dt) {
      is(t, name, *dt);
    } else {
      is(t, name, t.scalar_type());
    }
    const at::ScalarType x = t.scalar_type();
    if ((x != at::kHalf && x != at::kBFloat16) || (dtype_ != at::kFloat8_e4m3fn && x != dtype_))
      bad(name, ": expected dtype ", dtype_ == at::kFloat8_e4m3fn ? "Half or BFloat16" : c10::toString(dtype_), ", got ",
          c10::toString(x));
    if (t.dim() != 3 || t.size(2) != h_.head_dim || (n >= 0 && t.size(0) != n) || (h >= 0 && t.size(1) != h))
      bad(name, ": expected shape (", n >= 0 ? std::to_string(n) : "rows", ", ", h >= 0 ? std::to_string(h) : "heads", ", ",
          std::to_string(h_.head_dim), "), got ", shape_of(t));
    if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != h_.head_dim))
      bad(name, ": the heads of a row must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * h_.head_dim;
  }

  int64_t queries(const Tensor& q) const {
    const int64_t s = heads(q, "q", -1, -1);
    if (q.size(1) < 1 || q.size(1) % h_.n_kv_heads)
      bad("q: ", std::to_string(q.size(1)), " heads are no multiple of the ", std::to_string(h_.n_kv_heads), " KV heads");
    return s;
  }

  void rows(int64_t n, const Tensor& lens, const OptTensor& row_seq) const {
    exact(lens, "lengths", {n}, at::kInt);
    if (row_seq) exact(*row_seq, "row_seq", {n}, at::kInt);
    else if (n > h_.n_seqs) bad("q: ", std::to_string(n), " rows for ", std::to_string(h_.n_seqs), " sequences need row_seq");
  }

  // [n_seqs][Hkv][at least capacity] per-slot values; returns the slots.
  int64_t slots(const Tensor& t, const char* name, at::ScalarType dt) const {
    is(t, name, dt);
    if (t.dim() != 3 || t.size(0) != h_.n_seqs || t.size(1) != h_.n_kv_heads || t.size(2) < capacity())
      bad(name, ": expected (", std::to_string(h_.n_seqs), ", ", std::to_string(h_.n_kv_heads), ", at least ",
          std::to_string(capacity()), "), got ", shape_of(t));
    if (!t.is_contiguous()) bad(name, ": expected a contiguous tensor");
    return t.size(2);
  }

  rtp_paged_kv h_{};
  Tensor k_, v_, table_;
  OptTensor bounds_;
  c10::Device device_;
  at::ScalarType dtype_;
};

}  // namespace

PYBIND11_MODULE(_paged, m) {
  using namespace py::literals;
  m.doc() = "torch binding of the paged-cache operators; see paged.py";
  py::class_<PagedKV>(m, "PagedKV")
      .def(py::init<const Tensor&, const Tensor&, const Tensor&, double, double, const OptTensor&>(), "k"_a, "v"_a,
           "block_table"_a, py::kw_only(), "k_scale"_a = 1.0, "v_scale"_a = 1.0, "bounds"_a = py::none())
      .def_property_readonly("k", &PagedKV::k)
      .def_property_readonly("v", &PagedKV::v)
      .def_property_readonly("block_table", &PagedKV::table)
      .def_property_readonly("bounds", &PagedKV::bounds)
      .def_property_readonly("device", &PagedKV::device)
      .def_property_readonly("n_seqs", &PagedKV::n_seqs)
      .def_property_readonly("n_pages", &PagedKV::n_pages)
      .def_property_readonly("n_kv_heads", &PagedKV::n_kv_heads)
      .def_property_readonly("page_size", &PagedKV::page_size)
      .def_property_readonly("head_dim", &PagedKV::head_dim)
      .def_property_readonly("max_pages", &PagedKV::max_pages)
      .def_property_readonly("capacity", &PagedKV::capacity)
      .def("append", &PagedKV::append, "q"_a, "k"_a, "v"_a, "seq_lens"_a, py::kw_only(), "cu_new"_a = py::none(),
           "max_new"_a = py::none(), "positions"_a = py::none(), "q_weight"_a = py::none(), "k_weight"_a = py::none(),
           "eps"_a = 1e-6, "rope_base"_a = 1.0e6, "q_out"_a = py::none(), "slot_positions"_a = py::none(),
           "stream"_a = py::none())
      .def("update_bounds", &PagedKV::update_bounds, "seq_lens"_a, py::kw_only(), "stream"_a = py::none())
      .def("decode", &PagedKV::decode, "q"_a, "seq_lens"_a, py::kw_only(), "row_seq"_a = py::none(), "window"_a = 0,
           "n_sink"_a = 0, "sm_scale"_a = 0.0, "pages"_a = py::none(), "scores"_a = py::none(), "out"_a = py::none(),
           "return_lse"_a = false, "stream"_a = py::none())
      .def("select_pages", &PagedKV::select_pages, "q"_a, "seq_lens"_a, "top_pages"_a, py::kw_only(),
           "row_seq"_a = py::none(), "n_first"_a = 0, "n_recent"_a = 1, "stream"_a = py::none())
      .def("evict", &PagedKV::evict, "seq_lens"_a, "budget"_a, "scores"_a, "positions"_a, py::kw_only(), "n_recent"_a = 0,
           "n_sink"_a = 0, "out_scores"_a = py::none(), "out_positions"_a = py::none(), "stream"_a = py::none())
      .def("_errors", &PagedKV::errors, "stream"_a = py::none());
}
