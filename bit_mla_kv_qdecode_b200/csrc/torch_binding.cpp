// PyTorch binding of the operators around the decode: checks tensors, allocates
// outputs and workspaces, and calls the C entry points (include/mla_qcache.h) of
// the library that it links against. Nothing is computed here. The decode
// step of a small batch is a few microseconds on the device; the same checks
// written in Python took 8-12 us of host time a call.
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <limits>
#include <optional>
#include <string>

#include "mla_qcache.h"

namespace {

namespace py = pybind11;
using at::ScalarType;
using Tensor = at::Tensor;
using Opt = std::optional<at::Tensor>;
using Stream = std::optional<int64_t>;  // cudaStream_t; none: the current stream

constexpr int64_t kDc = 512, kDr = 64, kPage = 64;
constexpr int64_t kMaxSelected = 1 << 20;  // pages a query may attend

PyObject* g_error = nullptr;  // MlaError(function, code), kept for the life of the process

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const char* type_name(ScalarType t) {
  switch (t) {
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    default: return c10::toString(t);
  }
}

[[noreturn]] void bad_value(const std::string& why) { throw py::value_error(why); }

// Raise the error of an argument that does not fit (the contiguity check comes last).
[[noreturn]] void refuse(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape, int index) {
  const std::string n(name);
  if (t.scalar_type() != type)
    throw py::type_error(n + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (!t.is_cuda()) bad_value(n + " must be a CUDA tensor");
  if (t.sizes() != shape) bad_value(n + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.get_device() != index)
    bad_value(n + " must be on cuda:" + std::to_string(index) + ", got cuda:" + std::to_string(t.get_device()));
  bad_value(n + " must be contiguous");
}

bool fits(const Tensor& t, ScalarType type, at::IntArrayRef shape, int index) {
  return t.scalar_type() == type && t.is_cuda() && t.sizes() == shape && t.get_device() == index;
}

template <typename T = void>
T* arg(const Tensor& t, const char* name, ScalarType type, at::IntArrayRef shape, int index) {
  if (!fits(t, type, shape, index) || !t.is_contiguous()) refuse(t, name, type, shape, index);
  return static_cast<T*>(t.data_ptr());
}

template <typename T = void>
T* arg(const Opt& t, const char* name, ScalarType type, at::IntArrayRef shape, int index) {
  return t ? arg<T>(*t, name, type, shape, index) : nullptr;
}

// CUDA device of the tensor that the other arguments have to join, which has `dims` dimensions.
int device_of(const Tensor& t, const char* name, ScalarType type, int64_t dims) {
  if (t.dim() != dims)
    bad_value(std::string(name) + " must have " + std::to_string(dims) + " dimensions, got shape " + text(t.sizes()));
  if (!t.is_cuda() || t.scalar_type() != type) refuse(t, name, type, t.sizes(), 0);
  return t.get_device();
}

int as_int(int64_t v, const char* name) {
  if (v < std::numeric_limits<int>::min() || v > std::numeric_limits<int>::max())
    bad_value(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

int64_t page_count(int max_seq_len) { return max_seq_len > 0 ? (static_cast<int64_t>(max_seq_len) + kPage - 1) / kPage : 0; }

const mla_qcache_desc* description(int64_t address) { return reinterpret_cast<const mla_qcache_desc*>(address); }

// A quantized pool, which must hold every page of the description.
void* pool_of(const mla_qcache_desc* desc, const Tensor& pool, int index) {
  void* p = arg(pool, "pool", at::kByte, pool.sizes(), index);
  if (desc->num_pages > 0 && static_cast<size_t>(pool.numel()) < desc->num_pages * mla_qcache_page_bytes(desc))
    bad_value("pool is smaller than desc.num_pages pages");
  return p;
}

struct Table {
  const int32_t* p;
  int pages;
};
Table table_of(const Tensor& t, int64_t B, int index) {
  if (t.dim() != 2 || t.size(0) != B)
    bad_value("block_table must have shape (" + std::to_string(B) + ", max_pages), got " + text(t.sizes()));
  return {arg<int32_t>(t, "block_table", at::kInt, t.sizes(), index), as_int(t.size(1), "block_table")};
}

// Address and row stride of a bf16 tensor [B, n, ...] whose B * n rows are evenly spaced.
void* rows_of(const Tensor& t, const char* name, at::IntArrayRef shape, int index, int64_t& stride) {
  if (!fits(t, at::kBFloat16, shape, index)) refuse(t, name, at::kBFloat16, shape, index);
  const int64_t B = shape[0], n = shape[1];
  if (t.numel() && (t.stride(-1) != 1 || (B > 1 && n > 1 && t.stride(0) != n * t.stride(1))))
    bad_value(std::string(name) + " must have unit stride in its last dimension and evenly spaced rows");
  stride = n > 1 ? t.stride(1) : B > 1 ? t.stride(0) : 0;
  return t.data_ptr();
}

// Address and row stride of an optional bf16 output [rows, width] with unit stride in a row.
void* out_rows(const Opt& t, const char* name, int64_t rows, int64_t width, int index, int64_t& stride) {
  stride = 0;
  if (!t) return nullptr;
  if (!fits(*t, at::kBFloat16, {rows, width}, index)) refuse(*t, name, at::kBFloat16, {rows, width}, index);
  if (t->stride(1) != 1 || (rows > 1 && t->stride(0) < width))
    bad_value(std::string(name) + " must have unit stride in a row and rows that do not overlap");
  stride = rows > 1 ? t->stride(0) : width;
  return t->data_ptr();
}

// Uninitialised tensor for a kernel on `stream`: taken from that stream's memory,
// and not given back while the current stream may still read it.
Tensor empty(at::IntArrayRef shape, ScalarType type, int index, const Stream& stream) {
  const auto options = at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(index));
  if (stream) {
    const auto current = c10::cuda::getCurrentCUDAStream(index);
    if (reinterpret_cast<int64_t>(current.stream()) != *stream) {
      const auto other = *stream ? c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*stream), index)
                                 : c10::cuda::getDefaultCUDAStream(index);
      c10::cuda::CUDAStreamGuard guard(other);
      Tensor t = at::empty(shape, options);
      t.record_stream(current);
      return t;
    }
  }
  return at::empty(shape, options);
}

mla_stream_t handle(const Stream& stream, int index) {
  return stream ? reinterpret_cast<mla_stream_t>(*stream)
                : reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream(index).stream());
}

void check(const char* function, int code) {
  if (code == MLA_OK) return;
  PyErr_SetObject(g_error, py::reinterpret_borrow<py::object>(g_error)(function, code).ptr());
  throw py::error_already_set();
}

// Refuse, before outputs and workspaces are allocated for it, what the library would
// refuse after: a selection that cannot be, lengths that the table cannot hold.
void check_selection(const char* function, int64_t k, int64_t n_sink, int64_t n_recent) {
  if (k < 1 || k > kMaxSelected || n_sink < 0 || n_recent < 1 || n_sink > k || n_recent > k - n_sink)
    check(function, MLA_ERR_INVALID_ARG);
}
void check_capacity(const char* function, int64_t queries, int max_seq_len, int table_pages) {
  if (queries > 65535) check(function, MLA_ERR_UNSUPPORTED);
  if (queries > 0 && max_seq_len > table_pages * kPage) check(function, MLA_ERR_CAPACITY);
}

Opt append_norm_rope(int64_t desc_, const Tensor& pool, const Tensor& table, const Tensor& before, const Tensor& kv,
                     const Opt& weight, double eps, const Tensor& cos_sin, int pairs, const Opt& q, Opt q_out,
                     const Opt& positions, const Opt& new_lens, const Opt& rows_out, const Stream& stream) {
  const auto* desc = description(desc_);
  const int dev = device_of(kv, "kv", at::kBFloat16, 3);
  const int64_t B = kv.size(0), n = kv.size(1);
  int64_t kv_stride = 0, q_token = 0, q_head = 0, H = 0;
  const void* pkv = rows_of(kv, "kv", {B, n, kDc + kDr}, dev, kv_stride);
  const void* pq = nullptr;
  void* pqo = nullptr;
  if (q) {
    if (q->dim() != 4) bad_value("q must be a tensor [B, n, H, 64]");
    H = q->size(2);
    pq = rows_of(*q, "q", {B, n, H, kDr}, dev, q_token);
    q_head = H > 1 ? q->stride(2) : 0;
    if (!q_out) q_out = empty({B, n, H, kDr}, at::kBFloat16, dev, stream);
    pqo = arg(q_out, "q_out", at::kBFloat16, {B, n, H, kDr}, dev);
    if (H == 0) pq = pqo = nullptr;
  } else if (q_out) {
    bad_value("q_out needs q");
  }
  if (cos_sin.dim() != 2) bad_value("cos_sin must be a tensor [positions, 64]");
  const Table tab = table_of(table, B, dev);
  void* pp = pool_of(desc, pool, dev);
  const auto* pb = arg<int32_t>(before, "seq_lens_before", at::kInt, {B}, dev);
  const auto* pn = arg<int32_t>(new_lens, "new_lens", at::kInt, {B}, dev);
  const void* pw = arg(weight, "norm_weight", at::kBFloat16, {kDc}, dev);
  const auto* pc = arg<float>(cos_sin, "cos_sin", at::kFloat, {cos_sin.size(0), kDr}, dev);
  const auto* ppos = arg<int32_t>(positions, "positions", at::kInt, {B, n}, dev);
  void* pr = arg(rows_out, "rows_out", at::kBFloat16, {B, n, kDc + kDr}, dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  check("mla_qcache_append_norm_rope",
        mla_qcache_append_norm_rope(desc, pp, tab.p, tab.pages, pb, pn, pkv, kv_stride, pw, static_cast<float>(eps), pq,
                                    q_token, q_head, as_int(H, "q"), pqo, pc, as_int(cos_sin.size(0), "cos_sin"), ppos,
                                    pairs, pr, as_int(B, "kv"), as_int(n, "kv"), handle(stream, dev)));
  return q_out;
}

void qcache_read(int64_t desc_, const Tensor& pool, const Tensor& table, const Opt& start, const Tensor& cu_rows,
          int64_t max_rows, const Opt& out_c, const Opt& out_kr, const Stream& stream) {
  const auto* desc = description(desc_);
  const Opt& out = out_c ? out_c : out_kr;
  if (!out || out->dim() != 2) bad_value("out_c or out_kr must be given, as tensors [rows, width]");
  const int dev = device_of(cu_rows, "cu_rows", at::kInt, 1);
  const int64_t B = cu_rows.size(0) - 1, rows = out->size(0);
  if (B < 0) bad_value("cu_rows must have one entry more than there are requests");
  int64_t c_stride = 0, kr_stride = 0;
  void* pc = out_rows(out_c, "out_c", rows, kDc, dev, c_stride);
  void* pr = out_rows(out_kr, "out_kr", rows, kDr, dev, kr_stride);
  const Table tab = table_of(table, B, dev);
  const void* pp = pool_of(desc, pool, dev);
  const auto* ps = arg<int32_t>(start, "start", at::kInt, {B}, dev);
  const auto* pcu = arg<int32_t>(cu_rows, "cu_rows", at::kInt, {B + 1}, dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  check("mla_qcache_read", mla_qcache_read(desc, pp, tab.p, tab.pages, ps, pcu, as_int(max_rows, "max_rows"), rows, pc,
                                           c_stride, pr, kr_stride, as_int(B, "cu_rows"), handle(stream, dev)));
}

void page_digest(int64_t desc_, const Tensor& pool, const Tensor& table, const Tensor& before, int64_t n_new,
                 const Tensor& digests, const Opt& new_lens, const Stream& stream) {
  const auto* desc = description(desc_);
  const int dev = device_of(before, "seq_lens_before", at::kInt, 1);
  const int64_t B = before.size(0);
  const Table tab = table_of(table, B, dev);
  const void* pp = pool_of(desc, pool, dev);
  const auto* pb = arg<int32_t>(before, "seq_lens_before", at::kInt, {B}, dev);
  const auto* pn = arg<int32_t>(new_lens, "new_lens", at::kInt, {B}, dev);
  void* pd = arg(digests, "digests", at::kBFloat16, {desc->num_pages, kDc + kDr}, dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  check("mla_page_digest", mla_page_digest(desc, pp, tab.p, tab.pages, pb, pn, as_int(n_new, "n_new"), pd,
                                           as_int(B, "seq_lens_before"), handle(stream, dev)));
}

struct Queries {
  int dev;
  int64_t B, s_q, H;
  const void *c, *r;
};
Queries queries(const Tensor& q_c, const Tensor& q_r) {
  Queries q{};
  q.dev = device_of(q_c, "q_c", at::kBFloat16, 4);
  q.B = q_c.size(0);
  q.s_q = q_c.size(1);
  q.H = q_c.size(2);
  q.c = arg(q_c, "q_c", at::kBFloat16, {q.B, q.s_q, q.H, kDc}, q.dev);
  q.r = arg(q_r, "q_r", at::kBFloat16, {q.B, q.s_q, q.H, kDr}, q.dev);
  return q;
}

Tensor page_scores(const Tensor& table, const Tensor& seq_lens, int64_t max_seq_len_, const Tensor& digests,
                   const Tensor& q_c, const Tensor& q_r, double scale, const Opt& out_, const Stream& stream) {
  const Queries q = queries(q_c, q_r);
  const int max_seq_len = as_int(max_seq_len_, "max_seq_len");
  const int64_t pages = digests.dim() == 2 ? digests.size(0) : 0;
  const void* pd = arg(digests, "digests", at::kBFloat16, {pages, kDc + kDr}, q.dev);
  const Table tab = table_of(table, q.B, q.dev);
  const auto* pl = arg<int32_t>(seq_lens, "seq_lens", at::kInt, {q.B}, q.dev);
  check_capacity("mla_page_scores", q.B * q.s_q, max_seq_len, tab.pages);
  const int64_t shape[3] = {q.B, q.s_q, page_count(max_seq_len)};
  const Tensor out = out_ ? *out_ : empty(shape, at::kFloat, q.dev, stream);
  auto* po = arg<float>(out, "out", at::kFloat, shape, q.dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(q.dev));
  check("mla_page_scores",
        mla_page_scores(pd, as_int(pages, "digests"), tab.p, tab.pages, pl, max_seq_len, q.c, q.r, as_int(q.B, "q_c"),
                        as_int(q.s_q, "q_c"), as_int(q.H, "q_c"), static_cast<float>(scale), po, handle(stream, q.dev)));
  return out;
}

std::tuple<Tensor, Tensor, Tensor> select_pages(const Tensor& table, const Tensor& seq_lens, int64_t max_seq_len_,
                                                const Opt& scores, int64_t k, int64_t n_sink, int64_t n_recent,
                                                std::optional<int64_t> s_q_, const Opt& sel_table_, const Opt& sel_pages_,
                                                const Opt& sel_lens_, const Stream& stream) {
  if (!scores && !s_q_) bad_value("s_q is needed without scores");
  if (scores && scores->dim() != 3) bad_value("scores must be a tensor [B, s_q, pages]");
  const int64_t s_q = scores ? scores->size(1) : *s_q_;
  const int dev = device_of(seq_lens, "seq_lens", at::kInt, 1);
  const int64_t B = seq_lens.size(0);
  const int max_seq_len = as_int(max_seq_len_, "max_seq_len");
  check_selection("mla_select_pages", k, n_sink, n_recent);
  if (s_q < 1 || s_q > 65535) check("mla_select_pages", MLA_ERR_INVALID_ARG);
  const int64_t shape[3] = {B, s_q, k}, score_shape[3] = {B, s_q, page_count(max_seq_len)};
  const auto* ps = arg<float>(scores, "scores", at::kFloat, score_shape, dev);
  const Table tab = table_of(table, B, dev);
  const auto* pl = arg<int32_t>(seq_lens, "seq_lens", at::kInt, {B}, dev);
  check_capacity("mla_select_pages", B * s_q, max_seq_len, tab.pages);
  const Tensor t = sel_table_ ? *sel_table_ : empty(shape, at::kInt, dev, stream);
  const Tensor p = sel_pages_ ? *sel_pages_ : empty(shape, at::kInt, dev, stream);
  const Tensor l = sel_lens_ ? *sel_lens_ : empty({B, s_q}, at::kInt, dev, stream);
  auto* pt = arg<int32_t>(t, "sel_table", at::kInt, shape, dev);
  auto* pp = arg<int32_t>(p, "sel_pages", at::kInt, shape, dev);
  auto* pn = arg<int32_t>(l, "sel_lens", at::kInt, {B, s_q}, dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  check("mla_select_pages",
        mla_select_pages(tab.p, tab.pages, pl, max_seq_len, ps, as_int(B, "seq_lens"), as_int(s_q, "s_q"),
                         as_int(k, "k_pages"), as_int(n_sink, "n_sink"), as_int(n_recent, "n_recent"), pt, pp, pn,
                         handle(stream, dev)));
  return {t, p, l};
}

Tensor qdecode_sparse(int64_t desc_, const Tensor& pool, const Tensor& table, const Tensor& seq_lens, int64_t max_seq_len_,
                      const Opt& digests, const Tensor& q_c, const Tensor& q_r, double scale, int64_t k, int64_t n_sink,
                      int64_t n_recent, const Opt& out_, bool f32, const Opt& lse, int64_t num_splits,
                      const Opt& workspace_, unsigned flags, const Stream& stream) {
  const auto* desc = description(desc_);
  const Queries q = queries(q_c, q_r);
  const int max_seq_len = as_int(max_seq_len_, "max_seq_len"), B = as_int(q.B, "q_c"), s_q = as_int(q.s_q, "q_c"),
            H = as_int(q.H, "q_c"), k_pages = as_int(k, "k_pages"), splits = as_int(num_splits, "num_splits");
  const Table tab = table_of(table, q.B, q.dev);
  check_selection("mla_qdecode_sparse", k, n_sink, n_recent);
  check_capacity("mla_qdecode_sparse", q.B * q.s_q, max_seq_len, tab.pages);
  const int64_t shape[4] = {q.B, q.s_q, q.H, kDc};
  const Tensor out = out_ ? *out_ : empty(shape, f32 ? at::kFloat : at::kBFloat16, q.dev, stream);
  f32 = out.scalar_type() == at::kFloat;
  if (!f32 && out.scalar_type() != at::kBFloat16) throw py::type_error("out must be bfloat16 or float32");
  void* po = arg(out, "out", out.scalar_type(), shape, q.dev);
  const void* pp = pool_of(desc, pool, q.dev);
  const auto* pl = arg<int32_t>(seq_lens, "seq_lens", at::kInt, {q.B}, q.dev);
  const void* pd = arg(digests, "digests", at::kBFloat16, {desc->num_pages, kDc + kDr}, q.dev);
  auto* pe = arg<float>(lse, "lse", at::kFloat, {q.B, q.s_q, q.H}, q.dev);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(q.dev));  // the split plan is the device's
  const Tensor workspace =
      workspace_ ? *workspace_
                 : empty({static_cast<int64_t>(mla_qdecode_sparse_workspace_bytes(B, s_q, H, max_seq_len, k_pages, splits)) + 1},
                         at::kByte, q.dev, stream);
  void* pw = arg(workspace, "workspace", at::kByte, {workspace.numel()}, q.dev);
  check("mla_qdecode_sparse",
        mla_qdecode_sparse(desc, pp, tab.p, tab.pages, pl, max_seq_len, pd, q.c, q.r, B, s_q, H, static_cast<float>(scale),
                           k_pages, as_int(n_sink, "n_sink"), as_int(n_recent, "n_recent"), splits, pw,
                           static_cast<size_t>(workspace.numel()), po, f32, pe, flags, handle(stream, q.dev)));
  return out;
}

}  // namespace

PYBIND11_MODULE(_mla_torch, m) {
  m.def("set_error", [](const py::object& e) { g_error = py::object(e).release().ptr(); });
  m.def("append_norm_rope", &append_norm_rope);
  m.def("qcache_read", &qcache_read);
  m.def("page_digest", &page_digest);
  m.def("page_scores", &page_scores);
  m.def("select_pages", &select_pages);
  m.def("qdecode_sparse", &qdecode_sparse);
}
