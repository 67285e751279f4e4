// Python bindings of the rotary and draft-tree entry points (include/splitkv.h): argument checks,
// outputs and workspaces from torch's allocator, the current stream, one call.  No computation.
//
// These calls serve single tokens, where the host's time counts: reading the tensors here costs a
// few microseconds less a call than through ctypes (tree attention of one token: 24 us a call, 12 to 13.5 us
// from here).
#include <initializer_list>
#include <optional>
#include <string>
#include <tuple>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include "splitkv.h"

namespace py = pybind11;
using at::ScalarType;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

[[noreturn]] void refuse(const std::string& why) { throw py::value_error(why); }

// A status of the library as the package's SplitKVError.
void check(const char* fn, int status) {
  if (status == SPLITKV_OK) return;
  py::object error = py::module_::import("context_block_sparse_b200").attr("SplitKVError")(fn, status);
  PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(error.ptr())), error.ptr());
  throw py::error_already_set();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

using Shape = std::initializer_list<int64_t>;

// The tensor has that shape, type and device, and a contiguous last dimension.
void strided(const Tensor& t, const char* name, Shape shape, ScalarType dtype, int dev) {
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + " must be " + c10::toString(dtype) + ", not " + c10::toString(t.scalar_type()));
  if (!t.is_cuda() || t.get_device() != dev) refuse(std::string(name) + " must be a CUDA tensor on the device of the others");
  if (t.sizes() != at::IntArrayRef(shape))
    refuse(std::string(name) + " has shape " + shape_text(t.sizes()) + "; expected " + shape_text(shape));
  const int64_t d = t.dim();
  if (d > 0 && t.size(d - 1) > 1 && t.stride(d - 1) != 1)
    refuse("the last dimension of " + std::string(name) + " must be contiguous");
}

void dense(const Tensor& t, const char* name, Shape shape, ScalarType dtype, int dev) {
  strided(t, name, shape, dtype, dev);
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

int dtype_code(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case ScalarType::Float: return SPLITKV_DTYPE_F32;
    case ScalarType::BFloat16: return SPLITKV_DTYPE_BF16;
    case ScalarType::Half: return SPLITKV_DTYPE_F16;
    default: refuse(std::string(name) + " must be float32, bfloat16 or float16");
  }
}

int device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

void dims(const Tensor& t, const char* name, int64_t n, const char* what) {
  if (t.dim() != n) refuse(std::string(name) + " must be " + what);
}

int as_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return int(v);
}

int32_t* status_words(const OptTensor& s, int dev) {
  if (!s) return nullptr;
  dense(*s, "status", {2}, ScalarType::Int, dev);
  return s->data_ptr<int32_t>();
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

void set2(int64_t* out, const Tensor& t) {
  out[0] = t.stride(0);
  out[1] = t.stride(1);
}

// ------------------------------------------------------------------------------------ rotary
// Memory that q's own shape and order of dimensions describe, one element to a place.
Tensor like(const Tensor& t) { return at::empty_like(t); }

py::object rope(const Tensor& positions, const Tensor& freqs, double scale, const Tensor& q, const OptTensor& k,
                const OptTensor& q_out_, const OptTensor& k_out_, bool interleaved, bool adjoint) {
  const int dev = device_of(q, "q");
  splitkv_rope_args a{};
  a.dtype = dtype_code(q, "q");
  const ScalarType dt = q.scalar_type();
  dims(q, "q", 3, "[n, heads, head_dim]");
  const int64_t n = q.size(0), d = q.size(2);
  const bool pos64 = positions.scalar_type() == ScalarType::Long;
  dense(positions, "positions", {n}, pos64 ? ScalarType::Long : ScalarType::Int, dev);
  dense(freqs, "freqs", {freqs.numel()}, ScalarType::Double, dev);
  strided(q, "q", {n, q.size(1), d}, dt, dev);
  if (k) {
    dims(*k, "k", 3, "[n, heads, head_dim]");
    strided(*k, "k", {n, k->size(1), d}, dt, dev);
  }
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const Tensor q_out = q_out_ ? *q_out_ : like(q);
  Tensor k_out;
  if (k) k_out = k_out_ ? *k_out_ : like(*k);
  strided(q_out, "q_out", {n, q.size(1), d}, dt, dev);
  a.num_tokens = n;
  a.q_heads = as_int(q.size(1), "heads");
  a.head_dim = as_int(d, "head_dim");
  a.rotary_dim = as_int(2 * freqs.numel(), "freqs");
  a.flags = (interleaved ? SPLITKV_ROPE_INTERLEAVED : 0) | (adjoint ? SPLITKV_ROPE_ADJOINT : 0) |
            (pos64 ? SPLITKV_ROPE_POS64 : 0);
  a.scale = scale;
  a.positions = positions.const_data_ptr();
  a.freqs = static_cast<const double*>(freqs.const_data_ptr());
  a.q = q.const_data_ptr();
  a.q_out = q_out.data_ptr();
  set2(a.q_stride, q);
  set2(a.q_out_stride, q_out);
  if (k) {
    strided(k_out, "k_out", {n, k->size(1), d}, dt, dev);
    a.k_heads = as_int(k->size(1), "heads");
    a.k = k->const_data_ptr();
    a.k_out = k_out.data_ptr();
    set2(a.k_stride, *k);
    set2(a.k_out_stride, k_out);
  }
  check("splitkv_rope", splitkv_rope(&a, stream_of(dev)));
  if (!k) return py::cast(q_out);
  return py::make_tuple(q_out, k_out);
}

// --------------------------------------------------------------------------- tree attention
std::tuple<Tensor, Tensor> tree_attn(const Tensor& q, const Tensor& kb, const Tensor& vb, const Tensor& node_ptr,
                                     const OptTensor& mask, const Tensor& k_cache, const Tensor& v_cache,
                                     const Tensor& page_table, const Tensor& context_lens, double scale, int64_t max_nodes,
                                     std::optional<ScalarType> out_dtype, const OptTensor& o_, const OptTensor& lse_,
                                     const OptTensor& status, const OptTensor& ws_) {
  const int dev = device_of(q, "q");
  splitkv_tree_args a{};
  a.dtype = dtype_code(q, "q");
  const ScalarType dt = q.scalar_type();
  dims(q, "q", 3, "[nodes, heads, d]");
  dims(k_cache, "k_cache", 4, "[pages, page_size, heads, d]");
  dims(page_table, "page_table", 2, "[seqs, pages]");
  const int64_t nq = q.size(0), hq = q.size(1), d = q.size(2);
  const int64_t pages = k_cache.size(0), page = k_cache.size(1), hkv = k_cache.size(2);
  const int64_t B = page_table.size(0), max_pages = page_table.size(1);
  strided(q, "q", {nq, hq, d}, dt, dev);
  strided(kb, "kb", {nq, hkv, d}, dt, dev);
  strided(vb, "vb", {nq, hkv, d}, dt, dev);
  strided(k_cache, "k_cache", {pages, page, hkv, d}, dt, dev);
  strided(v_cache, "v_cache", {pages, page, hkv, d}, dt, dev);
  strided(page_table, "page_table", {B, max_pages}, ScalarType::Int, dev);
  dense(node_ptr, "node_ptr", {B + 1}, ScalarType::Int, dev);
  dense(context_lens, "context_lens", {B}, ScalarType::Int, dev);
  if (mask) {
    const ScalarType mt = mask->scalar_type();
    if (mt != ScalarType::Bool && mt != ScalarType::Byte) refuse("mask must be bool or uint8");
    if (mask->dim() != 2 || mask->size(1) < max_nodes)
      refuse("mask must be [nodes, columns] with " + std::to_string(max_nodes) + " (max_nodes) columns or more");
    strided(*mask, "mask", {nq, mask->size(1)}, mt, dev);
  }
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const ScalarType odt = o_ ? o_->scalar_type() : out_dtype ? *out_dtype : dt;
  const Tensor o = o_ ? *o_ : at::empty({nq, hq, d}, q.options().dtype(odt));
  const Tensor lse = lse_ ? *lse_ : at::empty({nq, hq}, q.options().dtype(ScalarType::Float));
  dense(o, "o", {nq, hq, d}, odt == dt ? dt : ScalarType::Float, dev);
  dense(lse, "lse", {nq, hq}, ScalarType::Float, dev);
  a.num_seqs = as_int(B, "seqs");
  a.num_nodes = as_int(nq, "nodes");
  a.max_nodes = as_int(max_nodes, "max_nodes");
  a.num_q_heads = as_int(hq, "heads");
  a.num_kv_heads = as_int(hkv, "heads");
  a.head_dim = as_int(d, "d");
  a.o_dtype = odt == dt ? a.dtype : SPLITKV_DTYPE_F32;
  a.page_size = as_int(page, "page_size");
  a.num_pages = as_int(pages, "pages");
  a.max_pages = as_int(max_pages, "pages");
  a.scale = float(scale);
  a.q = q.const_data_ptr();
  a.kb = kb.const_data_ptr();
  a.vb = vb.const_data_ptr();
  a.k_cache = k_cache.const_data_ptr();
  a.v_cache = v_cache.const_data_ptr();
  a.mask = mask ? mask->const_data_ptr() : nullptr;
  a.node_ptr = static_cast<const int32_t*>(node_ptr.const_data_ptr());
  a.context_lens = static_cast<const int32_t*>(context_lens.const_data_ptr());
  a.page_table = static_cast<const int32_t*>(page_table.const_data_ptr());
  a.o = o.data_ptr();
  a.lse = lse.data_ptr<float>();
  a.status = status_words(status, dev);
  set2(a.q_stride, q);
  set2(a.kb_stride, kb);
  set2(a.vb_stride, vb);
  for (int i = 0; i < 3; ++i) {
    a.k_stride[i] = k_cache.stride(i);
    a.v_stride[i] = v_cache.stride(i);
  }
  a.mask_stride = mask ? mask->stride(0) : 0;
  a.table_stride = page_table.stride(0);
  size_t bytes = 0;
  check("splitkv_tree_workspace_size", splitkv_tree_workspace_size(&a, &bytes));
  // without one given, the workspace is this call's own: calls on other streams and captured graphs share nothing
  Tensor ws;
  if (ws_) {
    if (!ws_->is_cuda() || ws_->get_device() != dev || !ws_->is_contiguous())
      refuse("ws must be a contiguous CUDA tensor on the device of the others");
    ws = *ws_;
    bytes = ws.numel() * ws.element_size();
  } else {
    ws = at::empty({int64_t(bytes)}, q.options().dtype(ScalarType::Byte));
  }
  check("splitkv_tree_attn", splitkv_tree_attn(&a, ws.data_ptr(), bytes, stream_of(dev)));
  return {o, lse};
}

// ------------------------------------------------------------------------------ verification
std::tuple<Tensor, Tensor, Tensor> tree_verify(const Tensor& target, const OptTensor& draft, const Tensor& tokens,
                                               const Tensor& parents, const Tensor& node_ptr, const Tensor& u_accept,
                                               const Tensor& u_sample, int64_t max_nodes, int64_t max_path,
                                               const OptTensor& status) {
  const int dev = device_of(target, "target");
  splitkv_verify_args a{};
  a.dtype = dtype_code(target, "target");
  dims(target, "target", 2, "[nodes, vocab]");
  dims(node_ptr, "node_ptr", 1, "[seqs + 1]");
  const int64_t nq = target.size(0), vocab = target.size(1), B = node_ptr.size(0) - 1;
  if (B < 0) refuse("node_ptr must be [seqs + 1]");
  if (max_path < 1) refuse("max_path must be positive");
  const ScalarType dt = target.scalar_type(), tok = tokens.scalar_type();
  strided(target, "target", {nq, vocab}, dt, dev);
  if (draft) strided(*draft, "draft", {nq, vocab}, dt, dev);
  if (tok != ScalarType::Int && tok != ScalarType::Long) refuse("tokens must be int32 or int64");
  dense(tokens, "tokens", {nq}, tok, dev);
  dense(parents, "parents", {nq}, ScalarType::Int, dev);
  dense(node_ptr, "node_ptr", {B + 1}, ScalarType::Int, dev);
  dense(u_accept, "u_accept", {nq}, ScalarType::Float, dev);
  dense(u_sample, "u_sample", {B}, ScalarType::Float, dev);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const Tensor path = at::empty({B, max_path}, parents.options());
  const Tensor count = at::empty({B}, parents.options());
  const Tensor next = at::empty({B}, tokens.options());
  a.num_seqs = as_int(B, "seqs");
  a.num_nodes = as_int(nq, "nodes");
  a.max_nodes = as_int(max_nodes, "max_nodes");
  a.vocab = as_int(vocab, "vocab");
  a.token_int64 = tok == ScalarType::Long;
  a.max_path = as_int(max_path, "max_path");
  a.target = target.const_data_ptr();
  a.draft = draft ? draft->const_data_ptr() : nullptr;
  a.tokens = tokens.const_data_ptr();
  a.parents = static_cast<const int32_t*>(parents.const_data_ptr());
  a.node_ptr = static_cast<const int32_t*>(node_ptr.const_data_ptr());
  a.u_accept = static_cast<const float*>(u_accept.const_data_ptr());
  a.u_sample = static_cast<const float*>(u_sample.const_data_ptr());
  a.path = path.data_ptr<int32_t>();
  a.count = count.data_ptr<int32_t>();
  a.next = next.data_ptr();
  a.status = status_words(status, dev);
  a.target_stride = target.stride(0);
  a.draft_stride = draft ? draft->stride(0) : 0;
  a.path_stride = max_path;
  check("splitkv_tree_verify", splitkv_tree_verify(&a, stream_of(dev)));
  return {path, count, next};
}

// ------------------------------------------------------------------------------------ commit
void tree_commit(const Tensor& k_cache, const Tensor& v_cache, const Tensor& page_table, const Tensor& context_lens,
                 const Tensor& kb, const Tensor& vb, const Tensor& node_ptr, const OptTensor& path, const OptTensor& count,
                 int64_t max_rows, const OptTensor& status) {
  const int dev = device_of(k_cache, "k_cache");
  const ScalarType dt = k_cache.scalar_type();
  const int64_t nd = k_cache.dim(), L = nd - 4;   // L: leading dimensions (0 or 1)
  if ((nd != 4 && nd != 5) || kb.dim() != nd - 1 || page_table.dim() != 2)
    refuse("the caches must be [layers, pages, page_size, heads, d] and kb, vb [layers, nodes, heads, d] (or all without "
           "layers), page_table [seqs, pages]");
  splitkv_commit_args a{};
  const int64_t layers = L ? k_cache.size(0) : 1, pages = k_cache.size(L), page = k_cache.size(L + 1);
  const int64_t hkv = k_cache.size(L + 2), d = k_cache.size(L + 3), nq = kb.size(L);
  const int64_t B = page_table.size(0), max_pages = page_table.size(1);
  for (const auto& [t, name] : {std::pair<const Tensor&, const char*>{k_cache, "k_cache"}, {v_cache, "v_cache"}}) {
    if (L)
      strided(t, name, {layers, pages, page, hkv, d}, dt, dev);
    else
      strided(t, name, {pages, page, hkv, d}, dt, dev);
    for (int64_t i = 0; i < nd; ++i)
      if (t.size(i) > 1 && t.stride(i) == 0) refuse(std::string(name) + " is written: its elements must not share memory");
  }
  for (const auto& [t, name] : {std::pair<const Tensor&, const char*>{kb, "kb"}, {vb, "vb"}}) {
    if (L)
      strided(t, name, {layers, nq, hkv, d}, dt, dev);
    else
      strided(t, name, {nq, hkv, d}, dt, dev);
  }
  strided(page_table, "page_table", {B, max_pages}, ScalarType::Int, dev);
  dense(node_ptr, "node_ptr", {B + 1}, ScalarType::Int, dev);
  dense(context_lens, "context_lens", {B}, ScalarType::Int, dev);
  if (path) {
    if (path->dim() != 2 || path->size(1) < max_rows)
      refuse("path must be [seqs, columns] with " + std::to_string(max_rows) + " (max_rows) columns or more");
    strided(*path, "path", {B, path->size(1)}, ScalarType::Int, dev);
    if (!count) refuse("path needs count");
    dense(*count, "count", {B}, ScalarType::Int, dev);
  }
  a.num_layers = as_int(layers, "layers");
  a.num_seqs = as_int(B, "seqs");
  a.num_nodes = as_int(nq, "nodes");
  a.max_rows = as_int(max_rows, "max_rows");
  a.num_kv_heads = as_int(hkv, "heads");
  a.head_dim = as_int(d, "d");
  a.elem_bytes = int(k_cache.element_size());
  a.page_size = as_int(page, "page_size");
  a.num_pages = as_int(pages, "pages");
  a.max_pages = as_int(max_pages, "pages");
  a.kb = kb.const_data_ptr();
  a.vb = vb.const_data_ptr();
  a.k_cache = k_cache.data_ptr();
  a.v_cache = v_cache.data_ptr();
  a.path = path ? static_cast<const int32_t*>(path->const_data_ptr()) : nullptr;
  a.count = path ? static_cast<const int32_t*>(count->const_data_ptr()) : nullptr;
  a.node_ptr = static_cast<const int32_t*>(node_ptr.const_data_ptr());
  a.context_lens = static_cast<const int32_t*>(context_lens.const_data_ptr());
  a.page_table = static_cast<const int32_t*>(page_table.const_data_ptr());
  a.status = status_words(status, dev);
  for (int i = 0; i < 3; ++i) {   // the layer's stride is 0 without layers
    a.kb_stride[i] = L + i > 0 ? kb.stride(L + i - 1) : 0;
    a.vb_stride[i] = L + i > 0 ? vb.stride(L + i - 1) : 0;
  }
  for (int i = 0; i < 4; ++i) {
    a.k_stride[i] = L + i > 0 ? k_cache.stride(L + i - 1) : 0;
    a.v_stride[i] = L + i > 0 ? v_cache.stride(L + i - 1) : 0;
  }
  a.path_stride = path ? path->stride(0) : 0;
  a.table_stride = page_table.stride(0);
  c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  check("splitkv_tree_commit", splitkv_tree_commit(&a, stream_of(dev)));
}

}  // namespace

PYBIND11_MODULE(_draft_ext, m) {
  m.def("splitkv_rope", &rope, py::arg("positions"), py::arg("freqs"), py::arg("scale"), py::arg("q"), py::arg("k"),
        py::arg("q_out"), py::arg("k_out"), py::arg("interleaved") = false, py::arg("adjoint") = false,
        "q', k' = the rotary positions (adjoint: their transpose) of q [n, Hq, d] and k [n, Hk, d] (or None) at "
        "positions [n]; rotary_dim = 2 * freqs.numel(); outputs are allocated where None is given");
  m.def("splitkv_tree_attn", &tree_attn, py::arg("q"), py::arg("kb"), py::arg("vb"), py::arg("node_ptr"), py::arg("mask"),
        py::arg("k_cache"), py::arg("v_cache"), py::arg("page_table"), py::arg("context_lens"), py::arg("scale"),
        py::arg("max_nodes"), py::arg("out_dtype") = py::none(), py::arg("o") = py::none(), py::arg("lse") = py::none(),
        py::arg("status") = py::none(), py::arg("ws") = py::none(),
        "o, lse = the attention of draft trees over their sequences' cached context and themselves");
  m.def("splitkv_tree_verify", &tree_verify, py::arg("target"), py::arg("draft"), py::arg("tokens"), py::arg("parents"),
        py::arg("node_ptr"), py::arg("u_accept"), py::arg("u_sample"), py::arg("max_nodes"), py::arg("max_path"),
        py::arg("status") = py::none(), "path, count, next = the verification of drafted tokens");
  m.def("splitkv_tree_commit", &tree_commit, py::arg("k_cache"), py::arg("v_cache"), py::arg("page_table"),
        py::arg("context_lens"), py::arg("kb"), py::arg("vb"), py::arg("node_ptr"), py::arg("path"), py::arg("count"),
        py::arg("max_rows"), py::arg("status") = py::none(),
        "copy the path's rows of kb, vb behind each sequence's context in the caches");
}
