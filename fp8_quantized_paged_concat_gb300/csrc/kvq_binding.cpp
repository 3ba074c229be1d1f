// kvq_binding.cpp -- the Python side of the calls that serve a model from the
// per-head NVFP4 cache, as a CPython extension: it checks the torch tensors
// (types, devices, shapes), allocates what the caller left out, and calls the
// C entry point on the tensors' device and the current stream.  These calls
// run once per layer and decoded token, where the same checks in Python take
// several times as long as the kernels: a single-token attention took 33 us
// of host time with them.
//
// The entry points' addresses come from the loaded library (bind), so that
// this module links against no particular build of it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>

#include "kvq.h"

namespace {

struct BadArgument {
  PyObject* type;
  std::string text;
};

[[noreturn]] void bad(const std::string& text) { throw BadArgument{PyExc_ValueError, text}; }
[[noreturn]] void pending() { throw BadArgument{nullptr, ""}; }   // a Python error is set already

struct Library {
  decltype(&kvq_qk_norm_rope) qk_norm_rope = nullptr;
  decltype(&kvq_window_attention_nvfp4_per_head) window = nullptr;
  decltype(&kvq_tree_attention_nvfp4_per_head) tree = nullptr;
  decltype(&kvq_compact_drafts_nvfp4_per_head) compact = nullptr;
  decltype(&kvq_per_head_attention_workspace_bytes) workspace_bytes = nullptr;
  decltype(&kvq_per_head_attention_default_splits) default_splits = nullptr;
  decltype(&kvq_last_error_string) last_error = nullptr;
};
Library lib;

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) bad(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

std::string shape_text(c10::IntArrayRef s) {
  std::ostringstream o;
  o << '[';
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << ']';
  return o.str();
}

// A tensor of that type and rank on device `index`, its innermost stride 1.
void check(const char* name, const at::Tensor& t, at::ScalarType type, int index, int64_t rank) {
  if (t.scalar_type() == type && t.is_cuda() && t.get_device() == index && t.dim() == rank &&
      (t.stride(-1) == 1 || t.size(-1) <= 1))
    return;
  std::ostringstream o;
  o << name << ": expected a CUDA " << type << " tensor of rank " << rank << " with unit inner stride on cuda:" << index
    << ", got " << t.scalar_type() << " of shape " << shape_text(t.sizes()) << ", strides " << shape_text(t.strides())
    << " on " << t.device();
  bad(o.str());
}

void shaped(const char* name, const at::Tensor& t, std::initializer_list<int64_t> shape) {
  const c10::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) bad(std::string(name) + ": expected shape " + shape_text(want) + ", got " + shape_text(t.sizes()));
}

// The device every other tensor of the call has to be on.
int device_of(const char* name, const at::Tensor& t) {
  if (!t.is_cuda()) bad(std::string(name) + ": expected a CUDA tensor");
  return t.get_device();
}

struct Strides {
  int64_t t, h;
};
// Token and head strides of [T, H, D] (a dimension of one element may carry any stride).
Strides head_strides(const at::Tensor& x) {
  const int64_t h = x.size(1) > 1 ? x.stride(1) : x.size(2);
  return {x.size(0) > 1 ? x.stride(0) : x.size(1) * h, h};
}
int64_t row_stride(const at::Tensor& x) { return x.size(0) > 1 ? x.stride(0) : x.size(1); }

int64_t integer(const char* name, PyObject* o, int64_t lo, int64_t hi) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) pending();
  if (v < lo || v > hi) bad(std::string(name) + ": out of range");
  return v;
}
int32_t int32(const char* name, PyObject* o) { return static_cast<int32_t>(integer(name, o, INT32_MIN, INT32_MAX)); }

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) pending();
  return static_cast<float>(v);
}

int32_t* status_word(PyObject* o, int index) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor("status", o);
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != index || t.numel() < 1)
    bad("status: expected an int32 tensor with at least one element on cuda:" + std::to_string(index));
  return static_cast<int32_t*>(t.data_ptr());
}

// The stream of the call: the current one of the device, a torch stream, or a raw handle.
cudaStream_t stream_of(PyObject* o, int index) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(index).stream();
  PyObject* handle = o;
  PyObject* owned = nullptr;
  if (!PyLong_Check(o)) {
    PyObject* at = PyObject_GetAttrString(o, "device_index");
    if (at == nullptr) pending();
    const long on = PyLong_AsLong(at);
    Py_DECREF(at);
    if (on == -1 && PyErr_Occurred()) pending();
    if (on != index) bad("stream: expected a stream of cuda:" + std::to_string(index) + ", the tensors' device");
    handle = owned = PyObject_GetAttrString(o, "cuda_stream");
    if (handle == nullptr) pending();
  }
  void* p = PyLong_AsVoidPtr(handle);
  Py_XDECREF(owned);
  if (p == nullptr && PyErr_Occurred()) pending();
  return static_cast<cudaStream_t>(p);
}

// Where a call runs: its tensors' device, and its stream.  What the call
// allocates comes from that stream's memory, so that nothing else still uses
// it and a workspace can be freed on return; results are known to the caller's
// current stream as well, and may be freed there.
class Scope {
 public:
  Scope(PyObject* stream_object, int dev) : device_(static_cast<c10::DeviceIndex>(dev)) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(dev);
    raw_ = stream_of(stream_object, dev);
    if (raw_ == current.stream()) return;
    callers_ = current;
    const auto index = static_cast<c10::DeviceIndex>(dev);
    guard_.reset_stream(raw_ == nullptr ? c10::cuda::getDefaultCUDAStream(index)
                                        : c10::cuda::getStreamFromExternal(raw_, index));
  }
  kvq_stream_t stream() const { return reinterpret_cast<kvq_stream_t>(raw_); }
  // (created here, not through the dispatcher: 1.0 against 1.3 us each)
  at::Tensor buffer(c10::IntArrayRef shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, device_.current_device().index()),
                                             std::nullopt));
  }
  at::Tensor result(c10::IntArrayRef shape, at::ScalarType type) const {
    at::Tensor t = buffer(shape, type);
    if (callers_) t.record_stream(*callers_);
    return t;
  }

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
  std::optional<c10::cuda::CUDAStream> callers_;
  cudaStream_t raw_ = nullptr;
};

struct CacheShape {
  int32_t layout, block_size, heads, head_size;
};
// A contiguous per-head cache (its last five dimensions, from `from` on).
CacheShape cache_shape(const at::Tensor& cache, int64_t from, PyObject* layout, int64_t head_size) {
  const bool nhd = PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "NHD") == 0;
  if (!nhd && !(PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "HND") == 0))
    bad("layout: expected one of ['HND', 'NHD']");
  const auto s = cache.sizes().slice(from), st = cache.strides().slice(from);
  bool contiguous = true;
  int64_t expect = 1;
  for (int i = 4; i >= 0; --i) {
    contiguous = contiguous && (s[i] <= 1 || st[i] == expect);
    expect *= s[i];
  }
  const int64_t full = s[4], block = nhd ? s[2] : s[3], heads = nhd ? s[3] : s[2];
  if (s[1] != 2 || !contiguous || full % 9 != 0 || (head_size >= 0 && full * 16 != head_size * 9) || block > INT32_MAX ||
      heads > INT32_MAX || full > INT32_MAX / 16)
    bad(std::string("kv_cache: expected a contiguous [P, 2, ") + (nhd ? "block_size, H" : "H, block_size") +
        ", D/2 + D/16] tensor" + (head_size >= 0 ? " with D = " + std::to_string(head_size) : std::string()) + ", got " +
        shape_text(cache.sizes()));
  return {nhd ? 0 : 1, static_cast<int32_t>(block), static_cast<int32_t>(heads), static_cast<int32_t>(full / 9 * 16)};
}

void must(kvq_status status, const char* name) {
  if (status == KVQ_OK) return;
  throw BadArgument{PyExc_RuntimeError,
                    std::string(name) + " failed (status " + std::to_string(status) + "): " + lib.last_error()};
}

int32_t dim(int64_t v) {
  if (v > INT32_MAX) bad("a dimension exceeds 2^31 - 1");
  return static_cast<int32_t>(v);
}

const float* scale_word(const char* name, PyObject* o, int index) {
  const at::Tensor& t = tensor(name, o);
  if (t.scalar_type() != at::kFloat || !t.is_cuda() || t.get_device() != index || t.numel() < 1)
    bad(std::string(name) + ": expected an fp32 scalar on cuda:" + std::to_string(index));
  return static_cast<const float*>(t.data_ptr());
}

// Runs a call's body; C++ exceptions become Python ones.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  try {
    if (lib.window == nullptr) throw BadArgument{PyExc_RuntimeError, "the library is not bound"};
    if (got != want) throw BadArgument{PyExc_TypeError, "wrong number of arguments"};
    return body();
  } catch (const BadArgument& e) {
    if (e.type != nullptr) PyErr_SetString(e.type, e.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* pair(const at::Tensor& a, const at::Tensor* b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = b != nullptr ? THPVariable_Wrap(*b) : Py_NewRef(Py_None);
  if (x == nullptr || y == nullptr) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_DECREF(x);
  Py_DECREF(y);
  return r;
}

// q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, q_out, k_out, status, stream
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor& q = tensor("q", a[0]);
    const int dev = device_of("q", q);
    check("q", q, at::kBFloat16, dev, 3);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    const at::Tensor& k = tensor("k", a[1]);
    check("k", k, at::kBFloat16, dev, 3);
    const int64_t KH = k.size(1);
    shaped("k", k, {T, KH, D});
    const at::Tensor &qw = tensor("q_weight", a[2]), &kw = tensor("k_weight", a[3]);
    check("q_weight", qw, at::kBFloat16, dev, 1);
    check("k_weight", kw, at::kBFloat16, dev, 1);
    shaped("q_weight", qw, {D});
    shaped("k_weight", kw, {D});
    const at::Tensor& pos = tensor("positions", a[4]);
    check("positions", pos, at::kLong, dev, 1);
    shaped("positions", pos, {T});
    const at::Tensor& table = tensor("cos_sin", a[5]);
    check("cos_sin", table, at::kFloat, dev, 2);
    const float eps = real(a[6]);
    const int interleaved = PyObject_IsTrue(a[7]);
    if (interleaved < 0) pending();
    const Scope scope(a[11], dev);
    const at::Tensor qo = a[8] == Py_None ? scope.result({T, H, D}, at::kBFloat16) : tensor("q_out", a[8]);
    const at::Tensor ko = a[9] == Py_None ? scope.result({T, KH, D}, at::kBFloat16) : tensor("k_out", a[9]);
    check("q_out", qo, at::kBFloat16, dev, 3);
    check("k_out", ko, at::kBFloat16, dev, 3);
    shaped("q_out", qo, {T, H, D});
    shaped("k_out", ko, {T, KH, D});
    const Strides sq = head_strides(q), sk = head_strides(k), sqo = head_strides(qo), sko = head_strides(ko);
    must(lib.qk_norm_rope(q.data_ptr(), sq.t, sq.h, k.data_ptr(), sk.t, sk.h, qw.data_ptr(), kw.data_ptr(),
                          static_cast<const int64_t*>(pos.data_ptr()), T, dim(H), dim(KH), dim(D),
                          static_cast<const float*>(table.data_ptr()), row_stride(table), table.size(0),
                          dim(table.size(1)), interleaved, eps, qo.data_ptr(), sqo.t, sqo.h, ko.data_ptr(), sko.t, sko.h,
                          status_word(a[10], dev), scope.stream()),
         "kvq_qk_norm_rope");
    return pair(qo, &ko);
  });
}

// q, query_start, seq_lens, tree_mask (None: window form), block_table, kv_cache, k_scale, v_scale, softmax_scale,
// max_query_len, max_seq_len, window, num_sinks, layout, num_splits, workspace, out, lse, status, stream
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 20, [&]() -> PyObject* {
    const at::Tensor& q = tensor("q", a[0]);
    const int dev = device_of("q", q);
    check("q", q, at::kBFloat16, dev, 3);
    const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
    const at::Tensor& start = tensor("query_start", a[1]);
    const at::Tensor& lens = tensor("seq_lens", a[2]);
    check("seq_lens", lens, at::kInt, dev, 1);
    const int64_t B = lens.size(0);
    check("query_start", start, at::kInt, dev, 1);
    shaped("query_start", start, {B + 1});
    const at::Tensor& table = tensor("block_table", a[4]);
    check("block_table", table, at::kInt, dev, 2);
    const int64_t W = table.size(1);
    shaped("block_table", table, {B, W});
    const at::Tensor& cache = tensor("kv_cache", a[5]);
    check("kv_cache", cache, at::kByte, dev, 5);
    const CacheShape c = cache_shape(cache, 0, a[13], D);
    const float *ks = scale_word("k_scale", a[6], dev), *vs = scale_word("v_scale", a[7], dev);
    const float scale = real(a[8]);
    const int32_t max_query = int32("max_query_len", a[9]), max_seq = int32("max_seq_len", a[10]);
    const int32_t window = int32("window", a[11]), sinks = int32("num_sinks", a[12]);
    const bool tree = a[3] != Py_None;
    const Scope scope(a[19], dev);
    const at::Tensor out = a[16] == Py_None ? scope.result({T, H, D}, at::kBFloat16) : tensor("out", a[16]);
    check("out", out, at::kBFloat16, dev, 3);
    shaped("out", out, {T, H, D});
    const bool want_lse = a[17] != Py_False;
    at::Tensor lse;
    if (want_lse) {
      lse = a[17] == Py_None ? scope.result({T, H}, at::kFloat) : tensor("lse", a[17]);
      check("lse", lse, at::kFloat, dev, 2);
      shaped("lse", lse, {T, H});
    }
    // the ranges of a block join in a cluster, or through a workspace
    int32_t use_workspace = 0;
    int32_t splits;
    if (a[14] == Py_None) {
      splits = lib.default_splits(max_query, dim(H), c.heads, c.head_size, dim(B), max_seq, window, sinks, tree,
                                  &use_workspace);
    } else {
      splits = int32("num_splits", a[14]);
      use_workspace = splits > KVQ_PER_HEAD_CLUSTER_SPLITS ||
                      (splits > 1 && c.heads > 0 && max_query * (H / c.heads) > KVQ_PER_HEAD_CLUSTER_ROWS);
    }
    at::Tensor workspace;
    if (a[15] != Py_None) {
      const at::Tensor& given = tensor("workspace", a[15]);
      if (!given.is_cuda() || given.get_device() != dev || !given.is_contiguous())
        bad("workspace: expected a contiguous tensor on cuda:" + std::to_string(dev));
      // default ranges that join without one run without it
      if (use_workspace || a[14] != Py_None) workspace = given;
    } else if (use_workspace && T > 0) {
      const int64_t bytes = lib.workspace_bytes(T, dim(H), c.head_size, splits);
      if (bytes > 0) workspace = scope.buffer({bytes}, at::kByte);
    }
    void* ws = workspace.defined() ? workspace.data_ptr() : nullptr;
    const int64_t ws_bytes = workspace.defined() ? workspace.numel() * static_cast<int64_t>(workspace.element_size()) : 0;
    const Strides sq = head_strides(q), so = head_strides(out);
    float* lse_ptr = want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
    const int64_t lse_stride = want_lse ? row_stride(lse) : 0;
    int32_t* status = status_word(a[18], dev);
    const kvq_stream_t stream = scope.stream();
    const auto* start_p = static_cast<const int32_t*>(start.data_ptr());
    const auto* lens_p = static_cast<const int32_t*>(lens.data_ptr());
    const auto* table_p = static_cast<const int32_t*>(table.data_ptr());
    const auto* cache_p = static_cast<const uint8_t*>(cache.data_ptr());
    if (tree) {
      const at::Tensor& mask = tensor("tree_mask", a[3]);
      check("tree_mask", mask, at::kLong, dev, 2);
      shaped("tree_mask", mask, {T, mask.size(1)});
      must(lib.tree(q.data_ptr(), sq.t, sq.h, T, dim(H), start_p, lens_p, dim(B), max_query,
                    static_cast<const uint64_t*>(mask.data_ptr()), row_stride(mask), dim(mask.size(1)), table_p,
                    row_stride(table), dim(W), cache_p, cache.size(0), c.block_size, c.layout, c.heads, c.head_size, ks,
                    vs, scale, out.data_ptr(), so.t, so.h, lse_ptr, lse_stride, max_seq, splits, ws, ws_bytes, status,
                    stream),
           "kvq_tree_attention_nvfp4_per_head");
    } else {
      must(lib.window(q.data_ptr(), sq.t, sq.h, T, dim(H), start_p, lens_p, dim(B), max_query, table_p,
                      row_stride(table), dim(W), cache_p, cache.size(0), c.block_size, c.layout, c.heads, c.head_size, ks,
                      vs, scale, window, sinks, out.data_ptr(), so.t, so.h, lse_ptr, lse_stride, max_seq, splits, ws,
                      ws_bytes, status, stream),
           "kvq_window_attention_nvfp4_per_head");
    }
    return pair(out, want_lse ? &lse : nullptr);
  });
}

// kv_cache, query_start, seq_lens, accepted, accepted_lens, block_table, layout, status, stream
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& cache = tensor("kv_cache", a[0]);
    const int dev = device_of("kv_cache", cache);
    if (cache.dim() != 5 && cache.dim() != 6) bad("kv_cache: expected a [P, 2, ...] or [L, P, 2, ...] tensor");
    check("kv_cache", cache, at::kByte, dev, cache.dim());
    const bool many = cache.dim() == 6;
    const int64_t layers = many ? cache.size(0) : 1;
    const CacheShape c = cache_shape(cache, many ? 1 : 0, a[6], -1);
    const at::Tensor& lens = tensor("seq_lens", a[2]);
    check("seq_lens", lens, at::kInt, dev, 1);
    const int64_t B = lens.size(0);
    const at::Tensor &start = tensor("query_start", a[1]), &counts = tensor("accepted_lens", a[4]);
    check("query_start", start, at::kInt, dev, 1);
    shaped("query_start", start, {B + 1});
    check("accepted_lens", counts, at::kInt, dev, 1);
    shaped("accepted_lens", counts, {B});
    const at::Tensor &accepted = tensor("accepted", a[3]), &table = tensor("block_table", a[5]);
    check("accepted", accepted, at::kInt, dev, 2);
    shaped("accepted", accepted, {B, accepted.size(1)});
    check("block_table", table, at::kInt, dev, 2);
    shaped("block_table", table, {B, table.size(1)});
    const Scope scope(a[8], dev);
    must(lib.compact(static_cast<uint8_t*>(cache.data_ptr()), dim(layers), many ? cache.stride(0) : 0,
                     cache.size(many ? 1 : 0), c.block_size, c.layout, c.heads, c.head_size,
                     static_cast<const int32_t*>(start.data_ptr()), static_cast<const int32_t*>(lens.data_ptr()), dim(B),
                     static_cast<const int32_t*>(accepted.data_ptr()), row_stride(accepted),
                     static_cast<const int32_t*>(counts.data_ptr()), dim(accepted.size(1)),
                     static_cast<const int32_t*>(table.data_ptr()), row_stride(table), dim(table.size(1)),
                     status_word(a[7], dev), scope.stream()),
         "kvq_compact_drafts_nvfp4_per_head");
    Py_RETURN_NONE;
  });
}

// bind({entry point: address}): the library whose entry points the calls use
PyObject* bind(PyObject*, PyObject* table) {
  Library found;
  const auto set = [&](const char* name, auto& fn) {
    PyObject* v = PyMapping_GetItemString(table, name);
    if (v == nullptr) return false;
    fn = reinterpret_cast<std::decay_t<decltype(fn)>>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    if (fn == nullptr && !PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s has no address", name);
    return fn != nullptr;
  };
  if (!set("kvq_qk_norm_rope", found.qk_norm_rope) || !set("kvq_window_attention_nvfp4_per_head", found.window) ||
      !set("kvq_tree_attention_nvfp4_per_head", found.tree) ||
      !set("kvq_compact_drafts_nvfp4_per_head", found.compact) ||
      !set("kvq_per_head_attention_workspace_bytes", found.workspace_bytes) ||
      !set("kvq_per_head_attention_default_splits", found.default_splits) ||
      !set("kvq_last_error_string", found.last_error))
    return nullptr;
  lib = found;
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_O, "bind({entry point: address})"},
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm_rope)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attention)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvq_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kvq_native() { return PyModule_Create(&module); }
