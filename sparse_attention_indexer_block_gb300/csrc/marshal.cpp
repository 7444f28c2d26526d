// Argument marshalling of the calls that run once a layer and step (attention,
// appends, trees): torch tensors to the functions of indexer.h. The work of a
// single call is some microseconds on the device, and reading a tensor's shape,
// strides, type and address from Python takes ten times as long as the call, so it
// is done here (one token appended with its queries, a call: 22 us from Python,
// 15 with the checks laid out for speed, 5.6 from here). Every refusal is an
// IndexerError, as in binding.py, which holds the functions' documentation.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include <cmath>
#include <initializer_list>
#include <string>
#include <type_traits>
#include <vector>

#include "../../include/indexer.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // IndexerError

// The functions of the library that the binding has loaded.
struct Library {
  decltype(&indexer_attend_paged) attend_paged;
  decltype(&indexer_attend_selected) attend_selected;
  decltype(&indexer_attend_tree) attend_tree;
  decltype(&indexer_attend_workspace_bytes) attend_workspace_bytes;
  decltype(&indexer_append_kv) append_kv;
  decltype(&indexer_insert_keys_mxfp4) insert_keys_mxfp4;
  decltype(&indexer_plan_tree) plan_tree;
  decltype(&indexer_commit_tree) commit_tree;
  decltype(&indexer_last_cuda_error) last_cuda_error;
};
Library g_lib = {};

struct Refusal {
  idx_status status;
  std::string what;
};
struct PythonError {};  // a Python exception is set

[[noreturn]] void refuse(const std::string& what, idx_status status = IDX_ERR_INVALID_ARG) {
  throw Refusal{status, what};
}

std::string shape_text(const Tensor& t) {
  std::string s = "(";
  for (int64_t n : t.sizes()) s += std::to_string(n) + ", ";
  return s + ")";
}

// ---------------------------------------------------------------------------
// arguments
// ---------------------------------------------------------------------------

const Tensor* maybe(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

const Tensor& tensor(PyObject* o, const char* what) {
  const Tensor* t = maybe(o, what);
  if (!t) refuse(std::string(what) + " is missing");
  return *t;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

// A number in [least, 2^31).
int32_t count(PyObject* o, const char* what, int64_t least = 0) {
  const int64_t v = integer(o);
  if (v < least || v > INT32_MAX) refuse(std::string(what) + " " + std::to_string(v));
  return static_cast<int32_t>(v);
}

// A contiguous tensor [n] of that type (n < 0: any size).
void need_vector(const Tensor& t, const char* what, at::ScalarType type, int64_t n) {
  if (t.scalar_type() != type) refuse(std::string(what) + " must be a tensor of " + at::toString(type));
  if (t.dim() != 1 || (n >= 0 && t.size(0) != n)) refuse(std::string(what) + " has shape " + shape_text(t));
  if (!t.is_contiguous()) refuse(std::string(what) + " must be contiguous");
}

// An int32 matrix of n rows (n < 0: any), contiguous in its columns.
void need_matrix(const Tensor& t, const char* what, int64_t n) {
  if (t.scalar_type() != at::kInt) refuse(std::string(what) + " must be an int32 tensor");
  if (t.dim() != 2 || (n >= 0 && t.size(0) != n)) refuse(std::string(what) + " has shape " + shape_text(t));
  if (!t.is_contiguous() && t.stride(1) != 1 && t.size(1) > 1)
    refuse(std::string(what) + " must be contiguous in its last dimension");
}

// Row stride of a matrix whose rows must not overlap.
int64_t row_stride(const Tensor& t, const char* what) {
  if (t.size(0) <= 1) return t.size(1);
  if (t.stride(0) < t.size(1)) refuse(std::string(what) + "'s rows overlap");
  return t.stride(0);
}

void need_error(const Tensor* e) {
  if (e && (e->element_size() != 4 || e->numel() < 1)) refuse("dev_error must be a tensor of a 32-bit word");
}

int need_device(std::initializer_list<const Tensor*> all) {
  const Tensor* first = *all.begin();
  if (!first->is_cuda()) refuse("tensors must be on a CUDA device");
  const int index = first->get_device();
  for (const Tensor* t : all)
    if (t && (!t->is_cuda() || t->get_device() != index)) refuse("tensors are on different devices");
  return index;
}

template <typename T>
T* at_of(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* at_of(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// The stream a call runs on, and is to allocate on: the current one of the tensors' device, or the
// caller's (a torch.cuda.Stream or a handle).
class On {
 public:
  On(int index, PyObject* stream) {
    if (stream == Py_None) {
      if (c10::cuda::current_device() != index) device_.set_index(static_cast<c10::DeviceIndex>(index));
      stream_ = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
      return;
    }
    void* handle;
    if (PyLong_Check(stream)) {
      handle = PyLong_AsVoidPtr(stream);
    } else {
      PyObject* of = PyObject_GetAttrString(stream, "device_index");
      if (!of) throw PythonError{};
      const long device = PyLong_AsLong(of);
      Py_DECREF(of);
      if (device != index && !PyErr_Occurred()) refuse("the stream is of another device than the tensors");
      PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
      if (!h) throw PythonError{};
      handle = PyLong_AsVoidPtr(h);
      Py_DECREF(h);
    }
    if (PyErr_Occurred()) throw PythonError{};
    stream_ = static_cast<cudaStream_t>(handle);
    given_.reset_stream(c10::cuda::getStreamFromExternal(stream_, static_cast<c10::DeviceIndex>(index)));
  }
  cudaStream_t stream() const { return stream_; }

 private:
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard given_;
  cudaStream_t stream_ = nullptr;
};

// Lets go of the interpreter's lock: an allocation may wait for the device, and so may a launch.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  const at::TensorOptions options = at::TensorOptions().dtype(type).device(like.device());
  const Unlocked unlocked;
  return at::empty(shape, options);
}

// Runs a function of the library without the interpreter's lock.
template <typename F>
idx_status unlocked(const F& f) {
  const Unlocked unlocked;
  return f();
}

void check(idx_status st) {
  if (st != IDX_OK) throw Refusal{st, st == IDX_ERR_CUDA ? g_lib.last_cuda_error() : ""};
}

// A new reference to a result: the caller's own object, or a new tensor's.
PyObject* result(PyObject* given, const Tensor& made) {
  if (given == Py_None) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}

// Calls f and turns what it throws into Python exceptions (what torch throws into torch's own:
// OutOfMemoryError among them).
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, const F& f) {
  if (n != want) return PyErr_Format(PyExc_TypeError, "%s: %zd arguments, not %zd", name, n, want);
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal& r) {
    PyObject* e = PyObject_CallFunction(g_error, "sis", name, static_cast<int>(r.status), r.what.c_str());
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  } catch (const PythonError&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

int32_t type_code(const Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return IDX_BF16;
  if (t.scalar_type() == at::kHalf) return IDX_FP16;
  refuse(std::string(what) + " is " + at::toString(t.scalar_type()) + ", not bfloat16 or float16", IDX_ERR_UNSUPPORTED);
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------

enum Form { kPaged, kSelected, kTree };

// (request or token, kv head) pairs: calls of more always use a workspace
constexpr int64_t kFewUnits = 304;

PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  static const char* const names[] = {"indexer_attend_paged", "indexer_attend_selected", "indexer_attend_tree"};
  const long form = n > 0 ? PyLong_AsLong(a[0]) : -1;
  if (form < kPaged || form > kTree) return PyErr_Format(PyExc_TypeError, "attend: form %ld", form);
  return guarded(names[form], n, 19, [&]() -> PyObject* {
    const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k_cache"), &v = tensor(a[3], "v_cache");
    const Tensor &table = tensor(a[4], "block_table"), &start = tensor(a[5], "query_start_loc");
    const Tensor *lens = maybe(a[6], "seq_lens"), *indices = maybe(a[7], "indices");
    const Tensor *out = maybe(a[9], "out"), *lse = maybe(a[10], "lse"), *ws = maybe(a[11], "workspace");
    const Tensor *error = maybe(a[12], "dev_error"), *masks = maybe(a[17], "masks");
    const Tensor* positions = maybe(a[18], "positions");
    if (q.dim() != 3 || k.dim() != 4 || v.dim() != 4)
      refuse("q must have 3 dimensions, k_cache and v_cache 4");
    idx_attend c{};
    c.dtype = type_code(q, "q");
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
      refuse("q, k_cache and v_cache differ in type");
    const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2), kv_heads = k.size(2);
    if (v.sizes() != k.sizes() || k.size(3) != dim)
      refuse("k_cache and v_cache must be [pages, 64, kv heads, head_dim of q]");
    if (k.size(1) != IDX_PAGE_TOKENS)
      refuse("pages of " + std::to_string(k.size(1)) + " tokens, not 64", IDX_ERR_UNSUPPORTED);
    if (dim != 64 && dim != 128)
      refuse("head_dim " + std::to_string(dim) + ", not 64 or 128", IDX_ERR_UNSUPPORTED);
    if (kv_heads < 1 || heads < 1 || heads % kv_heads)
      refuse(std::to_string(heads) + " heads over " + std::to_string(kv_heads) + " kv heads");
    if (q.stride(2) != 1 || k.stride(3) != 1 || v.stride(3) != 1)
      refuse("q, k_cache and v_cache must be contiguous in their last dimension");
    need_vector(start, "query_start_loc", at::kInt, -1);
    const int64_t reqs = start.size(0) - 1;
    if (reqs < 0) refuse("query_start_loc is empty");
    need_matrix(table, "block_table", reqs);
    if (table.size(1) < 1) refuse("block_table has no columns");
    c.bt_stride = row_stride(table, "block_table");
    if (form != kSelected) need_vector(tensor(a[6], "seq_lens"), "seq_lens", at::kInt, reqs);
    if (form == kSelected) {
      need_matrix(tensor(a[7], "indices"), "indices", tokens);
      if (indices->size(1) < 1) refuse("indices has no columns");
      c.indices_stride = tokens > 1 ? indices->stride(0) : indices->size(1);
      c.topk = static_cast<int32_t>(indices->size(1));
    }
    if (out && (out->sizes() != q.sizes() || out->scalar_type() != q.scalar_type() || !out->is_contiguous()))
      refuse("out must be a contiguous tensor of q's shape and type");
    if (lse && (lse->dim() != 2 || lse->size(0) != tokens || lse->size(1) != heads ||
                lse->scalar_type() != at::kFloat || !lse->is_contiguous()))
      refuse("lse must be a contiguous float32 tensor [tokens, heads]");
    c.max_query_len = count(a[14], "max_query_len");
    c.window = count(a[15], "window");
    c.sinks = count(a[16], "sinks");
    int64_t mask_stride = 0, words = 0;
    if (form == kTree) {
      need_matrix(tensor(a[17], "masks"), "masks", tokens);
      words = masks->size(1);
      if (words < 1) refuse("masks has no columns");
      mask_stride = row_stride(*masks, "masks");
      if (positions) need_vector(*positions, "positions", at::kInt, tokens);
      else if (c.window) refuse("a window needs positions");
    }
    need_error(error);
    if (tokens > INT32_MAX || heads > INT32_MAX || reqs > INT32_MAX || table.size(1) > INT32_MAX || words > INT32_MAX)
      refuse("sizes past 32 bits", IDX_ERR_UNSUPPORTED);
    c.scale = static_cast<float>(a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(dim)) : PyFloat_AsDouble(a[8]));
    if (PyErr_Occurred()) throw PythonError{};
    const int index =
        need_device({&q, &k, &v, &table, &start, lens, indices, out, lse, ws, error, masks, positions});
    const On on(index, a[13]);
    const Tensor made_out = out ? Tensor() : fresh(q.sizes(), q.scalar_type(), q);
    const Tensor made_lse = lse ? Tensor() : fresh({tokens, heads}, at::kFloat, q);
    c.q = q.data_ptr();
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.block_table = at_of<const int32_t>(table);
    c.seq_lens = at_of<const int32_t>(lens);
    c.query_start_loc = at_of<const int32_t>(start);
    c.indices = at_of<const int32_t>(indices);
    c.out = (out ? *out : made_out).data_ptr();
    c.lse = at_of<float>(lse ? *lse : made_lse);
    c.dev_error = at_of<uint32_t>(error);
    c.q_stride_token = q.stride(0);
    c.q_stride_head = q.stride(1);
    c.k_stride_page = k.stride(0);
    c.k_stride_token = k.stride(1);
    c.k_stride_head = k.stride(2);
    c.v_stride_page = v.stride(0);
    c.v_stride_token = v.stride(1);
    c.v_stride_head = v.stride(2);
    c.num_pages = k.size(0);
    c.bt_width = static_cast<int32_t>(table.size(1));
    c.num_reqs = static_cast<int32_t>(reqs);
    c.num_tokens = static_cast<int32_t>(tokens);
    c.num_heads = static_cast<int32_t>(heads);
    c.num_kv_heads = static_cast<int32_t>(kv_heads);
    c.head_dim = static_cast<int32_t>(dim);
    const auto run = [&](void* at, size_t bytes) {
      c.workspace = at;
      c.workspace_bytes = bytes;
      return unlocked([&] {
        return form == kPaged      ? g_lib.attend_paged(&c, on.stream())
               : form == kSelected ? g_lib.attend_selected(&c, on.stream())
                                   : g_lib.attend_tree(&c, at_of<const int32_t>(masks), mask_stride,
                                                         static_cast<int32_t>(words),
                                                         at_of<const int32_t>(positions), on.stream());
      });
    };
    if (ws) {
      check(run(ws->data_ptr(), ws->nbytes()));
    } else {
      // (small steps need no workspace: the call says so)
      idx_status st = IDX_ERR_WORKSPACE;
      if ((form == kSelected ? tokens : reqs) * kv_heads <= kFewUnits) st = run(nullptr, 0);
      if (st == IDX_ERR_WORKSPACE) {
        size_t bytes = 0;
        check(g_lib.attend_workspace_bytes(c.num_tokens, c.num_reqs, c.num_heads, c.num_kv_heads, c.head_dim,
                                             &bytes));
        const Tensor made = fresh({static_cast<int64_t>(bytes)}, at::kByte, q);
        st = run(made.data_ptr(), bytes);
      }
      check(st);
    }
    PyObject* r = PyTuple_New(2);
    if (!r) throw PythonError{};
    PyTuple_SET_ITEM(r, 0, result(a[9], made_out));
    PyTuple_SET_ITEM(r, 1, result(a[10], made_lse));
    return r;
  });
}

// ---------------------------------------------------------------------------
// new tokens into the caches
// ---------------------------------------------------------------------------

PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("indexer_append_kv", n, 12, [&]() -> PyObject* {
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
    const Tensor& slots = tensor(a[4], "slot_mapping");
    const Tensor *q = maybe(a[5], "q"), *positions = maybe(a[6], "positions"), *rotary = maybe(a[7], "rotary");
    const Tensor *q_out = maybe(a[9], "q_out"), *error = maybe(a[10], "dev_error");
    if (k.dim() != 3 || kc.dim() != 4) refuse("k and v must have 3 dimensions, k_cache and v_cache 4");
    idx_append c{};
    c.dtype = type_code(k, "k");
    const at::ScalarType type = k.scalar_type();
    if (v.scalar_type() != type || kc.scalar_type() != type || vc.scalar_type() != type)
      refuse("k, v, k_cache and v_cache differ in type");
    const int64_t tokens = k.size(0), kv_heads = k.size(1), dim = k.size(2);
    if (dim != 64 && dim != 128)
      refuse("head_dim " + std::to_string(dim) + ", not 64 or 128", IDX_ERR_UNSUPPORTED);
    if (v.sizes() != k.sizes() || kc.size(2) != kv_heads || kc.size(3) != dim || vc.sizes() != kc.sizes())
      refuse("k and v must be [tokens, kv heads, dim], the caches [pages, 64, kv heads, dim]");
    if (kc.size(1) != IDX_PAGE_TOKENS)
      refuse("pages of " + std::to_string(kc.size(1)) + " tokens, not 64", IDX_ERR_UNSUPPORTED);
    if (k.stride(2) != 1 || v.stride(2) != 1 || kc.stride(3) != 1 || vc.stride(3) != 1)
      refuse("k, v, k_cache and v_cache must be contiguous in their last dimension");
    need_vector(slots, "slot_mapping", at::kLong, tokens);
    if (!rotary) {
      if (q || positions || q_out) refuse("q, positions and q_out belong to a rotation");
    } else {
      if (rotary->scalar_type() != at::kFloat || rotary->dim() != 2)
        refuse("rotary must be a float32 tensor [positions, rotary_dim]");
      const int64_t turned = rotary->size(1);
      if (turned < 16 || turned % 16 || turned > dim)
        refuse("rotary_dim " + std::to_string(turned) + ", not a multiple of 16 up to " + std::to_string(dim),
               IDX_ERR_UNSUPPORTED);
      if (rotary->stride(1) != 1) refuse("rotary must be contiguous in its last dimension");
      need_vector(tensor(a[6], "positions"), "positions", at::kInt, tokens);
      c.rotary_dim = static_cast<int32_t>(turned);
      c.num_positions = rotary->size(0);
      c.rotary_stride = c.num_positions == 1 ? turned : rotary->stride(0);
      const int interleaved = PyObject_IsTrue(a[8]);
      if (interleaved < 0) throw PythonError{};
      c.interleaved = interleaved;
      if (q) {
        if (q->scalar_type() != type || q->dim() != 3 || q->size(0) != tokens || q->size(1) < 1 || q->size(2) != dim)
          refuse("q must be a tensor [tokens, heads, dim] of k's type");
        if (q->stride(2) != 1) refuse("q must be contiguous in its last dimension");
        if (q_out) {
          if (q_out->sizes() != q->sizes() || q_out->scalar_type() != type) refuse("q_out must be a tensor like q");
          if (q_out->stride(2) != 1) refuse("q_out must be contiguous in its last dimension");
        }
      } else if (q_out) {
        refuse("q_out without q");
      }
    }
    need_error(error);
    if (tokens > INT32_MAX || kv_heads > INT32_MAX || (q && q->size(1) > INT32_MAX))
      refuse("sizes past 32 bits", IDX_ERR_UNSUPPORTED);
    const int index = need_device({&k, &v, &kc, &vc, &slots, q, positions, rotary, q_out, error});
    const On on(index, a[11]);
    Tensor made;
    if (q) {
      if (!q_out) made = fresh(q->sizes(), type, *q);
      const Tensor& o = q_out ? *q_out : made;
      c.q = q->data_ptr();
      c.q_out = o.data_ptr();
      c.num_heads = static_cast<int32_t>(q->size(1));
      c.q_stride_token = q->stride(0);
      c.q_stride_head = q->stride(1);
      c.q_out_stride_token = o.stride(0);
      c.q_out_stride_head = o.stride(1);
    }
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.slot_mapping = at_of<const int64_t>(slots);
    c.positions = at_of<const int32_t>(positions);
    c.rotary = at_of<const float>(rotary);
    c.k_cache = kc.data_ptr();
    c.v_cache = vc.data_ptr();
    c.dev_error = at_of<uint32_t>(error);
    c.k_stride_token = k.stride(0);
    c.k_stride_head = k.stride(1);
    c.v_stride_token = v.stride(0);
    c.v_stride_head = v.stride(1);
    c.k_cache_stride_page = kc.stride(0);
    c.k_cache_stride_token = kc.stride(1);
    c.k_cache_stride_head = kc.stride(2);
    c.v_cache_stride_page = vc.stride(0);
    c.v_cache_stride_token = vc.stride(1);
    c.v_cache_stride_head = vc.stride(2);
    c.num_pages = kc.size(0);
    c.num_tokens = static_cast<int32_t>(tokens);
    c.num_kv_heads = static_cast<int32_t>(kv_heads);
    c.head_dim = static_cast<int32_t>(dim);
    check(unlocked([&] { return g_lib.append_kv(&c, on.stream()); }));
    if (!q) Py_RETURN_NONE;
    return result(a[9], made);
  });
}

PyObject* insert_keys_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("indexer_insert_keys_mxfp4", n, 6, [&]() -> PyObject* {
    const Tensor &k = tensor(a[0], "k"), &slots = tensor(a[1], "slot_mapping"), &cache = tensor(a[2], "index_cache");
    const Tensor *values = maybe(a[3], "values"), *error = maybe(a[4], "dev_error");
    if (k.dim() != 2 || k.scalar_type() != at::kBFloat16) refuse("k must be a bfloat16 tensor [tokens, 128]");
    const int64_t tokens = k.size(0), dim = k.size(1);
    if (dim != IDX_HEAD_DIM) refuse("keys of " + std::to_string(dim) + " values, not 128", IDX_ERR_UNSUPPORTED);
    if (k.stride(1) != 1) refuse("k must be contiguous in its last dimension");
    need_vector(slots, "slot_mapping", at::kLong, tokens);
    if (cache.scalar_type() != at::kByte || cache.dim() != 2 || cache.size(1) != IDX_MXFP4_PAGE_BYTES ||
        !cache.is_contiguous())
      refuse("index_cache must be a contiguous uint8 tensor [pages, 4352]");
    if (values && (values->sizes() != k.sizes() || values->scalar_type() != at::kBFloat16 || !values->is_contiguous()))
      refuse("values must be a contiguous bfloat16 tensor of k's shape");
    need_error(error);
    const int index = need_device({&k, &slots, &cache, values, error});
    const On on(index, a[5]);
    check(unlocked([&] {
      return g_lib.insert_keys_mxfp4(k.data_ptr(), tokens > 1 ? k.stride(0) : dim, at_of<const int64_t>(slots),
                                       tokens, static_cast<int32_t>(dim), at_of<uint8_t>(cache), cache.size(0),
                                       at_of<void>(values), at_of<uint32_t>(error), on.stream());
    }));
    return result(a[2], cache);
  });
}

// ---------------------------------------------------------------------------
// trees
// ---------------------------------------------------------------------------

PyObject* plan_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("indexer_plan_tree", n, 12, [&]() -> PyObject* {
    const Tensor &parents = tensor(a[0], "parents"), &lens = tensor(a[1], "seq_lens");
    const Tensor& start = tensor(a[2], "query_start_loc");
    const Tensor *masks = maybe(a[7], "masks"), *positions = maybe(a[8], "positions"), *paths = maybe(a[9], "paths");
    const Tensor* error = maybe(a[10], "dev_error");
    need_vector(parents, "parents", at::kInt, -1);
    const int64_t tokens = parents.size(0);
    need_vector(start, "query_start_loc", at::kInt, -1);
    const int64_t reqs = start.size(0) - 1;
    if (reqs < 0) refuse("query_start_loc is empty");
    need_vector(lens, "seq_lens", at::kInt, reqs);
    const int64_t words = (static_cast<int64_t>(count(a[3], "max_query_len", 1)) + 31) / 32;
    const int32_t window = count(a[4], "window"), sinks = count(a[5], "sinks"), width = count(a[6], "max_path");
    const auto need = [&](const Tensor* t, const char* what, int64_t columns) {
      if (!t) return;
      need_matrix(*t, what, tokens);
      if (t->size(1) != columns || !t->is_contiguous())
        refuse(std::string(what) + " must be contiguous, of " + std::to_string(columns) + " columns");
    };
    need(masks, "masks", words);
    need(paths, "paths", width);
    if (positions) need_vector(*positions, "positions", at::kInt, tokens);
    need_error(error);
    if (tokens > INT32_MAX || reqs > INT32_MAX) refuse("sizes past 32 bits", IDX_ERR_UNSUPPORTED);
    const int index = need_device({&parents, &lens, &start, masks, positions, paths, error});
    const On on(index, a[11]);
    const Tensor made_masks = masks ? Tensor() : fresh({tokens, words}, at::kInt, parents);
    const Tensor made_positions = positions ? Tensor() : fresh({tokens}, at::kInt, parents);
    const Tensor made_paths = paths || !width ? Tensor() : fresh({tokens, width}, at::kInt, parents);
    int32_t* const path = width ? at_of<int32_t>(paths ? *paths : made_paths) : nullptr;
    check(unlocked([&] {
      return g_lib.plan_tree(at_of<const int32_t>(parents), at_of<const int32_t>(lens),
                               at_of<const int32_t>(start), static_cast<int32_t>(reqs),
                               static_cast<int32_t>(tokens), window, sinks,
                               at_of<int32_t>(masks ? *masks : made_masks), static_cast<int32_t>(words),
                               at_of<int32_t>(positions ? *positions : made_positions), path, width,
                               at_of<uint32_t>(error), on.stream());
    }));
    PyObject* r = PyTuple_New(3);
    if (!r) throw PythonError{};
    PyTuple_SET_ITEM(r, 0, result(a[7], made_masks));
    PyTuple_SET_ITEM(r, 1, result(a[8], made_positions));
    if (!paths && !width) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 2, paths || width ? result(a[9], made_paths) : Py_None);
    return r;
  });
}

// idx_token_pool entries of a tensor [pages, 64, ...] or a uint8 index cache [pages, 8448 or 4352].
void add_pool(const Tensor& t, std::vector<idx_token_pool>* out) {
  if (t.dim() < 2 || t.size(0) < 1) refuse("a pool must be a tensor [pages, 64, ...] or a uint8 index cache");
  uint8_t* const at = at_of<uint8_t>(t);
  const int64_t pages = t.size(0);
  if (t.scalar_type() == at::kByte && t.dim() == 2 &&
      (t.size(1) == IDX_PAGE_BYTES || t.size(1) == IDX_MXFP4_PAGE_BYTES)) {
    const int64_t stride = pages > 1 ? t.stride(0) : t.size(1);
    if (t.stride(1) != 1 || stride < t.size(1) || stride % 4)
      refuse("an index cache's pages must be contiguous and of whole words");
    if (t.size(1) == IDX_PAGE_BYTES) {
      out->push_back({at, stride, IDX_HEAD_DIM, 0, 1, IDX_HEAD_DIM});
      out->push_back({at + IDX_PAGE_TOKENS * IDX_HEAD_DIM, stride, 4, 0, 1, 4});
    } else {
      constexpr int32_t kToken = IDX_MXFP4_PAGE_BYTES / IDX_PAGE_TOKENS;
      out->push_back({at, stride, kToken, 0, 1, kToken});
    }
    return;
  }
  if (t.size(1) != IDX_PAGE_TOKENS)
    refuse("pages of " + std::to_string(t.size(1)) + " tokens, not 64", IDX_ERR_UNSUPPORTED);
  const int64_t size = static_cast<int64_t>(t.element_size());
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0) refuse("a pool's tokens overlap");
  // a token's values from the last dimension up to where they stop being contiguous
  int64_t run = size, dim = t.dim() - 1;
  for (; dim >= 2 && (t.size(dim) == 1 || t.stride(dim) * size == run); --dim) run *= t.size(dim);
  int64_t pieces = 1, piece_stride = run;
  if (dim >= 2) {
    pieces = t.size(dim);
    piece_stride = t.stride(dim) * size;
    for (int64_t i = 2; i < dim; ++i)
      if (t.size(i) > 1) refuse("a pool's token must be one run of values or evenly spaced ones");
  }
  const int64_t token_stride = t.stride(1) * size, page_stride = pages > 1 ? t.stride(0) * size : token_stride;
  if (run == 0 || run % 4 || token_stride % 4 || page_stride % 4 || piece_stride % 4)
    refuse("a pool's tokens must be of whole 4-byte words");
  if (run > INT32_MAX || pieces > INT32_MAX) refuse("sizes past 32 bits", IDX_ERR_UNSUPPORTED);
  out->push_back({at, page_stride, token_stride, piece_stride, static_cast<int32_t>(pieces), static_cast<int32_t>(run)});
}

// The items of a list or tuple of pools.
struct Items {
  PyObject* fast;
  explicit Items(PyObject* o) : fast(PySequence_Fast(o, "pools must be a list of tensors")) {
    if (!fast) throw PythonError{};
  }
  ~Items() { Py_DECREF(fast); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  const Tensor& operator[](Py_ssize_t i) const { return tensor(PySequence_Fast_GET_ITEM(fast, i), "a pool"); }
};

// Pages of the pools (-1: no pool).
int64_t all_pools(const Items& items, std::vector<idx_token_pool>* out) {
  int64_t pages = -1;
  out->reserve(2 * items.size());
  for (Py_ssize_t i = 0; i < items.size(); ++i) {
    const Tensor& t = items[i];
    add_pool(t, out);
    if (pages >= 0 && t.size(0) != pages) refuse("the pools differ in pages");
    pages = t.size(0);
  }
  return pages;
}

PyObject* commit_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("indexer_commit_tree", n, 8, [&]() -> PyObject* {
    const Items items(a[0]);
    std::vector<idx_token_pool> pools;
    int64_t pages = all_pools(items, &pools);
    const Tensor &table = tensor(a[1], "block_table"), &lens = tensor(a[2], "seq_lens");
    const Tensor &start = tensor(a[3], "query_start_loc"), &accepted = tensor(a[4], "accepted");
    const Tensor *refs = maybe(a[5], "ref_counts"), *error = maybe(a[6], "dev_error");
    need_vector(start, "query_start_loc", at::kInt, -1);
    const int64_t reqs = start.size(0) - 1;
    if (reqs < 0) refuse("query_start_loc is empty");
    need_matrix(table, "block_table", reqs);
    if (table.size(1) < 1) refuse("block_table has no columns");
    need_vector(lens, "seq_lens", at::kInt, reqs);
    need_matrix(accepted, "accepted", reqs);
    if (refs) {
      need_vector(*refs, "ref_counts", at::kInt, pages);
      pages = refs->size(0);
    }
    if (pages < 0) refuse("neither pools nor ref_counts");
    const int64_t bt_stride = row_stride(table, "block_table"), stride = row_stride(accepted, "accepted");
    need_error(error);
    if (reqs > INT32_MAX || table.size(1) > INT32_MAX || accepted.size(1) > INT32_MAX)
      refuse("sizes past 32 bits", IDX_ERR_UNSUPPORTED);
    const int index = need_device({&table, &lens, &start, &accepted, refs, error});
    for (Py_ssize_t i = 0; i < items.size(); ++i)
      if (!items[i].is_cuda() || items[i].get_device() != index) refuse("tensors are on different devices");
    const On on(index, a[7]);
    check(unlocked([&] {
      return g_lib.commit_tree(pools.data(), static_cast<int32_t>(pools.size()), pages,
                                 at_of<const int32_t>(table), bt_stride, static_cast<int32_t>(table.size(1)),
                                 static_cast<int32_t>(reqs), at_of<int32_t>(lens), at_of<const int32_t>(start),
                                 at_of<const int32_t>(accepted), stride, static_cast<int32_t>(accepted.size(1)),
                                 at_of<int32_t>(refs), at_of<uint32_t>(error), on.stream());
    }));
    Py_RETURN_NONE;
  });
}

// The idx_token_pool entries of a list of pools, as tuples (for tests).
PyObject* token_pools(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("token_pools", n, 1, [&]() -> PyObject* {
    std::vector<idx_token_pool> pools;
    all_pools(Items(a[0]), &pools);
    PyObject* r = PyList_New(0);
    for (const idx_token_pool& p : pools) {
      PyObject* e = r ? Py_BuildValue("LLLii", static_cast<long long>(p.page_stride), static_cast<long long>(p.token_stride),
                                      static_cast<long long>(p.piece_stride), p.pieces, p.piece_bytes)
                      : nullptr;
      const bool ok = e && PyList_Append(r, e) == 0;
      Py_XDECREF(e);
      if (!ok) {
        Py_XDECREF(r);
        throw PythonError{};
      }
    }
    return r;
  });
}

// bind(handle): takes the functions from a library that dlopen has returned.
PyObject* bind(PyObject*, PyObject* handle) {
  void* const lib = PyLong_AsVoidPtr(handle);
  if (PyErr_Occurred()) return nullptr;
  Library found;
  const auto get = [&](auto* at, const char* name) -> bool {
    *at = reinterpret_cast<std::remove_reference_t<decltype(*at)>>(dlsym(lib, name));
    if (!*at) PyErr_Format(PyExc_RuntimeError, "the library does not export %s", name);
    return *at != nullptr;
  };
  if (!get(&found.attend_paged, "indexer_attend_paged") || !get(&found.attend_selected, "indexer_attend_selected") ||
      !get(&found.attend_tree, "indexer_attend_tree") ||
      !get(&found.attend_workspace_bytes, "indexer_attend_workspace_bytes") ||
      !get(&found.append_kv, "indexer_append_kv") ||
      !get(&found.insert_keys_mxfp4, "indexer_insert_keys_mxfp4") || !get(&found.plan_tree, "indexer_plan_tree") ||
      !get(&found.commit_tree, "indexer_commit_tree") || !get(&found.last_cuda_error, "indexer_last_cuda_error"))
    return nullptr;
  g_lib = found;
  Py_RETURN_NONE;
}

PyObject* set_error_class(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <typename F>
constexpr PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"attend", method(attend), METH_FASTCALL, nullptr},
    {"append_kv", method(append_kv), METH_FASTCALL, nullptr},
    {"insert_keys_mxfp4", method(insert_keys_mxfp4), METH_FASTCALL, nullptr},
    {"plan_tree", method(plan_tree), METH_FASTCALL, nullptr},
    {"commit_tree", method(commit_tree), METH_FASTCALL, nullptr},
    {"token_pools", method(token_pools), METH_FASTCALL, nullptr},
    {"bind", bind, METH_O, nullptr},
    {"set_error_class", set_error_class, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
