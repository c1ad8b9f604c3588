// Python side of the draft-tree and eviction calls: the checks of their tensors
// and the marshalling, as a CPython module.  A step makes these calls between
// kernels of a few microseconds; the same checks in Python take 0.4 us a tensor,
// longer than the launch itself (paged_tree_plan: 8.9 us from Python, of which
// its checks and ctypes took 5).  The module holds no kernel and no state but
// the addresses of the library's entry points, which the caller hands over.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "paged_attn.h"

namespace {

decltype(&paged_tree_plan) f_plan = nullptr;
decltype(&paged_tree_attn_ws) f_attn = nullptr;
decltype(&paged_tree_accept) f_accept = nullptr;
decltype(&paged_kv_evict) f_evict = nullptr;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

using Dims = std::initializer_list<int64_t>;

[[noreturn]] void refuse(const at::Tensor& t, const char* name, const std::string& want) {
  std::ostringstream s;
  s << name << ": " << want << " is wanted, got " << t.scalar_type() << " " << t.sizes()
    << " with strides " << t.strides() << " on " << t.device();
  throw Refused(s.str());
}

const at::Tensor& tensor_of(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + ": a tensor is wanted");
  return THPVariable_Unpack(o);
}

// The tensors of one call: all on the device of the first.
struct Call {
  c10::Device device{c10::kCPU};

  const at::Tensor& first(PyObject* o, const char* name) {
    const at::Tensor& t = tensor_of(o, name);
    if (!t.is_cuda()) {
      std::ostringstream s;
      s << name << ": a tensor on a CUDA device is wanted, got one on " << t.device();
      throw Refused(s.str());
    }
    device = t.device();
    return t;
  }
  void check(const at::Tensor& t, const char* name, at::ScalarType type, Dims shape) const {
    if (t.scalar_type() == type && t.device() == device && t.sizes() == at::IntArrayRef(shape) &&
        t.layout() == c10::kStrided && t.is_contiguous())
      return;
    std::ostringstream s;
    s << "contiguous " << type << " " << at::IntArrayRef(shape) << " on " << device;
    refuse(t, name, s.str());
  }
  template <typename T>
  T* get(PyObject* o, const char* name, at::ScalarType type, Dims shape) const {
    const at::Tensor& t = tensor_of(o, name);
    check(t, name, type, shape);
    return static_cast<T*>(t.data_ptr());
  }
  int32_t* i32(PyObject* o, const char* name, Dims shape) const {
    return get<int32_t>(o, name, at::kInt, shape);
  }
  int32_t* i32_or_null(PyObject* o, const char* name, Dims shape) const {
    return o == Py_None ? nullptr : i32(o, name, shape);
  }
  int32_t* err(PyObject* o) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor_of(o, "err");
    check(t, "err", at::kInt, {t.numel() < 1 ? 1 : t.numel()});
    return static_cast<int32_t*>(t.data_ptr());
  }
  // Contiguous device bytes of any type.
  void* bytes(PyObject* o, const char* name, size_t* n) const {
    const at::Tensor& t = tensor_of(o, name);
    if (t.device() != device || t.layout() != c10::kStrided || !t.is_contiguous()) {
      std::ostringstream s;
      s << "a contiguous tensor on " << device;
      refuse(t, name, s.str());
    }
    *n = t.nbytes();
    return t.data_ptr();
  }
  void* stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index()).stream();
    PyObject* x = PyObject_GetAttrString(o, "cuda_stream");
    void* p = x == nullptr ? nullptr : PyLong_AsVoidPtr(x);
    Py_XDECREF(x);
    if (PyErr_Occurred()) throw Refused("");
    return p;
  }
};

int32_t whole(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Refused("");
  if (x < INT32_MIN || x > INT32_MAX) throw Refused(std::string(name) + ": past 32 bits");
  return static_cast<int32_t>(x);
}

int32_t narrow(int64_t x, const char* name) {
  if (x > INT32_MAX) throw Refused(std::string(name) + ": a size past 32 bits");
  return static_cast<int32_t>(x);
}

float real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused("");
  return static_cast<float>(x);
}

int64_t rows_of(const at::Tensor& t, const char* name) {
  if (t.dim() < 1) refuse(t, name, "one dimension or more");
  return t.size(0);
}
int64_t width_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor_of(o, name);
  if (t.dim() < 1) refuse(t, name, "one dimension or more");
  return t.size(t.dim() - 1);
}

// A list of bf16 pools [num_blocks][Hkv][16][D] of one shape.
struct Pools {
  std::vector<void*> pointers;
  int64_t shape[4] = {0, 0, 0, 0};

  void read(Call& call, PyObject* list) {
    PyObject* seq = PySequence_Fast(list, "pools: a list of tensors is wanted");
    if (seq == nullptr) throw Refused("");
    struct Hold {
      PyObject* o;
      ~Hold() { Py_DECREF(o); }
    } hold{seq};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    pointers.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(seq, i);
      const at::Tensor& t = i == 0 ? call.first(o, "pools") : tensor_of(o, "pools");
      if (i == 0) {
        if (t.dim() != 4 || t.scalar_type() != at::kBFloat16)
          refuse(t, "pools", "BFloat16 [num_blocks][Hkv][16][D]");
        for (int d = 0; d < 4; ++d) shape[d] = t.size(d);
      }
      call.check(t, "pools", at::kBFloat16, {shape[0], shape[1], shape[2], shape[3]});
      pointers.push_back(t.data_ptr());
    }
  }
};

// f(args) -> pka_status, with what it throws as Python errors.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", wanted, given);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    Call c;
    const int64_t rows = rows_of(c.first(a[0], "parents"), "parents");
    const int64_t B = rows_of(tensor_of(a[2], "seq_lens"), "seq_lens");
    const int64_t width = width_of(a[3], "block_tables");
    const int32_t* parents = c.i32(a[0], "parents", {rows});
    const int32_t* first = c.i32(a[1], "query_start_loc", {B + 1});
    const int32_t* lens = c.i32(a[2], "seq_lens", {B});
    const int32_t* tables = c.i32(a[3], "block_tables", {B, width});
    uint64_t* masks = a[6] == Py_None
                          ? nullptr
                          : c.get<uint64_t>(a[6], "tree_masks", at::kLong, {rows});
    int32_t* positions = c.i32_or_null(a[7], "positions", {rows});
    int32_t* slots = c.i32_or_null(a[8], "slots", {rows});
    const int32_t* totals = c.i32_or_null(a[9], "total_lens", {B});
    const c10::cuda::OptionalCUDAGuard guard(c.device);
    return f_plan(parents, first, lens, totals, tables, narrow(width, "block_tables"),
                  whole(a[4], "num_blocks"), narrow(B, "seq_lens"), narrow(rows, "parents"),
                  whole(a[5], "max_query_len"), masks, positions, slots, c.err(a[10]),
                  c.stream(a[11]));
  });
}

PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    Call c;
    const at::Tensor& q = c.first(a[0], "q");
    if (q.dim() != 3) refuse(q, "q", "BFloat16 [total_q][Hq][D]");
    const int64_t rows = q.size(0), hq = q.size(1), d = q.size(2);
    const at::Tensor& k = tensor_of(a[2], "k_pool");
    if (k.dim() != 4 || k.size(2) != 16 || k.size(3) != d)
      refuse(k, "k_pool", "BFloat16 [num_blocks][Hkv][16][D] of q's D");
    const int64_t B = rows_of(tensor_of(a[7], "seq_lens"), "seq_lens");
    const int64_t width = width_of(a[4], "block_tables");
    const Dims pool{k.size(0), k.size(1), 16, d}, shape{rows, hq, d};
    c.check(q, "q", at::kBFloat16, shape);
    void* out = c.get<void>(a[1], "out", at::kBFloat16, shape);
    const pka_kv_pool kv{c.get<void>(a[2], "k_pool", at::kBFloat16, pool),
                         c.get<void>(a[3], "v_pool", at::kBFloat16, pool),
                         narrow(k.size(0), "k_pool"), narrow(k.size(1), "k_pool"), 16,
                         narrow(d, "q")};
    const int32_t* tables = c.i32(a[4], "block_tables", {B, width});
    const int32_t* first = c.i32(a[5], "query_start_loc", {B + 1});
    const uint64_t* masks = c.get<uint64_t>(a[6], "tree_masks", at::kLong, {rows});
    const int32_t* lens = c.i32(a[7], "seq_lens", {B});
    size_t space = 0;
    void* workspace = c.bytes(a[10], "workspace", &space);
    const pka_attn_params par{real(a[11]), real(a[12]), whole(a[13], "window"), c.err(a[14])};
    const c10::cuda::OptionalCUDAGuard guard(c.device);
    return f_attn(q.data_ptr(), out, &kv, tables, narrow(width, "block_tables"), first, masks, lens,
                  narrow(B, "seq_lens"), narrow(hq, "q"), narrow(rows, "q"),
                  whole(a[8], "max_query_len"), whole(a[9], "max_seq_len"), &par, workspace, space,
                  c.stream(a[15]));
  });
}

PyObject* accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    Call c;
    Pools p;
    p.read(c, a[0]);
    const int64_t rows = rows_of(
        p.pointers.empty() ? c.first(a[1], "parents") : tensor_of(a[1], "parents"), "parents");
    const int64_t B = rows_of(tensor_of(a[6], "seq_lens"), "seq_lens");
    const int64_t width = width_of(a[7], "path");
    const int32_t* parents = c.i32(a[1], "parents", {rows});
    const int32_t* tokens = c.i32(a[2], "tokens", {rows});
    const int32_t* targets = c.i32(a[3], "targets", {rows});
    const int32_t* slots = p.pointers.empty() ? c.i32_or_null(a[4], "slots", {rows})
                                              : c.i32(a[4], "slots", {rows});
    const int32_t* first = c.i32(a[5], "query_start_loc", {B + 1});
    const int32_t* lens = c.i32(a[6], "seq_lens", {B});
    int32_t* path = c.i32(a[7], "path", {B, width});
    int32_t* accepted = c.i32(a[8], "accepted", {B});
    int32_t* next = c.i32(a[9], "next_tokens", {B});
    int32_t* new_lens = c.i32(a[10], "new_seq_lens", {B});
    const c10::cuda::OptionalCUDAGuard guard(c.device);
    return f_accept(p.pointers.data(), narrow(p.pointers.size(), "pools"),
                    narrow(p.shape[0], "pools"), narrow(p.shape[1], "pools"),
                    narrow(p.shape[2], "pools"), narrow(p.shape[3], "pools"), parents, tokens,
                    targets, slots, first, lens, narrow(B, "seq_lens"), narrow(rows, "parents"),
                    narrow(width, "path"), path, accepted, next, new_lens, c.err(a[11]),
                    c.stream(a[12]));
  });
}

PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&] {
    Call c;
    Pools p;
    p.read(c, a[0]);
    if (p.pointers.empty() || p.pointers.size() % 2 != 0)
      throw Refused("pools: K and V of each layer are wanted, got " +
                    std::to_string(p.pointers.size()) + " pools");
    const int64_t layers = static_cast<int64_t>(p.pointers.size() / 2);
    const int64_t B = rows_of(tensor_of(a[4], "seq_lens"), "seq_lens");
    const int64_t width = width_of(a[3], "block_tables");
    const Dims shape{layers, B, p.shape[1], width * 16};
    const float* mass = c.get<float>(a[1], "key_mass", at::kFloat, shape);
    const int32_t* pos = c.i32(a[2], "key_pos", shape);
    const int32_t* tables = c.i32(a[3], "block_tables", {B, width});
    const int32_t* lens = c.i32(a[4], "seq_lens", {B});
    const int32_t* totals = c.i32_or_null(a[5], "total_lens", {B});
    float* new_mass = c.get<float>(a[9], "new_mass", at::kFloat, shape);
    int32_t* new_pos = c.i32(a[10], "new_pos", shape);
    int32_t* new_lens = c.i32(a[11], "new_seq_lens", {B});
    size_t space = 0;
    void* workspace = c.bytes(a[12], "workspace", &space);
    const int32_t* refs = c.i32_or_null(a[13], "refcounts", {p.shape[0]});
    const c10::cuda::OptionalCUDAGuard guard(c.device);
    return f_evict(p.pointers.data(), narrow(layers, "pools"), narrow(p.shape[0], "pools"),
                   narrow(p.shape[1], "pools"), narrow(p.shape[2], "pools"),
                   narrow(p.shape[3], "pools"), tables, narrow(width, "block_tables"), lens, totals,
                   narrow(B, "seq_lens"), whole(a[6], "budget"), whole(a[7], "sinks"),
                   whole(a[8], "recent"), mass, new_mass, pos, new_pos, new_lens, refs, workspace,
                   space, c.err(a[14]), c.stream(a[15]));
  });
}

// The library's entry points, in this order: plan, attention, acceptance, eviction.
PyObject* attach(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses are wanted");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
  }
  f_plan = reinterpret_cast<decltype(f_plan)>(p[0]);
  f_attn = reinterpret_cast<decltype(f_attn)>(p[1]);
  f_accept = reinterpret_cast<decltype(f_accept)>(p[2]);
  f_evict = reinterpret_cast<decltype(f_evict)>(p[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* attached(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (f_plan == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not attached");
    return nullptr;
  }
  return F(self, a, n);
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

}  // namespace

PyMODINIT_FUNC PyInit__native() {
  static PyMethodDef methods[] = {
      {"attach", fast(attach), METH_FASTCALL, "Takes the addresses of the library's entry points."},
      {"tree_plan", fast(attached<plan>), METH_FASTCALL, "paged_tree_plan: a pka_status."},
      {"tree_attn_ws", fast(attached<attn>), METH_FASTCALL, "paged_tree_attn_ws: a pka_status."},
      {"tree_accept", fast(attached<accept>), METH_FASTCALL, "paged_tree_accept: a pka_status."},
      {"kv_evict", fast(attached<evict>), METH_FASTCALL, "paged_kv_evict: a pka_status."},
      {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods,
                               nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}
