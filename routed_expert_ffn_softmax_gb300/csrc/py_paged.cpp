// Python side of the paged serving path (include/paged/moe_paged.h): checks tensors and makes the C calls.
//
// These calls are made per layer and token, and several take 4 to 10 us on the GPU. Checked attribute by attribute in
// Python and passed through ctypes, a call with 12 tensors took 9 us of host time, 6 of them checks; here it takes 3,
// most of it the launch. Everything is checked on every call; nothing is kept between calls.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "paged/moe_paged.h"

namespace {

constexpr at::ScalarType kI32 = at::kInt, kBf16 = at::kBFloat16, kF32 = at::kFloat, kU8 = at::kByte;

// One call's arguments. The first tensor settles the device; a failed check leaves a Python error set and ok() false.
class Args {
 public:
  Args(const char* fn, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : fn_(fn), args_(args), ok_(n == want) {
    if (!ok_) PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd expected", fn, n, want);
  }
  bool ok() const { return ok_; }

  const at::Tensor* tensor(const char* name) {
    if (!ok_) return nullptr;
    PyObject* o = args_[at_++];
    if (!THPVariable_Check(o)) {
      fail(PyExc_TypeError, name, "must be a tensor");
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  void dims(const char* name, const at::Tensor* t, int64_t n) {
    if (ok_ && t->dim() != n) {
      ok_ = false;
      PyErr_Format(PyExc_ValueError, "%s: %s must have %lld dimensions, got %lld", fn_, name, (long long)n, (long long)t->dim());
    }
  }
  // The address of a contiguous tensor of this type on the call's device.
  void* at(const char* name, const at::Tensor* t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    check(name, t, type, shape);
    if (ok_ && !t->is_contiguous()) fail(PyExc_ValueError, name, "must be contiguous");
    return ok_ ? t->data_ptr() : nullptr;
  }
  void* next(const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(name);
    return ok_ ? at(name, t, type, shape) : nullptr;
  }
  void* next_or_none(const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (ok_ && args_[at_] == Py_None) {
      ++at_;
      return nullptr;
    }
    return next(name, type, shape);
  }
  // Type, device and shape alone.
  void check(const char* name, const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
    if (!ok_) return;
    if (t->scalar_type() != type) return fail(PyExc_TypeError, name, "has the wrong type, expected ", at::toString(type));
    if (!t->is_cuda()) return fail(PyExc_ValueError, name, "must be on a CUDA device");
    if (device_ < 0) device_ = t->get_device();
    if (t->get_device() != device_) return fail(PyExc_ValueError, name, "must be on the same CUDA device as the other tensors");
    if (t->sizes() != shape) {
      ok_ = false;
      PyErr_Format(PyExc_ValueError, "%s: %s must have shape %s, got %s", fn_, name, text(shape).c_str(), text(t->sizes()).c_str());
    }
  }
  int integer(const char* name) {
    if (!ok_) return 0;
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(args_[at_++], &overflow);
    if (v == -1 && PyErr_Occurred()) {
      ok_ = false;
      return 0;
    }
    if (overflow || v > INT32_MAX || v < INT32_MIN) fail(PyExc_OverflowError, name, "does not fit 32 bits");
    return static_cast<int>(v);
  }
  float number() {
    if (!ok_) return 0.0f;
    const double v = PyFloat_AsDouble(args_[at_++]);
    if (v == -1.0 && PyErr_Occurred()) ok_ = false;
    return static_cast<float>(v);
  }
  int size(const at::Tensor* t, int64_t dim, const char* name) {
    if (!ok_) return 0;
    const int64_t n = t->size(dim);
    if (n > INT32_MAX) fail(PyExc_OverflowError, name, "is too long");
    return static_cast<int>(n);
  }
  void fail(PyObject* kind, const char* name, const char* what, const char* more = "") {
    ok_ = false;
    PyErr_Format(kind, "%s: %s %s%s", fn_, name, what, more);
  }
  // The call itself, with the tensors' device current, on the given stream or that device's current one.
  template <typename F>
  PyObject* call(F&& f) {
    if (!ok_) return nullptr;
    PyObject* s = args_[at_];
    void* stream = nullptr;
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
    } else {
      stream = PyLong_AsVoidPtr(s);
      if (!stream && PyErr_Occurred()) return nullptr;
    }
    c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device_));
    return PyLong_FromLong(f(static_cast<moe_stream_t>(stream)));
  }

 private:
  static std::string text(at::IntArrayRef v) {
    std::string s = "(";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
  }
  const char* fn_;
  PyObject* const* args_;
  Py_ssize_t at_ = 0;
  int64_t device_ = -1;
  bool ok_;
};

// No C++ exception may reach the interpreter.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

uint16_t* bf(void* p) { return static_cast<uint16_t*>(p); }
int32_t* in(void* p) { return static_cast<int32_t*>(p); }

// (ctx_lens, new_lens, page_size, num_pages, free_pages, free_count, block_table, seq_lens, cu_new, positions, slots,
//  free_left, workspace, stream)
PyObject* paged_plan(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_paged_plan", args, n, 14);
    const at::Tensor* ctx = a.tensor("ctx_lens");
    if (a.ok()) a.dims("ctx_lens", ctx, 1);
    const int B = a.size(ctx, 0, "ctx_lens");
    void* c = a.ok() ? a.at("ctx_lens", ctx, kI32, {B}) : nullptr;
    void* nw = a.next("new_lens", kI32, {B});
    const int page = a.integer("page_size"), pages = a.integer("num_pages");
    const at::Tensor* fr = a.tensor("free_pages");
    if (a.ok()) a.dims("free_pages", fr, 1);
    const int n_free = a.size(fr, 0, "free_pages");
    void* f = a.ok() ? a.at("free_pages", fr, kI32, {n_free}) : nullptr;
    void* count = a.next("free_count", kI32, {1});
    const at::Tensor* tb = a.tensor("block_table");
    if (a.ok()) a.dims("block_table", tb, 2);
    const int width = a.size(tb, 1, "block_table");
    void* t = a.ok() ? a.at("block_table", tb, kI32, {B, width}) : nullptr;
    void* lens = a.next("seq_lens", kI32, {B});
    void* cu = a.next("cu_new", kI32, {static_cast<int64_t>(B) + 1});
    const at::Tensor* ps = a.tensor("positions");
    if (a.ok()) a.dims("positions", ps, 1);
    const int rows = a.size(ps, 0, "positions");
    void* pos = a.ok() ? a.at("positions", ps, kI32, {rows}) : nullptr;
    void* slots = a.next("slots", kI32, {rows});
    void* left = a.next("free_left", kI32, {1});
    const at::Tensor* ws = a.tensor("workspace");
    void* w = a.ok() ? a.at("workspace", ws, kU8, {ws->numel()}) : nullptr;
    return a.call([&](moe_stream_t s) {
      return moe_paged_plan(in(c), in(nw), B, page, pages, in(f), n_free, in(count), in(t), width, in(lens), in(cu), in(pos),
                            in(slots), rows, in(left), w, ws->numel(), s);
    });
  });
}

// (qkv, q_weight, k_weight, eps, inv_freq, positions, slots, q_out, k_cache, v_cache, interleaved, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_qk_norm_rope", args, n, 12);
    const at::Tensor* x = a.tensor("qkv");
    if (a.ok() && (x->scalar_type() != kBf16 || !x->is_cuda())) a.fail(PyExc_TypeError, "qkv", "must be a bf16 CUDA tensor");
    if (a.ok() && !(THPVariable_Check(args[7]) && THPVariable_Check(args[8])))
      a.fail(PyExc_TypeError, "q_out and k_cache", "must be tensors");
    if (!a.ok()) return nullptr;
    const at::Tensor& qo = THPVariable_Unpack(args[7]);
    const at::Tensor& kc = THPVariable_Unpack(args[8]);
    a.dims("q_out", &qo, 3);
    a.dims("k_cache", &kc, 4);
    if (!a.ok()) return nullptr;
    const int N = a.size(&qo, 0, "q_out"), h_q = a.size(&qo, 1, "q_out"), d = a.size(&qo, 2, "q_out");
    const int pages = a.size(&kc, 0, "k_cache"), h_kv = a.size(&kc, 1, "k_cache"), page = a.size(&kc, 2, "k_cache");
    const int64_t width = (static_cast<int64_t>(h_q) + 2 * static_cast<int64_t>(h_kv)) * d;
    a.check("qkv", x, kBf16, {N, width});
    if (a.ok() && width > 1 && x->stride(1) != 1) a.fail(PyExc_ValueError, "qkv", "must have contiguous rows");
    void* qw = a.next_or_none("q_weight", kBf16, {d});
    void* kw = a.next_or_none("k_weight", kBf16, {d});
    const float eps = a.number();
    void* inv = nullptr;
    int rot = 0;
    if (a.ok()) {
      const at::Tensor* f = THPVariable_Check(args[4]) ? &THPVariable_Unpack(args[4]) : nullptr;
      if (f) a.dims("inv_freq", f, 1);
      const int pairs = f && a.ok() ? a.size(f, 0, "inv_freq") : 0;
      if (pairs > (1 << 20)) a.fail(PyExc_ValueError, "inv_freq", "is too long");
      inv = a.next_or_none("inv_freq", kF32, {pairs});
      rot = 2 * pairs;
    }
    void* pos = a.next("positions", kI32, {N});
    void* slots = a.next("slots", kI32, {N});
    void* q = a.next("q_out", kBf16, {N, h_q, d});
    void* k = a.next("k_cache", kBf16, {pages, h_kv, page, d});
    void* v = a.next("v_cache", kBf16, {pages, h_kv, page, d});
    const int inter = a.integer("interleaved");
    return a.call([&](moe_stream_t s) {
      return moe_qk_norm_rope(bf(x->data_ptr()), N > 1 ? x->stride(0) : width, N, h_q, h_kv, d, bf(qw), bf(kw), eps,
                              static_cast<const float*>(inv), rot, inter, in(pos), in(slots), bf(q), bf(k), bf(v), pages, page,
                              s);
    });
  });
}

// What the attention calls share: q, k_cache, v_cache, block_table, seq_lens, scale, out, workspace.
struct Attention {
  int N = 0, B = 0, h_q = 0, h_kv = 0, d = 0, pages = 0, page = 0, width = 0;
  void *q = nullptr, *k = nullptr, *v = nullptr, *table = nullptr, *lens = nullptr, *out = nullptr, *ws = nullptr;
  size_t ws_bytes = 0;
  float scale = 0.0f;
  void queries(Args& a) {
    const at::Tensor* t = a.tensor("q");
    if (a.ok()) a.dims("q", t, 3);
    N = a.size(t, 0, "q"), h_q = a.size(t, 1, "q"), d = a.size(t, 2, "q");
    if (a.ok()) q = a.at("q", t, kBf16, {N, h_q, d});
  }
  void rest(Args& a) {
    const at::Tensor* t = a.tensor("k_cache");
    if (a.ok()) a.dims("k_cache", t, 4);
    pages = a.size(t, 0, "k_cache"), h_kv = a.size(t, 1, "k_cache"), page = a.size(t, 2, "k_cache");
    if (a.ok()) k = a.at("k_cache", t, kBf16, {pages, h_kv, page, d});
    v = a.next("v_cache", kBf16, {pages, h_kv, page, d});
    t = a.tensor("block_table");
    if (a.ok()) a.dims("block_table", t, 2);
    B = a.size(t, 0, "block_table"), width = a.size(t, 1, "block_table");
    if (a.ok()) table = a.at("block_table", t, kI32, {B, width});
    lens = a.next("seq_lens", kI32, {B});
    scale = a.number();
    out = a.next("out", kBf16, {N, h_q, d});
    t = a.tensor("workspace");
    if (a.ok()) ws = a.at("workspace", t, kU8, {t->numel()});
    if (a.ok()) ws_bytes = t->numel();
  }
  void one_per_sequence(Args& a) {
    if (a.ok() && N != B) a.fail(PyExc_ValueError, "q", "must have one row per sequence");
  }
};

// (q, k_cache, v_cache, block_table, seq_lens, scale, out, workspace, window, n_sink, stream)
PyObject* gqa_paged_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_gqa_paged_decode", args, n, 11);
    Attention t;
    t.queries(a);
    t.rest(a);
    t.one_per_sequence(a);
    const int window = a.integer("window"), n_sink = a.integer("n_sink");
    return a.call([&](moe_stream_t s) {
      return moe_gqa_paged_decode(bf(t.q), bf(t.k), bf(t.v), in(t.table), in(t.lens), t.B, t.h_q, t.h_kv, t.d, t.pages, t.page,
                                  t.width, t.scale, window, n_sink, bf(t.out), t.ws, t.ws_bytes, s);
    });
  });
}

// (q, cu_q, k_cache, v_cache, block_table, seq_lens, scale, out, workspace, window, n_sink, stream)
PyObject* gqa_paged_prefill(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_gqa_paged_prefill", args, n, 12);
    Attention t;
    t.queries(a);
    const at::Tensor* c = a.tensor("cu_q");
    t.rest(a);
    void* cu = a.ok() ? a.at("cu_q", c, kI32, {static_cast<int64_t>(t.B) + 1}) : nullptr;
    const int window = a.integer("window"), n_sink = a.integer("n_sink");
    return a.call([&](moe_stream_t s) {
      return moe_gqa_paged_prefill(bf(t.q), in(cu), bf(t.k), bf(t.v), in(t.table), in(t.lens), t.N, t.B, t.h_q, t.h_kv, t.d,
                                   t.pages, t.page, t.width, t.scale, window, n_sink, bf(t.out), t.ws, t.ws_bytes, s);
    });
  });
}

// (q, prefix_table, prefix_len, k_cache, v_cache, block_table, seq_lens, scale, out, workspace, stream)
PyObject* gqa_prefix_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_gqa_prefix_decode", args, n, 11);
    Attention t;
    t.queries(a);
    int entries = 0;
    if (a.ok() && THPVariable_Check(args[1])) {
      a.dims("prefix_table", &THPVariable_Unpack(args[1]), 1);
      if (a.ok()) entries = a.size(&THPVariable_Unpack(args[1]), 0, "prefix_table");
    }
    void* shared = a.next_or_none("prefix_table", kI32, {entries});
    const int len = a.integer("prefix_len");
    t.rest(a);
    t.one_per_sequence(a);
    if (a.ok() && len > 0 && static_cast<int64_t>(entries) * t.page < len)
      a.fail(PyExc_ValueError, "prefix_table", "is shorter than prefix_len");
    return a.call([&](moe_stream_t s) {
      return moe_gqa_prefix_decode(bf(t.q), in(shared), len, bf(t.k), bf(t.v), in(t.table), in(t.lens), t.B, t.h_q, t.h_kv, t.d,
                                   t.pages, t.page, t.width, t.scale, bf(t.out), t.ws, t.ws_bytes, s);
    });
  });
}

#define PAGED_METHOD(name) {"moe_" #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PAGED_METHOD(paged_plan),        PAGED_METHOD(qk_norm_rope),      PAGED_METHOD(gqa_paged_decode),
                         PAGED_METHOD(gqa_paged_prefill), PAGED_METHOD(gqa_prefix_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
