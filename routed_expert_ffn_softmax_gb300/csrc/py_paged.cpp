// Python side of the paged serving path (include/paged/): checks tensors and makes the C calls.
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

#include "paged/moe_kv4.h"
#include "paged/moe_norm.h"
#include "paged/moe_paged.h"

namespace {

constexpr at::ScalarType kI32 = at::kInt, kBf16 = at::kBFloat16, kF32 = at::kFloat, kU8 = at::kByte, kI8 = at::kChar;

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
  void skip() { ++at_; }  // an argument that is None
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

// The 4-bit cache: [num_pages, h_kv, page_size / 16, 2304] bytes.
struct Kv4Cache {
  int pages = 0, h_kv = 0, page = 0;
  void* at = nullptr;
  void next(Args& a) {
    const at::Tensor* t = a.tensor("kv4_cache");
    if (a.ok()) a.dims("kv4_cache", t, 4);
    pages = a.size(t, 0, "kv4_cache"), h_kv = a.size(t, 1, "kv4_cache");
    const int blocks = a.size(t, 2, "kv4_cache");
    if (a.ok() && blocks > 1024) a.fail(PyExc_ValueError, "kv4_cache", "has too long pages");
    page = 16 * blocks;
    if (a.ok()) at = a.at("kv4_cache", t, kU8, {pages, h_kv, blocks, 2304});
  }
};

// What the calls that norm, rotate and store heads share.
struct Heads {
  int N = 0, h_q = 0, d = 0, rot = 0;
  const at::Tensor* x = nullptr;
  float eps = 0.0f;
  void *qw = nullptr, *kw = nullptr, *inv = nullptr;
  // q_out at its place among the arguments settles the sizes.
  void sizes(Args& a, PyObject* q_out) {
    x = a.tensor("qkv");
    if (a.ok() && (x->scalar_type() != kBf16 || !x->is_cuda())) a.fail(PyExc_TypeError, "qkv", "must be a bf16 CUDA tensor");
    if (a.ok() && !THPVariable_Check(q_out)) a.fail(PyExc_TypeError, "q_out", "must be a tensor");
    if (!a.ok()) return;
    const at::Tensor& qo = THPVariable_Unpack(q_out);
    a.dims("q_out", &qo, 3);
    N = a.size(&qo, 0, "q_out"), h_q = a.size(&qo, 1, "q_out"), d = a.size(&qo, 2, "q_out");
  }
  // The rows and their weights, for h_kv key/value heads; frequencies is the next argument but one.
  void rows(Args& a, int h_kv, PyObject* frequencies) {
    const int64_t w = width(h_kv);
    if (a.ok()) a.check("qkv", x, kBf16, {N, w});
    if (a.ok() && w > 1 && x->stride(1) != 1) a.fail(PyExc_ValueError, "qkv", "must have contiguous rows");
    qw = a.next_or_none("q_weight", kBf16, {d});
    kw = a.next_or_none("k_weight", kBf16, {d});
    eps = a.number();
    if (!a.ok()) return;
    const at::Tensor* f = THPVariable_Check(frequencies) ? &THPVariable_Unpack(frequencies) : nullptr;
    if (f) a.dims("inv_freq", f, 1);
    const int pairs = f && a.ok() ? a.size(f, 0, "inv_freq") : 0;
    if (pairs > (1 << 20)) a.fail(PyExc_ValueError, "inv_freq", "is too long");
    inv = a.next_or_none("inv_freq", kF32, {pairs});
    rot = 2 * pairs;
  }
  int64_t width(int h_kv) const { return (static_cast<int64_t>(h_q) + 2 * static_cast<int64_t>(h_kv)) * d; }
  int64_t stride(int h_kv) const { return N > 1 ? x->stride(0) : width(h_kv); }
};

// Positions with several axes: pair_axis [rot / 2] or None, positions [n_axes, N] with contiguous rows, or [N].
struct Axes {
  int n = 1;
  int64_t stride = 0;
  void *axis = nullptr, *positions = nullptr;
  void next(Args& a, const Heads& h) {
    axis = a.next_or_none("pair_axis", kI32, {h.rot / 2});
    const at::Tensor* t = a.tensor("positions");
    if (a.ok() && t->dim() == 1) {
      positions = a.at("positions", t, kI32, {h.N});
      return;
    }
    if (a.ok()) a.dims("positions", t, 2);
    n = a.size(t, 0, "positions");
    if (a.ok()) a.check("positions", t, kI32, {n, h.N});
    if (a.ok() && h.N > 1 && t->stride(1) != 1) a.fail(PyExc_ValueError, "positions", "must have contiguous rows");
    if (!a.ok()) return;
    stride = n > 1 ? t->stride(0) : h.N;
    positions = t->data_ptr();
  }
};

// (qkv, q_weight, k_weight, eps, inv_freq, [pair_axis,] positions, slots, q_out, k_cache, v_cache, interleaved, stream)
PyObject* qk_norm_to_bf16(const char* fn, bool several, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const int more = several ? 1 : 0;
    Args a(fn, args, n, 12 + more);
    if (!a.ok()) return nullptr;
    Heads h;
    h.sizes(a, args[7 + more]);
    if (a.ok() && !THPVariable_Check(args[8 + more])) a.fail(PyExc_TypeError, "k_cache", "must be a tensor");
    if (!a.ok()) return nullptr;
    const at::Tensor& kc = THPVariable_Unpack(args[8 + more]);
    a.dims("k_cache", &kc, 4);
    if (!a.ok()) return nullptr;
    const int pages = a.size(&kc, 0, "k_cache"), h_kv = a.size(&kc, 1, "k_cache"), page = a.size(&kc, 2, "k_cache");
    h.rows(a, h_kv, args[4]);
    Axes x;
    if (several) {
      x.next(a, h);
      if (a.ok() && !x.axis && h.rot > 0) a.fail(PyExc_TypeError, "pair_axis", "must be a tensor");
    } else {
      x.positions = a.next("positions", kI32, {h.N});
    }
    void* slots = a.next("slots", kI32, {h.N});
    void* q = a.next("q_out", kBf16, {h.N, h.h_q, h.d});
    void* k = a.next("k_cache", kBf16, {pages, h_kv, page, h.d});
    void* v = a.next("v_cache", kBf16, {pages, h_kv, page, h.d});
    const int inter = a.integer("interleaved");
    return a.call([&](moe_stream_t s) {
      const float* f = static_cast<const float*>(h.inv);
      const uint16_t* rows = bf(h.x->data_ptr());
      if (several)
        return moe_qk_norm_mrope(rows, h.stride(h_kv), h.N, h.h_q, h_kv, h.d, bf(h.qw), bf(h.kw), h.eps, f, in(x.axis), h.rot,
                                 inter, in(x.positions), x.stride, x.n, in(slots), bf(q), bf(k), bf(v), pages, page, s);
      return moe_qk_norm_rope(rows, h.stride(h_kv), h.N, h.h_q, h_kv, h.d, bf(h.qw), bf(h.kw), h.eps, f, h.rot, inter,
                              in(x.positions), in(slots), bf(q), bf(k), bf(v), pages, page, s);
    });
  });
}
PyObject* qk_norm_rope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return qk_norm_to_bf16("moe_qk_norm_rope", false, args, n);
}
PyObject* qk_norm_mrope(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return qk_norm_to_bf16("moe_qk_norm_mrope", true, args, n);
}

// (qkv, q_weight, k_weight, eps, inv_freq, pair_axis, positions, slots, q_out, kv4_cache, interleaved, stream)
PyObject* qk_norm_rope_kv4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_qk_norm_rope_kv4", args, n, 12);
    if (!a.ok()) return nullptr;
    Heads h;
    h.sizes(a, args[8]);
    if (a.ok() && !THPVariable_Check(args[9])) a.fail(PyExc_TypeError, "kv4_cache", "must be a tensor");
    if (!a.ok()) return nullptr;
    const at::Tensor& cache = THPVariable_Unpack(args[9]);
    a.dims("kv4_cache", &cache, 4);
    if (!a.ok()) return nullptr;
    h.rows(a, a.size(&cache, 1, "kv4_cache"), args[4]);
    Axes x;
    x.next(a, h);
    void* slots = a.next("slots", kI32, {h.N});
    void* q = a.next("q_out", kBf16, {h.N, h.h_q, h.d});
    Kv4Cache c;
    c.next(a);
    const int inter = a.integer("interleaved");
    return a.call([&](moe_stream_t s) {
      return moe_qk_norm_rope_kv4(bf(h.x->data_ptr()), h.stride(c.h_kv), h.N, h.h_q, c.h_kv, h.d, bf(h.qw), bf(h.kw), h.eps,
                                  static_cast<const float*>(h.inv), in(x.axis), h.rot, inter, in(x.positions), x.stride, x.n,
                                  in(slots), bf(q), static_cast<uint8_t*>(c.at), c.pages, c.page, s);
    });
  });
}

// (x, residual, weight, eps, residual_out, y, q, scales, stream)
PyObject* add_rms_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_add_rms_norm", args, n, 9);
    if (!a.ok()) return nullptr;
    const at::Tensor* x = args[0] == Py_None ? nullptr : a.tensor("x");
    if (!x) a.skip();
    const at::Tensor* r = a.tensor("residual");
    if (a.ok()) a.dims("residual", r, 2);
    const int N = a.size(r, 0, "residual"), H = a.size(r, 1, "residual");
    void* res = a.ok() ? a.at("residual", r, kBf16, {N, H}) : nullptr;
    if (a.ok() && x) a.check("x", x, kBf16, {N, H});
    if (a.ok() && x && H > 1 && x->stride(1) != 1) a.fail(PyExc_ValueError, "x", "must have contiguous rows");
    void* w = a.next_or_none("weight", kBf16, {H});
    const float eps = a.number();
    void* sum = a.next_or_none("residual_out", kBf16, {N, H});
    void* y = a.next_or_none("y", kBf16, {N, H});
    void* q = a.next_or_none("q", kI8, {N, H});
    void* scales = a.next_or_none("scales", kF32, {N, H / 128});
    return a.call([&](moe_stream_t s) {
      return moe_add_rms_norm(x ? bf(x->data_ptr()) : nullptr, x && N > 1 ? x->stride(0) : H, bf(res), bf(w), eps, N, H, bf(sum),
                              bf(y), static_cast<int8_t*>(q), static_cast<float*>(scales), s);
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
    lists(a);
  }
  void lists(Args& a) {  // block_table, seq_lens, scale, out, workspace
    const at::Tensor* t = a.tensor("block_table");
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

// (q, kv4_cache, block_table, seq_lens, scale, out, workspace, window, n_sink, stream)
PyObject* gqa_kv4_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_gqa_kv4_decode", args, n, 10);
    Attention t;
    t.queries(a);
    Kv4Cache c;
    c.next(a);
    t.lists(a);
    t.one_per_sequence(a);
    const int window = a.integer("window"), n_sink = a.integer("n_sink");
    return a.call([&](moe_stream_t s) {
      return moe_gqa_kv4_decode(bf(t.q), static_cast<uint8_t*>(c.at), in(t.table), in(t.lens), t.B, t.h_q, c.h_kv, t.d, c.pages,
                                c.page, t.width, t.scale, window, n_sink, bf(t.out), t.ws, t.ws_bytes, s);
    });
  });
}

// (kv4_cache, block_table, first, seq_lens, k_cache, v_cache, dst_table, workspace, stream)
PyObject* kv4_load(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a("moe_kv4_load", args, n, 9);
    Kv4Cache c;
    c.next(a);
    const at::Tensor* t = a.tensor("block_table");
    if (a.ok()) a.dims("block_table", t, 2);
    const int B = a.size(t, 0, "block_table"), width = a.size(t, 1, "block_table");
    void* table = a.ok() ? a.at("block_table", t, kI32, {B, width}) : nullptr;
    void* first = a.next_or_none("first", kI32, {B});
    void* lens = a.next("seq_lens", kI32, {B});
    t = a.tensor("k_cache");
    if (a.ok()) a.dims("k_cache", t, 4);
    const int pages = a.size(t, 0, "k_cache"), d = a.size(t, 3, "k_cache");
    void* k = a.ok() ? a.at("k_cache", t, kBf16, {pages, c.h_kv, c.page, d}) : nullptr;
    void* v = a.next("v_cache", kBf16, {pages, c.h_kv, c.page, d});
    t = a.tensor("dst_table");
    if (a.ok()) a.dims("dst_table", t, 2);
    const int dst_width = a.size(t, 1, "dst_table");
    void* dst = a.ok() ? a.at("dst_table", t, kI32, {B, dst_width}) : nullptr;
    t = a.tensor("workspace");
    void* w = a.ok() ? a.at("workspace", t, kU8, {t->numel()}) : nullptr;
    return a.call([&](moe_stream_t s) {
      return moe_kv4_load(static_cast<uint8_t*>(c.at), in(table), in(first), in(lens), B, c.h_kv, d, c.pages, c.page, width, bf(k),
                          bf(v), in(dst), pages, dst_width, w, t->numel(), s);
    });
  });
}

#define PAGED_METHOD(name) {"moe_" #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PAGED_METHOD(paged_plan),        PAGED_METHOD(qk_norm_rope),      PAGED_METHOD(gqa_paged_decode),
                         PAGED_METHOD(gqa_paged_prefill), PAGED_METHOD(gqa_prefix_decode), PAGED_METHOD(qk_norm_mrope),
                         PAGED_METHOD(qk_norm_rope_kv4),  PAGED_METHOD(gqa_kv4_decode),    PAGED_METHOD(kv4_load),
                         PAGED_METHOD(add_rms_norm),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
