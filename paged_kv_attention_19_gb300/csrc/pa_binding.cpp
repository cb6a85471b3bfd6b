// pa_binding.cpp -- the Python calls of the tree-drafting operators: checks of the tensors (type, shape,
// strides, device), then the C ABI on the tensors' device and stream.  In C++ because a step makes these
// calls often and small: the checks take about a microsecond here and ten or more in Python.
//
// Every function takes its arguments by position and returns None, a status of the C ABI, or a text
// that says what is wrong with an argument; __init__.py turns the last two into PaError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <sstream>
#include <string>

#include "pa_decode.h"

namespace {

struct Refused {
  std::string why;
};

template <typename... T>
[[noreturn]] void refuse(const T &...parts) {
  std::ostringstream s;
  (s << ... << parts);
  throw Refused{s.str()};
}

const char *kind_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kFloat: return "float32";
    case at::kBFloat16: return "bfloat16";
    case at::kByte: return "uint8";
    default: return c10::toString(t);
  }
}

// The arguments of one call, taken in order.
class Args {
 public:
  Args(PyObject *const *values, Py_ssize_t count, Py_ssize_t want) : v_(values) {
    if (count != want) refuse("takes ", (long)want, " arguments, got ", (long)count);
  }
  bool none() const { return v_[i_] == Py_None; }
  void skip() { ++i_; }

  const at::Tensor &tensor(const char *name) {
    PyObject *p = v_[i_++];
    if (!THPVariable_Check(p)) refuse(name, " has to be a tensor");
    return THPVariable_Unpack(p);
  }

  // A dense tensor of this type and shape on the call's device (the first tensor's).
  void *array(const char *name, at::ScalarType kind, std::initializer_list<int64_t> shape) {
    const at::Tensor &t = tensor(name);
    take_device(t);
    if (t.scalar_type() != kind || !same(t.sizes(), shape) || !t.is_contiguous() || t.device() != device())
      wrong(name, t, kind, shape, "dense ");
    return t.data_ptr();
  }
  void *optional(const char *name, at::ScalarType kind, std::initializer_list<int64_t> shape) {
    if (none()) {
      skip();
      return nullptr;
    }
    return array(name, kind, shape);
  }

  // Token rows of dense heads, any multiple of values apart.
  const at::Tensor &heads(const char *name, int64_t tokens, int64_t n, int64_t dim, long long *stride) {
    const at::Tensor &t = tensor(name);
    take_device(t);
    if (t.scalar_type() != at::kBFloat16 || !same(t.sizes(), {tokens, n, dim}) || t.device() != device() ||
        (dim > 1 && t.stride(2) != 1) || (n > 1 && t.stride(1) != dim))
      wrong(name, t, at::kBFloat16, {tokens, n, dim}, "");
    *stride = tokens > 1 ? t.stride(0) : n * dim;  // (a single token's stride says nothing)
    return t;
  }

  int integer(const char *name) {
    const long long x = PyLong_AsLongLong(v_[i_]);
    if (x == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(name, " has to be a whole number");
    }
    ++i_;
    if (x < INT_MIN || x > INT_MAX) refuse(name, " is out of range");
    return (int)x;
  }
  float real(const char *name) {
    const double x = PyFloat_AsDouble(v_[i_]);
    if (x == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse(name, " has to be a number");
    }
    ++i_;
    return (float)x;
  }

  at::Device device() const { return at::Device(at::DeviceType(kind_), (at::DeviceIndex)index_); }

  // The last argument: a stream (None: the current one of the tensors' device, a handle, or a torch stream).
  // Calls f(stream) with that device current; returns what the Python function returns.
  template <typename F>
  PyObject *launch(F f) {
    if (device().type() != at::kCUDA) refuse("the tensors are on ", device().str(), ", not on a GPU");
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != device().index()) guard.set_device(device());
    cudaStream_t stream = nullptr;
    PyObject *s = v_[i_];
    if (s == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(device().index()).stream();
    } else {
      PyObject *held = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
      void *p = held ? PyLong_AsVoidPtr(held) : nullptr;
      Py_XDECREF(held);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse("stream has to be None, a handle or a torch.cuda.Stream");
      }
      stream = static_cast<cudaStream_t>(p);
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = f(stream);
    Py_END_ALLOW_THREADS
    if (rc == PA_OK) Py_RETURN_NONE;
    return PyLong_FromLong(rc);
  }

 private:
  static bool same(at::IntArrayRef a, std::initializer_list<int64_t> b) {
    return a.size() == b.size() && std::equal(a.begin(), a.end(), b.begin());
  }
  void take_device(const at::Tensor &t) {
    if (index_ == -2) {
      kind_ = (int)t.device().type();
      index_ = t.device().index();
    }
  }
  [[noreturn]] void wrong(const char *name, const at::Tensor &t, at::ScalarType kind, std::initializer_list<int64_t> shape,
                          const char *dense) {
    std::ostringstream want;
    const char *sep = "";
    for (int64_t n : shape) {
      want << sep << n;
      sep = ", ";
    }
    refuse(name, " has to be a ", dense, kind_name(kind), " tensor of shape (", want.str(), ")", *dense ? "" : " whose heads are dense",
           " on ", device().str(), "; it is ", kind_name(t.scalar_type()), " ", t.sizes(), ", strides ", t.strides(), ", on ",
           t.device().str());
  }

  PyObject *const *v_;
  Py_ssize_t i_ = 0;
  int kind_ = 0, index_ = -2;  // the first tensor's device
};

const at::Tensor &peek(PyObject *const *v, Py_ssize_t count, Py_ssize_t i, const char *name, int dims) {
  if (i >= count || !THPVariable_Check(v[i])) refuse(name, " has to be a tensor");
  const at::Tensor &t = THPVariable_Unpack(v[i]);
  if (t.dim() != dims) refuse(name, " has to have ", dims, " dimensions; it has ", (long)t.dim());
  for (int64_t n : t.sizes())
    if (n > INT_MAX) refuse(name, " is too large");
  return t;
}

int64_t row_width(int fmt, int64_t D) { return fmt == 2 ? (D / 2 + D / 16 + 15) / 16 * 16 : D; }

template <typename F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const Refused &r) {
    return PyUnicode_FromStringAndSize(r.why.data(), (Py_ssize_t)r.why.size());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject *plan_step(PyObject *, PyObject *const *v, Py_ssize_t count) {
  return guarded([&] {
    Args a(v, count, 18);
    const int64_t B = peek(v, count, 0, "context_lens", 1).size(0), N = peek(v, count, 3, "free_list", 1).size(0),
                  W = peek(v, count, 5, "block_table", 2).size(1), T = peek(v, count, 11, "positions", 1).size(0);
    auto *lens = (const int32_t *)a.array("context_lens", at::kInt, {B});
    auto *news = (const int32_t *)a.array("new_lens", at::kInt, {B});
    auto *held = (const int32_t *)a.array("held_pages", at::kInt, {B});
    auto *list = (int32_t *)a.array("free_list", at::kInt, {N});
    auto *n_free = (const int32_t *)a.array("free_count", at::kInt, {1});
    auto *table = (int32_t *)a.array("block_table", at::kInt, {B, W});
    auto *lens_out = (int32_t *)a.array("context_lens_out", at::kInt, {B});
    auto *held_out = (int32_t *)a.array("held_pages_out", at::kInt, {B});
    auto *free_out = (int32_t *)a.array("free_count_out", at::kInt, {1});
    auto *start = (int32_t *)a.array("query_start", at::kInt, {B + 1});
    auto *slots = (int64_t *)a.array("slot_mapping", at::kLong, {T});
    auto *pos = (int32_t *)a.array("positions", at::kInt, {T});
    auto *parents = (const int32_t *)a.optional("parents", at::kInt, {T});
    auto *mask = (uint64_t *)a.optional("tree_mask", at::kLong, {T});
    auto *granted = (int32_t *)a.optional("granted", at::kInt, {B});
    auto *status = (uint32_t *)a.optional("status", at::kInt, {1});
    const int page = a.integer("page_size");
    return a.launch([&](cudaStream_t s) {
      return pa_plan_step_granted(lens, news, held, list, n_free, parents, table, lens_out, held_out, free_out, start, slots,
                                  pos, mask, granted, (int)B, page, (int)N, (int)W, (int)T, status, s);
    });
  });
}

PyObject *qk_norm_rope_write(PyObject *, PyObject *const *v, Py_ssize_t count) {
  return guarded([&] {
    Args a(v, count, 18);
    const int fmt = a.integer("format");
    const at::Tensor &q0 = peek(v, count, 1, "q", 3);
    const int64_t T = q0.size(0), Hq = q0.size(1), D = q0.size(2), Hkv = peek(v, count, 2, "k", 3).size(1);
    const at::Tensor &cs0 = peek(v, count, 6, "cos_sin", 2), &kp0 = peek(v, count, 10, "k_pool", 4);
    const int64_t far = cs0.size(0), rot = cs0.size(1), N = kp0.size(0), P = kp0.size(1), R = row_width(fmt, D);
    const at::ScalarType kind = fmt == 0 ? at::kBFloat16 : at::kByte;
    long long sq, sk, sv;
    const void *q = a.heads("q", T, Hq, D, &sq).data_ptr();
    const void *k = a.heads("k", T, Hkv, D, &sk).data_ptr();
    const void *val = a.heads("v", T, Hkv, D, &sv).data_ptr();
    const void *wq = a.optional("q_weight", at::kBFloat16, {D});
    const void *wk = a.optional("k_weight", at::kBFloat16, {D});
    auto *cs = (const float *)a.array("cos_sin", at::kFloat, {far, rot});
    auto *pos = (const int32_t *)a.array("positions", at::kInt, {T});
    auto *slots = (const int64_t *)a.array("slot_mapping", at::kLong, {T});
    void *out = a.array("q_out", at::kBFloat16, {T, Hq, D});
    void *kp = a.array("k_pool", kind, {N, P, Hkv, R});
    void *vp = a.array("v_pool", kind, {N, P, Hkv, R});
    auto *status = (uint32_t *)a.optional("status", at::kInt, {1});
    const float eps = a.real("eps");
    const int il = a.integer("interleaved");
    const float ks = a.real("k_scale"), vs = a.real("v_scale");
    return a.launch([&](cudaStream_t s) {
      if (fmt == 0)
        return pa_qk_norm_rope_write(q, k, val, wq, wk, cs, pos, slots, out, kp, vp, (int)T, (int)Hq, (int)Hkv, (int)D, sq, sk,
                                     sv, (int)rot, il, (int)far, eps, (int)P, (int)N, status, s);
      auto *f = fmt == 1 ? pa_qk_norm_rope_write_fp8 : pa_qk_norm_rope_write_nvfp4;
      return f(q, k, val, wq, wk, cs, pos, slots, out, kp, vp, (int)T, (int)Hq, (int)Hkv, (int)D, sq, sk, sv, (int)rot, il,
               (int)far, eps, ks, vs, (int)P, (int)N, status, s);
    });
  });
}

PyObject *tree_gqa(PyObject *, PyObject *const *v, Py_ssize_t count) {
  return guarded([&] {
    Args a(v, count, 20);
    const int fmt = a.integer("format");
    const at::Tensor &q0 = peek(v, count, 1, "q", 3), &kp0 = peek(v, count, 2, "k_pool", 4), &bt0 = peek(v, count, 4, "block_table", 2);
    const int64_t T = q0.size(0), Hq = q0.size(1), D = q0.size(2), N = kp0.size(0), P = kp0.size(1), Hkv = kp0.size(2);
    const int64_t B = bt0.size(0), W = bt0.size(1), R = row_width(fmt, D);
    const at::ScalarType kind = fmt == 0 ? at::kBFloat16 : at::kByte;
    const void *q = a.array("q", at::kBFloat16, {T, Hq, D});
    const void *kp = a.array("k_pool", kind, {N, P, Hkv, R});
    const void *vp = a.array("v_pool", kind, {N, P, Hkv, R});
    auto *bt = (const int32_t *)a.array("block_table", at::kInt, {B, W});
    auto *lens = (const int32_t *)a.array("context_lens", at::kInt, {B});
    auto *start = (const int32_t *)a.array("query_start", at::kInt, {B + 1});
    auto *mask = (const uint64_t *)a.array("tree_mask", at::kLong, {T});
    void *out = a.array("out", at::kBFloat16, {T, Hq, D});
    auto *lse = (float *)a.optional("lse", at::kFloat, {T, Hq});
    auto *granted = (const int32_t *)a.optional("granted", at::kInt, {B});
    const at::Tensor &ws = a.tensor("workspace");
    if (!ws.is_contiguous() || ws.device() != a.device()) refuse("workspace has to be a dense tensor on ", a.device().str());
    const int mq = a.integer("max_query");
    const float scale = a.real("scale"), ks = a.real("k_scale"), vs = a.real("v_scale");
    const int window = a.integer("window"), splits = a.integer("num_splits");
    int most = 0;
    if (a.none()) {
      a.skip();
      if (W * P > INT_MAX) refuse("block_table names more than 2^31 - 1 tokens a row: give max_context_len");
      most = (int)(W * P);
    } else {
      most = a.integer("max_context_len");
    }
    void *w = ws.data_ptr();
    const size_t wn = ws.nbytes();
    return a.launch([&](cudaStream_t s) {
      if (fmt == 0)
        return pa_tree_gqa_granted(q, kp, vp, bt, lens, start, mask, granted, out, lse, (int)B, (int)T, mq, (int)Hq, (int)Hkv,
                                   (int)D, (int)P, (int)N, (int)W, most, scale, window, splits, w, wn, s);
      auto *f = fmt == 1 ? pa_tree_gqa_fp8_granted : pa_tree_gqa_nvfp4_granted;
      return f(q, kp, vp, bt, lens, start, mask, granted, out, lse, (int)B, (int)T, mq, (int)Hq, (int)Hkv, (int)D, (int)P,
               (int)N, (int)W, most, scale, ks, vs, window, splits, w, wn, s);
    });
  });
}

PyObject *kv_compact(PyObject *, PyObject *const *v, Py_ssize_t count) {
  return guarded([&] {
    Args a(v, count, 11);
    if (!THPVariable_Check(v[0])) refuse("k_pool has to be a tensor");
    const at::Tensor &k = THPVariable_Unpack(v[0]);
    if (k.dim() != 4 && k.dim() != 5) refuse("k_pool has to have four or five dimensions; it has ", (long)k.dim());
    const int64_t L = k.dim() == 5 ? k.size(0) : 1, N = k.size(-4), P = k.size(-3), H = k.size(-2), R = k.size(-1);
    const at::Tensor &bt0 = peek(v, count, 2, "block_table", 2);
    const int64_t B = bt0.size(0), W = bt0.size(1), M = peek(v, count, 5, "accepted", 2).size(1);
    const at::ScalarType kind = k.scalar_type();
    void *kp, *vp;
    if (k.dim() == 5) {
      kp = a.array("k_pool", kind, {L, N, P, H, R});
      vp = a.array("v_pool", kind, {L, N, P, H, R});
    } else {
      kp = a.array("k_pool", kind, {N, P, H, R});
      vp = a.array("v_pool", kind, {N, P, H, R});
    }
    auto *bt = (const int32_t *)a.array("block_table", at::kInt, {B, W});
    auto *lens = (const int32_t *)a.array("context_lens", at::kInt, {B});
    auto *start = (const int32_t *)a.array("query_start", at::kInt, {B + 1});
    auto *acc = (const int32_t *)a.array("accepted", at::kInt, {B, M});
    auto *num = (const int32_t *)a.array("num_accepted", at::kInt, {B});
    auto *granted = (const int32_t *)a.optional("granted", at::kInt, {B});
    auto *out = (int32_t *)a.array("context_lens_out", at::kInt, {B});
    auto *status = (uint32_t *)a.optional("status", at::kInt, {1});
    const int64_t bytes = H * R * (int64_t)k.element_size();
    if (L > INT_MAX || N > INT_MAX || P > INT_MAX || bytes > INT_MAX) refuse("k_pool is too large");
    return a.launch([&](cudaStream_t s) {
      return pa_kv_compact_granted(kp, vp, bt, lens, start, acc, num, granted, out, (int)L, (int)B, (int)M, (int)bytes, (int)P,
                                   (int)N, (int)W, status, s);
    });
  });
}

#define PA_FUNCTION(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef functions[] = {PA_FUNCTION(plan_step), PA_FUNCTION(qk_norm_rope_write), PA_FUNCTION(tree_gqa),
                           PA_FUNCTION(kv_compact), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "pa_binding", "Tensor checks and calls of the C ABI.", -1, functions,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_pa_binding(void) { return PyModule_Create(&module); }
