// The Python side of the tables, the cache writes and the 8-bit cache: arguments checked and handed to
// the C ABI in one native call each.  A decode step's calls are short (3 to 7 us on the device), so
// what their checks cost counts: with ctypes and a Python check per tensor they took 8 to 11 us of
// host time and the attention 21, here 2.6 to 3.2 and 7 to 8 (two allocations and a launch of 2 us among
// them; GB300's Grace cores).  Nothing but marshalling happens here: the tensors' types, sizes, order
// and device are checked, as the C ABI, which checks everything else, sees addresses only.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <exception>

#include "scout.h"

namespace {

PyObject* g_error = nullptr;   // ScoutError
PyObject* g_memory = nullptr;  // torch.OutOfMemoryError

// The product of sizes; -1, which no tensor has, when it passes 64 bits.
template <class... A>
int64_t count(int64_t first, A... rest) {
  int64_t n = first;
  bool over = false;
  ((over = over || __builtin_mul_overflow(n, (int64_t)rest, &n)), ...);
  return over ? -1 : n;
}

// The arguments of one call, read in order; the first that does not fit sets the Python error and
// makes everything after it a no-op.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : at_(args), end_(args + n) {
    if (n != want) {
      PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, n);
      ok_ = false;
    }
  }
  bool ok() const { return ok_; }
  int device() const { return device_; }
  PyObject* raw() { return ok_ ? *at_++ : Py_None; }

  int64_t num() {
    if (!ok_) return 0;
    const long long v = PyLong_AsLongLong(*at_++);
    if (v == -1 && PyErr_Occurred()) ok_ = false;
    return v;
  }
  // a C int of the ABI
  int i32() {
    const int64_t v = num();
    if (ok_ && v != (int)v) {
      PyErr_Format(g_error, "%lld does not fit a 32-bit size", (long long)v);
      ok_ = false;
    }
    return (int)v;
  }
  double real() {
    if (!ok_) return 0.0;
    const double v = PyFloat_AsDouble(*at_++);
    if (v == -1.0 && PyErr_Occurred()) ok_ = false;
    return v;
  }

  // a tensor of any size; its device is looked at in settle()
  const at::Tensor* tensor(const char* name) {
    if (!ok_) return nullptr;
    PyObject* o = *at_++;
    if (!THPVariable_Check(o)) {
      fail("%s must be a CUDA tensor, got %s", name, Py_TYPE(o)->tp_name);
      return nullptr;
    }
    const at::Tensor* t = &THPVariable_Unpack(o);
    const int d = t->is_cuda() ? (int)t->get_device() : -1;
    if (device_ == kNone) device_ = d;
    if ((d < 0 || d != device_) && elsewhere_ == nullptr) elsewhere_ = name;
    return t;
  }
  // After the last tensor: all of them on one device, the current one.
  bool settle() {
    if (!ok_) return false;
    if (elsewhere_ != nullptr)
      fail("%s must be a CUDA tensor on the call's device", elsewhere_);
    else if (device_ != c10::cuda::current_device())
      fail("the tensors of a call must be on the current device, got cuda:%d", device_);
    return ok_;
  }
  // its address, once type, elements and contiguity fit
  void* sized(const at::Tensor* t, const char* name, at::ScalarType type, int64_t numel) {
    if (!ok_) return nullptr;
    if (t->scalar_type() != type || t->numel() != numel || !t->is_contiguous()) {
      fail("%s must be a contiguous CUDA tensor of %lld %s elements, got %lld %s%s", name, (long long)numel,
           c10::toString(type), (long long)t->numel(), c10::toString(t->scalar_type()),
           t->is_contiguous() ? "" : ", strided");
      return nullptr;
    }
    return t->data_ptr();
  }
  void* sized(const char* name, at::ScalarType type, int64_t numel) { return sized(tensor(name), name, type, numel); }
  // the same, or None
  const at::Tensor* optional(const char* name) {
    if (!ok_) return nullptr;
    if (*at_ == Py_None) {
      ++at_;
      return nullptr;
    }
    return tensor(name);
  }
  void* optional(const char* name, at::ScalarType type, int64_t numel) {
    const at::Tensor* t = optional(name);
    return t == nullptr ? nullptr : sized(t, name, type, numel);
  }
  // An output with room for `rows` rows, or None.  One without room has no address of its own but is still
  // asked for: it gets one that nothing is written to, so that what does not fit is reported.
  void* room(const at::Tensor* t, const char* name, at::ScalarType type, int rows, int64_t width) {
    if (t == nullptr) return nullptr;
    void* p = sized(t, name, type, count(rows, width));
    return rows == 0 ? reinterpret_cast<void*>(kNowhere) : p;
  }
  // rows [n_tokens][Hkv][D], each token's heads contiguous; ld: elements from a token to the next
  void* rows(const char* name, int Hkv, int64_t D, int64_t* n, int64_t* ld) {
    const at::Tensor* t = tensor(name);
    if (!ok_) return nullptr;
    if (t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(1) != Hkv || t->size(2) != D) {
      fail("%s must be a bf16 CUDA tensor [n_tokens][%d][%lld]", name, Hkv, (long long)D);
      return nullptr;
    }
    *n = t->size(0);
    if (*n != (int)*n) {
      fail("%s: %lld tokens do not fit a 32-bit size", name, (long long)*n);
      return nullptr;
    }
    if (*n > 0 && (t->stride(2) != 1 || (Hkv > 1 && t->stride(1) != D))) {
      fail("%s: the heads of a token must be contiguous", name);
      return nullptr;
    }
    *ld = *n > 1 ? t->stride(0) : Hkv * D;
    return t->data_ptr();
  }
  // None (the current stream of the call's device) or a torch.cuda.Stream; the last argument
  cudaStream_t stream(bool* given = nullptr) {
    if (!settle()) return nullptr;
    PyObject* o = *at_++;
    if (given != nullptr) *given = o != Py_None;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_).stream();
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    void* s = h != nullptr ? PyLong_AsVoidPtr(h) : nullptr;
    Py_XDECREF(h);
    if (PyErr_Occurred()) ok_ = false;
    return static_cast<cudaStream_t>(s);
  }
  template <class... A>
  void fail(const char* text, A... a) {
    if (ok_) PyErr_Format(g_error, text, a...);
    ok_ = false;
  }

 private:
  static constexpr int kNone = -2;
  static constexpr uintptr_t kNowhere = 256;
  PyObject* const* at_;
  PyObject* const* end_;
  int device_ = kNone;                // of the first tensor
  const char* elsewhere_ = nullptr;   // the first tensor that is not on it, or not on a GPU
  bool ok_ = true;
};

// The format of an 8-bit pool [n_slots][P][D]; V (or null) alike.
int format_of(Args& a, const at::Tensor* t, const at::Tensor* v, int P) {
  if (!a.ok()) return 0;
  const at::ScalarType s = t->scalar_type();
  if (s != at::kFloat8_e4m3fn && s != at::kFloat8_e5m2) {
    a.fail("an 8-bit pool must be float8_e4m3fn or float8_e5m2, got %s", c10::toString(s));
    return 0;
  }
  if (t->dim() != 3 || t->size(1) != P || (v != nullptr && (v->scalar_type() != s || v->sizes() != t->sizes())))
    a.fail("the pools must be [n_slots][%d][D] alike", P);
  else if (t->size(2) != (int)t->size(2))
    a.fail("a row of %lld elements does not fit a 32-bit size", (long long)t->size(2));
  return s == at::kFloat8_e4m3fn ? SCOUT_FP8_E4M3 : SCOUT_FP8_E5M2;
}

// The last size of a table's tensor: its blocks a sequence.
int last_size(Args& a, const at::Tensor* t, const char* name) {
  if (!a.ok()) return 0;
  const int64_t n = t->dim() > 0 ? t->size(-1) : 0;
  if (n != (int)n) a.fail("%s: %lld blocks do not fit a 32-bit size", name, (long long)n);
  return (int)n;
}
// The first size of a list, 0 without one.
int first_size(Args& a, const at::Tensor* t, const char* name) {
  if (!a.ok() || t == nullptr) return 0;
  const int64_t n = t->dim() > 0 ? t->size(0) : 0;
  if (n != (int)n) a.fail("%s: %lld entries do not fit a 32-bit size", name, (long long)n);
  return (int)n;
}

PyObject* done(int rc, const char* what) {
  if (rc == SCOUT_OK) Py_RETURN_NONE;
  PyErr_Format(g_error, "%s: %s", what, scout_status_string(rc));
  return nullptr;
}

// Runs f, with C++ exceptions as Python errors: an allocation that fails as PyTorch's own calls raise it.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (page_table, seq_len, free_slots | None, n_slots, B, Hkv, P, resident_bits, prev_len | None, cu_tokens | None,
//  slot_map | None, block_list | None, counts | None, status | None, stream | None)
PyObject* build_tables(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 15);
    const at::Tensor *pt = a.tensor("page_table"), *seq = a.tensor("seq_len"), *fr = a.optional("free_slots");
    const int64_t n_slots = a.num();
    const int B = a.i32(), Hkv = a.i32(), P = a.i32();
    const int cap = last_size(a, pt, "page_table");
    auto pt_p = static_cast<int32_t*>(a.sized(pt, "page_table", at::kInt, count(B, Hkv, cap)));
    auto seq_p = static_cast<const int32_t*>(a.sized(seq, "seq_len", at::kInt, B));
    const int64_t n_free = a.ok() && fr != nullptr ? fr->numel() : n_slots;
    auto fr_p = static_cast<const int32_t*>(fr != nullptr ? a.sized(fr, "free_slots", at::kInt, n_free) : nullptr);
    auto bits = static_cast<uint32_t*>(a.sized("resident_bits", at::kInt, count(B, Hkv, ((int64_t)cap + 31) / 32)));
    auto prev = static_cast<const int32_t*>(a.optional("prev_len", at::kInt, B));
    auto cu = static_cast<int32_t*>(a.optional("cu_tokens", at::kInt, (int64_t)B + 1));
    const at::Tensor* map = a.optional("slot_map");
    const int max_tokens = first_size(a, map, "slot_map");
    auto map_p = static_cast<int64_t*>(a.room(map, "slot_map", at::kLong, max_tokens, Hkv));
    const at::Tensor* list = a.optional("block_list");
    const int max_list = first_size(a, list, "block_list");
    auto list_p = static_cast<int32_t*>(a.room(list, "block_list", at::kInt, max_list, 2));
    auto counts = static_cast<int32_t*>(a.optional("counts", at::kInt, 3));
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    const cudaStream_t st = a.stream();
    if (n_free != (int)n_free) a.fail("%lld free slots do not fit a 32-bit size", (long long)n_free);
    if (!a.ok()) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = scout_build_tables(prev, seq_p, fr_p, (int)n_free, n_slots, B, Hkv, P, cap, pt_p, bits, cu, map_p, max_tokens,
                            list_p, max_list, counts, status, st);
    Py_END_ALLOW_THREADS;
    return done(rc, "scout_build_tables");
  });
}

// (K_pool, V_pool, Hkv, P, K_new, V_new, slot_map, status | None, stream | None)
PyObject* append_kv(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 9);
    const at::Tensor *kp = a.tensor("K_pool"), *vp = a.tensor("V_pool");
    const int Hkv = a.i32(), P = a.i32();
    if (a.ok() && (kp->dim() != 3 || kp->size(2) != (int)kp->size(2)))
      a.fail("K_pool must be a CUDA tensor [n_slots][%d][D]", P);
    if (!a.ok()) return nullptr;
    const int64_t slots = kp->size(0), D = kp->size(2), pool = count(slots, P, D);
    void *kpp = a.sized(kp, "K_pool", at::kBFloat16, pool), *vpp = a.sized(vp, "V_pool", at::kBFloat16, pool);
    int64_t nk = 0, nv = 0, ld_k = 0, ld_v = 0;
    void *k = a.rows("K_new", Hkv, D, &nk, &ld_k), *v = a.rows("V_new", Hkv, D, &nv, &ld_v);
    if (nk != nv) a.fail("K_new and V_new must hold the same tokens");
    auto map = static_cast<const int64_t*>(a.sized("slot_map", at::kLong, count(nk, Hkv)));
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    const cudaStream_t st = a.stream();
    if (!a.ok()) return nullptr;
    if (nk == 0) Py_RETURN_NONE;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = scout_append_kv(k, ld_k, v, ld_v, map, (int)nk, Hkv, (int)D, P, kpp, vpp, slots, status, st);
    Py_END_ALLOW_THREADS;
    return done(rc, "scout_append_kv");
  });
}

// (K_pool, V_pool, B, Hkv, P, K_new, V_new, page_table, seq_len, K_scale, V_scale, prev_len | None, status | None,
//  stream | None)
PyObject* append_kv8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 14);
    const at::Tensor *kp = a.tensor("K_pool"), *vp = a.tensor("V_pool");
    const int B = a.i32(), Hkv = a.i32(), P = a.i32();
    const int fmt = format_of(a, kp, vp, P);
    if (!a.ok()) return nullptr;
    const at::ScalarType type = kp->scalar_type();
    const int64_t slots = kp->size(0), D = kp->size(2), pool = count(slots, P, D);
    void *kpp = a.sized(kp, "K_pool", type, pool), *vpp = a.sized(vp, "V_pool", type, pool);
    int64_t nk = 0, nv = 0, ld_k = 0, ld_v = 0;
    void *k = a.rows("K_new", Hkv, D, &nk, &ld_k), *v = a.rows("V_new", Hkv, D, &nv, &ld_v);
    if (nk != nv) a.fail("K_new and V_new must hold the same tokens");
    const at::Tensor* pt = a.tensor("page_table");
    const int cap = last_size(a, pt, "page_table");
    auto pt_p = static_cast<const int32_t*>(a.sized(pt, "page_table", at::kInt, count(B, Hkv, cap)));
    auto seq = static_cast<const int32_t*>(a.sized("seq_len", at::kInt, B));
    auto ks = static_cast<float*>(a.sized("K_scale", at::kFloat, slots));
    auto vs = static_cast<float*>(a.sized("V_scale", at::kFloat, slots));
    auto prev = static_cast<const int32_t*>(a.optional("prev_len", at::kInt, B));
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    const cudaStream_t st = a.stream();
    if (!a.ok()) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = scout_append_kv8(fmt, k, ld_k, v, ld_v, (int)nk, prev, seq, pt_p, B, Hkv, (int)D, P, cap, kpp, vpp, ks, vs, slots,
                          status, st);
    Py_END_ALLOW_THREADS;
    return done(rc, "scout_append_kv8");
  });
}

// (kind, K_pool, B, Hkv, P, K_scale, page_table, seq_len, digest, block_list | None, status | None, stream | None)
PyObject* build_digest8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 12);
    const int kind = a.i32();
    const at::Tensor* kp = a.tensor("K_pool");
    const int B = a.i32(), Hkv = a.i32(), P = a.i32();
    const int fmt = format_of(a, kp, nullptr, P);
    if (!a.ok()) return nullptr;
    const int64_t slots = kp->size(0), D = kp->size(2);
    void* kpp = a.sized(kp, "K_pool", kp->scalar_type(), count(slots, P, D));
    auto ks = static_cast<const float*>(a.sized("K_scale", at::kFloat, slots));
    const at::Tensor* pt = a.tensor("page_table");
    const int cap = last_size(a, pt, "page_table");
    auto pt_p = static_cast<const int32_t*>(a.sized(pt, "page_table", at::kInt, count(B, Hkv, cap)));
    auto seq = static_cast<const int32_t*>(a.sized("seq_len", at::kInt, B));
    const bool minmax = kind == SCOUT_DIGEST_MINMAX;
    void* dg = a.sized("digest", minmax ? at::kBFloat16 : at::kFloat, count(B, Hkv, cap, D, minmax ? 2 : 1));
    const at::Tensor* list = a.optional("block_list");
    const int n_list = first_size(a, list, "block_list");
    auto list_p = static_cast<const int32_t*>(list != nullptr ? a.sized(list, "block_list", at::kInt, count(n_list, 2)) : nullptr);
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    const cudaStream_t st = a.stream();
    if (!a.ok()) return nullptr;
    if (list != nullptr && n_list == 0) Py_RETURN_NONE;  // an empty list, which has no address, is not "all blocks"
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = scout_build_digest8(kind, fmt, kpp, ks, slots, pt_p, seq, B, Hkv, (int)D, P, cap, list_p, n_list, dg, status, st);
    Py_END_ALLOW_THREADS;
    return done(rc, "scout_build_digest8");
  });
}

// (q, K_pool, V_pool, K_scale, V_scale, page_table, seq_len, res_list, res_count, B, Hq, Hkv, P, k, scale, workspace,
//  O_cpu, lse_cpu, O | None, lse | None, status | None, max_ctas | None, stream | None) -> (O, lse).  O_cpu and lse_cpu
// are both None for the partial alone.
PyObject* sparse_attn8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 23);
    const at::Tensor *q = a.tensor("q"), *kp = a.tensor("K_pool"), *vp = a.tensor("V_pool"), *ks = a.tensor("K_scale"),
                     *vs = a.tensor("V_scale"), *pt = a.tensor("page_table"), *seq = a.tensor("seq_len"),
                     *list = a.tensor("res_list"), *counts = a.tensor("res_count");
    const int B = a.i32(), Hq = a.i32(), Hkv = a.i32(), P = a.i32(), k = a.i32();
    const float scale = (float)a.real();
    const int fmt = format_of(a, kp, vp, P);
    if (!a.ok()) return nullptr;
    const at::ScalarType type = kp->scalar_type();
    const int64_t slots = kp->size(0), D = kp->size(2), pool = count(slots, P, D);
    const int cap = last_size(a, pt, "page_table");
    const void *q_p = a.sized(q, "q", at::kBFloat16, count(B, Hq, D)), *kpp = a.sized(kp, "K_pool", type, pool),
               *vpp = a.sized(vp, "V_pool", type, pool);
    auto ks_p = static_cast<const float*>(a.sized(ks, "K_scale", at::kFloat, slots));
    auto vs_p = static_cast<const float*>(a.sized(vs, "V_scale", at::kFloat, slots));
    auto pt_p = static_cast<const int32_t*>(a.sized(pt, "page_table", at::kInt, count(B, Hkv, cap)));
    auto seq_p = static_cast<const int32_t*>(a.sized(seq, "seq_len", at::kInt, B));
    auto list_p = static_cast<const int32_t*>(a.sized(list, "res_list", at::kInt, count(B, Hkv, k)));
    auto count_p = static_cast<const int32_t*>(a.sized(counts, "res_count", at::kInt, count(B, Hkv)));
    const at::Tensor* ws = a.tensor("workspace");
    const int64_t wsb = a.ok() ? ws->numel() : 0;
    void* ws_p = a.sized(ws, "workspace", at::kByte, wsb);
    const at::Tensor *oc = a.optional("O_cpu"), *lc = a.optional("lse_cpu");
    const bool merge = oc != nullptr || lc != nullptr;
    if (merge && (oc == nullptr || lc == nullptr)) a.fail("O_cpu and lse_cpu must be CUDA tensors");
    auto oc_p = static_cast<const float*>(merge ? a.sized(oc, "O_cpu", at::kFloat, count(B, Hq, D)) : nullptr);
    auto lc_p = static_cast<const float*>(merge ? a.sized(lc, "lse_cpu", at::kFloat, count(B, Hq)) : nullptr);
    const at::ScalarType otype = merge ? at::kBFloat16 : at::kFloat;
    const at::Tensor *o_given = a.optional("O"), *l_given = a.optional("lse");
    if (o_given != nullptr) a.sized(o_given, "O", otype, count(B, Hq, D));
    if (l_given != nullptr) a.sized(l_given, "lse", at::kFloat, count(B, Hq));
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    PyObject* max_ctas = a.raw();
    bool named = false;
    const cudaStream_t st = a.stream(&named);
    scout_launch launch = {};
    if (a.ok() && max_ctas != Py_None) {
      const long m = PyLong_AsLong(max_ctas);
      if (m == -1 && PyErr_Occurred()) return nullptr;
      if (m < 0 || m != (int)m) a.fail("max_ctas must be >= 0");
      launch.max_ctas = (int)m;
    }
    if (!a.ok()) return nullptr;
    at::Tensor O, lse;
    {
      // outputs made here come from the stream they are written on
      c10::cuda::OptionalCUDAStreamGuard on;
      if (named && (o_given == nullptr || l_given == nullptr))
        on.reset_stream(c10::cuda::getStreamFromExternal(st, (c10::DeviceIndex)a.device()));
      const at::TensorOptions opt = at::TensorOptions().device(q->device());
      O = o_given != nullptr ? *o_given : at::empty({B, Hq, D}, opt.dtype(otype));
      lse = l_given != nullptr ? *l_given : at::empty({B, Hq}, opt.dtype(at::kFloat));
    }
    void* o_p = O.data_ptr();
    auto l_p = static_cast<float*>(lse.data_ptr());
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = merge ? scout_sparse_attn8_merge(fmt, q_p, kpp, vpp, ks_p, vs_p, slots, pt_p, seq_p, list_p, count_p, B, Hq, Hkv,
                                          (int)D, P, cap, k, scale, oc_p, lc_p, o_p, l_p, ws_p, (size_t)wsb, status,
                                          &launch, st)
               : scout_sparse_attn8(fmt, q_p, kpp, vpp, ks_p, vs_p, slots, pt_p, seq_p, list_p, count_p, B, Hq, Hkv,
                                    (int)D, P, cap, k, scale, static_cast<float*>(o_p), l_p, ws_p, (size_t)wsb, status,
                                    &launch, st);
    Py_END_ALLOW_THREADS;
    if (rc != SCOUT_OK) return done(rc, merge ? "scout_sparse_attn8_merge" : "scout_sparse_attn8");
    PyObject *first = THPVariable_Wrap(O), *second = first != nullptr ? THPVariable_Wrap(lse) : nullptr;
    PyObject* both = second != nullptr ? PyTuple_Pack(2, first, second) : nullptr;
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
  });
}

// (ScoutError, torch.OutOfMemoryError)
PyObject* set_errors(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "2 arguments expected");
    return nullptr;
  }
  Py_XSETREF(g_error, Py_NewRef(args[0]));
  Py_XSETREF(g_memory, Py_NewRef(args[1]));
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}
PyMethodDef g_methods[] = {{"build_tables", fast(build_tables), METH_FASTCALL, nullptr},
                           {"append_kv", fast(append_kv), METH_FASTCALL, nullptr},
                           {"append_kv8", fast(append_kv8), METH_FASTCALL, nullptr},
                           {"build_digest8", fast(build_digest8), METH_FASTCALL, nullptr},
                           {"sparse_attn8", fast(sparse_attn8), METH_FASTCALL, nullptr},
                           {"set_errors", fast(set_errors), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#define SCOUT_TEXT_(x) #x
#define SCOUT_TEXT(x) SCOUT_TEXT_(x)

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&g_module);
  // the PyTorch whose headers this was built with: its objects are read by their layout there
  if (m != nullptr &&
      (PyModule_AddStringConstant(m, "torch_version", SCOUT_TEXT(TORCH_VERSION_MAJOR) "." SCOUT_TEXT(
                                      TORCH_VERSION_MINOR) "." SCOUT_TEXT(TORCH_VERSION_PATCH)) != 0 ||
       PyModule_AddIntConstant(m, "attn8_zero_bytes", SCOUT_SPARSE_ATTN8_ZERO_BYTES) != 0))
    Py_CLEAR(m);
  return m;
}
