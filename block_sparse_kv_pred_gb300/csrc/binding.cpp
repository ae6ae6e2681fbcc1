// The Python side of the tables, the cache writes, the 8-bit cache and a layer's row operators: arguments checked and handed to
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
    return ok_ ? tensor(*at_++, name) : nullptr;
  }
  const at::Tensor* tensor(PyObject* o, const char* name) {
    if (!ok_) return nullptr;
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
  // rows [n][heads][D] with any number of heads
  void* rows(const at::Tensor* t, const char* name, int64_t* n, int* heads, int64_t* D, int64_t* ld) {
    if (!ok_) return nullptr;
    if (t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(0) != (int)t->size(0) ||
        t->size(1) != (int)t->size(1) || t->size(2) != (int)t->size(2)) {
      fail("%s must be a bf16 CUDA tensor [n_tokens][heads][D] of 32-bit sizes", name);
      return nullptr;
    }
    *n = t->size(0);
    *heads = (int)t->size(1);
    *D = t->size(2);
    if (t->numel() > 0 && ((*D > 1 && t->stride(2) != 1) || (*heads > 1 && t->stride(1) != *D))) {
      fail("%s: the heads of a token must be contiguous", name);
      return nullptr;
    }
    *ld = *n > 1 ? t->stride(0) : *heads * *D;
    return t->data_ptr();
  }
  // a matrix [M][N] whose rows are contiguous; ld: elements from a row to the next
  void* matrix(const at::Tensor* t, const char* name, at::ScalarType type, int64_t M, int64_t N, int64_t* ld) {
    if (!ok_ || t == nullptr) return nullptr;
    if (t->scalar_type() != type || t->dim() != 2 || t->size(0) != M || t->size(1) != N ||
        (M > 0 && N > 1 && t->stride(1) != 1)) {
      fail("%s must be a %s CUDA tensor [%lld][%lld] with contiguous rows", name, c10::toString(type), (long long)M,
           (long long)N);
      return nullptr;
    }
    *ld = M > 1 ? t->stride(0) : N;
    return t->data_ptr();
  }
  // A tensor on the call's device or in host memory.  (What kind of host memory the C ABI looks at.)
  const at::Tensor* anywhere(const char* name) {
    if (!ok_) return nullptr;
    if (THPVariable_Check(*at_) && THPVariable_Unpack(*at_).is_cpu()) return &THPVariable_Unpack(*at_++);
    return tensor(name);
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

// One argument, a tuple (turns, rot_dim, layout, amplitude): a call with star arguments costs Python more.
scout_rope rope_of(Args& a) {
  scout_rope r = {};
  PyObject* o = a.raw();
  if (!a.ok()) return r;
  if (!PyTuple_CheckExact(o) || PyTuple_GET_SIZE(o) != 4) {
    a.fail("rope must be a Rope, got %s", Py_TYPE(o)->tp_name);
    return r;
  }
  const at::Tensor* t = a.tensor(PyTuple_GET_ITEM(o, 0), "rope.turns");
  const long rot_dim = PyLong_AsLong(PyTuple_GET_ITEM(o, 1));
  if (rot_dim != (int)rot_dim) a.fail("rope.rot_dim must fit 32 bits, got %ld", rot_dim);
  r.rot_dim = (int)rot_dim;
  r.layout = (int)PyLong_AsLong(PyTuple_GET_ITEM(o, 2));
  r.amplitude = (float)PyFloat_AsDouble(PyTuple_GET_ITEM(o, 3));
  if (a.ok() && PyErr_Occurred()) {
    PyErr_Clear();
    a.fail("rope must be a Rope: a number was expected");
  }
  r.turns = static_cast<const uint64_t*>(a.sized(t, "rope.turns", at::kLong, r.rot_dim / 2));
  return r;
}

// Outputs made here come from the stream they are written on (`named`: one that was given).
at::Tensor make(const at::Tensor* like, at::IntArrayRef sizes, at::ScalarType type, bool named, cudaStream_t st,
                int device) {
  c10::cuda::OptionalCUDAStreamGuard on;
  if (named) on.reset_stream(c10::cuda::getStreamFromExternal(st, (c10::DeviceIndex)device));
  return at::empty(sizes, at::TensorOptions().device(like->device()).dtype(type));
}

// (x, positions, rope, norm | None, eps, out | None, stream | None) -> out
PyObject* rotate(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 7);
    const at::Tensor* x = a.tensor("x");
    int64_t rows = 0, D = 0, ld_x = 0, rows_o = 0, D_o = 0, ld_o = 0;
    int heads = 0, heads_o = 0;
    const void* x_p = a.rows(x, "x", &rows, &heads, &D, &ld_x);
    auto pos = static_cast<const int32_t*>(a.sized("positions", at::kInt, rows));
    const scout_rope rope = rope_of(a);
    const void* norm = a.optional("norm", at::kBFloat16, D);
    const float eps = (float)a.real();
    const at::Tensor* given = a.optional("out");
    if (given != nullptr) {
      a.rows(given, "out", &rows_o, &heads_o, &D_o, &ld_o);
      if (rows_o != rows || heads_o != heads || D_o != D) a.fail("out must have the shape of x");
    }
    bool named = false;
    const cudaStream_t st = a.stream(&named);
    if (!a.ok()) return nullptr;
    const at::Tensor out = given != nullptr ? *given : make(x, {rows, heads, D}, at::kBFloat16, named, st, a.device());
    if (given == nullptr) ld_o = (int64_t)heads * D;
    if (rows > 0) {
      void* o_p = out.data_ptr();
      int rc;
      Py_BEGIN_ALLOW_THREADS;
      rc = scout_rotate(x_p, ld_x, o_p, ld_o, pos, (int)rows, heads, (int)D, &rope, norm, eps, st);
      Py_END_ALLOW_THREADS;
      if (rc != SCOUT_OK) return done(rc, "scout_rotate");
    }
    return THPVariable_Wrap(out);
  });
}

// The queries beside a write: q | None, q_norm | None, q_out | None, of n tokens.
struct Queries {
  const at::Tensor *q = nullptr, *given = nullptr;
  const void *p = nullptr, *norm = nullptr;
  at::Tensor out;
  int64_t ld = 0, ld_out = 0;
  int heads = 0;
  void read(Args& a, int64_t tokens, int64_t D) {
    q = a.optional("q");
    int64_t n = tokens, d = D, n_o = 0, d_o = 0;
    int h_o = 0;
    if (q != nullptr) {
      p = a.rows(q, "q", &n, &heads, &d, &ld);
      if (n != tokens || d != D || heads == 0) a.fail("q must hold the tokens of K_new, with heads of their size");
    }
    norm = a.optional("q_norm", at::kBFloat16, D);
    given = a.optional("q_out");
    if (q == nullptr && (norm != nullptr || given != nullptr)) a.fail("q_norm and q_out need q");
    if (given != nullptr) {
      a.rows(given, "q_out", &n_o, &h_o, &d_o, &ld_out);
      if (n_o != n || h_o != heads || d_o != d) a.fail("q_out must have the shape of q");
    }
  }
  // after the stream is known
  void* output(Args& a, int64_t tokens, int64_t D, bool named, cudaStream_t st) {
    if (q == nullptr) return nullptr;
    out = given != nullptr ? *given : make(q, {tokens, heads, D}, at::kBFloat16, named, st, a.device());
    if (given == nullptr) ld_out = (int64_t)heads * D;
    return out.data_ptr();
  }
  PyObject* result(int rc, const char* what) {
    if (rc != SCOUT_OK || q == nullptr) return done(rc, what);
    return THPVariable_Wrap(out);
  }
};

// (K_pool, V_pool, Hkv, P, K_new, V_new, positions, rope, k_norm | None, eps, slot_map, q | None, q_norm | None, q_out | None, status | None, stream | None) -> q_out | None
PyObject* append_rotated_kv(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 16);
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
    auto pos = static_cast<const int32_t*>(a.sized("positions", at::kInt, nk));
    const scout_rope rope = rope_of(a);
    const void* k_norm = a.optional("k_norm", at::kBFloat16, D);
    const float eps = (float)a.real();
    auto map = static_cast<const int64_t*>(a.sized("slot_map", at::kLong, count(nk, Hkv)));
    Queries q;
    q.read(a, nk, D);
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    bool named = false;
    const cudaStream_t st = a.stream(&named);
    if (!a.ok()) return nullptr;
    void* q_out = q.output(a, nk, D, named, st);
    int rc = SCOUT_OK;
    if (nk > 0) {
      Py_BEGIN_ALLOW_THREADS;
      rc = scout_append_rotated_kv(k, ld_k, v, ld_v, pos, &rope, k_norm, eps, map, (int)nk, Hkv, (int)D, P, kpp, vpp,
                                   slots, q.p, q.ld, q.heads, q.norm, q_out, q.ld_out, status, st);
      Py_END_ALLOW_THREADS;
    }
    return q.result(rc, "scout_append_rotated_kv");
  });
}

// (K_pool, V_pool, B, Hkv, P, K_new, V_new, rope, k_norm | None, eps, page_table, seq_len,
//  K_scale, V_scale, prev_len | None, positions | None, q | None, q_norm | None, q_out | None, status | None,
//  stream | None) -> q_out | None
PyObject* append_rotated_kv8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 21);
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
    const scout_rope rope = rope_of(a);
    const void* k_norm = a.optional("k_norm", at::kBFloat16, D);
    const float eps = (float)a.real();
    const at::Tensor* pt = a.tensor("page_table");
    const int cap = last_size(a, pt, "page_table");
    auto pt_p = static_cast<const int32_t*>(a.sized(pt, "page_table", at::kInt, count(B, Hkv, cap)));
    auto seq = static_cast<const int32_t*>(a.sized("seq_len", at::kInt, B));
    auto ks = static_cast<float*>(a.sized("K_scale", at::kFloat, slots));
    auto vs = static_cast<float*>(a.sized("V_scale", at::kFloat, slots));
    auto prev = static_cast<const int32_t*>(a.optional("prev_len", at::kInt, B));
    auto pos = static_cast<const int32_t*>(a.optional("positions", at::kInt, nk));
    Queries q;
    q.read(a, nk, D);
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    bool named = false;
    const cudaStream_t st = a.stream(&named);
    if (!a.ok()) return nullptr;
    void* q_out = q.output(a, nk, D, named, st);
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = scout_append_rotated_kv8(fmt, k, ld_k, v, ld_v, (int)nk, pos, &rope, k_norm, eps, prev, seq, pt_p, B, Hkv, (int)D,
                                  P, cap, kpp, vpp, ks, vs, slots, q.p, q.ld, q.heads, q.norm, q_out, q.ld_out, status, st);
    Py_END_ALLOW_THREADS;
    return q.result(rc, "scout_append_rotated_kv8");
  });
}

// (X, W, positions, rope, norm | None, eps, Q | None, status | None, max_ctas | None, stream | None) -> Q
PyObject* predict_q_rotated(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 10);
    const at::Tensor *x = a.tensor("X"), *w = a.tensor("W");
    if (a.ok() && (x->dim() != 2 || w->dim() != 2 || x->size(0) != (int)x->size(0) || x->size(1) != (int)x->size(1) ||
                   w->size(0) != (int)w->size(0)))
      a.fail("X must be [M][K] and W [N][K], of 32-bit sizes");
    if (!a.ok()) return nullptr;
    const int64_t M = x->size(0), K = x->size(1), N = w->size(0);
    const void *x_p = a.sized(x, "X", at::kBFloat16, count(M, K)), *w_p = a.sized(w, "W", at::kBFloat16, count(N, K));
    auto pos = static_cast<const int32_t*>(a.sized("positions", at::kInt, M));
    const scout_rope rope = rope_of(a);
    const void* norm = a.optional("norm", at::kBFloat16, 128);
    const float eps = (float)a.real();
    const at::Tensor* given = a.optional("Q");
    if (given != nullptr) a.sized(given, "Q", at::kBFloat16, count(M, N));
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
    const at::Tensor Q = given != nullptr ? *given : make(x, {M, N}, at::kBFloat16, named, st, a.device());
    void* q_p = Q.data_ptr();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = scout_predict_q_rotated(x_p, w_p, q_p, (int)M, (int)N, (int)K, pos, &rope, norm, eps, status, &launch, st);
    Py_END_ALLOW_THREADS;
    return rc != SCOUT_OK ? done(rc, "scout_predict_q_rotated") : THPVariable_Wrap(Q);
  });
}

// (K_pool, V_pool, B, Hkv, P, K_scale | None, V_scale | None, page_table, seq_len, K_out, V_out, block_list | None,
//  status | None, stream | None).  Without scales the pools are bf16.
PyObject* read_kv(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 14);
    const at::Tensor *kp = a.tensor("K_pool"), *vp = a.tensor("V_pool");
    const int B = a.i32(), Hkv = a.i32(), P = a.i32();
    const at::Tensor *ks = a.optional("K_scale"), *vs = a.optional("V_scale");
    const bool codes = ks != nullptr || vs != nullptr;
    if (codes && (ks == nullptr || vs == nullptr)) a.fail("K_scale and V_scale must be CUDA tensors");
    if (a.ok() && (kp->dim() != 3 || kp->size(2) != (int)kp->size(2)))
      a.fail("K_pool must be a CUDA tensor [n_slots][%d][D]", P);
    const int fmt = codes ? format_of(a, kp, vp, P) : 0;
    if (!a.ok()) return nullptr;
    const at::ScalarType type = codes ? kp->scalar_type() : at::kBFloat16;
    const int64_t slots = kp->size(0), D = kp->size(2), pool = count(slots, P, D);
    const void *kpp = a.sized(kp, "K_pool", type, pool), *vpp = a.sized(vp, "V_pool", type, pool);
    auto ks_p = static_cast<const float*>(codes ? a.sized(ks, "K_scale", at::kFloat, slots) : nullptr);
    auto vs_p = static_cast<const float*>(codes ? a.sized(vs, "V_scale", at::kFloat, slots) : nullptr);
    const at::Tensor* pt = a.tensor("page_table");
    const int cap = last_size(a, pt, "page_table");
    auto pt_p = static_cast<const int32_t*>(a.sized(pt, "page_table", at::kInt, count(B, Hkv, cap)));
    auto seq = static_cast<const int32_t*>(a.sized("seq_len", at::kInt, B));
    const at::Tensor* out[2] = {a.anywhere("K_out"), a.anywhere("V_out")};
    int64_t stride[3] = {0, 0, 0}, T = 0;
    if (a.ok()) {
      const at::Tensor &k = *out[0], &v = *out[1];
      if (k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 || k.dim() != 4 || k.size(0) != B ||
          k.size(1) != Hkv || k.size(3) != D || v.sizes() != k.sizes() || k.is_cuda() != v.is_cuda())
        a.fail("K_out and V_out must be bf16 tensors [%d][%d][T][%lld] alike", B, Hkv, (long long)D);
      else if (k.numel() > 0)
        for (int i = 0; i < 4; ++i) {
          if (k.size(i) == 1) continue;
          if (k.stride(i) != v.stride(i) || k.stride(i) == 0 || (i == 3 && k.stride(3) != 1))
            a.fail("K_out and V_out must have the same strides, with contiguous rows that do not overlap");
          else if (i < 3)
            stride[i] = k.stride(i);
        }
      T = k.dim() == 4 ? k.size(2) : 0;
    }
    const at::Tensor* list = a.optional("block_list");
    const int n_list = first_size(a, list, "block_list");
    auto list_p =
        static_cast<const int32_t*>(list != nullptr ? a.sized(list, "block_list", at::kInt, count(n_list, 2)) : nullptr);
    auto status = static_cast<int32_t*>(a.optional("status", at::kInt, 1));
    const cudaStream_t st = a.stream();
    if (!a.ok()) return nullptr;
    if (list != nullptr && n_list == 0) Py_RETURN_NONE;  // an empty list, which has no address, is not "all blocks"
    void *ko = out[0]->data_ptr(), *vo = out[1]->data_ptr();
    const int host = out[0]->is_cuda() ? 0 : 1;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = codes ? scout_read_kv8(fmt, kpp, vpp, ks_p, vs_p, slots, pt_p, seq, B, Hkv, (int)D, P, cap, list_p, n_list, ko, vo,
                                stride[0], stride[1], stride[2], T, host, status, st)
               : scout_read_kv(kpp, vpp, slots, pt_p, seq, B, Hkv, (int)D, P, cap, list_p, n_list, ko, vo, stride[0],
                               stride[1], stride[2], T, host, status, st);
    Py_END_ALLOW_THREADS;
    return done(rc, codes ? "scout_read_kv8" : "scout_read_kv");
  });
}

// (kind, Y | None, H, w, eps, b | None, w_post | None, b_post | None, gate | None, alpha, H_out | None, X | None,
//  w_ahead | None, b_ahead | None, X_ahead | None, stream | None) -> (H_out, X) or (H_out, X, X_ahead)
PyObject* add_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 16);
    const int kind = a.i32();
    const at::Tensor *y = a.optional("Y"), *h = a.tensor("H"), *w = a.tensor("w");
    const float eps = (float)a.real();
    if (a.ok() && (h->dim() != 2 || h->size(0) != (int)h->size(0) || h->size(1) != (int)h->size(1)))
      a.fail("H must be [M][N], of 32-bit sizes");
    if (!a.ok()) return nullptr;
    const int64_t M = h->size(0), N = h->size(1);
    const at::ScalarType wide = h->scalar_type();
    if (wide != at::kBFloat16 && wide != at::kFloat) a.fail("H must be bf16 or fp32, got %s", c10::toString(wide));
    int64_t ld_y = N, ld_h = N, ld_o = N, ld_g = 0;
    const void* y_p = a.matrix(y, "Y", at::kBFloat16, M, N, &ld_y);
    const void* h_p = a.matrix(h, "H", wide, M, N, &ld_h);
    const void* w_p = a.sized(w, "w", at::kBFloat16, N);
    const void* b_p = a.optional("b", at::kBFloat16, N);
    const void *wp_p = a.optional("w_post", at::kBFloat16, N), *bp_p = a.optional("b_post", at::kBFloat16, N);
    const at::Tensor* gate = a.optional("gate");
    const void* g_p = nullptr;
    if (a.ok() && gate != nullptr) {
      g_p = gate->dim() == 1 ? a.sized(gate, "gate", at::kBFloat16, N)
                             : a.matrix(gate, "gate", at::kBFloat16, M, N, &ld_g);
      if (gate->dim() == 1) ld_g = 0;
    }
    const float alpha = (float)a.real();
    const at::Tensor *h_out = a.optional("H_out"), *x = a.optional("X");
    a.matrix(h_out, "H_out", wide, M, N, &ld_o);
    if (h_out != nullptr && y == nullptr) a.fail("H_out needs Y: without it the stream stays as it is");
    if (x != nullptr) a.sized(x, "X", at::kBFloat16, count(M, N));
    const void* wa_p = a.optional("w_ahead", at::kBFloat16, N);
    const void* ba_p = a.optional("b_ahead", at::kBFloat16, N);
    const at::Tensor* xa = a.optional("X_ahead");
    if (xa != nullptr) a.sized(xa, "X_ahead", at::kBFloat16, count(M, N));
    if (wa_p == nullptr && (ba_p != nullptr || xa != nullptr)) a.fail("b_ahead and X_ahead need w_ahead");
    bool named = false;
    const cudaStream_t st = a.stream(&named);
    if (!a.ok()) return nullptr;
    at::Tensor H_out, X, XA;
    H_out = h_out != nullptr ? *h_out : y == nullptr ? *h : make(h, {M, N}, wide, named, st, a.device());
    X = x != nullptr ? *x : make(h, {M, N}, at::kBFloat16, named, st, a.device());
    if (wa_p != nullptr) XA = xa != nullptr ? *xa : make(h, {M, N}, at::kBFloat16, named, st, a.device());
    if (M > 0) {
      void *ho_p = y != nullptr ? H_out.data_ptr() : nullptr, *x_p = X.data_ptr(),
           *xa_p = wa_p != nullptr ? XA.data_ptr() : nullptr;
      int rc;
      Py_BEGIN_ALLOW_THREADS;
      rc = scout_add_norm(kind, y_p, ld_y, wp_p, bp_p, g_p, ld_g, alpha, wide == at::kFloat ? SCOUT_FP32 : SCOUT_BF16, h_p,
                          ld_h, ho_p, ld_o, w_p, b_p, x_p, wa_p, ba_p, xa_p, (int)M, (int)N, eps, st);
      Py_END_ALLOW_THREADS;
      if (rc != SCOUT_OK) return done(rc, "scout_add_norm");
    }
    PyObject* out[3] = {THPVariable_Wrap(H_out), THPVariable_Wrap(X), wa_p != nullptr ? THPVariable_Wrap(XA) : nullptr};
    PyObject* all = nullptr;
    if (out[0] != nullptr && out[1] != nullptr && (wa_p == nullptr || out[2] != nullptr))
      all = wa_p != nullptr ? PyTuple_Pack(3, out[0], out[1], out[2]) : PyTuple_Pack(2, out[0], out[1]);
    for (PyObject* o : out) Py_XDECREF(o);
    return all;
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
                           {"rotate", fast(rotate), METH_FASTCALL, nullptr},
                           {"append_rotated_kv", fast(append_rotated_kv), METH_FASTCALL, nullptr},
                           {"append_rotated_kv8", fast(append_rotated_kv8), METH_FASTCALL, nullptr},
                           {"predict_q_rotated", fast(predict_q_rotated), METH_FASTCALL, nullptr},
                           {"read_kv", fast(read_kv), METH_FASTCALL, nullptr},
                           {"add_norm", fast(add_norm), METH_FASTCALL, nullptr},
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
