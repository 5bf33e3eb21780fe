// The compiled half of _paged.py: argument checks, output allocation and the
// calls of the b200attn_paged_* entry points, on torch tensors. Nothing here
// computes. A decoding step makes these calls once per layer around kernels of
// a few microseconds; checks and conversions in Python with ctypes took 5-12 us
// a call, more than most of the kernels.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/record_stream.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/b200attn.h"

namespace {

// The library's entry points (the library may be another build of it), and
// whether tensors of any device are let through (tests with stand-ins).
decltype(&b200attn_paged_slots) fn_slots = nullptr;
decltype(&b200attn_paged_append) fn_append = nullptr;
decltype(&b200attn_paged_fwd) fn_fwd = nullptr;
decltype(&b200attn_paged_fwd_workspace_bytes) fn_ws = nullptr;
bool any_device = false;

struct Refused : std::invalid_argument {  // becomes ValueError
  using std::invalid_argument::invalid_argument;
};

std::string describe(PyObject* o) {
  if (!THPVariable_Check(o)) return Py_TYPE(o)->tp_name;
  const at::Tensor& t = THPVariable_Unpack(o);
  std::string s = c10::toString(t.scalar_type());
  s += " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] on " + t.device().str();
}

[[noreturn]] void refuse(const char* name, const std::string& what, PyObject* got) {
  throw Refused(std::string(name) + " must be " + what + ", got " + describe(got));
}

bool given(PyObject* o) { return o != nullptr && o != Py_None; }

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on_gpu(const at::Tensor& t) { return t.is_cuda() || any_device; }

int64_t integer(PyObject* o, const char* name) {
  PyObject* i = PyNumber_Index(o);
  if (!i) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be an integer");
  }
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(i, &overflow);
  Py_DECREF(i);
  if (overflow != 0) throw Refused(std::string(name) + " is out of range");
  return v;
}

int int32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) throw Refused(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

// A contiguous int32 [n] tensor on `dev` (any n where n < 0).
const at::Tensor& ints(PyObject* o, const char* name, int64_t n, const c10::Device* dev) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kInt || t->dim() != 1 || (n >= 0 && t->size(0) != n) || !t->is_contiguous() ||
      !on_gpu(*t) || (dev && t->device() != *dev))
    refuse(name, "a contiguous int32 CUDA tensor" + (n >= 0 ? " [" + std::to_string(n) + "]" : std::string(" [n]")) +
                     (dev ? " on " + dev->str() : std::string()), o);
  return *t;
}

struct Table {
  int* ptr;
  size_t row;
  int width;
};

Table table_of(PyObject* o, int64_t batch, const c10::Device& dev) {
  const at::Tensor* t = tensor(o);
  if (t && t->scalar_type() == at::kInt && t->dim() == 2 && t->device() == dev) {
    const int64_t width = t->size(1), row = t->size(0) == 1 ? width : t->stride(0);
    if (t->size(0) == batch && width > 0 && (width == 1 || t->stride(1) == 1) && row >= width)
      return {static_cast<int*>(t->data_ptr()), static_cast<size_t>(row), int32(width, "block_table's width")};
  }
  refuse("block_table",
         "int32 [" + std::to_string(batch) + ", pages] on " + dev.str() + " with contiguous rows that do not overlap", o);
}

struct Rows {
  const at::Tensor* t;
  int64_t n, heads, stride;
};

// bf16 [tokens, heads, d], each token contiguous, tokens any multiple of 8 elements apart.
Rows rows_of(PyObject* o, const char* name, int64_t d, const c10::Device& dev) {
  const at::Tensor* t = tensor(o);
  if (t && t->scalar_type() == at::kBFloat16 && t->dim() == 3 && t->device() == dev) {
    const int64_t n = t->size(0), h = t->size(1), stride = n > 1 ? t->stride(0) : h * d;
    if (t->size(2) == d && h > 0 && t->stride(2) == 1 && (h == 1 || t->stride(1) == d) && stride >= h * d &&
        stride % 8 == 0)
      return {t, n, h, stride};
  }
  refuse(name, "bf16 [tokens, heads, " + std::to_string(d) + "] on " + dev.str() +
                   " with contiguous heads, tokens that do not overlap and are a multiple of 8 elements apart", o);
}

// The cache tensors as the library takes them.
struct Cache {
  b200attn_paged_cache c;
  c10::Device dev;
};

const float* scale_of(PyObject* o, const char* name, int64_t heads, const c10::Device& dev) {
  if (!given(o)) throw Refused(std::string(name) + " is required for an e4m3 cache");
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != heads || t->device() != dev ||
      !t->is_contiguous())
    refuse(name, "contiguous fp32 [" + std::to_string(heads) + "] on " + dev.str(), o);
  return static_cast<const float*>(t->data_ptr());
}

Cache cache_of(PyObject* ko, PyObject* vo, PyObject* k_scale, PyObject* v_scale) {
  const at::Tensor *k = tensor(ko), *v = tensor(vo);
  for (auto [t, o, name] : {std::tuple{k, ko, "k_cache"}, std::tuple{v, vo, "v_cache"}})
    if (!t || t->dim() != 4 || !on_gpu(*t) || t->stride(3) != 1)
      refuse(name, "a 4-D [pages, page_size, H, d] CUDA tensor, d fastest", o);
  if (v->device() != k->device() || v->scalar_type() != k->scalar_type() || v->size(0) != k->size(0) ||
      v->size(1) != k->size(1) || v->size(2) != k->size(2))
    refuse("v_cache", "like k_cache (" + describe(ko) + ") in device, dtype, pages, page_size and heads", vo);
  const bool bf16 = k->scalar_type() == at::kBFloat16;
  if (!bf16 && k->scalar_type() != at::kFloat8_e4m3fn && k->scalar_type() != at::kByte)
    refuse("k_cache", "bf16 or e4m3", ko);
  Cache r{{}, k->device()};
  b200attn_paged_cache& c = r.c;
  c.num_pages = int32(k->size(0), "pages"), c.page_size = int32(k->size(1), "page_size"), c.Hkv = int32(k->size(2), "heads");
  c.d_qk = int32(k->size(3), "d"), c.d_v = int32(v->size(3), "d");
  if (c.num_pages < 1 || c.page_size < 1 || c.Hkv < 1) refuse("k_cache", "of at least one page, row and head", ko);
  if (bf16 && (given(k_scale) || given(v_scale))) throw Refused("scales are for e4m3 caches");
  c.dtype = bf16 ? B200ATTN_BF16 : B200ATTN_FP8_E4M3;
  c.k_scale = bf16 ? nullptr : scale_of(k_scale, "k_scale", c.Hkv, r.dev);
  c.v_scale = bf16 ? nullptr : scale_of(v_scale, "v_scale", c.Hkv, r.dev);
  // a dimension of one may come with any stride: what it would be
  auto strides = [&](const at::Tensor& t, const char* name, PyObject* o, int64_t& page, int64_t& token, int64_t& head) {
    const int64_t d = t.size(3), esz = bf16 ? 2 : 1;
    head = c.Hkv > 1 ? t.stride(2) : d;
    token = c.page_size > 1 ? t.stride(1) : c.Hkv * d;
    page = c.num_pages > 1 ? t.stride(0) : c.page_size * c.Hkv * d;
    if (page <= 0 || token <= 0 || head <= 0 || ((page | token | head) * esz & 15))
      refuse(name, "of strides that are positive multiples of 16 bytes", o);
  };
  strides(*k, "k_cache", ko, c.k_page_stride, c.k_token_stride, c.k_head_stride);
  strides(*v, "v_cache", vo, c.v_page_stride, c.v_token_stride, c.v_head_stride);
  c.k = k->data_ptr(), c.v = v->data_ptr();
  return r;
}

at::Tensor empty(c10::IntArrayRef shape, at::ScalarType dtype, const c10::Device& dev) {
  if (dev.is_cuda()) return at::Tensor(at::detail::empty_cuda(shape, dtype, dev, std::nullopt));
  return at::empty(shape, c10::TensorOptions().dtype(dtype).device(dev));
}

// n elements of a 1-D tensor from `at` on, in its storage.
at::Tensor part(const at::Tensor& of, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(), of.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// The tensors' device as the current one for the call, and the stream to launch on.
//
// A stream the caller names is the current one while the call allocates: memory
// belongs to the stream it was allocated on, so a workspace of the caller's current
// stream could still be in use there when the kernels begin, and would be handed out
// again when the call returns, under the kernels still running. What is returned is
// recorded on the caller's stream too (result), where it may be read and let go.
struct Launch {
  c10::cuda::OptionalCUDAGuard guard;
  c10::cuda::OptionalCUDAStreamGuard on;
  std::optional<c10::cuda::CUDAStream> callers;  // where the launch stream is another one
  void* stream = nullptr;
  Launch(const c10::Device& dev, PyObject* s) {
    if (dev.is_cuda()) guard.set_device(dev);
    uintptr_t handle = 0;
    if (given(s)) {
      handle = static_cast<uintptr_t>(PyLong_AsUnsignedLongLongMask(s));
      stream = reinterpret_cast<void*>(handle);
    }
    if (!dev.is_cuda()) return;
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(dev.index());
    if (!given(s)) {
      stream = now.stream();
      return;
    }
    if (handle == 1) handle = 0;  // cudaStreamLegacy: the default stream
    if (reinterpret_cast<cudaStream_t>(handle) == now.stream()) return;
    callers = now;
    on.reset_stream(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(handle), dev.index()));
  }
  void result(const at::Tensor& t) const {
    if (callers && t.defined()) t.record_stream(*callers);
  }
};

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) throw std::runtime_error("wrong number of arguments");
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (!type) PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// slots(block_table, context_lens, new_lens, total, page_size, free_pages, free_head, free_head_out, stream)
// -> (cu_seqlens, kv_lens, positions, slots[, free_head_out]), or the library's status
PyObject* slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& ctx = ints(a[1], "context_lens", -1, nullptr);
    const int64_t B = ctx.size(0);
    if (B < 1) refuse("context_lens", "of at least one request", a[1]);
    const c10::Device dev = ctx.device();
    const at::Tensor& nw = ints(a[2], "new_lens", B, &dev);
    const Table table = table_of(a[0], B, dev);
    const int total = int32(integer(a[3], "total"), "total"), ps = int32(integer(a[4], "page_size"), "page_size");
    if (total < 0 || ps < 1) throw Refused("total must not be negative and page_size at least 1");
    const int *free = nullptr, *head = nullptr;
    int count = 0;
    at::Tensor head_out;
    if (given(a[5])) {
      const at::Tensor& pages = ints(a[5], "free_pages", -1, &dev);
      head = static_cast<const int*>(ints(a[6], "free_head", 1, &dev).data_ptr());
      count = int32(pages.size(0), "free_pages' size");
      free = count ? static_cast<const int*>(pages.data_ptr()) : head;  // an empty list: an address, never read
      if (given(a[7])) head_out = ints(a[7], "free_head_out", 1, &dev);
    } else if (given(a[6]) || given(a[7])) {
      throw Refused("free_head goes with free_pages");
    }
    Launch l(dev, a[8]);
    // one allocation: cu_seqlens, kv_lens, positions, slots, head
    const at::Tensor all = empty({2 * B + 2 + 2 * static_cast<int64_t>(total)}, at::kInt, dev);
    at::Tensor cu = part(all, 0, B + 1), kv = part(all, B + 1, B);
    at::Tensor pos = part(all, 2 * B + 1, total), slot = part(all, 2 * B + 1 + total, total);
    if (free && !head_out.defined()) head_out = part(all, 2 * B + 1 + 2 * static_cast<int64_t>(total), 1);
    l.result(all);
    const int rc = fn_slots(table.ptr, table.row, table.width, static_cast<const int*>(ctx.data_ptr()),
                            static_cast<const int*>(nw.data_ptr()), int32(B, "batch"), total, ps, free, count, head,
                            free ? static_cast<int*>(head_out.data_ptr()) : nullptr, static_cast<int*>(cu.data_ptr()),
                            static_cast<int*>(kv.data_ptr()), static_cast<int*>(pos.data_ptr()),
                            static_cast<int*>(slot.data_ptr()), l.stream);
    if (rc != 0) return PyLong_FromLong(rc);
    PyObject* out = PyTuple_New(free ? 5 : 4);
    if (!out) return nullptr;
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(std::move(cu)));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(std::move(kv)));
    PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(std::move(pos)));
    PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(std::move(slot)));
    if (free) PyTuple_SET_ITEM(out, 4, THPVariable_Wrap(std::move(head_out)));
    return out;
  });
}

// append(k, v, k_cache, v_cache, slots, k_scale, v_scale, stream) -> the library's status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Cache c = cache_of(a[2], a[3], a[5], a[6]);
    const Rows k = rows_of(a[0], "k", c.c.d_qk, c.dev), v = rows_of(a[1], "v", c.c.d_v, c.dev);
    if (k.heads != c.c.Hkv || v.heads != c.c.Hkv || v.n != k.n)
      throw Refused("k and v must have the cache's " + std::to_string(c.c.Hkv) + " heads and the same number of tokens");
    const at::Tensor& slot = ints(a[4], "slots", k.n, &c.dev);
    Launch l(c.dev, a[7]);
    return PyLong_FromLong(fn_append(k.t->data_ptr(), v.t->data_ptr(), k.stride, v.stride, int32(k.n, "tokens"), &c.c,
                                     static_cast<const int*>(slot.data_ptr()), l.stream));
  });
}

// fwd(q, k_cache, v_cache, block_table, cu_seqlens, kv_lens, max_seqlen_q, causal, softmax_scale, k_scale, v_scale, out,
//     return_lse, workspace, stream) -> out, or (out, lse), or the library's status
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Cache c = cache_of(a[1], a[2], a[9], a[10]);
    const c10::Device& dev = c.dev;
    const Rows q = rows_of(a[0], "q", c.c.d_qk, dev);
    if (q.heads % c.c.Hkv != 0) throw Refused("the query heads must be a multiple of the cache's heads");
    const at::Tensor& kv = ints(a[5], "kv_lens", -1, &dev);
    const int64_t B = kv.size(0);
    if (B < 1) refuse("kv_lens", "of at least one request", a[5]);
    const at::Tensor& cu = ints(a[4], "cu_seqlens", B + 1, &dev);
    const Table table = table_of(a[3], B, dev);
    const int total = int32(q.n, "tokens"), Hq = int32(q.heads, "heads");
    int64_t max_q = given(a[6]) ? integer(a[6], "max_seqlen_q") : total;
    if (max_q < 1 && total > 0) throw Refused("max_seqlen_q must be at least 1");
    if (max_q > total) max_q = total;
    const int causal = PyObject_IsTrue(a[7]), want_lse = PyObject_IsTrue(a[12]);
    if (causal < 0 || want_lse < 0) return nullptr;
    double scale = 0.0;
    if (given(a[8])) {
      scale = PyFloat_AsDouble(a[8]);
      if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    Launch l(dev, a[14]);
    at::Tensor out, lse, ws;
    if (given(a[11])) {
      const at::Tensor* t = tensor(a[11]);
      if (!t || t->scalar_type() != at::kBFloat16 || t->device() != dev || !t->is_contiguous() || t->dim() != 3 ||
          t->size(0) != total || t->size(1) != Hq || t->size(2) != c.c.d_v)
        refuse("out", "contiguous bf16 [" + std::to_string(total) + ", " + std::to_string(Hq) + ", " +
                          std::to_string(c.c.d_v) + "] on " + dev.str(), a[11]);
      out = *t;
    } else {
      out = empty({total, Hq, c.c.d_v}, at::kBFloat16, dev);
      l.result(out);
    }
    if (want_lse) lse = empty({Hq, total}, at::kFloat, dev);
    l.result(lse);
    if (given(a[13])) {
      const at::Tensor* t = tensor(a[13]);
      if (!t || t->device() != dev || !t->is_contiguous()) refuse("workspace", "contiguous on " + dev.str(), a[13]);
      ws = *t;
    }
    if (total > 0) {
      if (!ws.defined())
        ws = empty({static_cast<int64_t>(fn_ws(total, static_cast<int>(max_q), Hq, c.c.Hkv))}, at::kByte, dev);
      const int rc = fn_fwd(q.t->data_ptr(), q.stride, &c.c, table.ptr, table.row, table.width,
                            static_cast<const int*>(cu.data_ptr()), static_cast<const int*>(kv.data_ptr()),
                            int32(B, "batch"), total, static_cast<int>(max_q), Hq, causal, static_cast<float>(scale),
                            out.data_ptr(), want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws.data_ptr(),
                            ws.nbytes(), l.stream);
      if (rc != 0) return PyLong_FromLong(rc);
    }
    PyObject* o = given(a[11]) ? Py_NewRef(a[11]) : THPVariable_Wrap(std::move(out));
    if (!want_lse || !o) return o;
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, o);
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(std::move(lse)));
    return both;
  });
}

// bind(slots, append, fwd, workspace_bytes, any_device): addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    auto address = [&](int i) { return static_cast<uintptr_t>(integer(a[i], "an address")); };
    fn_slots = reinterpret_cast<decltype(fn_slots)>(address(0));
    fn_append = reinterpret_cast<decltype(fn_append)>(address(1));
    fn_fwd = reinterpret_cast<decltype(fn_fwd)>(address(2));
    fn_ws = reinterpret_cast<decltype(fn_ws)>(address(3));
    any_device = PyObject_IsTrue(a[4]) == 1;
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<slots>("slots"), method<append>("append"), method<fwd>("fwd"), method<bind>("bind"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
