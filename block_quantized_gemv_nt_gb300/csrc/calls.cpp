// calls.cpp — the torch side of a step's calls over the paged 4-bit cache: checks of the
// tensors, then the C entry point.  The same in Python cost 5 us a call, more than the
// launch (3 us) and most of the kernels of a decode step.
//
// Every function returns the entry point's nt_status; a tensor that does not fit raises
// ValueError and calls nothing.  Streams: None (torch's current one of the device), an
// address, or an object with cuda_stream.  Other Python threads run while the library works:
// a launch waits where the stream's queue is full.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "../../include/nt.h"

namespace {

struct Refused {
  const char* why;
};

const at::Tensor& tensor(PyObject* o, const char* why) {
  if (!THPVariable_Check(o)) throw Refused{why};
  return THPVariable_Unpack(o);
}
int index_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
void need(bool ok, const char* why) {
  if (!ok) throw Refused{why};
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw std::exception();
  return v;
}
void* address(PyObject* o) {
  if (o == Py_None) return nullptr;
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw std::exception();
  return p;
}
void* stream_of(PyObject* o, int index) {
  if (o == Py_None) return index < 0 ? nullptr : c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(index)).stream();
  if (PyLong_Check(o)) return address(o);
  PyObject* s = PyObject_GetAttrString(o, "cuda_stream");
  if (!s) throw std::exception();
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw std::exception();
  return p;
}
template <typename P>
P* data(const at::Tensor& t) {
  return static_cast<P*>(t.data_ptr());
}

// a contiguous int32 tensor of n values on the device
int32_t* ints(PyObject* o, int64_t n, int index, const char* why) {
  const at::Tensor& t = tensor(o, why);
  need(t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n && t.is_contiguous() && index_of(t) == index, why);
  return data<int32_t>(t);
}
int32_t* ints_or_null(PyObject* o, int64_t n, int index, const char* why) {
  return o == Py_None ? nullptr : ints(o, n, index, why);
}

// rows' format: fp32 or f16
int row_fmt(const at::Tensor& t, const char* why) {
  if (t.scalar_type() == at::kFloat) return NT_F32;
  need(t.scalar_type() == at::kHalf, why);
  return NT_F16;
}

// the interpreter is let go of while one lives: for the library's call only
struct Released {
  PyThreadState* state = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(state); }
};

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.why);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

// (read, ctx, cache, n_kvh, head_dim, index, k, v, slots, stream)
PyObject* kv4_rows(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 10, [&] {
    const char* why = "k and v: rows [n][n_kvh][head_dim] on the cache's device, alike in layout";
    const int index = int(integer(a[5]));
    const at::Tensor &k = tensor(a[6], why), &v = tensor(a[7], why);
    need(k.dim() == 3 && k.size(1) == integer(a[3]) && k.size(2) == integer(a[4]) && k.stride(2) == 1 &&
             v.sizes() == k.sizes() && v.strides() == k.strides() && v.scalar_type() == k.scalar_type() &&
             index_of(k) == index && index_of(v) == index,
         why);
    const int64_t n = k.size(0);
    why = "slots: a contiguous int64 tensor on the cache's device, one for each row";
    const at::Tensor& s = tensor(a[8], why);
    need(s.scalar_type() == at::kLong && s.dim() == 1 && s.size(0) == n && s.is_contiguous() && index_of(s) == index, why);
    const int fmt = row_fmt(k, "rows must be float32 or float16");
    nt_ctx* ctx = static_cast<nt_ctx*>(address(a[1]));
    const nt_kv4* cache = static_cast<const nt_kv4*>(address(a[2]));
    void *kp = data<void>(k), *vp = data<void>(v), *stream = stream_of(a[9], index);
    const int64_t *slots = data<int64_t>(s), tok = k.stride(0), head = k.stride(1);
    const bool read = a[0] == Py_True;
    const Released others;
    if (read) return nt_kv4_read(ctx, cache, fmt, kp, vp, n, tok, head, slots, stream);
    return nt_kv4_append(ctx, cache, fmt, kp, vp, n, tok, head, slots, stream);
  });
}

// (ctx, cache, head_dim, index, q, out, q_start, held, table, stream)
PyObject* attn_kv4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 10, [&] {
    const char* why = "q: contiguous float32 [n_tok][n_qh][head_dim] on the cache's device";
    const int index = int(integer(a[3]));
    const at::Tensor& q = tensor(a[4], why);
    need(q.dim() == 3 && q.size(2) == integer(a[2]) && q.scalar_type() == at::kFloat && q.is_contiguous() &&
             index_of(q) == index,
         why);
    const at::Tensor& out = tensor(a[5], "out: like q");
    need(out.sizes() == q.sizes() && out.scalar_type() == at::kFloat && out.is_contiguous() && index_of(out) == index,
         "out: like q");
    why = "table: a contiguous int32 tensor [n_req][max_pages], all on one device";
    const at::Tensor& table = tensor(a[8], why);
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous() && index_of(table) == index, why);
    const int64_t n_req = table.size(0);
    const int32_t* q_start = ints(a[6], n_req + 1, index, "q_start: a contiguous int32 tensor of n_req + 1 on the tables' device");
    const int32_t* held = ints(a[7], n_req, index, "held: a contiguous int32 tensor of n_req on the tables' device");
    need(n_req <= 1 << 20 && q.size(1) <= 1 << 20, "more requests or heads than the library takes");
    nt_ctx* ctx = static_cast<nt_ctx*>(address(a[0]));
    const nt_kv4* cache = static_cast<const nt_kv4*>(address(a[1]));
    void* stream = stream_of(a[9], index);
    const float* from = data<float>(q);
    float* to = data<float>(out);
    const int32_t* pages = data<int32_t>(table);
    const int64_t n_tok = q.size(0), n_qh = q.size(1), width = table.size(1);
    const Released others;
    return nt_attn_kv4(ctx, from, cache, to, int(n_qh), n_tok, int(n_req), q_start, held, pages, width, stream);
  });
}

// (ctx, index, table, held, free, n_free, n_new, q_start, slots, positions, keep, held_out, n_free_out, stream)
PyObject* kv4_pages(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 14, [&] {
    const int index = int(integer(a[1]));
    const char* why = "table: a contiguous int32 tensor [n_req][max_pages], all on one device";
    const at::Tensor& table = tensor(a[2], why);
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous() && index_of(table) == index, why);
    const int64_t R = table.size(0);
    need(R <= 1 << 20, "more requests than the library takes");
    int32_t* held = ints(a[3], R, index, "held: a contiguous int32 tensor of n_req on the tables' device");
    why = "free: a contiguous int32 tensor of n_pages on the tables' device";
    const at::Tensor& free = tensor(a[4], why);
    need(free.scalar_type() == at::kInt && free.dim() == 1 && free.is_contiguous() && index_of(free) == index, why);
    int32_t* n_free = ints(a[5], 1, index, "n_free: a contiguous int32 tensor of 1 on the tables' device");
    const int32_t* n_new = ints(a[6], R, index, "n_new: a contiguous int32 tensor of n_req on the tables' device");
    int32_t* q_start = ints(a[7], R + 1, index, "q_start: a contiguous int32 tensor of n_req + 1 on the tables' device");
    why = "slots: a contiguous int64 tensor on the tables' device";
    const at::Tensor& slots = tensor(a[8], why);
    need(slots.scalar_type() == at::kLong && slots.dim() == 1 && slots.is_contiguous() && index_of(slots) == index, why);
    int32_t* positions = ints(a[9], slots.size(0), index, "positions: a contiguous int32 tensor as long as slots");
    const int32_t* keep = ints_or_null(a[10], R, index, "keep: a contiguous int32 tensor of n_req on the tables' device");
    int32_t* held_out = ints_or_null(a[11], R, index, "held_out: a contiguous int32 tensor of n_req on the tables' device");
    int32_t* n_free_out = ints_or_null(a[12], 1, index, "n_free_out: a contiguous int32 tensor of 1 on the tables' device");
    nt_ctx* ctx = static_cast<nt_ctx*>(address(a[0]));
    void* stream = stream_of(a[13], index);
    int32_t *entries = data<int32_t>(table), *stack = data<int32_t>(free);
    int64_t* to = data<int64_t>(slots);
    const int64_t width = table.size(1), n_pages = free.size(0), n_tok = slots.size(0);
    const Released others;
    return nt_kv4_pages(ctx, int(R), entries, width, held, keep, n_new, stack, n_pages, n_free, held_out ? held_out : held,
                        n_free_out ? n_free_out : n_free, q_start, to, positions, n_tok, stream);
  });
}

// (ctx, plan, head_dim, index, ((x, y), ...), positions, pos0, stream)
PyObject* rope_rows(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 8, [&] {
    const char* few = "rows: one to three pairs of float32 or float16 tensors";
    need(PyTuple_Check(a[4]) && PyTuple_GET_SIZE(a[4]) >= 1 && PyTuple_GET_SIZE(a[4]) <= 3, few);
    const int n_jobs = int(PyTuple_GET_SIZE(a[4])), index = int(integer(a[3]));
    const int64_t hd = integer(a[2]);
    const char* why = "rows: [n][n_heads][head_dim] on the context's device, alike in type, contiguous channels";
    nt_rope_job jobs[3];
    int64_t n = 0;
    int fmt = 0;
    for (int i = 0; i < n_jobs; ++i) {
      PyObject* pair = PyTuple_GET_ITEM(a[4], i);
      need(PyTuple_Check(pair) && PyTuple_GET_SIZE(pair) == 2, few);
      const at::Tensor &x = tensor(PyTuple_GET_ITEM(pair, 0), few), &y = tensor(PyTuple_GET_ITEM(pair, 1), few);
      const int f = row_fmt(x, few);
      need(x.dim() == 3 && x.size(2) == hd && y.sizes() == x.sizes() && x.stride(2) == 1 && y.stride(2) == 1 &&
               y.scalar_type() == x.scalar_type() && index_of(x) == index && index_of(y) == index && x.size(1) <= 1 << 20 &&
               (i == 0 || (f == fmt && x.size(0) == n)),
           why);
      fmt = f;
      n = x.size(0);
      jobs[i] = {data<void>(x), data<void>(y), int(x.size(1)), x.stride(0), x.stride(1), y.stride(0), y.stride(1)};
    }
    const int32_t* positions = ints_or_null(a[5], n, index, "positions: a contiguous int32 tensor, one for each row");
    nt_ctx* ctx = static_cast<nt_ctx*>(address(a[0]));
    const nt_rope_plan* plan = static_cast<const nt_rope_plan*>(address(a[1]));
    const int64_t pos0 = integer(a[6]);
    void* stream = stream_of(a[7], index);
    const Released others;
    return nt_rope_rows(ctx, plan, fmt, jobs, n_jobs, n, positions, pos0, stream);
  });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"kv4_rows", fast(kv4_rows), METH_FASTCALL, nullptr},
                         {"attn_kv4", fast(attn_kv4), METH_FASTCALL, nullptr},
                         {"kv4_pages", fast(kv4_pages), METH_FASTCALL, nullptr},
                         {"rope_rows", fast(rope_rows), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "nt_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_nt_calls() { return PyModule_Create(&module); }
