// The quick way into the long-context calls from Python: one C call checks the
// tensors, allocates the outputs and calls libpagedattn, in 2-3 us besides the
// launches, where the same steps in Python take 8-15 us -- more than the
// kernels of a small step.
//
// Every function takes the common form of its call (default outputs,
// workspace and stream) and returns its result, or None when anything is not
// as it must be or not as it is handled here.  The caller (_binding.py) then
// takes its own way, which makes every check again, by name, and handles the
// rest: nothing is launched before a None.  Once the library's call has been made
// it is not made again: its failure is raised, and the results are Python objects
// before it.
#include <Python.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "pagedattn.h"

namespace {

struct Library {
  decltype(&pa_block_key_bounds) bounds;
  decltype(&pa_select_blocks_workspace_bytes) select_bytes;
  decltype(&pa_select_blocks) select;
  decltype(&pa_decode_sparse_workspace_bytes) sparse_bytes;
  decltype(&pa_paged_attention_decode_sparse) sparse;
  decltype(&pa_decode_weights_workspace_bytes) weights_bytes;
  decltype(&pa_paged_attention_decode_weights) weights;
  decltype(&pa_evict_tokens) evict;
} lib;

struct No {};  // not for the quick way

// An argument that must be a contiguous CUDA tensor of `type` with `nd`
// dimensions on the current device.
struct Dev {
  int index;
  const at::Tensor &operator()(PyObject *o, at::ScalarType type, int nd) const {
    if (!THPVariable_CheckExact(o)) throw No{};
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != type || t.dim() != nd || !t.is_contiguous() ||
        t.requires_grad())
      throw No{};
    for (int i = 0; i < nd; ++i)
      if (t.size(i) > INT_MAX) throw No{};
    return t;
  }
  // the device error word, or null for None
  int32_t *err(PyObject *o) const {
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) throw No{};
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != index || t.scalar_type() != at::kInt || !t.is_contiguous() || t.numel() < 1)
      throw No{};
    return static_cast<int32_t *>(t.data_ptr());
  }
};

int integer(PyObject *o) {
  if (!PyLong_CheckExact(o)) throw No{};
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over || v > INT_MAX || v < INT_MIN) throw No{};
  return (int)v;
}
int integer_or(PyObject *o, int64_t otherwise) {
  if (o != Py_None) return integer(o);
  if (otherwise > INT_MAX) throw No{};
  return (int)otherwise;
}
int size(const at::Tensor &t, int i) { return (int)t.size(i); }
void need(bool ok) {
  if (!ok) throw No{};
}

struct Workspace {
  void *p = nullptr;
  size_t bytes = 0;
};

// The workspace that _binding.py keeps for (device, stream), if it is there
// and large enough; a captured call never takes it.
Workspace workspace(PyObject *cache, size_t bytes, int device, cudaStream_t stream) {
  if (bytes == 0) return {};
  if (stream && c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) throw No{};
  PyObject *key = Py_BuildValue("(iK)", device, (unsigned long long)(uintptr_t)stream);
  if (!key) throw No{};
  PyObject *o = PyDict_GetItemWithError(cache, key);  // borrowed
  Py_DECREF(key);
  if (!o || !THPVariable_Check(o)) throw No{};
  const at::Tensor &t = THPVariable_Unpack(o);
  const size_t have = (size_t)t.numel() * t.element_size();
  if (have < bytes) throw No{};
  return {t.data_ptr(), have};
}

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, int device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (at::DeviceIndex)device)));
}

// A reference of its own.
struct Ref {
  PyObject *p;
  explicit Ref(PyObject *o) : p(o) {
    if (!p) throw No{};
  }
  Ref(const Ref &) = delete;
  ~Ref() { Py_XDECREF(p); }
  // The result of a call that returned `status`, or its failure raised as the
  // binding raises it.
  PyObject *after(int status, const char *call) {
    PyObject *r = p;
    if (status == PA_OK) {
      p = nullptr;
      return r;
    }
    PyObject *m = PyImport_ImportModule("paged_kv_cache_262_gb300._binding");
    PyObject *x = m ? PyObject_CallMethod(m, "_check", "is", status, call) : nullptr;
    Py_XDECREF(m);
    if (x) {  // (it raises)
      Py_DECREF(x);
      PyErr_SetString(PyExc_RuntimeError, call);
    }
    return nullptr;
  }
};

template <class F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n == want) return f();
  } catch (const No &) {
  } catch (...) {  // an allocation or a driver call that failed: the other way reports it
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

constexpr at::ScalarType kBf = at::kBFloat16, kI = at::kInt, kF = at::kFloat;

// k_pool, bounds, block_tables, context_lens, start_lens, max_new_tokens, max_context_len, err_flag, -> True
PyObject *bounds(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    const Dev dev{c10::cuda::current_device()};
    const at::Tensor &k = dev(a[0], kBf, 4), &b = dev(a[1], kBf, 4), &bt = dev(a[2], kI, 2), &ctx = dev(a[3], kI, 1);
    const int S = size(ctx, 0), B = size(k, 2);
    need(size(b, 0) == size(k, 0) && size(b, 1) == size(k, 1) && size(b, 2) == 2 && size(b, 3) == size(k, 3) &&
         size(bt, 0) >= S);
    const int32_t *start = nullptr;
    if (a[4] != Py_None) {
      const at::Tensor &t = dev(a[4], kI, 1);
      need(size(t, 0) >= S);
      start = static_cast<const int32_t *>(t.data_ptr());
    }
    const int most = integer_or(a[6], (int64_t)size(bt, 1) * B), max_new = integer_or(a[5], most);
    const pa_decode_desc d{S, size(k, 1), size(k, 1), size(k, 3), B, size(k, 0), size(bt, 1), most, 1.f};
    int32_t *err = dev.err(a[7]);
    cudaStream_t st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    Py_INCREF(Py_True);
    Ref r(Py_True);
    return r.after(lib.bounds(&d, k.data_ptr(), static_cast<const int32_t *>(bt.data_ptr()),
                              static_cast<const int32_t *>(ctx.data_ptr()), start, max_new, b.data_ptr(), err, st),
                   "pa_block_key_bounds");
  });
}

// q, bounds, block_tables, context_lens, num_select, block_size, sink_blocks, recent_blocks, max_context_len,
// err_flag, workspaces -> selected
PyObject *select(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const Dev dev{c10::cuda::current_device()};
    const at::Tensor &q = dev(a[0], kBf, 3), &b = dev(a[1], kBf, 4), &bt = dev(a[2], kI, 2), &ctx = dev(a[3], kI, 1);
    const int S = size(q, 0), Hkv = size(b, 1), k = integer(a[4]), B = integer(a[5]);
    need(size(b, 2) == 2 && size(q, 2) == size(b, 3) && size(bt, 0) >= S && size(ctx, 0) >= S && k > 0);
    const pa_decode_desc d{S,          size(q, 1), Hkv, size(b, 3), B, size(b, 0), size(bt, 1),
                           integer_or(a[8], (int64_t)size(bt, 1) * B), 1.f};
    cudaStream_t st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    int32_t *err = dev.err(a[9]);
    const Workspace ws = workspace(a[10], lib.select_bytes(&d), dev.index, st);
    const int sink = integer(a[6]), recent = integer(a[7]);
    at::Tensor out = fresh({S, Hkv, k}, kI, dev.index);
    Ref r(THPVariable_Wrap(out));
    return r.after(lib.select(&d, q.data_ptr(), b.data_ptr(), static_cast<const int32_t *>(bt.data_ptr()),
                              static_cast<const int32_t *>(ctx.data_ptr()), k, sink, recent,
                              static_cast<int32_t *>(out.data_ptr()), ws.p, ws.bytes, err, st),
                   "pa_select_blocks");
  });
}

struct Decode {
  const at::Tensor &q, &k, &v, &bt, &ctx;
  pa_decode_desc d;
};

// q, k_pool, v_pool, block_tables, context_lens at a[0..4]
Decode decode(const Dev &dev, PyObject *const *a, PyObject *scale, PyObject *max_ctx) {
  const at::Tensor &q = dev(a[0], kBf, 3), &k = dev(a[1], kBf, 4), &v = dev(a[2], kBf, 4), &bt = dev(a[3], kI, 2),
                   &ctx = dev(a[4], kI, 1);
  const int S = size(q, 0), B = size(k, 2), D = size(k, 3);
  need(v.sizes() == k.sizes() && size(q, 2) == D && size(bt, 0) >= S && size(ctx, 0) >= S && D > 0);
  double sc;
  if (scale == Py_None) {
    sc = 1.0 / std::sqrt((double)D);
  } else {
    need(PyFloat_CheckExact(scale));
    sc = PyFloat_AS_DOUBLE(scale);
  }
  return Decode{q, k, v, bt, ctx, pa_decode_desc{S, size(q, 1), size(k, 1), D, B, size(k, 0), size(bt, 1),
                                                 integer_or(max_ctx, (int64_t)size(bt, 1) * B), (float)sc}};
}

// q, k_pool, v_pool, block_tables, context_lens, selected, scale, max_context_len, err_flag, workspaces -> out
PyObject *sparse(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const Dev dev{c10::cuda::current_device()};
    const Decode x = decode(dev, a, a[6], a[7]);
    const at::Tensor &sel = dev(a[5], kI, 3);
    const int k = size(sel, 2);
    need(size(sel, 0) >= x.d.num_seqs && size(sel, 1) == x.d.num_kv_heads);
    cudaStream_t st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    int32_t *err = dev.err(a[8]);
    const Workspace ws = workspace(a[9], lib.sparse_bytes(&x.d, k), dev.index, st);
    at::Tensor out = fresh(x.q.sizes(), kBf, dev.index);
    Ref r(THPVariable_Wrap(out));
    return r.after(lib.sparse(&x.d, x.q.data_ptr(), x.k.data_ptr(), x.v.data_ptr(),
                              static_cast<const int32_t *>(x.bt.data_ptr()),
                              static_cast<const int32_t *>(x.ctx.data_ptr()),
                              static_cast<const int32_t *>(sel.data_ptr()), k, out.data_ptr(), ws.p, ws.bytes, err, st),
                   "pa_paged_attention_decode_sparse");
  });
}

struct Weights {
  const at::Tensor &in, &out;
  const int32_t *rows;
};

// weights, weights_out or None, weight_rows or None
Weights weight_rows(const Dev &dev, PyObject *w, PyObject *wo, PyObject *rows, const pa_decode_desc &d) {
  const at::Tensor &in = dev(w, kF, 3), &out = wo == Py_None ? in : dev(wo, kF, 3);
  need(out.sizes() == in.sizes() && size(in, 1) == d.num_kv_heads && size(in, 2) >= d.max_context_len);
  const char *p = static_cast<const char *>(in.data_ptr()), *q = static_cast<const char *>(out.data_ptr());
  const size_t bytes = (size_t)in.numel() * 4;
  need(p == q || p >= q + bytes || q >= p + bytes);
  if (rows == Py_None) {
    need(size(in, 0) >= d.num_seqs);
    return {in, out, nullptr};
  }
  const at::Tensor &r = dev(rows, kI, 1);
  need(size(r, 0) >= d.num_seqs);
  return {in, out, static_cast<const int32_t *>(r.data_ptr())};
}

// q, k_pool, v_pool, block_tables, context_lens, weights, weights_out, weight_rows, scale, max_context_len, err_flag,
// workspaces -> out
PyObject *weights(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject * {
    const Dev dev{c10::cuda::current_device()};
    const Decode x = decode(dev, a, a[8], a[9]);
    const Weights w = weight_rows(dev, a[5], a[6], a[7], x.d);
    cudaStream_t st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    int32_t *err = dev.err(a[10]);
    const Workspace ws = workspace(a[11], lib.weights_bytes(&x.d), dev.index, st);
    at::Tensor out = fresh(x.q.sizes(), kBf, dev.index);
    Ref r(THPVariable_Wrap(out));
    return r.after(lib.weights(&x.d, x.q.data_ptr(), x.k.data_ptr(), x.v.data_ptr(),
                               static_cast<const int32_t *>(x.bt.data_ptr()),
                               static_cast<const int32_t *>(x.ctx.data_ptr()),
                               static_cast<const float *>(w.in.data_ptr()), static_cast<float *>(w.out.data_ptr()),
                               w.rows, size(w.in, 0), size(w.in, 2), out.data_ptr(), ws.p, ws.bytes, err, st),
                   "pa_paged_attention_decode_weights");
  });
}

// k_pool, v_pool, block_tables, context_lens, keep_lens, weights, max_keep_len, sink_tokens, recent_tokens,
// dst_tables, weights_out, weight_rows, max_context_len, err_flag -> (kept, new_lens)
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject * {
    const Dev dev{c10::cuda::current_device()};
    const at::Tensor &k = dev(a[0], kBf, 4), &v = dev(a[1], kBf, 4), &bt = dev(a[2], kI, 2), &ctx = dev(a[3], kI, 1),
                     &keep = dev(a[4], kI, 1);
    const int S = size(ctx, 0), Hkv = size(k, 1), B = size(k, 2), mk = integer(a[6]);
    need(v.sizes() == k.sizes() && mk > 0 && size(bt, 0) >= S && size(keep, 0) >= S);
    const int32_t *dst = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor &t = dev(a[9], kI, 2);
      need(size(t, 0) >= S && size(t, 1) == size(bt, 1));
      dst = static_cast<const int32_t *>(t.data_ptr());
    }
    const pa_decode_desc d{S, Hkv, Hkv, size(k, 3), B, size(k, 0), size(bt, 1),
                           integer_or(a[12], (int64_t)size(bt, 1) * B), 1.f};
    const Weights w = weight_rows(dev, a[5], a[10], a[11], d);
    cudaStream_t st = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
    int32_t *err = dev.err(a[13]);
    const int sink = integer(a[7]), recent = integer(a[8]);
    at::Tensor kept = fresh({S, Hkv, mk}, kI, dev.index), lens = fresh({S}, kI, dev.index);
    Ref k_(THPVariable_Wrap(kept)), l_(THPVariable_Wrap(lens)), r(PyTuple_Pack(2, k_.p, l_.p));
    return r.after(lib.evict(&d, k.data_ptr(), v.data_ptr(), static_cast<const int32_t *>(bt.data_ptr()), dst,
                             static_cast<const int32_t *>(ctx.data_ptr()),
                             static_cast<const int32_t *>(keep.data_ptr()), mk, sink, recent,
                             static_cast<const float *>(w.in.data_ptr()), static_cast<float *>(w.out.data_ptr()),
                             w.rows, size(w.in, 0), size(w.in, 2), static_cast<int32_t *>(kept.data_ptr()),
                             static_cast<int32_t *>(lens.data_ptr()), err, st),
                   "pa_evict_tokens");
  });
}

// bind(addresses of the library's calls, in the order of Library)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  void *p[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes 8 addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  lib.bounds = reinterpret_cast<decltype(lib.bounds)>(p[0]);
  lib.select_bytes = reinterpret_cast<decltype(lib.select_bytes)>(p[1]);
  lib.select = reinterpret_cast<decltype(lib.select)>(p[2]);
  lib.sparse_bytes = reinterpret_cast<decltype(lib.sparse_bytes)>(p[3]);
  lib.sparse = reinterpret_cast<decltype(lib.sparse)>(p[4]);
  lib.weights_bytes = reinterpret_cast<decltype(lib.weights_bytes)>(p[5]);
  lib.weights = reinterpret_cast<decltype(lib.weights)>(p[6]);
  lib.evict = reinterpret_cast<decltype(lib.evict)>(p[7]);
  Py_RETURN_NONE;
}

#define PA_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_FAST(bounds),  PA_FAST(select), PA_FAST(sparse), PA_FAST(weights),
                         PA_FAST(evict),   PA_FAST(bind),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_pa_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_fastcall(void) {
  PyObject *m = PyModule_Create(&module_def);
  // the torch that it was compiled against, and may be used with
  if (m && PyModule_AddStringConstant(m, "torch_version", PA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
