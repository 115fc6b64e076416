// The compiled half of the Python binding for the calls of a verify step that
// a decoder makes back to back (append_kv, append_mla, verify_attn_scaled,
// verify_attn_mla_scaled): reads torch tensors into va_tensor descriptors and
// calls the C ABI. Marshalling fifteen tensors through ctypes takes 20 us on a
// Grace core, several times what the kernels of a small step take; here it
// takes well under one.
//
// Every function takes positional arguments (tensors or None, numbers), checks
// types, ranks and devices as the ctypes half does, and returns the va_status.
// C++ exceptions become Python errors; the GIL is released around the call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "verify_attn.h"

namespace {

// The descriptors of one call, and the device they share.
struct Args {
  static constexpr int kMax = 16;
  va_tensor d[kMax];
  int n = 0;
  bool any = false;
  c10::Device device{c10::kCPU};

  // Reads `o` (a tensor or None) into *out; false with a Python error set.
  bool add(PyObject* o, va_tensor** out) {
    *out = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "expected a tensor or None, not %s", Py_TYPE(o)->tp_name);
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    int32_t code;
    switch (t.scalar_type()) {
      case at::kBFloat16: code = VA_BF16; break;
      case at::kFloat8_e4m3fn: code = VA_FP8_E4M3; break;
      case at::kInt: code = VA_INT32; break;
      case at::kFloat: code = VA_FP32; break;
      default:
        PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
        return false;
    }
    if (t.dim() > 4) {
      PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
      return false;
    }
    if (any && t.device() != device) {
      PyErr_Format(PyExc_ValueError, "tensors on different devices: %s and %s", device.str().c_str(),
                   t.device().str().c_str());
      return false;
    }
    any = true;
    device = t.device();
    if (n == kMax) {
      PyErr_SetString(PyExc_ValueError, "too many tensors");
      return false;
    }
    va_tensor& v = d[n++];
    v.data = t.numel() > 0 && !device.is_meta() ? t.data_ptr() : nullptr;
    v.dtype = code;
    v.ndim = (int32_t)t.dim();
    for (int i = 0; i < v.ndim; ++i) {
      v.shape[i] = t.size(i);
      v.stride[i] = t.stride(i);
    }
    *out = &v;
    return true;
  }

  // The call runs on a GPU.
  bool on_cuda(const char* where) const {
    if (any && device.is_cuda()) return true;
    PyErr_Format(PyExc_ValueError, "%s: tensors must be on a CUDA device, not %s", where, device.str().c_str());
    return false;
  }
};

// A stream argument: a handle, or None for the current stream of the device.
bool read_stream(PyObject* o, c10::Device device, cudaStream_t* out) {
  if (o == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    return true;
  }
  *out = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
  return !PyErr_Occurred();
}

bool read_int(PyObject* o, int32_t* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "a 32-bit integer is expected");
    return false;
  }
  *out = (int32_t)v;
  return true;
}

bool read_float(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return false;
  *out = (float)v;
  return true;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
  return false;
}

// Runs `fn` (which returns a PyObject*) with C++ exceptions turned into Python's.
template <class F>
PyObject* guarded(F fn) {
  try {
    return fn();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// The C call with its device current and the GIL released.
template <class F>
PyObject* status_of(c10::Device device, F call) {
  va_status s;
  {
    c10::cuda::CUDAGuard guard(device);
    Py_BEGIN_ALLOW_THREADS;
    s = call();
    Py_END_ALLOW_THREADS;
  }
  return PyLong_FromLong(s);
}

bool read_rope(Args& args, PyObject* cos_sin, PyObject* positions, PyObject* interleaved, va_rope* rope,
               const va_rope** out) {
  va_tensor *cs, *pos;
  if (!args.add(cos_sin, &cs) || !args.add(positions, &pos) || !read_int(interleaved, &rope->interleaved)) return false;
  if (!cs && pos) {
    PyErr_SetString(PyExc_ValueError, "positions without cos_sin");
    return false;
  }
  rope->cos_sin = cs;
  rope->positions = pos;
  *out = cs ? rope : nullptr;
  return true;
}

// append_kv(q, k, v, block_table, cu_seqlens_q, seqused_k, k_descale, v_descale,
//           k_scales, v_scales, q_out, k_cache, v_cache, cos_sin, positions, interleaved, stream)
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 17)) return nullptr;
    Args args;
    va_tensor* t[13];
    for (int i = 0; i < 13; ++i)
      if (!args.add(a[i], &t[i])) return nullptr;
    va_rope rope;
    const va_rope* r;
    cudaStream_t stream;
    if (!read_rope(args, a[13], a[14], a[15], &rope, &r) || !args.on_cuda("append_kv") ||
        !read_stream(a[16], args.device, &stream))
      return nullptr;
    return status_of(args.device, [&] {
      return verify_attn_append_kv(t[0], t[1], t[2], t[3], t[4], t[5], r, t[6], t[7], t[8], t[9], t[10], t[11], t[12],
                                   stream);
    });
  });
}

// append_mla(q_pe, latent, k_pe, block_table, cu_seqlens_q, seqused_k, descale,
//            scales, q_pe_out, kv_cache, cos_sin, positions, interleaved, stream)
PyObject* append_mla(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 14)) return nullptr;
    Args args;
    va_tensor* t[10];
    for (int i = 0; i < 10; ++i)
      if (!args.add(a[i], &t[i])) return nullptr;
    va_rope rope;
    const va_rope* r;
    cudaStream_t stream;
    if (!read_rope(args, a[10], a[11], a[12], &rope, &r) || !args.on_cuda("append_mla") ||
        !read_stream(a[13], args.device, &stream))
      return nullptr;
    return status_of(args.device, [&] {
      return verify_attn_append_mla(t[0], t[1], t[2], t[3], t[4], t[5], r, t[6], t[7], t[8], t[9], stream);
    });
  });
}

// A workspace for one call, from torch's allocator on the call's stream: calls
// on other streams, and calls captured into other graphs, get others.
class CallWorkspace {
 public:
  CallWorkspace(size_t bytes, cudaStream_t stream) {
    // (the allocator's blocks are 512-byte aligned)
    p_ = bytes > 0 ? c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, stream) : nullptr;
  }
  ~CallWorkspace() {
    if (p_) c10::cuda::CUDACachingAllocator::raw_delete(p_);
  }
  CallWorkspace(const CallWorkspace&) = delete;
  CallWorkspace& operator=(const CallWorkspace&) = delete;
  void* get() const { return p_; }

 private:
  void* p_ = nullptr;
};

// The attention calls' tail: workspace (a tensor or None), num_splits, event, stream.
// Without a workspace the call's own is given back behind it, so its waits report
// to the library's status word.
struct Tail {
  void* ws = nullptr;
  size_t bytes = 0;
  int32_t splits = 0;
  void* event = nullptr;
  cudaStream_t stream = nullptr;

  int32_t splits_arg() const { return ws || splits < 0 ? splits : splits | VA_LIBRARY_STATUS; }

  bool read(PyObject* workspace, PyObject* num_splits, PyObject* ev, PyObject* st, c10::Device device) {
    if (!read_int(num_splits, &splits) || !read_stream(st, device, &stream)) return false;
    event = PyLong_AsVoidPtr(ev);
    if (PyErr_Occurred()) return false;
    if (workspace == Py_None) return true;
    if (!THPVariable_Check(workspace)) {
      PyErr_SetString(PyExc_TypeError, "workspace: a tensor or None");
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(workspace);
    if (t.device() != device || !t.is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "workspace: a contiguous tensor on the call's device");
      return false;
    }
    char* p = static_cast<char*>(t.numel() > 0 ? t.data_ptr() : nullptr);
    const size_t off = (256 - reinterpret_cast<uintptr_t>(p) % 256) % 256;
    bytes = t.numel() * t.element_size();
    bytes = bytes > off ? bytes - off : 0;
    ws = p ? p + off : nullptr;
    if (!ws) {  // an empty workspace is too small, not absent
      PyErr_SetString(PyExc_ValueError, "workspace: empty");
      return false;
    }
    return true;
  }
};

// verify_attn_scaled(q, k_cache, v_cache, k_scales, v_scales, block_table, cu_seqlens_q, seqused_k, out, sinks,
//                    max_seqlen_q, max_seqlen_k, softmax_scale, window_left, softcap, workspace, num_splits, event, stream)
PyObject* attn_scaled(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 19)) return nullptr;
    Args args;
    va_tensor* t[10];
    for (int i = 0; i < 10; ++i)
      if (!args.add(a[i], &t[i])) return nullptr;
    int32_t max_q, max_k;
    float scale;
    va_options opt;
    Tail tail;
    if (!read_int(a[10], &max_q) || !read_int(a[11], &max_k) || !read_float(a[12], &scale) ||
        !read_int(a[13], &opt.window_left) || !read_float(a[14], &opt.softcap) ||
        !args.on_cuda("verify_attn_scaled") || !tail.read(a[15], a[16], a[17], a[18], args.device))
      return nullptr;
    opt.sinks = t[9];
    c10::cuda::CUDAGuard guard(args.device);
    size_t need = 0;  // 0: the arguments have no plan, and the call says why
    if (!tail.ws && t[0] && t[1] && t[7] && t[0]->ndim == 3 && t[1]->ndim == 4 && t[7]->ndim == 1 &&
        t[7]->shape[0] <= INT32_MAX && t[1]->shape[2] <= INT32_MAX && t[0]->shape[1] <= INT32_MAX)
      need = verify_attn_workspace_size((int32_t)t[7]->shape[0], (int32_t)t[1]->shape[2], (int32_t)t[0]->shape[1],
                                        max_q, max_k, VA_FP8_E4M3, tail.splits);
    const CallWorkspace own(need, tail.stream);
    void* ws = tail.ws ? tail.ws : own.get();
    return status_of(args.device, [&] {
      return verify_attn_scaled(t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], max_q, max_k, scale, t[8], &opt, ws,
                                tail.ws ? tail.bytes : need, tail.splits_arg(), tail.event, tail.stream);
    });
  });
}

// verify_attn_mla_scaled(q, kv_cache, scales, block_table, cu_seqlens_q, seqused_k, out,
//                        max_seqlen_q, max_seqlen_k, softmax_scale, workspace, num_splits, event, stream)
PyObject* attn_mla_scaled(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (!arity(n, 14)) return nullptr;
    Args args;
    va_tensor* t[7];
    for (int i = 0; i < 7; ++i)
      if (!args.add(a[i], &t[i])) return nullptr;
    int32_t max_q, max_k;
    float scale;
    Tail tail;
    if (!read_int(a[7], &max_q) || !read_int(a[8], &max_k) || !read_float(a[9], &scale) ||
        !args.on_cuda("verify_attn_mla_scaled") || !tail.read(a[10], a[11], a[12], a[13], args.device))
      return nullptr;
    c10::cuda::CUDAGuard guard(args.device);
    size_t need = 0;
    if (!tail.ws && t[0] && t[5] && t[0]->ndim == 3 && t[5]->ndim == 1 && t[5]->shape[0] <= INT32_MAX &&
        t[0]->shape[1] <= INT32_MAX)
      need = verify_attn_mla_workspace_size((int32_t)t[5]->shape[0], (int32_t)t[0]->shape[1], max_q, max_k, tail.splits);
    const CallWorkspace own(need, tail.stream);
    void* ws = tail.ws ? tail.ws : own.get();
    return status_of(args.device, [&] {
      return verify_attn_mla_scaled(t[0], t[1], t[2], t[3], t[4], t[5], max_q, max_k, scale, t[6], ws,
                                    tail.ws ? tail.bytes : need, tail.splits_arg(), tail.event, tail.stream);
    });
  });
}

PyMethodDef kMethods[] = {
    {"append_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_kv)), METH_FASTCALL, nullptr},
    {"append_mla", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_mla)), METH_FASTCALL, nullptr},
    {"attn_scaled", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn_scaled)), METH_FASTCALL, nullptr},
    {"attn_mla_scaled", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn_mla_scaled)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "va_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_va_binding() { return PyModule_Create(&kModule); }
