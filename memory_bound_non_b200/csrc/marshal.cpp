// Argument marshalling of the NVFP4 operators for the Python binding: tensors
// are checked (type, shape, device, contiguity) and handed to the C entry point
// whose address the caller passes.  A call with a dozen tensors costs about a
// microsecond here, against ten when each check is a Python expression, which
// is more than the kernels of a decoding step take.
#include <Python.h>

#include <algorithm>
#include <climits>
#include <initializer_list>
#include <string>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "frt.h"

namespace {

PyObject* g_error = nullptr;  // FrtError(fn, status, message)

struct Error {
  int status;
  std::string message;
};
struct PythonError {};  // a Python exception is set

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

using Shape = std::initializer_list<int64_t>;

// One call: its device is that of the first tensor.
struct Call {
  const char* fn;
  int device = -1;

  [[noreturn]] void invalid(const std::string& message) const { throw Error{FRT_ERR_INVALID_ARG, message}; }

  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) invalid(std::string(name) + " is not a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) invalid(std::string(name) + ": tensor is not on a CUDA device");
    if (!t.is_contiguous()) invalid(std::string(name) + ": tensor is not contiguous");
    if (device < 0) device = t.get_device();
    if (t.get_device() != device)
      invalid(std::string(name) + " is on device " + std::to_string(t.get_device()) + ", expected " +
              std::to_string(device));
    return t;
  }
  template <typename T = void>
  T* pointer(PyObject* o, const char* name, at::ScalarType type, Shape shape) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
      invalid(std::string(name) + " is " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type));
    if (t.sizes() != at::IntArrayRef(shape))
      invalid(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(at::IntArrayRef(shape)));
    return static_cast<T*>(t.data_ptr());
  }
  // None is NULL
  template <typename T = void>
  T* optional(PyObject* o, const char* name, at::ScalarType type, Shape shape) {
    return o == Py_None ? nullptr : pointer<T>(o, name, type, shape);
  }
  // a status word: int32, any shape
  int32_t* status(PyObject* o) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "status");
    if (t.scalar_type() != at::kInt || t.numel() < 1) invalid("status is not an int32 tensor");
    return static_cast<int32_t*>(t.data_ptr());
  }
  uint8_t* bytes(PyObject* o, const char* name, int64_t n) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kByte || t.numel() != n)
      invalid(std::string(name) + " holds " + std::to_string(t.numel()) + " elements of " +
              c10::toString(t.scalar_type()) + ", expected " + std::to_string(n) + " bytes");
    return static_cast<uint8_t*>(t.data_ptr());
  }
  frt_dtype dtype(const at::Tensor& t) const {
    if (t.scalar_type() == at::kHalf) return FRT_F16;
    if (t.scalar_type() == at::kBFloat16) return FRT_BF16;
    invalid(std::string(c10::toString(t.scalar_type())) + " is not a supported 16-bit type");
  }
  void dims(const at::Tensor& t, const char* name, int64_t n) const {
    if (t.dim() != n) invalid(std::string(name) + " has shape " + text(t.sizes()) + ", expected " +
                              std::to_string(n) + " dimensions");
  }
  int integer(PyObject* o, const char* name) const {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    if (v < INT_MIN || v > INT_MAX) invalid(std::string(name) + " does not fit 32 bits");
    return (int)v;
  }
  float real(PyObject* o) const {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)v;
  }
  // None: the current stream of the call's device; a torch stream, or a handle
  cudaStream_t stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* handle = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (handle == nullptr) throw PythonError{};
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (p == nullptr && PyErr_Occurred()) throw PythonError{};
    return static_cast<cudaStream_t>(p);
  }
  void check(frt_status st, const char* what) const {
    if (st != FRT_OK) throw Error{(int)st, what};
  }
};

// Makes the call's device current for its duration.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(int device) {
    if (c10::cuda::current_device() != device) guard.set_index((c10::DeviceIndex)device);
  }
};

template <typename F>
F entry(PyObject* address) {
  return reinterpret_cast<F>(PyLong_AsVoidPtr(address));
}

// Runs body(call, args) for a call with exactly N arguments.
template <int N, typename Body>
PyObject* run(const char* fn, Py_ssize_t n, Body body) {
  Call call{fn};
  try {
    if (n != N) call.invalid("expected " + std::to_string(N) + " arguments, got " + std::to_string(n));
    body(call);
    Py_RETURN_NONE;
  } catch (const PythonError&) {
    return nullptr;
  } catch (const Error& e) {
    PyObject* value = PyObject_CallFunction(g_error, "sis", fn, e.status, e.message.c_str());
    if (value != nullptr) {
      PyErr_SetObject(g_error, value);
      Py_DECREF(value);
    }
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

const char* describe(PyObject* status_string, frt_status st) {
  return entry<decltype(&frt_status_string)>(status_string)(st);
}

struct Cache {
  uint8_t *k_codes, *k_sf, *v_codes, *v_sf;
  float* scales;
  int capacity;
};
Cache cache(Call& c, PyObject* const* a, int64_t hkv, int64_t hd) {
  const at::Tensor& k = c.tensor(a[0], "k_codes");
  c.dims(k, "k_codes", 3);
  const int64_t cap = k.size(0);
  if (cap > INT_MAX) c.invalid("the capacity does not fit 32 bits");
  Cache r;
  r.capacity = (int)cap;
  r.k_codes = c.pointer<uint8_t>(a[0], "k_codes", at::kByte, {cap, hkv, hd / 2});
  r.k_sf = c.pointer<uint8_t>(a[1], "k_sf", at::kByte, {(cap + 3) / 4, hkv, hd / 16, 4});
  r.v_codes = c.pointer<uint8_t>(a[2], "v_codes", at::kByte, {cap, hkv, hd / 2});
  r.v_sf = c.pointer<uint8_t>(a[3], "v_sf", at::kByte, {(cap + 3) / 4, hkv, hd / 16, 4});
  r.scales = c.pointer<float>(a[4], "kv_scales", at::kFloat, {2});
  return r;
}

// address, status_string, qkv, q_norm_w, k_norm_w, cos, sin, positions, slots,
// q_out, k_codes, k_sf, v_codes, v_sf, kv_scales, status, Hq, Hkv, hd, eps,
// stream
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run<21>("frt_qkv_norm_rope_nvfp4_kvcache", n, [&](Call& c) {
    const at::Tensor& qkv = c.tensor(a[2], "qkv");
    const frt_dtype dt = c.dtype(qkv);
    c.dims(qkv, "qkv", 2);
    const at::ScalarType type = qkv.scalar_type();
    const int64_t M = qkv.size(0);
    const int hq = c.integer(a[16], "Hq"), hkv = c.integer(a[17], "Hkv"), hd = c.integer(a[18], "hd");
    if (hq <= 0 || hkv <= 0 || hd <= 0) c.invalid("Hq, Hkv and hd must be positive");
    void* x = c.pointer(a[2], "qkv", type, {M, ((int64_t)hq + 2 * (int64_t)hkv) * hd});
    void* qw = c.optional(a[3], "q_norm_w", type, {hd});
    void* kw = c.optional(a[4], "k_norm_w", type, {hd});
    const at::Tensor& cos = c.tensor(a[5], "cos_tab");
    c.dims(cos, "cos_tab", 2);
    const int64_t max_pos = cos.size(0);
    float* ct = c.pointer<float>(a[5], "cos_tab", at::kFloat, {max_pos, hd / 2});
    float* st = c.pointer<float>(a[6], "sin_tab", at::kFloat, {max_pos, hd / 2});
    int32_t* pos = c.pointer<int32_t>(a[7], "positions", at::kInt, {M});
    int32_t* slots = c.optional<int32_t>(a[8], "slots", at::kInt, {M});
    void* q = c.pointer(a[9], "q_out", type, {M, hq, hd});
    const Cache kv = cache(c, a + 10, hkv, hd);
    int32_t* status = c.status(a[15]);
    const float eps = c.real(a[19]);
    if (M > INT_MAX || max_pos > INT_MAX) c.invalid("a size does not fit 32 bits");
    const cudaStream_t stream = c.stream(a[20]);
    OnDevice on(c.device);
    const frt_status r = entry<decltype(&frt_qkv_norm_rope_nvfp4_kvcache)>(a[0])(
        x, qw, kw, ct, st, pos, slots, q, kv.k_codes, kv.k_sf, kv.v_codes, kv.v_sf, kv.scales, status, (int)M, hq, hkv,
        hd, (int)max_pos, kv.capacity, eps, dt, stream);
    if (r != FRT_OK) c.check(r, describe(a[1], r));
  });
}

// address, status_string, k_codes, k_sf, v_codes, v_sf, kv_scales, slots, k_out,
// v_out, status, stream
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run<12>("frt_nvfp4_kvcache_read", n, [&](Call& c) {
    const at::Tensor& out = c.tensor(a[8], "k_out");
    const frt_dtype dt = c.dtype(out);
    c.dims(out, "k_out", 3);
    const int64_t rows = out.size(0), hkv = out.size(1), hd = out.size(2);
    const Cache kv = cache(c, a + 2, hkv, hd);
    int32_t* slots = c.optional<int32_t>(a[7], "slots", at::kInt, {rows});
    void* v = c.pointer(a[9], "v_out", out.scalar_type(), {rows, hkv, hd});
    int32_t* status = c.status(a[10]);
    if (rows > INT_MAX || hkv > INT_MAX || hd > INT_MAX) c.invalid("a size does not fit 32 bits");
    const cudaStream_t stream = c.stream(a[11]);
    OnDevice on(c.device);
    const frt_status r = entry<decltype(&frt_nvfp4_kvcache_read)>(a[0])(
        kv.k_codes, kv.k_sf, kv.v_codes, kv.v_sf, kv.scales, slots, out.data_ptr(), v, status, (int)rows, (int)hkv,
        (int)hd, kv.capacity, dt, stream);
    if (r != FRT_OK) c.check(r, describe(a[1], r));
  });
}

// address, status_string, workspace_bytes (address), q, k_codes, k_sf, v_codes,
// v_sf, kv_scales, kv_len, q_indptr, page_table, out, workspace, status, window,
// page_size, max_q_len, max_kv_len, softmax_scale, stream
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run<21>("frt_attn_nvfp4_kvcache", n, [&](Call& c) {
    const at::Tensor& q = c.tensor(a[3], "q");
    const frt_dtype dt = c.dtype(q);
    c.dims(q, "q", 3);
    const int64_t M = q.size(0), hq = q.size(1), hd = q.size(2);
    const at::Tensor& k = c.tensor(a[4], "k_codes");
    c.dims(k, "k_codes", 3);
    const int64_t hkv = k.size(1);
    const Cache kv = cache(c, a + 4, hkv, hd);
    int32_t* kv_len = c.pointer<int32_t>(a[9], "kv_len", at::kInt, {M});
    int64_t n_seqs = 1, max_pages = 0;
    int32_t *indptr = nullptr, *table = nullptr;
    if (a[10] != Py_None) {
      n_seqs = c.tensor(a[10], "q_indptr").numel() - 1;
      if (n_seqs < 1) c.invalid("q_indptr holds no sequence");
      indptr = c.pointer<int32_t>(a[10], "q_indptr", at::kInt, {n_seqs + 1});
    }
    if (a[11] != Py_None) {
      const at::Tensor& t = c.tensor(a[11], "page_table");
      c.dims(t, "page_table", 2);
      max_pages = t.size(1);
      table = c.pointer<int32_t>(a[11], "page_table", at::kInt, {n_seqs, max_pages});
    }
    void* out = c.pointer(a[12], "out", q.scalar_type(), {M, hq, hd});
    int32_t* status = c.status(a[14]);
    const int window = c.integer(a[15], "window"), page_size = c.integer(a[16], "page_size");
    if (M > INT_MAX || hq > INT_MAX || hkv > INT_MAX || hd > INT_MAX || n_seqs > INT_MAX || max_pages > INT_MAX)
      c.invalid("a size does not fit 32 bits");
    const int max_q = a[17] == Py_None ? (int)(M > 0 ? M : 1) : c.integer(a[17], "max_q_len");
    const int64_t holds = table != nullptr ? max_pages * page_size : kv.capacity;
    const int max_kv = a[18] == Py_None ? (int)std::min<int64_t>(std::max<int64_t>(holds, 0), 0x7FFFFF00)
                                        : c.integer(a[18], "max_kv_len");
    const float scale = c.real(a[19]);
    const cudaStream_t stream = c.stream(a[20]);
    OnDevice on(c.device);
    at::Tensor own;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[13] != Py_None) {
      const at::Tensor& t = c.tensor(a[13], "workspace");
      ws = t.data_ptr();
      ws_bytes = t.nbytes();
    } else {
      ws_bytes = entry<decltype(&frt_attn_nvfp4_workspace_bytes)>(a[2])((int)M, (int)n_seqs, (int)hq, (int)hkv, (int)hd,
                                                                      max_q, max_kv);
      if (ws_bytes > 0) {
        // allocated on the launching stream, so that its memory is reused only behind this call
        c10::cuda::OptionalCUDAStreamGuard guard;
        if (a[20] != Py_None) guard.reset_stream(c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)c.device));
        own = at::empty({(int64_t)ws_bytes}, q.options().dtype(at::kByte));
        ws = own.data_ptr();
      }
    }
    const frt_status r = entry<decltype(&frt_attn_nvfp4_kvcache)>(a[0])(
        q.data_ptr(), kv.k_codes, kv.k_sf, kv.v_codes, kv.v_sf, kv.scales, kv_len, indptr, table, out, ws, ws_bytes,
        status, (int)M, (int)n_seqs, (int)hq, (int)hkv, (int)hd, kv.capacity, page_size, (int)max_pages, max_q, max_kv,
        window, scale, dt, stream);
    if (r != FRT_OK) c.check(r, describe(a[1], r));
  });
}

// address, status_string, x, x_scales, x_sf, w_codes, w_sf, w_scale, bias, y,
// x_format, sf_layout, stream
PyObject* matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run<13>("frt_matvec_nvfp4", n, [&](Call& c) {
    const at::Tensor& y = c.tensor(a[9], "y");
    const frt_dtype dt = c.dtype(y);
    c.dims(y, "y", 2);
    const at::Tensor& w = c.tensor(a[5], "w_codes");
    c.dims(w, "w_codes", 2);
    const int64_t M = y.size(0), N = y.size(1), K = 2 * w.size(1);
    if (M > INT_MAX || N > INT_MAX || K > INT_MAX) c.invalid("a size does not fit 32 bits");
    const frt_x_format format = (frt_x_format)c.integer(a[10], "x_format");
    const frt_sf_layout layout = (frt_sf_layout)c.integer(a[11], "sf_layout");
    const auto sf_bytes = [&](int64_t rows) {
      return layout == FRT_SF_SWIZZLED_128X4 ? (rows + 127) / 128 * 128 * ((K / 16 + 3) / 4 * 4) : rows * (K / 16);
    };
    void* x = c.pointer(a[2], "x", format == FRT_X_16BIT ? y.scalar_type() : at::kByte,
                        {M, format == FRT_X_NVFP4 ? K / 2 : K});
    float* xs = nullptr;
    if (format == FRT_X_E4M3_BLOCK)
      xs = c.pointer<float>(a[3], "x_scales", at::kFloat, {M, (K + 127) / 128});
    else if (format != FRT_X_16BIT)
      xs = c.pointer<float>(a[3], "x_scales", at::kFloat, {1});
    uint8_t* xsf = format == FRT_X_NVFP4 ? c.bytes(a[4], "x_sf", sf_bytes(M)) : nullptr;
    uint8_t* wc = c.pointer<uint8_t>(a[5], "w_codes", at::kByte, {N, K / 2});
    uint8_t* wsf = c.bytes(a[6], "w_sf", sf_bytes(N));
    float* ws = c.pointer<float>(a[7], "w_scale", at::kFloat, {1});
    void* bias = c.optional(a[8], "bias", y.scalar_type(), {N});
    const cudaStream_t stream = c.stream(a[12]);
    OnDevice on(c.device);
    const frt_status r = entry<decltype(&frt_matvec_nvfp4)>(a[0])(x, xs, xsf, wc, wsf, ws, bias, y.data_ptr(), (int)M,
                                                                (int)N, (int)K, format, layout, dt, stream);
    if (r != FRT_OK) c.check(r, describe(a[1], r));
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define FRT_FAST(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FRT_FAST(write),
                         FRT_FAST(read),
                         FRT_FAST(attend),
                         FRT_FAST(matvec),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", FRT_BUILT_FOR) != 0) {  // the version of torch
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
