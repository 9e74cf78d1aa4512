// attn_binding.cpp — the Python face of the attention layers' operators: checks torch
// tensors, allocates outputs and calls the C ABI of include/gdn.h.
//
// A CPython extension over torch's C++ tensors instead of ctypes calls: these
// operators take a few microseconds on the GPU for the batches of a decoding step,
// and reading shapes, strides, types and addresses of ten tensors through Python
// attributes took 6 to 13 us a call.  The library's functions are called through
// the addresses that init() gets, so the CUDA library is loaded in one place.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "gdn.h"

namespace {

decltype(&gdn_kv_append) p_append;
decltype(&gdn_kv_gather) p_gather;
decltype(&gdn_attn_decode_paged) p_decode;
decltype(&gdn_attn_decode_paged_workspace_size) p_decode_ws;
decltype(&gdn_attn_prefill) p_prefill;
decltype(&gdn_qk_norm_rope) p_rope;
decltype(&gdn_kv_append_rope) p_append_rope;
decltype(&gdn_attn_prefill_paged) p_prefill_paged;
decltype(&gdn_attn_prefill_paged_workspace_size) p_prefill_paged_ws;
PyObject* g_check;  // check(status, name): raises GdnError

struct Refused {  // a Python exception to raise
  PyObject* type;
  std::string what;
};
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

std::string list(std::initializer_list<int64_t> shape) {
  std::string s = "[";
  for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + "]";
}

bool has_shape(const at::Tensor& t, std::initializer_list<int64_t> shape) {
  return t.sizes() == c10::IntArrayRef(shape.begin(), shape.size());
}

const at::Tensor& ints(PyObject* o, std::initializer_list<int64_t> shape, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!(t.scalar_type() == at::kInt && t.is_cuda() && has_shape(t, shape) && t.is_contiguous()))
    value_error(std::string(name) + " must be " + list(shape) + " int32 on the GPU, contiguous");
  return t;
}

const at::Tensor& rows(PyObject* o, std::initializer_list<int64_t> shape, const char* name,
                       bool dense = false) {
  const at::Tensor& t = tensor(o, name);
  if (!(t.scalar_type() == at::kBFloat16 && t.is_cuda() && has_shape(t, shape) &&
        (!dense || t.is_contiguous())))
    value_error(std::string(name) + " must be " + list(shape) + " bfloat16 on the GPU" +
                (dense ? ", contiguous" : ""));
  return t;
}

// Elements between the tokens of t [T, heads, D]: the heads of a token lie side by
// side, the tokens may be apart (a slice of a fused projection).
int64_t token_stride(const at::Tensor& t, const char* name) {
  const int64_t T = t.size(0), H = t.size(1), D = t.size(2);
  if (t.is_contiguous()) return H * D;
  if (t.stride(2) != 1 || (H > 1 && t.stride(1) != D))
    value_error(std::string(name) + ": a token's heads must be contiguous");
  return T > 1 ? t.stride(0) : H * D;
}

int64_t dim(const at::Tensor& t, int64_t n, const char* name, const char* what) {
  if (t.dim() != n) value_error(std::string(name) + " must be " + what);
  return 0;
}

// The tensors' common device: the call launches there, whatever the current one is.
c10::Device one_device(std::initializer_list<const at::Tensor*> tensors) {
  const c10::Device d = (*tensors.begin())->device();
  for (const at::Tensor* t : tensors)
    if (t->device() != d) value_error("tensors must be on one device, got " + d.str() + " and " + t->device().str());
  return d;
}

struct Cache {  // a paged cache's tensors and sizes
  c10::Device device = c10::Device(c10::kCPU);
  const void *k, *v;
  const uint8_t *ke = nullptr, *ve = nullptr;
  const int32_t* table;
  int64_t P, h_kv, page, D, N, max_pages;
  gdn_cache_dtype dtype;
  at::TensorOptions options;  // of rows read back
  void with(std::initializer_list<const at::Tensor*> tensors) const {
    if (one_device(tensors) != device)
      value_error("tensors must be on the cache's device " + device.str() + ", got " + one_device(tensors).str());
  }
  Cache(PyObject* k_pages, PyObject* v_pages, PyObject* page_table, PyObject* k_exp, PyObject* v_exp) {
    const at::Tensor &kp = tensor(k_pages, "k_pages"), &vp = tensor(v_pages, "v_pages");
    const at::Tensor& pt = tensor(page_table, "page_table");
    if (kp.scalar_type() == at::kBFloat16) dtype = GDN_CACHE_BF16;
    else if (kp.scalar_type() == at::kFloat8_e4m3fn) dtype = GDN_CACHE_E4M3;
    else throw Refused{PyExc_TypeError, std::string("pages must be bfloat16 or float8_e4m3fn, got ") +
                                            c10::toString(kp.scalar_type())};
    if (!(kp.dim() == 4 && vp.sizes() == kp.sizes() && vp.scalar_type() == kp.scalar_type() &&
          kp.is_contiguous() && vp.is_contiguous() && kp.is_cuda() && vp.is_cuda()))
      value_error("k_pages / v_pages must be [num_pages, h_kv, page_size, D] of one dtype on the GPU, "
                  "contiguous");
    P = kp.size(0);
    h_kv = kp.size(1);
    page = kp.size(2);
    D = kp.size(3);
    if (dtype == GDN_CACHE_E4M3) {
      auto exps = [&](PyObject* o) -> const uint8_t* {
        if (o != Py_None) {
          const at::Tensor& t = tensor(o, "k_exp / v_exp");
          if (has_shape(t, {P, h_kv, page}) && t.scalar_type() == at::kByte && t.is_cuda() && t.is_contiguous())
            return static_cast<const uint8_t*>(t.data_ptr());
        }
        value_error("k_exp / v_exp must be [num_pages, h_kv, page_size] uint8 on the GPU, contiguous");
      };
      ke = exps(k_exp);
      ve = exps(v_exp);
    }
    if (!(pt.dim() == 2 && pt.scalar_type() == at::kInt && pt.is_cuda() && pt.is_contiguous()))
      value_error("page_table must be [num_seqs, max_pages] int32 on the GPU, contiguous");
    N = pt.size(0);
    max_pages = pt.size(1);
    k = kp.data_ptr();
    v = vp.data_ptr();
    table = static_cast<const int32_t*>(pt.data_ptr());
    options = kp.options().dtype(at::kBFloat16);
    device = one_device({&kp, &vp, &pt});
    if (dtype == GDN_CACHE_E4M3) one_device({&kp, &tensor(k_exp, "k_exp"), &tensor(v_exp, "v_exp")});
  }
};

// Where a call launches: on its tensors' device and the given stream, or that device's
// current one; and the tensors that belong on the stream.  What a call on another stream
// than the current one allocates comes from that stream's own memory: a block of the
// current stream's may still be written by work queued there.  An output of such a call is
// not given out again before the current stream, where the caller gets it, has passed the
// point where it is freed; a tensor of the caller's not before the call's stream has.
struct Launch {
  c10::cuda::OptionalCUDAGuard on;  // only where another device is the current one
  cudaStream_t handle;
  bool other;  // than the current one
  Launch(c10::Device device, PyObject* o) {
    if (c10::cuda::current_device() != device.index()) on.set_device(device);
    const cudaStream_t current = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    handle = current;
    if (o != Py_None) {
      PyObject* h = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream")
                                                             : PyNumber_Long(o);
      if (!h) throw python_error();
      handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
      Py_DECREF(h);
      if (PyErr_Occurred()) throw python_error();
      if (handle == cudaStreamLegacy) handle = nullptr;  // the same stream, as torch names it
    }
    other = handle != current;
  }
  c10::cuda::CUDAStream of_torch(c10::DeviceIndex device) const {
    return c10::cuda::getStreamFromExternal(handle, device);
  }
  // (past the dispatcher: a call with two outputs takes 4.7 us of host time, with at::empty 5.1)
  static at::Tensor empty(c10::IntArrayRef shape, const at::TensorOptions& options) {
    return at::Tensor(at::detail::empty_cuda(shape, options));
  }
  at::Tensor scratch(c10::IntArrayRef shape, const at::TensorOptions& options) const {
    if (!other) return empty(shape, options);
    const c10::cuda::CUDAStreamGuard on(of_torch(options.device().index()));
    return empty(shape, options);
  }
  at::Tensor output(c10::IntArrayRef shape, const at::TensorOptions& options) const {
    at::Tensor t = scratch(shape, options);
    if (other) t.record_stream(c10::cuda::getCurrentCUDAStream(t.device().index()));
    return t;
  }
  const at::Tensor& given(const at::Tensor& t) const {
    if (other) t.record_stream(of_torch(t.device().index()));
    return t;
  }
  gdn_stream_t abi() const { return reinterpret_cast<gdn_stream_t>(handle); }
};

void check(gdn_status st, const char* name) {
  if (st == GDN_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", static_cast<int>(st), name);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, name);
  throw python_error();
}

float scale_of(PyObject* o, int64_t D) {
  if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  const double s = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw python_error();
  return static_cast<float>(s);
}

int32_t as32(int64_t n) {  // sizes beyond 32 bits: a value that the library refuses
  return n > INT32_MAX ? INT32_MAX : static_cast<int32_t>(n);
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

const int32_t* i32_of(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }

// kv_append(k, v, k_pages, v_pages, page_table, cu_seqlens, start_pos, k_exp, v_exp, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Cache c(a[2], a[3], a[4], a[7], a[8]);
    const at::Tensor& k0 = tensor(a[0], "k");
    dim(k0, 3, "k", "[T, h_kv, D]");
    const int64_t T = k0.size(0);
    const at::Tensor &k = rows(a[0], {T, c.h_kv, c.D}, "k"), &v = rows(a[1], {T, c.h_kv, c.D}, "v");
    const at::Tensor &cu = ints(a[5], {c.N + 1}, "cu_seqlens"), &st = ints(a[6], {c.N}, "start_pos");
    c.with({&k, &v, &cu, &st});
    const Launch s(c.device, a[9]);
    check(p_append(k.data_ptr(), v.data_ptr(), token_stride(k, "k"), token_stride(v, "v"),
                   const_cast<void*>(c.k), const_cast<void*>(c.v), const_cast<uint8_t*>(c.ke),
                   const_cast<uint8_t*>(c.ve), c.table, i32_of(cu), i32_of(st), as32(c.N), T, as32(c.h_kv),
                   as32(c.D), as32(c.page), as32(c.P), as32(c.max_pages), c.dtype, s.abi()),
          "gdn_kv_append");
    Py_RETURN_NONE;
  });
}

// kv_gather(k_pages, v_pages, page_table, cu_seqlens, start_pos, total, k_exp, v_exp, k, v, stream)
PyObject* kv_gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Cache c(a[0], a[1], a[2], a[6], a[7]);
    const int64_t T = PyLong_AsLongLong(a[5]);
    if (PyErr_Occurred()) throw python_error();
    if (T < 0) value_error("total_tokens must not be negative");
    const at::Tensor &cu = ints(a[3], {c.N + 1}, "cu_seqlens"), &st = ints(a[4], {c.N}, "start_pos");
    c.with({&cu, &st});
    const Launch s(c.device, a[10]);
    auto out = [&](PyObject* o, const char* name) {
      return o == Py_None ? s.output({T, c.h_kv, c.D}, c.options) : s.given(rows(o, {T, c.h_kv, c.D}, name));
    };
    const at::Tensor k = out(a[8], "k"), v = out(a[9], "v");
    c.with({&k, &v});
    check(p_gather(k.data_ptr(), v.data_ptr(), token_stride(k, "k"), token_stride(v, "v"), c.k, c.v, c.ke,
                   c.ve, c.table, i32_of(cu), i32_of(st), as32(c.N), T, as32(c.h_kv), as32(c.D),
                   as32(c.page), as32(c.P), as32(c.max_pages), c.dtype, s.abi()),
          "gdn_kv_gather");
    PyObject *pk = THPVariable_Wrap(k), *pv = THPVariable_Wrap(v);
    return pk && pv ? Py_BuildValue("(NN)", pk, pv) : nullptr;
  });
}

// attn_decode_paged(q, k_pages, v_pages, page_table, cache_len, k_exp, v_exp, scale, o, workspace, stream)
PyObject* attn_decode_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Cache c(a[1], a[2], a[3], a[5], a[6]);
    const at::Tensor& q0 = tensor(a[0], "q");
    dim(q0, 3, "q", "[B, h_q, D]");
    const int64_t h_q = q0.size(1);
    const at::Tensor& q = rows(a[0], {c.N, h_q, c.D}, "q");
    const at::Tensor& len = ints(a[4], {c.N}, "cache_len");
    const float scale = scale_of(a[7], c.D);
    c.with({&q, &len});
    const Launch s(c.device, a[10]);
    const at::Tensor o = a[8] == Py_None ? s.output({c.N, h_q, c.D}, c.options)
                                         : s.given(rows(a[8], {c.N, h_q, c.D}, "o", true));
    at::Tensor ws;
    if (a[9] == Py_None) {
      ws = s.scratch({(int64_t)p_decode_ws(as32(h_q), as32(c.h_kv), as32(c.D))}, c.options.dtype(at::kByte));
    } else {
      ws = tensor(a[9], "workspace");
      if (!(ws.is_cuda() && ws.is_contiguous())) value_error("workspace must be on the GPU, contiguous");
    }
    c.with({&o, &ws});
    check(p_decode(q.data_ptr(), token_stride(q, "q"), c.k, c.v, c.ke, c.ve, c.table, i32_of(len), o.data_ptr(),
                   as32(c.N), as32(h_q), as32(c.h_kv), as32(c.D), as32(c.page), as32(c.P), as32(c.max_pages),
                   c.dtype, scale, ws.numel() ? ws.data_ptr() : nullptr, ws.nbytes(), s.abi()),
          "gdn_attn_decode_paged");
    return THPVariable_Wrap(o);
  });
}

// attn_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k, scale, o, stream)
PyObject* attn_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor &q0 = tensor(a[0], "q"), &k0 = tensor(a[1], "k");
    dim(q0, 3, "q", "[Tq, h_q, D]");
    dim(k0, 3, "k", "[Tk, h_kv, D]");
    const int64_t Tq = q0.size(0), h_q = q0.size(1), D = q0.size(2), Tk = k0.size(0), h_kv = k0.size(1);
    const at::Tensor &q = rows(a[0], {Tq, h_q, D}, "q"), &k = rows(a[1], {Tk, h_kv, D}, "k");
    const at::Tensor& v = rows(a[2], {Tk, h_kv, D}, "v");
    const int64_t N = tensor(a[3], "cu_seqlens_q").numel() - 1;
    const at::Tensor& cq = ints(a[3], {N + 1}, "cu_seqlens_q");
    const at::Tensor& ck = a[4] == Py_None ? cq : ints(a[4], {N + 1}, "cu_seqlens_k");
    if (N < 0) value_error("cu_seqlens_q must have at least one entry");
    const float scale = scale_of(a[5], D);
    const Launch s(one_device({&q, &k, &v, &cq, &ck}), a[7]);
    const at::Tensor o = a[6] == Py_None ? s.output({Tq, h_q, D}, q.options())
                                         : s.given(rows(a[6], {Tq, h_q, D}, "o", true));
    one_device({&q, &o});
    check(p_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), i32_of(cq), i32_of(ck), as32(N), Tq,
                    Tk, as32(h_q), as32(h_kv), as32(D), token_stride(q, "q"), token_stride(k, "k"),
                    token_stride(v, "v"), GDN_BF16, scale, s.abi()),
          "gdn_attn_prefill");
    return THPVariable_Wrap(o);
  });
}

// A count that may be None (0); a negative one is refused.
int32_t count_of(PyObject* o, const char* name) {
  if (o == Py_None) return 0;
  const int64_t n = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) throw python_error();
  if (n < 0) value_error(std::string(name) + " must not be negative");
  return as32(n);
}

// attn_prefill_paged(q, k_pages, v_pages, page_table, cu_seqlens_q, cache_len, k_exp, v_exp, window, sinks, scale,
//                    o, workspace, stream)
PyObject* attn_prefill_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Cache c(a[1], a[2], a[3], a[6], a[7]);
    const at::Tensor& q0 = tensor(a[0], "q");
    dim(q0, 3, "q", "[T, h_q, D]");
    const int64_t T = q0.size(0), h_q = q0.size(1);
    const at::Tensor& q = rows(a[0], {T, h_q, c.D}, "q");
    const at::Tensor &cu = ints(a[4], {c.N + 1}, "cu_seqlens_q"), &len = ints(a[5], {c.N}, "cache_len");
    const int32_t window = count_of(a[8], "window"), sinks = count_of(a[9], "sinks");
    if (a[8] != Py_None && window == 0) value_error("window must be positive, or None");
    const float scale = scale_of(a[10], c.D);
    c.with({&q, &cu, &len});
    const Launch s(c.device, a[13]);
    const at::Tensor o = a[11] == Py_None ? s.output({T, h_q, c.D}, c.options)
                                          : s.given(rows(a[11], {T, h_q, c.D}, "o", true));
    at::Tensor ws;
    if (a[12] == Py_None) {
      ws = s.scratch({(int64_t)p_prefill_paged_ws(as32(h_q), as32(c.h_kv), as32(c.D), c.dtype, T)}, c.options.dtype(at::kByte));
    } else {
      ws = tensor(a[12], "workspace");
      if (!(ws.is_cuda() && ws.is_contiguous())) value_error("workspace must be on the GPU, contiguous");
      s.given(ws);
    }
    c.with({&o, &ws});
    check(p_prefill_paged(q.data_ptr(), token_stride(q, "q"), c.k, c.v, c.ke, c.ve, c.table, i32_of(cu), i32_of(len),
                          o.data_ptr(), as32(c.N), T, as32(h_q), as32(c.h_kv), as32(c.D), as32(c.page), as32(c.P),
                          as32(c.max_pages), c.dtype, scale, window, sinks, ws.numel() ? ws.data_ptr() : nullptr,
                          ws.nbytes(), s.abi()),
          "gdn_attn_prefill_paged");
    return THPVariable_Wrap(o);
  });
}

struct Rotation {  // how heads are normalised and turned, and the positions
  const at::Tensor* tensors[4];  // those given, for one_device
  int given = 0;
  const int32_t* positions = nullptr;
  const float *freq, *qw = nullptr, *kw = nullptr;
  int64_t axes = 1, rotary;
  float eps = 0.f;
  uint32_t options = 0;
  std::string axis_of;  // a byte for each frequency
  Rotation(PyObject* pos, PyObject* inv_freq, PyObject* q_weight, PyObject* k_weight, PyObject* norm_eps,
           PyObject* axes_, PyObject* interleaved, int64_t T, int64_t D) {
    auto floats = [&](PyObject* o, int64_t n, const char* name) {
      const at::Tensor& t = tensor(o, name);
      if (!(t.scalar_type() == at::kFloat && t.is_cuda() && t.dim() == 1 && (n < 0 || t.numel() == n) && t.is_contiguous()))
        value_error(std::string(name) + " must be [" + (n < 0 ? "rotary_dim / 2" : std::to_string(n)) +
                    "] float32 on the GPU, contiguous");
      tensors[given++] = &t;
      return static_cast<const float*>(t.data_ptr());
    };
    freq = floats(inv_freq, -1, "inv_freq");
    rotary = 2 * tensors[0]->numel();
    if (axes_ != Py_None) {
      PyObject* bytes = PyBytes_FromObject(axes_);
      if (!bytes) throw python_error();
      axis_of.assign(PyBytes_AS_STRING(bytes), static_cast<size_t>(PyBytes_GET_SIZE(bytes)));
      Py_DECREF(bytes);
      if (static_cast<int64_t>(axis_of.size()) != rotary / 2)
        value_error("axes must have an entry for each of the " + std::to_string(rotary / 2) + " frequencies");
    }
    if (pos != Py_None) {
      const at::Tensor& t = tensor(pos, "positions");
      if (axes_ != Py_None && t.dim() == 2) axes = t.size(0);
      const bool shape = axes_ == Py_None ? has_shape(t, {T}) : has_shape(t, {axes, T});
      if (!(t.scalar_type() == at::kInt && t.is_cuda() && shape && t.is_contiguous()))
        value_error(std::string("positions must be ") + (axes_ == Py_None ? list({T}) : "[axes, " + std::to_string(T) + "]") +
                    " int32 on the GPU, contiguous");
      for (const char c : axis_of)
        if (static_cast<uint8_t>(c) >= axes) value_error("axes must be below " + std::to_string(axes) + ", the axes of positions");
      tensors[given++] = &t;
      positions = static_cast<const int32_t*>(t.data_ptr());
    } else if (axes_ != Py_None) {
      value_error("axes need positions");
    }
    if (norm_eps != Py_None) {
      eps = static_cast<float>(PyFloat_AsDouble(norm_eps));
      if (PyErr_Occurred()) throw python_error();
      options |= GDN_ROPE_RMSNORM;
      if (q_weight != Py_None) qw = floats(q_weight, D, "q_weight");
      if (k_weight != Py_None) kw = floats(k_weight, D, "k_weight");
    } else if (q_weight != Py_None || k_weight != Py_None) {
      value_error("q_weight / k_weight need norm_eps");
    }
    const int yes = PyObject_IsTrue(interleaved);
    if (yes < 0) throw python_error();
    if (yes) options |= GDN_ROPE_INTERLEAVED;
  }
  const uint8_t* of() const { return axis_of.empty() ? nullptr : reinterpret_cast<const uint8_t*>(axis_of.data()); }
  void on(c10::Device d) const {
    for (int i = 0; i < given; ++i)
      if (tensors[i]->device() != d) value_error("tensors must be on one device, got " + d.str() + " and " + tensors[i]->device().str());
  }
};

// qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, norm_eps, axes, interleaved, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor &q0 = tensor(a[0], "q"), &k0 = tensor(a[1], "k");
    dim(q0, 3, "q", "[T, h_q, D]");
    dim(k0, 3, "k", "[T, h_kv, D]");
    const int64_t T = q0.size(0), h_q = q0.size(1), D = q0.size(2), h_kv = k0.size(1);
    const at::Tensor &q = rows(a[0], {T, h_q, D}, "q"), &k = rows(a[1], {T, h_kv, D}, "k");
    if (a[2] == Py_None) value_error("positions must be given");
    const Rotation r(a[2], a[3], a[4], a[5], a[6], a[7], a[8], T, D);
    const c10::Device device = one_device({&q, &k});
    r.on(device);
    const Launch s(device, a[11]);
    auto out = [&](PyObject* o, int64_t h, const char* name) {
      return o == Py_None ? s.output({T, h, D}, q.options()) : s.given(rows(o, {T, h, D}, name));
    };
    const at::Tensor qo = out(a[9], h_q, "q_out"), ko = out(a[10], h_kv, "k_out");
    one_device({&q, &qo, &ko});
    check(p_rope(q.data_ptr(), k.data_ptr(), token_stride(q, "q"), token_stride(k, "k"), qo.data_ptr(), ko.data_ptr(),
                 token_stride(qo, "q_out"), token_stride(ko, "k_out"), r.positions, as32(r.axes), r.of(), r.freq,
                 as32(r.rotary), r.qw, r.kw, r.eps, T, as32(h_q), as32(h_kv), as32(D), GDN_BF16, r.options, s.abi()),
          "gdn_qk_norm_rope");
    PyObject *pq = THPVariable_Wrap(qo), *pk = THPVariable_Wrap(ko);
    return pq && pk ? Py_BuildValue("(NN)", pq, pk) : nullptr;
  });
}

// kv_append_rope(q, k, v, k_pages, v_pages, page_table, cu_seqlens, start_pos, positions, inv_freq, q_weight,
//                k_weight, norm_eps, axes, interleaved, k_exp, v_exp, q_out, stream)
PyObject* kv_append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&]() -> PyObject* {
    const Cache c(a[3], a[4], a[5], a[15], a[16]);
    const at::Tensor& k0 = tensor(a[1], "k");
    dim(k0, 3, "k", "[T, h_kv, D]");
    const int64_t T = k0.size(0);
    const at::Tensor &k = rows(a[1], {T, c.h_kv, c.D}, "k"), &v = rows(a[2], {T, c.h_kv, c.D}, "v");
    const at::Tensor &cu = ints(a[6], {c.N + 1}, "cu_seqlens"), &st = ints(a[7], {c.N}, "start_pos");
    int64_t h_q = 0, q_stride = 0, o_stride = 0;
    if (a[0] != Py_None) {
      dim(tensor(a[0], "q"), 3, "q", "[T, h_q, D]");
      h_q = tensor(a[0], "q").size(1);
      const at::Tensor& q = rows(a[0], {T, h_q, c.D}, "q");
      c.with({&q});
      q_stride = token_stride(q, "q");
    } else if (a[17] != Py_None) {
      value_error("q_out needs q");
    }
    const Rotation r(a[8], a[9], a[10], a[11], a[12], a[13], a[14], T, c.D);
    c.with({&k, &v, &cu, &st});
    r.on(c.device);
    const Launch s(c.device, a[18]);
    at::Tensor qo;
    if (h_q > 0) {
      qo = a[17] == Py_None ? s.output({T, h_q, c.D}, c.options) : s.given(rows(a[17], {T, h_q, c.D}, "q_out"));
      c.with({&qo});
      o_stride = token_stride(qo, "q_out");
    }
    check(p_append_rope(h_q > 0 ? tensor(a[0], "q").data_ptr() : nullptr, k.data_ptr(), v.data_ptr(), q_stride,
                        token_stride(k, "k"), token_stride(v, "v"), h_q > 0 ? qo.data_ptr() : nullptr, o_stride,
                        const_cast<void*>(c.k), const_cast<void*>(c.v), const_cast<uint8_t*>(c.ke),
                        const_cast<uint8_t*>(c.ve), c.table, i32_of(cu), i32_of(st), r.positions, as32(r.axes), r.of(),
                        r.freq, as32(r.rotary), r.qw, r.kw, r.eps, as32(c.N), T, as32(h_q), as32(c.h_kv), as32(c.D),
                        as32(c.page), as32(c.P), as32(c.max_pages), c.dtype, r.options, s.abi()),
          "gdn_kv_append_rope");
    if (h_q == 0) Py_RETURN_NONE;
    return THPVariable_Wrap(qo);
  });
}

// token_stride(t): what the calls take for the distance of t's tokens
PyObject* token_stride_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    dim(tensor(a[0], "t"), 3, "t", "[T, heads, D]");
    return PyLong_FromLongLong(token_stride(tensor(a[0], "t"), "t"));
  });
}

// one_device(t, u): None where the calls take both tensors together
PyObject* one_device_py(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    one_device({&tensor(a[0], "t"), &tensor(a[1], "u")});
    Py_RETURN_NONE;
  });
}

// init(check, addresses of the functions)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int kFunctions = 9;
  return guarded(n, 1 + kFunctions, [&]() -> PyObject* {
    void* p[kFunctions];
    for (int i = 0; i < kFunctions; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i + 1]);
      if (PyErr_Occurred()) throw python_error();
    }
    p_append = reinterpret_cast<decltype(p_append)>(p[0]);
    p_gather = reinterpret_cast<decltype(p_gather)>(p[1]);
    p_decode = reinterpret_cast<decltype(p_decode)>(p[2]);
    p_decode_ws = reinterpret_cast<decltype(p_decode_ws)>(p[3]);
    p_prefill = reinterpret_cast<decltype(p_prefill)>(p[4]);
    p_rope = reinterpret_cast<decltype(p_rope)>(p[5]);
    p_append_rope = reinterpret_cast<decltype(p_append_rope)>(p[6]);
    p_prefill_paged = reinterpret_cast<decltype(p_prefill_paged)>(p[7]);
    p_prefill_paged_ws = reinterpret_cast<decltype(p_prefill_paged_ws)>(p[8]);
    Py_INCREF(a[0]);
    Py_XDECREF(g_check);
    g_check = a[0];
    Py_RETURN_NONE;
  });
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("init", init),
                         FAST("kv_append", kv_append),
                         FAST("kv_gather", kv_gather),
                         FAST("attn_decode_paged", attn_decode_paged),
                         FAST("attn_prefill", attn_prefill),
                         FAST("attn_prefill_paged", attn_prefill_paged),
                         FAST("qk_norm_rope", qk_norm_rope),
                         FAST("kv_append_rope", kv_append_rope),
                         FAST("token_stride", token_stride_py),
                         FAST("one_device", one_device_py),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_binding() { return PyModule_Create(&module); }
