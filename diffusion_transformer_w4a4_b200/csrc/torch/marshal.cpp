// Argument marshalling of the calls between a block's projections and of the FP8 layer: from torch tensors to the C
// interface, with the checks that need a tensor (type, device, shape, contiguity; the library checks the rest).
//
// Small calls are bound by the host: through ctypes and tensor attributes read one by one, a query/key norm of one token
// takes 15 us and an attention 10 us of Python, against 3 and 14 us on the GPU.  Here the fields are read directly.
// The library's functions come as addresses, so that this module serves the release and the debug library alike.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <exception>
#include <string>

#include "svdq.h"

namespace {

decltype(&svdq_qk_norm_rope) g_norm = nullptr;
decltype(&svdq_cross_attn) g_attn = nullptr;
decltype(&svdq_fp8_forward) g_fp8 = nullptr;
decltype(&svdq_fp8_workspace_size) g_fp8_size = nullptr;
PyObject* g_error = nullptr;      // SvdqError(status, where)
PyObject* g_new_status = nullptr;  // attn_status(device index), which calls set_status
PyObject* g_out_of_memory = nullptr;  // torch.OutOfMemoryError
constexpr int kDevices = 64;
int32_t* g_status[kDevices] = {};

struct PyError {};  // a Python exception is set
[[noreturn]] void value_error(const std::string& s) {
  PyErr_SetString(PyExc_ValueError, s.c_str());
  throw PyError();
}
// Text of a message's parts (no streams: their locale may come from another copy of the C++ library in the process).
std::string text(const char* s) { return s; }
std::string text(int64_t v) { return std::to_string(v); }
std::string text(const c10::Device& d) { return d.str(); }
std::string text(at::ScalarType t) { return c10::toString(t); }
std::string text(at::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}
template <class... A>
[[noreturn]] void refuse(const A&... a) {
  value_error((text(a) + ...));
}

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a torch tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw PyError();
  }
  return THPVariable_Unpack(o);
}

// A bf16 [batch, tokens, heads, dim] view on `device`.
svdq_heads heads(const char* name, const at::Tensor& t, const c10::Device& device) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || !t.is_cuda())
    refuse(name, ": expected a bf16 CUDA tensor [batch, tokens, heads, dim], got ", t.scalar_type(), " ", t.sizes(),
           " on ", t.device());
  if (t.device() != device) refuse(name, " on ", t.device(), ", q on ", device);
  const auto st = t.strides();
  if (st[3] != 1 && t.size(3) > 1) refuse(name, ": the last dimension must be contiguous");
  return {t.data_ptr(), st[0], st[1], st[2]};
}
// A contiguous tensor of a given type and shape on `device`.
void* aux(const char* name, const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const c10::Device& device) {
  if (t.scalar_type() != type || t.device() != device || t.sizes() != shape || !t.is_contiguous())
    refuse(name, ": expected a contiguous ", type, " tensor ", shape, " on ", device, ", got ", t.scalar_type(), " ",
           t.sizes(), " on ", t.device());
  return t.data_ptr();
}

int32_t* status_of(PyObject* o, const c10::Device& device) {
  if (o != Py_None) return (int32_t*)aux("status", tensor("status", o), at::kInt, {1}, device);
  const int i = device.index();
  if (i < 0 || i >= kDevices) refuse("no status word on ", device);
  if (!g_status[i]) {
    PyObject* r = PyObject_CallFunction(g_new_status, "i", i);
    if (!r) throw PyError();
    Py_DECREF(r);
    if (!g_status[i]) refuse("no status word on ", device);
  }
  return g_status[i];
}
void* stream_of(PyObject* o, const c10::Device& device) {
  if (o == Py_None) return (void*)c10::cuda::getCurrentCUDAStream(device.index()).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) throw PyError();
  return p;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return v;
}

// Memory of stream `owner` that a call on `stream` uses: the allocator hands it to nobody before the call is done, though it
// be dropped earlier.  A raw handle's stream is not noted, as it may be destroyed before the memory is freed.
void note_use(const at::Tensor& t, void* owner, const c10::cuda::CUDAStream& stream) {
  const cudaStream_t handle = stream.stream();
  if ((void*)handle == owner) return;
  if (handle && stream == c10::cuda::getStreamFromExternal(handle, stream.device_index())) return;
  t.record_stream(stream);
}

[[noreturn]] void raise_status(int status, const char* where) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PyError();
}
// call() with `device` current; a status other than SVDQ_OK raises.
template <class F>
void run(const c10::Device& device, const char* where, F&& call) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != device.index()) guard.set_index(device.index());
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = call();
  Py_END_ALLOW_THREADS;
  if (st != SVDQ_OK) raise_status(st, where);
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const PyError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory ? g_out_of_memory : PyExc_MemoryError, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// qk_norm_rope(q, k, q_weight, k_weight, eps, rope, positions, pairs, out_q, out_k, status, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor& q = tensor("q", a[0]);
    const c10::Device device = q.device();
    const bool both = a[1] != Py_None;
    svdq_norm_rope_args args[2];
    at::Tensor out[2];
    const float* table = nullptr;
    int64_t rows = 0, rot = 0, dim = 0;
    for (int i = 0; i < (both ? 2 : 1); ++i) {
      const at::Tensor& x = i ? tensor("k", a[1]) : q;
      svdq_norm_rope_args& r = args[i];
      r.x = heads(i ? "k" : "q", x, device);
      if (i == 0) {
        dim = x.size(3);
        if (a[5] != Py_None) {
          const at::Tensor& t = tensor("rope", a[5]);
          if (t.dim() != 3 || t.size(2) != 2) refuse("rope: expected [rows, rot/2, 2], got ", t.sizes());
          table = (const float*)aux("rope", t, at::kFloat, t.sizes(), device);
          rows = t.size(0);
          rot = 2 * t.size(1);
        } else if (a[6] != Py_None) {
          refuse("positions need a rope table");
        }
      } else if (x.size(3) != dim) {
        refuse("heads of ", dim, " (q) and ", x.size(3), " (k)");
      }
      r.batch = x.size(0);
      r.tokens = x.size(1);
      r.heads = x.size(2);
      PyObject* w = a[2 + i];
      r.weight = w == Py_None ? nullptr : aux(i ? "k_weight" : "q_weight", tensor("weight", w), at::kBFloat16, {dim}, device);
      r.rope = table;
      r.rope_rows = rows;
      r.positions = a[6] == Py_None ? nullptr
                                    : (const int32_t*)aux(i ? "positions (for k)" : "positions", tensor("positions", a[6]),
                                                          at::kInt, {r.batch, r.tokens}, device);
      if (a[8 + i] == Py_None) {
        out[i] = at::empty_like(x);
        const auto st = out[i].strides();
        r.y = {out[i].data_ptr(), st[0], st[1], st[2]};
      } else {
        const at::Tensor& o = tensor(i ? "out_k" : "out_q", a[8 + i]);
        r.y = heads(i ? "out_k" : "out_q", o, device);
        if (o.sizes() != x.sizes()) refuse(i ? "out_k: " : "out_q: ", o.sizes(), " for ", x.sizes());
      }
    }
    const float eps = (float)number(a[4]);
    const int pairs = (int)integer(a[7]);
    int32_t* status = status_of(a[10], device);
    void* stream = stream_of(a[11], device);
    run(device, "svdq_qk_norm_rope",
        [&] { return g_norm(&args[0], both ? &args[1] : nullptr, dim, rot, pairs, eps, status, stream); });
    PyObject* r[2] = {nullptr, nullptr};
    for (int i = 0; i < (both ? 2 : 1); ++i) r[i] = a[8 + i] == Py_None ? THPVariable_Wrap(out[i]) : Py_NewRef(a[8 + i]);
    if (!both) return r[0];
    PyObject* t = PyTuple_Pack(2, r[0], r[1]);
    Py_DECREF(r[0]);
    Py_DECREF(r[1]);
    return t;
  });
}

// cross_attn(q, k, v, kv_len, kv_mask, scale, out, status, stream)
PyObject* cross_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]);
    const c10::Device device = q.device();
    svdq_attn_args r;
    r.q = heads("q", q, device);
    r.k = heads("k", k, device);
    r.v = heads("v", v, device);
    r.batch = q.size(0);
    r.q_tokens = q.size(1);
    r.kv_tokens = k.size(1);
    r.heads = q.size(2);
    r.kv_heads = k.size(2);
    r.dim = q.size(3);
    if (k.sizes() != v.sizes() || k.size(0) != r.batch || k.size(3) != r.dim)
      refuse("q ", q.sizes(), ", k ", k.sizes(), ", v ", v.sizes(), " do not fit");
    r.kv_len = a[3] == Py_None ? nullptr
                               : (const int32_t*)aux("kv_len", tensor("kv_len", a[3]), at::kInt, {r.batch}, device);
    r.kv_mask = nullptr;
    r.mask_stride = 0;
    if (a[4] != Py_None) {
      const at::Tensor& m = tensor("kv_mask", a[4]);
      if ((m.scalar_type() != at::kByte && m.scalar_type() != at::kBool) || m.device() != device || m.dim() != 2 ||
          m.size(0) != r.batch || m.size(1) != r.kv_tokens || (r.kv_tokens > 1 && m.stride(1) != 1))
        refuse("kv_mask: expected uint8 or bool [", r.batch, ", ", r.kv_tokens, "] on ", device, ", rows contiguous, got ",
               m.scalar_type(), " ", m.sizes(), " on ", m.device());
      r.kv_mask = (const uint8_t*)m.data_ptr();
      r.mask_stride = m.stride(0);
    }
    r.scale = a[5] == Py_None ? (float)std::pow((double)r.dim, -0.5) : (float)number(a[5]);
    at::Tensor out;
    if (a[6] == Py_None) {
      out = at::empty_like(q);
      const auto st = out.strides();
      r.o = {out.data_ptr(), st[0], st[1], st[2]};
    } else {
      const at::Tensor& o = tensor("out", a[6]);
      r.o = heads("out", o, device);
      if (o.sizes() != q.sizes()) refuse("out ", o.sizes(), " for q ", q.sizes());
    }
    int32_t* status = status_of(a[7], device);
    void* stream = stream_of(a[8], device);
    run(device, "svdq_cross_attn", [&] { return g_attn(&r, status, stream); });
    return a[6] == Py_None ? THPVariable_Wrap(out) : Py_NewRef(a[6]);
  });
}

// fp8_forward(handle, N, K, device index, memory, x, out, stream, id) -> y, or None where there is no workspace for so many
// tokens yet.  The memory: (buffer whose end is the workspace, handle of its stream, weights, handle of theirs), or None.
// With an output the stream may be a handle other than the current stream's, and torch's id of it.
PyObject* fp8_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const auto* layer = (const svdq_fp8_layer*)PyLong_AsVoidPtr(a[0]);
    const int64_t N = integer(a[1]), K = integer(a[2]);
    const c10::Device device(c10::DeviceType::CUDA, (c10::DeviceIndex)integer(a[3]));
    if (PyErr_Occurred()) throw PyError();
    const at::Tensor& x = tensor("x", a[5]);
    if (x.scalar_type() != at::kBFloat16 || !x.is_cuda() || !x.is_contiguous() || x.dim() < 1 || x.size(-1) != K)
      refuse("expected a contiguous bf16 CUDA tensor [..., ", K, "], got ", x.scalar_type(), " ", x.sizes());
    if (x.device() != device) refuse("input on ", x.device(), ", layer on ", device);
    const int64_t M = x.numel() / K;
    PyObject* const w = a[4];
    if (w == Py_None) Py_RETURN_NONE;
    if (!PyTuple_Check(w) || PyTuple_GET_SIZE(w) != 4) refuse("memory: expected a tuple of four");
    const at::Tensor &buf = tensor("buffer", PyTuple_GET_ITEM(w, 0)), &blob = tensor("weights", PyTuple_GET_ITEM(w, 2));
    void *const buf_owner = PyLong_AsVoidPtr(PyTuple_GET_ITEM(w, 1)), *const blob_owner = PyLong_AsVoidPtr(PyTuple_GET_ITEM(w, 3));
    if (PyErr_Occurred()) throw PyError();
    size_t size = 0;
    if (const int st = g_fp8_size(layer, M, &size)) raise_status(st, "svdq_fp8_workspace_size");
    if ((size_t)buf.numel() < size) Py_RETURN_NONE;
    uint8_t* const ws = (uint8_t*)buf.data_ptr() + ((size_t)buf.numel() - size);
    at::Tensor made;
    const at::Tensor* y = &made;
    if (a[6] == Py_None) {
      made = at::empty({M, N}, x.options());
    } else {
      y = &tensor("out", a[6]);
      if (y->scalar_type() != at::kBFloat16 || y->device() != device || !y->is_contiguous() || y->numel() != M * N)
        refuse("expected a contiguous bf16 output [", M, ", ", N, "] on ", device);
    }
    const c10::cuda::CUDAStream stream =
        a[7] == Py_None ? c10::cuda::getCurrentCUDAStream(device.index())
                        : c10::cuda::CUDAStream::unpack3(integer(a[8]), device.index(), c10::DeviceType::CUDA);
    if (a[7] != Py_None && (a[6] == Py_None || (void*)stream.stream() != PyLong_AsVoidPtr(a[7])))
      refuse("not a stream of ", device, " that is known by its id");
    note_use(buf, buf_owner, stream);
    note_use(blob, blob_owner, stream);
    run(device, "svdq_fp8_forward", [&] {
      return g_fp8(layer, x.data_ptr(), M, y->data_ptr(), ws, size, (void*)stream.stream());
    });
    return a[6] == Py_None ? THPVariable_Wrap(made) : Py_NewRef(a[6]);
  });
}

// bind(addresses of svdq_qk_norm_rope, svdq_cross_attn, svdq_fp8_forward and svdq_fp8_workspace_size, SvdqError,
//      attn_status, torch.OutOfMemoryError, torch.__version__).  Tensors are read by their layout in the torch that this was
// compiled against: another one is refused.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const char* torch_version = PyUnicode_AsUTF8(a[7]);
    if (!torch_version) throw PyError();
    if (std::strcmp(torch_version, SVDQ_TORCH_VERSION) != 0) {
      PyErr_Format(PyExc_RuntimeError,
                   "_marshal.so was built for torch " SVDQ_TORCH_VERSION ", this is %s: build it again with "
                   "`python -m diffusion_transformer_w4a4_b200.build`",
                   torch_version);
      throw PyError();
    }
    g_norm = (decltype(g_norm))PyLong_AsVoidPtr(a[0]);
    g_attn = (decltype(g_attn))PyLong_AsVoidPtr(a[1]);
    g_fp8 = (decltype(g_fp8))PyLong_AsVoidPtr(a[2]);
    g_fp8_size = (decltype(g_fp8_size))PyLong_AsVoidPtr(a[3]);
    if (PyErr_Occurred()) throw PyError();
    g_error = Py_NewRef(a[4]);
    g_new_status = Py_NewRef(a[5]);
    g_out_of_memory = Py_NewRef(a[6]);
    Py_RETURN_NONE;
  });
}
// set_status(device index, address of its status word)
PyObject* set_status(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    const long long i = integer(a[0]);
    if (i < 0 || i >= kDevices) refuse("device ", (int64_t)i);
    g_status[i] = (int32_t*)PyLong_AsVoidPtr(a[1]);
    if (PyErr_Occurred()) throw PyError();
    Py_RETURN_NONE;
  });
}

// current_stream(device index) -> handle
PyObject* current_stream(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    return PyLong_FromVoidPtr((void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)integer(a[0])).stream());
  });
}

PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
                         {"set_status", (PyCFunction)(void (*)())set_status, METH_FASTCALL, nullptr},
                         {"current_stream", (PyCFunction)(void (*)())current_stream, METH_FASTCALL, nullptr},
                         {"qk_norm_rope", (PyCFunction)(void (*)())qk_norm_rope, METH_FASTCALL, nullptr},
                         {"cross_attn", (PyCFunction)(void (*)())cross_attn, METH_FASTCALL, nullptr},
                         {"fp8_forward", (PyCFunction)(void (*)())fp8_forward, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  if (Py_Version >> 16 != PY_VERSION_HEX >> 16) {
    PyErr_SetString(PyExc_ImportError, "built for Python " PY_VERSION);
    return nullptr;
  }
  return PyModule_Create(&module_def);
}
