// _rcx_torch: marshalling of the calls that a decoding step makes (rotation by
// several axes, block-scaled KV cache, attention over it) from torch tensors to
// the C ABI of librcx.so.  These kernels run for a few microseconds, so the
// call is kept shorter than they are: views, device and stream are read here in
// about a microsecond, where the ctypes binding spends six (a decoding step's
// attention: 14.4 us a call through ctypes, of which 4.9 in the C call).
//
// Each function checks what the C ABI cannot see (types, devices, dimensions of
// torch tensors) and raises TypeError or ValueError; the C call's status is
// returned for the Python side to raise.
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/rcx.h"

namespace {

// Thrown after the Python error is set.
struct PyError {};

[[noreturn]] void value_error(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  throw PyError();
}

const at::Tensor* tensor(PyObject* x, const char* name, bool optional = false) {
  if (optional && x == Py_None) return nullptr;
  if (!THPVariable_Check(x)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch tensor", name);
    throw PyError();
  }
  return &THPVariable_Unpack(x);
}

long long integer(PyObject* x) {
  const long long v = PyLong_AsLongLong(x);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return v;
}

// Before a call writes t behind autograd's back: refuses what torch's own in-place
// operations refuse, a tensor that gradients are wanted of.
void check_output(const at::Tensor* t, const char* name) {
  if (t && t->requires_grad() && at::GradMode::is_enabled()) {
    PyErr_Format(PyExc_ValueError, "%s would be written in place, but it requires grad: pass another output, or call under "
                                   "torch.no_grad()", name);
    throw PyError();
  }
}

// After the write: autograd then sees that what it saved has changed.
void written(const at::Tensor* t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

rcx_tensor null_view() {
  rcx_tensor t = {};
  return t;
}

rcx_tensor view4(const at::Tensor& t) {
  rcx_tensor r = {};
  if (t.layout() != at::kStrided) value_error("expected a strided tensor");
  switch (t.scalar_type()) {
    case at::kFloat: r.dtype = RCX_F32; break;
    case at::kBFloat16: r.dtype = RCX_BF16; break;
    case at::kChar: r.dtype = RCX_I8; break;
    case at::kFloat8_e4m3fn: r.dtype = RCX_E4M3; break;
    default:
      PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
      throw PyError();
  }
  if (t.dim() != 4) value_error("expected a 4-D [B, N, H, d] tensor");
  r.ptr = t.data_ptr();
  for (int i = 0; i < 4; ++i) {
    r.shape[i] = t.size(i);
    r.stride[i] = t.stride(i);
  }
  return r;
}

rcx_tensor lse_view(const at::Tensor& t) {
  if (t.dim() != 3 || t.scalar_type() != at::kFloat) value_error("expected a 3-D [B, H, N] float32 tensor");
  rcx_tensor r = {};
  r.ptr = t.data_ptr();
  r.dtype = RCX_F32;
  for (int i = 0; i < 3; ++i) {
    r.shape[i] = t.size(i);
    r.stride[i] = t.stride(i);
  }
  r.shape[3] = r.stride[3] = 1;
  return r;
}

// The CUDA device of all tensors of a call.
struct OneDevice {
  int index = -1;
  void add(const at::Tensor* t) {
    if (!t) return;
    if (!t->is_cuda()) {
      PyErr_Format(PyExc_ValueError, "expected CUDA tensors, got one on %s", t->device().str().c_str());
      throw PyError();
    }
    const int i = t->get_device();
    if (index < 0) index = i;
    if (i != index) {
      PyErr_Format(PyExc_ValueError, "tensors on different devices: cuda:%d and cuda:%d", index, i);
      throw PyError();
    }
  }
};

const int64_t* per_sequence(PyObject* x, const char* name, int64_t B, OneDevice& dev) {
  const at::Tensor* t = tensor(x, name, true);
  if (!t) return nullptr;
  if (t->scalar_type() != at::kLong || t->dim() != 1 || t->size(0) != B || (B > 1 && t->stride(0) != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous int64 [%lld] tensor", name, (long long)B);
    throw PyError();
  }
  dev.add(t);
  return t->data_ptr<int64_t>();
}

// Makes the device current for the call; the stream is torch's current one there.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit OnDevice(int index) {
    guard.set_index((c10::DeviceIndex)index);
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
  }
};

const rcx_kv_blocks* blocks(PyObject* address) {
  return reinterpret_cast<const rcx_kv_blocks*>((uintptr_t)integer(address));
}

// C++ exceptions (an allocation that fails) and PyError end at the boundary.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const PyError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

struct Buffer {                       // a contiguous host buffer, released with the scope
  Py_buffer b;
  explicit Buffer(PyObject* x) {
    if (PyObject_GetBuffer(x, &b, PyBUF_C_CONTIGUOUS)) throw PyError();
  }
  ~Buffer() { PyBuffer_Release(&b); }
};

// (q, k, q_out, k_out, inv_freq float64 [d/2], axis int32 [d/2], positions, flags) -> status
PyObject* rope_axes_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor *q = tensor(a[0], "q", true), *k = tensor(a[1], "k", true);
    const at::Tensor *qo = tensor(a[2], "q_out", true), *ko = tensor(a[3], "k_out", true);
    const at::Tensor* pos = tensor(a[6], "positions");
    const at::Tensor* ref = q ? q : k;
    if (!ref || (q && !qo) || (k && !ko)) value_error("an operand or its output is missing");
    const rcx_tensor tq = q ? view4(*q) : null_view(), tk = k ? view4(*k) : null_view();
    const int64_t B = ref->size(0), N = ref->size(1), d = ref->size(3);
    if (pos->scalar_type() != at::kLong || pos->dim() != 3 || pos->size(1) != B || pos->size(2) != N) {
      PyErr_Format(PyExc_ValueError, "positions must be an int64 [axes, %lld, %lld] tensor", (long long)B, (long long)N);
      throw PyError();
    }
    if (N > 1 && pos->stride(2) != 1) value_error("positions must have unit stride over tokens");
    const Buffer inv(a[4]), axis(a[5]);
    if (inv.b.len != d / 2 * 8 || axis.b.len != d / 2 * 4) value_error("inv_freq and axis need d/2 entries");
    OneDevice dev;
    dev.add(ref);
    dev.add(k);
    dev.add(pos);
    if (q) dev.add(qo);
    if (k) dev.add(ko);
    const rcx_tensor tqo = q ? view4(*qo) : null_view(), tko = k ? view4(*ko) : null_view();
    const long long flags = integer(a[7]);
    check_output(q ? qo : nullptr, "q_out");
    check_output(k ? ko : nullptr, "k_out");
    OnDevice on(dev.index);
    const int st = rcx_rope_axes_apply(
        tq, tk, tqo, tko, pos->data_ptr<int64_t>(), (int)std::min<int64_t>(pos->size(0), 1 << 20), pos->stride(0),
        pos->stride(1), static_cast<const double*>(inv.b.buf), static_cast<const int32_t*>(axis.b.buf), (int)flags,
        on.stream);
    if (st == RCX_OK) {
      written(q ? qo : nullptr);
      written(k ? ko : nullptr);
    }
    return PyLong_FromLong(st);
  });
}

// (k, v, pool, address, start, count) -> status
PyObject* kv_block_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor *k = tensor(a[0], "k"), *v = tensor(a[1], "v");
    OneDevice dev;
    dev.add(tensor(a[2], "pool"));
    dev.add(k);
    dev.add(v);
    const rcx_tensor tk = view4(*k), tv = view4(*v);
    const int64_t* start = per_sequence(a[4], "start", k->size(0), dev);
    const int64_t* count = per_sequence(a[5], "count", k->size(0), dev);
    OnDevice on(dev.index);
    return PyLong_FromLong(rcx_kv_block_append(tk, tv, blocks(a[3]), start, count, on.stream));
  });
}

// (pool, address, B, lengths, n, k_out, v_out, bf16) -> (status, k_out, v_out); outputs that are None are made
PyObject* kv_block_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor* pool = tensor(a[0], "pool");
    const int64_t B = integer(a[2]), len = integer(a[4]);
    if (len < 0) value_error("n must not be negative");
    OneDevice dev;
    dev.add(pool);
    at::Tensor out[2];
    for (int i = 0; i < 2; ++i) {
      const at::Tensor* given = tensor(a[5 + i], "output", true);
      if (given) {
        dev.add(given);
        check_output(given, i ? "v_out" : "k_out");
        out[i] = *given;
      } else {
        out[i] = at::empty({B, len, pool->size(2), pool->size(3)},
                           pool->options().dtype(integer(a[7]) ? at::kBFloat16 : at::kFloat));
      }
      if (out[i].dim() != 4 || out[i].size(1) != len) value_error("outputs must hold n tokens: [B, n, Hkv, d]");
    }
    const int64_t* lengths = per_sequence(a[3], "lengths", B, dev);
    OnDevice on(dev.index);
    const int st = rcx_kv_block_read(blocks(a[1]), lengths, view4(out[0]), view4(out[1]), on.stream);
    for (int i = 0; i < 2; ++i)
      if (st == RCX_OK && a[5 + i] != Py_None) written(&out[i]);
    return Py_BuildValue("iNN", st, THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
  });
}

// (q, pool, address, start, count, o, lse, window, n_sink, temperature, workspace, want_lse)
// -> (status, o, lse); o, lse and workspace that are None are made
PyObject* attn_kv_block_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor *q = tensor(a[0], "q"), *o_in = tensor(a[5], "o", true), *lse_in = tensor(a[6], "lse", true);
    const at::Tensor* ws_in = tensor(a[10], "workspace", true);
    OneDevice dev;
    dev.add(tensor(a[1], "pool"));
    dev.add(q);
    dev.add(o_in);
    dev.add(lse_in);
    dev.add(ws_in);
    const rcx_tensor tq = view4(*q);
    const rcx_kv_blocks* cache = blocks(a[2]);
    const int64_t* start = per_sequence(a[3], "start", q->size(0), dev);
    const int64_t* count = per_sequence(a[4], "count", q->size(0), dev);
    const long long window = integer(a[7]), n_sink = integer(a[8]);
    const double t = PyFloat_AsDouble(a[9]);
    if (t == -1.0 && PyErr_Occurred()) throw PyError();
    const int want_lse = PyObject_IsTrue(a[11]);
    if (want_lse < 0) throw PyError();
    check_output(o_in, "o");
    check_output(lse_in, "lse");
    OnDevice on(dev.index);
    const at::Tensor o = o_in ? *o_in : at::empty(q->sizes(), q->options());
    at::Tensor lse, ws;
    if (lse_in) lse = *lse_in;
    else if (want_lse) lse = at::empty({q->size(0), q->size(2), q->size(1)}, q->options().dtype(at::kFloat));
    if (ws_in) {
      ws = *ws_in;
      if (!ws.is_contiguous()) value_error("workspace must be contiguous");
    } else {
      const int64_t need = rcx_attn_kv_block_workspace_size(tq, cache);
      ws = at::empty({std::max<int64_t>(need, 256)}, q->options().dtype(at::kByte));
    }
    const int st = rcx_attn_kv_block_fwd(tq, cache, start, count, view4(o), lse.defined() ? lse_view(lse) : null_view(),
                                         window, n_sink, t, ws.data_ptr(), (int64_t)ws.nbytes(), on.stream);
    if (st == RCX_OK) {
      written(o_in);
      written(lse_in);
    }
    PyObject* l = lse.defined() ? THPVariable_Wrap(lse) : Py_NewRef(Py_None);
    return Py_BuildValue("iNN", st, THPVariable_Wrap(o), l);
  });
}

#define RCX_METHOD(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RCX_METHOD(rope_axes_apply), RCX_METHOD(kv_block_append), RCX_METHOD(kv_block_read),
                         RCX_METHOD(attn_kv_block_fwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rcx_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rcx_torch(void) { return PyModule_Create(&module); }
