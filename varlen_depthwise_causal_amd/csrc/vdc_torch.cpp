// The recurrent layer's calls on torch tensors: checks, outputs, workspaces and the
// current stream, and then the C entry points of libvdc.so (include/vdc.h).  Module
// layer has the signatures and their documentation; this is their body, in C++
// because a single token's kernel takes less time than the same checks in Python.
// Built by _build.py into _vdc_torch.so beside libvdc.so.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>
#include <string>

#include "vdc.h"

namespace {

using at::Tensor;
using c10::Device;
using c10::ScalarType;

// What a call refuses, as the Python exception of that type.
struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }

std::string str(c10::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}
std::string name_of(ScalarType t) { return c10::toString(t); }

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// A tensor, or null for None.
const Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

void* ptr(const Tensor& t) { return t.data_ptr(); }
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// ------------------------------------------------------------------ checks --

void on_device(const Tensor& t, const char* what, Device dev) {
  if (t.device() != dev) value_error(std::string(what) + " must be a device tensor on " + dev.str());
}

// Row stride of a BF16 [S, C] activation whose rows are dense.
int64_t rows(const Tensor& t, const char* what, int64_t S, int64_t C, Device dev) {
  if (t.scalar_type() != ScalarType::BFloat16) type_error(std::string(what) + " must be bfloat16");
  if (t.dim() != 2 || t.size(0) != S || t.size(1) != C)
    value_error(std::string(what) + " must be " + str({S, C}) + ", got " + str(t.sizes()));
  on_device(t, what, dev);
  if (C != 1 && t.stride(1) != 1 && t.numel() > 0)
    value_error(std::string(what) + " must have dense rows, got strides " + str(t.strides()));
  // One row has no stride of its own, and neither has a row of a tensor without
  // elements.
  if (S <= 1 || C == 0) return C;
  if (t.stride(0) < C) value_error("the rows of " + std::string(what) + " overlap (strides " + str(t.strides()) + ")");
  return t.stride(0);
}

// Sizes, device and row stride of the activation that gives them.
struct Act {
  const Tensor& t;
  int64_t S, C, stride;
  Device dev;
  Act(PyObject* o, const char* what) : t(tensor(o, what)), S(0), C(0), stride(0), dev(t.device()) {
    if (t.dim() != 2) value_error(std::string(what) + " must be [rows, C], got " + str(t.sizes()));
    S = t.size(0);
    C = t.size(1);
    stride = rows(t, what, S, C, dev);
    if (!t.is_cuda()) value_error(std::string(what) + " must be a device tensor");
  }
};

void dense(const Tensor& t, const char* what, ScalarType type, c10::IntArrayRef shape, Device dev) {
  if (t.scalar_type() != type)
    type_error(std::string(what) + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
  if (t.sizes() != shape) value_error(std::string(what) + " must be " + str(shape) + ", got " + str(t.sizes()));
  on_device(t, what, dev);
  if (!t.is_contiguous()) value_error(std::string(what) + " must be contiguous");
}

int code_of(ScalarType t, const char* what) {
  if (t == ScalarType::Float) return VDC_F32;
  if (t == ScalarType::BFloat16) return VDC_BF16;
  type_error(std::string(what) + " must be float32 or bfloat16, got " + name_of(t));
}
// dtype code of an FP32 or BF16 parameter [C].
int param(const Tensor& t, const char* what, int64_t C, Device dev) {
  const int code = code_of(t.scalar_type(), what);
  dense(t, what, t.scalar_type(), {C}, dev);
  return code;
}

int64_t documents(const Tensor& cu, Device dev) {
  if (cu.scalar_type() != ScalarType::Int || cu.dim() != 1 || cu.numel() < 1)
    value_error("cu_seqlens must be a non-empty 1-D int32 tensor");
  dense(cu, "cu_seqlens", ScalarType::Int, cu.sizes(), dev);
  return cu.numel() - 1;
}

// A new tensor, past the dispatcher, which takes 0.25 us of a call's 4 to 10.
Tensor fresh(c10::IntArrayRef sizes, ScalarType type, Device dev) {
  return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}
Tensor fresh_as(const Tensor& t) { return fresh(t.sizes(), t.scalar_type(), t.device()); }

// The caller's output, or a new one.
Tensor output(PyObject* o, const char* what, int64_t S, int64_t C, Device dev) {
  if (o == Py_None) return fresh({S, C}, ScalarType::BFloat16, dev);
  const Tensor& t = tensor(o, what);
  dense(t, what, ScalarType::BFloat16, {S, C}, dev);
  return t;
}

struct Workspace {
  Tensor t;
  void* p = nullptr;
  size_t n = 0;
  Workspace(PyObject* o, size_t need, Device dev) {
    if (o != Py_None) {
      t = tensor(o, "workspace");
      if (t.device() != dev || !t.is_contiguous())
        value_error("workspace must be a contiguous device tensor on " + dev.str());
    } else if (need) {
      t = fresh({(int64_t)need}, ScalarType::Byte, dev);
    } else {
      return;
    }
    p = t.data_ptr();
    n = (size_t)t.numel() * t.element_size();
  }
};

hipStream_t stream_of(Device dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

// ------------------------------------------------------------------ results --

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap(const Tensor* t) {
  if (t) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}
template <class... T>
PyObject* tuple(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(T));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, wrap(t)), ...);
  return out;
}

// A status other than VDC_OK as the package's VdcError.
struct Status {
  int rc;
  const char* what;
};
void check(int rc, const char* what) {
  if (rc) throw Status{rc, what};
}

PyObject* attribute(const char* module, const char* name) {
  PyObject* m = PyImport_ImportModule(module);
  PyObject* a = m ? PyObject_GetAttrString(m, name) : nullptr;
  Py_XDECREF(m);
  return a;
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const Status& s) {
    if (PyObject* cls = attribute("varlen_depthwise_causal_amd._lib", "VdcError")) {
      PyObject* err = PyObject_CallFunction(cls, "is", s.rc, s.what);
      if (err) PyErr_SetObject(cls, err);
      Py_XDECREF(err);
      Py_DECREF(cls);
    }
  } catch (const c10::OutOfMemoryError& e) {
    if (PyObject* cls = attribute("torch", "OutOfMemoryError")) {
      PyErr_SetString(cls, e.what_without_backtrace());
      Py_DECREF(cls);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw 0;  // the error is set
  return (float)v;
}

// ---------------------------------------------- gated linear recurrence --

// (x, r, i, decay, z, scale): the arguments that the recurrence's calls share.
vdc_recurrence recurrence(const Act& x, PyObject* const* a) {
  vdc_recurrence v = {};
  const Tensor &r = tensor(a[1], "r"), &i = tensor(a[2], "i"), &decay = tensor(a[3], "decay");
  const Tensor* z = maybe(a[4], "z");
  v.S = x.S;
  v.C = x.C;
  v.x_stride = x.stride;
  v.r_stride = rows(r, "r", x.S, x.C, x.dev);
  v.i_stride = rows(i, "i", x.S, x.C, x.dev);
  v.z_stride = z ? rows(*z, "z", x.S, x.C, x.dev) : x.C;
  v.decay_dtype = param(decay, "decay", x.C, x.dev);
  v.scale = number(a[5]);
  v.x = ptr(x.t);
  v.r = ptr(r);
  v.i = ptr(i);
  v.z = ptr(z);
  v.decay = ptr(decay);
  return v;
}

// The cache and what chooses its slots.
void cache(vdc_recurrence* v, const Tensor* state, const Tensor* index, const Tensor* resume, int64_t sequences,
           Device dev) {
  if (!state) {
    if (index || resume) value_error("state_index and resume need a state");
    return;
  }
  if (state->dim() != 2) value_error("state must be [slots, " + std::to_string(v->C) + "]");
  v->slots = state->size(0);
  dense(*state, "state", ScalarType::Float, {v->slots, v->C}, dev);
  if (index) dense(*index, "state_index", ScalarType::Int, {sequences}, dev);
  else if (sequences > v->slots)
    value_error("state has " + std::to_string(v->slots) + " slots for " + std::to_string(sequences) + " sequences");
  if (resume) {
    if (resume->scalar_type() != ScalarType::Bool && resume->scalar_type() != ScalarType::Byte)
      type_error("resume must be bool or uint8, got " + name_of(resume->scalar_type()));
    dense(*resume, "resume", resume->scalar_type(), {sequences}, dev);
  }
  v->state = static_cast<float*>(ptr(state));
  v->state_index = static_cast<const int32_t*>(ptr(index));
  v->resume = static_cast<const uint8_t*>(ptr(resume));
}

// (x, r, i, decay, z, scale, cu_seqlens, state, state_index, resume, keep, out, workspace)
PyObject* recurrence_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Act x(a[0], "x");
    vdc_recurrence v = recurrence(x, a);
    const Tensor& cu = tensor(a[6], "cu_seqlens");
    v.num_docs = documents(cu, x.dev);
    v.cu_seqlens = static_cast<const int32_t*>(ptr(cu));
    const Tensor* state = maybe(a[7], "state");
    cache(&v, state, maybe(a[8], "state_index"), maybe(a[9], "resume"), v.num_docs, x.dev);
    const bool keeps = a[10] != Py_None && a[10] != Py_False;
    Tensor keep;
    if (keeps) {
      if (state) value_error("keep is for the training forward, without a state");
      const int64_t kept = gated_recurrence_keep_rows(x.S);
      if (a[10] == Py_True) {
        keep = fresh({kept, x.C}, ScalarType::Float, x.dev);
      } else {
        keep = tensor(a[10], "keep");
        dense(keep, "keep", ScalarType::Float, {kept, x.C}, x.dev);
      }
    }
    const Tensor out = output(a[11], "out", x.S, x.C, x.dev);
    const Workspace ws(a[12], gated_recurrence_workspace_bytes(VDC_FWD, x.S, x.C), x.dev);
    const c10::DeviceGuard guard(x.dev);
    check(gated_recurrence_fwd(&v, ptr(out), keeps ? static_cast<float*>(ptr(keep)) : nullptr, ws.p, ws.n,
                               stream_of(x.dev)),
          "gated_recurrence_fwd");
    return keeps ? tuple(out, keep) : wrap(out);
  });
}

// (x, r, i, decay, z, scale, cu_seqlens, dy, keep, workspace)
PyObject* recurrence_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Act x(a[0], "x");
    vdc_recurrence v = recurrence(x, a);
    const Tensor &cu = tensor(a[6], "cu_seqlens"), &dy = tensor(a[7], "dy"), &keep = tensor(a[8], "keep");
    v.num_docs = documents(cu, x.dev);
    v.cu_seqlens = static_cast<const int32_t*>(ptr(cu));
    const int64_t dys = rows(dy, "dy", x.S, x.C, x.dev);
    dense(keep, "keep", ScalarType::Float, {gated_recurrence_keep_rows(x.S), x.C}, x.dev);
    const Tensor dx = output(Py_None, "dx", x.S, x.C, x.dev), dr = fresh_as(dx), di = fresh_as(dx),
                 ddecay = fresh_as(tensor(a[3], "decay"));
    const Tensor dz = v.z || a[4] != Py_None ? fresh_as(dx) : Tensor();
    const Tensor* gate = dz.defined() ? &dz : nullptr;
    const Workspace ws(a[9], gated_recurrence_workspace_bytes(VDC_BWD, x.S, x.C), x.dev);
    const c10::DeviceGuard guard(x.dev);
    check(gated_recurrence_bwd(&v, ptr(dy), dys, static_cast<const float*>(ptr(keep)), ptr(dx), ptr(dr), ptr(di),
                               ptr(ddecay), ptr(gate), ws.p, ws.n, stream_of(x.dev)),
          "gated_recurrence_bwd");
    return tuple(dx, dr, di, ddecay, gate);
  });
}

// (x, r, i, decay, z, scale, state, state_index, out)
PyObject* recurrence_update(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    if (a[6] == Py_None) value_error("gated_recurrence_update needs a state");
    const Act x(a[0], "x");
    vdc_recurrence v = recurrence(x, a);
    cache(&v, &tensor(a[6], "state"), maybe(a[7], "state_index"), nullptr, x.S, x.dev);
    const Tensor out = output(a[8], "out", x.S, x.C, x.dev);
    const c10::DeviceGuard guard(x.dev);
    check(gated_recurrence_update(&v, ptr(out), stream_of(x.dev)), "gated_recurrence_update");
    return wrap(out);
  });
}

// ------------------------------------------------------------ layer norm --

// (x, weight, bias, residual, eps, out, stream_out)
PyObject* norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Act x(a[0], "x");
    const Tensor& w = tensor(a[1], "weight");
    const Tensor *b = maybe(a[2], "bias"), *res = maybe(a[3], "residual");
    const int wd = param(w, "weight", x.C, x.dev), bd = b ? param(*b, "bias", x.C, x.dev) : 0;
    const float eps = number(a[4]);
    const int64_t rs = res ? rows(*res, "residual", x.S, x.C, x.dev) : x.C;
    if (!res && a[6] != Py_None) value_error("stream_out needs a residual");
    const Tensor out = output(a[5], "out", x.S, x.C, x.dev);
    const Tensor sum = res ? output(a[6], "stream_out", x.S, x.C, x.dev) : x.t;
    const c10::DeviceGuard guard(x.dev);
    check(layer_norm_fwd(ptr(x.t), x.stride, ptr(res), rs, ptr(w), wd, ptr(b), bd, x.S, x.C, eps, ptr(out),
                         res ? ptr(sum) : nullptr, stream_of(x.dev)),
          "layer_norm_fwd");
    return tuple(out, sum);
  });
}

// (s, weight, dy, bias, dstream, eps, workspace)
PyObject* norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const Act s(a[0], "s");
    const Tensor &w = tensor(a[1], "weight"), &dy = tensor(a[2], "dy");
    const Tensor *b = maybe(a[3], "bias"), *ds = maybe(a[4], "dstream");
    const int64_t dys = rows(dy, "dy", s.S, s.C, s.dev), dss = ds ? rows(*ds, "dstream", s.S, s.C, s.dev) : s.C;
    const int wd = param(w, "weight", s.C, s.dev), bd = b ? param(*b, "bias", s.C, s.dev) : 0;
    const float eps = number(a[5]);
    const Tensor dx = output(Py_None, "dx", s.S, s.C, s.dev), dw = fresh_as(w), db = b ? fresh_as(*b) : Tensor();
    const Tensor* dbias = b ? &db : nullptr;
    const Workspace ws(a[6], layer_norm_workspace_bytes(s.S, s.C), s.dev);
    const c10::DeviceGuard guard(s.dev);
    check(layer_norm_bwd(ptr(s.t), s.stride, ptr(w), wd, ptr(dy), dys, ptr(ds), dss, s.S, s.C, eps, ptr(dx), ptr(dw),
                         ptr(dbias), bd, ws.p, ws.n, stream_of(s.dev)),
          "layer_norm_bwd");
    return tuple(dx, dw, dbias);
  });
}

// ------------------------------------------------------ states put aside --

// (state, codes, scales, state_index, pool_index)
PyObject* pool(PyObject* const* a, Py_ssize_t n, bool back) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Tensor &state = tensor(a[0], "state"), &codes = tensor(a[1], "codes"), &scales = tensor(a[2], "scales");
    const Tensor *si = maybe(a[3], "state_index"), *pi = maybe(a[4], "pool_index");
    const int dtype = code_of(state.scalar_type(), "state");
    if (!state.is_cuda()) value_error("state must be a device tensor");
    if (state.dim() < 2 || !state.is_contiguous()) value_error("state must be a contiguous [slots, ...] cache");
    const Device dev = state.device();
    const int64_t slots = state.size(0);
    int64_t E = 1;
    for (int64_t d = 1; d < state.dim(); ++d) E *= state.size(d);
    const ScalarType type = codes.scalar_type();
    if (type != ScalarType::Char && type != ScalarType::Float8_e4m3fn)
      type_error("codes must be int8 or float8_e4m3fn, got " + name_of(type));
    if (codes.dim() != 2 || codes.size(1) != E)
      value_error("codes must be [pool, " + std::to_string(E) + "], got " + str(codes.sizes()));
    const int64_t places = codes.size(0);
    dense(codes, "codes", type, {places, E}, dev);
    dense(scales, "scales", ScalarType::Float, {places, (E + 63) / 64}, dev);
    const int64_t count = si ? si->numel() : pi ? pi->numel() : slots;
    if (si) dense(*si, "state_index", ScalarType::Int, {count}, dev);
    if (pi) dense(*pi, "pool_index", ScalarType::Int, {count}, dev);
    if ((!si && count > slots) || (!pi && count > places))
      value_error(std::to_string(count) + " states do not fit " + std::to_string(slots) + " slots and " +
                  std::to_string(places) + " places");
    const int code = type == ScalarType::Char ? VDC_INT8 : VDC_E4M3;
    const int32_t *slot = static_cast<const int32_t*>(ptr(si)), *place = static_cast<const int32_t*>(ptr(pi));
    float* s = static_cast<float*>(ptr(scales));
    const c10::DeviceGuard guard(dev);
    if (back)
      check(state_dequantize(ptr(codes), code, s, places, place, ptr(state), dtype, slots, E, slot, count,
                             stream_of(dev)),
            "state_dequantize");
    else
      check(state_quantize(ptr(state), dtype, slots, E, slot, ptr(codes), code, s, places, place, count,
                           stream_of(dev)),
            "state_quantize");
    Py_RETURN_NONE;
  });
}
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return pool(a, n, false); }
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return pool(a, n, true); }

#define VDC_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {VDC_METHOD(recurrence_fwd), VDC_METHOD(recurrence_bwd), VDC_METHOD(recurrence_update),
                         VDC_METHOD(norm_fwd),       VDC_METHOD(norm_bwd),       VDC_METHOD(quantize),
                         VDC_METHOD(dequantize),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vdc_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vdc_torch() { return PyModule_Create(&module); }
