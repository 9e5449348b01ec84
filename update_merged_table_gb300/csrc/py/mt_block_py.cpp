// The dense block's calls for Python (block.py): argument checks, output
// tensors and the call of the C ABI, in one step of native code.
//
// A call on a few rows (a token being served) takes a few microseconds on the
// GPU; checked and marshalled from Python it cost 12 to 34 us of host time on
// the Grace CPU, here 4 to 7.  Nothing is computed here: the functions of
// libmt.so arrive as addresses (init), and tensors are read and made with
// torch's own C++ interface.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>
#include <string>

#include "mt.h"

namespace {

decltype(&mt_pack8) f_pack8;
decltype(&mt_unpack8) f_unpack8;
decltype(&mt_group_linear_forward) f_linear_forward;
decltype(&mt_group_linear_backward) f_linear_backward;
decltype(&mt_gated_norm_forward) f_norm_forward;
decltype(&mt_gated_norm_backward) f_norm_backward;
PyObject* g_mt_error;       // the MTError class
PyObject* g_out_of_memory;  // torch's

// Thrown where a Python error has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}

void check(int rc, const char* what) {
  if (rc == MT_OK) return;
  PyObject* e = PyObject_CallFunction(g_mt_error, "is", rc, what);
  if (e != nullptr) {
    PyErr_SetObject(g_mt_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(what) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

at::ScalarType type_of(int dtype) { return dtype == MT_F32 ? at::kFloat : at::kBFloat16; }

std::string shape(int64_t n, int64_t d) {
  return "[" + (n < 0 ? std::string("n") : std::to_string(n)) + ", " + std::to_string(d) + "]";
}

// A row tensor [n, d] (n = -1: any number of rows, returned) of this type on this device: columns contiguous, rows not
// overlapping.
mt_rows rows(PyObject* o, const char* what, int64_t& n, int64_t d, at::ScalarType type, int device) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 2) raise(PyExc_ValueError, std::string(what) + " must be a 2-D CUDA tensor");
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, std::string(what) + " must be " + (type == at::kFloat ? "float32" : "bfloat16"));
  if (!t.is_cuda() || t.device().index() != device)
    raise(PyExc_ValueError, std::string(what) + " is on " + t.device().str() + ", not on cuda:" + std::to_string(device));
  if ((n >= 0 && t.size(0) != n) || t.size(1) != d)
    raise(PyExc_ValueError, std::string(what) + " must be " + shape(n, d) + ", not " + shape(t.size(0), t.size(1)));
  n = t.size(0);
  int64_t ld = t.stride(0);
  if (d > 1 && t.stride(1) != 1) raise(PyExc_ValueError, std::string("the columns of ") + what + " must be contiguous");
  if (n <= 1) ld = d;  // there is no next row
  else if (ld < d) raise(PyExc_ValueError, std::string("the rows of ") + what + " overlap");
  return mt_rows{t.data_ptr(), ld, nullptr, nullptr};
}

mt_rows none_rows() { return mt_rows{nullptr, 0, nullptr, nullptr}; }

// A contiguous tensor of this type and shape on this device (d1 < 0: one dimension).
void* whole(PyObject* o, const char* what, at::ScalarType type, int device, int64_t d0, int64_t d1, int64_t d2 = -1) {
  const at::Tensor& t = tensor(o, what);
  const int64_t dims = d1 < 0 ? 1 : d2 < 0 ? 2 : 3;
  const bool fits = t.dim() == dims && t.size(0) == d0 && (dims < 2 || t.size(1) == d1) && (dims < 3 || t.size(2) == d2);
  if (!fits || t.scalar_type() != type || !t.is_cuda() || t.device().index() != device || !t.is_contiguous()) {
    std::string s = "[" + std::to_string(d0) + (d1 < 0 ? "" : ", " + std::to_string(d1)) + (d2 < 0 ? "" : ", " + std::to_string(d2)) + "]";
    raise(PyExc_ValueError, std::string(what) + " must be a contiguous " + c10::toString(type) + " CUDA tensor " + s +
                                " on cuda:" + std::to_string(device));
  }
  return t.data_ptr();
}

const int64_t* offsets_of(PyObject* o, int64_t groups, int device) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).scalar_type() != at::kLong)
    raise(PyExc_TypeError, "offsets must be a contiguous int64 CUDA tensor [" + std::to_string(groups + 1) + "]");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.dim() != 1 || t.size(0) != groups + 1 || !t.is_cuda() || t.device().index() != device || !t.is_contiguous())
    raise(PyExc_TypeError, "offsets must be a contiguous int64 CUDA tensor [" + std::to_string(groups + 1) + "] on cuda:" +
                               std::to_string(device));
  return static_cast<const int64_t*>(t.data_ptr());
}

at::Tensor make(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)device)));
}
at::Tensor make_codes(int64_t n, int64_t d, int device) { return make({n, d}, at::kChar, device); }
at::Tensor make_exps(int64_t n, int64_t d, int device) {
  return make({n, (d + MT_PACK_BLOCK - 1) / MT_PACK_BLOCK}, at::kByte, device);
}

// The device made current, and its current stream.
struct On {
  explicit On(int device) : guard((c10::DeviceIndex)device), stream(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream()) {}
  c10::cuda::CUDAGuard guard;
  void* stream;
};

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* wrap_or_none(const std::optional<at::Tensor>& t) {
  if (t.has_value()) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", got, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
    return nullptr;
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// Both parts of a checkpoint of rows [n, d].
mt_rows saved_parts(PyObject* codes, PyObject* exps, const char* what, int64_t n, int64_t d, int device) {
  mt_rows r = none_rows();
  r.codes = static_cast<int8_t*>(whole(codes, what, at::kChar, device, n, d));
  r.exps = static_cast<uint8_t*>(whole(exps, what, at::kByte, device, n, (d + MT_PACK_BLOCK - 1) / MT_PACK_BLOCK));
  return r;
}
// The saved rows of a backward: plain, or (codes, exps).
mt_rows saved(PyObject* o, const char* what, int64_t& n, int64_t d, at::ScalarType type, int device) {
  if (o == Py_None) return none_rows();
  if (!PyTuple_Check(o)) return rows(o, what, n, d, type, device);
  return saved_parts(PyTuple_GET_ITEM(o, 0), PyTuple_GET_ITEM(o, 1), what, n, d, device);
}

// init(addresses of the six functions in order, MTError, torch.OutOfMemoryError)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    f_pack8 = reinterpret_cast<decltype(f_pack8)>(integer(a[0]));
    f_unpack8 = reinterpret_cast<decltype(f_unpack8)>(integer(a[1]));
    f_linear_forward = reinterpret_cast<decltype(f_linear_forward)>(integer(a[2]));
    f_linear_backward = reinterpret_cast<decltype(f_linear_backward)>(integer(a[3]));
    f_norm_forward = reinterpret_cast<decltype(f_norm_forward)>(integer(a[4]));
    f_norm_backward = reinterpret_cast<decltype(f_norm_backward)>(integer(a[5]));
    Py_INCREF(a[6]);
    g_mt_error = a[6];
    Py_INCREF(a[7]);
    g_out_of_memory = a[7];
    Py_RETURN_NONE;
  });
}

// pack8(x, codes or None, exps or None) -> (codes, exps)
PyObject* pack8(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 3, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    if (x.dim() != 2 || !x.is_cuda()) raise(PyExc_ValueError, "x must be a 2-D CUDA tensor");
    if (x.scalar_type() != at::kFloat && x.scalar_type() != at::kBFloat16)
      raise(PyExc_TypeError, "rows must be float32 or bfloat16");
    const int device = x.device().index();
    int64_t n = -1;
    const int64_t d = x.size(1);
    if (d < 1 || d > MT_MAX_BLOCK_DIM) raise(PyExc_ValueError, "x must have 1 to 8192 columns");
    const mt_rows r = rows(a[0], "x", n, d, x.scalar_type(), device);
    On on(device);
    at::Tensor codes, exps;
    if (a[1] != Py_None) {
      const int64_t nb = (d + MT_PACK_BLOCK - 1) / MT_PACK_BLOCK;
      whole(a[1], "out", at::kChar, device, n, d);
      whole(a[2], "out", at::kByte, device, n, nb);
      codes = THPVariable_Unpack(a[1]);
      exps = THPVariable_Unpack(a[2]);
    } else {
      codes = make_codes(n, d, device);
      exps = make_exps(n, d, device);
    }
    check(f_pack8(r.data, r.ld, n, (int32_t)d, x.scalar_type() == at::kFloat ? MT_F32 : MT_BF16,
                  static_cast<int8_t*>(codes.data_ptr()), static_cast<uint8_t*>(exps.data_ptr()), on.stream),
          "mt_pack8");
    return Py_BuildValue("(NN)", wrap(codes), wrap(exps));
  });
}

// unpack8(codes, exps, dtype code, out or None) -> rows
PyObject* unpack8(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 4, [&]() -> PyObject* {
    const at::Tensor& codes = tensor(a[0], "p");
    if (codes.dim() != 2 || !codes.is_cuda()) raise(PyExc_ValueError, "the codes of p must be a 2-D CUDA tensor");
    const int device = codes.device().index();
    int64_t n = codes.size(0);
    const int64_t d = codes.size(1);
    if (d < 1 || d > MT_MAX_BLOCK_DIM) raise(PyExc_ValueError, "p must have 1 to 8192 columns");
    const mt_rows p = saved_parts(a[0], a[1], "p", n, d, device);
    const int dtype = (int)integer(a[2]);
    On on(device);
    mt_rows r;
    at::Tensor out;
    if (a[3] != Py_None) {
      r = rows(a[3], "out", n, d, type_of(dtype), device);
      out = THPVariable_Unpack(a[3]);
    } else {
      out = make({n, d}, type_of(dtype), device);
      r = mt_rows{out.data_ptr(), d, nullptr, nullptr};
    }
    check(f_unpack8(p.codes, p.exps, n, (int32_t)d, dtype, r.data, r.ld, on.stream), "mt_unpack8");
    return wrap(out);
  });
}

// linear_forward(groups, in, out, dtype, device, status, x, w, offsets, y or None) -> y
PyObject* linear_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 10, [&]() -> PyObject* {
    const int64_t groups = integer(a[0]), k = integer(a[1]), m = integer(a[2]);
    const int dtype = (int)integer(a[3]), device = (int)integer(a[4]);
    const at::ScalarType type = type_of(dtype);
    int64_t n = -1;
    const mt_rows x = rows(a[6], "x", n, k, type, device);
    const void* w = whole(a[7], "weight", type, device, groups, m, k);
    const int64_t* off = offsets_of(a[8], groups, device);
    On on(device);
    at::Tensor y;
    mt_rows r;
    if (a[9] != Py_None) {
      r = rows(a[9], "out", n, m, type, device);
      y = THPVariable_Unpack(a[9]);
    } else {
      y = make({n, m}, type, device);
      r = mt_rows{y.data_ptr(), m, nullptr, nullptr};
    }
    check(f_linear_forward(x.data, x.ld, w, off, (int32_t)groups, n, (int32_t)k, (int32_t)m, dtype, r.data, r.ld,
                           reinterpret_cast<int32_t*>(integer(a[5])), on.stream),
          "mt_group_linear_forward");
    return wrap(y);
  });
}

// linear_backward(groups, in, out, dtype, device, status, dy, x or (codes, exps) or None, w or None, offsets, dx or None,
// dw or None, want_dx, want_dw, ws or None) -> (dx, dw)
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 15, [&]() -> PyObject* {
    const int64_t groups = integer(a[0]), k = integer(a[1]), m = integer(a[2]);
    const int dtype = (int)integer(a[3]), device = (int)integer(a[4]);
    const at::ScalarType type = type_of(dtype);
    const bool want_dx = integer(a[12]) != 0, want_dw = integer(a[13]) != 0;
    int64_t n = -1;
    const mt_rows dy = rows(a[6], "dy", n, m, type, device);
    if (want_dw && a[7] == Py_None) raise(PyExc_TypeError, "x must be a CUDA tensor or a Packed8");
    const mt_rows x = want_dw ? saved(a[7], "x", n, k, type, device) : none_rows();
    const void* w = want_dx ? whole(a[8], "weight", type, device, groups, m, k) : nullptr;
    const int64_t* off = offsets_of(a[9], groups, device);
    On on(device);
    std::optional<at::Tensor> dx, dw;
    mt_rows rdx = none_rows();
    float* pdw = nullptr;
    if (want_dx) {
      if (a[10] != Py_None) {
        rdx = rows(a[10], "out_dx", n, k, type, device);
        dx = THPVariable_Unpack(a[10]);
      } else {
        dx = make({n, k}, type, device);
        rdx = mt_rows{dx->data_ptr(), k, nullptr, nullptr};
      }
    }
    if (want_dw) {
      if (a[11] != Py_None) {
        pdw = static_cast<float*>(whole(a[11], "out_dw", at::kFloat, device, groups, m, k));
        dw = THPVariable_Unpack(a[11]);
      } else {
        dw = make({groups, m, k}, at::kFloat, device);
        pdw = static_cast<float*>(dw->data_ptr());
      }
    }
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (want_dw) {
      const at::Tensor& t = tensor(a[14], "the workspace");
      ws = t.data_ptr();
      ws_bytes = (size_t)t.numel();
    }
    // an empty batch has no dx rows to point at: only dw is asked for
    if (n > 0 || want_dw)
      check(f_linear_backward(dy.data, dy.ld, want_dw ? &x : nullptr, w, off, (int32_t)groups, n, (int32_t)k, (int32_t)m, dtype,
                              n > 0 ? rdx.data : nullptr, rdx.ld, pdw, reinterpret_cast<int32_t*>(integer(a[5])), ws, ws_bytes,
                              on.stream),
            "mt_group_linear_backward");
    return Py_BuildValue("(NN)", wrap_or_none(dx), wrap_or_none(dw));
  });
}

// groups, dim, dtype, kind, gate, eps, device, status, post_weight, post_bias, scale, pre_weight, pre_bias, offsets
constexpr int kNormArgs = 14;
mt_gated_norm norm_config(PyObject* const* a) {
  mt_gated_norm c{};
  c.groups = (int32_t)integer(a[0]);
  c.dim = (int32_t)integer(a[1]);
  c.dtype = (int32_t)integer(a[2]);
  c.kind = (int32_t)integer(a[3]);
  c.gate = (int32_t)integer(a[4]);
  c.eps = (float)PyFloat_AsDouble(a[5]);
  const int device = (int)integer(a[6]);
  c.status = reinterpret_cast<int32_t*>(integer(a[7]));
  static const char* const names[] = {"post_weight", "post_bias", "scale", "pre_weight", "pre_bias"};
  const float** const to[] = {&c.post_weight, &c.post_bias, &c.scale, &c.pre_weight, &c.pre_bias};
  for (int i = 0; i < 5; ++i) {
    PyObject* o = a[8 + i];
    if (o == Py_None) continue;
    const bool flat = c.groups == 1 && THPVariable_Check(o) && THPVariable_Unpack(o).dim() == 1;
    *to[i] = static_cast<const float*>(flat ? whole(o, names[i], at::kFloat, device, c.dim, -1)
                                            : whole(o, names[i], at::kFloat, device, c.groups, c.dim));
  }
  if (a[13] != Py_None) c.offsets = offsets_of(a[13], c.groups, device);
  else if (c.groups != 1) raise(PyExc_ValueError, "several groups need offsets");
  return c;
}

// An output row tensor: the caller's, or a new one.
mt_rows output(PyObject* given, const char* what, int64_t& n, int64_t d, at::ScalarType type, int device,
               std::optional<at::Tensor>& t) {
  if (given != Py_None) {
    const mt_rows r = rows(given, what, n, d, type, device);
    t = THPVariable_Unpack(given);
    return r;
  }
  t = make({n, d}, type, device);
  return mt_rows{t->data_ptr(), d, nullptr, nullptr};
}

// norm_forward(config..., x, y or None, u or None, z or None, h or None, pack bits y u z h)
//   -> (z or None without y, h or None, codes and exps of the checkpoints asked for ...)
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, kNormArgs + 6, [&]() -> PyObject* {
    mt_gated_norm c = norm_config(a);
    const int device = (int)integer(a[6]);
    const at::ScalarType type = type_of(c.dtype);
    PyObject* const* b = a + kNormArgs;
    int64_t n = -1;
    const mt_rows x = rows(b[0], "x", n, c.dim, type, device);
    mt_rows r[4];  // y, u, z, h
    const bool has_y = b[1] != Py_None, has_h = c.pre_weight != nullptr;
    r[0] = has_y ? rows(b[1], "y", n, c.dim, type, device) : none_rows();
    r[1] = b[2] != Py_None ? rows(b[2], "u", n, c.dim, type, device) : none_rows();
    r[2] = r[3] = none_rows();
    c.n = n;
    if (!has_y) c.gate = MT_GATE_NONE;
    On on(device);
    std::optional<at::Tensor> z, h;
    if (has_y) r[2] = output(b[3], "out_z", n, c.dim, type, device, z);
    if (has_h) r[3] = output(b[4], "out_h", n, c.dim, type, device, h);
    const int pack = (int)integer(b[5]);
    at::Tensor packed[8];
    int made = 0;
    for (int i = 0; i < 4; ++i) {
      if (!(pack >> i & 1)) continue;
      packed[made] = make_codes(n, c.dim, device);
      packed[made + 1] = make_exps(n, c.dim, device);
      r[i].codes = static_cast<int8_t*>(packed[made].data_ptr());
      r[i].exps = static_cast<uint8_t*>(packed[made + 1].data_ptr());
      made += 2;
    }
    if (n > 0) check(f_norm_forward(&c, &x, &r[0], &r[1], &r[2], &r[3], on.stream), "mt_gated_norm_forward");
    PyObject* out = PyTuple_New(2 + made);
    if (out == nullptr) throw Raised{};
    PyTuple_SET_ITEM(out, 0, wrap_or_none(z));
    PyTuple_SET_ITEM(out, 1, wrap_or_none(h));
    for (int i = 0; i < made; ++i) PyTuple_SET_ITEM(out, 2 + i, wrap(packed[i]));
    return out;
  });
}

// norm_backward(config..., dz or None, dh or None, y, u, z (each rows, (codes, exps) or None), dx, dy, du (each or None), ws)
//   -> (dx, dy or None, du or None, gradient or None for each of the five parameters)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, kNormArgs + 9, [&]() -> PyObject* {
    mt_gated_norm c = norm_config(a);
    const int device = (int)integer(a[6]);
    const at::ScalarType type = type_of(c.dtype);
    PyObject* const* b = a + kNormArgs;
    int64_t n = -1;
    // the first of dh and dz that is there says how many rows there are
    const mt_rows dh = b[1] != Py_None ? rows(b[1], "dh", n, c.dim, type, device) : none_rows();
    const mt_rows dz = b[0] != Py_None ? rows(b[0], "dz", n, c.dim, type, device) : none_rows();
    const mt_rows y = saved(b[2], "y", n, c.dim, type, device), u = saved(b[3], "u", n, c.dim, type, device);
    const mt_rows z = c.pre_weight != nullptr ? saved(b[4], "z", n, c.dim, type, device) : none_rows();
    const bool has_y = b[2] != Py_None, has_u = b[3] != Py_None;
    c.n = n;
    if (!has_y) c.gate = MT_GATE_NONE;
    On on(device);
    std::optional<at::Tensor> dx, dy, du;
    const mt_rows rdx = output(b[5], "out_dx", n, c.dim, type, device, dx);
    const mt_rows rdy = has_y ? output(b[6], "out_dy", n, c.dim, type, device, dy) : none_rows();
    const mt_rows rdu = has_u ? output(b[7], "out_du", n, c.dim, type, device, du) : none_rows();
    const float* const there[] = {c.post_weight, c.post_bias, c.scale, c.pre_weight, c.pre_bias};
    float* grads[5] = {};
    std::optional<at::Tensor> sums[5];
    for (int i = 0; i < 5; ++i) {
      if (there[i] == nullptr) continue;
      sums[i] = make({c.groups, c.dim}, at::kFloat, device);
      grads[i] = static_cast<float*>(sums[i]->data_ptr());
    }
    const at::Tensor& ws = tensor(b[8], "the workspace");
    check(f_norm_backward(&c, &dz, &dh, &y, &u, &z, &rdx, &rdy, &rdu, grads[0], grads[1], grads[2], grads[3], grads[4],
                          ws.data_ptr(), (size_t)ws.numel(), on.stream),
          "mt_gated_norm_backward");
    PyObject* out = PyTuple_New(8);
    if (out == nullptr) throw Raised{};
    PyTuple_SET_ITEM(out, 0, wrap_or_none(dx));
    PyTuple_SET_ITEM(out, 1, wrap_or_none(dy));
    PyTuple_SET_ITEM(out, 2, wrap_or_none(du));
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(out, 3 + i, wrap_or_none(sums[i]));
    return out;
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init),           FAST(pack8),        FAST(unpack8),       FAST(linear_forward),
                         FAST(linear_backward), FAST(norm_forward), FAST(norm_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mt_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mt_block(void) { return PyModule_Create(&module); }
