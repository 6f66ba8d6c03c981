// torch_calls.cpp -- the host side of the 4-bit route's calls and of the heads'
// rotation: torch tensors checked and handed to libi8 (include/i8.h), outputs and
// workspaces allocated by torch.  fp4.py and serving.py document the calls and
// give their defaults.
//
// A CPython extension and not ctypes, because a small call is the host's time: one
// token through a layer is 5 us of the GPU's, and 21 us of the host's by ctypes, most
// of it in the interpreter and in torch.empty's argument parser with the caches cold
// from the launch before.
//
// Nothing leaves a function here by a C++ exception: Refusal (an argument that is
// refused) becomes its Python error, and what torch throws the one that torch's own
// functions raise (torch.OutOfMemoryError where there is no room for an output).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "../../include/i8.h"

namespace {

PyObject* g_rows_type = nullptr;   // FP4Rows
PyObject* g_error_type = nullptr;  // I8Error(status, what)

struct Refusal {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse_type(std::string what) { throw Refusal{PyExc_TypeError, std::move(what)}; }
[[noreturn]] void refuse(std::string what) { throw Refusal{PyExc_ValueError, std::move(what)}; }

const char* dtype_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : t == at::kByte ? "torch.uint8" : t == at::kInt ? "torch.int32" : "torch.float32";
}

// A CUDA tensor of a type and a number of dimensions, on device `index` (-1: any).
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType dtype, int64_t dims, int index) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != dtype) refuse_type(std::string(name) + " must be " + dtype_name(dtype));
  if (t.dim() != dims) refuse(std::string(name) + " must be " + std::to_string(dims) + "-D");
  if (index >= 0 && t.get_device() != index) refuse(std::string(name) + " must be on cuda:" + std::to_string(index));
  return t;
}

// The address of a contiguous vector of n elements; None: null, where that is allowed.
const void* vector(PyObject* o, const char* name, at::ScalarType dtype, int64_t n, int index, bool none = true) {
  if (none && o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name, dtype, 1, index);
  if (t.size(0) != n) refuse(std::string(name) + " must have " + std::to_string(n) + " elements, got " + std::to_string(t.size(0)));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

struct Matrix {
  void* p;
  int64_t ld;
};
// A matrix with unit stride along its rows.
Matrix matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
  if (t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(name) + " must be (" + std::to_string(rows) + ", " + std::to_string(cols) + "), got (" +
           std::to_string(t.size(0)) + ", " + std::to_string(t.size(1)) + ")");
  if (t.stride(1) != 1 && cols > 1) refuse(std::string(name) + " must have unit stride along its rows");
  if (rows <= 1) return {t.data_ptr(), cols};  // the stride of a single row says nothing
  if (t.stride(0) < cols) refuse(std::string(name) + " rows overlap");
  return {t.data_ptr(), t.stride(0)};
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType dtype, int index) {
  return at::empty(size, at::TensorOptions().dtype(dtype).device(at::Device(at::kCUDA, static_cast<at::DeviceIndex>(index))));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refusal{nullptr, {}};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, {}};
  return v;
}
PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Refusal{nullptr, {}};
  return o;
}

// ----------------------------------------------------------------- rows
constexpr int64_t kTile[2] = {2048, 1024};  // bytes of block scales of 128 rows by 256 elements

// FP4Rows on a device.
i8_fp4_rows rows_of(PyObject* o, const std::string& name, int index) {
  if (reinterpret_cast<PyObject*>(Py_TYPE(o)) != g_rows_type) refuse_type(name + " must be FP4Rows");
  PyObject* const row = PyTuple_GET_ITEM(o, 2);
  const at::Tensor& codes = tensor(PyTuple_GET_ITEM(o, 0), (name + ".codes").c_str(), at::kByte, 2, index);
  const at::Tensor& scales = tensor(PyTuple_GET_ITEM(o, 1), (name + ".block_scales").c_str(), at::kByte, 3, index);
  const int64_t n = codes.size(0), half = codes.size(1), size = scales.size(2);
  if ((size != kTile[0] && size != kTile[1]) || scales.size(0) != (n + 127) / 128 || scales.size(1) != (half + 127) / 128)
    refuse(name + ".block_scales must be [ceil(rows / 128), ceil(K / 256), 2048 or 1024]");
  if (!codes.is_contiguous() || !scales.is_contiguous()) refuse(name + " must be contiguous");
  return {codes.data_ptr(), scales.data_ptr(),
          static_cast<const float*>(vector(row, (name + ".row_scales").c_str(), at::kFloat, n, index)), n, 2 * half,
          size == kTile[0] ? I8_FP4_NV16 : I8_FP4_MX32};
}
int device_of_rows(PyObject* o, const char* name) {
  if (reinterpret_cast<PyObject*>(Py_TYPE(o)) != g_rows_type) refuse_type(std::string(name) + " must be FP4Rows");
  return tensor(PyTuple_GET_ITEM(o, 0), (std::string(name) + ".codes").c_str(), at::kByte, 2, -1).get_device();
}

// Fresh rows, or those of `given` where they are of these sizes.
struct NewRows {
  at::Tensor codes, scales, row;
  i8_fp4_rows rows;
};
NewRows new_rows(PyObject* given, int64_t n, int64_t K, int fmt, bool scaled, int index) {
  NewRows r;
  if (given != Py_None) {
    r.rows = rows_of(given, "out", index);
    if (r.rows.rows != n || r.rows.K != K || r.rows.fmt != fmt || scaled != (PyTuple_GET_ITEM(given, 2) != Py_None))
      refuse("out must be FP4Rows.empty of the rows' sizes and format");
    return r;
  }
  r.codes = empty({n, K / 2}, at::kByte, index);
  r.scales = empty({(n + 127) / 128, (K + 255) / 256, kTile[fmt]}, at::kByte, index);
  if (scaled) r.row = empty({n}, at::kFloat, index);
  r.rows = {r.codes.data_ptr(), r.scales.data_ptr(), scaled ? static_cast<const float*>(r.row.data_ptr()) : nullptr, n, K, fmt};
  return r;
}
// FP4Rows of them: `given`, or a new one.
PyObject* finish_rows(PyObject* given, const NewRows& r) {
  if (given != Py_None) return Py_NewRef(given);
  // (a tuple's subclass, filled here: its own constructor runs in the interpreter)
  PyTypeObject* const type = reinterpret_cast<PyTypeObject*>(g_rows_type);
  PyObject* const made = type->tp_alloc(type, 3);
  if (!made) throw Refusal{nullptr, {}};
  try {
    PyTuple_SET_ITEM(made, 0, wrap(r.codes));
    PyTuple_SET_ITEM(made, 1, wrap(r.scales));
    PyTuple_SET_ITEM(made, 2, r.row.defined() ? wrap(r.row) : Py_NewRef(Py_None));
  } catch (...) {
    Py_DECREF(made);
    throw;
  }
  return made;
}

// bf16 [rows, K] to quantize.
struct Source {
  void* p;
  int64_t rows, K, ld;
  int index;
};
Source source(PyObject* o) {
  const at::Tensor& t = tensor(o, "x", at::kBFloat16, 2, -1);
  const int64_t rows = t.size(0), K = t.size(1);
  if (K == 0 || K % 32 != 0) refuse("x's width must be a multiple of 32");
  const Matrix m = matrix(t, "x", rows, K);
  return {m.p, rows, K, m.ld, static_cast<int>(t.get_device())};
}

struct Output {
  at::Tensor fresh;
  Matrix m;
  PyObject* give(PyObject* out) const { return out != Py_None ? Py_NewRef(out) : wrap(fresh); }
};
Output output(PyObject* o, const char* name, int64_t rows, int64_t cols, int index) {
  Output out;
  if (o != Py_None) {
    out.m = matrix(tensor(o, name, at::kBFloat16, 2, index), name, rows, cols);
  } else {
    out.fresh = empty({rows, cols}, at::kBFloat16, index);
    out.m = {out.fresh.data_ptr(), cols};
  }
  return out;
}

// The library's call on the current stream of device `index`, made the current
// device for the call where it is not.
template <typename Call>
void run(const char* name, int index, Call call) {
  i8_status status;
  {
    const c10::cuda::OptionalCUDAGuard guard(at::Device(at::kCUDA, static_cast<at::DeviceIndex>(index)));
    const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<at::DeviceIndex>(index)).stream();
    PyThreadState* const state = PyEval_SaveThread();  // a launch may wait for room in the stream
    status = call(reinterpret_cast<i8_stream_t>(stream));
    PyEval_RestoreThread(state);
  }
  if (status == I8_OK) return;
  PyObject* const e = PyObject_CallFunction(g_error_type, "is", static_cast<int>(status), name);
  if (e) {
    PyErr_SetObject(g_error_type, e);
    Py_DECREF(e);
  }
  throw Refusal{nullptr, {}};
}

// ----------------------------------------------------------------- calls
// quant_rows(x, fmt, out) -> FP4Rows
PyObject* quant_rows(PyObject* const* a) {
  const Source x = source(a[0]);
  const int fmt = static_cast<int>(integer(a[1]));
  const NewRows r = new_rows(a[2], x.rows, x.K, fmt, fmt == I8_FP4_NV16, x.index);
  run("i8_quant_rows_fp4", x.index, [&](i8_stream_t st) {
    return i8_quant_rows_fp4(x.p, x.rows, x.K, x.ld, fmt, const_cast<void*>(r.rows.codes),
                             const_cast<void*>(r.rows.block_scales), const_cast<float*>(r.rows.row_scales), st);
  });
  return finish_rows(a[2], r);
}

// norm_rows(x, residual, weight, eps, fmt, residual_out, out) -> FP4Rows or (FP4Rows, h)
PyObject* norm_rows(PyObject* const* a) {
  const Source x = source(a[0]);
  const void* const weight = vector(a[2], "weight", at::kBFloat16, x.K, x.index);
  const float eps = static_cast<float>(number(a[3]));
  const int fmt = static_cast<int>(integer(a[4]));
  Matrix res{nullptr, 0};
  Output h{{}, {nullptr, 0}};
  if (a[1] != Py_None) {
    res = matrix(tensor(a[1], "residual", at::kBFloat16, 2, x.index), "residual", x.rows, x.K);
    h = output(a[5], "residual_out", x.rows, x.K, x.index);
  } else if (a[5] != Py_None) {
    refuse("residual_out without a residual");
  }
  const NewRows r = new_rows(a[6], x.rows, x.K, fmt, true, x.index);
  run("i8_add_rmsnorm_quant_fp4", x.index, [&](i8_stream_t st) {
    return i8_add_rmsnorm_quant_fp4(x.p, x.rows, x.K, x.ld, res.p, res.ld, weight, eps, fmt, const_cast<void*>(r.rows.codes),
                                    const_cast<void*>(r.rows.block_scales), const_cast<float*>(r.rows.row_scales), h.m.p,
                                    h.m.ld, st);
  });
  PyObject* const rows = finish_rows(a[6], r);
  if (a[1] == Py_None) return rows;
  PyObject* sum = nullptr;
  try {
    sum = h.give(a[5]);
  } catch (...) {
    Py_DECREF(rows);
    throw;
  }
  PyObject* const both = PyTuple_Pack(2, rows, sum);
  Py_DECREF(rows);
  Py_DECREF(sum);
  if (!both) throw Refusal{nullptr, {}};
  return both;
}

// gemm(a, w, bias, out) -> y
PyObject* gemm(PyObject* const* a) {
  const int index = device_of_rows(a[0], "a");
  const i8_fp4_rows t = rows_of(a[0], "a", index), w = rows_of(a[1], "w", index);
  if (t.K != w.K || t.fmt != w.fmt) refuse("a and w must have the same K and format");
  const void* const bias = vector(a[2], "bias", at::kBFloat16, w.rows, index);
  const Output y = output(a[3], "out", t.rows, w.rows, index);
  run("i8_gemm_fp4_bias_bf16", index,
      [&](i8_stream_t st) { return i8_gemm_fp4_bias_bf16(&t, &w, bias, y.m.p, y.m.ld, st); });
  return y.give(a[3]);
}

// gemm_gated(a, gate, up, gate_bias, up_bias, activation, out) -> y
PyObject* gemm_gated(PyObject* const* a) {
  const int index = device_of_rows(a[0], "a");
  const i8_fp4_rows t = rows_of(a[0], "a", index), g = rows_of(a[1], "gate", index), u = rows_of(a[2], "up", index);
  if (t.K != g.K || t.fmt != g.fmt || u.K != g.K || u.fmt != g.fmt || u.rows != g.rows)
    refuse("a, gate and up must have the same K and format, gate and up the same rows");
  const void* const gb = vector(a[3], "gate_bias", at::kBFloat16, g.rows, index);
  const void* const ub = vector(a[4], "up_bias", at::kBFloat16, g.rows, index);
  const int act = static_cast<int>(integer(a[5]));
  const Output y = output(a[6], "out", t.rows, g.rows, index);
  run("i8_gemm_fp4_gated_bf16", index,
      [&](i8_stream_t st) { return i8_gemm_fp4_gated_bf16(&t, &g, &u, gb, ub, act, y.m.p, y.m.ld, st); });
  return y.give(a[6]);
}

struct Workspace {
  at::Tensor fresh;
  void* p;
  size_t bytes;
};
Workspace workspace(PyObject* o, const Source& x, int fmt) {
  Workspace ws;
  if (o == Py_None) {
    ws.bytes = i8_linear_fp4_workspace_bytes(x.rows, x.K, fmt);
    ws.fresh = empty({static_cast<int64_t>(ws.bytes)}, at::kByte, x.index);
    ws.p = ws.fresh.data_ptr();
    return ws;
  }
  if (!THPVariable_Check(o)) refuse_type("workspace must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != x.index || !t.is_contiguous())
    refuse("workspace must be contiguous and on cuda:" + std::to_string(x.index));
  ws.p = t.data_ptr();
  ws.bytes = static_cast<size_t>(t.numel()) * t.element_size();
  return ws;
}

// linear(x, w, bias, out, workspace) -> y
PyObject* linear(PyObject* const* a) {
  const Source x = source(a[0]);
  const i8_fp4_rows w = rows_of(a[1], "w", x.index);
  if (w.K != x.K) refuse("x and w must have the same K");
  const void* const bias = vector(a[2], "bias", at::kBFloat16, w.rows, x.index);
  const Output y = output(a[3], "out", x.rows, w.rows, x.index);
  const Workspace ws = workspace(a[4], x, w.fmt);
  run("i8_linear_fp4", x.index, [&](i8_stream_t st) {
    return i8_linear_fp4(x.p, x.rows, x.K, x.ld, &w, bias, y.m.p, y.m.ld, ws.p, ws.bytes, st);
  });
  return y.give(a[3]);
}

// linear_gated(x, gate, up, gate_bias, up_bias, activation, out, workspace) -> y
PyObject* linear_gated(PyObject* const* a) {
  const Source x = source(a[0]);
  const i8_fp4_rows g = rows_of(a[1], "gate", x.index), u = rows_of(a[2], "up", x.index);
  if (g.K != x.K || u.K != x.K || u.fmt != g.fmt || u.rows != g.rows)
    refuse("x, gate and up must have the same K, gate and up the same rows and format");
  const void* const gb = vector(a[3], "gate_bias", at::kBFloat16, g.rows, x.index);
  const void* const ub = vector(a[4], "up_bias", at::kBFloat16, g.rows, x.index);
  const int act = static_cast<int>(integer(a[5]));
  const Output y = output(a[6], "out", x.rows, g.rows, x.index);
  const Workspace ws = workspace(a[7], x, g.fmt);
  run("i8_gated_linear_fp4", x.index, [&](i8_stream_t st) {
    return i8_gated_linear_fp4(x.p, x.rows, x.K, x.ld, &g, &u, gb, ub, act, y.m.p, y.m.ld, ws.p, ws.bytes, st);
  });
  return y.give(a[6]);
}

// bf16 [tokens, heads, head_dim] with unit stride along head_dim.
struct Heads {
  void* p;
  int64_t token, head;
};
Heads heads(const at::Tensor& t, const char* name, int64_t tokens, int64_t n, int64_t dim) {
  if (t.size(0) != tokens || t.size(1) != n || t.size(2) != dim)
    refuse(std::string(name) + " must be (" + std::to_string(tokens) + ", " + std::to_string(n) + ", " + std::to_string(dim) + ")");
  if (t.stride(2) != 1 && dim > 1) refuse(std::string(name) + " must have unit stride along head_dim");
  // the stride along a dimension of one element says nothing
  return {t.data_ptr(), tokens > 1 ? t.stride(0) : 0, n > 1 ? t.stride(1) : 0};
}

// rotate(q, k, positions, inv_freq, q_weight, k_weight, eps, sections, interleaved, out) -> (q, k)
PyObject* rotate(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q", at::kBFloat16, 3, -1);
  const int index = static_cast<int>(q.get_device());
  const at::Tensor& k = tensor(a[1], "k", at::kBFloat16, 3, index);
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), Hk = k.size(1);
  const Heads qi = heads(q, "q", T, Hq, D), ki = heads(k, "k", T, Hk, D);
  const at::Tensor& freq = tensor(a[3], "inv_freq", at::kFloat, 1, index);
  const int64_t half = freq.size(0);
  if (!freq.is_contiguous()) refuse("inv_freq must be contiguous");
  if (!THPVariable_Check(a[2])) refuse_type("positions must be a torch.Tensor");
  const at::Tensor& where = tensor(a[2], "positions", at::kInt, THPVariable_Unpack(a[2]).dim() == 2 ? 2 : 1, index);
  int64_t axes = 1;
  Matrix pos{nullptr, T};
  if (where.dim() == 2) {
    axes = where.size(0);
    if (a[7] == Py_None) refuse("positions of several axes need sections");
    pos = matrix(where, "positions", axes, T);
  } else {
    pos.p = const_cast<void*>(vector(a[2], "positions", at::kInt, T, index, false));
  }
  int32_t sections[4] = {static_cast<int32_t>(half), 0, 0, 0};
  if (a[7] != Py_None) {
    PyObject* const seq = PySequence_Fast(a[7], "sections must be a sequence of counts");
    if (!seq) throw Refusal{nullptr, {}};
    int64_t sum = 0;
    const int64_t n = PySequence_Fast_GET_SIZE(seq);
    bool good = n == axes && n <= 4;
    for (int64_t i = 0; good && i < n; ++i) {
      const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
      if (v == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw Refusal{nullptr, {}};
      }
      good = v >= 0 && v <= half;
      sections[i] = static_cast<int32_t>(v);
      sum += v;
    }
    Py_DECREF(seq);
    if (!good || sum != half) refuse("sections must be one count of pairs an axis (4 at most), together len(inv_freq)");
  }
  const void* const qw = vector(a[4], "q_weight", at::kBFloat16, D, index);
  const void* const kw = vector(a[5], "k_weight", at::kBFloat16, D, index);
  const float eps = static_cast<float>(number(a[6]));
  const int interleaved = PyObject_IsTrue(a[8]);
  if (interleaved < 0) throw Refusal{nullptr, {}};
  at::Tensor fresh_q, fresh_k;
  Heads qo, ko;
  const bool given = a[9] != Py_None;
  if (given) {
    if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 2) refuse_type("out must be two tensors");
    qo = heads(tensor(PyTuple_GET_ITEM(a[9], 0), "out[0]", at::kBFloat16, 3, index), "out[0]", T, Hq, D);
    ko = heads(tensor(PyTuple_GET_ITEM(a[9], 1), "out[1]", at::kBFloat16, 3, index), "out[1]", T, Hk, D);
  } else {
    fresh_q = empty({T, Hq, D}, at::kBFloat16, index);
    fresh_k = empty({T, Hk, D}, at::kBFloat16, index);
    qo = {fresh_q.data_ptr(), Hq * D, D};
    ko = {fresh_k.data_ptr(), Hk * D, D};
  }
  run("i8_heads_rmsnorm_rotate", index, [&](i8_stream_t st) {
    return i8_heads_rmsnorm_rotate(qi.p, qi.token, qi.head, Hq, ki.p, ki.token, ki.head, Hk, T, D, qw, kw, eps,
                                   static_cast<const int32_t*>(pos.p), pos.ld, axes, sections,
                                   static_cast<const float*>(freq.data_ptr()), 2 * half, interleaved, qo.p, qo.token,
                                   qo.head, ko.p, ko.token, ko.head, st);
  });
  if (given) return Py_NewRef(a[9]);
  PyObject* const both = PyTuple_New(2);
  if (!both) throw Refusal{nullptr, {}};
  for (int i = 0; i < 2; ++i) {
    PyObject* const one = THPVariable_Wrap(i == 0 ? fresh_q : fresh_k);
    if (!one) {
      Py_DECREF(both);
      throw Refusal{nullptr, {}};
    }
    PyTuple_SET_ITEM(both, i, one);
  }
  return both;
}

// The types that the calls make: FP4Rows, I8Error.
PyObject* types(PyObject* const* a) {
  Py_XSETREF(g_rows_type, Py_NewRef(a[0]));
  Py_XSETREF(g_error_type, Py_NewRef(a[1]));
  return Py_NewRef(Py_None);
}

template <PyObject* (*CALL)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", ARGS, n);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return CALL(args);
  } catch (const Refusal& r) {
    if (r.type) PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*CALL)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<CALL, ARGS>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<types, 2>("types"),       method<quant_rows, 3>("quant_rows"),
                           method<norm_rows, 7>("norm_rows"), method<gemm, 4>("gemm"),
                           method<gemm_gated, 7>("gemm_gated"), method<linear, 5>("linear"),
                           method<linear_gated, 8>("linear_gated"), method<rotate, 10>("rotate"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
