// binding.cpp — the calls of the kernels behind a decode step's logits, without ctypes: a Python module that looks at the
// tensors, takes their pointers and sizes and calls the C entry point.
//
// These kernels take a few microseconds, of which looking at a dozen arguments in Python would be as much again.  Each function
// returns the entry point's code, or -1 where an argument is not of the usual kind; the caller then looks at them one by
// one for a message (or, where they are right all the same, calls through ctypes).  The entry points' addresses are
// handed in by bind(), so this module belongs to whichever library is loaded.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/orpo_pages.h"

namespace {

decltype(&orpo_logits_adjust) g_adjust;
decltype(&orpo_beam_history) g_history;
decltype(&orpo_pages_advance) g_advance;
decltype(&orpo_pages_copy) g_copy;
decltype(&orpo_pages_release) g_release;
decltype(&orpo_pages_compact) g_compact;

constexpr long kUnusual = -1;

// Reads the arguments in order; `ok` turns false on the first that is not of the usual kind.
struct Args {
  PyObject* const* args;
  Py_ssize_t at = 0;
  bool ok = true;
  int64_t device = -1;

  PyObject* next() { return args[at++]; }
  int64_t whole() {
    PyObject* const o = next();
    if (!PyLong_Check(o)) return ok = false, 0;
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return v;
  }
  float real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return (float)v;
  }
  // A torch.cuda.Stream, or None for the current one; and which device is current.
  void* stream() {
    PyObject* const o = next();
    device = c10::cuda::current_device();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    PyObject* const handle = PyObject_GetAttrString(o, "cuda_stream");
    void* const s = handle ? PyLong_AsVoidPtr(handle) : nullptr;
    Py_XDECREF(handle);
    if (PyErr_Occurred()) PyErr_Clear(), ok = false;
    return s;
  }
  // A CUDA tensor on the call's device; nullptr for None where that is allowed.
  const at::Tensor* tensor(bool none = false) {
    PyObject* const o = next();
    if (o == Py_None) return ok = ok && none, nullptr;
    if (!THPVariable_Check(o)) return ok = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device) return ok = false, nullptr;
    return &t;
  }
  const at::Tensor* of(at::ScalarType type, bool none = false) {
    const at::Tensor* t = tensor(none);
    ok = ok && (!t || t->scalar_type() == type);
    return t;
  }
  const at::Tensor* ints(bool none = false) { return of(at::kInt, none); }
};

bool vector_of(const at::Tensor* t, int64_t n) { return t->dim() == 1 && t->size(0) == n && t->is_contiguous(); }
// A matrix with rows of n (n < 0: any) contiguous elements, and its pitch.
bool matrix_of(const at::Tensor* t, int64_t rows, int64_t n, int64_t& pitch) {
  if (t->dim() != 2 || (rows >= 0 && t->size(0) != rows) || (n >= 0 && t->size(1) != n)) return false;
  pitch = t->size(0) > 1 ? t->stride(0) : t->size(1);
  return (t->stride(1) == 1 || t->size(1) <= 1) && pitch >= t->size(1);
}
template <class T>
T* data(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

template <class Call>
PyObject* called(Call call) {
  long code = kUnusual;
  PyThreadState* const state = PyEval_SaveThread();
  try {
    code = call();
  } catch (...) {  // a tensor without storage
  }
  PyEval_RestoreThread(state);
  return PyLong_FromLong(code);
}

PyObject* unusual() { return PyLong_FromLong(kUnusual); }

// stream, logits, beams, status, history, length, prompt, repetition, presence, frequency, no_repeat, bias_token, bias_value,
// masks, mask_row
PyObject* adjust(Args a) {
  void* const stream = a.stream();
  const at::Tensor* const x = a.tensor();
  const int64_t beams = a.whole();
  const at::Tensor *const status = a.ints(), *const history = a.ints(true), *const length = a.ints(true), *const prompt = a.ints(true);
  const float repetition = a.real(), presence = a.real(), frequency = a.real();
  const int64_t no_repeat = a.whole();
  const at::Tensor *const bias_token = a.ints(true), *const bias_value = a.of(at::kFloat, true), *const masks = a.tensor(true),
                   *const mask_row = a.ints(true);
  int64_t ld = 0, ld_history = 0, ld_bias = 0, ld_masks = 0, ld_value = 0;
  if (!a.ok || !status || !(x->scalar_type() == at::kFloat || x->scalar_type() == at::kBFloat16) || !matrix_of(x, -1, -1, ld)) return unusual();
  const int64_t rows = x->size(0), V = x->size(1);
  if (beams < 1 || beams > INT32_MAX || rows % beams || no_repeat < INT32_MIN || no_repeat > INT32_MAX) return unusual();
  const int64_t batch = rows / beams;
  if (history && (!length || !matrix_of(history, rows, -1, ld_history) || !vector_of(length, batch) || (prompt && !vector_of(prompt, batch))))
    return unusual();
  if ((bias_token == nullptr) != (bias_value == nullptr) || (masks == nullptr) != (mask_row == nullptr)) return unusual();
  if (bias_token) {
    if (bias_token->dim() == 1 ? !(bias_token->is_contiguous() && vector_of(bias_value, bias_token->size(0)))
                               : !(matrix_of(bias_token, batch, -1, ld_bias) && matrix_of(bias_value, batch, bias_token->size(1), ld_value) && ld_value == ld_bias))
      return unusual();
  }
  if (masks && (!(masks->scalar_type() == at::kInt || masks->scalar_type() == at::kUInt32) || !matrix_of(masks, -1, (V + 31) / 32, ld_masks) ||
                !vector_of(mask_row, rows)))
    return unusual();
  return called([&] {
    return g_adjust(x->data_ptr(), ld, x->scalar_type() == at::kBFloat16, batch, (int)beams, V, data<int32_t>(history), ld_history,
                    history ? history->size(1) : 0, data<int32_t>(length), data<int32_t>(prompt), repetition, presence, frequency, (int)no_repeat,
                    data<int32_t>(bias_token), data<float>(bias_value), ld_bias, bias_token ? bias_token->size(-1) : 0, data<uint32_t>(masks),
                    ld_masks, masks ? masks->size(0) : 0, data<int32_t>(mask_row), data<int32_t>(status), stream);
  });
}

// stream, history, parent, token, length, status
PyObject* history(Args a) {
  void* const stream = a.stream();
  const at::Tensor *const h = a.ints(), *const parent = a.ints(), *const token = a.ints(), *const length = a.ints(), *const status = a.ints();
  int64_t ld = 0, ld_parent = 0, ld_token = 0;
  if (!a.ok || !matrix_of(parent, -1, -1, ld_parent)) return unusual();
  const int64_t batch = parent->size(0), beams = parent->size(1);
  if (beams > INT32_MAX || !matrix_of(h, batch * beams, -1, ld) || !matrix_of(token, batch, beams, ld_token) || !vector_of(length, batch))
    return unusual();
  return called([&] {
    return g_history(data<int32_t>(h), ld, h->size(1), data<int32_t>(parent), ld_parent, data<int32_t>(token), ld_token, data<int32_t>(length),
                     batch, (int)beams, data<int32_t>(status), stream);
  });
}

bool moves_of(const at::Tensor* moves, const at::Tensor* n_moves) {
  return moves->dim() == 2 && moves->size(1) == 3 && moves->is_contiguous() && vector_of(n_moves, 1);
}

// stream, table, refs, page, parent, length, more, most, moves, n_moves, workspace, status
PyObject* advance(Args a) {
  void* const stream = a.stream();
  const at::Tensor *const table = a.ints(), *const refs = a.ints();
  const int64_t page = a.whole();
  const at::Tensor *const parent = a.ints(true), *const length = a.ints(), *const more = a.ints(true);
  const int64_t most = a.whole();
  const at::Tensor *const moves = a.ints(), *const n_moves = a.ints(), *const workspace = a.of(at::kByte), *const status = a.ints();
  int64_t ld = 0, ld_parent = 0;
  if (!a.ok || !matrix_of(table, -1, -1, ld) || length->dim() != 1 || length->size(0) < 1 || !length->is_contiguous()) return unusual();
  const int64_t batch = length->size(0), rows = table->size(0), beams = rows / batch;
  if (rows != batch * beams || beams > INT32_MAX || !vector_of(refs, refs->numel()) || (parent && !matrix_of(parent, batch, beams, ld_parent)) ||
      (more && !vector_of(more, batch)) || !moves_of(moves, n_moves) || !workspace->is_contiguous())
    return unusual();
  return called([&] {
    return g_advance(data<int32_t>(table), ld, table->size(1), data<int32_t>(refs), refs->numel(), page, data<int32_t>(parent), ld_parent,
                     data<int32_t>(length), data<int32_t>(more), most, batch, (int)beams, data<int32_t>(moves), moves->size(0),
                     data<int32_t>(n_moves), workspace->data_ptr(), (size_t)workspace->numel(), data<int32_t>(status), stream);
  });
}

// stream, pool, moves, n_moves, status
PyObject* copy(Args a) {
  void* const stream = a.stream();
  const at::Tensor *const pool = a.tensor(), *const moves = a.ints(), *const n_moves = a.ints(), *const status = a.ints();
  if (!a.ok || pool->dim() != 5 || !pool->is_contiguous() || !moves_of(moves, n_moves)) return unusual();
  return called([&] {
    return g_copy(pool->data_ptr(), pool->size(0), pool->size(1), pool->size(2), pool->size(3), pool->size(4) * (int64_t)pool->element_size(),
                  data<int32_t>(moves), moves->size(0), data<int32_t>(n_moves), data<int32_t>(status), stream);
  });
}

// stream, table, refs, ended, status
PyObject* release(Args a) {
  void* const stream = a.stream();
  const at::Tensor *const table = a.ints(), *const refs = a.ints(), *const ended = a.tensor(true), *const status = a.ints();
  int64_t ld = 0;
  if (!a.ok || !matrix_of(table, -1, -1, ld) || !vector_of(refs, refs->numel())) return unusual();
  const int64_t rows = table->size(0), batch = ended ? ended->numel() : rows, beams = batch > 0 ? rows / batch : 1;
  if (rows != batch * beams || beams > INT32_MAX ||
      (ended && !((ended->scalar_type() == at::kByte || ended->scalar_type() == at::kBool) && vector_of(ended, batch))))
    return unusual();
  return called([&] {
    return g_release(data<int32_t>(table), ld, table->size(1), data<int32_t>(refs), refs->numel(), data<uint8_t>(ended), batch, (int)beams,
                     data<int32_t>(status), stream);
  });
}

// stream, table, refs, page, new_table, new_refs, live, moves, n_moves, workspace, status
PyObject* compact(Args a) {
  void* const stream = a.stream();
  const at::Tensor *const table = a.ints(), *const refs = a.ints();
  const int64_t page = a.whole();
  const at::Tensor *const new_table = a.ints(), *const new_refs = a.ints(), *const live = a.ints(), *const moves = a.ints(),
                   *const n_moves = a.ints(), *const workspace = a.of(at::kByte), *const status = a.ints();
  int64_t ld = 0, ld_new = 0;
  if (!a.ok || !matrix_of(table, -1, -1, ld) || !matrix_of(new_table, table->size(0), table->size(1), ld_new) ||
      !vector_of(refs, refs->numel()) || !vector_of(new_refs, refs->numel()) || !vector_of(live, 1) || !moves_of(moves, n_moves) ||
      !workspace->is_contiguous())
    return unusual();
  return called([&] {
    return g_compact(data<int32_t>(table), ld, table->size(1), table->size(0), data<int32_t>(refs), refs->numel(), page, data<int32_t>(new_table),
                     ld_new, data<int32_t>(new_refs), data<int32_t>(live), data<int32_t>(moves), moves->size(0), data<int32_t>(n_moves),
                     workspace->data_ptr(), (size_t)workspace->numel(), data<int32_t>(status), stream);
  });
}

// Whatever a tensor cannot be asked (a layout without strides, storage that is not there) makes the call an unusual one.
template <PyObject* (*f)(Args), int kArgs>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f(Args{args});
  } catch (...) {
    return unusual();
  }
}

// The addresses of the six entry points, in the order above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void** const to[] = {reinterpret_cast<void**>(&g_adjust), reinterpret_cast<void**>(&g_history), reinterpret_cast<void**>(&g_advance),
                       reinterpret_cast<void**>(&g_copy),   reinterpret_cast<void**>(&g_release), reinterpret_cast<void**>(&g_compact)};
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    *to[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<bind>("bind"),
                           method<guarded<adjust, 15>>("adjust"),
                           method<guarded<history, 6>>("history"),
                           method<guarded<advance, 12>>("advance"),
                           method<guarded<copy, 5>>("copy"),
                           method<guarded<release, 5>>("release"),
                           method<guarded<compact, 11>>("compact"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "orpo_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_orpo_binding(void) { return PyModule_Create(&g_module); }
