// The calls of f8.py on their plain form: checks, output tensors, stream and
// launch in one step.
//
// A decoding step calls these operators on a few tokens, where the kernels take
// a few microseconds and the Python side of a call took longer: the norm of one
// token 13.3 us, of which 3.5 us were the library's call and launch.  Each
// function here takes the plain form of its call -- tensors of the right types,
// shapes and strides, new outputs -- and returns None for anything else; the
// Python code then makes the same call step by step, or says what is wrong.
//
// The library's entry points come in as addresses (bind), so that this file
// links against no particular copy of it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/prune24_f8.h"

namespace {

decltype(&rms_norm) p_norm = nullptr;
decltype(&gated_act) p_gate = nullptr;
decltype(&spmm24_f8) p_product = nullptr;

constexpr at::ScalarType F8 = at::kFloat8_e4m3fn;

// dtype code of a stream's type, -1 for others
int stream_code(at::ScalarType t) { return t == at::kBFloat16 ? P24_BF16 : t == at::kFloat ? P24_F32 : -1; }
at::ScalarType type_of(int code) { return code == P24_F8 ? F8 : code == P24_BF16 ? at::kBFloat16 : at::kFloat; }

bool is_none(PyObject* o) { return o == Py_None; }

// A 2-D device tensor with unit stride along its rows.
bool rows(PyObject* o, const at::Tensor*& t, int64_t& ld) {
  if (!THPVariable_CheckExact(o)) return false;
  t = &THPVariable_Unpack(o);
  if (!t->is_cuda() || t->dim() != 2 || t->layout() != at::kStrided) return false;
  if (t->stride(1) != 1 || t->size(0) < 1 || t->size(1) < 1) return false;
  ld = t->stride(0);
  return ld >= t->size(1);
}

bool same_rows(const at::Tensor& t, const at::Tensor& like) {
  return t.scalar_type() == like.scalar_type() && t.device() == like.device() && t.size(0) == like.size(0) &&
         t.size(1) == like.size(1);
}

const float* vec(PyObject* o, int64_t n, const at::Device& dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.device() != dev || t.scalar_type() != at::kFloat || t.dim() != 1 || t.size(0) != n ||
      !t.is_contiguous())
    return nullptr;
  return static_cast<const float*>(t.data_ptr());
}

at::Tensor make(std::initializer_list<int64_t> shape, at::ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), type, dev, std::nullopt);
}

// A new tokens x width output; in 8 bits its scales lie behind the values in the
// same allocation (the two are used and freed together, and one allocation is
// half a microsecond less).
at::Tensor make_rows(int64_t tokens, int64_t width, int code, const at::Device& dev, at::Tensor& scale) {
  if (code != P24_F8) return make({tokens, width}, type_of(code), dev);
  const int64_t at = (tokens * width + 15) / 16 * 16;
  const at::Tensor buf = make({at + 4 * tokens}, at::kByte, dev);
  auto part = [&](at::ScalarType type, std::initializer_list<int64_t> shape, int64_t first) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(c10::IntArrayRef(shape.begin(), shape.size()));
    t.unsafeGetTensorImpl()->set_storage_offset(first);
    return t;
  };
  scale = part(at::kFloat, {tokens}, at / 4);
  return part(F8, {tokens, width}, 0);
}

void* stream_of(const at::Device& dev) { return c10::hip::getCurrentHIPStream(dev.index()).stream(); }

// "not the plain form": a failed conversion of an argument leaves no error behind
PyObject* none() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (values, scale or None, h or None) as a tuple
PyObject* give(const at::Tensor& y, const at::Tensor& scale, const at::Tensor& h) {
  PyObject* out = PyTuple_New(3);
  if (!out) return nullptr;
  const at::Tensor* parts[3] = {&y, &scale, &h};
  for (int i = 0; i < 3; ++i) {
    PyObject* o = parts[i]->defined() ? THPVariable_Wrap(*parts[i]) : (Py_INCREF(Py_None), Py_None);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, o);
  }
  return out;
}

// No C++ exception leaves a function that Python calls: it becomes the one that torch's own calls
// raise (an allocation's torch.OutOfMemoryError among them).
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// norm(x, weight, residual, eps, code)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5 || !p_norm) return none();
    const at::Tensor *x, *r = nullptr;
    int64_t ldx, ldr = 0;
    if (!rows(a[0], x, ldx)) return none();
    const int xc = stream_code(x->scalar_type());
    if (xc < 0) return none();
    const int64_t tokens = x->size(0), width = x->size(1);
    const at::Device dev = x->device();
    const float* w = vec(a[1], width, dev);
    if (!w || !PyFloat_CheckExact(a[3])) return none();
    if (!is_none(a[2]) && (!rows(a[2], r, ldr) || !same_rows(*r, *x))) return none();
    const long code = PyLong_AsLong(a[4]);
    at::Tensor s, h, y = make_rows(tokens, width, (int)code, dev, s);
    if (r) h = make({tokens, width}, x->scalar_type(), dev);
    const p24_status st =
        p_norm(x->data_ptr(), xc, ldx, r ? r->data_ptr() : nullptr, ldr, w, (float)PyFloat_AS_DOUBLE(a[3]), tokens,
               width, r ? h.data_ptr() : nullptr, width, y.data_ptr(), (int)code, width,
               s.defined() ? (float*)s.data_ptr() : nullptr, stream_of(dev));
    return st == P24_OK ? give(y, s, h) : none();
  });
}

// gate(gate, up, act, code)
PyObject* gate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4 || !p_gate) return none();
    const at::Tensor *g, *u = nullptr;
    int64_t ldg, ldu = 0;
    if (!rows(a[0], g, ldg)) return none();
    const int xc = stream_code(g->scalar_type());
    if (xc < 0) return none();
    if (!is_none(a[1]) && (!rows(a[1], u, ldu) || !same_rows(*u, *g))) return none();
    const int64_t tokens = g->size(0), width = g->size(1);
    const at::Device dev = g->device();
    const long act = PyLong_AsLong(a[2]), code = PyLong_AsLong(a[3]);
    at::Tensor s, y = make_rows(tokens, width, (int)code, dev, s);
    const p24_status st = p_gate(g->data_ptr(), xc, ldg, u ? u->data_ptr() : nullptr, ldu, (int)act, tokens, width,
                                 y.data_ptr(), (int)code, width, s.defined() ? (float*)s.data_ptr() : nullptr,
                                 stream_of(dev));
    return st == P24_OK ? give(y, s, at::Tensor()) : none();
  });
}

// product(data, w_scale, M, K, values, x_scale, code, bias, act, residual) -> Y
PyObject* product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10 || !p_product) return none();
    const at::Tensor *x, *r = nullptr;
    int64_t ldx, ldr = 0;
    if (!THPVariable_CheckExact(a[0]) || !rows(a[4], x, ldx) || x->scalar_type() != F8) return none();
    const at::Tensor& data = THPVariable_Unpack(a[0]);
    const int64_t M = PyLong_AsLongLong(a[2]), K = PyLong_AsLongLong(a[3]), N = x->size(0);
    const at::Device dev = x->device();
    const float *ws = vec(a[1], M, dev), *xs = vec(a[5], N, dev), *bias = nullptr;
    if (!ws || !xs || data.device() != dev || x->size(1) != K || M < 1) return none();
    if (data.scalar_type() != at::kByte || !data.is_contiguous() ||
        data.numel() < (M + 127) / 128 * ((K + 127) / 128) * 2 * 5120)
      return none();
    if (!is_none(a[7]) && !(bias = vec(a[7], M, dev))) return none();
    const long code = PyLong_AsLong(a[6]), act = PyLong_AsLong(a[8]);
    if (!is_none(a[9]) && (!rows(a[9], r, ldr) || r->scalar_type() != type_of((int)code) || r->device() != dev ||
                           r->size(0) != N || r->size(1) != M))
      return none();
    at::Tensor y = make({N, M}, type_of((int)code), dev);
    const p24_status st =
        p_product(data.data_ptr(), ws, M, K, x->data_ptr(), ldx, xs, N, y.data_ptr(), (int)code, M, bias, (int)act,
                  r ? r->data_ptr() : nullptr, ldr, stream_of(dev));
    if (st != P24_OK) return none();
    return THPVariable_Wrap(y);
  });
}

// bind(rms_norm, gated_act, spmm24_f8): their addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
    return nullptr;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_norm = reinterpret_cast<decltype(p_norm)>(p[0]);
  p_gate = reinterpret_cast<decltype(p_gate)>(p[1]);
  p_product = reinterpret_cast<decltype(p_product)>(p[2]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), "set the library's entry points"},
                         {"norm", FAST(norm), "rms_norm with new outputs, or None"},
                         {"gate", FAST(gate), "gated_act with new outputs, or None"},
                         {"product", FAST(product), "spmm24_f8 with a new output, or None"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_f8_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__f8_call(void) { return PyModule_Create(&module); }
