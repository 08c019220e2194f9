// The calls of f8.py, experts.py and f8_block.py on their plain form: checks, output tensors, stream and
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
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/prune24_experts.h"
#include "../../include/prune24_f8.h"
#include "../../include/prune24_f8_block.h"

namespace {

decltype(&rms_norm) p_norm = nullptr;
decltype(&gated_act) p_gate = nullptr;
decltype(&spmm24_f8) p_product = nullptr;
decltype(&experts_route) p_route = nullptr;
decltype(&experts_route_workspace) p_route_ws = nullptr;
decltype(&spmm24_f8_grouped) p_grouped = nullptr;
decltype(&experts_combine) p_combine = nullptr;
decltype(&quantize_f8_block) p_quantize = nullptr;
decltype(&gemm_f8_block) p_block = nullptr;

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

// Part of a byte buffer as a tensor, from its element `first` on.
at::Tensor part_of(const at::Tensor& buf, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t first) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                          c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(c10::IntArrayRef(shape.begin(), shape.size()));
  t.unsafeGetTensorImpl()->set_storage_offset(first);
  return t;
}

// A new tokens x width output; in 8 bits its scales lie behind the values in the
// same allocation (the two are used and freed together, and one allocation is
// half a microsecond less).
at::Tensor make_rows(int64_t tokens, int64_t width, int code, const at::Device& dev, at::Tensor& scale) {
  if (code != P24_F8) return make({tokens, width}, type_of(code), dev);
  const int64_t at = (tokens * width + 15) / 16 * 16;
  const at::Tensor buf = make({at + 4 * tokens}, at::kByte, dev);
  scale = part_of(buf, at::kFloat, {tokens}, at / 4);
  return part_of(buf, F8, {tokens, width}, 0);
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

// The operators below run on the current device only; on another one the Python code makes it current first.
bool current(const at::Device& dev) { return dev.index() == c10::hip::current_device(); }

// Contiguous int32 or fp32 of `n` values in `dims` dimensions; its address, or nullptr.
template <typename T>
const T* flat(PyObject* o, at::ScalarType type, int dims, int64_t n, const at::Device& dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.device() != dev || t.scalar_type() != type || t.dim() != dims || t.numel() != n || !t.is_contiguous())
    return nullptr;
  return static_cast<const T*>(t.data_ptr());
}

PyObject* give_all(std::initializer_list<const at::Tensor*> parts) {
  PyObject* out = PyTuple_New((Py_ssize_t)parts.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* t : parts) {
    PyObject* o = THPVariable_Wrap(*t);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// route(logits, k, score, bias, normalize, scale) -> (experts, weights, offsets, tokens, positions), parts of
// one allocation
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* l;
    int64_t ldl;
    if (n != 6 || !p_route || !rows(a[0], l, ldl)) return none();
    const int code = stream_code(l->scalar_type());
    const at::Device dev = l->device();
    if (code < 0 || !current(dev) || !PyLong_CheckExact(a[1]) || !PyFloat_CheckExact(a[5])) return none();
    const int64_t T = l->size(0), E = l->size(1), k = PyLong_AsLongLong(a[1]);
    if (k < 1 || k > E || E > P24_EXPERTS_MAX || k > P24_EXPERTS_K_MAX || T > (1 << 18)) return none();
    const float* bias = nullptr;
    if (!is_none(a[3]) && !(bias = vec(a[3], E, dev))) return none();
    const int64_t each = (T * k + 3) / 4 * 4;
    const int64_t ws = 4 * each + E + 1, need = (int64_t)p_route_ws(T, E);      // the workspace lies behind the outputs
    const at::Tensor buf = make({4 * ws + need}, at::kByte, dev);
    const at::Tensor experts = part_of(buf, at::kInt, {T, k}, 0), weights = part_of(buf, at::kFloat, {T, k}, each),
                     tokens = part_of(buf, at::kInt, {T * k}, 2 * each), positions = part_of(buf, at::kInt, {T, k}, 3 * each),
                     offsets = part_of(buf, at::kInt, {E + 1}, 4 * each);
    const p24_status st =
        p_route(l->data_ptr(), code, ldl, T, E, k, (int)PyLong_AsLong(a[2]), bias, (int)PyLong_AsLong(a[4]),
                (float)PyFloat_AS_DOUBLE(a[5]), (int32_t*)experts.data_ptr(), (float*)weights.data_ptr(),
                (int32_t*)offsets.data_ptr(), (int32_t*)tokens.data_ptr(), (int32_t*)positions.data_ptr(),
                (int32_t*)buf.data_ptr() + ws, (size_t)need, stream_of(dev));
    if (st != P24_OK) return none();
    return give_all({&experts, &weights, &offsets, &tokens, &positions});
  });
}

// grouped(data, w_scale, E, M, K, values, x_scale, offsets, tokens, code, bias, act) -> Y
PyObject* grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* x;
    int64_t ldx;
    if (n != 12 || !p_grouped || !THPVariable_CheckExact(a[0]) || !rows(a[5], x, ldx) || x->scalar_type() != F8) return none();
    const at::Tensor& data = THPVariable_Unpack(a[0]);
    const int64_t E = PyLong_AsLongLong(a[2]), M = PyLong_AsLongLong(a[3]), K = PyLong_AsLongLong(a[4]), N = x->size(0);
    const at::Device dev = x->device();
    if (E < 1 || M < 1 || !current(dev) || x->size(1) != K) return none();
    const float *ws = flat<float>(a[1], at::kFloat, 2, E * M, dev), *xs = vec(a[6], N, dev), *bias = nullptr;
    const int32_t *offsets = flat<int32_t>(a[7], at::kInt, 1, E + 1, dev), *tokens = nullptr;
    if (!ws || THPVariable_Unpack(a[1]).size(0) != E || !xs || !offsets || data.device() != dev) return none();
    if (data.scalar_type() != at::kByte || !data.is_contiguous() ||
        data.numel() < E * ((M + 127) / 128 * ((K + 127) / 128) * 2 * 5120))
      return none();
    int64_t R = N;
    if (!is_none(a[8])) {
      if (!THPVariable_CheckExact(a[8])) return none();
      R = THPVariable_Unpack(a[8]).numel();
      if (R < 1 || !(tokens = flat<int32_t>(a[8], at::kInt, 1, R, dev))) return none();
    }
    if (!is_none(a[10]) && (!(bias = flat<float>(a[10], at::kFloat, 2, E * M, dev)) || THPVariable_Unpack(a[10]).size(0) != E))
      return none();
    const long code = PyLong_AsLong(a[9]), act = PyLong_AsLong(a[11]);
    at::Tensor y = make({R, M}, type_of((int)code), dev);
    const p24_status st = p_grouped(data.data_ptr(), ws, E, M, K, x->data_ptr(), ldx, xs, N, offsets, tokens, R, y.data_ptr(),
                                    (int)code, M, bias, (int)act, stream_of(dev));
    return st == P24_OK ? THPVariable_Wrap(y) : none();
  });
}

// combine(Z, positions, weights, residual, code or -1) -> y
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *z, *r = nullptr;
    int64_t ldz, ldr = 0;
    if (n != 5 || !p_combine || !rows(a[0], z, ldz) || !THPVariable_CheckExact(a[1])) return none();
    const at::Tensor& p = THPVariable_Unpack(a[1]);
    const at::Device dev = z->device();
    const int zc = stream_code(z->scalar_type());
    if (zc < 0 || !current(dev) || p.dim() != 2 || p.size(0) < 1 || p.size(1) < 1) return none();
    const int64_t T = p.size(0), k = p.size(1), width = z->size(1);
    const int32_t* pos = flat<int32_t>(a[1], at::kInt, 2, T * k, dev);
    const float* w = flat<float>(a[2], at::kFloat, 2, T * k, dev);
    if (!pos || !w || THPVariable_Unpack(a[2]).size(0) != T) return none();
    long code = PyLong_AsLong(a[4]);
    if (!is_none(a[3])) {
      if (!rows(a[3], r, ldr) || r->device() != dev || r->size(0) != T || r->size(1) != width) return none();
      const int rc = stream_code(r->scalar_type());
      if (rc < 0 || (code >= 0 && code != rc)) return none();
      code = rc;
    }
    if (code < 0) code = zc;
    at::Tensor y = make({T, width}, type_of((int)code), dev);
    const p24_status st = p_combine(z->data_ptr(), zc, ldz, z->size(0), pos, w, T, k, width, r ? r->data_ptr() : nullptr, ldr,
                                    y.data_ptr(), (int)code, width, stream_of(dev));
    return st == P24_OK ? THPVariable_Wrap(y) : none();
  });
}

// quantize(x, up, act) -> (values, scale), parts of one allocation; for widths whose rows start on 16 bytes
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x, *u = nullptr;
    int64_t ldx, ldu = 0;
    if (n != 3 || !p_quantize || !rows(a[0], x, ldx)) return none();
    const int xc = stream_code(x->scalar_type());
    const at::Device dev = x->device();
    const int64_t tokens = x->size(0), width = x->size(1), blocks = (width + 127) / 128;
    if (xc < 0 || width % 16 || !current(dev)) return none();
    if (!is_none(a[1]) && (!rows(a[1], u, ldu) || !same_rows(*u, *x))) return none();
    const at::Tensor buf = make({tokens * width + 4 * blocks * tokens}, at::kByte, dev);
    const at::Tensor v = part_of(buf, F8, {tokens, width}, 0), s = part_of(buf, at::kFloat, {blocks, tokens}, tokens * width / 4);
    const p24_status st = p_quantize(x->data_ptr(), xc, ldx, u ? u->data_ptr() : nullptr, ldu, (int)PyLong_AsLong(a[2]),
                                     tokens, width, v.data_ptr(), width, (float*)s.data_ptr(), tokens, stream_of(dev));
    return st == P24_OK ? give_all({&v, &s}) : none();
  });
}

// block_product(W values, W scale, values, scale, code, bias, act, residual) -> Y
PyObject* block_product(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *w, *x, *r = nullptr;
    int64_t ldw, ldx, ldr = 0;
    if (n != 8 || !p_block || !rows(a[0], w, ldw) || !rows(a[2], x, ldx) || w->scalar_type() != F8 || x->scalar_type() != F8)
      return none();
    const at::Device dev = x->device();
    const int64_t M = w->size(0), K = x->size(1), N = x->size(0), blocks = (K + 127) / 128, mb = (M + 127) / 128;
    if (w->size(1) != K || w->device() != dev || !current(dev)) return none();
    const float *ws = flat<float>(a[1], at::kFloat, 2, mb * blocks, dev), *xs = flat<float>(a[3], at::kFloat, 2, blocks * N, dev),
                *bias = nullptr;
    if (!ws || !xs || THPVariable_Unpack(a[1]).size(0) != mb || THPVariable_Unpack(a[3]).size(0) != blocks) return none();
    if (!is_none(a[5]) && !(bias = vec(a[5], M, dev))) return none();
    const long code = PyLong_AsLong(a[4]), act = PyLong_AsLong(a[6]);
    if (!is_none(a[7]) && (!rows(a[7], r, ldr) || r->scalar_type() != type_of((int)code) || r->device() != dev ||
                           r->size(0) != N || r->size(1) != M))
      return none();
    at::Tensor y = make({N, M}, type_of((int)code), dev);
    const p24_status st = p_block(w->data_ptr(), ldw, ws, M, K, x->data_ptr(), ldx, xs, N, N, y.data_ptr(), (int)code, M, bias,
                                  (int)act, r ? r->data_ptr() : nullptr, ldr, stream_of(dev));
    return st == P24_OK ? THPVariable_Wrap(y) : none();
  });
}

// bind(rms_norm, gated_act, spmm24_f8, experts_route, spmm24_f8_grouped, experts_combine, quantize_f8_block,
// gemm_f8_block, experts_route_workspace): their addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int COUNT = 9;
  if (n != COUNT) {
    PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
    return nullptr;
  }
  void* p[COUNT];
  for (int i = 0; i < COUNT; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_norm = reinterpret_cast<decltype(p_norm)>(p[0]);
  p_gate = reinterpret_cast<decltype(p_gate)>(p[1]);
  p_product = reinterpret_cast<decltype(p_product)>(p[2]);
  p_route = reinterpret_cast<decltype(p_route)>(p[3]);
  p_grouped = reinterpret_cast<decltype(p_grouped)>(p[4]);
  p_combine = reinterpret_cast<decltype(p_combine)>(p[5]);
  p_quantize = reinterpret_cast<decltype(p_quantize)>(p[6]);
  p_block = reinterpret_cast<decltype(p_block)>(p[7]);
  p_route_ws = reinterpret_cast<decltype(p_route_ws)>(p[8]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), "set the library's entry points"},
                         {"norm", FAST(norm), "rms_norm with new outputs, or None"},
                         {"gate", FAST(gate), "gated_act with new outputs, or None"},
                         {"product", FAST(product), "spmm24_f8 with a new output, or None"},
                         {"route", FAST(route), "experts_route with new outputs, or None"},
                         {"grouped", FAST(grouped), "spmm24_f8_grouped with a new output, or None"},
                         {"combine", FAST(combine), "experts_combine with a new output, or None"},
                         {"quantize", FAST(quantize), "quantize_f8_block with new outputs, or None"},
                         {"block_product", FAST(block_product), "gemm_f8_block with a new output, or None"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_f8_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__f8_call(void) { return PyModule_Create(&module); }
