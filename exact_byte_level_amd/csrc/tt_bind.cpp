// tt_bind.cpp -- Python binding of the serving calls: takes tensors, checks
// them and calls the C ABI (include/tt_serve.h).
//
// A serving step of one request is a few microseconds on the GPU; reading the
// dozen tensors of a call from Python costs about 10 us, here one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstring>
#include <initializer_list>

#include "tt_serve.h"

namespace {

using at::ScalarType;

// The calls of the library, set once by connect().
struct {
  decltype(&tt_plan_blocks) plan_blocks;
  decltype(&tt_release_blocks) release_blocks;
  decltype(&tt_token_bits) token_bits;
  decltype(&tt_grammar_bits) grammar_bits;
  decltype(&tt_grammar_advance) grammar_advance;
  decltype(&tt_shape_logits) shape_logits;
} tt;

PyObject* raw_stream = nullptr;  // torch's look-up of a device's current stream

const char* type_name(ScalarType t) {
  switch (t) {
    case ScalarType::Int: return "int32";
    case ScalarType::Long: return "int64";
    case ScalarType::Float: return "float32";
    case ScalarType::Half: return "float16";
    case ScalarType::BFloat16: return "bfloat16";
    case ScalarType::Bool: return "bool";
    case ScalarType::Byte: return "uint8";
    default: return c10::toString(t);
  }
}

// The arguments of one call: the first fault sets a Python error and stays.
struct Call {
  int dev = -1;
  bool ok = true;

  bool fail(const char* format, ...) {
    if (!ok) return false;
    va_list list;
    va_start(list, format);
    PyErr_FormatV(PyExc_ValueError, format, list);
    va_end(list);
    return ok = false;
  }

  const at::Tensor* tensor(PyObject* o, const char* name) {
    if (!ok) return nullptr;
    if (!THPVariable_Check(o)) {
      fail("%s: a tensor is needed", name);
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }

  // The tensor whose device, which has to be the current one, the others share.
  void device(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) return;
    if (!t->is_cuda()) {
      fail("%s is not on a GPU", name);
      return;
    }
    dev = (int)t->get_device();
    int now = -1;
    if (hipGetDevice(&now) != hipSuccess || now != dev)
      fail("%s is on cuda:%d, the current device is cuda:%d", name, dev, now);
  }

  bool fits(const at::Tensor* t, const char* name, ScalarType type, int dims) {
    if (!t) return false;
    if (t->scalar_type() == type && t->dim() == dims && t->is_cuda() && t->get_device() == dev) return true;
    return fail("%s: a %d-d %s tensor on cuda:%d is needed, got a %d-d %s tensor on %s", name, dims, type_name(type), dev,
                (int)t->dim(), type_name(t->scalar_type()), t->device().str().c_str());
  }

  // Address of a 1-d tensor without gaps; of None, nothing.
  void* vec(PyObject* o, const char* name, ScalarType type, int64_t size = -1, int64_t* length = nullptr) {
    if (!ok || o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o, name);
    if (!fits(t, name, type, 1)) return nullptr;
    const int64_t n = t->size(0);
    if (size >= 0 && n != size) fail("%s has %lld entries, not %lld", name, (long long)n, (long long)size);
    if (n > 1 && t->stride(0) != 1) fail("%s has gaps between its entries", name);
    if (length) *length = n;
    return t->data_ptr();
  }

  // Address and row stride of a 2-d tensor whose rows are without gaps.
  void* mat(PyObject* o, const char* name, ScalarType type, int64_t* stride, int64_t rows, int64_t least,
            int64_t* count = nullptr, int64_t* width = nullptr) {
    if (!ok || o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o, name);
    if (!fits(t, name, type, 2)) return nullptr;
    const int64_t n = t->size(0), m = t->size(1);
    if (rows >= 0 && n != rows) fail("%s has %lld rows, not %lld", name, (long long)n, (long long)rows);
    if (m < least) fail("%s has rows of %lld entries, %lld are needed", name, (long long)m, (long long)least);
    if (n > 0 && m > 1 && t->stride(1) != 1) fail("%s has gaps within its rows", name);
    *stride = t->stride(0);
    if (count) *count = n;
    if (width) *width = m;
    return t->data_ptr();
  }

  int64_t number(PyObject* o) {
    if (!ok) return 0;
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) ok = false;
    return v;
  }

  bool truth(PyObject* o) {
    const int v = ok ? PyObject_IsTrue(o) : 0;
    if (v < 0) ok = false;
    return v > 0;
  }

  // Returns rc after a call that wrote into these tensors (or None): autograd, which may have kept one of them for a
  // gradient, goes by their versions.
  int wrote(int rc, std::initializer_list<PyObject*> tensors) {
    for (PyObject* o : tensors)
      if (o != Py_None && !THPVariable_Unpack(o).is_inference()) THPVariable_Unpack(o).unsafeGetTensorImpl()->bump_version();
    return rc;
  }

  // The stream given (its address), or the device's current one.
  hipStream_t stream(PyObject* o) {
    if (!ok) return nullptr;
    if (o != Py_None) return reinterpret_cast<hipStream_t>(number(o));
    PyObject* at = PyLong_FromLong(dev);
    PyObject* got = at ? PyObject_CallFunctionObjArgs(raw_stream, at, nullptr) : nullptr;
    Py_XDECREF(at);
    void* p = got ? PyLong_AsVoidPtr(got) : nullptr;
    Py_XDECREF(got);
    if (PyErr_Occurred()) ok = false;
    return reinterpret_cast<hipStream_t>(p);
  }
};

template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t needed, F f) {
  if (given != needed) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    Call c;
    const int rc = f(c);
    return c.ok ? PyLong_FromLong(rc) : nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// lengths, table, free_blocks, n_free, block_size, slots, out_n, offsets, positions, rows, out_lengths, out_n_free, stream
PyObject* plan(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 13, [&](Call& c) -> int {
    tt_plan_args a{};
    c.device(v[0], "lengths");
    a.lengths = (const int32_t*)c.vec(v[0], "lengths", ScalarType::Int, -1, &a.rows);
    a.table = (int32_t*)c.mat(v[1], "table", ScalarType::Int, &a.table_stride, a.rows, 0, nullptr, &a.width);
    a.free_blocks = (const int32_t*)c.vec(v[2], "free_blocks", ScalarType::Int, -1, &a.free_cap);
    a.n_free = (const int32_t*)c.vec(v[3], "n_free", ScalarType::Int, 1);
    a.block_size = c.number(v[4]);
    a.slots = (int64_t*)c.vec(v[5], "slots", ScalarType::Long, -1, &a.places);
    a.out_n = (int64_t*)c.vec(v[6], "out_n", ScalarType::Long, 1);
    a.offsets = (const int64_t*)c.vec(v[7], "offsets", ScalarType::Long, a.rows + 1);
    a.positions = (int32_t*)c.vec(v[8], "positions", ScalarType::Int, a.places);
    a.row_of = (int32_t*)c.vec(v[9], "rows", ScalarType::Int, a.places);
    a.out_lengths = v[10] == Py_None ? const_cast<int32_t*>(a.lengths)
                                     : (int32_t*)c.vec(v[10], "out_lengths", ScalarType::Int, a.rows);
    a.out_n_free = v[11] == Py_None ? const_cast<int32_t*>(a.n_free)
                                    : (int32_t*)c.vec(v[11], "out_n_free", ScalarType::Int, 1);
    const hipStream_t st = c.stream(v[12]);
    if (!c.ok) return 0;
    return c.wrote(tt.plan_blocks(&a, st), {v[1], v[5], v[6], v[8], v[9], v[v[10] == Py_None ? 0 : 10], v[v[11] == Py_None ? 3 : 11]});
  });
}

// lengths, done, table, free_blocks, n_free, block_size, out_n, out_lengths, out_n_free, stream
PyObject* release(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 10, [&](Call& c) -> int {
    int64_t rows = 0, stride = 0, width = 0, cap = 0;
    c.device(v[0], "lengths");
    auto* lengths = (int32_t*)c.vec(v[0], "lengths", ScalarType::Int, -1, &rows);
    const at::Tensor* d = c.tensor(v[1], "done");
    if (d && d->scalar_type() != ScalarType::Bool && d->scalar_type() != ScalarType::Byte)
      c.fail("done: truth values are needed, got %s", type_name(d->scalar_type()));
    auto* done = (const uint8_t*)c.vec(v[1], "done", d ? d->scalar_type() : ScalarType::Bool, rows);
    auto* table = (const int32_t*)c.mat(v[2], "table", ScalarType::Int, &stride, rows, 0, nullptr, &width);
    auto* free_blocks = (int32_t*)c.vec(v[3], "free_blocks", ScalarType::Int, -1, &cap);
    auto* n_free = (int32_t*)c.vec(v[4], "n_free", ScalarType::Int, 1);
    const int64_t block_size = c.number(v[5]);
    auto* out_n = (int64_t*)c.vec(v[6], "out_n", ScalarType::Long, 1);
    auto* out_lengths = v[7] == Py_None ? lengths : (int32_t*)c.vec(v[7], "out_lengths", ScalarType::Int, rows);
    auto* out_n_free = v[8] == Py_None ? n_free : (int32_t*)c.vec(v[8], "out_n_free", ScalarType::Int, 1);
    const hipStream_t st = c.stream(v[9]);
    if (!c.ok) return 0;
    return c.wrote(tt.release_blocks(lengths, done, rows, block_size, table, stride, width, free_blocks, cap, n_free,
                                     out_lengths, out_n_free, out_n, st),
                   {v[3], v[6], v[v[7] == Py_None ? 0 : 7], v[v[8] == Py_None ? 4 : 8]});
  });
}

// ids, bits, vocab, offsets, add, stream
PyObject* token_bits(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 6, [&](Call& c) -> int {
    int64_t count = 0, bounds = 2, stride = 0;
    c.device(v[1], "bits");
    const int64_t vocab = c.number(v[2]);
    auto* ids = (const int32_t*)c.vec(v[0], "ids", ScalarType::Int, -1, &count);
    auto* offsets = (const int64_t*)c.vec(v[3], "offsets", ScalarType::Long, -1, &bounds);
    auto* bits = (int32_t*)c.mat(v[1], "bits", ScalarType::Int, &stride, bounds - 1, (vocab + 31) / 32);
    const bool add = c.truth(v[4]);
    const hipStream_t st = c.stream(v[5]);
    return c.ok ? c.wrote(tt.token_bits(ids, count, offsets, bounds - 1, vocab, bits, stride, add, st), {v[1]}) : 0;
  });
}

// The grammar's and the strings' fields, as their Python objects keep them.
tt_grammar grammar_of(Call& c, PyObject* fields, PyObject* dev) {
  tt_grammar g{};
  char* data = nullptr;
  Py_ssize_t size = 0;
  if (c.ok && (PyBytes_AsStringAndSize(fields, &data, &size) < 0 || size != (Py_ssize_t)sizeof(g))) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a grammar and token strings are needed");
    c.ok = false;
  }
  if (c.ok) std::memcpy(&g, data, sizeof(g));
  if (c.number(dev) != c.dev) c.fail("the grammar, the token strings and the states have to be on one device");
  return g;
}

// fields, device of the grammar and strings, states, bits, vocab, stream
PyObject* grammar_bits(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 6, [&](Call& c) -> int {
    int64_t rows = 0, stride = 0;
    c.device(v[2], "states");
    const tt_grammar g = grammar_of(c, v[0], v[1]);
    const int64_t vocab = c.number(v[4]);
    auto* states = (const int32_t*)c.vec(v[2], "states", ScalarType::Int, -1, &rows);
    auto* bits = (int32_t*)c.mat(v[3], "bits", ScalarType::Int, &stride, rows, (vocab + 31) / 32);
    const hipStream_t st = c.stream(v[5]);
    return c.ok ? c.wrote(tt.grammar_bits(&g, states, rows, bits, stride, vocab, st), {v[3]}) : 0;
  });
}

// fields, device of the grammar and strings, states, chosen, out_states, stream
PyObject* grammar_advance(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 6, [&](Call& c) -> int {
    int64_t rows = 0;
    c.device(v[2], "states");
    const tt_grammar g = grammar_of(c, v[0], v[1]);
    auto* states = (int32_t*)c.vec(v[2], "states", ScalarType::Int, -1, &rows);
    auto* chosen = (const int32_t*)c.vec(v[3], "chosen", ScalarType::Int, rows);
    auto* out = v[4] == Py_None ? states : (int32_t*)c.vec(v[4], "out_states", ScalarType::Int, rows);
    const hipStream_t st = c.stream(v[5]);
    return c.ok ? c.wrote(tt.grammar_advance(&g, states, chosen, rows, out, st), {v[v[4] == Py_None ? 2 : 4]}) : 0;
  });
}

int64_t logits_type(ScalarType t) {
  return t == ScalarType::Float ? TT_F32 : t == ScalarType::Half ? TT_F16 : t == ScalarType::BFloat16 ? TT_BF16 : -1;
}

// logits, out, seen, generated, n_generated, repetition, frequency, presence, bias_offsets, bias_ids, bias_values,
// allowed, allowed_rows, temperature, stream
PyObject* shape(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(n, 15, [&](Call& c) -> int {
    tt_shape_args a{};
    c.device(v[0], "logits");
    const at::Tensor *x = c.tensor(v[0], "logits"), *y = c.tensor(v[1], "out");
    if (!x || !y) return 0;
    a.in_type = logits_type(x->scalar_type());
    a.out_type = logits_type(y->scalar_type());
    if (a.in_type < 0 || a.out_type < 0 || (a.out_type != a.in_type && a.out_type != TT_F32))
      c.fail("logits %s to %s: float32, float16 or bfloat16 to itself or to float32 is needed",
             type_name(x->scalar_type()), type_name(y->scalar_type()));
    int64_t wide = 0;
    a.logits = c.mat(v[0], "logits", x->scalar_type(), &a.logits_stride, -1, 0, &a.rows, &a.vocab);
    a.out = c.mat(v[1], "out", y->scalar_type(), &a.out_stride, a.rows, 0, nullptr, &wide);
    if (wide != a.vocab) c.fail("out has rows of %lld entries, not %lld", (long long)wide, (long long)a.vocab);
    const int64_t words = (a.vocab + 31) / 32;
    a.seen = (const int32_t*)c.mat(v[2], "seen", ScalarType::Int, &a.seen_stride, a.rows, words);
    a.generated = (const int32_t*)c.mat(v[3], "generated", ScalarType::Int, &a.generated_stride, a.rows, 0, nullptr,
                                        &a.generated_cap);
    a.n_generated = (const int32_t*)c.vec(v[4], "n_generated", ScalarType::Int, a.rows);
    a.repetition = (const float*)c.vec(v[5], "repetition", ScalarType::Float, a.rows);
    a.frequency = (const float*)c.vec(v[6], "frequency", ScalarType::Float, a.rows);
    a.presence = (const float*)c.vec(v[7], "presence", ScalarType::Float, a.rows);
    if ((v[8] == Py_None) != (v[9] == Py_None) || (v[8] == Py_None) != (v[10] == Py_None))
      c.fail("bias_offsets, bias_ids and bias_values belong together");
    a.bias_offsets = (const int64_t*)c.vec(v[8], "bias_offsets", ScalarType::Long, a.rows + 1);
    a.bias_ids = (const int32_t*)c.vec(v[9], "bias_ids", ScalarType::Int, -1, &a.n_bias);
    a.bias_values = (const float*)c.vec(v[10], "bias_values", ScalarType::Float, a.n_bias);
    if (v[11] == Py_None && v[12] != Py_None) c.fail("allowed_rows without allowed");
    a.allowed = (const int32_t*)c.mat(v[11], "allowed", ScalarType::Int, &a.allowed_stride, v[12] == Py_None ? a.rows : -1,
                                      words, &a.allowed_count);
    // without a single set there is no address, but the rows still go by them
    if (v[11] != Py_None && !a.allowed) a.allowed = (const int32_t*)a.logits;
    a.allowed_rows = (const int32_t*)c.vec(v[12], "allowed_rows", ScalarType::Int, a.rows);
    a.temperature = (const float*)c.vec(v[13], "temperature", ScalarType::Float, a.rows);
    const hipStream_t st = c.stream(v[14]);
    return c.ok ? c.wrote(tt.shape_logits(&a, st), {v[1]}) : 0;
  });
}

// Addresses of the six calls, in the order above.
PyObject* connect(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != (Py_ssize_t)(sizeof(tt) / sizeof(void*))) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  void* at[sizeof(tt) / sizeof(void*)];
  for (Py_ssize_t i = 0; i < n; ++i) {
    at[i] = PyLong_AsVoidPtr(v[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  std::memcpy(&tt, at, sizeof(tt));
  Py_RETURN_NONE;
}

#define CALL(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(connect),         CALL(plan),  CALL(release), CALL(token_bits), CALL(grammar_bits),
                         CALL(grammar_advance), CALL(shape), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) {
  PyObject* torch_c = PyImport_ImportModule("torch._C");
  if (!torch_c) return nullptr;
  raw_stream = PyObject_GetAttrString(torch_c, "_cuda_getCurrentRawStream");
  Py_DECREF(torch_c);
  return raw_stream ? PyModule_Create(&module) : nullptr;
}
