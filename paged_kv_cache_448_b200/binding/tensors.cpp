// tensors.cpp — the calls of the 4-bit cache and of the page operators on torch
// tensors (module _tensors): each checks its tensors in full and makes one call
// of the C ABI (include/paged.h) on the tensors' device.
//
// These calls launch kernels of a few microseconds. The same checks in Python
// cost 5 to 7 us a call, and the argument conversions of ctypes 2 to 3 us more
// (a decode call of 24 arguments over four small sequences 10.5 us in all);
// here a call is bounded by its launch.
//
// Every function returns the call's pa_status, 0 for success; what is wrong
// with a tensor raises ValueError (TypeError for what is no tensor).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "paged.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct TypeProblem : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw TypeProblem(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// t has this type and shape (-1: any extent), is contiguous and on device dev.
void check(const Tensor& t, const char* name, ScalarType type, std::initializer_list<int64_t> shape,
           int dev) {
  bool ok = t.scalar_type() == type && t.dim() == static_cast<int64_t>(shape.size());
  int64_t i = 0;
  if (ok)
    for (int64_t n : shape) {
      ok &= n < 0 || t.size(i) == n;
      ++i;
    }
  if (ok && t.is_contiguous() && t.get_device() == dev) return;
  std::ostringstream s;
  s << name << " must be a contiguous " << type << " tensor of shape [";
  i = 0;
  for (int64_t n : shape) {
    s << (i++ ? ", " : "");
    if (n < 0) s << "*";
    else s << n;
  }
  s << "] on the call's device, not " << t.scalar_type() << " " << t.sizes() << " on " << t.device()
    << (t.is_contiguous() ? "" : ", not contiguous");
  bad(s.str());
}

struct Rows {  // two 16-bit tensors [tokens, heads, head_dim] alike
  pa_dtype type;
  int64_t tokens, heads, dim;
  int dev;
};

Rows check_rows(const Tensor& x, const Tensor& y, const char* xname, const char* yname) {
  const ScalarType t = x.scalar_type();
  if ((t != at::kHalf && t != at::kBFloat16) || x.dim() != 3 || !x.is_contiguous())
    bad(std::string(xname) + " must be a contiguous f16 or bf16 [tokens, heads, head_dim] tensor");
  const Rows r{t == at::kHalf ? PA_F16 : PA_BF16, x.size(0), x.size(1), x.size(2),
               static_cast<int>(x.get_device())};
  check(y, yname, t, {r.tokens, r.heads, r.dim}, r.dev);
  if (r.dim <= 0 || r.heads <= 0) bad(std::string(xname) + " has no heads or no head_dim");
  return r;
}

struct Planes {
  uint8_t *kc, *vc, *ks, *vs;
  int64_t blocks, heads, block_size;
};

Planes check_planes(PyObject* const* o, int64_t dim, int dev) {
  const Tensor &kc = tensor(o[0], "key_cache"), &vc = tensor(o[1], "value_cache"),
               &ks = tensor(o[2], "k_scales"), &vs = tensor(o[3], "v_scales");
  if (kc.dim() != 4)
    bad("key_cache must be [num_blocks, num_kv_heads, block_size, head_dim / 2]");
  const int64_t nb = kc.size(0), h = kc.size(1), bs = kc.size(2);
  check(kc, "key_cache", at::kByte, {nb, h, bs, dim / 2}, dev);
  check(vc, "value_cache", at::kByte, {nb, h, bs, dim / 2}, dev);
  check(ks, "k_scales", at::kByte, {nb, h, bs, dim / 32}, dev);
  check(vs, "v_scales", at::kByte, {nb, h, bs, dim / 32}, dev);
  auto p = [](const Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); };
  return {p(kc), p(vc), p(ks), p(vs), nb, h, bs};
}

int32_t* ints(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

int32_t i32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " does not fit in 32 bits");
  return static_cast<int32_t>(v);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeProblem(std::string(name) + " must be an integer");
  }
  return v;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeProblem(std::string(name) + " must be a number");
  }
  return v;
}

// Other Python threads run while this lives: a launch waits for room in the
// GPU's queue, and what empties the queue may need them (a host callback).
struct WithoutLock {
  PyThreadState* state = PyEval_SaveThread();
  WithoutLock() = default;
  WithoutLock(const WithoutLock&) = delete;
  ~WithoutLock() { PyEval_RestoreThread(state); }
};

// call(stream) with device dev current and the interpreter lock released (call
// touches no Python object); stream None: the device's current one, else the
// handle (an integer).
template <class F>
PyObject* launch(int dev, PyObject* stream, F call) {
  if (dev < 0) bad("tensors must be on a CUDA device");
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
  void* handle =
      stream == Py_None
          ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream())
          : PyLong_AsVoidPtr(stream);
  if (!handle && PyErr_Occurred()) {
    PyErr_Clear();
    throw TypeProblem("stream must be a CUDA stream");
  }
  long status;
  {
    const WithoutLock unlocked;
    status = call(static_cast<pa_stream_t>(handle));
  }
  return PyLong_FromLong(status);
}

template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F body) {
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", given, wanted);
    return nullptr;
  }
  try {
    return body();
  } catch (const TypeProblem& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// key, value, four planes, slot_mapping, stream
template <class Call>
PyObject* rows_call(PyObject* const* a, Py_ssize_t n, Call call) {
  return guarded(n, 8, [&] {
    const Tensor &key = tensor(a[0], "key"), &value = tensor(a[1], "value");
    const Rows r = check_rows(key, value, "key", "value");
    const Planes p = check_planes(a + 2, r.dim, r.dev);
    if (p.heads != r.heads)
      bad("the cache has " + std::to_string(p.heads) + " kv-heads, key " + std::to_string(r.heads));
    const Tensor& slots = tensor(a[6], "slot_mapping");
    check(slots, "slot_mapping", at::kInt, {r.tokens}, r.dev);
    return launch(r.dev, a[7], [&](pa_stream_t s) {
      return call(key.data_ptr(), value.data_ptr(), p.kc, p.vc, p.ks, p.vs, ints(slots),
                  i32(r.tokens, "tokens"), i32(r.heads, "heads"), i32(r.dim, "head_dim"),
                  i32(p.block_size, "block_size"), p.blocks, r.type, s);
    });
  });
}

PyObject* write_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return rows_call(a, n, pa_reshape_and_cache_mxfp4);
}
PyObject* read_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return rows_call(a, n, pa_gather_cache_mxfp4);
}

// out, query, four planes, block_tables, context_lens, max_context_len, scale,
// partition_tokens, workspace, stream
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Tensor &out = tensor(a[0], "out"), &query = tensor(a[1], "query");
    const Rows r = check_rows(query, out, "query", "out");
    const Planes p = check_planes(a + 2, r.dim, r.dev);
    const Tensor &bt = tensor(a[6], "block_tables"), &cl = tensor(a[7], "context_lens"),
                 &ws = tensor(a[11], "workspace");
    check(bt, "block_tables", at::kInt, {r.tokens, -1}, r.dev);
    check(cl, "context_lens", at::kInt, {r.tokens}, r.dev);
    check(ws, "workspace", at::kByte, {-1}, r.dev);
    const int32_t max_ctx = i32(integer(a[8], "max_context_len"), "max_context_len");
    const float scale = static_cast<float>(number(a[9], "scale"));
    const int32_t part = i32(integer(a[10], "partition_tokens"), "partition_tokens");
    return launch(r.dev, a[12], [&](pa_stream_t s) {
      return pa_decode_mxfp4(out.data_ptr(), query.data_ptr(), p.kc, p.vc, p.ks, p.vs, ints(bt),
                             i32(bt.size(1), "max_blocks_per_seq"), ints(cl), max_ctx,
                             i32(r.tokens, "sequences"), i32(r.heads, "heads"),
                             i32(p.heads, "kv_heads"), i32(r.dim, "head_dim"),
                             i32(p.block_size, "block_size"), p.blocks, scale, r.type, part,
                             ws.data_ptr(), static_cast<size_t>(ws.numel()), s);
    });
  });
}

// out, query, cu_query_lens, max_query_len, four planes, block_tables,
// context_lens, max_context_len, scale, workspace, stream
PyObject* chunked_prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Tensor &out = tensor(a[0], "out"), &query = tensor(a[1], "query");
    const Rows r = check_rows(query, out, "query", "out");
    const Planes p = check_planes(a + 4, r.dim, r.dev);
    const Tensor &cu = tensor(a[2], "cu_query_lens"), &bt = tensor(a[8], "block_tables"),
                 &cl = tensor(a[9], "context_lens"), &ws = tensor(a[12], "workspace");
    check(bt, "block_tables", at::kInt, {-1, -1}, r.dev);
    const int64_t seqs = bt.size(0);
    check(cl, "context_lens", at::kInt, {seqs}, r.dev);
    check(cu, "cu_query_lens", at::kInt, {seqs + 1}, r.dev);
    check(ws, "workspace", at::kByte, {-1}, r.dev);
    const int32_t max_q = i32(integer(a[3], "max_query_len"), "max_query_len");
    const int32_t max_ctx = i32(integer(a[10], "max_context_len"), "max_context_len");
    const float scale = static_cast<float>(number(a[11], "scale"));
    return launch(r.dev, a[13], [&](pa_stream_t s) {
      return pa_chunked_prefill_mxfp4(
          out.data_ptr(), query.data_ptr(), ints(cu), i32(r.tokens, "tokens"), max_q, p.kc, p.vc,
          p.ks, p.vs, ints(bt), i32(bt.size(1), "max_blocks_per_seq"), ints(cl), max_ctx,
          i32(seqs, "sequences"), i32(r.heads, "heads"), i32(p.heads, "kv_heads"),
          i32(r.dim, "head_dim"), i32(p.block_size, "block_size"), p.blocks, scale, r.type,
          ws.data_ptr(), static_cast<size_t>(ws.numel()), s);
    });
  });
}

int32_t* error_word(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "error_word");
  check(t, "error_word", at::kInt, {1}, dev);
  return ints(t);
}

// address of the pa_plane array, planes, blocks, device, block_size,
// block_tables, context_lens, parents, fresh_blocks, new_block_tables,
// new_context_lens, error_word, stream
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    auto planes = reinterpret_cast<const pa_plane*>(integer(a[0], "planes"));
    const int32_t count = i32(integer(a[1], "planes"), "planes");
    const int64_t blocks = integer(a[2], "blocks");
    const int dev = static_cast<int>(integer(a[3], "device"));
    const int32_t bs = i32(integer(a[4], "block_size"), "block_size");
    const Tensor &bt = tensor(a[5], "block_tables"), &cl = tensor(a[6], "context_lens"),
                 &parents = tensor(a[7], "parents"), &fresh = tensor(a[8], "fresh_blocks"),
                 &nbt = tensor(a[9], "new_block_tables"), &ncl = tensor(a[10], "new_context_lens");
    check(bt, "block_tables", at::kInt, {-1, -1}, dev);
    const int64_t seqs = bt.size(0), width = bt.size(1), children = parents.numel();
    check(cl, "context_lens", at::kInt, {seqs}, dev);
    check(parents, "parents", at::kInt, {children}, dev);
    check(fresh, "fresh_blocks", at::kInt, {children}, dev);
    check(nbt, "new_block_tables", at::kInt, {children, width}, dev);
    check(ncl, "new_context_lens", at::kInt, {children}, dev);
    int32_t* err = error_word(a[11], dev);
    return launch(dev, a[12], [&](pa_stream_t s) {
      return pa_fork_sequences(planes, count, blocks, bs, ints(bt), i32(seqs, "sequences"),
                               i32(width, "max_blocks_per_seq"), ints(cl), ints(parents),
                               ints(fresh), i32(children, "children"), ints(nbt), ints(ncl), err, s);
    });
  });
}

// address of the pa_plane array, planes, blocks, device, moves, block_tables
// (or None), error_word, stream
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    auto planes = reinterpret_cast<const pa_plane*>(integer(a[0], "planes"));
    const int32_t count = i32(integer(a[1], "planes"), "planes");
    const int64_t blocks = integer(a[2], "blocks");
    const int dev = static_cast<int>(integer(a[3], "device"));
    const Tensor& moves = tensor(a[4], "moves");
    check(moves, "moves", at::kInt, {-1, 2}, dev);
    int32_t* table = nullptr;
    int64_t entries = 0;
    if (a[5] != Py_None) {
      const Tensor& bt = tensor(a[5], "block_tables");
      check(bt, "block_tables", at::kInt, {-1, -1}, dev);
      table = ints(bt);
      entries = bt.numel();
    }
    int32_t* err = error_word(a[6], dev);
    return launch(dev, a[7], [&](pa_stream_t s) {
      return pa_compact_blocks(planes, count, blocks, ints(moves), i32(moves.size(0), "moves"),
                               table, entries, err, s);
    });
  });
}

PyMethodDef methods[] = {
    {"write_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(write_rows)), METH_FASTCALL, nullptr},
    {"read_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read_rows)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL, nullptr},
    {"chunked_prefill", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(chunked_prefill)), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fork)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
