// binding.cpp -- the Python binding of the decoder-block entry points as a CPython extension: the
// checks and the marshalling of ops.rotary, ops.cache_append and ops.cache_attention.
//
// These run once per token of a generation, on kernels of 2 to 6 us.  Asking a dozen tensors for
// their types, shapes and addresses from Python and handing them over by ctypes took 15 to 21 us a
// call on the GB300's Arm host; here one of one launch takes 4.4 to 5.7.  The functions
// take every argument by position (ops.py gives them names and defaults) and return the output, or
// the status of include/b2b.h if the library refused.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <stdexcept>
#include <string>

#include "b2b.h"

namespace {

struct TypeRefusal : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueRefusal : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};      // an exception that Python has already

std::string text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

const char* dtype_text(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw TypeRefusal(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef sizes) {
  if (!t.is_cuda()) throw ValueRefusal(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() != type)
    throw TypeRefusal(std::string(name) + " has dtype " + dtype_text(t.scalar_type()) + ", expected " +
                      dtype_text(type));
  if (t.sizes() != sizes)
    throw ValueRefusal(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(sizes));
}

void same_device(const at::Tensor& t, const char* name, c10::Device dev) {
  if (t.device() != dev)
    throw ValueRefusal(std::string(name) + " is on " + t.device().str() + ", the other operands on " +
                       dev.str() + ": all operands and the output must be on one device");
}

// A contiguous operand's address.
void* dense(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef sizes,
            c10::Device dev) {
  check(t, name, type, sizes);
  if (!t.is_contiguous()) throw ValueRefusal(std::string(name) + " must be contiguous");
  same_device(t, name, dev);
  return t.data_ptr();
}

// The token stride of a [T, H, D] operand whose heads and channels are dense.
int64_t rows(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef sizes,
             c10::Device dev) {
  check(t, name, type, sizes);
  same_device(t, name, dev);
  const int64_t T = sizes[0], H = sizes[1], D = sizes[2];
  if (t.stride(2) != 1 || (H > 1 && t.stride(1) != D))
    throw ValueRefusal(std::string(name) + " must have dense heads and channels, got strides " +
                       text(t.strides()));
  return T > 1 ? t.stride(0) : H * D;
}

b2b_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kHalf) return B2B_F16;
  if (t.scalar_type() == at::kBFloat16) return B2B_BF16;
  throw TypeRefusal(std::string("expected float16 or bfloat16, got ") + dtype_text(t.scalar_type()));
}

void three(const at::Tensor& t, const char* name) {
  if (t.dim() != 3)
    throw ValueRefusal(std::string(name) + " has shape " + text(t.sizes()) + ", expected three dimensions");
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}
// As integer, for a 32-bit argument of the library; what does not fit is refused there.
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  if (v != static_cast<int32_t>(v)) throw ValueRefusal("an integer argument is out of range");
  return static_cast<int32_t>(v);
}
int32_t narrow(int64_t v, const char* what) {
  if (v > INT32_MAX) throw ValueRefusal(std::string(what) + " is out of range");
  return static_cast<int32_t>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}

// The device of the first operand made current, and the stream of the call: the current one, a
// torch.cuda.Stream or a raw handle.  What the call allocates comes from that stream's memory.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> on;
  cudaStream_t stream;

  Place(c10::Device dev, PyObject* given) {
    device.set_device(dev);
    if (given == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    int64_t handle;
    if (PyLong_Check(given)) {
      handle = integer(given);
    } else {
      PyObject* h = PyObject_GetAttrString(given, "cuda_stream");
      if (h == nullptr) throw PythonError();
      handle = PyLong_AsLongLong(h);
      Py_DECREF(h);
      if (handle == -1 && PyErr_Occurred()) throw PythonError();
    }
    stream = reinterpret_cast<cudaStream_t>(handle);
    on.emplace(c10::cuda::getStreamFromExternal(stream, dev.index()));
  }
};

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(dev));
}

struct Table {
  const float* data = nullptr;
  int64_t positions = 0;
  int32_t rot = 0;
};

Table table_of(PyObject* o, c10::Device dev) {
  Table t;
  if (o == Py_None) return t;
  const at::Tensor& v = tensor(o, "table");
  if (v.dim() != 3 || v.size(2) != 2)
    throw ValueRefusal("table has shape " + text(v.sizes()) + ", expected [positions, rot / 2, 2]");
  t.data = static_cast<const float*>(dense(v, "table", at::kFloat, v.sizes(), dev));
  t.positions = v.size(0);
  t.rot = narrow(2 * v.size(1), "table");
  return t;
}

// Arguments at[0..7]: k_cache, v_cache, k_scale, v_scale, page_table, lens, starts, max_new.
b2b_cache cache_of(PyObject* const* at, int64_t T, c10::Device dev) {
  b2b_cache c;
  const at::Tensor& k = tensor(at[0], "k_cache");
  if (k.dim() != 4)
    throw ValueRefusal("k_cache has shape " + text(k.sizes()) + ", expected [pages, heads, page size, head size]");
  const int64_t scales[2] = {k.size(0), k.size(1)};
  c.k = dense(k, "k_cache", at::kFloat8_e4m3fn, k.sizes(), dev);
  c.v = dense(tensor(at[1], "v_cache"), "v_cache", at::kFloat8_e4m3fn, k.sizes(), dev);
  c.k_scale = static_cast<float*>(dense(tensor(at[2], "k_scale"), "k_scale", at::kFloat, scales, dev));
  c.v_scale = static_cast<float*>(dense(tensor(at[3], "v_scale"), "v_scale", at::kFloat, scales, dev));
  c.pages = k.size(0);
  c.heads = narrow(k.size(1), "k_cache");
  c.page_size = narrow(k.size(2), "k_cache");
  c.head_dim = narrow(k.size(3), "k_cache");
  const at::Tensor& table = tensor(at[4], "page_table");
  if (table.dim() != 2)
    throw ValueRefusal("page_table has shape " + text(table.sizes()) + ", expected [sequences, pages]");
  c.batch = narrow(table.size(0), "page_table");
  c.max_pages = narrow(table.size(1), "page_table");
  c.page_table = static_cast<const int32_t*>(dense(table, "page_table", at::kInt, table.sizes(), dev));
  const int64_t B[1] = {table.size(0)}, B1[1] = {table.size(0) + 1};
  c.lens = static_cast<const int32_t*>(dense(tensor(at[5], "lens"), "lens", at::kInt, B, dev));
  c.starts = at[6] == Py_None
                 ? nullptr
                 : static_cast<const int32_t*>(dense(tensor(at[6], "starts"), "starts", at::kInt, B1, dev));
  if (at[7] == Py_None)
    c.max_new = narrow(c.starts != nullptr ? T : T / (c.batch > 0 ? c.batch : 1), "the number of rows");
  else
    c.max_new = integer32(at[7]);
  return c;
}

PyObject* answer(b2b_status st, const at::Tensor& out) {
  return st == B2B_OK ? THPVariable_Wrap(out) : PyLong_FromLong(st);
}
PyObject* answer(b2b_status st, PyObject* out) {
  if (st != B2B_OK) return PyLong_FromLong(st);
  Py_INCREF(out);
  return out;
}

// rotary(x, table, positions, layout, inverse, out, stream)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const b2b_dtype dt = dtype_of(x);
  three(x, "x");
  const c10::Device dev = x.device();
  const int64_t ldx = rows(x, "x", x.scalar_type(), x.sizes(), dev);
  if (a[1] == Py_None) throw TypeRefusal("table must be a torch.Tensor");
  const Table t = table_of(a[1], dev);
  const int64_t T[1] = {x.size(0)};
  const void* positions = dense(tensor(a[2], "positions"), "positions", at::kInt, T, dev);
  const int64_t row = x.size(1) * x.size(2);
  int64_t ldo = row;
  if (a[5] != Py_None) ldo = rows(tensor(a[5], "out"), "out", x.scalar_type(), x.sizes(), dev);
  Place place(dev, a[6]);
  at::Tensor made;
  if (a[5] == Py_None) made = empty(x.sizes(), x.scalar_type(), dev);
  void* out = a[5] == Py_None ? made.data_ptr() : THPVariable_Unpack(a[5]).data_ptr();
  const b2b_status st = b2b_rotary(
      dt, T[0], narrow(x.size(1), "x"), narrow(x.size(2), "x"), t.rot,
      static_cast<b2b_rotary_layout>(integer32(a[3])), integer32(a[4]), x.data_ptr(), ldx, t.data,
      t.positions, static_cast<const int32_t*>(positions), out, ldo, place.stream);
  return a[5] == Py_None ? answer(st, made) : answer(st, a[5]);
}

// cache_append(k, v, [cache: 8], table, layout, q, q_out, stream)
PyObject* cache_append(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k");
  const b2b_dtype dt = dtype_of(k);
  three(k, "k");
  if (!k.is_cuda()) throw ValueRefusal("k must be a CUDA tensor");
  const c10::Device dev = k.device();
  const int64_t T = k.size(0);
  const b2b_cache c = cache_of(a + 2, T, dev);
  const int64_t shape[3] = {T, c.heads, c.head_dim};
  const int64_t ldk = rows(k, "k", k.scalar_type(), shape, dev);
  const at::Tensor& v = tensor(a[1], "v");
  const int64_t ldv = rows(v, "v", k.scalar_type(), shape, dev);
  const Table t = table_of(a[10], dev);
  const bool queries = a[12] != Py_None, own = queries && a[13] == Py_None;
  if (queries && t.data == nullptr && a[10] == Py_None)
    throw ValueRefusal("q is given to be rotated: it needs a table");
  if (!queries && a[13] != Py_None) throw ValueRefusal("q_out is given without q");
  int64_t ldq = 0, ldqo = 0, q_heads = 0;
  const void* q = nullptr;
  if (queries) {
    const at::Tensor& qt = tensor(a[12], "q");
    three(qt, "q");
    q_heads = qt.size(1);
    const int64_t q_shape[3] = {T, q_heads, c.head_dim};
    ldq = rows(qt, "q", k.scalar_type(), q_shape, dev);
    ldqo = own ? q_heads * c.head_dim : rows(tensor(a[13], "q_out"), "q_out", k.scalar_type(), q_shape, dev);
    q = qt.data_ptr();
  }
  Place place(dev, a[14]);
  at::Tensor made;
  void* q_out = nullptr;
  if (own) made = empty({T, q_heads, c.head_dim}, k.scalar_type(), dev);
  if (queries) q_out = own ? made.data_ptr() : THPVariable_Unpack(a[13]).data_ptr();
  const b2b_status st = b2b_cache_append(
      dt, &c, T, k.data_ptr(), ldk, v.data_ptr(), ldv, t.data, t.positions, t.rot,
      static_cast<b2b_rotary_layout>(integer32(a[11])), q, ldq, narrow(q_heads, "q"), q_out, ldqo,
      place.stream);
  return own ? answer(st, made) : answer(st, a[13]);
}

// cache_attention(q, [cache: 8], scale, softcap, slopes, out, workspace, stream)
PyObject* cache_attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const b2b_dtype dt = dtype_of(q);
  three(q, "q");
  const c10::Device dev = q.device();
  const int64_t ldq = rows(q, "q", q.scalar_type(), q.sizes(), dev);
  const int64_t T = q.size(0), heads = q.size(1), D = q.size(2);
  const b2b_cache c = cache_of(a + 1, T, dev);
  if (D != c.head_dim)
    throw ValueRefusal("q has head size " + std::to_string(D) + ", the cache " + std::to_string(c.head_dim));
  const float scale = static_cast<float>(a[9] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(a[9]));
  const int64_t H[1] = {heads};
  const void* slopes =
      a[11] == Py_None ? nullptr : dense(tensor(a[11], "slopes"), "slopes", at::kFloat, H, dev);
  void* out = a[12] == Py_None ? nullptr
                               : dense(tensor(a[12], "out"), "out", q.scalar_type(), q.sizes(), dev);
  Place place(dev, a[14]);
  at::Tensor made, space;
  if (out == nullptr) {
    made = empty(q.sizes(), q.scalar_type(), dev);
    out = made.data_ptr();
  }
  int64_t bytes = 0;
  void* work = nullptr;
  if (a[13] == Py_None) {
    const b2b_status st = b2b_cache_attention_workspace(&c, T, narrow(heads, "q"), &bytes);
    if (st != B2B_OK) return PyLong_FromLong(st);
    if (bytes > 0) {
      space = empty({bytes}, at::kByte, dev);
      work = space.data_ptr();
    }
  } else {
    const at::Tensor& w = tensor(a[13], "workspace");
    bytes = w.numel();
    const int64_t n[1] = {bytes};
    work = dense(w, "workspace", at::kByte, n, dev);
  }
  const b2b_status st = b2b_cache_attention(
      dt, &c, T, q.data_ptr(), ldq, narrow(heads, "q"), scale, static_cast<float>(number(a[10])),
      static_cast<const float*>(slopes), out, work, bytes, place.stream);
  return a[12] == Py_None ? answer(st, made) : answer(st, a[12]);
}

// cache_attention_workspace(T, q_heads, [cache: 8]): bytes, or a negative status
PyObject* cache_attention_workspace(PyObject* const* a) {
  const at::Tensor& k = tensor(a[2], "k_cache");
  if (!k.is_cuda()) throw ValueRefusal("k_cache must be a CUDA tensor");
  const int64_t T = integer(a[0]);
  const b2b_cache c = cache_of(a + 2, T, k.device());
  c10::cuda::OptionalCUDAGuard device(k.device());
  int64_t bytes = 0;
  const b2b_status st = b2b_cache_attention_workspace(&c, T, integer32(a[1]), &bytes);
  return PyLong_FromLongLong(st == B2B_OK ? bytes : -static_cast<int64_t>(st));
}

// No C++ exception leaves the module: the refusals above as what they are, torch's own (memory that
// has run out, say) as torch's Python functions raise them.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const TypeRefusal& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueRefusal& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const PythonError&) {
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

#define ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(rotary, 7), ENTRY(cache_append, 15), ENTRY(cache_attention, 15),
                         ENTRY(cache_attention_workspace, 10), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
