// binding.cpp -- the Python binding of the decoder-block entry points as a CPython extension: the
// checks and the marshalling of ops.rotary and of ops.cache_append, cache_attention,
// cache_tree_attention, cache_pages, cache_copy and cache_compact.
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
    case at::kLong: return "torch.int64";
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

// Arguments at[0..3]: k_cache, v_cache, k_scale, v_scale.
b2b_cache pool_of(PyObject* const* at, c10::Device dev) {
  b2b_cache c = {};
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
  return c;
}

// Arguments at[0], at[1]: page_table, lens.
void sequences_of(PyObject* const* at, b2b_cache& c, c10::Device dev) {
  const at::Tensor& table = tensor(at[0], "page_table");
  if (table.dim() != 2)
    throw ValueRefusal("page_table has shape " + text(table.sizes()) + ", expected [sequences, pages]");
  c.batch = narrow(table.size(0), "page_table");
  c.max_pages = narrow(table.size(1), "page_table");
  c.page_table = static_cast<const int32_t*>(dense(table, "page_table", at::kInt, table.sizes(), dev));
  const int64_t B[1] = {table.size(0)};
  c.lens = static_cast<const int32_t*>(dense(tensor(at[1], "lens"), "lens", at::kInt, B, dev));
}

// Arguments at[0..7]: k_cache, v_cache, k_scale, v_scale, page_table, lens, starts, max_new.
b2b_cache cache_of(PyObject* const* at, int64_t T, c10::Device dev) {
  b2b_cache c = pool_of(at, dev);
  sequences_of(at + 4, c, dev);
  const int64_t B1[1] = {static_cast<int64_t>(c.batch) + 1};
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

// Arguments q, cache[0..7], rest[0..5]: scale, softcap, slopes, out, workspace, stream, and for drafted
// trees masks and positions.
PyObject* attention(PyObject* q_at, PyObject* const* cache, PyObject* const* rest, PyObject* masks_at,
                    PyObject* positions_at) {
  const at::Tensor& q = tensor(q_at, "q");
  const b2b_dtype dt = dtype_of(q);
  three(q, "q");
  const c10::Device dev = q.device();
  const int64_t ldq = rows(q, "q", q.scalar_type(), q.sizes(), dev);
  const int64_t T = q.size(0), heads = q.size(1), D = q.size(2);
  const b2b_cache c = cache_of(cache, T, dev);
  if (D != c.head_dim)
    throw ValueRefusal("q has head size " + std::to_string(D) + ", the cache " + std::to_string(c.head_dim));
  const uint64_t* masks = nullptr;
  const int32_t* positions = nullptr;
  int32_t words = 0;
  if (masks_at != nullptr) {
    const at::Tensor& m = tensor(masks_at, "masks");
    if (m.dim() != 2)
      throw ValueRefusal("masks has shape " + text(m.sizes()) + ", expected [rows, words]");
    const int64_t shape[2] = {T, m.size(1)}, rows_of[1] = {T};
    masks = static_cast<const uint64_t*>(dense(m, "masks", at::kLong, shape, dev));
    words = narrow(m.size(1), "masks");
    if (static_cast<int64_t>(words) * 64 < c.max_new)
      throw ValueRefusal("masks has " + std::to_string(words) + " words of 64 bits a row, too few for " +
                         std::to_string(c.max_new) + " new tokens");
    if (positions_at != Py_None)
      positions = static_cast<const int32_t*>(
          dense(tensor(positions_at, "positions"), "positions", at::kInt, rows_of, dev));
  }
  const float scale = static_cast<float>(rest[0] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(rest[0]));
  const int64_t H[1] = {heads};
  const void* slopes =
      rest[2] == Py_None ? nullptr : dense(tensor(rest[2], "slopes"), "slopes", at::kFloat, H, dev);
  void* out = rest[3] == Py_None ? nullptr
                                 : dense(tensor(rest[3], "out"), "out", q.scalar_type(), q.sizes(), dev);
  Place place(dev, rest[5]);
  at::Tensor made, space;
  if (out == nullptr) {
    made = empty(q.sizes(), q.scalar_type(), dev);
    out = made.data_ptr();
  }
  int64_t bytes = 0;
  void* work = nullptr;
  if (rest[4] == Py_None) {
    const b2b_status st =
        (masks_at != nullptr ? b2b_cache_tree_attention_workspace : b2b_cache_attention_workspace)(
            &c, T, narrow(heads, "q"), &bytes);
    if (st != B2B_OK) return PyLong_FromLong(st);
    if (bytes > 0) {
      space = empty({bytes}, at::kByte, dev);
      work = space.data_ptr();
    }
  } else {
    const at::Tensor& w = tensor(rest[4], "workspace");
    bytes = w.numel();
    const int64_t n[1] = {bytes};
    work = dense(w, "workspace", at::kByte, n, dev);
  }
  const float softcap = static_cast<float>(number(rest[1]));
  const auto* bias = static_cast<const float*>(slopes);
  const b2b_status st =
      masks_at != nullptr
          ? b2b_cache_tree_attention(dt, &c, T, q.data_ptr(), ldq, narrow(heads, "q"), masks, words,
                                     positions, scale, softcap, bias, out, work, bytes, place.stream)
          : b2b_cache_attention(dt, &c, T, q.data_ptr(), ldq, narrow(heads, "q"), scale, softcap, bias,
                                out, work, bytes, place.stream);
  return rest[3] == Py_None ? answer(st, made) : answer(st, rest[3]);
}

// cache_attention(q, [cache: 8], scale, softcap, slopes, out, workspace, stream)
PyObject* cache_attention(PyObject* const* a) { return attention(a[0], a + 1, a + 9, nullptr, nullptr); }

// cache_tree_attention(q, masks, [cache: 8], positions, scale, softcap, slopes, out, workspace, stream)
PyObject* cache_tree_attention(PyObject* const* a) { return attention(a[0], a + 2, a + 11, a[1], a[10]); }

PyObject* attention_workspace(PyObject* const* a, bool tree) {
  const at::Tensor& k = tensor(a[2], "k_cache");
  if (!k.is_cuda()) throw ValueRefusal("k_cache must be a CUDA tensor");
  const int64_t T = integer(a[0]);
  const b2b_cache c = cache_of(a + 2, T, k.device());
  c10::cuda::OptionalCUDAGuard device(k.device());
  int64_t bytes = 0;
  const b2b_status st = (tree ? b2b_cache_tree_attention_workspace : b2b_cache_attention_workspace)(
      &c, T, integer32(a[1]), &bytes);
  return PyLong_FromLongLong(st == B2B_OK ? bytes : -static_cast<int64_t>(st));
}

// cache_attention_workspace(T, q_heads, [cache: 8]): bytes, or a negative status; the same for trees
PyObject* cache_attention_workspace(PyObject* const* a) { return attention_workspace(a, false); }
PyObject* cache_tree_attention_workspace(PyObject* const* a) { return attention_workspace(a, true); }

// An optional int32 operand of n elements.
const int32_t* ints(PyObject* o, const char* name, int64_t n, c10::Device dev) {
  const int64_t shape[1] = {n};
  return o == Py_None ? nullptr : static_cast<const int32_t*>(dense(tensor(o, name), name, at::kInt, shape, dev));
}

// cache_pages(page_table, lens, pages, page_size, parents, kept, new, table_out, lens_out, copies, left,
// workspace, stream): the four outputs, all given or all None
PyObject* cache_pages(PyObject* const* a) {
  const at::Tensor& table = tensor(a[0], "page_table");
  if (!table.is_cuda()) throw ValueRefusal("page_table must be a CUDA tensor");
  const c10::Device dev = table.device();
  b2b_cache c = {};
  sequences_of(a, c, dev);
  const int64_t pages = integer(a[2]);
  const int32_t page_size = integer32(a[3]);
  int64_t rows = c.batch;
  static const char* const lists[3] = {"parents", "kept", "new"};
  bool sized = false;
  for (int i = 0; i < 3; ++i) {                      // the first list that is given says how many rows follow
    if (a[4 + i] == Py_None || sized) continue;
    const at::Tensor& t = tensor(a[4 + i], lists[i]);
    if (t.dim() != 1)
      throw ValueRefusal(std::string(lists[i]) + " has shape " + text(t.sizes()) + ", expected one dimension");
    rows = t.size(0);
    sized = true;
  }
  const int32_t* list[3];
  for (int i = 0; i < 3; ++i) list[i] = ints(a[4 + i], lists[i], rows, dev);
  if (a[4] == Py_None && rows != c.batch)
    throw ValueRefusal("without parents each of the " + std::to_string(c.batch) + " sequences is followed, not " +
                       std::to_string(rows));
  const int64_t shapes[4][2] = {{rows, c.max_pages}, {rows, 1}, {rows, 3}, {1, 1}};
  static const int dims[4] = {2, 1, 2, 1};
  static const char* const names[4] = {"the table", "the lengths", "the copies", "the count left"};
  int32_t* out[4];
  const bool own = a[7] == Py_None;
  if (!own)
    for (int i = 0; i < 4; ++i)
      out[i] = static_cast<int32_t*>(dense(tensor(a[7 + i], names[i]), names[i], at::kInt,
                                           at::IntArrayRef(shapes[i], static_cast<size_t>(dims[i])), dev));
  Place place(dev, a[12]);
  at::Tensor made[4], space;
  if (own)
    for (int i = 0; i < 4; ++i) {
      made[i] = empty(at::IntArrayRef(shapes[i], static_cast<size_t>(dims[i])), at::kInt, dev);
      out[i] = static_cast<int32_t*>(made[i].data_ptr());
    }
  int64_t bytes = 0;
  void* work = nullptr;
  if (a[11] == Py_None) {
    const b2b_status st = b2b_cache_pages_workspace(pages, narrow(rows, "the number of rows"), &bytes);
    if (st != B2B_OK) return PyLong_FromLong(st);
    if (bytes > 0) {
      space = empty({bytes}, at::kByte, dev);
      work = space.data_ptr();
    }
  } else {
    const at::Tensor& w = tensor(a[11], "workspace");
    bytes = w.numel();
    const int64_t n[1] = {bytes};
    work = dense(w, "workspace", at::kByte, n, dev);
  }
  const b2b_status st = b2b_cache_pages(
      page_size, pages, c.batch, c.max_pages, c.page_table, c.lens, narrow(rows, "the number of rows"),
      list[0], list[1], list[2], out[0], out[1], out[2], out[3], work, bytes, place.stream);
  if (st != B2B_OK) return PyLong_FromLong(st);
  PyObject* all = PyTuple_New(4);
  if (all == nullptr) throw PythonError();
  for (int i = 0; i < 4; ++i) {
    PyObject* o = own ? THPVariable_Wrap(made[i]) : a[7 + i];
    if (o == nullptr) {
      Py_DECREF(all);
      throw PythonError();
    }
    if (!own) Py_INCREF(o);
    PyTuple_SET_ITEM(all, i, o);
  }
  return all;
}

// cache_copy(k_cache, v_cache, k_scale, v_scale, copies, stream)
PyObject* cache_copy(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k_cache");
  if (!k.is_cuda()) throw ValueRefusal("k_cache must be a CUDA tensor");
  const c10::Device dev = k.device();
  const b2b_cache c = pool_of(a, dev);
  const at::Tensor& copies = tensor(a[4], "copies");
  const int64_t shape[2] = {copies.dim() > 0 ? copies.size(0) : 0, 3};
  const void* pairs = dense(copies, "copies", at::kInt, shape, dev);
  Place place(dev, a[5]);
  return answer(b2b_cache_copy(&c, shape[0], static_cast<const int32_t*>(pairs), place.stream), Py_None);
}

// cache_compact(k_cache, v_cache, k_scale, v_scale, page_table, lens, first, tokens, counts, stream)
PyObject* cache_compact(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k_cache");
  if (!k.is_cuda()) throw ValueRefusal("k_cache must be a CUDA tensor");
  const c10::Device dev = k.device();
  b2b_cache c = pool_of(a, dev);
  sequences_of(a + 4, c, dev);
  if (a[6] == Py_None || a[8] == Py_None) throw TypeRefusal("first and counts must be torch.Tensors");
  const int32_t* first = ints(a[6], "first", c.batch, dev);
  const int32_t* counts = ints(a[8], "counts", c.batch, dev);
  const at::Tensor& tokens = tensor(a[7], "tokens");
  const int64_t shape[2] = {c.batch, tokens.dim() == 2 ? tokens.size(1) : 0};
  const void* kept = dense(tokens, "tokens", at::kInt, shape, dev);
  Place place(dev, a[9]);
  return answer(b2b_cache_compact(&c, first, static_cast<const int32_t*>(kept), narrow(shape[1], "tokens"),
                                  counts, place.stream),
                Py_None);
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
                         ENTRY(cache_attention_workspace, 10), ENTRY(cache_tree_attention, 17),
                         ENTRY(cache_tree_attention_workspace, 10), ENTRY(cache_pages, 13),
                         ENTRY(cache_copy, 6), ENTRY(cache_compact, 10), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
