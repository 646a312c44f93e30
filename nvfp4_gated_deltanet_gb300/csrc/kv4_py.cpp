// The Python face of the kv4_* calls (module _kv4): checks and marshals the
// tensors of kv4.py natively. A decode step's calls take a few microseconds on
// the GPU; through ctypes one of them cost 18 microseconds of host time.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <string>

#include "gdn.h"

namespace {

struct Bad : std::exception {  // -> ValueError
  std::string text;
  explicit Bad(std::string s) : text(std::move(s)) {}
  const char *what() const noexcept override { return text.c_str(); }
};
struct Status : std::exception {  // -> GdnError
  int status;
  const char *call;
  Status(int s, const char *c) : status(s), call(c) {}
};
struct Raised : std::exception {};  // a Python error is set

void check(int status, const char *call) {
  if (status != GDN_OK) throw Status(status, call);
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw Bad(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
int64_t whole(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}
bool given(PyObject *o) { return o != Py_None; }

bool is_bf16(const at::Tensor &t) {
  const auto d = t.scalar_type();
  return d == at::kBFloat16 || d == at::kShort || d == at::kUInt16;
}
const int32_t *i32(PyObject *o, const char *name, int dims) {
  const at::Tensor &t = tensor(o, name);
  if (t.scalar_type() != at::kInt || t.dim() != dims || !t.is_cuda() || !t.is_contiguous())
    throw Bad(std::string(name) + ": expected a contiguous int32 CUDA tensor of " + std::to_string(dims) + " dimension(s)");
  return t.const_data_ptr<int32_t>();
}
int as_int(int64_t v, const char *name) {
  if (v > 0x7fffffffLL) throw Bad(std::string(name) + ": too large");
  return (int)v;
}
int32_t *status_word(PyObject *o) {
  if (!given(o)) return nullptr;
  i32(o, "dev_status", 1);
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.numel() < 1) throw Bad("dev_status: expected one element");
  return t.data_ptr<int32_t>();
}
// A call runs on the device of its first tensor (its pages): every other tensor
// and the stream must be of that device too. With it the current one, the stream
// used by default, the launches and what is kept per device are that device's.
struct Named {
  const char *name;
  PyObject *o;
};
c10::Device device_of(std::initializer_list<Named> tensors, PyObject *stream) {
  const Named &first = *tensors.begin();
  const c10::Device dev = tensor(first.o, first.name).device();
  if (!dev.is_cuda()) throw Bad(std::string(first.name) + ": expected a CUDA tensor");
  for (const Named &t : tensors) {
    if (!given(t.o)) continue;
    const c10::Device d = tensor(t.o, t.name).device();
    if (d != dev)
      throw Bad(std::string(t.name) + ": is on " + d.str() + ", but " + first.name + " is on the CUDA device " + dev.str());
  }
  if (given(stream)) {
    PyObject *v = PyObject_GetAttrString(stream, "device_index");  // torch's streams have one
    if (!v) {
      PyErr_Clear();
      return dev;
    }
    const long long i = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Raised();
    if (i != dev.index())
      throw Bad("stream: is of CUDA device " + std::to_string(i) + ", but " + first.name + " is on " + dev.str());
  }
  return dev;
}
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(c10::Device d) {
    if (c10::cuda::current_device() != d.index()) guard.set_device(d);
  }
};
// The stream on the current device
cudaStream_t stream_of(PyObject *o) {
  if (!given(o)) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject *v = PyObject_GetAttrString(o, "cuda_stream");
  if (!v) throw Raised();
  const unsigned long long s = PyLong_AsUnsignedLongLong(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) throw Raised();
  return reinterpret_cast<cudaStream_t>(s);
}

kv4_cache cache(PyObject *o, PyObject *ks, PyObject *vs) {
  const at::Tensor &p = tensor(o, "pages");
  if (p.scalar_type() != at::kByte || p.dim() != 4 || !p.is_cuda() || !p.is_contiguous())
    throw Bad("pages: expected a contiguous uint8 CUDA tensor [num_pages][Hkv][page_tokens / 16][18 d]");
  if (p.size(3) % 18) throw Bad("pages: the last dimension is 18 * head_dim bytes");
  return {p.data_ptr<uint8_t>(), as_int(p.size(0), "pages"), as_int(16 * p.size(2), "pages"), as_int(p.size(1), "pages"),
          as_int(p.size(3) / 18, "pages"), (float)number(ks), (float)number(vs)};
}
float scale_of(PyObject *o, const kv4_cache &c) { return given(o) ? (float)number(o) : 1.0f / std::sqrt((float)c.head_dim); }
kv4_batch batch(PyObject *table, PyObject *kv_len, PyObject *q_start, int64_t rows) {
  kv4_batch b{};
  b.block_table = i32(table, "block_table", 2);
  b.kv_len = i32(kv_len, "kv_len", 1);
  b.q_start = given(q_start) ? i32(q_start, "q_start", 1) : nullptr;
  const at::Tensor &t = THPVariable_Unpack(table);
  b.B = as_int(t.size(0), "block_table");
  b.max_pages = as_int(t.size(1), "block_table");
  b.T = as_int(rows, "rows");
  if (THPVariable_Unpack(kv_len).size(0) != b.B || (b.q_start && THPVariable_Unpack(q_start).size(0) != b.B + 1))
    throw Bad("block_table, kv_len and q_start disagree on the number of sequences");
  return b;
}
// BF16 rows [T][heads][d] whose heads lie together (heads < 0: any number); the row stride in elements
int64_t rows_stride(const at::Tensor &t, const char *name, int heads, int d) {
  if (!is_bf16(t) || !t.is_cuda() || t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || t.size(2) != d)
    throw Bad(std::string(name) + ": expected BF16 CUDA rows [T][" + (heads >= 0 ? std::to_string(heads) : "heads") + "][" +
              std::to_string(d) + "]");
  if (t.size(0) > 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != d)))
    throw Bad(std::string(name) + ": a row's heads must lie together in memory");
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * d;
}
// A new tensor, without the dispatcher's microsecond
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) {
  return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
// The given output, checked, or a new one of the type. For work on `stream` it is
// allocated as that stream's: a block that the current stream has freed may still
// be in use there, and nothing orders the two. The caller goes on with it on the
// current stream, so it is recorded there.
at::Tensor output(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like,
                  PyObject *stream) {
  if (!given(o)) {
    if (!given(stream)) return fresh(shape, type, like);
    const c10::cuda::CUDAStream here = c10::cuda::getCurrentCUDAStream(like.device().index());
    c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream_of(stream), like.device().index()));
    at::Tensor t = fresh(shape, type, like);
    if (t.numel() > 0) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), here);
    return t;
  }
  const at::Tensor &t = tensor(o, name);
  const bool typed = type == at::kBFloat16 ? is_bf16(t) : t.scalar_type() == type;
  if (!typed || t.sizes() != shape || !t.is_cuda() || !t.is_contiguous())
    throw Bad(std::string(name) + ": expected a contiguous CUDA tensor of its shape and type");
  return t;
}
// Device scratch of n bytes for work on `s`: allocated as that stream's, so that it is reused in its order
at::Tensor workspace(PyObject *o, size_t n, const at::Tensor &like, PyObject *stream, cudaStream_t s, size_t &bytes) {
  if (given(o)) {
    const at::Tensor &t = tensor(o, "workspace");
    if (!t.is_cuda() || !t.is_contiguous()) throw Bad("workspace: expected a contiguous CUDA tensor");
    bytes = t.numel() * t.element_size();
    return t;
  }
  bytes = n;
  if (n == 0) return at::Tensor();
  if (!given(stream)) return fresh({(int64_t)n}, at::kByte, like);
  c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(s, like.device().index()));
  return fresh({(int64_t)n}, at::kByte, like);
}
void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
const uint16_t *u16(const at::Tensor &t) { return static_cast<const uint16_t *>(t.const_data_ptr()); }
uint16_t *u16_out(const at::Tensor &t) { return static_cast<uint16_t *>(t.data_ptr()); }
PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
  PyObject *r = PyTuple_New(2);
  if (!r) throw Raised();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(b));
  return r;
}

// k v pages table kv_len k_scale v_scale q_start dev_status stream
PyObject *append(PyObject *const *a) {
  const OnDevice on(device_of({{"pages", a[2]}, {"k", a[0]}, {"v", a[1]}, {"block_table", a[3]},
                               {"kv_len", a[4]}, {"q_start", a[7]}, {"dev_status", a[8]}}, a[9]));
  const kv4_cache c = cache(a[2], a[5], a[6]);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const int64_t ks = rows_stride(k, "k", c.n_kv_heads, c.head_dim), vs = rows_stride(v, "v", c.n_kv_heads, c.head_dim);
  if (k.size(0) != v.size(0)) throw Bad("k and v have different numbers of rows");
  const kv4_batch b = batch(a[3], a[4], a[7], k.size(0));
  check(kv4_append(&c, &b, u16(k), ks, u16(v), vs, status_word(a[8]), stream_of(a[9])), "kv4_append");
  Py_RETURN_NONE;
}
// pages table kv_len k_scale v_scale rows q_start k v dev_status stream
PyObject *read(PyObject *const *a) {
  const OnDevice on(device_of({{"pages", a[0]}, {"block_table", a[1]}, {"kv_len", a[2]}, {"q_start", a[6]},
                               {"k", a[7]}, {"v", a[8]}, {"dev_status", a[9]}}, a[10]));
  const kv4_cache c = cache(a[0], a[3], a[4]);
  const int64_t rows = whole(a[5]);
  if (rows < 0) throw Bad("rows: expected a number of rows");
  kv4_batch b = batch(a[1], a[2], a[6], rows);
  b.zero_padding = !given(a[7]) | !given(a[8]) << 1;  // rows that nobody writes are zeros in outputs made here
  const int64_t shape[3] = {rows, c.n_kv_heads, c.head_dim};
  const at::Tensor &p = THPVariable_Unpack(a[0]);
  const at::Tensor k = output(a[7], "k", shape, at::kBFloat16, p, a[10]),
                   v = output(a[8], "v", shape, at::kBFloat16, p, a[10]);
  check(kv4_read(&c, &b, u16_out(k), u16_out(v), status_word(a[9]), stream_of(a[10])), "kv4_read");
  return pair(k, v);
}
// q pages table kv_len k_scale v_scale sm_scale out lse return_lse workspace dev_status stream
PyObject *decode(PyObject *const *a) {
  const bool want = truth(a[9]);
  const OnDevice on(device_of({{"pages", a[1]}, {"q", a[0]}, {"block_table", a[2]}, {"kv_len", a[3]},
                               {"out", a[7]}, {"lse", a[8]}, {"workspace", a[10]},
                               {"dev_status", a[11]}}, a[12]));
  const kv4_cache c = cache(a[1], a[4], a[5]);
  const at::Tensor &q = tensor(a[0], "q");
  if (q.dim() != 3 && q.dim() != 4) throw Bad("q: expected [B][Hq][d] or [B][r][Hq][d]");
  const bool four = q.dim() == 4;
  const int64_t B = q.size(0), r = four ? q.size(1) : 1, Hq = q.size(four ? 2 : 1);
  if (!is_bf16(q) || !q.is_cuda() || q.size(-1) != c.head_dim)
    throw Bad("q: expected BF16 CUDA rows [B][heads][" + std::to_string(c.head_dim) + "]");
  if (q.numel() > 0 && (q.stride(-1) != 1 || (Hq > 1 && q.stride(-2) != c.head_dim)))
    throw Bad("q: a row's heads must lie together in memory");
  const int64_t row = r > 1 ? q.stride(1) : B > 1 ? q.stride(0) : Hq * c.head_dim;
  if (r > 1 && B > 1 && q.stride(0) != r * row) throw Bad("q: the rows of all sequences must be evenly spaced");
  const kv4_batch b = batch(a[2], a[3], Py_None, B * r);
  if (b.B != B) throw Bad("q and block_table disagree on the number of sequences");
  const at::Tensor out = output(a[7], "out", q.sizes(), at::kBFloat16, q, a[12]);
  const at::Tensor lse = want || given(a[8]) ? output(a[8], "lse", q.sizes().slice(0, q.dim() - 1), at::kFloat, q, a[12])
                                              : at::Tensor();
  const cudaStream_t s = stream_of(a[12]);
  size_t n;
  const at::Tensor ws = workspace(a[10], kv4_decode_workspace(&c, &b, as_int(Hq, "q")), q, a[12], s, n);
  check(kv4_decode(&c, &b, u16(q), row, as_int(Hq, "q"), scale_of(a[6], c), u16_out(out), static_cast<float *>(ptr(lse)),
                   ptr(ws), n, status_word(a[11]), s),
        "kv4_decode");
  return want ? pair(out, lse) : THPVariable_Wrap(out);
}
// q pages table kv_len q_start k_scale v_scale total_kv sm_scale out lse return_lse workspace dev_status stream
PyObject *prefill(PyObject *const *a) {
  const bool want = truth(a[11]);
  const OnDevice on(device_of({{"pages", a[1]}, {"q", a[0]}, {"block_table", a[2]}, {"kv_len", a[3]},
                               {"q_start", a[4]}, {"out", a[9]}, {"lse", a[10]}, {"workspace", a[12]},
                               {"dev_status", a[13]}}, a[14]));
  const kv4_cache c = cache(a[1], a[5], a[6]);
  const at::Tensor &q = tensor(a[0], "q");
  const int64_t qs = rows_stride(q, "q", -1, c.head_dim);
  const int Hq = as_int(q.size(1), "q");
  kv4_batch b = batch(a[2], a[3], a[4], q.size(0));
  b.zero_padding = !given(a[9]) | !given(a[10]) << 1;
  const int64_t total = given(a[7]) ? whole(a[7]) : (int64_t)b.B * b.max_pages * c.page_tokens;
  const at::Tensor out = output(a[9], "out", q.sizes(), at::kBFloat16, q, a[14]);
  const at::Tensor lse = want || given(a[10]) ? output(a[10], "lse", q.sizes().slice(0, 2), at::kFloat, q, a[14])
                                               : at::Tensor();
  const cudaStream_t s = stream_of(a[14]);
  size_t n;
  const at::Tensor ws = workspace(a[12], kv4_prefill_workspace(&c, &b, total, Hq), q, a[14], s, n);
  check(kv4_prefill(&c, &b, total, u16(q), qs, Hq, scale_of(a[8], c), u16_out(out), static_cast<float *>(ptr(lse)), ptr(ws),
                    n, status_word(a[13]), s),
        "kv4_prefill");
  return want ? pair(out, lse) : THPVariable_Wrap(out);
}

struct Layers {
  uint8_t *p;
  int layers, num;
  int64_t stride, bytes;
};
Layers layers_of(PyObject *o) {
  const at::Tensor &t = tensor(o, "pages");
  if (t.scalar_type() != at::kByte || (t.dim() != 4 && t.dim() != 5) || !t.is_cuda())
    throw Bad("pages: expected a uint8 CUDA tensor [num_pages][Hkv][groups][18 d] or [layers][num_pages]...");
  const int k = (int)t.dim() - 4;
  int64_t size = 1;
  for (int i = 3; i >= 0; --i) {
    if (t.size(i + k) != 1 && t.stride(i + k) != size) throw Bad("pages: a layer's pages must be contiguous");
    if (i > 0) size *= t.size(i + k);
  }
  return {t.data_ptr<uint8_t>(), k ? as_int(t.size(0), "pages") : 1, as_int(t.size(k), "pages"), k ? t.stride(0) : 0, size};
}
// pages src dst dev_status stream
PyObject *copy_pages(PyObject *const *a) {
  const OnDevice on(device_of({{"pages", a[0]}, {"src", a[1]}, {"dst", a[2]}, {"dev_status", a[3]}}, a[4]));
  const Layers l = layers_of(a[0]);
  const int32_t *src = i32(a[1], "src", 1), *dst = i32(a[2], "dst", 1);
  const int64_t n = THPVariable_Unpack(a[1]).size(0);
  if (THPVariable_Unpack(a[2]).size(0) != n) throw Bad("src and dst have different lengths");
  check(kv4_copy_pages(l.p, l.layers, l.stride, l.num, l.bytes, src, dst, as_int(n, "src"), status_word(a[3]), stream_of(a[4])),
        "kv4_copy_pages");
  Py_RETURN_NONE;
}
// pages table tables_out page_map n_live workspace dev_status stream
PyObject *compact(PyObject *const *a) {
  const OnDevice on(device_of({{"pages", a[0]}, {"block_table", a[1]}, {"tables_out", a[2]},
                               {"page_map", a[3]}, {"n_live", a[4]}, {"workspace", a[5]},
                               {"dev_status", a[6]}}, a[7]));
  const Layers l = layers_of(a[0]);
  const int32_t *table = i32(a[1], "block_table", 2);
  const at::Tensor &t = THPVariable_Unpack(a[1]), &p = THPVariable_Unpack(a[0]);
  const int64_t num[1] = {l.num}, one[1] = {1};
  const at::Tensor out = output(a[2], "tables_out", t.sizes(), at::kInt, p, a[7]),
                   map = output(a[3], "page_map", num, at::kInt, p, a[7]),
                   live = output(a[4], "n_live", one, at::kInt, p, a[7]);
  const cudaStream_t s = stream_of(a[7]);
  size_t n;
  const at::Tensor ws = workspace(a[5], kv4_compact_workspace(l.num), p, a[7], s, n);
  check(kv4_compact(l.p, l.layers, l.stride, l.num, l.bytes, table, as_int(t.size(0), "block_table"),
                    as_int(t.size(1), "block_table"), out.data_ptr<int32_t>(), map.data_ptr<int32_t>(),
                    live.data_ptr<int32_t>(), ptr(ws), n, status_word(a[6]), s),
        "kv4_compact");
  PyObject *r = PyTuple_New(3);
  if (!r) throw Raised();
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(map));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(live));
  return r;
}

// No C++ exception crosses into Python.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised &) {
  } catch (const Bad &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Status &e) {
    PyObject *m = PyImport_ImportModule("nvfp4_gated_deltanet_gb300");
    PyObject *cls = m ? PyObject_GetAttrString(m, "GdnError") : nullptr;
    PyObject *v = cls ? PyObject_CallFunction(cls, "is", e.status, e.call) : nullptr;
    if (v) PyErr_SetObject(cls, v);
    Py_XDECREF(v);
    Py_XDECREF(cls);
    Py_XDECREF(m);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define KV4_METHOD(f, n) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {KV4_METHOD(append, 10), KV4_METHOD(read, 11), KV4_METHOD(decode, 13), KV4_METHOD(prefill, 15),
                         KV4_METHOD(copy_pages, 5), KV4_METHOD(compact, 8), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv4", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv4() { return PyModule_Create(&module); }
