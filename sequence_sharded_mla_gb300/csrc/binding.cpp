// Python entry of the rotary, cache-append, shared-prefix, attention-weight,
// eviction and e4m3 grouped-query calls (and the combine that follows them):
// argument checks, output allocation and the C call, without a Python object per
// pointer.  A decode step's calls are a few microseconds of GPU work each, so
// checks written in Python (10 to 30 us a call on the Grace host) would be what
// bounds them.
//
// Every call runs on the tensors' device, on the given stream or the device's
// current one; outputs and workspaces that it allocates belong to that stream.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "mla_dcp.h"

namespace {

PyObject* g_error = nullptr;   // MLAError(status, where)

// A Python exception on its way to the interpreter.
struct Raise {
  PyObject* type;
  std::string what;
};
struct Raised {};              // already set

[[noreturn]] void type_error(const std::string& s) { throw Raise{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Raise{PyExc_ValueError, s}; }

std::string dims_of(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, const char* name, const c10::Device* dev) {
  if (!t.is_cuda()) value_error(std::string(name) + " must be on a CUDA device");
  if (dev != nullptr && t.device() != *dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", expected " + dev->str());
}

// A contiguous tensor of one of `types` with `ndim` dimensions, on `dev` if given.
const at::Tensor& check(PyObject* o, const char* name, std::initializer_list<at::ScalarType> types,
                        int ndim, const c10::Device* dev) {
  const at::Tensor& t = tensor(o, name);
  bool found = false;
  for (at::ScalarType s : types) found |= t.scalar_type() == s;
  if (!found)
    type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + " is not " +
               c10::toString(*types.begin()));
  on_device(t, name, dev);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  if (t.dim() != ndim)
    value_error(std::string(name) + " must have " + std::to_string(ndim) + " dims, got " +
                std::to_string(t.dim()));
  return t;
}

void shape_is(const at::Tensor& t, const char* name, at::IntArrayRef want) {
  if (t.sizes() != want)
    value_error(std::string(name) + " must be " + dims_of(want) + ", got " + dims_of(t.sizes()));
}

// Contiguous memory of `type` that holds a tensor of shape `want`: one of that
// shape, or with more entries in front, or of another number of dimensions.
const at::Tensor& room(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef want,
                       const c10::Device& dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + " is not " +
               c10::toString(type));
  on_device(t, name, &dev);
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  int64_t need = 1;
  for (int64_t n : want) need *= n;
  if (t.numel() < need) value_error(std::string(name) + " is too small");
  if (t.dim() == (int64_t)want.size() && t.sizes().slice(1) != want.slice(1))
    value_error(std::string(name) + " must be " + dims_of(want) + ", got " + dims_of(t.sizes()));
  return t;
}

int to_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v != (int)v) value_error(std::string(name) + " is out of range");
  return (int)v;
}

// A dimension as a C int.
int small(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(std::string(name) + " has too many entries");
  return (int)v;
}

double to_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

bool to_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

struct Ref {                   // an owned Python reference
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) {
    if (p == nullptr) throw Raised{};
  }
  Ref(const Ref&) = delete;
  ~Ref() { Py_DECREF(p); }
};

PyObject* name_of(const char* s) { return PyUnicode_InternFromString(s); }

// Makes a device, and a given stream, current for the call.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard given;
  void* stream;
  Place(const c10::Device& dev, PyObject* s) {
    if (s == Py_None) {
      device.set_device(dev);
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    const c10::cuda::CUDAStream cs = stream_of(dev, s);
    if (cs.device() != dev)
      value_error("stream is on " + cs.device().str() + ", expected " + dev.str());
    given.reset_stream(cs);
    stream = cs.stream();
  }
  // A torch stream, or any object with the CUDA handle of a stream of the
  // device as `cuda_stream`.
  static c10::cuda::CUDAStream stream_of(const c10::Device& dev, PyObject* s) {
    static PyObject* const kId = name_of("stream_id");
    static PyObject* const kIndex = name_of("device_index");
    static PyObject* const kType = name_of("device_type");
    static PyObject* const kHandle = name_of("cuda_stream");
    if (!PyObject_HasAttr(s, kId)) {
      const Ref handle(PyObject_GetAttr(s, kHandle));
      void* const h = PyLong_AsVoidPtr(handle.p);
      if (h == nullptr && PyErr_Occurred()) throw Raised{};
      return c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(h), dev.index());
    }
    const Ref id(PyObject_GetAttr(s, kId)), index(PyObject_GetAttr(s, kIndex)),
        type(PyObject_GetAttr(s, kType));
    const long long i = PyLong_AsLongLong(id.p);
    if (i == -1 && PyErr_Occurred()) throw Raised{};
    return c10::cuda::CUDAStream::unpack3(i, (c10::DeviceIndex)to_int(index.p, "stream"),
                                          (c10::DeviceType)to_int(type.p, "stream"));
  }
};

// A new tensor on the current device and stream (a Place's), without the
// dispatcher: half of torch.empty's 1.5 us.
at::Tensor make(at::IntArrayRef sizes, at::ScalarType t) {
  return at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(),
                                   c10::DispatchKeySet(c10::DispatchKey::CUDA), t, std::nullopt);
}

// `given` if it is not None, else the wrapped `t`: a new reference.
PyObject* give(PyObject* given, const at::Tensor& t) {
  if (given != nullptr && given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw Raised{};
  return o;
}

void status(mla_status st, const char* where) {
  if (st == MLA_OK) return;
  const Ref e(PyObject_CallFunction(g_error, "is", (int)st, where));
  PyErr_SetObject(g_error, e.p);
  throw Raised{};
}

// Runs a C entry without the interpreter lock.
template <class F>
mla_status unlocked(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const mla_status st = f();
  PyEval_RestoreThread(s);
  return st;
}

template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raise& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const Raised&) {
  } catch (const c10::OutOfMemoryError& e) {
    static PyObject* const oom = [] {
      PyObject* m = PyImport_ImportModule("torch");
      PyObject* t = m != nullptr ? PyObject_GetAttrString(m, "OutOfMemoryError") : nullptr;
      Py_XDECREF(m);
      if (t == nullptr) PyErr_Clear();
      return t != nullptr ? t : PyExc_RuntimeError;
    }();
    PyErr_SetString(oom, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

bool want_args(const char* name, Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
  return false;
}

// ------------------------------------------------------------- shared pieces
// Elements between the tokens of t [B, q_len, ...] whose last `dims`
// dimensions are contiguous (a view of a wider projection output will do).
int64_t token_stride(const at::Tensor& t, const char* name, int dims) {
  if (t.scalar_type() != at::kBFloat16)
    type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) +
               " is not BFloat16");
  on_device(t, name, nullptr);
  if (t.dim() != 2 + dims)
    value_error(std::string(name) + " must have " + std::to_string(2 + dims) + " dims, got " +
                std::to_string(t.dim()));
  int64_t width = 1;
  for (int d = 1 + dims; d > 1; --d) {
    if (t.size(d) != 1 && t.stride(d) != width)
      value_error(std::string(name) + ": a token's values must be contiguous");
    width *= t.size(d);
  }
  const int64_t B = t.size(0), q_len = t.size(1);
  if (t.is_contiguous()) return width;
  const int64_t step = q_len > 1 ? t.stride(1) : B > 1 ? t.stride(0) : width;
  if (q_len > 1 && B > 1 && t.stride(0) != q_len * step)
    value_error(std::string(name) + ": tokens must be evenly spaced");
  if (t.numel() > 0 && step < width) value_error(std::string(name) + ": tokens overlap");
  return step;
}

struct RopeArg {
  mla_rope r;
  bool given;
};

RopeArg rope_arg(PyObject* o, const c10::Device& dev) {
  RopeArg a{};
  if (o == Py_None) return a;
  static PyObject* const kInv = name_of("inv_freq");
  static PyObject* const kFirst = name_of("first_dim");
  static PyObject* const kInter = name_of("interleaved");
  static PyObject* const kFactor = name_of("attention_factor");
  const Ref inv(PyObject_GetAttr(o, kInv)), first(PyObject_GetAttr(o, kFirst)),
      inter(PyObject_GetAttr(o, kInter)), factor(PyObject_GetAttr(o, kFactor));
  const at::Tensor& t = check(inv.p, "rope.inv_freq", {at::kDouble}, 1, &dev);
  a.given = true;
  a.r.inv_freq = t.const_data_ptr<double>();
  a.r.rot_dim = small(2 * t.numel(), "rope.inv_freq");
  a.r.first_dim = to_int(first.p, "rope.first_dim");
  a.r.interleaved = to_bool(inter.p);
  a.r.attention_factor = (float)to_double(factor.p);
  return a;
}

const int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape, const c10::Device& dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = check(o, name, {at::kInt}, (int)shape.size(), &dev);
  shape_is(t, name, shape);
  return t.const_data_ptr<int32_t>();
}

mla_tokens tokens_arg(int64_t B, int64_t q_len, PyObject* seq_lens, PyObject* q_lens,
                      PyObject* positions, const c10::Device& dev) {
  mla_tokens t;
  t.batch = small(B, "the batch");
  t.q_len = small(q_len, "q_len");
  t.seq_lens = ints(seq_lens, "seq_lens", {B}, dev);
  t.q_lens = ints(q_lens, "q_lens", {B}, dev);
  t.positions = ints(positions, "positions", {B, q_len}, dev);
  return t;
}

// Rows to rotate: x and where they go.
struct RowsArg {
  const at::Tensor* x = nullptr;
  at::Tensor out;
  int64_t xs = 0, ys = 0;
};

// `out` checked (x itself, or memory of its own); a new tensor comes later.
RowsArg rows_arg(PyObject* px, PyObject* pout, const char* name) {
  RowsArg r;
  r.x = &tensor(px, name);
  r.xs = r.ys = token_stride(*r.x, name, 2);
  if (pout == Py_None) {
    r.ys = r.x->size(2) * r.x->size(3);
    return r;
  }
  const std::string oname = std::string(name) + "_out";
  r.out = tensor(pout, oname.c_str());
  if (pout == px) return r;
  r.ys = token_stride(r.out, oname.c_str(), 2);
  shape_is(r.out, oname.c_str(), r.x->sizes());
  if (r.out.device() != r.x->device())
    value_error(oname + " is on " + r.out.device().str() + ", expected " + r.x->device().str());
  const auto a = (uintptr_t)r.x->const_data_ptr(), b = (uintptr_t)r.out.const_data_ptr();
  if (a == b) {
    if (r.xs != r.ys && r.x->size(0) * r.x->size(1) > 1)
      value_error(oname + " overlaps " + name + " with other strides");
    r.ys = r.xs;
  } else if (r.x->numel() > 0) {
    // the bytes from the first token to the end of the last; with equal strides
    // they may be columns of one tensor, apart in every token
    const int64_t last = r.x->size(0) * r.x->size(1) - 1, width = r.x->size(2) * r.x->size(3);
    if (a < b + 2 * (last * r.ys + width) && b < a + 2 * (last * r.xs + width)) {
      const int64_t step = 2 * r.xs, gap = (int64_t)(a < b ? b - a : a - b) % step;
      if (r.xs != r.ys || gap < 2 * width || step - gap < 2 * width)
        value_error(oname + " overlaps " + name);
    }
  }
  return r;
}

// The gqa_block_pages descriptor of an e4m3 (or bf16, without scales) cache.
gqa_block_pages block_pages(PyObject* pk, PyObject* pv, PyObject* pks, PyObject* pvs,
                            const c10::Device& dev) {
  const at::Tensor& k = tensor(pk, "k_cache");
  const bool bf16 = k.scalar_type() == at::kBFloat16;
  if (bf16) {
    if (pks != Py_None || pvs != Py_None)
      value_error("k_scale and v_scale are only for fp8 caches");
    check(pk, "k_cache", {at::kBFloat16}, 4, &dev);
  } else {
    check(pk, "k_cache", {at::kFloat8_e4m3fn, at::kByte}, 4, &dev);
  }
  const at::Tensor& v = check(pv, "v_cache", {k.scalar_type()}, 4, &dev);
  shape_is(v, "v_cache", k.sizes());
  if (k.size(3) != 128) value_error("k_cache and v_cache must be [P, 64, Hkv, 128]");
  gqa_block_pages p{};
  p.k = k.mutable_data_ptr();
  p.v = v.mutable_data_ptr();
  p.dtype = bf16 ? MLA_KV_BF16 : MLA_KV_FP8_E4M3;
  p.num_pages = small(k.size(0), "k_cache");
  p.page_size = small(k.size(1), "k_cache");
  p.num_kv_heads = small(k.size(2), "k_cache");
  if (bf16) return p;
  if (pks == Py_None || pvs == Py_None) value_error("fp8 caches need k_scale and v_scale");
  const at::Tensor& ks = check(pks, "k_scale", {at::kFloat}, 3, &dev);
  const at::Tensor& vs = check(pvs, "v_scale", {at::kFloat}, 3, &dev);
  const int64_t n = ks.size(1);
  if (n < 1 || k.size(1) % n != 0) value_error("k_scale must be [P, 64 / block, Hkv]");
  p.block = (int)(k.size(1) / n);
  shape_is(ks, "k_scale", {k.size(0), n, k.size(2)});
  shape_is(vs, "v_scale", {k.size(0), n, k.size(2)});
  p.k_scale = ks.mutable_data_ptr<float>();
  p.v_scale = vs.mutable_data_ptr<float>();
  return p;
}

// The mla_kv_pages descriptor of a bf16 or e4m3 latent cache.
mla_kv_pages latent_pages(PyObject* pkv, PyObject* pscale, const c10::Device& dev) {
  const at::Tensor& kv = tensor(pkv, "kv");
  mla_kv_pages pages{};
  if (kv.scalar_type() == at::kBFloat16) {
    if (pscale != Py_None) value_error("kv_scale is only for fp8 caches");
    pages.dtype = MLA_KV_BF16;
  } else if (kv.scalar_type() == at::kByte || kv.scalar_type() == at::kFloat8_e4m3fn) {
    if (pscale == Py_None) value_error("fp8 caches need kv_scale");
    pages.dtype = MLA_KV_FP8_E4M3;
  } else {
    type_error(std::string("kv dtype ") + c10::toString(kv.scalar_type()) + " unsupported");
  }
  check(pkv, "kv", {kv.scalar_type()}, 3, &dev);
  if (kv.size(1) != 64 || kv.size(2) != 576) value_error("kv must be [P, 64, 576]");
  pages.data = kv.mutable_data_ptr();
  pages.num_pages = small(kv.size(0), "kv");
  pages.page_size = 64;
  if (pscale != Py_None) {
    const at::Tensor& sc = check(pscale, "kv_scale", {at::kFloat}, 2, &dev);
    shape_is(sc, "kv_scale", {kv.size(0), kv.size(1)});
    pages.scale = sc.mutable_data_ptr<float>();
  }
  return pages;
}

// fp32 rows [B, width] whose values are contiguous; floats between rows.
int64_t row_stride(const at::Tensor& t, const char* name, int64_t B, const c10::Device& dev) {
  if (t.scalar_type() != at::kFloat)
    type_error(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + " is not Float");
  on_device(t, name, &dev);
  if (t.dim() != 2 || t.size(0) != B)
    value_error(std::string(name) + " must be [B, width] with the batch of seq_lens");
  if (t.size(1) > 1 && t.stride(1) != 1)
    value_error(std::string(name) + ": a request's values must be contiguous");
  const int64_t step = B > 1 ? t.stride(0) : t.size(1);
  if (step < t.size(1)) value_error(std::string(name) + ": rows overlap");
  return step;
}

// What both cache appends take besides the cache and the new rows.
struct Append {
  const int32_t* block_table;
  int max_pages, shard_id, num_shards, heads = 0;
  mla_tokens tok;
  RopeArg rope;
  RowsArg q;
  PyObject *pq, *pq_out, *pws, *pstream;
};

// a: block_table, seq_lens, rope, q, q_out, q_lens, positions, shard_id,
// num_shards, workspace, stream
Append append_arg(PyObject* const* a, int64_t B, int64_t q_len, int64_t width,
                  const c10::Device& dev) {
  Append p;
  const at::Tensor& bt = check(a[0], "block_table", {at::kInt}, 2, &dev);
  if (a[1] == Py_None) type_error("seq_lens must be a torch.Tensor");
  if (bt.size(0) != B)
    value_error("block_table and the new tokens disagree on the number of requests");
  p.block_table = bt.const_data_ptr<int32_t>();
  p.max_pages = small(bt.size(1), "block_table");
  p.tok = tokens_arg(B, q_len, a[1], a[5], a[6], dev);
  p.rope = rope_arg(a[2], dev);
  p.pq = a[3];
  p.pq_out = a[4];
  if (a[3] == Py_None) {
    if (a[4] != Py_None) value_error("q_out without q");
  } else {
    p.q = rows_arg(a[3], a[4], "q");
    if (p.q.x->device() != dev)
      value_error("q is on " + p.q.x->device().str() + ", expected " + dev.str());
    shape_is(*p.q.x, "q", {B, q_len, p.q.x->size(2), width});
    p.heads = small(p.q.x->size(2), "q");
  }
  p.shard_id = to_int(a[7], "shard_id");
  p.num_shards = to_int(a[8], "num_shards");
  p.pws = a[9];
  p.pstream = a[10];
  if (a[9] != Py_None) check(a[9], "workspace", {at::kByte}, 1, &dev);
  return p;
}

// Allocates what the caller left out, runs `call`, and answers (q_out, workspace).
template <class F>
PyObject* run_append(Append& p, const c10::Device& dev, const char* where, F&& call) {
  const Place place(dev, p.pstream);
  at::Tensor ws;
  if (p.pws != Py_None) ws = THPVariable_Unpack(p.pws);
  else ws = at::zeros({256}, at::TensorOptions().dtype(at::kByte).device(dev));
  if (p.q.x != nullptr && !p.q.out.defined()) p.q.out = make(p.q.x->sizes(), at::kBFloat16);
  const void* q = p.q.x != nullptr ? p.q.x->const_data_ptr() : nullptr;
  void* q_out = p.q.x != nullptr ? p.q.out.mutable_data_ptr() : nullptr;
  void* wp = ws.mutable_data_ptr();
  const size_t wb = (size_t)ws.numel();
  const mla_rope* rope = p.rope.given ? &p.rope.r : nullptr;
  status(unlocked([&] { return call(q, q_out, rope, wp, wb, place.stream); }), where);
  PyObject* first = Py_None;
  if (p.pq == Py_None) Py_INCREF(first);
  else first = give(p.pq_out, p.q.out);
  const Ref a(first), b(give(p.pws, ws));
  return PyTuple_Pack(2, a.p, b.p);
}

// ------------------------------------------------------------------ entries
// x, rope, seq_lens, q_lens, positions, out, stream
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("rope_apply", n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    RowsArg r = rows_arg(a[0], a[5], "x");
    const c10::Device dev = r.x->device();
    if (a[2] == Py_None && a[4] == Py_None) value_error("give seq_lens or positions");
    const mla_tokens tok = tokens_arg(r.x->size(0), r.x->size(1), a[2], a[3], a[4], dev);
    if (a[1] == Py_None) type_error("rope must be a Rope");
    const RopeArg rope = rope_arg(a[1], dev);
    const int H = small(r.x->size(2), "x"), D = small(r.x->size(3), "x");
    const Place place(dev, a[6]);
    if (!r.out.defined()) r.out = make(r.x->sizes(), at::kBFloat16);
    const void* x = r.x->const_data_ptr();
    void* y = r.out.mutable_data_ptr();
    status(unlocked([&] {
             return mla_rope_apply(x, r.xs, y, r.ys, &tok, H, D, &rope.r, place.stream);
           }),
           "mla_rope_apply");
    return give(a[5], r.out);
  });
}

// latent, kv, kv_scale, then as append_arg
PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("latent_append", n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "latent");
    const int64_t xs = token_stride(x, "latent", 1);
    const c10::Device dev = x.device();
    if (x.size(2) != 576) value_error("latent must be [B, q_len, 576]");
    const mla_kv_pages pages = latent_pages(a[1], a[2], dev);
    Append p = append_arg(a + 3, x.size(0), x.size(1), 576, dev);
    const void* xp = x.const_data_ptr();
    return run_append(p, dev, "mla_cache_append",
                      [&](const void* q, void* q_out, const mla_rope* rope, void* ws, size_t wb,
                          void* stream) {
                        return mla_cache_append(xp, xs, &pages, p.block_table, p.max_pages, &p.tok,
                                                rope, q, p.q.xs, q_out, p.q.ys, p.heads,
                                                p.shard_id, p.num_shards, ws, wb, stream);
                      });
  });
}

// k, v, k_cache, v_cache, k_scale, v_scale, then as append_arg
PyObject* heads_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("heads_append", n, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int64_t ks = token_stride(k, "k", 2), vs = token_stride(v, "v", 2);
    const c10::Device dev = k.device();
    on_device(v, "v", &dev);
    shape_is(v, "v", k.sizes());
    const gqa_block_pages pages = block_pages(a[2], a[3], a[4], a[5], dev);
    shape_is(k, "k", {k.size(0), k.size(1), pages.num_kv_heads, 128});
    Append p = append_arg(a + 6, k.size(0), k.size(1), 128, dev);
    const void *kp = k.const_data_ptr(), *vp = v.const_data_ptr();
    return run_append(p, dev, "gqa_cache_append",
                      [&](const void* q, void* q_out, const mla_rope* rope, void* ws, size_t wb,
                          void* stream) {
                        return gqa_cache_append(kp, ks, vp, vs, &pages, p.block_table, p.max_pages,
                                                &p.tok, rope, q, p.q.xs, q_out, p.q.ys, p.heads,
                                                p.shard_id, p.num_shards, ws, wb, stream);
                      });
  });
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, num_shards,
// layout (number), shard_id, causal, softmax_scale, out_partial, lse_partial,
// workspace, stream, q_lens
PyObject* attend_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("attend_fp8", n, 17)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = check(a[0], "q", {at::kBFloat16}, 4, nullptr);
    const c10::Device dev = q.device();
    const int64_t B = q.size(0), q_len = q.size(1), H = q.size(2), D = q.size(3);
    if (tensor(a[1], "k_cache").scalar_type() == at::kBFloat16)
      type_error("k_cache must hold e4m3 codes; gqa_decode_partial takes bf16 caches");
    const gqa_block_pages pages = block_pages(a[1], a[2], a[3], a[4], dev);
    const at::Tensor& bt = check(a[5], "block_table", {at::kInt}, 2, &dev);
    const at::Tensor& sl = check(a[6], "seq_lens", {at::kInt}, 1, &dev);
    if (bt.size(0) != B || sl.size(0) != B)
      value_error("q, block_table and seq_lens disagree on the number of requests");
    const int32_t* q_lens = ints(a[16], "q_lens", {B}, dev);
    const int num_shards = to_int(a[7], "num_shards"), layout = to_int(a[8], "layout");
    const int shard_id = to_int(a[9], "shard_id");
    gqa_shape sh{};
    sh.batch = small(B, "q");
    sh.q_len = small(q_len, "q");
    sh.num_heads = small(H, "q");
    sh.num_kv_heads = pages.num_kv_heads;
    sh.head_dim = small(D, "q");
    sh.causal = to_bool(a[10]);
    sh.softmax_scale =
        a[11] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)to_double(a[11]);
    const int64_t n_out = shard_id == MLA_ALL_SHARDS ? std::max(num_shards, 1) : 1;
    at::Tensor out, lse, ws;
    if (a[12] != Py_None) {
      out = check(a[12], "out_partial", {at::kFloat}, 5, &dev);
      shape_is(out, "out_partial", {n_out, B, q_len, H, D});
    }
    if (a[13] != Py_None) {
      lse = check(a[13], "lse_partial", {at::kFloat}, 4, &dev);
      shape_is(lse, "lse_partial", {n_out, B, q_len, H});
    }
    if (a[14] != Py_None) ws = check(a[14], "workspace", {at::kByte}, 1, &dev);
    const Place place(dev, a[15]);
    if (!ws.defined()) {
      const size_t need = gqa_fp8_workspace_size(&sh, num_shards, shard_id);
      ws = make({(int64_t)std::max(need, (size_t)256)}, at::kByte);
    }
    // refused shapes come back as a status before anything is written
    if (num_shards <= 8) {
      if (!out.defined()) out = make({n_out, B, q_len, H, D}, at::kFloat);
      if (!lse.defined()) lse = make({n_out, B, q_len, H}, at::kFloat);
    }
    const void* qp = q.const_data_ptr();
    const int32_t *btp = bt.const_data_ptr<int32_t>(), *slp = sl.const_data_ptr<int32_t>();
    const int max_pages = small(bt.size(1), "block_table");
    float* op = out.defined() ? out.mutable_data_ptr<float>() : nullptr;
    float* lp = lse.defined() ? lse.mutable_data_ptr<float>() : nullptr;
    void* wp = ws.mutable_data_ptr();
    const size_t wb = (size_t)ws.numel();
    status(unlocked([&] {
             return gqa_decode_partial_fp8(qp, &pages, btp, max_pages, slp, q_lens, &sh, shard_id,
                                           num_shards, (mla_layout)layout, op, lp, wp, wb,
                                           place.stream);
           }),
           "gqa_decode_partial_fp8");
    const Ref r0(give(a[12], out)), r1(give(a[13], lse)), r2(give(a[14], ws));
    return PyTuple_Pack(3, r0.p, r1.p, r2.p);
  });
}

// partials, lses, out, lse_out, stream
PyObject* shard_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("shard_combine", n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& p = check(a[0], "partials", {at::kFloat}, 5, nullptr);
    const c10::Device dev = p.device();
    const at::Tensor& l = check(a[1], "lses", {at::kFloat}, 4, &dev);
    const int64_t B = p.size(1), q_len = p.size(2), H = p.size(3), D = p.size(4);
    gqa_shape sh{};
    sh.batch = small(B, "partials");
    sh.q_len = small(q_len, "partials");
    sh.num_heads = small(H, "partials");
    sh.num_kv_heads = 1;
    sh.head_dim = small(D, "partials");
    sh.softmax_scale = 1.0f;
    const int N = small(p.size(0), "partials");
    at::Tensor out, lse;
    shape_is(l, "lses", {N, B, q_len, H});
    if (a[2] != Py_None) out = room(a[2], "out", at::kBFloat16, {B, q_len, H, D}, dev);
    if (a[3] != Py_None) lse = room(a[3], "lse_out", at::kFloat, {B, q_len, H}, dev);
    const Place place(dev, a[4]);
    if (!out.defined()) out = make({B, q_len, H, D}, at::kBFloat16);
    if (!lse.defined()) lse = make({B, q_len, H}, at::kFloat);
    const float *pp = p.const_data_ptr<float>(), *lp = l.const_data_ptr<float>();
    void* op = out.mutable_data_ptr();
    float* lo = static_cast<float*>(lse.mutable_data_ptr());
    status(unlocked([&] { return gqa_shard_combine(pp, lp, N, &sh, op, lo, place.stream); }),
           "gqa_shard_combine");
    const Ref r0(give(a[2], out)), r1(give(a[3], lse));
    return PyTuple_Pack(2, r0.p, r1.p);
  });
}

// A latent step's shape from q [B, q_len, H, 576].
mla_shape latent_shape(const at::Tensor& q, PyObject* causal, PyObject* scale, const int32_t* q_lens) {
  if (q.size(3) != 576) value_error("q must be [B, q_len, H, 576]");
  mla_shape sh{};
  sh.batch = small(q.size(0), "q");
  sh.q_len = small(q.size(1), "q");
  sh.num_heads = small(q.size(2), "q");
  sh.causal = to_bool(causal);
  sh.softmax_scale = (float)to_double(scale);
  sh.q_lens = q_lens;
  return sh;
}

// q, kv, kv_scale, block_table, seq_lens, group_starts, prefix_lens, causal,
// softmax_scale, out_partial, lse_partial, workspace, stream, q_lens
PyObject* prefix_partial(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("prefix_partial", n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = check(a[0], "q", {at::kBFloat16}, 4, nullptr);
    const c10::Device dev = q.device();
    const int64_t B = q.size(0);
    const mla_kv_pages pages = latent_pages(a[1], a[2], dev);
    const at::Tensor& bt = check(a[3], "block_table", {at::kInt}, 2, &dev);
    const at::Tensor& sl = check(a[4], "seq_lens", {at::kInt}, 1, &dev);
    if (bt.size(0) != B || sl.size(0) != B)
      value_error("q, block_table and seq_lens disagree on the number of requests");
    const mla_shape sh = latent_shape(q, a[7], a[8], ints(a[13], "q_lens", {B}, dev));
    const at::Tensor& pl = check(a[6], "prefix_lens", {at::kInt}, 1, &dev);
    const at::Tensor& gs = check(a[5], "group_starts", {at::kInt}, 1, &dev);
    shape_is(gs, "group_starts", {pl.size(0) + 1});
    at::Tensor out, lse, ws;
    const int64_t ql = q.size(1), H = q.size(2);
    if (a[9] != Py_None) {
      out = check(a[9], "out_partial", {at::kFloat}, 5, &dev);
      shape_is(out, "out_partial", {2, B, ql, H, 512});
    }
    if (a[10] != Py_None) {
      lse = check(a[10], "lse_partial", {at::kFloat}, 4, &dev);
      shape_is(lse, "lse_partial", {2, B, ql, H});
    }
    if (a[11] != Py_None) ws = check(a[11], "workspace", {at::kByte}, 1, &dev);
    const int groups = small(pl.size(0), "prefix_lens"), mp = small(bt.size(1), "block_table");
    const Place place(dev, a[12]);
    if (!ws.defined()) {
      const size_t need = mla_prefix_workspace_size(&sh, groups, mp, pages.dtype);
      ws = make({(int64_t)std::max(need, (size_t)256)}, at::kByte);
    }
    if (!out.defined()) out = make({2, B, ql, H, 512}, at::kFloat);
    if (!lse.defined()) lse = make({2, B, ql, H}, at::kFloat);
    const void* qp = q.const_data_ptr();
    const int32_t *btp = bt.const_data_ptr<int32_t>(), *slp = sl.const_data_ptr<int32_t>();
    const int32_t *gp = gs.const_data_ptr<int32_t>(), *pp = pl.const_data_ptr<int32_t>();
    float *op = out.mutable_data_ptr<float>(), *lp = lse.mutable_data_ptr<float>();
    void* wp = ws.mutable_data_ptr();
    const size_t wb = (size_t)ws.numel();
    status(unlocked([&] {
             return mla_prefix_partial(qp, &pages, btp, mp, slp, &sh, gp, pp, groups, op, lp, wp, wb,
                                       place.stream);
           }),
           "mla_prefix_partial");
    const Ref r0(give(a[9], out)), r1(give(a[10], lse)), r2(give(a[11], ws));
    return PyTuple_Pack(3, r0.p, r1.p, r2.p);
  });
}

// q, kv, kv_scale, block_table, seq_lens, lse, weights, out, causal,
// softmax_scale, q_lens, workspace, stream
PyObject* attention_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("attention_weights", n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& q = check(a[0], "q", {at::kBFloat16}, 4, nullptr);
    const c10::Device dev = q.device();
    const int64_t B = q.size(0);
    const mla_kv_pages pages = latent_pages(a[1], a[2], dev);
    const at::Tensor& bt = check(a[3], "block_table", {at::kInt}, 2, &dev);
    const at::Tensor& sl = check(a[4], "seq_lens", {at::kInt}, 1, &dev);
    if (bt.size(0) != B || sl.size(0) != B)
      value_error("q, block_table and seq_lens disagree on the number of requests");
    const mla_shape sh = latent_shape(q, a[8], a[9], ints(a[10], "q_lens", {B}, dev));
    const at::Tensor& lse = check(a[5], "lse", {at::kFloat}, 3, &dev);
    shape_is(lse, "lse", q.sizes().slice(0, 3));
    at::Tensor before, out, ws;
    int64_t bs = 0, os = 0;
    if (a[6] != Py_None) {
      before = tensor(a[6], "weights");
      bs = row_stride(before, "weights", B, dev);
    }
    if (a[7] != Py_None) {
      out = tensor(a[7], "out");
      os = row_stride(out, "out", B, dev);
      if (before.defined()) shape_is(before, "weights", out.sizes());
    }
    const int64_t width = out.defined() ? out.size(1) : before.defined() ? before.size(1) : bt.size(1) * 64;
    if (a[11] != Py_None) ws = check(a[11], "workspace", {at::kByte}, 1, &dev);
    const int w = small(width, "weights"), mp = small(bt.size(1), "block_table");
    const Place place(dev, a[12]);
    if (!ws.defined()) {
      const size_t need = mla_attention_weights_workspace_size(&sh, pages.dtype);
      ws = make({(int64_t)std::max(need, (size_t)256)}, at::kByte);
    }
    if (!out.defined()) {
      out = at::zeros({B, width}, at::TensorOptions().dtype(at::kFloat).device(dev));
      os = width;
    }
    const void* qp = q.const_data_ptr();
    const int32_t *btp = bt.const_data_ptr<int32_t>(), *slp = sl.const_data_ptr<int32_t>();
    const float* lp = lse.const_data_ptr<float>();
    const float* bp = before.defined() ? before.const_data_ptr<float>() : nullptr;
    float* op = out.mutable_data_ptr<float>();
    void* wp = ws.mutable_data_ptr();
    const size_t wb = (size_t)ws.numel();
    status(unlocked([&] {
             return mla_attention_weights(qp, &pages, btp, mp, slp, &sh, lp, bp, bs, op, os, w, wp,
                                          wb, place.stream);
           }),
           "mla_attention_weights");
    const Ref r0(give(a[7], out)), r1(give(a[11], ws));
    return PyTuple_Pack(2, r0.p, r1.p);
  });
}

// kv, kv_scale, block_table, seq_lens, weights, keep, new_block_table,
// keep_first, recent, kept, new_seq_lens, weights_out, workspace, stream
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!want_args("cache_evict", n, 14)) return nullptr;
  return guarded([&]() -> PyObject* {
    on_device(tensor(a[0], "kv"), "kv", nullptr);
    const c10::Device dev = THPVariable_Unpack(a[0]).device();
    const mla_kv_pages pages = latent_pages(a[0], a[1], dev);
    const at::Tensor& sl = check(a[3], "seq_lens", {at::kInt}, 1, &dev);
    const int64_t B = sl.size(0);
    const at::Tensor& bt = check(a[2], "block_table", {at::kInt}, 2, &dev);
    const at::Tensor& nbt = check(a[6], "new_block_table", {at::kInt}, 2, &dev);
    if (bt.size(0) != B || nbt.size(0) != B)
      value_error("block_table, new_block_table and seq_lens disagree on the number of requests");
    const at::Tensor& w = tensor(a[4], "weights");
    const int64_t step = row_stride(w, "weights", B, dev);
    if (a[5] == Py_None) type_error("keep must be a torch.Tensor");
    const int32_t* keep = ints(a[5], "keep", {B}, dev);
    const int32_t* first = ints(a[7], "keep_first", {B}, dev);
    const int recent = to_int(a[8], "recent");
    at::Tensor kept, lens, wo, ws;
    if (a[9] != Py_None) {
      kept = check(a[9], "kept", {at::kInt}, 2, &dev);
      if (kept.size(0) != B) value_error("kept must have a row for every request");
    }
    const int64_t max_keep = kept.defined() ? kept.size(1) : nbt.size(1) * 64;
    if (a[10] != Py_None) {
      lens = check(a[10], "new_seq_lens", {at::kInt}, 1, &dev);
      shape_is(lens, "new_seq_lens", {B});
    }
    if (a[11] != Py_None) {
      wo = check(a[11], "weights_out", {at::kFloat}, 2, &dev);
      shape_is(wo, "weights_out", {B, max_keep});
    }
    if (a[12] != Py_None) ws = check(a[12], "workspace", {at::kByte}, 1, &dev);
    const int batch = small(B, "seq_lens"), mk = small(max_keep, "kept");
    const int width = small(w.size(1), "weights"), mp = small(bt.size(1), "block_table");
    const int nmp = small(nbt.size(1), "new_block_table");
    const Place place(dev, a[13]);
    if (!ws.defined()) ws = at::zeros({256}, at::TensorOptions().dtype(at::kByte).device(dev));
    if (!kept.defined()) kept = make({B, max_keep}, at::kInt);
    if (!lens.defined()) lens = make({B}, at::kInt);
    if (!wo.defined()) wo = make({B, max_keep}, at::kFloat);
    const int32_t *btp = bt.const_data_ptr<int32_t>(), *nbp = nbt.const_data_ptr<int32_t>();
    const int32_t* slp = sl.const_data_ptr<int32_t>();
    const float* wp = w.const_data_ptr<float>();
    int32_t *lp = lens.mutable_data_ptr<int32_t>(), *kp = kept.mutable_data_ptr<int32_t>();
    float* wop = wo.mutable_data_ptr<float>();
    void* wsp = ws.mutable_data_ptr();
    const size_t wb = (size_t)ws.numel();
    status(unlocked([&] {
             return mla_cache_evict(&pages, btp, mp, slp, batch, wp, step, width, keep, first,
                                    recent, nbp, nmp, lp, kp, mk, wop, wsp, wb, place.stream);
           }),
           "mla_cache_evict");
    const Ref r0(give(a[10], lens)), r1(give(a[9], kept)), r2(give(a[11], wo)), r3(give(a[12], ws));
    return PyTuple_Pack(4, r0.p, r1.p, r2.p, r3.p);
  });
}

// inv_freq of a Rope: float64, one dimension, contiguous, on a CUDA device
PyObject* check_frequencies(PyObject*, PyObject* o) {
  return guarded([&]() -> PyObject* {
    check(o, "inv_freq", {at::kDouble}, 1, nullptr);
    Py_RETURN_NONE;
  });
}

PyObject* set_error(PyObject*, PyObject* o) {
  Py_INCREF(o);
  Py_XDECREF(g_error);
  g_error = o;
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef kMethods[] = {
    {"rope_apply", fast(&rope_apply), METH_FASTCALL, nullptr},
    {"latent_append", fast(&latent_append), METH_FASTCALL, nullptr},
    {"heads_append", fast(&heads_append), METH_FASTCALL, nullptr},
    {"attend_fp8", fast(&attend_fp8), METH_FASTCALL, nullptr},
    {"shard_combine", fast(&shard_combine), METH_FASTCALL, nullptr},
    {"prefix_partial", fast(&prefix_partial), METH_FASTCALL, nullptr},
    {"attention_weights", fast(&attention_weights), METH_FASTCALL, nullptr},
    {"cache_evict", fast(&cache_evict), METH_FASTCALL, nullptr},
    {"check_frequencies", check_frequencies, METH_O, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
