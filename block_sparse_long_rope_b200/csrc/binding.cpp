// Native half of the torch binding for the calls of a serving step, which are
// short enough that checking their tensors from Python would take longer than
// the kernels (16 to 21 us a call; 3.7 to 4 us from here). star.py holds the
// public functions; these take their arguments in order, check them, make the
// tensors' device current and call the C ABI of the libstar.so that bind() was
// given. They return its status, which star.py turns into an error.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string.h>

#include <exception>

#include "star.h"

namespace {

decltype(&star_rope_scaled) rope_scaled_fn;
decltype(&star_batch_plan) batch_plan_fn;
decltype(&star_kv8_append) kv8_append_fn;
decltype(&star_kv8_attend) kv8_attend_fn;

// A Python error is set: unwinds to the entry point.
struct Raised {};

template <typename... Args>
[[noreturn]] void raise(PyObject* type, const char* fmt, Args... args) {
  PyErr_Format(type, fmt, args...);
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const at::Tensor& bf16(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16)
    raise(PyExc_TypeError, "%s must be bfloat16, got %s", name, c10::toString(t.scalar_type()));
  return t;
}
// A contiguous int32 tensor, of n entries where n >= 0.
const at::Tensor& ints(PyObject* o, const char* name, int64_t n = -1) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt || !t.is_contiguous())
    raise(PyExc_ValueError, "%s must be a contiguous int32 tensor", name);
  if (n >= 0 && t.numel() != n)
    raise(PyExc_ValueError, "%s must have %lld entries, it has %lld", name, (long long)n, (long long)t.numel());
  return t;
}
int as_int(int64_t v, const char* name) {
  if (v > INT32_MAX || v < INT32_MIN) raise(PyExc_ValueError, "%s (%lld) does not fit int32", name, (long long)v);
  return static_cast<int>(v);
}
int to_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return as_int(v, name);
}
void* data(const at::Tensor& t) { return t.data_ptr(); }

// The one CUDA device of a call's tensors, and the stream that it runs on.
class Place {
 public:
  void on(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a CUDA tensor", name);
    const int d = t.device().index();
    if (dev_ < 0) dev_ = d;
    else if (d != dev_)
      raise(PyExc_ValueError, "%s is on cuda:%d, the other tensors on cuda:%d", name, d, dev_);
  }
  // Makes the device current; a given stream has to be its own.
  void* enter(PyObject* stream) {
    uint64_t handle = 0;
    if (stream != Py_None) {
      const int d = attribute(stream, "device_index");
      if (d != dev_) raise(PyExc_ValueError, "the stream is on cuda:%d, the tensors on cuda:%d", d, dev_);
      handle = attribute(stream, "cuda_stream");
    }
    if (c10::cuda::current_device() != dev_) guard_.set_index(dev_);
    if (stream != Py_None) return reinterpret_cast<void*>(handle);
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev_)).stream();
  }

 private:
  static uint64_t attribute(PyObject* o, const char* name) {
    PyObject* v = PyObject_GetAttrString(o, name);
    if (!v) throw Raised{};
    const uint64_t x = PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Raised{};
    return x;
  }
  int dev_ = -1;
  c10::cuda::OptionalCUDAGuard guard_;
};

struct Cache {
  int kind, pages, heads, page_len, dim;
};
Cache cache(const at::Tensor& kp, const at::Tensor& vp, const at::Tensor& ks, const at::Tensor& vs) {
  Cache c;
  c.kind = kp.scalar_type() == at::kFloat8_e4m3fn ? STAR_KV8_E4M3 : kp.scalar_type() == at::kChar ? STAR_KV8_INT8 : -1;
  if (c.kind < 0 || vp.scalar_type() != kp.scalar_type())
    raise(PyExc_TypeError, "k_pages and v_pages must both be float8_e4m3fn or int8, got %s and %s",
          c10::toString(kp.scalar_type()), c10::toString(vp.scalar_type()));
  if (kp.dim() != 4 || vp.sizes() != kp.sizes())
    raise(PyExc_ValueError, "k_pages and v_pages must have one shape [num_pages, Hkv, page_len, D]");
  const at::Tensor* scales[2] = {&ks, &vs};
  const char* names[2] = {"k_scale", "v_scale"};
  for (int i = 0; i < 2; ++i)
    if (scales[i]->scalar_type() != at::kFloat || scales[i]->dim() != 2 || scales[i]->size(0) != kp.size(0) ||
        scales[i]->size(1) != kp.size(1))
      raise(PyExc_ValueError, "%s must be float32 [num_pages, Hkv]", names[i]);
  const at::Tensor* all[4] = {&kp, &vp, &ks, &vs};
  const char* all_names[4] = {"k_pages", "v_pages", "k_scale", "v_scale"};
  for (int i = 0; i < 4; ++i)
    if (!all[i]->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", all_names[i]);
  c.pages = as_int(kp.size(0), "num_pages");
  c.heads = as_int(kp.size(1), "Hkv");
  c.page_len = as_int(kp.size(2), "page_len");
  c.dim = as_int(kp.size(3), "D");
  return c;
}
const at::Tensor& space(PyObject* o) {
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  return t;
}
size_t bytes(const at::Tensor& t) { return static_cast<size_t>(t.numel()) * t.element_size(); }

// Runs one entry point's body with n arguments; nothing but a Python error leaves it.
template <typename Body>
PyObject* entry(Py_ssize_t got, Py_ssize_t n, Body body) {
  try {
    if (got != n) raise(PyExc_TypeError, "%zd arguments expected, got %zd", n, got);
    return PyLong_FromLong(body());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* bind(PyObject*, PyObject* handle) {
  void* lib = PyLong_AsVoidPtr(handle);
  if (PyErr_Occurred()) return nullptr;
  rope_scaled_fn = reinterpret_cast<decltype(rope_scaled_fn)>(dlsym(lib, "star_rope_scaled"));
  batch_plan_fn = reinterpret_cast<decltype(batch_plan_fn)>(dlsym(lib, "star_batch_plan"));
  kv8_append_fn = reinterpret_cast<decltype(kv8_append_fn)>(dlsym(lib, "star_kv8_append"));
  kv8_attend_fn = reinterpret_cast<decltype(kv8_attend_fn)>(dlsym(lib, "star_kv8_attend"));
  if (!rope_scaled_fn || !batch_plan_fn || !kv8_append_fn || !kv8_attend_fn) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks the serving entry points");
    return nullptr;
  }
  Py_RETURN_NONE;
}

// x, y, inv_freq (a buffer of doubles), mscale, interleaved, transpose, pos, pos0, stream
PyObject* rope_scaled(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 9, [&]() -> star_status {
    const at::Tensor &x = bf16(a[0], "x"), &y = bf16(a[1], "y");
    if (x.dim() != 4 || y.sizes() != x.sizes()) raise(PyExc_ValueError, "x and y must have one shape [B, S, H, D]");
    if (x.stride(3) != 1 || y.stride(3) != 1) raise(PyExc_ValueError, "head_dim must be contiguous");
    const int B = as_int(x.size(0), "B"), S = as_int(x.size(1), "S");
    const double m = PyFloat_AsDouble(a[3]);
    const int inter = PyObject_IsTrue(a[4]), turn = PyObject_IsTrue(a[5]);
    const long long pos0 = PyLong_AsLongLong(a[7]);
    if (PyErr_Occurred()) throw Raised{};
    Py_buffer f;
    if (PyObject_GetBuffer(a[2], &f, PyBUF_CONTIG_RO | PyBUF_FORMAT)) throw Raised{};
    struct Release {
      Py_buffer* b;
      ~Release() { PyBuffer_Release(b); }
    } release{&f};
    if (f.itemsize != 8 || !f.format || f.format[strspn(f.format, "<=@")] != 'd')
      raise(PyExc_TypeError, "inv_freq must hold doubles");
    const int32_t* pos = nullptr;
    int64_t pos_stride = 0;
    Place place;
    if (a[6] != Py_None) {
      const at::Tensor& p = tensor(a[6], "pos");
      const bool one = p.dim() == 1 && p.size(0) == S, two = p.dim() == 2 && p.size(0) == B && p.size(1) == S;
      if (p.scalar_type() != at::kInt || !(one || two) || (S > 1 && p.stride(-1) != 1))
        raise(PyExc_ValueError, "pos must be int32 [S] or [B, S], contiguous in S");
      place.on(x, "x");
      place.on(p, "pos");
      pos = static_cast<const int32_t*>(data(p));
      pos_stride = two ? p.stride(0) : 0;
    }
    place.on(x, "x");
    place.on(y, "y");
    void* stream = place.enter(a[8]);
    const int64_t xs[3] = {x.stride(0), x.stride(1), x.stride(2)}, ys[3] = {y.stride(0), y.stride(1), y.stride(2)};
    return rope_scaled_fn(data(x), xs, data(y), ys, pos, pos_stride, pos0, B, S, as_int(x.size(2), "H"),
                          as_int(x.size(3), "D"), 2 * as_int(f.len / 8, "len(inv_freq)"),
                          static_cast<const double*>(f.buf), m, inter, turn, stream);
  });
}

// ctx_len, new_len, free_pages, free_begin, page_len, block_table, cu_new, pos, slot, run_start,
// kv_len, free_next, workspace, stream
PyObject* batch_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 14, [&]() -> star_status {
    const at::Tensor& table = ints(a[5], "block_table");
    if (table.dim() != 2) raise(PyExc_ValueError, "block_table must be [B, max_pages]");
    const int64_t B = table.size(0);
    const at::Tensor &free_pages = ints(a[2], "free_pages"), &pos = ints(a[7], "pos");
    const int64_t cap = pos.numel();
    const at::Tensor &ctx = ints(a[0], "ctx_len", B), &add = ints(a[1], "new_len", B), &kv = ints(a[10], "kv_len", B),
                     &cu = ints(a[6], "cu_new", B + 1), &slot = ints(a[8], "slot", cap),
                     &begin = ints(a[3], "free_begin", 1), &next = ints(a[11], "free_next", 1),
                     &runs = ints(a[9], "run_start"), &ws = space(a[12]);
    Place place;
    place.on(table, "block_table");
    place.on(ctx, "ctx_len");
    place.on(add, "new_len");
    place.on(free_pages, "free_pages");
    place.on(begin, "free_begin");
    place.on(cu, "cu_new");
    place.on(pos, "pos");
    place.on(slot, "slot");
    place.on(runs, "run_start");
    place.on(kv, "kv_len");
    place.on(next, "free_next");
    place.on(ws, "workspace");
    const int page_len = to_int(a[4], "page_len");
    void* stream = place.enter(a[13]);
    auto p = [](const at::Tensor& t) { return static_cast<int32_t*>(data(t)); };
    return batch_plan_fn(p(ctx), p(add), as_int(B, "B"), p(free_pages), as_int(free_pages.numel(), "num_free"),
                         p(begin), page_len, p(table), as_int(table.size(1), "max_pages"), p(cu), p(pos), p(slot),
                         as_int(cap, "n_cap"), p(runs), as_int(runs.numel() - 1, "run_cap"), p(kv), p(next),
                         data(ws), bytes(ws), stream);
  });
}

// k, v, slot, run_start, k_pages, v_pages, k_scale, v_scale, workspace, stream
PyObject* kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 10, [&]() -> star_status {
    const at::Tensor &kp = tensor(a[4], "k_pages"), &vp = tensor(a[5], "v_pages"), &ks = tensor(a[6], "k_scale"),
                     &vs = tensor(a[7], "v_scale");
    const Cache c = cache(kp, vp, ks, vs);
    const at::Tensor &k = bf16(a[0], "k"), &v = bf16(a[1], "v");
    const at::Tensor* rows[2] = {&k, &v};
    const char* names[2] = {"k", "v"};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor& t = *rows[i];
      if (t.dim() != 3 || t.size(1) != c.heads || t.size(2) != c.dim || t.size(0) != k.size(0))
        raise(PyExc_ValueError, "%s must be [n, %d, %d]", names[i], c.heads, c.dim);
      if (t.stride(2) != 1) raise(PyExc_ValueError, "%s must be contiguous in head_dim", names[i]);
    }
    const at::Tensor &slot = ints(a[2], "slot", k.size(0)), &runs = ints(a[3], "run_start"),
                     &ws = space(a[8]);
    Place place;
    place.on(k, "k");
    place.on(v, "v");
    place.on(slot, "slot");
    place.on(runs, "run_start");
    place.on(kp, "k_pages");
    place.on(vp, "v_pages");
    place.on(ks, "k_scale");
    place.on(vs, "v_scale");
    place.on(ws, "workspace");
    void* stream = place.enter(a[9]);
    const int64_t kst[2] = {k.stride(0), k.stride(1)}, vst[2] = {v.stride(0), v.stride(1)};
    return kv8_append_fn(data(k), kst, data(v), vst, as_int(k.size(0), "n"), c.heads, c.dim,
                         static_cast<int32_t*>(data(slot)), static_cast<int32_t*>(data(runs)),
                         as_int(runs.numel() - 1, "run_cap"), data(kp), data(vp), static_cast<float*>(data(ks)),
                         static_cast<float*>(data(vs)), c.pages, c.page_len, c.kind, data(ws), bytes(ws), stream);
  });
}

// q, cu_new, kv_len, block_table, k_pages, v_pages, k_scale, v_scale, o, workspace, max_new, max_kv,
// lse, stream
PyObject* kv8_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry(n, 14, [&]() -> star_status {
    const at::Tensor &kp = tensor(a[4], "k_pages"), &vp = tensor(a[5], "v_pages"), &ks = tensor(a[6], "k_scale"),
                     &vs = tensor(a[7], "v_scale");
    const Cache c = cache(kp, vp, ks, vs);
    const at::Tensor &q = bf16(a[0], "q"), &o = bf16(a[8], "o");
    if (q.dim() != 3 || q.size(2) != c.dim || q.stride(2) != 1)
      raise(PyExc_ValueError, "q must be [n, Hq, %d], contiguous in head_dim", c.dim);
    if (o.sizes() != q.sizes() || !o.is_contiguous()) raise(PyExc_ValueError, "o must be contiguous, of q's shape");
    const at::Tensor& table = ints(a[3], "block_table");
    if (table.dim() != 2) raise(PyExc_ValueError, "block_table must be [B, max_pages]");
    const at::Tensor &cu = ints(a[1], "cu_new", table.size(0) + 1), &kv = ints(a[2], "kv_len", table.size(0)),
                     &ws = space(a[9]);
    Place place;
    place.on(q, "q");
    place.on(o, "o");
    float* lse = nullptr;
    if (a[12] != Py_None) {
      const at::Tensor& l = tensor(a[12], "lse");
      if (l.scalar_type() != at::kFloat || l.dim() != 2 || l.size(0) != q.size(1) || l.size(1) != q.size(0) ||
          !l.is_contiguous())
        raise(PyExc_ValueError, "lse must be contiguous float32 [%lld, %lld]", (long long)q.size(1),
              (long long)q.size(0));
      place.on(l, "lse");
      lse = static_cast<float*>(data(l));
    }
    place.on(cu, "cu_new");
    place.on(kv, "kv_len");
    place.on(table, "block_table");
    place.on(kp, "k_pages");
    place.on(vp, "v_pages");
    place.on(ks, "k_scale");
    place.on(vs, "v_scale");
    place.on(ws, "workspace");
    const int max_new = to_int(a[10], "max_new"), max_kv = to_int(a[11], "max_kv");
    void* stream = place.enter(a[13]);
    const int64_t qst[2] = {q.stride(0), q.stride(1)};
    return kv8_attend_fn(data(q), qst, as_int(q.size(0), "n"), static_cast<int32_t*>(data(cu)),
                         static_cast<int32_t*>(data(kv)), as_int(table.size(0), "B"),
                         static_cast<int32_t*>(data(table)), as_int(table.size(1), "max_pages"), data(kp), data(vp),
                         static_cast<float*>(data(ks)), static_cast<float*>(data(vs)), c.pages, c.page_len, c.kind,
                         as_int(q.size(1), "Hq"), c.heads, c.dim, max_new, max_kv, data(o), lse, data(ws), bytes(ws),
                         stream);
  });
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"rope_scaled", fast(rope_scaled), METH_FASTCALL, nullptr},
                         {"batch_plan", fast(batch_plan), METH_FASTCALL, nullptr},
                         {"kv8_append", fast(kv8_append), METH_FASTCALL, nullptr},
                         {"kv8_attend", fast(kv8_attend), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
