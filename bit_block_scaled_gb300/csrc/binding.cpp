// Python binding of the calls around the layer (grouped routing, norms, cache,
// attention): argument marshalling only, in C++ because these calls are as
// short as a Python function that looks at a few tensors. Each function takes
// what the Python function of the same name takes and returns its status code;
// arguments of the wrong type, shape or layout are MOE_ERR_INVALID_ARG, and
// nothing is launched.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <initializer_list>

#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/moe4.h"

namespace {

struct Bad {};  // an argument that does not fit

void need(bool ok) {
  if (!ok) throw Bad();
}

// A tensor argument, or none.
struct Arg {
  const at::Tensor *t = nullptr;
  explicit Arg(PyObject *o) {
    if (o == Py_None) return;
    need(THPVariable_Check(o));
    t = &THPVariable_Unpack(o);
    need(t->layout() == at::kStrided);
  }
  explicit operator bool() const { return t != nullptr; }
  void *ptr() const { return t ? t->data_ptr() : nullptr; }
  at::ScalarType type() const { return t->scalar_type(); }
  int64_t size(int i) const { return t->sizes()[i]; }
  int64_t stride(int i) const { return t->strides()[i]; }
  int64_t dim() const { return t->dim(); }
  // a contiguous tensor of n values of a type, or none
  void *flat(at::ScalarType type, int64_t n) const {
    if (!t) return nullptr;
    need(t->scalar_type() == type && t->numel() == n && t->is_contiguous());
    return t->data_ptr();
  }
};

int type_code(at::ScalarType t) {
  if (t == at::kBFloat16) return MOE_BF16;
  if (t == at::kHalf) return MOE_FP16;
  need(t == at::kFloat);
  return MOE_FP32;
}

int int_of(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad();
  need(v >= INT32_MIN && v <= INT32_MAX);
  return (int)v;
}

float float_of(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Bad();
  return (float)v;
}

// The memory of a ctypes structure; none is null.
template <typename T>
T *struct_of(PyObject *o) {
  if (o == Py_None) return nullptr;
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw Bad();
  T *p = static_cast<T *>(b.buf);
  const bool fits = b.len >= (Py_ssize_t)sizeof(T);
  PyBuffer_Release(&b);  // the caller's argument keeps the object
  need(fits);
  return p;
}

// The one device that all are on, which is current for the rest of the call: the library launches there. Where there
// is but one, it is (asking and setting take 0.15 us, as long as the rest of a call).
struct Together {
  c10::OptionalDeviceGuard guard;
  Together(const Arg &t, std::initializer_list<const Arg *> others) {
    const c10::Device d = t.t->device();
    for (const Arg *o : others) need(!*o || o->t->device() == d);
    if (!d.is_cuda() || c10::cuda::device_count() > 1) guard.reset_device(d);
  }
};

// A structure's address is in the memory of t's device, as far as it says (0: it does not): CUDA device i is i + 1,
// host memory -1, anything else -2.
void beside(int place, const Arg &t) {
  const c10::Device d = t.t->device();
  need(!place || place == (d.is_cuda() ? d.index() + 1 : d.is_cpu() ? -1 : -2));
}

// A workspace that holds the status word.
void workspace(const Arg &ws) { need((bool)ws && ws.t->is_contiguous() && (int64_t)ws.t->nbytes() >= MOE_STATUS_BYTES); }

// A stream object, a raw handle, or None: the current stream of the tensor's device.
moe_stream_t stream_of(PyObject *o, const Arg &t) {
  if (o == Py_None) need(t.t->is_cuda());
  if (o == Py_None) return (moe_stream_t)c10::cuda::getCurrentCUDAStream(t.t->device().index()).stream();
  if (PyLong_Check(o)) return (moe_stream_t)PyLong_AsVoidPtr(o);
  PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Bad();
  void *p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return (moe_stream_t)p;
}

// Runs f, whose result is a status code; whatever is thrown becomes one too.
template <typename F>
PyObject *status(Py_ssize_t n, Py_ssize_t want, F f) {
  int code;
  try {
    need(n == want);
    code = f();
  } catch (const Bad &) {
    code = MOE_ERR_INVALID_ARG;
  } catch (...) {
    code = MOE_ERR_CUDA;
  }
  PyErr_Clear();
  return PyLong_FromLong(code);
}

// logits, sel_bias, k, router, topk_ids, topk_weights, ws, stream
PyObject *route_grouped(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status(n, 8, [&]() -> int {
    const Arg l(a[0]), bias(a[1]), ids(a[4]), w(a[5]), ws(a[6]);
    need(l && l.dim() == 2 && ids && w);
    workspace(ws);
    const Together on(l, {&bias, &ids, &w, &ws});
    const int64_t T = l.size(0), E = l.size(1);
    const int k = int_of(a[2]);
    need(T <= INT32_MAX && E <= INT32_MAX && k >= 0 && (l.stride(1) == 1 || E <= 1));
    return moe_route_grouped(l.ptr(), type_code(l.type()), T > 1 ? l.stride(0) : E,
                             static_cast<float *>(bias.flat(at::kFloat, E)), (int)T, (int)E, k,
                             struct_of<moe_router_t>(a[3]), static_cast<int32_t *>(ids.flat(at::kInt, T * k)),
                             static_cast<float *>(w.flat(at::kFloat, T * k)), ws.ptr(), stream_of(a[7], l));
  });
}

// moe_norm_t with the length of its parameters behind it (0: it has none), and where they are
struct PlacedNorm {
  moe_norm_t norm;
  int32_t width, place;
};

// moe_kv_cache_t with where its data is
struct PlacedCache {
  moe_kv_cache_t cache;
  int32_t place;
};

// z, residual, gate, post, alpha, h_out, pre, y_out, stream
PyObject *residual_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status(n, 9, [&]() -> int {
    const Arg z(a[0]), r(a[1]), gate(a[2]), h(a[5]), y(a[7]);
    const Arg &act = z ? z : y ? y : r;
    need((bool)act && act.dim() == 2);
    const Arg &res = r ? r : h ? h : act;
    const Together on(act, {&z, &r, &gate, &h, &y});
    const int64_t T = act.size(0), H = act.size(1);
    need(T <= INT32_MAX && H <= INT32_MAX);
    auto rows = [&](const Arg &t, const Arg &like) -> int64_t {  // its stride over rows
      if (!t) return 0;
      need(t.dim() == 2 && t.type() == like.type() && t.size(0) == T && t.size(1) == H);
      need(t.stride(1) == 1 || H <= 1);
      return T > 1 ? t.stride(0) : (H + 7) / 8 * 8;  // the stride of a single row does not matter
    };
    const int64_t zs = rows(z, act), rs = rows(r, res), hs = rows(h, res), ys = rows(y, act);
    int64_t gst = 0, gsh = 0;
    if (gate) {
      need(gate.dim() == 2 && gate.type() == act.type());
      const int64_t gt = gate.size(0), gh = gate.size(1);
      need((gt == T || gt == 1) && (gh == H || gh == 1));
      gst = gt > 1 ? gate.stride(0) : 0;
      gsh = gh > 1 ? gate.stride(1) : 0;
    }
    const PlacedNorm *post = struct_of<PlacedNorm>(a[3]), *pre = struct_of<PlacedNorm>(a[6]);
    for (const PlacedNorm *p : {post, pre})
      if (p) {
        need(!p->width || p->width == H);
        beside(p->place, act);
      }
    return moe_residual_norm(z.ptr(), zs, r.ptr(), rs, gate.ptr(), gst, gsh, (int)T, (int)H, type_code(act.type()),
                             type_code(res.type()), post ? &post->norm : nullptr, float_of(a[4]), h.ptr(), hs,
                             pre ? &pre->norm : nullptr, y.ptr(), ys, stream_of(a[8], act));
  });
}

// Strides over the first two dimensions of a [T, heads, D] tensor.
struct Rows3 {
  int64_t t, h;
  Rows3(const Arg &x, int64_t T, int64_t heads, int64_t D) {
    need(x.dim() == 3 && x.size(0) == T && x.size(1) == heads && x.size(2) == D && (x.stride(2) == 1 || D == 1));
    t = T > 1 ? x.stride(0) : heads * D;
    h = heads > 1 ? x.stride(1) : D;
  }
};

// k, v, slots, cache, ws, stream
PyObject *kv_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status(n, 6, [&]() -> int {
    const Arg k(a[0]), v(a[1]), slots(a[2]), ws(a[4]);
    const PlacedCache *pc = struct_of<PlacedCache>(a[3]);
    need(k && v && slots && pc && k.type() == v.type());
    workspace(ws);
    const Together on(k, {&v, &slots, &ws});
    beside(pc->place, k);
    const moe_kv_cache_t *c = &pc->cache;
    const int64_t T = slots.t->numel();
    need(T <= INT32_MAX);
    const Rows3 ks(k, T, c->kv_heads, c->head_dim), vs(v, T, c->kv_heads, c->head_dim);
    return moe_kv_write(k.ptr(), v.ptr(), type_code(k.type()), ks.t, ks.h, vs.t, vs.h,
                        static_cast<int32_t *>(slots.flat(at::kInt, T)), (int)T, c, ws.ptr(), stream_of(a[5], k));
  });
}

// cache, slots, k_out, v_out, ws, stream
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status(n, 6, [&]() -> int {
    const Arg slots(a[1]), k(a[2]), v(a[3]), ws(a[4]);
    const PlacedCache *pc = struct_of<PlacedCache>(a[0]);
    const Arg &one = k ? k : v;
    need(one && slots && pc && (!v || v.type() == one.type()));
    workspace(ws);
    const Together on(slots, {&k, &v, &ws});
    beside(pc->place, slots);
    const moe_kv_cache_t *c = &pc->cache;
    const int64_t T = slots.t->numel();
    need(T <= INT32_MAX);
    int64_t s[4] = {0, 0, 0, 0};
    if (k) {
      const Rows3 x(k, T, c->kv_heads, c->head_dim);
      s[0] = x.t, s[1] = x.h;
    }
    if (v) {
      const Rows3 x(v, T, c->kv_heads, c->head_dim);
      s[2] = x.t, s[3] = x.h;
    }
    return moe_kv_read(c, static_cast<int32_t *>(slots.flat(at::kInt, T)), (int)T, k.ptr(), v.ptr(), type_code(one.type()),
                       s[0], s[1], s[2], s[3], ws.ptr(), stream_of(a[5], slots));
  });
}

// q, cache, block_table, seq_lens, out, ws, scale, window, sinks, lse, stream
PyObject *attn_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return status(n, 11, [&]() -> int {
    const Arg q(a[0]), table(a[2]), lens(a[3]), out(a[4]), ws(a[5]), sinks(a[8]), lse(a[9]);
    const PlacedCache *pc = struct_of<PlacedCache>(a[1]);
    need(q && pc && table && lens && out && ws && q.dim() == 3 && out.type() == q.type());
    const Together on(q, {&table, &lens, &out, &ws, &sinks, &lse});
    beside(pc->place, q);
    const moe_kv_cache_t *c = &pc->cache;
    const int64_t B = q.size(0), heads = q.size(1), D = q.size(2);
    need(D == c->head_dim && B <= INT32_MAX && heads <= INT32_MAX);
    need(table.dim() == 2 && table.type() == at::kInt && table.size(0) == B && ws.type() == at::kByte);
    const int64_t pages = table.size(1);
    need(pages <= INT32_MAX && (table.stride(1) == 1 || pages <= 1));
    const Rows3 qs(q, B, heads, D), os(out, B, heads, D);
    return moe_attn_decode(q.ptr(), type_code(q.type()), qs.t, qs.h, c, static_cast<int32_t *>(table.ptr()),
                           B > 1 ? table.stride(0) : pages, (int)pages,
                           static_cast<int32_t *>(lens.flat(at::kInt, B)), (int)B, (int)heads, float_of(a[6]),
                           int_of(a[7]), static_cast<float *>(sinks.flat(at::kFloat, heads)), out.ptr(), os.t, os.h,
                           static_cast<float *>(lse.flat(at::kFloat, B * heads)), ws.ptr(), (size_t)ws.t->numel(),
                           stream_of(a[10], q));
  });
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(route_grouped), FAST(residual_norm), FAST(kv_write), FAST(kv_read), FAST(attn_decode),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
