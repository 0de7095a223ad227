// Tensors to the C entry points of rotary positions, differential attention and its decoding: checks of
// shapes, types, strides and devices, the outputs, the device and the stream.
//
// A decoding step's kernel is shorter than the interpreter takes to look at five tensors, so these calls
// do that here: mesh_rope of one token of 64 sequences costs the host 5 us, where the same checks and a
// ctypes call of 27 arguments took 16.  The functions take positional arguments only and return the
// outputs, or a status code where the entry point refuses; the package's functions give them names,
// defaults and documentation.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <initializer_list>
#include <sstream>
#include <string>

#include "mesh_attn.h"

namespace {

// The library is opened by path; bind() takes its functions' addresses.
decltype(&mesh_attn_rope) rope_fn = nullptr;
decltype(&mesh_attn_diff_fwd) fwd_fn = nullptr;
decltype(&mesh_attn_diff_bwd) bwd_fn = nullptr;
decltype(&mesh_attn_diff_decode) decode_fn = nullptr;

const at::Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}
at::Tensor tensor_or_none(PyObject* o, const char* name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

void expect_args(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got); }

int64_t integer(PyObject* o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}
void* pointer(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}
int32_t i32(int64_t x) {
  TORCH_CHECK_VALUE(x <= INT32_MAX, "sizes must be below 2^31");
  return (int32_t)x;
}

mesh_attn_dtype dtype_code(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return MESH_ATTN_BF16;
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, "unsupported dtype ", t.scalar_type(),
                   ": use torch.bfloat16 or torch.float32");
  return MESH_ATTN_F32;
}

// The CUDA device that all tensors are on (those that are there at all).
c10::Device one_device(std::initializer_list<const at::Tensor*> ts) {
  const c10::Device d = (*ts.begin())->device();
  bool ok = d.is_cuda();
  for (const at::Tensor* t : ts) ok = ok && (!t->defined() || t->device() == d);
  if (!ok) {
    std::ostringstream s;
    for (const at::Tensor* t : ts)
      if (t->defined()) s << " " << t->device();
    TORCH_CHECK_VALUE(false, "tensors must be on one CUDA device; got", s.str());
  }
  return d;
}

void contiguous(std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    TORCH_CHECK_VALUE(!t->defined() || t->is_contiguous(),
                      "q, k, v, lam, the gradients and the outputs must be contiguous");
}
// ts, where they are there, are as q: contiguous, of its shape and dtype.
void like(const at::Tensor& q, std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    TORCH_CHECK_VALUE(!t->defined() || (t->sizes() == q.sizes() && t->scalar_type() == q.scalar_type()),
                      "O, O2 and dO must have q's shape and dtype, dQ, dK, dV and dlam those of q, k, v and lam");
  contiguous(ts);
}

// What the kernels write besides the outputs: nbytes() of an expanded tensor counts memory that is not there, and
// a status block is MESH_ATTN_STATUS_WORDS long whatever the tensor's size.
void check_scratch(const at::Tensor& ws, const at::Tensor& status) {
  TORCH_CHECK_VALUE(ws.is_contiguous(), "workspace must be contiguous");
  TORCH_CHECK_VALUE(status.scalar_type() == at::kInt && status.is_contiguous() && status.numel() >= MESH_ATTN_STATUS_WORDS,
                    "status must be ", MESH_ATTN_STATUS_WORDS, " or more contiguous int32 (new_status)");
}

void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The stream of a call: the one given (its handle), or the device's current one.
cudaStream_t stream_of(PyObject* given, c10::Device d) {
  return given == Py_None ? c10::cuda::getCurrentCUDAStream(d.index()).stream() : static_cast<cudaStream_t>(pointer(given));
}

// A C entry point, without the interpreter's lock (a full launch queue blocks it).
template <typename F>
int call(c10::Device d, F&& f) {
  const c10::DeviceGuard guard(d);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) throw python_error();
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o;
    if (t->defined()) {
      o = THPVariable_Wrap(*t);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    if (!o) {
      Py_DECREF(out);
      throw python_error();
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 4);
  rope_fn = reinterpret_cast<decltype(rope_fn)>(pointer(a[0]));
  fwd_fn = reinterpret_cast<decltype(fwd_fn)>(pointer(a[1]));
  bwd_fn = reinterpret_cast<decltype(bwd_fn)>(pointer(a[2]));
  decode_fn = reinterpret_cast<decltype(decode_fn)>(pointer(a[3]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- rotary positions

// MeshRope's numbers as bytes: this header, the frequencies, the axes.
struct RopeHeader {
  int32_t d, groups, pairs, axes, adjacent, reserved;
};

// (handle, q, k, positions, q_out, k_out, inverse, stream); k and k_out None together, either output None
// for a new dense tensor
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 8);
  TORCH_CHECK_TYPE(PyBytes_Check(a[0]), "rope must be a MeshRope");
  RopeHeader h;
  const char* raw = PyBytes_AS_STRING(a[0]);
  TORCH_CHECK_VALUE(PyBytes_GET_SIZE(a[0]) >= (Py_ssize_t)sizeof(h), "rope is not of a MeshRope");
  std::memcpy(&h, raw, sizeof(h));
  TORCH_CHECK_VALUE(h.pairs >= 0 && PyBytes_GET_SIZE(a[0]) == (Py_ssize_t)(sizeof(h) + 12 * (size_t)h.pairs),
                    "rope is not of a MeshRope");
  const at::Tensor &q = tensor(a[1], "q"), &pos = tensor(a[3], "positions");
  const at::Tensor k = tensor_or_none(a[2], "k");
  at::Tensor q_out = tensor_or_none(a[4], "q_out"), k_out = tensor_or_none(a[5], "k_out");
  TORCH_CHECK_VALUE(q.dim() == 4 && q.size(3) == h.d, "q must be [B, H, S, ", h.d, "]");
  TORCH_CHECK_VALUE(k.defined() || !k_out.defined(), "k and k_out go together");
  const int64_t B = q.size(0), S = q.size(2);
  if (k.defined())
    TORCH_CHECK_VALUE(k.dim() == 4 && k.size(0) == B && k.size(2) == S && k.size(3) == h.d,
                      "q and k must agree in batch, tokens and columns");
  const at::ScalarType type = q.scalar_type();
  for (const auto& [x, y] : {std::pair<const at::Tensor*, const at::Tensor*>{&q, &q_out}, {&k, &k_out}}) {
    if (!x->defined()) continue;
    TORCH_CHECK_VALUE(x->scalar_type() == type && (!y->defined() || y->scalar_type() == type),
                      "q, k and the outputs must be of one dtype");
    TORCH_CHECK_VALUE(!y->defined() || y->sizes() == x->sizes(), "an output must have its input's shape");
    TORCH_CHECK_VALUE(!x->numel() || (x->stride(3) == 1 && (!y->defined() || y->stride(3) == 1)),
                      "the columns of a head must be consecutive");
  }
  const mesh_attn_dtype dt = dtype_code(q);
  TORCH_CHECK_VALUE(pos.scalar_type() == at::kInt || pos.scalar_type() == at::kLong, "positions must be int32 or int64");
  // [axes, B, S], [axes, S] or, for one axis, [B, S] or [S]: the axes' strides, 0 where it is the same for all
  int64_t ps[3] = {0, 0, 0};
  bool fits = false;
  const int64_t nd = pos.dim();
  if (nd >= 1 && nd <= 3 && pos.size(nd - 1) == S) {
    ps[2] = pos.stride(nd - 1);
    const auto batch = [&](int64_t i) {
      ps[1] = pos.size(i) == 1 ? 0 : pos.stride(i);
      return pos.size(i) == 1 || pos.size(i) == B;
    };
    if (nd == 1) {
      fits = h.axes == 1;
    } else if (nd == 2 && h.axes == 1) {
      fits = batch(0);
    } else {
      ps[0] = pos.stride(0);
      fits = pos.size(0) == h.axes && (nd == 2 || batch(1));
    }
  }
  TORCH_CHECK_VALUE(fits, "positions must be [", h.axes, ", S] or [", h.axes, ", B, S] with B = ", B, ", S = ", S, "; got ",
                    pos.sizes());
  const c10::Device dev = one_device({&q, &pos, &k, &q_out, &k_out});
  if (!q_out.defined()) q_out = at::empty(q.sizes(), q.options());
  if (k.defined() && !k_out.defined()) k_out = at::empty(k.sizes(), k.options());
  const auto strides = [](const at::Tensor& t, int64_t(&s)[3]) {
    for (int i = 0; i < 3; ++i) s[i] = t.defined() ? t.stride(i) : 0;
  };
  int64_t qs[3], qos[3], ks[3], kos[3];
  strides(q, qs), strides(q_out, qos), strides(k, ks), strides(k_out, kos);
  const int32_t inverse = (int32_t)integer(a[6]), Bi = i32(B), Hq = i32(q.size(1)), Hk = k.defined() ? i32(k.size(1)) : 0;
  const cudaStream_t st = stream_of(a[7], dev);
  const double* freq = reinterpret_cast<const double*>(raw + sizeof(h));  // 8-byte aligned behind the object's own header
  const int32_t* axis = reinterpret_cast<const int32_t*>(raw + sizeof(h) + 8 * (size_t)h.pairs);
  const int rc = call(dev, [&] {
    return rope_fn(dt, Bi, S, h.d, Hq, q.data_ptr(), qs, q_out.data_ptr(), qos, Hk, data(k), ks, data(k_out), kos, h.groups,
                   h.pairs, h.axes, freq, axis, h.adjacent, inverse, pos.data_ptr(), (int32_t)(8 * pos.element_size()), ps, st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&q_out, &k_out});
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- differential attention

struct Sizes {
  mesh_attn_dtype dt;
  int32_t B, Hq, Hkv, d, lam_n;
  int64_t S;  // of q
};

// q, k, v and lam that fit together; k's and v's strides and lengths are the caller's to check
Sizes diff_sizes(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& lam) {
  TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4 && v.sizes() == k.sizes(), "q must be [B, Hq, S, d], k and v [B, Hkv, S, d]");
  TORCH_CHECK_VALUE(k.size(0) == q.size(0) && k.size(3) == q.size(3), "q, k and v must agree in batch and columns");
  TORCH_CHECK_VALUE(k.size(1) >= 1 && q.size(1) % k.size(1) == 0, "Hq must be a multiple of Hkv: ", q.size(1), " and ", k.size(1));
  TORCH_CHECK_VALUE(lam.dim() == 1 && (lam.size(0) == q.size(1) || lam.size(0) == 1),
                    "lam must be [Hq], or [1] for one value for all heads");
  const at::ScalarType t = q.scalar_type();
  TORCH_CHECK_VALUE(k.scalar_type() == t && v.scalar_type() == t && lam.scalar_type() == t, "q, k, v and lam must be of one dtype");
  contiguous({&q, &lam});
  return {dtype_code(q), i32(q.size(0)), i32(q.size(1)), i32(k.size(1)), i32(q.size(3)), i32(lam.size(0)), q.size(2)};
}

void check_lse(const at::Tensor& lse, const Sizes& z) {
  TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.sizes() == at::IntArrayRef({z.B, z.Hq, 2, z.S}),
                    "LSE must be fp32 [B, Hq, 2, S] (S = 1 in decoding)");
  contiguous({&lse});
}

float scale_of(PyObject* o, const Sizes& z) {
  if (o == Py_None) return (float)(1.0 / std::sqrt((double)(z.d / 2)));
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)x;
}

// A plan as the calls take it: (handle, S, {device index: tables}, {device index: the stream that owns their memory})
struct PlanRef {
  const mesh_attn_plan* handle;
  PyObject *tables, *streams;
};
PlanRef plan_of(PyObject* o, const Sizes& z, const at::Tensor& k) {
  TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4, "plan must be a Plan");
  const int64_t S = integer(PyTuple_GET_ITEM(o, 1));
  TORCH_CHECK_VALUE(z.S == S && k.size(2) == S, "the plan is for S = ", S, "; q has ", z.S, " tokens, k and v ", k.size(2));
  return {static_cast<const mesh_attn_plan*>(pointer(PyTuple_GET_ITEM(o, 0))), PyTuple_GET_ITEM(o, 2), PyTuple_GET_ITEM(o, 3)};
}

// The plan's tables for a call on `st`.  Where that is not the stream that owns their memory, the memory stays
// theirs until the call has run, though the plan may be dropped before.
at::Tensor tables_for(const PlanRef& p, c10::Device d, cudaStream_t st) {
  PyObject* key = PyLong_FromLong(d.index());
  if (!key) throw python_error();
  PyObject* t = PyDict_GetItemWithError(p.tables, key);
  PyObject* owner = t ? PyDict_GetItemWithError(p.streams, key) : nullptr;
  Py_DECREF(key);
  if (PyErr_Occurred()) throw python_error();
  if (!t) return at::Tensor();
  const at::Tensor& x = tensor(t, "tables");
  if (!owner || pointer(owner) != st) x.record_stream(c10::cuda::getStreamFromExternal(st, d.index()).unwrap());
  return x;
}

// (plan, q, k, v, lam, scale, O, O2, LSE, with_o2, workspace, status, stream); outputs None for new ones.
// Returns None where the plan has no tables on the device yet.
PyObject* diff_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 13);
  const at::Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &lam = tensor(a[4], "lam");
  at::Tensor O = tensor_or_none(a[6], "O"), O2 = tensor_or_none(a[7], "O2"), lse = tensor_or_none(a[8], "LSE");
  const at::Tensor &ws = tensor(a[10], "workspace"), &status = tensor(a[11], "status");
  const Sizes z = diff_sizes(q, k, v, lam);
  contiguous({&k, &v});
  like(q, {&O, &O2});
  if (lse.defined()) check_lse(lse, z);
  check_scratch(ws, status);
  const c10::Device dev = one_device({&q, &k, &v, &lam, &ws, &status, &O, &O2, &lse});
  const PlanRef plan = plan_of(a[0], z, k);
  const float scale = scale_of(a[5], z);
  const cudaStream_t st = stream_of(a[12], dev);
  const at::Tensor tables = tables_for(plan, dev, st);
  if (!tables.defined()) Py_RETURN_NONE;
  if (!O.defined()) O = at::empty(q.sizes(), q.options());
  if (!O2.defined() && integer(a[9])) O2 = at::empty(q.sizes(), q.options());
  if (!lse.defined()) lse = at::empty({z.B, z.Hq, 2, z.S}, q.options().dtype(at::kFloat));
  const int rc = call(dev, [&] {
    return fwd_fn(plan.handle, tables.data_ptr(), z.dt, z.B, z.Hq, z.Hkv, z.d, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                  lam.data_ptr(), z.lam_n, scale, O.data_ptr(), data(O2), static_cast<float*>(lse.data_ptr()), ws.data_ptr(),
                  ws.nbytes(), static_cast<int32_t*>(status.data_ptr()), st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&O, &O2, &lse});
  END_HANDLE_TH_ERRORS
}

// (plan, q, k, v, lam, O, O2, LSE, dO, scale, dQ, dK, dV, dlam, workspace, status, stream); gradients None for new ones.
// Returns None where the plan has no tables on the device yet.
PyObject* diff_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 17);
  const at::Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &lam = tensor(a[4], "lam");
  const at::Tensor &O = tensor(a[5], "O"), &O2 = tensor(a[6], "O2"), &lse = tensor(a[7], "LSE"), &dO = tensor(a[8], "dO");
  at::Tensor dQ = tensor_or_none(a[10], "dQ"), dK = tensor_or_none(a[11], "dK"), dV = tensor_or_none(a[12], "dV"),
             dlam = tensor_or_none(a[13], "dlam");
  const at::Tensor &ws = tensor(a[14], "workspace"), &status = tensor(a[15], "status");
  const Sizes z = diff_sizes(q, k, v, lam);
  contiguous({&k, &v});
  like(q, {&O, &O2, &dO, &dQ});
  like(k, {&dK, &dV});
  like(lam, {&dlam});
  check_lse(lse, z);
  check_scratch(ws, status);
  const c10::Device dev = one_device({&q, &k, &v, &lam, &O, &O2, &lse, &dO, &ws, &status, &dQ, &dK, &dV, &dlam});
  const PlanRef plan = plan_of(a[0], z, k);
  const float scale = scale_of(a[9], z);
  const cudaStream_t st = stream_of(a[16], dev);
  const at::Tensor tables = tables_for(plan, dev, st);
  if (!tables.defined()) Py_RETURN_NONE;
  if (!dQ.defined()) dQ = at::empty(q.sizes(), q.options());
  if (!dK.defined()) dK = at::empty(k.sizes(), k.options());
  if (!dV.defined()) dV = at::empty(v.sizes(), v.options());
  if (!dlam.defined()) dlam = at::empty(lam.sizes(), lam.options());
  if (!q.numel()) {  // no rows: sums over nothing
    const c10::StreamGuard guard(c10::cuda::getStreamFromExternal(st, dev.index()).unwrap());
    for (const at::Tensor* t : {&dK, &dV, &dlam}) t->zero_();
    return tuple_of({&dQ, &dK, &dV, &dlam});
  }
  const int rc = call(dev, [&] {
    return bwd_fn(plan.handle, tables.data_ptr(), z.dt, z.B, z.Hq, z.Hkv, z.d, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                  lam.data_ptr(), z.lam_n, O.data_ptr(), O2.data_ptr(), static_cast<const float*>(lse.data_ptr()),
                  dO.data_ptr(), scale, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), dlam.data_ptr(), ws.data_ptr(),
                  ws.nbytes(), static_cast<int32_t*>(status.data_ptr()), st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&dQ, &dK, &dV, &dlam});
  END_HANDLE_TH_ERRORS
}

// (q, k, v, lam): raises where they do not fit together or are not on one CUDA device
PyObject* diff_check(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 4);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &lam = tensor(a[3], "lam");
  diff_sizes(q, k, v, lam);
  one_device({&q, &k, &v, &lam});
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, lens, lam, scale, O, LSE, workspace, status, stream); outputs None for new ones
PyObject* diff_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 11);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache"), &lens = tensor(a[3], "lens"),
                   &lam = tensor(a[4], "lam");
  at::Tensor O = tensor_or_none(a[6], "O"), lse = tensor_or_none(a[7], "LSE");
  const at::Tensor &ws = tensor(a[8], "workspace"), &status = tensor(a[9], "status");
  const Sizes z = diff_sizes(q, k, v, lam);
  const int64_t T = k.size(2);
  TORCH_CHECK_VALUE(z.S == 1, "q must hold one token a sequence: [B, Hq, 1, d]");
  TORCH_CHECK_VALUE(lens.dim() == 1 && lens.size(0) == z.B && lens.scalar_type() == at::kInt && lens.is_contiguous(),
                    "lens must be contiguous int32 [B]");
  TORCH_CHECK_VALUE(!T || (k.stride(3) == 1 && v.stride(3) == 1), "the columns of the caches must be consecutive");
  like(q, {&O});
  if (lse.defined()) check_lse(lse, z);
  check_scratch(ws, status);
  const c10::Device dev = one_device({&q, &k, &v, &lens, &lam, &ws, &status, &O, &lse});
  const float scale = scale_of(a[5], z);
  const cudaStream_t st = stream_of(a[10], dev);
  if (!O.defined()) O = at::empty(q.sizes(), q.options());
  if (!lse.defined()) lse = at::empty({z.B, z.Hq, 2, 1}, q.options().dtype(at::kFloat));
  int64_t ks[3], vs[3];
  for (int i = 0; i < 3; ++i) ks[i] = k.stride(i), vs[i] = v.stride(i);
  const int rc = call(dev, [&] {
    return decode_fn(z.dt, z.B, z.Hq, z.Hkv, z.d, T, q.data_ptr(), k.data_ptr(), ks, v.data_ptr(), vs,
                     static_cast<const int32_t*>(lens.data_ptr()), lam.data_ptr(), z.lam_n, scale, O.data_ptr(),
                     static_cast<float*>(lse.data_ptr()), ws.data_ptr(), ws.nbytes(), static_cast<int32_t*>(status.data_ptr()),
                     st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&O, &lse});
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind),     ENTRY(rope),       ENTRY(diff_fwd), ENTRY(diff_bwd),
                         ENTRY(diff_check), ENTRY(diff_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
