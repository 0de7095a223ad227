// Tensors to the C entry points of rotary positions, differential attention and its decoding, the paged cache and
// range-masked attention: checks of shapes, types, strides and devices, the outputs, the device and the stream.
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
decltype(&mesh_attn_paged_append) append_fn = nullptr;
decltype(&mesh_attn_paged_attn) paged_fn = nullptr;
decltype(&mesh_attn_range_fwd) range_fwd_fn = nullptr;
decltype(&mesh_attn_range_bwd) range_bwd_fn = nullptr;

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
  expect_args(n, 8);
  rope_fn = reinterpret_cast<decltype(rope_fn)>(pointer(a[0]));
  fwd_fn = reinterpret_cast<decltype(fwd_fn)>(pointer(a[1]));
  bwd_fn = reinterpret_cast<decltype(bwd_fn)>(pointer(a[2]));
  decode_fn = reinterpret_cast<decltype(decode_fn)>(pointer(a[3]));
  append_fn = reinterpret_cast<decltype(append_fn)>(pointer(a[4]));
  paged_fn = reinterpret_cast<decltype(paged_fn)>(pointer(a[5]));
  range_fwd_fn = reinterpret_cast<decltype(range_fwd_fn)>(pointer(a[6]));
  range_bwd_fn = reinterpret_cast<decltype(range_bwd_fn)>(pointer(a[7]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- rotary positions

// MeshRope's numbers as bytes: this header, the frequencies, the axes.
struct RopeHeader {
  int32_t d, groups, pairs, axes, adjacent, reserved;
};
struct RopeRef {
  RopeHeader h;
  const double* freq;
  const int32_t* axis;
};
RopeRef rope_of(PyObject* o) {
  TORCH_CHECK_TYPE(PyBytes_Check(o), "rope must be a MeshRope");
  RopeRef r;
  const char* raw = PyBytes_AS_STRING(o);
  TORCH_CHECK_VALUE(PyBytes_GET_SIZE(o) >= (Py_ssize_t)sizeof(r.h), "rope is not of a MeshRope");
  std::memcpy(&r.h, raw, sizeof(r.h));
  TORCH_CHECK_VALUE(r.h.pairs >= 0 && PyBytes_GET_SIZE(o) == (Py_ssize_t)(sizeof(r.h) + 12 * (size_t)r.h.pairs),
                    "rope is not of a MeshRope");
  r.freq = reinterpret_cast<const double*>(raw + sizeof(r.h));  // 8-byte aligned behind the object's own header
  r.axis = reinterpret_cast<const int32_t*>(raw + sizeof(r.h) + 8 * (size_t)r.h.pairs);
  return r;
}

// (handle, q, k, positions, q_out, k_out, inverse, stream); k and k_out None together, either output None
// for a new dense tensor
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 8);
  const RopeRef rope_ref = rope_of(a[0]);
  const RopeHeader& h = rope_ref.h;
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
  const double* freq = rope_ref.freq;
  const int32_t* axis = rope_ref.axis;
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

// ---------------------------------------------------------------- a paged cache

// The cache and the batch over it: pages, table, offsets and lengths that fit together.
struct Cache {
  int32_t Hkv, d, n_pages, page, B, max_pages;
  int64_t ks[3], vs[3], table_s;
  const int32_t *table, *offsets, *lens;
};
Cache cache_of(const at::Tensor& kp, const at::Tensor& vp, const at::Tensor& table, const at::Tensor& offsets, const at::Tensor& lens) {
  TORCH_CHECK_VALUE(kp.dim() == 4 && vp.sizes() == kp.sizes(), "k_pages and v_pages must be [n_pages, Hkv, page, d]");
  TORCH_CHECK_VALUE(vp.scalar_type() == kp.scalar_type(), "k_pages and v_pages must be of one dtype");
  TORCH_CHECK_VALUE(!kp.numel() || (kp.stride(3) == 1 && vp.stride(3) == 1), "the columns of the pages must be consecutive");
  TORCH_CHECK_VALUE(table.dim() == 2 && table.scalar_type() == at::kInt && (table.size(1) <= 1 || table.stride(1) == 1),
                    "table must be int32 [B, pages], its rows consecutive");
  const int64_t B = table.size(0);
  TORCH_CHECK_VALUE(offsets.dim() == 1 && offsets.size(0) == B + 1 && offsets.scalar_type() == at::kInt && offsets.is_contiguous(),
                    "offsets must be contiguous int32 [B + 1] with B = ", B);
  TORCH_CHECK_VALUE(lens.dim() == 1 && lens.size(0) == B && lens.scalar_type() == at::kInt && lens.is_contiguous(),
                    "lens must be contiguous int32 [B] with B = ", B);
  Cache c{};
  c.Hkv = i32(kp.size(1)), c.d = i32(kp.size(3)), c.n_pages = i32(kp.size(0)), c.page = i32(kp.size(2));
  c.B = i32(B), c.max_pages = i32(table.size(1));
  for (int i = 0; i < 3; ++i) c.ks[i] = kp.stride(i), c.vs[i] = vp.stride(i);
  c.table_s = table.stride(0);
  c.table = static_cast<const int32_t*>(table.data_ptr());
  c.offsets = static_cast<const int32_t*>(offsets.data_ptr());
  c.lens = static_cast<const int32_t*>(lens.data_ptr());
  return c;
}
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}
void check_status_block(const at::Tensor& status) {
  TORCH_CHECK_VALUE(status.scalar_type() == at::kInt && status.is_contiguous() && status.numel() >= MESH_ATTN_STATUS_WORDS,
                    "status must be ", MESH_ATTN_STATUS_WORDS, " or more contiguous int32 (new_status)");
}

// (rope or None, q or None, k, v, k_pages, v_pages, table, offsets, lens, positions or None, q_out or None, status, stream)
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 13);
  RopeRef rope{};
  if (a[0] != Py_None) rope = rope_of(a[0]);
  const at::Tensor q = tensor_or_none(a[1], "q");
  const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v"), &kp = tensor(a[4], "k_pages"), &vp = tensor(a[5], "v_pages");
  const at::Tensor &table = tensor(a[6], "table"), &offsets = tensor(a[7], "offsets"), &lens = tensor(a[8], "lens");
  const at::Tensor pos = tensor_or_none(a[9], "positions");
  at::Tensor q_out = tensor_or_none(a[10], "q_out");
  const at::Tensor& status = tensor(a[11], "status");
  const Cache c = cache_of(kp, vp, table, offsets, lens);
  TORCH_CHECK_VALUE(a[0] == Py_None || rope.h.d == c.d, "rope is for heads of ", rope.h.d, " columns; the pages have ", c.d);
  TORCH_CHECK_VALUE(k.dim() == 3 && k.size(1) == c.Hkv && k.size(2) == c.d && v.sizes() == k.sizes(), "k and v must be [N, ", c.Hkv,
                    ", ", c.d, "]");
  const int64_t N = k.size(0);
  const at::ScalarType type = kp.scalar_type();
  TORCH_CHECK_VALUE(q.defined() || !q_out.defined(), "q and q_out go together");
  if (q.defined())
    TORCH_CHECK_VALUE(q.dim() == 3 && q.size(0) == N && q.size(2) == c.d && (!q_out.defined() || q_out.sizes() == q.sizes()),
                      "q and q_out must be [N, Hq, ", c.d, "] with N = ", N);
  for (const at::Tensor* t : std::initializer_list<const at::Tensor*>{&q, &k, &v, &q_out})
    if (t->defined()) {
      TORCH_CHECK_VALUE(t->scalar_type() == type, "q, k, v and the pages must be of one dtype");
      TORCH_CHECK_VALUE(!t->numel() || t->stride(2) == 1, "the columns of a head must be consecutive");
    }
  check_status_block(status);
  int64_t ps[2] = {0, 0};
  if (pos.defined()) {
    TORCH_CHECK_VALUE(a[0] != Py_None, "positions without a rope");
    TORCH_CHECK_VALUE(pos.scalar_type() == at::kInt || pos.scalar_type() == at::kLong, "positions must be int32 or int64");
    const bool one = pos.dim() == 1 && rope.h.axes == 1 && pos.size(0) == N;
    const bool all = pos.dim() == 2 && pos.size(0) == rope.h.axes && pos.size(1) == N;
    TORCH_CHECK_VALUE(one || all, "positions must be [", rope.h.axes, ", N] ([N] for one axis) with N = ", N, "; got ", pos.sizes());
    if (all) ps[0] = pos.stride(0);
    ps[1] = pos.stride(pos.dim() - 1);
  }
  const mesh_attn_dtype dt = dtype_code(kp);
  const c10::Device dev = one_device({&kp, &vp, &k, &v, &table, &offsets, &lens, &status, &q, &q_out, &pos});
  if (q.defined() && !q_out.defined()) q_out = at::empty(q.sizes(), q.options());
  const auto strides = [](const at::Tensor& t, int64_t(&s)[2]) {
    for (int i = 0; i < 2; ++i) s[i] = t.defined() ? t.stride(i) : 0;
  };
  int64_t qs[2], qos[2], ks[2], vs[2];
  strides(q, qs), strides(q_out, qos), strides(k, ks), strides(v, vs);
  const int32_t Hq = q.defined() ? i32(q.size(1)) : 0;
  const cudaStream_t st = stream_of(a[12], dev);
  const int rc = call(dev, [&] {
    return append_fn(dt, N, c.B, Hq, c.Hkv, c.d, data(q), qs, data(q_out), qos, k.data_ptr(), ks, v.data_ptr(), vs, c.n_pages, c.page,
                     kp.data_ptr(), c.ks, vp.data_ptr(), c.vs, c.table, c.max_pages, c.table_s, c.offsets, c.lens,
                     a[0] == Py_None ? 1 : rope.h.groups, rope.h.pairs, a[0] == Py_None ? 1 : rope.h.axes, rope.freq, rope.axis,
                     rope.h.adjacent, data(pos), pos.defined() ? (int32_t)(8 * pos.element_size()) : 0, ps,
                     static_cast<int32_t*>(status.data_ptr()), st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&q_out});
  END_HANDLE_TH_ERRORS
}

void check_slopes(const at::Tensor& slopes, int64_t Hq) {
  TORCH_CHECK_VALUE(!slopes.defined() || (slopes.dim() == 1 && slopes.size(0) == Hq && slopes.scalar_type() == at::kFloat &&
                                          slopes.is_contiguous()),
                    "slopes must be contiguous fp32 [Hq] with Hq = ", Hq);
}
float scale_or(PyObject* o, int32_t d) { return o == Py_None ? (float)(1.0 / std::sqrt((double)d)) : (float)number(o); }

// (q, k_pages, v_pages, table, offsets, lens, max_new, scale, cap, slopes or None, window, O, LSE, workspace, status, stream)
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 16);
  const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
  const at::Tensor &table = tensor(a[3], "table"), &offsets = tensor(a[4], "offsets"), &lens = tensor(a[5], "lens");
  const at::Tensor slopes = tensor_or_none(a[9], "slopes");
  at::Tensor O = tensor_or_none(a[11], "O"), lse = tensor_or_none(a[12], "LSE");
  const at::Tensor &ws = tensor(a[13], "workspace"), &status = tensor(a[14], "status");
  const Cache c = cache_of(kp, vp, table, offsets, lens);
  TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == c.d, "q must be [N, Hq, ", c.d, "]");
  TORCH_CHECK_VALUE(c.Hkv >= 1 && q.size(1) % c.Hkv == 0, "Hq must be a multiple of Hkv: ", q.size(1), " and ", c.Hkv);
  TORCH_CHECK_VALUE(q.scalar_type() == kp.scalar_type(), "q and the pages must be of one dtype");
  TORCH_CHECK_VALUE(!q.numel() || q.stride(2) == 1, "the columns of a head must be consecutive");
  const int64_t N = q.size(0), Hq = q.size(1);
  check_slopes(slopes, Hq);
  TORCH_CHECK_VALUE(!O.defined() || (O.sizes() == q.sizes() && O.scalar_type() == q.scalar_type() && O.is_contiguous()),
                    "O must be contiguous, of q's shape and dtype");
  TORCH_CHECK_VALUE(!lse.defined() || (lse.sizes() == at::IntArrayRef({N, Hq}) && lse.scalar_type() == at::kFloat && lse.is_contiguous()),
                    "LSE must be contiguous fp32 [N, Hq]");
  check_scratch(ws, status);
  const mesh_attn_dtype dt = dtype_code(q);
  const c10::Device dev = one_device({&q, &kp, &vp, &table, &offsets, &lens, &ws, &status, &slopes, &O, &lse});
  const int64_t max_new = integer(a[6]), window = integer(a[10]);
  const float scale = scale_or(a[7], c.d), cap = (float)number(a[8]);
  const cudaStream_t st = stream_of(a[15], dev);
  if (!O.defined()) O = at::empty(q.sizes(), q.options());
  if (!lse.defined()) lse = at::empty({N, Hq}, q.options().dtype(at::kFloat));
  const int64_t qs[2] = {q.stride(0), q.stride(1)};
  const int32_t Hq32 = i32(Hq);
  const int rc = call(dev, [&] {
    return paged_fn(dt, N, c.B, Hq32, c.Hkv, c.d, q.data_ptr(), qs, c.n_pages, c.page, kp.data_ptr(), c.ks, vp.data_ptr(), c.vs,
                    c.table, c.max_pages, c.table_s, c.offsets, c.lens, max_new, scale, cap, static_cast<const float*>(data(slopes)),
                    window, O.data_ptr(), static_cast<float*>(lse.data_ptr()), ws.data_ptr(), ws.nbytes(),
                    static_cast<int32_t*>(status.data_ptr()), st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&O, &lse});
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- range-masked attention

struct RangeSizes {
  mesh_attn_dtype dt;
  int32_t B, Hq, Hkv, d;
  int64_t S, mask_s;
};
RangeSizes range_sizes(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v, const at::Tensor& lo, const at::Tensor& hi,
                       const at::Tensor& slopes) {
  TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4 && v.sizes() == k.sizes(), "q must be [B, Hq, S, d], k and v [B, Hkv, S, d]");
  TORCH_CHECK_VALUE(k.size(0) == q.size(0) && k.size(2) == q.size(2) && k.size(3) == q.size(3),
                    "q, k and v must agree in batch, tokens and columns");
  TORCH_CHECK_VALUE(k.size(1) >= 1 && q.size(1) % k.size(1) == 0, "Hq must be a multiple of Hkv: ", q.size(1), " and ", k.size(1));
  TORCH_CHECK_VALUE(k.scalar_type() == q.scalar_type() && v.scalar_type() == q.scalar_type(), "q, k and v must be of one dtype");
  TORCH_CHECK_VALUE(q.is_contiguous() && k.is_contiguous() && v.is_contiguous(), "q, k and v must be contiguous");
  const int64_t B = q.size(0), S = q.size(2);
  const auto fits = [&](const at::Tensor& t) {
    return t.scalar_type() == at::kInt && t.is_contiguous() &&
           ((t.dim() == 1 && t.size(0) == S) || (t.dim() == 2 && t.size(1) == S && (t.size(0) == B || t.size(0) == 1)));
  };
  TORCH_CHECK_VALUE(fits(lo) && fits(hi) && lo.sizes() == hi.sizes(), "lo and hi must be contiguous int32 [S] or [B, S] with B = ", B,
                    ", S = ", S);
  check_slopes(slopes, q.size(1));
  return {dtype_code(q), i32(B), i32(q.size(1)), i32(k.size(1)), i32(q.size(3)), S, lo.dim() == 2 && lo.size(0) > 1 ? S : 0};
}
void check_range_lse(const at::Tensor& lse, const RangeSizes& z) {
  TORCH_CHECK_VALUE(lse.scalar_type() == at::kFloat && lse.sizes() == at::IntArrayRef({z.B, z.Hq, z.S}) && lse.is_contiguous(),
                    "LSE must be contiguous fp32 [B, Hq, S]");
}
void like_range(const at::Tensor& q, std::initializer_list<const at::Tensor*> ts) {
  for (const at::Tensor* t : ts)
    TORCH_CHECK_VALUE(!t->defined() || (t->sizes() == q.sizes() && t->scalar_type() == q.scalar_type() && t->is_contiguous()),
                      "O, dO and dQ must be contiguous, of q's shape and dtype, dK and dV of k's");
}
const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }

// (q, k, v, lo, hi, slopes or None): raises where they do not fit together or are not on one CUDA device
PyObject* range_check(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 6);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &lo = tensor(a[3], "lo"),
                   &hi = tensor(a[4], "hi");
  const at::Tensor slopes = tensor_or_none(a[5], "slopes");
  range_sizes(q, k, v, lo, hi, slopes);
  one_device({&q, &k, &v, &lo, &hi, &slopes});
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (q, k, v, lo, hi, scale, cap, slopes or None, O, LSE, workspace, status, stream); outputs None for new ones
PyObject* range_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 13);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &lo = tensor(a[3], "lo"),
                   &hi = tensor(a[4], "hi");
  const at::Tensor slopes = tensor_or_none(a[7], "slopes");
  at::Tensor O = tensor_or_none(a[8], "O"), lse = tensor_or_none(a[9], "LSE");
  const at::Tensor &ws = tensor(a[10], "workspace"), &status = tensor(a[11], "status");
  const RangeSizes z = range_sizes(q, k, v, lo, hi, slopes);
  like_range(q, {&O});
  if (lse.defined()) check_range_lse(lse, z);
  check_scratch(ws, status);
  const c10::Device dev = one_device({&q, &k, &v, &lo, &hi, &ws, &status, &slopes, &O, &lse});
  const float scale = scale_or(a[5], z.d), cap = (float)number(a[6]);
  const cudaStream_t st = stream_of(a[12], dev);
  if (!O.defined()) O = at::empty(q.sizes(), q.options());
  if (!lse.defined()) lse = at::empty({z.B, z.Hq, z.S}, q.options().dtype(at::kFloat));
  const int rc = call(dev, [&] {
    return range_fwd_fn(z.dt, z.B, z.Hq, z.Hkv, z.S, z.d, q.data_ptr(), k.data_ptr(), v.data_ptr(), ints(lo), ints(hi), z.mask_s,
                        static_cast<const float*>(data(slopes)), scale, cap, O.data_ptr(), static_cast<float*>(lse.data_ptr()),
                        ws.data_ptr(), ws.nbytes(), static_cast<int32_t*>(status.data_ptr()), st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&O, &lse});
  END_HANDLE_TH_ERRORS
}

// (q, k, v, lo, hi, O, LSE, dO, scale, cap, slopes or None, dQ, dK, dV, workspace, status, stream); gradients None for new ones
PyObject* range_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 17);
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &lo = tensor(a[3], "lo"),
                   &hi = tensor(a[4], "hi");
  const at::Tensor &O = tensor(a[5], "O"), &lse = tensor(a[6], "LSE"), &dO = tensor(a[7], "dO");
  const at::Tensor slopes = tensor_or_none(a[10], "slopes");
  at::Tensor dQ = tensor_or_none(a[11], "dQ"), dK = tensor_or_none(a[12], "dK"), dV = tensor_or_none(a[13], "dV");
  const at::Tensor &ws = tensor(a[14], "workspace"), &status = tensor(a[15], "status");
  const RangeSizes z = range_sizes(q, k, v, lo, hi, slopes);
  like_range(q, {&O, &dO, &dQ});
  like_range(k, {&dK, &dV});
  check_range_lse(lse, z);
  check_scratch(ws, status);
  const c10::Device dev = one_device({&q, &k, &v, &lo, &hi, &O, &lse, &dO, &ws, &status, &slopes, &dQ, &dK, &dV});
  const float scale = scale_or(a[8], z.d), cap = (float)number(a[9]);
  const cudaStream_t st = stream_of(a[16], dev);
  if (!dQ.defined()) dQ = at::empty(q.sizes(), q.options());
  if (!dK.defined()) dK = at::empty(k.sizes(), k.options());
  if (!dV.defined()) dV = at::empty(v.sizes(), v.options());
  if (!q.numel()) {  // no rows: sums over nothing
    const c10::StreamGuard guard(c10::cuda::getStreamFromExternal(st, dev.index()).unwrap());
    for (const at::Tensor* t : {&dK, &dV}) t->zero_();
    return tuple_of({&dQ, &dK, &dV});
  }
  const int rc = call(dev, [&] {
    return range_bwd_fn(z.dt, z.B, z.Hq, z.Hkv, z.S, z.d, q.data_ptr(), k.data_ptr(), v.data_ptr(), ints(lo), ints(hi), z.mask_s,
                        static_cast<const float*>(data(slopes)), O.data_ptr(), static_cast<const float*>(lse.data_ptr()),
                        dO.data_ptr(), scale, cap, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws.data_ptr(), ws.nbytes(),
                        static_cast<int32_t*>(status.data_ptr()), st);
  });
  if (rc) return PyLong_FromLong(rc);
  return tuple_of({&dQ, &dK, &dV});
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind),     ENTRY(rope),       ENTRY(diff_fwd), ENTRY(diff_bwd),
                         ENTRY(diff_check), ENTRY(diff_decode), ENTRY(paged_append), ENTRY(paged_attn),
                         ENTRY(range_check), ENTRY(range_fwd), ENTRY(range_bwd), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
