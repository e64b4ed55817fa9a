// fa_bind.cpp -- argument marshalling of the decoding-step operators: what the
// package's qk_norm_rope, qk_norm_rope_backward, qk_norm_rope_append,
// decode_tree, verify_tree and compact_tree do between the caller's tensors and
// the C ABI (checks, outputs, pointers, the stream).
//
// Why native: these calls last 2 to 20 us on the GPU, and a decoding step makes
// them one after another, so the host's time per call is what the caller waits
// for.  The same checks in Python, through ctypes, took 12 to 28 us per call.
//
// The library's entry points are handed over as addresses (bind), so that this
// module and the ctypes binding use the one loaded copy.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "fa.h"

namespace {

decltype(&fa_qk_norm_rope) p_rope;
decltype(&fa_qk_norm_rope_append) p_append;
decltype(&fa_qk_norm_rope_backward) p_rope_backward;
decltype(&fa_decode_tree_fwd) p_tree;
decltype(&fa_verify_tree) p_verify;
decltype(&fa_compact_tree) p_compact;

struct Refused {
  PyObject* type;
  std::string text;
};
[[noreturn]] void bad_value(const std::string& text) { throw Refused{PyExc_ValueError, text}; }
[[noreturn]] void bad_type(const std::string& text) { throw Refused{PyExc_TypeError, text}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
void dims(const at::Tensor& t, const char* name, int n, const char* shape) {
  if (t.dim() != n) bad_value(std::string(name) + " must be " + shape);
}
int head_dtype(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return FA_BF16;
  if (t.scalar_type() == at::kHalf) return FA_FP16;
  bad_type(std::string(name) + " must be bf16 or fp16");
}
void same_dtype(const at::Tensor& t, const char* name, const at::Tensor& like) {
  if (t.scalar_type() != like.scalar_type())
    bad_type(std::string(name) + " must have the same dtype as the other heads");
}
void is_type(const at::Tensor& t, const char* name, at::ScalarType type, const char* type_name) {
  if (t.scalar_type() != type)
    bad_type(std::string(name) + " must be a " + type_name + " CUDA tensor");
}
void same_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) {
    std::string s = std::string(name) + " must have shape (";
    for (auto n : shape) s += std::to_string(n) + ", ";
    bad_value(s + ")");
  }
}
void contiguous(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) bad_value(std::string(name) + " must be a contiguous CUDA tensor");
}
void int32(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  is_type(t, name, at::kInt, "int32");
  same_shape(t, name, shape);
  contiguous(t, name);
}

// The current device, which all tensors must be on: kernels launch there.
struct Device {
  int index;
  explicit Device(const at::Tensor& first) {
    if (!first.is_cuda()) bad_value("tensors must be CUDA tensors on the current device");
    index = first.get_device();
    if (index != c10::cuda::current_device())
      bad_value("tensors must be CUDA tensors on the current device");
  }
  void has(const at::Tensor& t) const {
    if (!t.is_cuda() || t.get_device() != index)
      bad_value("tensors must be CUDA tensors on the current device");
  }
};

// The call's stream (None: torch's current one).  New outputs belong to it, so
// that their memory is neither still in use nor reused too early elsewhere.
struct Stream {
  cudaStream_t handle;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  Stream(PyObject* o, int device) {
    if (o == Py_None) {
      handle = c10::cuda::getCurrentCUDAStream(device).stream();
      return;
    }
    PyObject* v = PyObject_HasAttrString(o, "cuda_stream")
                      ? PyObject_GetAttrString(o, "cuda_stream")
                      : PyNumber_Index(o);
    if (!v) throw python_error();
    handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    if (PyErr_Occurred()) throw python_error();
    // (The legacy stream's handle is another name of the null stream.)
    const cudaStream_t own = handle == cudaStreamLegacy ? nullptr : handle;
    guard.emplace(c10::cuda::getStreamFromExternal(own, device));
  }
};

// A new tensor on the current device: at::empty without its dispatch.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const Device& dev) {
  return at::detail::empty_cuda(sizes, type, at::Device(at::kCUDA, dev.index), std::nullopt);
}
at::Tensor output(PyObject* given, const char* name, const at::Tensor& like, const Device& dev) {
  if (given == Py_None) return fresh(like.sizes(), like.scalar_type(), dev);
  const at::Tensor& t = tensor(given, name);
  if (t.scalar_type() != like.scalar_type() || t.sizes() != like.sizes())
    bad_value(std::string(name) + " must have the input's shape and dtype");
  contiguous(t, name);
  dev.has(t);
  return t;
}

// Stride between the tokens of [..., H, D]: heads contiguous, tokens at one
// stride (a slice of a packed projection is fine).
int64_t token_stride(const at::Tensor& t, const char* name) {
  const auto n = t.sizes(), st = t.strides();
  const int64_t k = t.dim(), H = n[k - 2], D = n[k - 1];
  if (t.numel() == 0) return H * D;
  bool ok = (st[k - 1] == 1 || D == 1) && (st[k - 2] == D || H == 1);
  int64_t stride = -1, step = 0;  // step: what the next leading axis must have
  for (int64_t i = k - 3; i >= 0 && ok; --i) {
    if (n[i] == 1) continue;
    if (stride < 0)
      stride = st[i];
    else
      ok = st[i] == step;
    step = st[i] * n[i];
  }
  if (!ok) bad_value(std::string(name) + ": heads must be contiguous and tokens at one stride");
  return stride < 0 ? H * D : stride;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
int narrow(int64_t v) {  // a size that the C ABI takes as an int
  return v > INT32_MAX ? INT32_MAX : static_cast<int>(v);
}

// The library's calls run without the interpreter's lock: a launch may wait for
// room in the stream's queue, and what makes room can need the lock (a host
// function in Python).
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... Args>
int unlocked(F* f, Args... args) {
  const Unlocked u;
  return f(args...);
}

PyObject* wrapped(std::initializer_list<at::Tensor> ts) {
  if (ts.size() == 1) return THPVariable_Wrap(*ts.begin());
  PyObject* r = PyTuple_New(ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const auto& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// The norm and rotation's shared arguments.
struct Heads {
  const at::Tensor &q, &k, &qw, &kw, &freq;
  const at::Tensor* pos = nullptr;
  int64_t T = 1, qs, ks;
  int Hq, Hkv, D, code;
  Heads(PyObject* const* a)
      : q(tensor(a[0], "q")), k(tensor(a[1], "k")), qw(tensor(a[2], "q_weight")),
        kw(tensor(a[3], "k_weight")), freq(tensor(a[4], "inv_freq")) {
    const int64_t n = q.dim();
    if (n < 2 || k.dim() != n) bad_value("q and k must be [..., heads, D]");
    D = narrow(q.size(n - 1));
    Hq = narrow(q.size(n - 2));
    Hkv = narrow(k.size(n - 2));
    if (k.sizes().slice(0, n - 2) != q.sizes().slice(0, n - 2) || k.size(n - 1) != D)
      bad_value("q and k must share their leading shape and head dimension");
    for (int64_t i = 0; i < n - 2; ++i) T *= q.size(i);
    code = head_dtype(q, "q");
    same_dtype(k, "k", q);
    same_dtype(qw, "q_weight", q);
    same_dtype(kw, "k_weight", q);
    const int64_t wd[1] = {D};
    same_shape(qw, "q_weight", wd);
    same_shape(kw, "k_weight", wd);
    is_type(freq, "inv_freq", at::kFloat, "float32");
    dims(freq, "inv_freq", 1, "[rot_dim / 2]");
    contiguous(qw, "q_weight");
    contiguous(kw, "k_weight");
    contiguous(freq, "inv_freq");
    qs = token_stride(q, "q");
    ks = token_stride(k, "k");
  }
  void positions(PyObject* o) {
    pos = &tensor(o, "positions");
    int32(*pos, "positions", q.sizes().slice(0, q.dim() - 2));
  }
  void on(const Device& d) const {
    for (const at::Tensor* t : {&k, &qw, &kw, &freq}) d.has(*t);
    if (pos) d.has(*pos);
  }
  int rot() const { return narrow(2 * freq.size(0)); }
};

// A paged cache [num_pages, page_size, Hkv, D], page table [B, max_pages] and
// lengths [B].
struct Pages {
  const at::Tensor &k, &v, &table, &lens;
  int num_pages, page_size, Hkv, D, max_pages;
  Pages(PyObject* kp, PyObject* vp, PyObject* tp, PyObject* lp, int64_t B, bool layers)
      : k(tensor(kp, "kpages")), v(tensor(vp, "vpages")), table(tensor(tp, "page_table")),
        lens(tensor(lp, "seqlens")) {
    const int64_t n = k.dim();
    if (n != 4 && !(layers && n == 5))
      bad_value(layers ? "kpages must be [num_pages,page_size,Hkv,D] or [layers,...]"
                       : "kpages must be [num_pages,page_size,Hkv,D]");
    same_shape(v, "vpages", k.sizes());
    same_dtype(v, "vpages", k);
    dims(table, "page_table", 2, "[B,max_pages]");
    const int64_t ts[2] = {B, table.size(1)}, ls[1] = {B};
    int32(table, "page_table", ts);
    int32(lens, "seqlens", ls);
    contiguous(k, "kpages");
    contiguous(v, "vpages");
    num_pages = narrow(k.size(n - 4));
    page_size = narrow(k.size(n - 3));
    Hkv = narrow(k.size(n - 2));
    D = narrow(k.size(n - 1));
    max_pages = narrow(table.size(1));
  }
  void on(const Device& d) const {
    for (const at::Tensor* t : {&k, &v, &table, &lens}) d.has(*t);
  }
};

const int32_t* i32(const at::Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); }
const float* f32(const at::Tensor& t) { return static_cast<const float*>(t.const_data_ptr()); }

// (q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, q_out, k_out, stream)
PyObject* norm_rope(PyObject* const* a) {
  Heads h(a);
  h.positions(a[5]);
  const Device dev(h.q);
  h.on(dev);
  Stream s(a[10], dev.index);
  const at::Tensor qo = output(a[8], "q_out", h.q, dev), ko = output(a[9], "k_out", h.k, dev);
  const int st = unlocked(
      p_rope, h.q.const_data_ptr(), h.k.const_data_ptr(), qo.data_ptr(), ko.data_ptr(),
      h.qw.const_data_ptr(), h.kw.const_data_ptr(), f32(h.freq), i32(*h.pos), h.T, h.Hq, h.Hkv, h.D,
      h.rot(), h.qs, h.ks, (float)number(a[6]), truth(a[7]), h.code, s.handle);
  return st ? PyLong_FromLong(st) : wrapped({qo, ko});
}

// (q, k, q_weight, k_weight, inv_freq, positions, eps, interleaved, dq_out, dk_out, stream)
PyObject* norm_rope_backward(PyObject* const* a) {
  Heads h(a);
  h.positions(a[5]);
  const at::Tensor &gq = tensor(a[8], "dq_out"), &gk = tensor(a[9], "dk_out");
  same_dtype(gq, "dq_out", h.q);
  same_dtype(gk, "dk_out", h.q);
  same_shape(gq, "dq_out", h.q.sizes());
  same_shape(gk, "dk_out", h.k.sizes());
  contiguous(gq, "dq_out");
  contiguous(gk, "dk_out");
  const Device dev(h.q);
  h.on(dev);
  dev.has(gq);
  dev.has(gk);
  Stream s(a[10], dev.index);
  const at::Tensor dq = fresh(h.q.sizes(), h.q.scalar_type(), dev);
  const at::Tensor dk = fresh(h.k.sizes(), h.k.scalar_type(), dev);
  const at::Tensor dqw = fresh({h.D}, at::kFloat, dev), dkw = fresh({h.D}, at::kFloat, dev);
  const int st = unlocked(
      p_rope_backward, gq.const_data_ptr(), gk.const_data_ptr(), h.q.const_data_ptr(),
      h.k.const_data_ptr(), h.qw.const_data_ptr(), h.kw.const_data_ptr(), f32(h.freq), i32(*h.pos),
      dq.data_ptr(), dk.data_ptr(), static_cast<float*>(dqw.data_ptr()),
      static_cast<float*>(dkw.data_ptr()), h.T, h.Hq, h.Hkv, h.D, h.rot(), h.qs, h.ks,
      (float)number(a[6]), truth(a[7]), h.code, s.handle);
  return st ? PyLong_FromLong(st) : wrapped({dq, dk, dqw, dkw});
}

// (q, k, q_weight, k_weight, inv_freq, v, kpages, vpages, page_table, seqlens, eps, positions,
//  interleaved, q_out, stream)
PyObject* append(PyObject* const* a) {
  Heads h(a);
  dims(h.q, "q", 4, "[B,N,Hq,D]");
  const at::Tensor& v = tensor(a[5], "v");
  same_dtype(v, "v", h.q);
  same_shape(v, "v", h.k.sizes());
  const int64_t vs = token_stride(v, "v");
  const Pages p(a[6], a[7], a[8], a[9], h.q.size(0), false);
  same_dtype(p.k, "kpages", h.q);
  if (p.Hkv != h.Hkv || p.D != h.D) bad_value("kpages must be [num_pages,page_size,Hkv,D]");
  if (a[11] != Py_None) h.positions(a[11]);
  const Device dev(h.q);
  h.on(dev);
  dev.has(v);
  p.on(dev);
  Stream s(a[14], dev.index);
  const at::Tensor qo = output(a[13], "q_out", h.q, dev);
  const int st = unlocked(
      p_append, h.q.const_data_ptr(), h.k.const_data_ptr(), v.const_data_ptr(), qo.data_ptr(),
      p.k.data_ptr(), p.v.data_ptr(), h.qw.const_data_ptr(), h.kw.const_data_ptr(), f32(h.freq),
      h.pos ? i32(*h.pos) : nullptr, i32(p.table), i32(p.lens), narrow(h.q.size(0)),
      narrow(h.q.size(1)), h.Hq, h.Hkv, p.num_pages, p.page_size, p.max_pages, h.D, h.rot(), h.qs,
      h.ks, vs, (float)number(a[10]), truth(a[12]), h.code, s.handle);
  return st ? PyLong_FromLong(st) : wrapped({qo});
}

// (q, kpages, vpages, page_table, seqlens, parents, scale, out, stream, lse)
PyObject* tree(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  dims(q, "q", 4, "[B,N,Hq,D]");
  const int code = head_dtype(q, "q");
  const int64_t B = q.size(0), N = q.size(1), Hq = q.size(2);
  const Pages p(a[1], a[2], a[3], a[4], B, false);
  same_dtype(p.k, "kpages", q);
  if (p.D != q.size(3)) bad_value("kpages must be [num_pages,page_size,Hkv,D]");
  const at::Tensor& parents = tensor(a[5], "parents");
  const int64_t bn[2] = {B, N}, rows[3] = {B, N, Hq};
  int32(parents, "parents", bn);
  contiguous(q, "q");
  const Device dev(q);
  p.on(dev);
  dev.has(parents);
  Stream s(a[8], dev.index);
  const at::Tensor out = output(a[7], "out", q, dev);
  at::Tensor lse;
  const bool want = a[9] != Py_None && a[9] != Py_False;
  if (a[9] == Py_True) {
    lse = fresh(rows, at::kFloat, dev);
  } else if (want) {
    lse = tensor(a[9], "lse");
    if (lse.scalar_type() != at::kFloat) bad_value("lse must be a float32 tensor [B,N,Hq]");
    same_shape(lse, "lse", rows);
    contiguous(lse, "lse");
    dev.has(lse);
  }
  const int st = unlocked(
      p_tree, q.const_data_ptr(), p.k.const_data_ptr(), p.v.const_data_ptr(), i32(p.table),
      i32(p.lens), i32(parents), out.data_ptr(),
      want ? static_cast<float*>(lse.data_ptr()) : nullptr, narrow(B), narrow(N), narrow(Hq), p.Hkv,
      p.num_pages, p.page_size, p.max_pages, p.D, (float)number(a[6]), code, s.handle);
  if (st) return PyLong_FromLong(st);
  return want ? wrapped({out, lse}) : wrapped({out});
}

// (target_probs, draft_probs, tokens, parents, uniforms, stream)
PyObject* verify(PyObject* const* a) {
  const at::Tensor& p = tensor(a[0], "target_probs");
  dims(p, "target_probs", 3, "[B,N,V]");
  is_type(p, "target_probs", at::kFloat, "float32");
  const at::Tensor* q = a[1] == Py_None ? nullptr : &tensor(a[1], "draft_probs");
  const at::Tensor &tokens = tensor(a[2], "tokens"), &parents = tensor(a[3], "parents"),
                   &u = tensor(a[4], "uniforms");
  const int64_t bn[2] = {p.size(0), p.size(1)}, b1[1] = {p.size(0)};
  if (q) {
    is_type(*q, "draft_probs", at::kFloat, "float32");
    same_shape(*q, "draft_probs", p.sizes());
    contiguous(*q, "draft_probs");
  }
  is_type(u, "uniforms", at::kFloat, "float32");
  same_shape(u, "uniforms", bn);
  contiguous(p, "target_probs");
  contiguous(u, "uniforms");
  int32(tokens, "tokens", bn);
  int32(parents, "parents", bn);
  const Device dev(p);
  if (q) dev.has(*q);
  dev.has(tokens);
  dev.has(parents);
  dev.has(u);
  Stream s(a[5], dev.index);
  const at::Tensor path = fresh(bn, at::kInt, dev), count = fresh(b1, at::kInt, dev),
                   next = fresh(b1, at::kInt, dev);
  const int st =
      unlocked(p_verify, f32(p), q ? f32(*q) : nullptr, i32(tokens), i32(parents), f32(u),
               static_cast<int32_t*>(path.data_ptr()), static_cast<int32_t*>(count.data_ptr()),
               static_cast<int32_t*>(next.data_ptr()), narrow(bn[0]), narrow(bn[1]),
               narrow(p.size(2)), s.handle);
  return st ? PyLong_FromLong(st) : wrapped({path, count, next});
}

// (kpages, vpages, page_table, seqlens, path, count, seqlens_out, stream)
PyObject* compact(PyObject* const* a) {
  const at::Tensor &path = tensor(a[4], "path"), &count = tensor(a[5], "count");
  dims(path, "path", 2, "[B,N]");
  const int64_t B = path.size(0), b1[1] = {B};
  const Pages p(a[0], a[1], a[2], a[3], B, true);
  head_dtype(p.k, "kpages");
  int32(path, "path", path.sizes());
  int32(count, "count", b1);
  const Device dev(p.k);
  p.on(dev);
  dev.has(path);
  dev.has(count);
  Stream s(a[7], dev.index);
  const at::Tensor out = output(a[6], "seqlens_out", p.lens, dev);
  const int st = unlocked(
      p_compact, p.k.data_ptr(), p.v.data_ptr(), i32(p.table), i32(p.lens), i32(path), i32(count),
      static_cast<int32_t*>(out.data_ptr()), p.k.dim() == 5 ? narrow(p.k.size(0)) : 1, narrow(B),
      narrow(path.size(1)), p.Hkv, p.num_pages, p.page_size, p.max_pages, p.D, s.handle);
  return st ? PyLong_FromLong(st) : wrapped({out});
}

// (tensor): its token stride.
PyObject* stride_of(PyObject* const* a) {
  return PyLong_FromLongLong(token_stride(tensor(a[0], "x"), "x"));
}

// (addresses of the library's six entry points)
PyObject* bind(PyObject* const* a) {
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) throw python_error();
  }
  p_rope = reinterpret_cast<decltype(p_rope)>(p[0]);
  p_append = reinterpret_cast<decltype(p_append)>(p[1]);
  p_rope_backward = reinterpret_cast<decltype(p_rope_backward)>(p[2]);
  p_tree = reinterpret_cast<decltype(p_tree)>(p[3]);
  p_verify = reinterpret_cast<decltype(p_verify)>(p[4]);
  p_compact = reinterpret_cast<decltype(p_compact)>(p[5]);
  Py_RETURN_NONE;
}

// A call with exactly N positional arguments; results, or a status other than
// FA_OK as an int.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind, 6>("bind"),
                         method<norm_rope, 11>("qk_norm_rope"),
                         method<norm_rope_backward, 11>("qk_norm_rope_backward"),
                         method<append, 15>("qk_norm_rope_append"),
                         method<tree, 10>("decode_tree"),
                         method<verify, 6>("verify_tree"),
                         method<compact, 8>("compact_tree"),
                         method<stride_of, 1>("token_stride"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_bind() {
  PyObject* m = PyModule_Create(&module);
  // The torch whose headers were compiled in: the package checks it on loading.
  if (m && PyModule_AddStringConstant(m, "torch_version", FA_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
