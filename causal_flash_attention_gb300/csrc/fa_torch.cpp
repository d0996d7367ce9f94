// Native part of the Python binding: the span, ragged, query/key-preparation and latent
// calls of libfa (include/fa.h) on torch tensors. Each function checks its
// tensors (a tensor on another device, of another type or size would have the
// kernels read memory that is not its own), allocates what the caller did not
// give, and makes one call of the library; no computation happens here.
//
// A serving step is a handful of such calls whose kernels take 5 to 10 us, so the
// host side of a call counts: through ctypes and Python checks a forward one cost
// 17 to 28 us (allocations included), here 5 to 6, of which the library and the
// launch are 1.7 to 3.6 (a backward: 11 to 13 us).
//
// The library is given by its dlopen handle (the first argument of every
// function), so that these calls and the ctypes ones always use the same copy.
// A function returns its tensors, or the library's negative error code as an int;
// bad tensors raise ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <sstream>
#include <string>
#include <utility>

#include "../../include/fa.h"

namespace {

using at::Tensor;

struct BadArgument {
  std::string text;
};

// The entry points of the library last called.
struct Library {
  void* handle = nullptr;
  decltype(&fa_fwd_span) fwd_span;
  decltype(&fa_bwd_span) bwd_span;
  decltype(&fa_bwd_span_workspace_bytes) bwd_span_bytes;
  decltype(&fa_fwd_ragged_paged) ragged;
  decltype(&fa_fwd_ragged_paged_workspace_bytes) ragged_bytes;
  decltype(&fa_qk_norm_rope) norm_rope;
  decltype(&fa_qk_norm_rope_bwd) norm_rope_bwd;
  decltype(&fa_qk_norm_rope_bwd_workspace_bytes) norm_rope_bwd_bytes;
  decltype(&fa_qk_norm_rope_append) append;
};

// Those of latent attention, found by themselves on their first use: the calls above also run on the handle of
// a library that has only theirs, as the binding's own tests give them. (The package loads none without these.)
struct LatentLibrary {
  void* handle = nullptr;
  decltype(&fa_fwd_latent) fwd;
  decltype(&fa_bwd_latent) bwd;
  decltype(&fa_bwd_latent_workspace_bytes) bwd_bytes;
  decltype(&fa_fwd_latent_paged) paged;
  decltype(&fa_fwd_latent_paged_workspace_bytes) paged_bytes;
  decltype(&fa_latent_append) append;
};

template <typename F>
void find(void* handle, const char* name, F& f) {
  f = reinterpret_cast<F>(dlsym(handle, name));
  if (!f) throw BadArgument{std::string("the library has no ") + name};
}

const Library& library(PyObject* o) {
  static Library lib;   // guarded by the interpreter lock
  void* handle = PyLong_AsVoidPtr(o);
  if (handle == lib.handle && handle) return lib;
  if (!handle) throw BadArgument{"no library handle"};
  Library l;
  find(handle, "fa_fwd_span", l.fwd_span);
  find(handle, "fa_bwd_span", l.bwd_span);
  find(handle, "fa_bwd_span_workspace_bytes", l.bwd_span_bytes);
  find(handle, "fa_fwd_ragged_paged", l.ragged);
  find(handle, "fa_fwd_ragged_paged_workspace_bytes", l.ragged_bytes);
  find(handle, "fa_qk_norm_rope", l.norm_rope);
  find(handle, "fa_qk_norm_rope_bwd", l.norm_rope_bwd);
  find(handle, "fa_qk_norm_rope_bwd_workspace_bytes", l.norm_rope_bwd_bytes);
  find(handle, "fa_qk_norm_rope_append", l.append);
  l.handle = handle;
  lib = l;
  return lib;
}

const LatentLibrary& latent_library(PyObject* o) {
  static LatentLibrary lib;   // guarded by the interpreter lock
  void* handle = PyLong_AsVoidPtr(o);
  if (handle == lib.handle && handle) return lib;
  if (!handle) throw BadArgument{"no library handle"};
  LatentLibrary l;
  find(handle, "fa_fwd_latent", l.fwd);
  find(handle, "fa_bwd_latent", l.bwd);
  find(handle, "fa_bwd_latent_workspace_bytes", l.bwd_bytes);
  find(handle, "fa_fwd_latent_paged", l.paged);
  find(handle, "fa_fwd_latent_paged_workspace_bytes", l.paged_bytes);
  find(handle, "fa_latent_append", l.append);
  l.handle = handle;
  lib = l;
  return lib;
}

// ------------------------------------------------------------- arguments --
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw BadArgument{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
Tensor maybe(PyObject* o, const char* name) { return o == Py_None ? Tensor() : tensor(o, name); }

float real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw BadArgument{""};
  return static_cast<float>(x);
}
int integer(PyObject* o) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw BadArgument{""};
  if (x != static_cast<int>(x)) throw BadArgument{"an integer argument does not fit into 32 bits"};
  return static_cast<int>(x);
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw BadArgument{""};
  return x == 1;
}

int dtype_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return FA_F32;
    case at::kHalf: return FA_F16;
    case at::kBFloat16: return FA_BF16;
    default: return -1;
  }
}

std::string describe(const Tensor& t) {
  std::ostringstream s;
  s << (t.is_contiguous() ? "a " : "a strided ") << t.scalar_type() << " tensor " << t.sizes()
    << " on " << t.device();
  return s.str();
}
[[noreturn]] void misfit(const char* name, const Tensor& t, const char* kind, at::Device dev,
                         at::ScalarType dt, at::IntArrayRef sizes) {
  std::ostringstream s;
  s << name << " must be a " << kind << dt << " tensor " << sizes << " on " << dev << ", not "
    << describe(t);
  throw BadArgument{s.str()};
}

using Sizes = std::initializer_list<int64_t>;

// t has to be contiguous, on dev, of this type and size
void fit(const char* name, const Tensor& t, at::Device dev, at::ScalarType dt, at::IntArrayRef sizes) {
  if (t.device() != dev || t.scalar_type() != dt || t.sizes() != sizes || !t.is_contiguous())
    misfit(name, t, "contiguous ", dev, dt, sizes);
}
void fit(const char* name, const Tensor& t, at::Device dev, at::ScalarType dt, Sizes sizes) {
  fit(name, t, dev, dt, at::IntArrayRef(sizes.begin(), sizes.size()));
}

at::Device cuda_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw BadArgument{std::string(name) + " must be a CUDA tensor"};
  return t.device();
}

void four_dims(const Tensor& t, const char* what) {
  if (t.dim() != 4) throw BadArgument{what};
}

template <typename T>
T* data(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

// Other Python threads run while a call allocates and launches, either of which may wait
// for the GPU (memory to be freed, a full launch queue). From here to end() nothing
// touches a Python object.
class Released {
  PyThreadState* state_ = PyEval_SaveThread();

 public:
  Released() = default;
  Released(const Released&) = delete;
  ~Released() { end(); }
  void end() {
    if (state_) PyEval_RestoreThread(state_);
    state_ = nullptr;
  }
};

// Where a call runs and allocates: the tensors' device, and the current stream
// or the one given by its handle. Memory comes from that stream's own pool, so
// that its earlier and later users are ordered with the call.
struct Place {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  fa_stream_t stream;
  Place(at::Device dev, PyObject* o) : device(dev) {
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
      return;
    }
    stream = static_cast<fa_stream_t>(PyLong_AsVoidPtr(o));
    if (PyErr_Occurred()) throw BadArgument{""};
    guard.emplace(c10::cuda::getStreamFromExternal(stream, dev.index()));
  }
};

// (allocated without the operator dispatch of at::empty: a call's few outputs are a
// good part of its host time)
Tensor empty(at::IntArrayRef sizes, at::Device dev, at::ScalarType dt) {
  return Tensor(at::detail::empty_cuda(sizes, dt, dev, std::nullopt));
}
// [B, H, S, d], laid out [B, S, H, d]
Tensor empty_tokens_first(int64_t B, int64_t H, int64_t S, int64_t d, at::Device dev, at::ScalarType dt) {
  return Tensor(at::detail::empty_strided_cuda({B, H, S, d}, {S * H * d, d, H * d, 1}, dt, dev));
}
Tensor workspace_of(size_t bytes, at::Device dev) {
  return empty({static_cast<int64_t>(bytes)}, dev, at::kByte);
}
size_t workspace_bytes(const Tensor& t, at::Device dev) {
  if (!t.defined()) return 0;
  if (t.device() != dev || !t.is_contiguous()) {
    std::ostringstream s;
    s << "workspace must be contiguous and on " << dev;
    throw BadArgument{s.str()};
  }
  return t.nbytes();
}

// Sizes go to the library as 32-bit integers.
int narrow(int64_t x) {
  if (x > 0x7fffffff) throw BadArgument{"a dimension does not fit into 32 bits"};
  return static_cast<int>(x);
}

PyObject* tensors(std::initializer_list<Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o;
    if (t.defined()) {
      o = THPVariable_Wrap(t);
    } else {
      o = Py_None;
      Py_INCREF(o);
    }
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// ------------------------------------------------------------------ spans --
struct SpanDims {
  int B, Hq, Hkv, Sq, Skv, d;
};
SpanDims span_inputs(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& begin,
                     const Tensor& end, const Tensor& slopes) {
  const at::Device dev = cuda_device(q, "q");
  four_dims(q, "q and k must be [B, H, S, d]");
  four_dims(k, "q and k must be [B, H, S, d]");
  const auto dt = q.scalar_type();
  const int64_t B = q.size(0), Sq = q.size(2), d = q.size(3), Hkv = k.size(1), Skv = k.size(2);
  if (!q.is_contiguous()) throw BadArgument{"q must be contiguous"};
  fit("k", k, dev, dt, {B, Hkv, Skv, d});
  fit("v", v, dev, dt, {B, Hkv, Skv, d});
  fit("key_begin", begin, dev, at::kInt, {B, Sq});
  fit("key_end", end, dev, at::kInt, {B, Sq});
  if (slopes.defined()) fit("slopes", slopes, dev, at::kFloat, {q.size(1)});
  return {narrow(B), narrow(q.size(1)), narrow(Hkv), narrow(Sq), narrow(Skv), narrow(d)};
}

float scale_of(PyObject* o, int d) {
  return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : real(o);
}

// (handle, q, k, v, key_begin, key_end, out, lse, softcap, slopes, scale, stream)
PyObject* span_forward(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  const Tensor &begin = tensor(a[4], "key_begin"), &end = tensor(a[5], "key_end");
  Tensor out = maybe(a[6], "out"), lse = maybe(a[7], "lse");
  const Tensor slopes = maybe(a[9], "slopes");
  const SpanDims n = span_inputs(q, k, v, begin, end, slopes);
  const float scale = scale_of(a[10], n.d), softcap = real(a[8]);
  const Place at(q.device(), a[11]);
  Released released;
  if (out.defined()) fit("out", out, q.device(), q.scalar_type(), q.sizes());
  else out = empty(q.sizes(), q.device(), q.scalar_type());
  if (lse.defined()) fit("lse", lse, q.device(), at::kFloat, q.sizes().slice(0, 3));
  else lse = empty(q.sizes().slice(0, 3), q.device(), at::kFloat);
  const int rc = lib.fwd_span(q.data_ptr(), k.data_ptr(), v.data_ptr(), data<int>(begin),
                              data<int>(end), out.data_ptr(), data<float>(lse), n.B, n.Hq, n.Hkv,
                              n.Sq, n.Skv, n.d, scale, softcap, data<float>(slopes),
                              dtype_code(q), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({out, lse});
}

// (handle, q, k, v, key_begin, key_end, out, dout, lse, dq, dk, dv, workspace, softcap, slopes,
//  scale, stream)
PyObject* span_backward(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  const Tensor &begin = tensor(a[4], "key_begin"), &end = tensor(a[5], "key_end");
  const Tensor &out = tensor(a[6], "out"), &dout = tensor(a[7], "dout"), &lse = tensor(a[8], "lse");
  Tensor dq = maybe(a[9], "dq"), dk = maybe(a[10], "dk"), dv = maybe(a[11], "dv");
  Tensor ws = maybe(a[12], "workspace");
  const Tensor slopes = maybe(a[14], "slopes");
  const SpanDims n = span_inputs(q, k, v, begin, end, slopes);
  const at::Device dev = q.device();
  const auto dt = q.scalar_type();
  fit("out", out, dev, dt, q.sizes());
  fit("dout", dout, dev, dt, q.sizes());
  fit("lse", lse, dev, at::kFloat, q.sizes().slice(0, 3));
  const float scale = scale_of(a[15], n.d), softcap = real(a[13]);
  const Place at(dev, a[16]);
  Released released;
  for (auto& [name, g, like] : {std::tuple<const char*, Tensor&, const Tensor&>{"dq", dq, q},
                                {"dk", dk, k}, {"dv", dv, k}}) {
    if (g.defined()) fit(name, g, dev, dt, like.sizes());
    else g = empty(like.sizes(), dev, dt);
  }
  if (!ws.defined()) ws = workspace_of(lib.bwd_span_bytes(n.B, n.Hq, n.Hkv, n.Sq, n.Skv, n.d), dev);
  const int rc = lib.bwd_span(q.data_ptr(), k.data_ptr(), v.data_ptr(), data<int>(begin),
                              data<int>(end), out.data_ptr(), dout.data_ptr(), data<float>(lse),
                              dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), n.B, n.Hq, n.Hkv, n.Sq,
                              n.Skv, n.d, scale, softcap, data<float>(slopes), dtype_code(q),
                              ws.data_ptr(), workspace_bytes(ws, dev), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({dq, dk, dv});
}

// ----------------------------------------------------------------- ragged --
struct CacheDims {
  int block_size, num_blocks, max_blocks;
};
CacheDims cache_inputs(at::Device dev, at::ScalarType dt, int64_t B, int64_t Hkv, int64_t d,
                       const Tensor& kc, const Tensor& vc, const Tensor& table, const Tensor& lens) {
  if (kc.dim() != 4 || table.dim() != 2)
    throw BadArgument{"caches [num_blocks,Hkv,block_size,d], table [B,max_blocks]"};
  fit("k_cache", kc, dev, dt, {kc.size(0), Hkv, kc.size(2), d});
  fit("v_cache", vc, dev, dt, kc.sizes());
  fit("block_table", table, dev, at::kInt, {B, table.size(1)});
  fit("seq_lens", lens, dev, at::kInt, {B});
  return {narrow(kc.size(2)), narrow(kc.size(0)), narrow(table.size(1))};
}

// (handle, q, k_cache, v_cache, block_table, seq_lens, out, lse, workspace, window, softcap,
//  slopes, scale, stream)
PyObject* ragged(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
  const Tensor &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seq_lens");
  Tensor out = maybe(a[6], "out"), lse = maybe(a[7], "lse"), ws = maybe(a[8], "workspace");
  const Tensor slopes = maybe(a[11], "slopes");
  const at::Device dev = cuda_device(q, "q");
  const auto dt = q.scalar_type();
  if (q.dim() != 4 || kc.dim() != 4 || !q.is_contiguous())
    throw BadArgument{"q [B,Hq,Sq,d] contiguous, caches [num_blocks,Hkv,block_size,d]"};
  const int B = narrow(q.size(0)), Hq = narrow(q.size(1)), Sq = narrow(q.size(2)), d = narrow(q.size(3));
  const int Hkv = narrow(kc.size(1));
  const CacheDims c = cache_inputs(dev, dt, B, Hkv, d, kc, vc, table, lens);
  if (slopes.defined()) fit("slopes", slopes, dev, at::kFloat, {Hq});
  const int window = integer(a[9]);
  const float scale = scale_of(a[12], d), softcap = real(a[10]);
  const Place at(dev, a[13]);
  Released released;
  if (out.defined()) fit("out", out, dev, dt, q.sizes());
  else out = empty(q.sizes(), dev, dt);
  if (lse.defined()) fit("lse", lse, dev, at::kFloat, q.sizes().slice(0, 3));
  else lse = empty(q.sizes().slice(0, 3), dev, at::kFloat);
  if (!ws.defined())
    ws = workspace_of(lib.ragged_bytes(B, Hq, Hkv, Sq, d, c.block_size, c.max_blocks), dev);
  const int rc = lib.ragged(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), data<int>(table),
                            data<int>(lens), out.data_ptr(), data<float>(lse), B, Hq, Hkv, Sq, d,
                            c.block_size, c.num_blocks, c.max_blocks, window, scale, softcap,
                            data<float>(slopes), dtype_code(q),
                            ws.data_ptr(), workspace_bytes(ws, dev), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({out, lse});
}

// ---------------------------------------------------- query / key heads --
// The fa_view of a [B, H, S, d] tensor of any strides but the last.
fa_view view(const char* name, const Tensor& t, at::Device dev, at::ScalarType dt, Sizes sizes,
             bool written = false) {
  const at::IntArrayRef want(sizes.begin(), sizes.size());
  if (t.device() != dev || t.scalar_type() != dt || t.sizes() != want) misfit(name, t, "", dev, dt, want);
  const auto st = t.strides();
  if (st[3] != 1) throw BadArgument{std::string(name) + ": the elements of a head must be contiguous"};
  if (written && !t.is_contiguous()) {
    std::pair<int64_t, int64_t> dims[3] = {{st[0], want[0]}, {st[1], want[1]}, {st[2], want[2]}};
    std::sort(dims, dims + 3);
    int64_t reach = want[3];
    for (const auto& [stride, n] : dims) {
      if (n <= 1) continue;
      if (stride < reach) throw BadArgument{std::string(name) + ": elements overlap in memory"};
      reach = stride * n;
    }
  }
  // a dimension of one row has no stride to keep aligned
  return fa_view{t.data_ptr(), want[0] > 1 ? st[0] : 0, want[1] > 1 ? st[1] : 0, want[2] > 1 ? st[2] : 0};
}

struct RopeArgs {
  Tensor turns, positions, wq, wk;
  int rope_dim = 0;
};
RopeArgs rope_inputs(at::Device dev, at::ScalarType dt, int64_t B, int64_t S, int64_t d,
                     PyObject* turns, PyObject* positions, PyObject* wq, PyObject* wk) {
  RopeArgs r;
  r.turns = maybe(turns, "turns");
  r.positions = maybe(positions, "positions");
  r.wq = maybe(wq, "q_weight");
  r.wk = maybe(wk, "k_weight");
  if (r.turns.defined()) {
    fit("turns", r.turns, dev, at::kLong, {r.turns.numel()});
    r.rope_dim = narrow(2 * r.turns.numel());
  }
  if (r.positions.defined()) fit("positions", r.positions, dev, at::kInt, {B, S});
  if (r.wq.defined()) fit("q_weight", r.wq, dev, dt, {d});
  if (r.wk.defined()) fit("k_weight", r.wk, dev, dt, {d});
  return r;
}

struct HeadDims {
  at::Device dev;
  at::ScalarType dt;
  int B, Hq, Hkv, S, d;
};
HeadDims head_dims(const Tensor& q, const Tensor& k, const char* name) {
  const at::Device dev = cuda_device(q, name);
  four_dims(q, "q [B,Hq,S,d] and k [B,Hkv,S,d] (any strides but the last)");
  four_dims(k, "q [B,Hq,S,d] and k [B,Hkv,S,d] (any strides but the last)");
  return {dev, q.scalar_type(), narrow(q.size(0)), narrow(q.size(1)), narrow(k.size(1)),
          narrow(q.size(2)), narrow(q.size(3))};
}

// (handle, q, k, q_out, k_out, turns, positions, q_weight, k_weight, eps, interleaved,
//  rope_scale, stream)
PyObject* norm_rope(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k");
  Tensor qo = maybe(a[3], "q_out"), ko = maybe(a[4], "k_out");
  const HeadDims n = head_dims(q, k, "q");
  const RopeArgs r = rope_inputs(n.dev, n.dt, n.B, n.S, n.d, a[5], a[6], a[7], a[8]);
  const Sizes qs = {n.B, n.Hq, n.S, n.d}, ks = {n.B, n.Hkv, n.S, n.d};
  const fa_view vq = view("q", q, n.dev, n.dt, qs), vk = view("k", k, n.dev, n.dt, ks);
  const float eps = real(a[9]), rope_scale = real(a[11]);
  const bool interleaved = truth(a[10]);
  const Place at(n.dev, a[12]);
  Released released;
  if (!qo.defined()) qo = empty(q.sizes(), n.dev, n.dt);
  if (!ko.defined()) ko = empty(k.sizes(), n.dev, n.dt);
  const fa_view vqo = view("q_out", qo, n.dev, n.dt, qs, true);
  const fa_view vko = view("k_out", ko, n.dev, n.dt, ks, true);
  const int rc = lib.norm_rope(&vq, &vk, &vqo, &vko, data<void>(r.wq), data<void>(r.wk), eps,
                               data<int>(r.positions), data<unsigned long long>(r.turns), r.rope_dim,
                               interleaved, rope_scale, n.B, n.Hq, n.Hkv, n.S, n.d, dtype_code(q),
                               at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({qo, ko});
}

// (handle, dq_out, dk_out, q, k, dq, dk, dq_weight, dk_weight, workspace, turns, positions,
//  q_weight, k_weight, eps, interleaved, rope_scale, allocate, stream); allocate: give what is
//  missing, dq and dk as projections lay q and k out
PyObject* norm_rope_bwd(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &dqo = tensor(a[1], "dq_out"), &dko = tensor(a[2], "dk_out");
  const Tensor q = maybe(a[3], "q"), k = maybe(a[4], "k");
  Tensor dq = maybe(a[5], "dq"), dk = maybe(a[6], "dk"), dwq = maybe(a[7], "dq_weight"),
         dwk = maybe(a[8], "dk_weight"), ws = maybe(a[9], "workspace");
  const HeadDims n = head_dims(dqo, dko, "dq_out");
  const RopeArgs r = rope_inputs(n.dev, n.dt, n.B, n.S, n.d, a[10], a[11], a[12], a[13]);
  const Sizes qs = {n.B, n.Hq, n.S, n.d}, ks = {n.B, n.Hkv, n.S, n.d};
  const fa_view vdqo = view("dq_out", dqo, n.dev, n.dt, qs), vdko = view("dk_out", dko, n.dev, n.dt, ks);
  fa_view vq{}, vk{};
  if (q.defined()) vq = view("q", q, n.dev, n.dt, qs);
  if (k.defined()) vk = view("k", k, n.dev, n.dt, ks);
  const float eps = real(a[14]), rope_scale = real(a[16]);
  const bool interleaved = truth(a[15]), allocate = truth(a[17]);
  const Place at(n.dev, a[18]);
  Released released;
  if (allocate) {
    if (!dq.defined()) dq = empty_tokens_first(n.B, n.Hq, n.S, n.d, n.dev, n.dt);
    if (!dk.defined()) dk = empty_tokens_first(n.B, n.Hkv, n.S, n.d, n.dev, n.dt);
    if (r.wq.defined()) {
      dwq = empty({n.d}, n.dev, at::kFloat);
      dwk = empty({n.d}, n.dev, at::kFloat);
      ws = workspace_of(lib.norm_rope_bwd_bytes(n.B, n.Hq, n.Hkv, n.S, n.d, 1), n.dev);
    }
  } else if (!dq.defined() || !dk.defined()) {
    throw BadArgument{"dq and dk must be tensors"};
  }
  const fa_view vdq = view("dq", dq, n.dev, n.dt, qs, true), vdk = view("dk", dk, n.dev, n.dt, ks, true);
  if (dwq.defined()) fit("dq_weight", dwq, n.dev, at::kFloat, {n.d});
  if (dwk.defined()) fit("dk_weight", dwk, n.dev, at::kFloat, {n.d});
  const int rc = lib.norm_rope_bwd(
      &vdqo, &vdko, q.defined() ? &vq : nullptr, k.defined() ? &vk : nullptr, &vdq, &vdk,
      data<float>(dwq), data<float>(dwk), data<void>(r.wq), data<void>(r.wk), eps,
      data<int>(r.positions), data<unsigned long long>(r.turns), r.rope_dim, interleaved, rope_scale,
      n.B, n.Hq, n.Hkv, n.S, n.d, dtype_code(dqo), data<void>(ws),
      workspace_bytes(ws, n.dev), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({dq, dk, dwq, dwk});
}

// (handle, q, k, v, q_out, k_cache, v_cache, block_table, seq_lens, turns, q_weight, k_weight,
//  eps, interleaved, rope_scale, stream)
PyObject* append(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  Tensor qo = maybe(a[4], "q_out");
  const Tensor &kc = tensor(a[5], "k_cache"), &vc = tensor(a[6], "v_cache");
  const Tensor &table = tensor(a[7], "block_table"), &lens = tensor(a[8], "seq_lens");
  const HeadDims n = head_dims(q, k, "q");
  const RopeArgs r = rope_inputs(n.dev, n.dt, n.B, n.S, n.d, a[9], Py_None, a[10], a[11]);
  const CacheDims c = cache_inputs(n.dev, n.dt, n.B, n.Hkv, n.d, kc, vc, table, lens);
  const Sizes qs = {n.B, n.Hq, n.S, n.d}, ks = {n.B, n.Hkv, n.S, n.d};
  const fa_view vq = view("q", q, n.dev, n.dt, qs), vk = view("k", k, n.dev, n.dt, ks),
                vv = view("v", v, n.dev, n.dt, ks);
  const float eps = real(a[12]), rope_scale = real(a[14]);
  const bool interleaved = truth(a[13]);
  const Place at(n.dev, a[15]);
  Released released;
  if (!qo.defined()) qo = empty(q.sizes(), n.dev, n.dt);
  const fa_view vqo = view("q_out", qo, n.dev, n.dt, qs, true);
  const int rc = lib.append(&vq, &vk, &vv, &vqo, kc.data_ptr(), vc.data_ptr(), data<int>(table),
                            data<int>(lens), data<void>(r.wq), data<void>(r.wk), eps,
                            data<unsigned long long>(r.turns), r.rope_dim, interleaved, rope_scale,
                            n.B, n.Hq, n.Hkv, n.S, n.d, c.block_size, c.num_blocks, c.max_blocks,
                            dtype_code(q), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(qo);
}

// append, then ragged over the cache with it. What either refuses is found out before the
// append writes: the ragged call is made first without a workspace, which the library looks
// at after everything else.
// (handle, q, k, v, k_cache, v_cache, block_table, seq_lens, turns, q_weight, k_weight, eps,
//  interleaved, rope_scale, window, softcap, slopes, scale, stream)
PyObject* step(PyObject* const* a) {
  const Library lib = library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  const Tensor &kc = tensor(a[4], "k_cache"), &vc = tensor(a[5], "v_cache");
  const Tensor &table = tensor(a[6], "block_table"), &lens = tensor(a[7], "seq_lens");
  const Tensor slopes = maybe(a[16], "slopes");
  const HeadDims n = head_dims(q, k, "q");
  const RopeArgs r = rope_inputs(n.dev, n.dt, n.B, n.S, n.d, a[8], Py_None, a[9], a[10]);
  const CacheDims c = cache_inputs(n.dev, n.dt, n.B, n.Hkv, n.d, kc, vc, table, lens);
  const Sizes qs = {n.B, n.Hq, n.S, n.d}, ks = {n.B, n.Hkv, n.S, n.d};
  const fa_view vq = view("q", q, n.dev, n.dt, qs), vk = view("k", k, n.dev, n.dt, ks),
                vv = view("v", v, n.dev, n.dt, ks);
  if (slopes.defined()) fit("slopes", slopes, n.dev, at::kFloat, {n.Hq});
  const float eps = real(a[11]), rope_scale = real(a[13]), softcap = real(a[15]);
  const float scale = scale_of(a[17], n.d);
  const bool interleaved = truth(a[12]);
  const int window = integer(a[14]);
  const Place at(n.dev, a[18]);
  Released released;
  const Tensor qo = empty(q.sizes(), n.dev, n.dt), out = empty(q.sizes(), n.dev, n.dt);
  const Tensor lse = empty(q.sizes().slice(0, 3), n.dev, at::kFloat);
  const Tensor ws =
      workspace_of(lib.ragged_bytes(n.B, n.Hq, n.Hkv, n.S, n.d, c.block_size, c.max_blocks), n.dev);
  const fa_view vqo = view("q_out", qo, n.dev, n.dt, qs, true);
  auto attend = [&](void* workspace, size_t bytes) {
    return lib.ragged(qo.data_ptr(), kc.data_ptr(), vc.data_ptr(), data<int>(table), data<int>(lens),
                      out.data_ptr(), data<float>(lse), n.B, n.Hq, n.Hkv, n.S, n.d, c.block_size,
                      c.num_blocks, c.max_blocks, window, scale, softcap, data<float>(slopes),
                      dtype_code(q), workspace, bytes, at.stream);
  };
  int rc = attend(nullptr, 0);
  if (rc == FA_ERR_WORKSPACE)
    rc = lib.append(&vq, &vk, &vv, &vqo, kc.data_ptr(), vc.data_ptr(), data<int>(table),
                    data<int>(lens), data<void>(r.wq), data<void>(r.wk), eps,
                    data<unsigned long long>(r.turns), r.rope_dim, interleaved, rope_scale, n.B, n.Hq,
                    n.Hkv, n.S, n.d, c.block_size, c.num_blocks, c.max_blocks, dtype_code(q),
                    at.stream);
  if (rc == FA_OK) rc = attend(ws.data_ptr(), workspace_bytes(ws, n.dev));
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({out, lse});
}

// ----------------------------------------------------------------- latent --
constexpr int64_t kRope = 64;   // elements of the rotated key part

// The fa_view of a [B, S, d] tensor (no heads).
fa_view flat_view(const char* name, const Tensor& t, at::Device dev, at::ScalarType dt, int64_t B, int64_t S,
                  int64_t d, bool written = false) {
  const Sizes sizes = {B, S, d};
  const at::IntArrayRef want(sizes.begin(), sizes.size());
  if (t.device() != dev || t.scalar_type() != dt || t.sizes() != want) misfit(name, t, "", dev, dt, want);
  return view(name, t.unsqueeze(1), dev, dt, {B, 1, S, d}, written);
}

struct LatentInputs {
  at::Device dev;
  at::ScalarType dt;
  int B, H, Sq, Skv, d;
  fa_view q, k, kr, v;
};
LatentInputs latent_inputs(const Tensor& q, const Tensor& k, const Tensor& kr, const Tensor& v,
                           const Tensor& begin, const Tensor& end) {
  const at::Device dev = cuda_device(q, "q");
  four_dims(q, "q [B,H,Sq,d+64], k and v [B,H,Skv,d], k_rope [B,Skv,64] (any strides but the last)");
  four_dims(k, "q [B,H,Sq,d+64], k and v [B,H,Skv,d], k_rope [B,Skv,64] (any strides but the last)");
  LatentInputs n{dev, q.scalar_type(), narrow(q.size(0)), narrow(q.size(1)), narrow(q.size(2)),
                 narrow(k.size(2)), narrow(k.size(3)), {}, {}, {}, {}};
  n.q = view("q", q, dev, n.dt, {n.B, n.H, n.Sq, n.d + kRope});
  n.k = view("k", k, dev, n.dt, {n.B, n.H, n.Skv, n.d});
  n.kr = flat_view("k_rope", kr, dev, n.dt, n.B, n.Skv, kRope);
  n.v = view("v", v, dev, n.dt, {n.B, n.H, n.Skv, n.d});
  if (begin.defined() != end.defined()) throw BadArgument{"key_begin and key_end go together"};
  if (begin.defined()) {
    fit("key_begin", begin, dev, at::kInt, {n.B, n.Sq});
    fit("key_end", end, dev, at::kInt, {n.B, n.Sq});
  }
  return n;
}

// (handle, q, k, k_rope, v, key_begin, key_end, out, lse, scale, stream)
PyObject* latent_forward(PyObject* const* a) {
  const LatentLibrary lib = latent_library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &kr = tensor(a[3], "k_rope"), &v = tensor(a[4], "v");
  const Tensor begin = maybe(a[5], "key_begin"), end = maybe(a[6], "key_end");
  Tensor out = maybe(a[7], "out"), lse = maybe(a[8], "lse");
  const LatentInputs n = latent_inputs(q, k, kr, v, begin, end);
  const float scale = scale_of(a[9], n.d + static_cast<int>(kRope));
  const Place at(n.dev, a[10]);
  Released released;
  if (!out.defined()) out = empty_tokens_first(n.B, n.H, n.Sq, n.d, n.dev, n.dt);
  const fa_view vo = view("out", out, n.dev, n.dt, {n.B, n.H, n.Sq, n.d}, true);
  if (lse.defined()) fit("lse", lse, n.dev, at::kFloat, {n.B, n.H, n.Sq});
  else lse = empty({n.B, n.H, n.Sq}, n.dev, at::kFloat);
  const int rc = lib.fwd(&n.q, &n.k, &n.kr, &n.v, data<int>(begin), data<int>(end), &vo, data<float>(lse), n.B,
                                n.H, n.Sq, n.Skv, n.d, scale, dtype_code(q), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({out, lse});
}

// (handle, q, k, k_rope, v, key_begin, key_end, out, dout, lse, dq, dk, dk_rope, dv, workspace,
//  scale, stream)
PyObject* latent_backward(PyObject* const* a) {
  const LatentLibrary lib = latent_library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &kr = tensor(a[3], "k_rope"), &v = tensor(a[4], "v");
  const Tensor begin = maybe(a[5], "key_begin"), end = maybe(a[6], "key_end");
  const Tensor &out = tensor(a[7], "out"), &dout = tensor(a[8], "dout"), &lse = tensor(a[9], "lse");
  Tensor dq = maybe(a[10], "dq"), dk = maybe(a[11], "dk"), dkr = maybe(a[12], "dk_rope"), dv = maybe(a[13], "dv");
  Tensor ws = maybe(a[14], "workspace");
  const LatentInputs n = latent_inputs(q, k, kr, v, begin, end);
  const Sizes os = {n.B, n.H, n.Sq, n.d}, ks = {n.B, n.H, n.Skv, n.d};
  const fa_view vo = view("out", out, n.dev, n.dt, os), vg = view("dout", dout, n.dev, n.dt, os);
  fit("lse", lse, n.dev, at::kFloat, {n.B, n.H, n.Sq});
  const float scale = scale_of(a[15], n.d + static_cast<int>(kRope));
  const Place at(n.dev, a[16]);
  Released released;
  if (!dq.defined()) dq = empty_tokens_first(n.B, n.H, n.Sq, n.d + kRope, n.dev, n.dt);
  if (!dk.defined()) dk = empty_tokens_first(n.B, n.H, n.Skv, n.d, n.dev, n.dt);
  if (!dkr.defined()) dkr = empty({n.B, n.Skv, kRope}, n.dev, n.dt);
  if (!dv.defined()) dv = empty_tokens_first(n.B, n.H, n.Skv, n.d, n.dev, n.dt);
  if (!ws.defined()) ws = workspace_of(lib.bwd_bytes(n.B, n.H, n.Sq, n.Skv, n.d), n.dev);
  const fa_view vdq = view("dq", dq, n.dev, n.dt, {n.B, n.H, n.Sq, n.d + kRope}, true);
  const fa_view vdk = view("dk", dk, n.dev, n.dt, ks, true), vdv = view("dv", dv, n.dev, n.dt, ks, true);
  const fa_view vdkr = flat_view("dk_rope", dkr, n.dev, n.dt, n.B, n.Skv, kRope, true);
  const int rc = lib.bwd(&n.q, &n.k, &n.kr, &n.v, data<int>(begin), data<int>(end), &vo, &vg, data<float>(lse),
                                &vdq, &vdk, &vdkr, &vdv, n.B, n.H, n.Sq, n.Skv, n.d, scale, dtype_code(q),
                                ws.data_ptr(), workspace_bytes(ws, n.dev), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({dq, dk, dkr, dv});
}

// A cache [num_blocks, block_size, rank + 64] with its table and lengths; its rank.
int latent_cache(CacheDims& c, at::Device dev, at::ScalarType dt, int64_t B, const Tensor& cache, const Tensor& table,
                 const Tensor& lens) {
  if (cache.dim() != 3 || table.dim() != 2 || cache.size(2) <= kRope)
    throw BadArgument{"cache [num_blocks,block_size,rank+64], table [B,max_blocks]"};
  fit("cache", cache, dev, dt, cache.sizes());
  fit("block_table", table, dev, at::kInt, {B, table.size(1)});
  fit("seq_lens", lens, dev, at::kInt, {B});
  c = {narrow(cache.size(1)), narrow(cache.size(0)), narrow(table.size(1))};
  return narrow(cache.size(2) - kRope);
}

// (handle, q, cache, block_table, seq_lens, tree_masks, out, lse, workspace, window, scale, stream)
PyObject* latent_paged(PyObject* const* a) {
  const LatentLibrary lib = latent_library(a[0]);
  const Tensor &q = tensor(a[1], "q"), &cache = tensor(a[2], "cache");
  const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
  const Tensor tree = maybe(a[5], "tree_masks");
  Tensor out = maybe(a[6], "out"), lse = maybe(a[7], "lse"), ws = maybe(a[8], "workspace");
  const at::Device dev = cuda_device(q, "q");
  const auto dt = q.scalar_type();
  four_dims(q, "q must be [B,H,Sq,rank+64] (any strides but the last)");
  const int B = narrow(q.size(0)), H = narrow(q.size(1)), Sq = narrow(q.size(2));
  CacheDims c;
  const int rank = latent_cache(c, dev, dt, B, cache, table, lens);
  const fa_view vq = view("q", q, dev, dt, {B, H, Sq, rank + kRope});
  if (tree.defined()) fit("tree_masks", tree, dev, at::kLong, {B, Sq});
  const int window = integer(a[9]);
  const float scale = real(a[10]);
  const Place at(dev, a[11]);
  Released released;
  if (out.defined()) fit("out", out, dev, dt, {B, H, Sq, rank});
  else out = empty({B, H, Sq, rank}, dev, dt);
  if (lse.defined()) fit("lse", lse, dev, at::kFloat, {B, H, Sq});
  else lse = empty({B, H, Sq}, dev, at::kFloat);
  if (!ws.defined()) ws = workspace_of(lib.paged_bytes(B, H, Sq, rank, c.block_size, c.max_blocks), dev);
  const int rc = lib.paged(&vq, cache.data_ptr(), data<int>(table), data<int>(lens), data<long long>(tree),
                                  out.data_ptr(), data<float>(lse), B, H, Sq, rank, c.block_size, c.num_blocks,
                                  c.max_blocks, window, scale, dtype_code(q), ws.data_ptr(),
                                  workspace_bytes(ws, dev), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : tensors({out, lse});
}

// (handle, latent, k_rope, q_rope, q_out, cache, block_table, seq_lens, positions, weight, turns, eps,
//  interleaved, rope_scale, stream)
PyObject* latent_append(PyObject* const* a) {
  const LatentLibrary lib = latent_library(a[0]);
  const Tensor &latent = tensor(a[1], "latent"), &kr = tensor(a[2], "k_rope"), &qr = tensor(a[3], "q_rope");
  Tensor qo = maybe(a[4], "q_out");
  const Tensor &cache = tensor(a[5], "cache"), &table = tensor(a[6], "block_table"), &lens = tensor(a[7], "seq_lens");
  const Tensor positions = maybe(a[8], "positions"), weight = maybe(a[9], "weight");
  const Tensor& turns = tensor(a[10], "turns");
  const at::Device dev = cuda_device(latent, "latent");
  const auto dt = latent.scalar_type();
  if (latent.dim() != 3 || qr.dim() != 4)
    throw BadArgument{"latent [B,Sq,rank], k_rope [B,Sq,64], q_rope [B,H,Sq,64] (any strides but the last)"};
  const int B = narrow(latent.size(0)), Sq = narrow(latent.size(1)), H = narrow(qr.size(1));
  CacheDims c;
  const int rank = latent_cache(c, dev, dt, B, cache, table, lens);
  const Sizes qs = {B, H, Sq, kRope};
  const fa_view vl = flat_view("latent", latent, dev, dt, B, Sq, rank), vk = flat_view("k_rope", kr, dev, dt, B, Sq, kRope),
                vq = view("q_rope", qr, dev, dt, qs);
  fit("turns", turns, dev, at::kLong, {kRope / 2});
  if (positions.defined()) fit("positions", positions, dev, at::kInt, {B, Sq});
  if (weight.defined()) fit("weight", weight, dev, dt, {rank});
  const float eps = real(a[11]), rope_scale = real(a[13]);
  const bool interleaved = truth(a[12]);
  const Place at(dev, a[14]);
  Released released;
  if (!qo.defined()) qo = empty({B, H, Sq, kRope}, dev, dt);
  const fa_view vqo = view("q_out", qo, dev, dt, qs, true);
  const int rc = lib.append(&vl, &vk, &vq, &vqo, cache.data_ptr(), data<int>(table), data<int>(lens),
                                   data<int>(positions), data<void>(weight), eps, data<unsigned long long>(turns),
                                   interleaved, rope_scale, B, H, Sq, rank, c.block_size, c.num_blocks, c.max_blocks,
                                   dtype_code(latent), at.stream);
  released.end();
  return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(qo);
}

// ----------------------------------------------------------------- module --
// Nothing thrown leaves a function: bad arguments become ValueError (or the
// Python error already set), anything else RuntimeError.
template <PyObject* (*f)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, not %zd", N, n);
    return nullptr;
  }
  try {
    return f(args);
  } catch (const BadArgument& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.text.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* type = nullptr;
    if (PyObject* torch = PyImport_ImportModule("torch")) {
      type = PyObject_GetAttrString(torch, "OutOfMemoryError");
      Py_DECREF(torch);
    }
    PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*f)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<span_forward, 12>("span_forward"), method<span_backward, 17>("span_backward"),
    method<ragged, 14>("ragged"),             method<norm_rope, 13>("norm_rope"),
    method<norm_rope_bwd, 19>("norm_rope_bwd"), method<append, 16>("append"),
    method<step, 19>("step"),
    method<latent_forward, 11>("latent_forward"), method<latent_backward, 17>("latent_backward"),
    method<latent_paged, 12>("latent_paged"), method<latent_append, 15>("latent_append"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module_def); }
