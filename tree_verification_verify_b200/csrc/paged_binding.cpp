// Python binding of the paged calls of include/tree_verify.h: argument checks
// and marshalling only, in C++ because a call's checks took 13 us of Python
// where the launch itself takes 4 (a decoding step makes a few such calls per
// layer).  The library's functions are handed in as addresses by
// init(functions, error); nothing of the library is linked here.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>

#include <cstdarg>
#include <map>
#include <utility>

#include "../../include/tree_verify.h"

// The torch and Python this is built for, for the build and the package to look
// up without loading it.
extern "C" __attribute__((used, visibility("default"))) const char tv_paged_built_against[] = TV_BUILT_AGAINST;

namespace {

// ------------------------------------------------------------------ errors

PyObject* g_error = nullptr;                      // the package's TVError

struct Refused {};                                // a Python error is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list ap;
  va_start(ap, format);
  PyErr_FormatV(g_error, format, ap);
  va_end(ap);
  throw Refused{};
}
void need(bool ok, const char* message) {
  if (!ok) refuse("%s", message);
}

// --------------------------------------------------------------- functions

struct Functions {
  decltype(&tree_verify_attn_paged) attn;
  decltype(&tree_verify_attn_paged_workspace_size) attn_ws;
  decltype(&tree_accept_probs) accept;
  decltype(&tree_commit_kv_paged) commit;
  decltype(&tree_commit_kv_paged_workspace_size) commit_ws;
  decltype(&tree_pages_update) update;
  decltype(&tree_pages_update_workspace_size) update_ws;
  decltype(&tree_pages_compact) compact;
  decltype(&tree_pages_compact_workspace_size) compact_ws;
  decltype(&tv_status_string) status;
} g_fn;

void check(tv_status st, const char* what) {
  if (st != TV_OK) refuse("%s: %s (status %d)", what, g_fn.status(st), static_cast<int>(st));
}

// ----------------------------------------------------------------- tensors

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == nullptr || o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}

// A call's tensors must share one CUDA device; the call runs there.
struct Device {
  int index = -1;
  void add(const at::Tensor* t) {
    if (!t) return;
    if (!t->is_cuda()) refuse("tensors must live on a CUDA device (there is no CPU path)");
    const int d = t->get_device();
    if (index < 0) index = d;
    else if (d != index) refuse("tensors must share one device");
  }
};

// A required tensor of the call.
const at::Tensor& arg(PyObject* o, const char* name, Device& dev) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse("%s must be a tensor", name);
  dev.add(t);
  return *t;
}
const at::Tensor* opt(PyObject* o, const char* name, Device& dev) {
  const at::Tensor* t = tensor(o, name);
  dev.add(t);
  return t;
}

// A size for one of the ABI's 32-bit fields.
int32_t i32(int64_t size, const char* name) {
  if (size > INT32_MAX) refuse("%s must be below 2^31", name);
  return static_cast<int32_t>(size);
}

bool is_shape(const at::Tensor& t, at::IntArrayRef s) { return t.sizes() == s; }

int dtype(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return TV_BF16;
  if (t.scalar_type() == at::kFloat) return TV_FP32;
  refuse("%s must be bf16 or fp32", name);
}

template <typename T = int32_t>
T* vec(const at::Tensor* t, int64_t n, const char* name, at::ScalarType st = at::kInt) {
  if (!t) return nullptr;
  if (t->scalar_type() != st || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    refuse("%s must be contiguous int32 of shape (%lld,)", name, static_cast<long long>(n));
  return static_cast<T*>(t->data_ptr());
}

// An int32 table of `rows` rows (and `cols` columns, when not -1), each contiguous.
int32_t* table(const at::Tensor& t, int64_t rows, int64_t cols, const char* name) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != rows || (cols >= 0 && t.size(1) != cols) ||
      (t.size(1) > 1 && t.stride(1) != 1 && t.numel() > 0))
    refuse("%s must be int32 with %lld contiguous rows", name, static_cast<long long>(rows));
  return static_cast<int32_t*>(t.data_ptr());
}

void pair(const at::Tensor& k, const at::Tensor& v, const char* name) {
  if (k.scalar_type() != v.scalar_type() || k.sizes() != v.sizes() || k.strides() != v.strides())
    refuse("%s K and V must share shape, strides and dtype", name);
  if (k.stride(-1) != 1) refuse("%s K/V must have a contiguous last dimension", name);
}

uint32_t* status_word(const at::Tensor* t) {
  if (!t) return nullptr;
  if (t->element_size() != 4 || t->numel() < 1) refuse("dev_status must be one int32");
  return static_cast<uint32_t*>(t->data_ptr());
}

// ------------------------------------------------------------------ streams

// The call's device and stream: allocations and launches go there.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  cudaStream_t stream;
  int index;
  Place(const Device& dev, PyObject* raw) : index(dev.index) {
    need(index >= 0, "tensors must live on a CUDA device (there is no CPU path)");
    if (raw != Py_None) {
      stream = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
      if (PyErr_Occurred()) throw Refused{};
      guard.reset_stream(c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(index)));
    } else {
      device.set_index(static_cast<c10::DeviceIndex>(index));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    }
  }
  at::Tensor empty(at::IntArrayRef s, at::ScalarType t) const {
    return at::empty(s, at::TensorOptions().dtype(t).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
  }
};

constexpr size_t kTicketBytes = 64 * 1024;

// Scratch per (device, stream): made on that stream, its ticket counters
// zeroed once and left zero by every call.  Never freed at exit (the process
// takes it back), only outgrown.
void* scratch(const Place& at, size_t bytes, at::Tensor& own) {
  static auto* kept = new std::map<std::pair<int, cudaStream_t>, at::Tensor>();
  const int64_t n = static_cast<int64_t>(bytes) + 256;
  at::Tensor* t = &own;
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(at.stream, &capturing) == cudaSuccess && capturing != cudaStreamCaptureStatusNone) {
    // part of the graph: no other graph or stream can meet it
    own = at.empty({n}, at::kByte);
    own.narrow(0, 0, std::min<int64_t>(n, kTicketBytes + 256)).zero_();
  } else {
    t = &(*kept)[{at.index, at.stream}];
    if (!t->defined() || t->numel() < n) {
      *t = at.empty({n}, at::kByte);
      t->narrow(0, 0, std::min<int64_t>(n, kTicketBytes + 256)).zero_();
    }
  }
  return reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(t->data_ptr()) + 255) & ~static_cast<uintptr_t>(255));
}

template <typename A, typename Run, typename Size>
void run(const Place& at, const char* name, const A& a, Run call, Size size) {
  const size_t bytes = size(&a);                  // 0: the call itself says what is wrong
  at::Tensor own;
  void* ws = bytes ? scratch(at, bytes, own) : nullptr;
  check(call(&a, ws, bytes, at.stream), name);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// Converts what a call throws; no exception leaves this file.  Running out of
// memory is torch's own error, as from any of its allocations.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Refused&) {
  } catch (const c10::OutOfMemoryError&) {
    torch::translate_exception_to_python(std::current_exception());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// ---------------------------------------------------------------- attention

// q, k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, parent,
// n_nodes, scale, out, lse, want_lse, dev_status, stream, prefix_only
PyObject* attn(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 16)) return nullptr;
  return guarded([&]() -> PyObject* {
    Device dev;
    const at::Tensor& q = arg(v[0], "q", dev);
    const at::Tensor& k = arg(v[1], "k_pages", dev);
    const at::Tensor& vp = arg(v[2], "v_pages", dev);
    const at::Tensor& pt = arg(v[3], "page_table", dev);
    const at::Tensor& len = arg(v[4], "prefix_len", dev);
    const at::Tensor& kt = arg(v[5], "k_tree", dev);
    const at::Tensor& vt = arg(v[6], "v_tree", dev);
    const at::Tensor& par = arg(v[7], "parent", dev);
    const at::Tensor* nn = opt(v[8], "n_nodes", dev);
    const double scale = PyFloat_AsDouble(v[9]);
    if (PyErr_Occurred()) throw Refused{};
    const at::Tensor* out = opt(v[10], "out", dev);
    const at::Tensor* lse = opt(v[11], "lse", dev);
    const bool want_lse = PyObject_IsTrue(v[12]) == 1;
    const at::Tensor* st = opt(v[13], "dev_status", dev);
    const Place at(dev, v[14]);
    tv_attn_paged_args a = {};
    a.dtype = dtype(q, "q");
    need(q.dim() == 4 && q.stride(3) == 1, "q must be [B][T][Hq][d] with a contiguous last dimension");
    const int64_t B = q.size(0), T = q.size(1), Hq = q.size(2), d = q.size(3);
    need(k.dim() == 4 && kt.dim() == 4, "K/V must be [num_pages][page_size][Hkv][d] and [B][T][Hkv][d]");
    pair(k, vp, "the pool's");
    pair(kt, vt, "tree");
    need(k.scalar_type() == q.scalar_type() && kt.scalar_type() == q.scalar_type() && k.size(3) == d,
         "K/V must share q's dtype and d");
    need(is_shape(kt, {B, T, k.size(2), d}), "tree K/V must be [B][T][Hkv][d]");
    at::Tensor out_new, lse_new;
    if (!out) {
      out_new = at.empty({B, T, Hq, d}, q.scalar_type());
      out = &out_new;
    }
    need(out->sizes() == q.sizes() && out->scalar_type() == q.scalar_type() && out->stride(3) == 1,
         "out must have q's shape and dtype with a contiguous last dimension");
    if (!lse && want_lse) {
      lse_new = at.empty({B, T, Hq}, at::kFloat);
      lse = &lse_new;
    }
    need(!lse || (is_shape(*lse, {B, T, Hq}) && lse->scalar_type() == at::kFloat && lse->is_contiguous()),
         "lse must be contiguous fp32 [B][T][Hq]");
    a.B = i32(B, "B"); a.T = i32(T, "T"); a.Hq = i32(Hq, "Hq"); a.Hkv = i32(k.size(2), "Hkv"); a.d = i32(d, "d");
    a.num_pages = i32(k.size(0), "num_pages"); a.page_size = i32(k.size(1), "page_size");
    a.q = q.data_ptr(); a.q_sb = q.stride(0); a.q_st = q.stride(1); a.q_sh = q.stride(2);
    a.k_pages = k.data_ptr(); a.v_pages = vp.data_ptr();
    a.kv_sp = k.stride(0); a.kv_sr = k.stride(1); a.kv_sh = k.stride(2);
    a.page_table = table(pt, B, -1, "page_table"); a.pt_sb = pt.stride(0); a.max_pages = i32(pt.size(1), "max_pages");
    a.prefix_len = vec(&len, B, "prefix_len");
    a.k_tree = kt.data_ptr(); a.v_tree = vt.data_ptr();
    a.kt_sb = kt.stride(0); a.kt_st = kt.stride(1); a.kt_sh = kt.stride(2);
    a.parent = table(par, B, T, "parent"); a.parent_sb = par.stride(0);
    a.n_nodes = vec(nn, B, "n_nodes");
    a.scale = static_cast<float>(scale);
    a.out = out->data_ptr(); a.o_sb = out->stride(0); a.o_st = out->stride(1); a.o_sh = out->stride(2);
    a.lse = lse ? static_cast<float*>(lse->data_ptr()) : nullptr;
    a.dev_status = status_word(st);
    a.prefix_only = PyObject_IsTrue(v[15]) == 1;
    run(at, "tree_verify_attn_paged", a, g_fn.attn, g_fn.attn_ws);
    PyObject* o = out == &out_new ? wrap(out_new) : same(v[10]);
    PyObject* l = lse == &lse_new ? wrap(lse_new) : same(lse ? v[11] : Py_None);
    PyObject* r = PyTuple_Pack(2, o, l);
    Py_XDECREF(o);
    Py_XDECREF(l);
    return r;
  });
}

// --------------------------------------------------------------- acceptance

const at::Tensor* probs(const at::Tensor* t, const char* name, at::IntArrayRef s) {
  if (t && (t->scalar_type() != at::kFloat || t->sizes() != s || (s[2] > 1 && t->stride(2) != 1)))
    refuse("%s must be fp32 [B][T][V] with contiguous rows", name);
  return t;
}

// target_probs, draft_tokens, parent, u_child, u_sample, draft_probs,
// n_nodes, mode, dev_status, stream, n_accepted, accepted_nodes, out_tokens
PyObject* accept(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    Device dev;
    const at::Tensor& p = arg(v[0], "target_probs", dev);
    const at::Tensor& tok = arg(v[1], "draft_tokens", dev);
    const at::Tensor& par = arg(v[2], "parent", dev);
    const at::Tensor* uc = opt(v[3], "u_child", dev);
    const at::Tensor* us = opt(v[4], "u_sample", dev);
    const at::Tensor* q = opt(v[5], "draft_probs", dev);
    const at::Tensor* nn = opt(v[6], "n_nodes", dev);
    const at::Tensor* st = opt(v[8], "dev_status", dev);
    const at::Tensor* have[3] = {opt(v[10], "n_accepted", dev), opt(v[11], "accepted_nodes", dev),
                                 opt(v[12], "out_tokens", dev)};
    const Place at(dev, v[9]);
    need(p.dim() == 3, "target_probs must be [B][T][V]");
    const int64_t B = p.size(0), T = p.size(1), V = p.size(2);
    probs(&p, "target_probs", p.sizes());
    probs(q, "draft_probs", p.sizes());
    for (const at::Tensor* u : {uc, us})
      need(!u || (u->scalar_type() == at::kDouble && is_shape(*u, {B, T}) && u->is_contiguous()),
           "u_child and u_sample must be contiguous fp64 [B][T]");
    tv_accept_probs_args a = {};
    a.B = i32(B, "B"); a.T = i32(T, "T"); a.V = i32(V, "V");
    a.target_probs = static_cast<const float*>(p.data_ptr()); a.tp_sb = p.stride(0); a.tp_st = p.stride(1);
    if (q) {
      a.draft_probs = static_cast<const float*>(q->data_ptr()); a.dp_sb = q->stride(0); a.dp_st = q->stride(1);
    }
    a.draft_tokens = table(tok, B, T, "draft_tokens"); a.tok_sb = tok.stride(0);
    a.parent = table(par, B, T, "parent"); a.parent_sb = par.stride(0);
    a.n_nodes = vec(nn, B, "n_nodes");
    a.u_child = uc ? static_cast<const double*>(uc->data_ptr()) : nullptr;
    a.u_sample = us ? static_cast<const double*>(us->data_ptr()) : nullptr;
    a.mode = static_cast<int32_t>(PyLong_AsLong(v[7]));
    at::Tensor made[3];
    const int64_t cols[3] = {-1, T, T + 1};
    int32_t* ptr[3];
    for (int i = 0; i < 3; ++i) {
      if (!have[i]) {
        made[i] = i == 0 ? at.empty({B}, at::kInt) : at.empty({B, cols[i]}, at::kInt);
        have[i] = &made[i];
      }
      const at::Tensor& t = *have[i];
      need(t.scalar_type() == at::kInt && t.is_contiguous() &&
               (i == 0 ? is_shape(t, {B}) : is_shape(t, {B, cols[i]})),
           "outputs must be contiguous int32: n_accepted [B], accepted_nodes [B][T], out_tokens [B][T+1]");
      ptr[i] = static_cast<int32_t*>(t.data_ptr());
    }
    a.n_accepted = ptr[0]; a.accepted_nodes = ptr[1]; a.out_tokens = ptr[2];
    a.dev_status = status_word(st);
    check(g_fn.accept(&a, at.stream), "tree_accept_probs");
    PyObject* o[3];
    for (int i = 0; i < 3; ++i) o[i] = have[i] == &made[i] ? wrap(made[i]) : same(v[10 + i]);
    PyObject* r = PyTuple_Pack(3, o[0], o[1], o[2]);
    for (PyObject* x : o) Py_XDECREF(x);
    return r;
  });
}

// ---------------------------------------------------------------- KV commit

// A tensor with an optional leading layer dimension: its layers, the layer
// stride, and where its other dimensions begin.
struct Layers {
  int64_t n, stride;
  int at;
  explicit Layers(const at::Tensor& t) : n(t.dim() == 5 ? t.size(0) : 1), stride(t.dim() == 5 ? t.stride(0) : 0), at(t.dim() == 5) {}
};

template <typename A>
Layers pool(A& a, const at::Tensor& k, const at::Tensor& v) {
  a.dtype = dtype(k, "K/V");
  need(k.dim() == 4 || k.dim() == 5, "the pool must be [num_pages][page_size][Hkv][d], with a leading layer dimension or not");
  pair(k, v, "the pool's");
  const Layers l(k);
  a.layers = i32(l.n, "layers"); a.kv_sl = l.stride;
  a.num_pages = i32(k.size(l.at), "num_pages"); a.page_size = i32(k.size(l.at + 1), "page_size");
  a.Hkv = i32(k.size(l.at + 2), "Hkv"); a.d = i32(k.size(l.at + 3), "d");
  a.kv_sp = k.stride(l.at); a.kv_sr = k.stride(l.at + 1); a.kv_sh = k.stride(l.at + 2);
  a.k_pages = k.data_ptr(); a.v_pages = v.data_ptr();
  return l;
}

// k_pages, v_pages, page_table, prefix_len, k_tree, v_tree, n_accepted,
// accepted_nodes, prefix_len_out, dev_status, stream
PyObject* commit(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    Device dev;
    const at::Tensor& k = arg(v[0], "k_pages", dev);
    const at::Tensor& vp = arg(v[1], "v_pages", dev);
    const at::Tensor& pt = arg(v[2], "page_table", dev);
    const at::Tensor& len = arg(v[3], "prefix_len", dev);
    const at::Tensor& kt = arg(v[4], "k_tree", dev);
    const at::Tensor& vt = arg(v[5], "v_tree", dev);
    const at::Tensor& na = arg(v[6], "n_accepted", dev);
    const at::Tensor& acc = arg(v[7], "accepted_nodes", dev);
    const at::Tensor* lo = opt(v[8], "prefix_len_out", dev);
    const at::Tensor* st = opt(v[9], "dev_status", dev);
    const Place at(dev, v[10]);
    tv_commit_paged_args a = {};
    const Layers l = pool(a, k, vp);
    need(kt.dim() == k.dim(), "tree K/V must be [layers][B][T][Hkv][d], with the pool's layer dimension or without");
    pair(kt, vt, "tree");
    const Layers t(kt);
    const int64_t B = kt.size(t.at), T = kt.size(t.at + 1);
    need(kt.scalar_type() == k.scalar_type() && t.n == l.n && kt.size(t.at + 2) == a.Hkv && kt.size(t.at + 3) == a.d,
         "tree K/V must be [layers][B][T][Hkv][d] of the pool's dtype");
    a.B = i32(B, "B"); a.T = i32(T, "T");
    a.k_tree = kt.data_ptr(); a.v_tree = vt.data_ptr();
    a.kt_sl = t.stride; a.kt_sb = kt.stride(t.at); a.kt_st = kt.stride(t.at + 1); a.kt_sh = kt.stride(t.at + 2);
    a.page_table = table(pt, B, -1, "page_table"); a.pt_sb = pt.stride(0); a.max_pages = i32(pt.size(1), "max_pages");
    a.prefix_len = vec(&len, B, "prefix_len");
    a.prefix_len_out = lo ? vec(lo, B, "prefix_len_out") : vec(&len, B, "prefix_len");
    a.n_accepted = vec(&na, B, "n_accepted");
    a.accepted_nodes = table(acc, B, T, "accepted_nodes"); a.acc_sb = acc.stride(0);
    a.dev_status = status_word(st);
    run(at, "tree_commit_kv_paged", a, g_fn.commit, g_fn.commit_ws);
    return same(lo ? v[8] : v[3]);
  });
}

// -------------------------------------------------------------- page tables

PyObject* two(const at::Tensor* a, const at::Tensor& a_new, PyObject* a_old, const at::Tensor* b,
              const at::Tensor& b_new, PyObject* b_old) {
  PyObject* x = a == &a_new ? wrap(a_new) : same(a_old);
  PyObject* y = b == &b_new ? wrap(b_new) : same(b_old);
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// k_pages, v_pages, page_table, source, keep, grow, pinned, out, n_free,
// dev_status, stream
PyObject* update(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    Device dev;
    const at::Tensor& k = arg(v[0], "k_pages", dev);
    const at::Tensor& vp = arg(v[1], "v_pages", dev);
    const at::Tensor& pt = arg(v[2], "page_table", dev);
    const at::Tensor& src = arg(v[3], "source", dev);
    const at::Tensor& keep = arg(v[4], "keep", dev);
    const at::Tensor& grow = arg(v[5], "grow", dev);
    const at::Tensor* pin = opt(v[6], "pinned", dev);
    const at::Tensor* out = opt(v[7], "out", dev);
    const at::Tensor* nf = opt(v[8], "n_free", dev);
    const at::Tensor* st = opt(v[9], "dev_status", dev);
    const Place at(dev, v[10]);
    tv_pages_update_args a = {};
    pool(a, k, vp);
    need(pt.dim() == 2 && src.dim() == 1, "page_table must be [B_in][max_pages], source [B]");
    const int64_t B = src.size(0);
    a.B_in = i32(pt.size(0), "B_in"); a.max_pages_in = i32(pt.size(1), "max_pages"); a.B = i32(B, "B");
    a.page_table = table(pt, pt.size(0), -1, "page_table"); a.pt_sb = pt.stride(0);
    a.source = vec(&src, B, "source"); a.keep = vec(&keep, B, "keep"); a.grow = vec(&grow, B, "grow");
    a.pinned = vec(pin, a.num_pages, "pinned");
    at::Tensor out_new, nf_new;
    if (!out) {
      out_new = at.empty({B, pt.size(1)}, at::kInt);
      out = &out_new;
    }
    if (!nf) {
      nf_new = at.empty({1}, at::kInt);
      nf = &nf_new;
    }
    a.page_table_out = table(*out, B, -1, "out"); a.po_sb = out->stride(0); a.max_pages = i32(out->size(1), "max_pages");
    a.n_free = vec(nf, 1, "n_free");
    a.dev_status = status_word(st);
    run(at, "tree_pages_update", a, g_fn.update, g_fn.update_ws);
    return two(out, out_new, v[7], nf, nf_new, v[8]);
  });
}

// k_pages, v_pages, page_table, length, pinned, out, n_used, dev_status, stream
PyObject* compact(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (!arity(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    Device dev;
    const at::Tensor& k = arg(v[0], "k_pages", dev);
    const at::Tensor& vp = arg(v[1], "v_pages", dev);
    const at::Tensor& pt = arg(v[2], "page_table", dev);
    const at::Tensor& len = arg(v[3], "length", dev);
    const at::Tensor* pin = opt(v[4], "pinned", dev);
    const at::Tensor* out = opt(v[5], "out", dev);
    const at::Tensor* nu = opt(v[6], "n_used", dev);
    const at::Tensor* st = opt(v[7], "dev_status", dev);
    const Place at(dev, v[8]);
    tv_pages_compact_args a = {};
    pool(a, k, vp);
    need(pt.dim() == 2, "page_table must be [B][max_pages]");
    const int64_t B = pt.size(0);
    a.B = i32(B, "B"); a.max_pages = i32(pt.size(1), "max_pages");
    a.page_table = table(pt, B, -1, "page_table"); a.pt_sb = pt.stride(0);
    a.length = vec(&len, B, "length");
    a.pinned = vec(pin, a.num_pages, "pinned");
    at::Tensor out_new, nu_new;
    if (!out) {
      out_new = at.empty({B, pt.size(1)}, at::kInt);
      out = &out_new;
    }
    if (!nu) {
      nu_new = at.empty({1}, at::kInt);
      nu = &nu_new;
    }
    a.page_table_out = table(*out, B, pt.size(1), "out"); a.po_sb = out->stride(0);
    a.n_used = vec(nu, 1, "n_used");
    a.dev_status = status_word(st);
    run(at, "tree_pages_compact", a, g_fn.compact, g_fn.compact_ws);
    return two(out, out_new, v[5], nu, nu_new, v[6]);
  });
}

// ------------------------------------------------------------------- module

// init({name: address}, TVError)
PyObject* init(PyObject*, PyObject* args) {
  PyObject *fns, *error;
  if (!PyArg_ParseTuple(args, "O!O", &PyDict_Type, &fns, &error)) return nullptr;
  bool ok = true;
  auto take = [&](auto& f, const char* name) {
    PyObject* x = PyDict_GetItemString(fns, name);
    void* p = x ? PyLong_AsVoidPtr(x) : nullptr;
    if (!p) {
      ok = false;
      if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "%s", name);
    }
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p);
  };
  take(g_fn.attn, "tree_verify_attn_paged");
  take(g_fn.attn_ws, "tree_verify_attn_paged_workspace_size");
  take(g_fn.accept, "tree_accept_probs");
  take(g_fn.commit, "tree_commit_kv_paged");
  take(g_fn.commit_ws, "tree_commit_kv_paged_workspace_size");
  take(g_fn.update, "tree_pages_update");
  take(g_fn.update_ws, "tree_pages_update_workspace_size");
  take(g_fn.compact, "tree_pages_compact");
  take(g_fn.compact_ws, "tree_pages_compact_workspace_size");
  take(g_fn.status, "tv_status_string");
  if (!ok) return nullptr;
  Py_XDECREF(g_error);
  Py_INCREF(error);
  g_error = error;
  Py_RETURN_NONE;
}


PyMethodDef g_methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attn)), METH_FASTCALL, nullptr},
    {"accept", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(accept)), METH_FASTCALL, nullptr},
    {"commit", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(commit)), METH_FASTCALL, nullptr},
    {"update", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(update)), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(compact)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) { return PyModule_Create(&g_module); }
