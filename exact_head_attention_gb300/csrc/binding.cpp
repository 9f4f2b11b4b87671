// The Python calls of the operators between projections and attention, and of drafted trees: argument checks, allocation and
// the C-ABI call in compiled code, for calls whose kernels take a few microseconds.  Marshalled in Python by ctypes, a call
// that rotates one token took 17.5 us on the host; here it takes 7 to 8, of which its two outputs and the launch are 6.6.  exattn.py has the signatures and their documentation.
//
// The library itself (libexattn.so) knows nothing of torch: this module links against it and is loaded by exattn.py alone.
#include <Python.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/variable.h>

#include "../../include/exattn.h"

namespace {

struct BadValue {
  std::string text;
};
struct BadType {
  std::string text;
};
struct Failed {
  attn_status status;
  const char* where;
};
struct PythonError {};  // already set

PyObject* error_class = nullptr;  // AttnError

void require(bool ok, const char* text) {
  if (!ok) throw BadValue{text};
}

const at::Tensor* tensor_or_none(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw BadType{"a tensor is wanted"};
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o) {
  const at::Tensor* t = tensor_or_none(o);
  if (!t) throw BadType{"a tensor is wanted"};
  return *t;
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
PyObject* wrapped(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!out) throw PythonError{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(out, i++, wrapped(t));
  return out;
}

// Runs `body` with C++ exceptions and refusals turned into Python's.
template <typename Body>
PyObject* guarded(Body&& body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const BadValue& e) {
    PyErr_SetString(PyExc_ValueError, e.text.c_str());
  } catch (const BadType& e) {
    PyErr_SetString(PyExc_TypeError, e.text.c_str());
  } catch (const Failed& e) {
    if (PyObject* x = PyObject_CallFunction(error_class, "is", static_cast<int>(e.status), e.where)) {
      PyErr_SetObject(error_class, x);
      Py_DECREF(x);
    }
  } catch (const PythonError&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

template <typename Call>
void library(const char* where, Call&& call) {
  attn_status st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  if (st != ATTN_OK) throw Failed{st, where};
}

attn_dtype dtype_code(at::ScalarType t) {
  if (t == at::kBFloat16) return ATTN_BF16;
  if (t == at::kHalf) return ATTN_FP16;
  throw BadType{std::string("unsupported dtype ") + c10::toString(t) + "; expected bfloat16 or float16"};
}

struct View {
  void* p = nullptr;
  attn_strides s = {0, 0, 0};
};
View view_of(const at::Tensor* t) {
  View v;
  if (!t) return v;
  const auto s = t->strides();
  require(s[3] == 1, "tensors must have a contiguous last dimension");
  v.p = t->data_ptr();
  v.s = {s[0], s[1], s[2]};
  return v;
}
View view_of(const at::Tensor& t) { return t.defined() ? view_of(&t) : View{}; }
// A caller's tensor that must be as another is.
View view_like(const at::Tensor* t, const at::Tensor* like) {
  require(!t || (like && t->sizes() == like->sizes() && t->scalar_type() == like->scalar_type() && t->get_device() == like->get_device()),
          "tensors must match in shape, dtype and device");
  return view_of(t);
}
at::Tensor empty_as(const at::Tensor* t) { return t ? at::empty_like(*t) : at::Tensor(); }

const int* int32_of(const at::Tensor* t, long B, int index, const char* text) {
  if (!t) return nullptr;
  require(t->scalar_type() == at::kInt && t->dim() == 1 && t->size(0) == B && t->get_device() == index && t->is_contiguous(), text);
  return static_cast<const int*>(t->data_ptr());
}

// Two [B, H, N, d] tensors, one of which may be missing.
struct Pair {
  const at::Tensor *q, *k;
  long B, N, d, H, Hk;
  int index;
  at::ScalarType dtype;

  Pair(const at::Tensor* q_, const at::Tensor* k_) : q(q_), k(k_) {
    const at::Tensor* x = q ? q : k;
    require(x, "one of the tensors is needed");
    require(x->is_cuda(), "tensors must be CUDA tensors");
    require(x->dim() == 4 && (!k || k->dim() == 4), "tensors must be [B, H, N, d]");
    B = x->size(0);
    N = x->size(2);
    d = x->size(3);
    H = q ? q->size(1) : 0;
    Hk = k ? k->size(1) : 0;
    require(B <= INT32_MAX && N <= INT32_MAX && d <= INT32_MAX && H <= INT32_MAX && Hk <= INT32_MAX, "tensors are too large");
    index = x->get_device();
    dtype = x->scalar_type();
    if (q && k) {
      require(k->size(0) == B && k->size(2) == N && k->size(3) == d, "tensors must be [B, H, N, d] with the same B, N and d");
      require(k->scalar_type() == dtype && k->get_device() == index, "tensors must be of one dtype, on one device");
    }
  }
};

struct RopeArgs {
  const at::Tensor *freq, *start, *offsets, *q_weight, *k_weight;
  long layout;
  double amplitude, eps;
};

attn_rope rope_of(const RopeArgs& a, long B, long N, long d, at::ScalarType dtype, int index) {
  attn_rope r = {};
  if (a.freq) {
    require(a.freq->scalar_type() == at::kDouble && a.freq->dim() == 1 && a.freq->is_contiguous() && a.freq->get_device() == index,
            "freq must be a contiguous float64 tensor [rotary_dim / 2] on the tensors' device");
    require(a.freq->numel() <= d, "freq must be [rotary_dim / 2]");
    r.rotary_dim = 2 * static_cast<int>(a.freq->numel());
    r.freq = r.rotary_dim ? static_cast<const double*>(a.freq->data_ptr()) : nullptr;
  }
  r.start = int32_of(a.start, B, index, "start must be a contiguous int32 tensor of one entry a sequence on the tensors' device");
  if (a.offsets) {
    const at::Tensor& o = *a.offsets;
    const bool rows = o.dim() == 2;
    require(o.scalar_type() == at::kInt && o.get_device() == index && (rows || o.dim() == 1) && o.size(-1) == N &&
                (!rows || o.size(0) == 1 || o.size(0) == B) && (N <= 1 || o.stride(-1) == 1),
            "offsets must be an int32 tensor [B, N], [1, N] or [N], last dimension contiguous, on the tensors' device");
    r.offsets = static_cast<const int*>(o.data_ptr());
    r.offset_stride = rows && o.size(0) > 1 ? o.stride(0) : 0;
  }
  const at::Tensor* weights[2] = {a.q_weight, a.k_weight};
  for (const at::Tensor* w : weights)
    require(!w || ((w->scalar_type() == at::kFloat || w->scalar_type() == dtype) && w->dim() == 1 && w->size(0) == d && w->get_device() == index &&
                   w->is_contiguous()),
            "weights must be contiguous [d], float32 or of the tensors' dtype, on their device");
  if (a.q_weight && a.k_weight && a.q_weight->scalar_type() != a.k_weight->scalar_type()) throw BadType{"both weights must be of one dtype"};
  const at::Tensor* w = a.q_weight ? a.q_weight : a.k_weight;
  r.q_weight = a.q_weight ? a.q_weight->data_ptr() : nullptr;
  r.k_weight = a.k_weight ? a.k_weight->data_ptr() : nullptr;
  r.weight_fp32 = w && w->scalar_type() == at::kFloat;
  r.layout = static_cast<int>(a.layout);
  r.amplitude = static_cast<float>(a.amplitude);
  r.eps = static_cast<float>(a.eps);
  return r;
}

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw BadType{"wrong number of arguments"};
}

// q, k, freq, start, offsets, layout, amplitude, q_weight, k_weight, eps, out q, out k
PyObject* rope_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 12);
    const Pair x(tensor_or_none(a[0]), tensor_or_none(a[1]));
    const attn_dtype code = dtype_code(x.dtype);
    const RopeArgs ra = {tensor_or_none(a[2]), tensor_or_none(a[3]), tensor_or_none(a[4]), tensor_or_none(a[7]), tensor_or_none(a[8]),
                         integer(a[5]), real(a[6]), real(a[9])};
    const attn_rope rope = rope_of(ra, x.B, x.N, x.d, x.dtype, x.index);
    const View q = view_of(x.q), k = view_of(x.k);
    const at::Tensor *to_q = tensor_or_none(a[10]), *to_k = tensor_or_none(a[11]);
    const bool given = to_q || to_k;
    require(!given || (!to_q == !x.q && !to_k == !x.k), "out must be a pair of what q and k are");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(x.index));
    const at::Tensor oq = given ? (to_q ? *to_q : at::Tensor()) : empty_as(x.q), ok = given ? (to_k ? *to_k : at::Tensor()) : empty_as(x.k);
    const View vq = given ? view_like(to_q, x.q) : view_of(oq), vk = given ? view_like(to_k, x.k) : view_of(ok);
    if (x.B && x.N && (x.H || x.Hk)) {
      void* stream = stream_of(x.index);
      library("attn_rope_fwd", [&] {
        return attn_rope_fwd(q.p, q.s, k.p, k.s, vq.p, vq.s, vk.p, vk.s, static_cast<int>(x.B), static_cast<int>(x.H), static_cast<int>(x.Hk),
                             static_cast<int>(x.N), static_cast<int>(x.d), &rope, code, stream);
      });
    }
    return tuple_of({oq, ok});
  });
}

// dq, dk, q, k, freq, start, offsets, layout, amplitude, q_weight, k_weight, eps, workspace
PyObject* rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 13);
    const Pair x(tensor_or_none(a[0]), tensor_or_none(a[1]));
    const attn_dtype code = dtype_code(x.dtype);
    const RopeArgs ra = {tensor_or_none(a[4]), tensor_or_none(a[5]), tensor_or_none(a[6]), tensor_or_none(a[9]), tensor_or_none(a[10]),
                         integer(a[7]), real(a[8]), real(a[11])};
    const attn_rope rope = rope_of(ra, x.B, x.N, x.d, x.dtype, x.index);
    const bool nq = ra.q_weight && x.H, nk = ra.k_weight && x.Hk;
    const at::Tensor *in_q = tensor_or_none(a[2]), *in_k = tensor_or_none(a[3]), *workspace = tensor_or_none(a[12]);
    require((!nq || in_q) && (!nk || in_k), "the gradients of a norm need its input");
    require(!workspace || (workspace->get_device() == x.index && workspace->is_contiguous()),
            "the workspace must be contiguous and on the tensors' device");
    const View dq = view_of(x.q), dk = view_of(x.k), q = view_like(nq ? in_q : nullptr, x.q), k = view_like(nk ? in_k : nullptr, x.k);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(x.index));
    const at::Tensor oq = empty_as(x.q), ok = empty_as(x.k);
    const bool some = x.B && x.N && (x.H || x.Hk);
    // weights without a head or token behind them have gradients of zero
    auto gradient = [&](const at::Tensor* w, bool normed) { return !w ? at::Tensor() : normed && some ? at::empty_like(*w) : at::zeros_like(*w); };
    const at::Tensor wq = gradient(ra.q_weight, nq), wk = gradient(ra.k_weight, nk);
    if (some) {
      at::Tensor space;
      size_t bytes = 0;
      if (nq || nk) {
        bytes = attn_rope_bwd_workspace_size(static_cast<int>(x.d));
        if (workspace) {
          space = *workspace;
          bytes = workspace->nbytes();
        } else {
          space = at::empty({static_cast<int64_t>(bytes)}, (x.q ? x.q : x.k)->options().dtype(at::kByte));
        }
      }
      const View vq = view_of(oq), vk = view_of(ok);
      void *stream = stream_of(x.index), *at_space = space.defined() ? space.data_ptr() : nullptr;
      void *pq = nq ? wq.data_ptr() : nullptr, *pk = nk ? wk.data_ptr() : nullptr;
      library("attn_rope_bwd", [&] {
        return attn_rope_bwd(dq.p, dq.s, dk.p, dk.s, q.p, q.s, k.p, k.s, vq.p, vq.s, vk.p, vk.s, pq, pk, static_cast<int>(x.B),
                             static_cast<int>(x.H), static_cast<int>(x.Hk), static_cast<int>(x.N), static_cast<int>(x.d), &rope, code, at_space,
                             bytes, stream);
      });
    }
    return tuple_of({oq, ok, wq, wk});
  });
}

// k, v, k_scale, v_scale, page_table: the attn_cache of checked tensors, as bytes
PyObject* cache_struct(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 5);
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]), &ks = tensor(a[2]), &vs = tensor(a[3]), &table = tensor(a[4]);
    const at::ScalarType t = k.scalar_type();
    if ((t != at::kFloat8_e4m3fn && t != at::kChar) || v.scalar_type() != t)
      throw BadType{std::string("unsupported cache dtypes ") + c10::toString(t) + ", " + c10::toString(v.scalar_type()) +
                    "; expected float8_e4m3fn or int8 for both"};
    if (ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat || table.scalar_type() != at::kInt)
      throw BadType{"scales must be float32 and the page table int32"};
    require(k.dim() == 4 && k.sizes() == v.sizes() && table.dim() == 2, "k, v must be [num_pages, heads, page, d] and the page table [B, width]");
    require(ks.dim() == 2 && ks.size(0) == k.size(0) && ks.size(1) == k.size(1) && ks.sizes() == vs.sizes(), "scales must be [num_pages, heads]");
    for (const at::Tensor* x : {&k, &v, &ks, &vs, &table})
      require(x->is_cuda() && x->get_device() == k.get_device() && x->is_contiguous(), "cache tensors must be contiguous and on one CUDA device");
    for (int i = 0; i < 4; ++i) require(k.size(i) <= INT32_MAX, "tensors are too large");
    require(table.size(0) <= INT32_MAX && table.size(1) <= INT32_MAX, "tensors are too large");
    attn_cache c = {};
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    c.k_scale = static_cast<float*>(ks.data_ptr());
    c.v_scale = static_cast<float*>(vs.data_ptr());
    c.page_table = static_cast<const int*>(table.data_ptr());
    c.num_pages = static_cast<int>(k.size(0));
    c.heads = static_cast<int>(k.size(1));
    c.page_size = static_cast<int>(k.size(2));
    c.d = static_cast<int>(k.size(3));
    c.table_width = static_cast<int>(table.size(1));
    c.format = t == at::kChar ? ATTN_CACHE_INT8 : ATTN_CACHE_E4M3;
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&c), sizeof(c));
  });
}

// A QuantCache: the address of its attn_cache, its device and its sequences.
struct Cache {
  const attn_cache* c;
  int index;
  long B;

  Cache(PyObject* address, PyObject* device, PyObject* rows)
      : c(static_cast<const attn_cache*>(PyLong_AsVoidPtr(address))), index(static_cast<int>(integer(device))), B(integer(rows)) {
    if (!c && PyErr_Occurred()) throw PythonError{};
  }
  // A 16-bit [B, H, N, d] view that goes with the cache.
  View view(const at::Tensor* t, at::ScalarType dtype) const {
    if (!t) return View{};
    require(t->dim() == 4 && t->size(0) == B && t->size(3) == c->d, "tensors must be [B, H, N, d] with the page table's B and the cache's d");
    require(t->get_device() == index && t->scalar_type() == dtype, "tensors must be of one dtype, on the cache's device");
    return view_of(t);
  }
  const int* int32(const at::Tensor* t, const char* text) const { return int32_of(t, B, index, text); }
};
constexpr char kStart[] = "start must be a contiguous int32 tensor of one entry a sequence on the cache's device";
constexpr char kCount[] = "count must be a contiguous int32 tensor of one entry a sequence on the cache's device";
constexpr char kLens[] = "lens must be a contiguous int32 tensor of one entry a sequence on the cache's device";

// address, device, B, k, v, freq, start, count, offsets, q, layout, amplitude, q_weight, k_weight, eps, position_start, out
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 17);
    const Cache cache(a[0], a[1], a[2]);
    const at::Tensor &k = tensor(a[3]), &v = tensor(a[4]);
    const at::Tensor *q = tensor_or_none(a[9]), *out = tensor_or_none(a[16]);
    require(k.dim() == 4 && k.sizes() == v.sizes() && k.size(1) == cache.c->heads, "k and v must be [B, heads, N, d] with the cache's heads");
    const at::ScalarType dtype = k.scalar_type();
    const attn_dtype code = dtype_code(dtype);
    const View vk = cache.view(&k, dtype), vv = cache.view(&v, dtype), vq = cache.view(q, dtype);
    const long N = k.size(2), H = q ? q->size(1) : 0;
    require(N <= INT32_MAX && H <= INT32_MAX, "tensors are too large");
    require(!q || q->size(2) == N, "q must be [B, H, N, d] of the new tokens");
    const RopeArgs ra = {tensor_or_none(a[5]), tensor_or_none(a[15]), tensor_or_none(a[8]), tensor_or_none(a[12]), tensor_or_none(a[13]),
                         integer(a[10]), real(a[11]), real(a[14])};
    require(q || (!ra.q_weight && !out), "a weight or an output for queries that are not there");
    const int *start = cache.int32(tensor_or_none(a[6]), kStart), *counts = cache.int32(tensor_or_none(a[7]), kCount);
    const attn_rope rope = rope_of(ra, cache.B, N, cache.c->d, dtype, cache.index);
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(cache.index));
    const View given = view_like(out, q);
    const at::Tensor to = out ? *out : empty_as(q);
    const View vo = out ? given : view_of(to);
    if (cache.B && N) {
      void* stream = stream_of(cache.index);
      library("attn_cache_append", [&] {
        return attn_cache_append(cache.c, vq.p, vq.s, vo.p, vo.s, vk.p, vk.s, vv.p, vv.s, start, counts, static_cast<int>(cache.B),
                                 static_cast<int>(H), static_cast<int>(N), &rope, code, stream);
      });
    }
    return wrapped(to);
  });
}

// address, device, B, q, lens, tree, scale, workspace
PyObject* forward_cache_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 8);
    const Cache cache(a[0], a[1], a[2]);
    const at::Tensor &q = tensor(a[3]), &tree = tensor(a[5]);
    const at::ScalarType dtype = q.scalar_type();
    const View vq = cache.view(&q, dtype);
    const attn_dtype code = dtype_code(dtype);
    const long H = q.size(1), Nq = q.size(2), words = (Nq + 31) / 32;
    require(H <= INT32_MAX && Nq <= INT32_MAX, "tensors are too large");
    require(tree.scalar_type() == at::kInt && tree.get_device() == cache.index && tree.is_contiguous() && tree.dim() == 3 &&
                (tree.size(0) == 1 || tree.size(0) == cache.B) && tree.size(1) == Nq && tree.size(2) == words,
            "tree must be a contiguous int32 tensor [B, Nq, ceil(Nq / 32)] or [1, ...] on the cache's device");
    const int* lens = cache.int32(&tensor(a[4]), kLens);
    const float scale = static_cast<float>(a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(cache.c->d)) : real(a[6]));
    const at::Tensor* workspace = tensor_or_none(a[7]);
    require(!workspace || (workspace->get_device() == cache.index && workspace->is_contiguous()),
            "the workspace must be contiguous and on the cache's device");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(cache.index));
    const at::Tensor o = at::empty_like(q), lse = at::empty({cache.B, H, Nq}, q.options().dtype(at::kFloat));
    if (cache.B && H && Nq) {
      at::Tensor space;
      size_t bytes;
      if (workspace) {
        space = *workspace;
        bytes = workspace->nbytes();
      } else {
        bytes = attn_fwd_cache_workspace_size(cache.c, static_cast<int>(cache.B), static_cast<int>(H), static_cast<int>(Nq));
        space = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
      }
      const View vo = view_of(o);
      void *stream = stream_of(cache.index), *at_space = space.data_ptr(), *at_lse = lse.data_ptr(), *at_tree = tree.data_ptr();
      const long long stride = tree.size(0) > 1 ? Nq * words : 0;
      library("attn_fwd_cache_tree", [&] {
        return attn_fwd_cache_tree(vq.p, vq.s, cache.c, lens, static_cast<const uint32_t*>(at_tree), stride, vo.p, vo.s,
                                   static_cast<float*>(at_lse), static_cast<int>(cache.B), static_cast<int>(H), static_cast<int>(Nq), scale, code,
                                   at_space, bytes, stream);
      });
    }
    return tuple_of({o, lse});
  });
}

// parents
PyObject* draft_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 1);
    const at::Tensor& parents = tensor(a[0]);
    require(parents.scalar_type() == at::kInt && parents.is_cuda() && (parents.dim() == 1 || parents.dim() == 2) && parents.is_contiguous(),
            "parents must be a contiguous int32 CUDA tensor [B, N] or [N]");
    const long B = parents.dim() == 1 ? 1 : parents.size(0), N = parents.size(-1);
    require(B <= INT32_MAX && N <= INT32_MAX, "tensors are too large");
    const int index = parents.get_device();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    const at::Tensor mask = at::empty({B, N, (N + 31) / 32}, parents.options()), depth = at::empty({B, N}, parents.options());
    if (B && N) {
      void *stream = stream_of(index), *at_parents = parents.data_ptr(), *at_mask = mask.data_ptr(), *at_depth = depth.data_ptr();
      library("attn_draft_tree", [&] {
        return attn_draft_tree(static_cast<const int*>(at_parents), static_cast<uint32_t*>(at_mask), static_cast<int*>(at_depth),
                               static_cast<int>(B), static_cast<int>(N), stream);
      });
    }
    return tuple_of({mask, depth});
  });
}

// Any number of tensors, or None: whether one is a leaf whose gradient a living autograd graph adds up on another stream than
// the current one.  (Torch keeps a leaf's node of that, and its stream, for as long as a graph of it lives.)
PyObject* leaf_elsewhere(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    for (Py_ssize_t i = 0; i < n; ++i) {
      const at::Tensor* t = tensor_or_none(a[i]);
      if (!t || !t->is_cuda() || !t->requires_grad()) continue;
      const auto node = torch::autograd::impl::try_get_grad_accumulator(*t);
      if (!node) continue;
      const auto stream = node->stream();
      if (stream && *stream != c10::cuda::getCurrentCUDAStream(t->get_device()).unwrap()) Py_RETURN_TRUE;
    }
    Py_RETURN_FALSE;
  });
}

// The class that library failures are raised as.
PyObject* set_error_class(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(error_class);
  error_class = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<rope_forward>("rope_forward"),
                         method<rope_backward>("rope_backward"),
                         method<cache_append>("cache_append"),
                         method<forward_cache_tree>("forward_cache_tree"),
                         method<draft_tree>("draft_tree"),
                         method<cache_struct>("cache_struct"),
                         method<leaf_elsewhere>("leaf_elsewhere"),
                         {"set_error_class", set_error_class, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&definition); }
