// fast.cpp - the short way through the window and cache bindings (module _fast).
//
// For a short sequence the kernels take a few microseconds, and the Python
// binding's checks, allocations and ctypes call take 6 to 20.  Each function here
// does the same in one step for the common call: tensors of the right shapes on
// the current device, the current stream, a workspace of its own.  It returns
// None without having done anything where a call is not that, or where the
// library refuses its arguments; window.py and cache.py then take their own way,
// which says what is wrong.  A failed launch is raised here and not tried again:
// part of the call may have run.  Other Python threads run while a call allocates
// and launches, as they do while ctypes calls: a launch waits where the stream's
// queue is full.  Host time of a call by ctypes and by this way: windowed forward
// 12.4 and 4.8 us, backward 19.8 and 9.1, decoding 15.7 and 5.1, append 8.1 and
// 2.8, reserve 8.6 and 3.3, fork 15.6 and 6.1, free 6.4 and 2.3, compact 14.3 and
// 6.4.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "../../include/fa_b200_cache.h"
#include "../../include/fa_b200_window.h"

namespace {

using at::Tensor;

// A strided tensor on the current device.
const Tensor* cuda_tensor(PyObject* o) {
  if (!THPVariable_Check(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.get_device() != c10::cuda::current_device())
    return nullptr;
  return &t;
}

// A contiguous one of this type.
const Tensor* dense(PyObject* o, at::ScalarType type) {
  const Tensor* t = cuda_tensor(o);
  return t && t->scalar_type() == type && t->is_contiguous() ? t : nullptr;
}

const Tensor* dense_int(PyObject* o, int64_t dim) {
  const Tensor* t = dense(o, at::kInt);
  return t && t->dim() == dim ? t : nullptr;
}

bool get_int(PyObject* o, int& v) {
  if (!PyLong_Check(o)) return false;
  int overflow = 0;
  const long long x = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (overflow || x < INT_MIN || x > INT_MAX) return false;
  v = int(x);
  return true;
}

bool get_scale(PyObject* o, int64_t d, float& v) {
  if (o == Py_None)
    v = float(std::pow(double(d), -0.5));
  else if (PyFloat_Check(o))
    v = float(PyFloat_AS_DOUBLE(o));
  else
    return false;
  return true;
}

bool get_elem(const Tensor& t, int& elem) {
  if (t.scalar_type() == at::kBFloat16)
    elem = FA_ELEM_BF16;
  else if (t.scalar_type() == at::kHalf)
    elem = FA_ELEM_F16;
  else
    return false;
  return true;
}

bool fits(std::initializer_list<int64_t> sizes) {
  for (const int64_t n : sizes)
    if (n > INT_MAX) return false;
  return true;
}

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::Device on) {
  return at::detail::empty_cuda(sizes, type, on, std::nullopt);
}

Tensor bytes(size_t n, c10::Device on) { return empty({int64_t(n)}, at::kByte, on); }

void* stream_of(c10::Device on) { return c10::cuda::getCurrentCUDAStream(on.index()).stream(); }

int32_t* ints(const Tensor* t) { return static_cast<int32_t*>(t->data_ptr()); }

template <typename... T>
PyObject* tuple_of(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t)), ...);
  return r;
}

// What a call that did not return FA_OK leads to.  Only a launch can fail after
// something has been launched; the other statuses are refusals before that.  (A
// second compaction after one whose copy was not launched would find the counts
// moved and nothing left to do.)
PyObject* not_ok(const char* call, int status) {
  if (status != FA_ERR_LAUNCH) Py_RETURN_NONE;
  PyObject* fa = PyImport_ImportModule("flashattention_bf16_fwd_b200.fa");
  PyObject* r = fa ? PyObject_CallMethod(fa, "_check", "si", call, status) : nullptr;   // raises
  Py_XDECREF(fa);
  return r;
}

// Other Python threads run while one of these lives (an exception ends it too).
// What the call needs of its tensors is read before.  0.1 us of a call's 2.1 to 9.
class NoGil {
 public:
  NoGil() : state_(PyEval_SaveThread()) {}
  ~NoGil() { PyEval_RestoreThread(state_); }
  NoGil(const NoGil&) = delete;
  NoGil& operator=(const NoGil&) = delete;

 private:
  PyThreadState* state_;
};

#define FA_IF(condition) \
  if (!(condition)) Py_RETURN_NONE

// q, k and v of the windowed calls: [B,H,N,d] and two [B,Hkv,N,d] with Hkv dividing H.
struct Heads {
  const Tensor *q, *k, *v;
  int elem;
};

bool get_heads(PyObject* const* a, Heads& h) {
  h.q = cuda_tensor(a[0]);
  if (!h.q || h.q->dim() != 4 || !h.q->is_contiguous() || !get_elem(*h.q, h.elem)) return false;
  h.k = dense(a[1], h.q->scalar_type());
  h.v = dense(a[2], h.q->scalar_type());
  if (!h.k || !h.v || h.k->dim() != 4 || h.k->sizes() != h.v->sizes()) return false;
  const auto q = h.q->sizes(), k = h.k->sizes();
  return k[0] == q[0] && k[1] > 0 && q[1] % k[1] == 0 && k[2] == q[2] && k[3] == q[3] && fits({q[0], q[1], q[2], q[3]});
}

// (q, k, v, window, sinks, scale, fix_mode) -> (o, lse)
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads h;
  int window, sinks, fix_mode;
  float scale;
  FA_IF(n == 7 && get_heads(a, h) && get_int(a[3], window) && get_int(a[4], sinks) &&
        get_scale(a[5], h.q->size(3), scale) && get_int(a[6], fix_mode));
  const int B = int(h.q->size(0)), H = int(h.q->size(1)), Hkv = int(h.k->size(1)), N = int(h.q->size(2)),
            d = int(h.q->size(3));
  const at::ScalarType type = h.q->scalar_type();
  const c10::Device on = h.q->device();
  const void *q = h.q->data_ptr(), *k = h.k->data_ptr(), *v = h.v->data_ptr();
  Tensor o, lse;
  int status;
  {
    const NoGil no_gil;
    o = empty({B, H, N, d}, type, on);
    lse = empty({B, H, N}, at::kFloat, on);
    status = fa_window_fwd(q, k, v, o.data_ptr(), lse.data_ptr<float>(), B, H, Hkv, N, d, window, sinks, scale,
                           fix_mode, h.elem, stream_of(on));
  }
  if (status) return not_ok("fa_window_fwd", status);
  return tuple_of(o, lse);
  END_HANDLE_TH_ERRORS
}

// (q, k, v, o, lse, do, window, sinks, scale) -> (dq, dk, dv)
PyObject* window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Heads h;
  int window, sinks;
  float scale;
  FA_IF(n == 9 && get_heads(a, h) && get_int(a[6], window) && get_int(a[7], sinks) &&
        get_scale(a[8], h.q->size(3), scale));
  const auto s = h.q->sizes();
  const at::ScalarType type = h.q->scalar_type();
  const Tensor *to = dense(a[3], type), *tlse = dense(a[4], at::kFloat), *tdout = dense(a[5], type);
  FA_IF(to && tlse && tdout && to->sizes() == s && tdout->sizes() == s && tlse->sizes() == s.slice(0, 3));
  const int B = int(s[0]), H = int(s[1]), Hkv = int(h.k->size(1)), N = int(s[2]), d = int(s[3]);
  const size_t need = fa_window_bwd_workspace_size(B, H, Hkv, N, d, window, sinks);
  FA_IF(need);
  const c10::Device on = h.q->device();
  const void *q = h.q->data_ptr(), *k = h.k->data_ptr(), *v = h.v->data_ptr(), *o = to->data_ptr(),
             *dout = tdout->data_ptr();
  const float* lse = static_cast<const float*>(tlse->data_ptr());
  Tensor dq, dk, dv;
  int status;
  {
    const NoGil no_gil;
    dq = empty({B, H, N, d}, type, on);
    dk = empty({B, Hkv, N, d}, type, on);
    dv = empty({B, Hkv, N, d}, type, on);
    const Tensor ws = bytes(need, on);
    status = fa_window_bwd(q, k, v, o, lse, dout, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), need, B,
                           H, Hkv, N, d, window, sinks, scale, h.elem, stream_of(on));
  }
  if (status) return not_ok("fa_window_bwd", status);
  return tuple_of(dq, dk, dv);
  END_HANDLE_TH_ERRORS
}

// The pages of one layer, or with `layers` of [L, ...] too, and the tables.
struct Cache {
  const Tensor *k = nullptr, *v = nullptr, *refs = nullptr, *table = nullptr, *lens = nullptr;
  int elem = 0;
  int64_t L = 0, P = 0, Hkv = 0, page = 0, d = 0, S = 0, M = 0;
};

bool get_pages(PyObject* k, PyObject* v, bool layers, Cache& c) {
  c.k = cuda_tensor(k);
  if (!c.k || !c.k->is_contiguous() || !get_elem(*c.k, c.elem)) return false;
  c.v = dense(v, c.k->scalar_type());
  const auto s = c.k->sizes();
  const size_t n = s.size();
  if (!c.v || s != c.v->sizes() || !(n == 4 || (layers && n == 5))) return false;
  c.L = n == 5 ? s[0] : 1;
  c.P = s[n - 4];
  c.Hkv = s[n - 3];
  c.page = s[n - 2];
  c.d = s[n - 1];
  return c.Hkv > 0 && fits({c.L, c.P, c.Hkv, c.page, c.d});
}

bool get_table(PyObject* table, PyObject* lens, Cache& c) {
  c.table = dense_int(table, 2);
  c.lens = dense_int(lens, 1);
  if (!c.table || !c.lens || c.lens->size(0) != c.table->size(0)) return false;
  c.S = c.table->size(0);
  c.M = c.table->size(1);
  return fits({c.S, c.M});
}

// Elements between the tokens of t [*, heads, d], whose heads are contiguous; 0: it is not that.
int64_t row_stride(const Tensor* t, int64_t heads, int64_t d, at::ScalarType type) {
  if (!t || t->dim() != 3 || t->size(1) != heads || t->size(2) != d || t->scalar_type() != type) return 0;
  if (t->is_contiguous()) return heads * d;
  if (t->size(0) < 2 || t->stride(2) != 1 || (heads > 1 && t->stride(1) != d)) return 0;
  return t->stride(0);
}

// What the calls take of a cache, read before other threads may run.
struct Raw {
  void *k, *v;
  int32_t *refs, *table, *lens;
  int L, P, Hkv, page, d, S, M;
  c10::Device on;
  explicit Raw(const Cache& c)
      : k(c.k ? c.k->data_ptr() : nullptr), v(c.v ? c.v->data_ptr() : nullptr), refs(c.refs ? ints(c.refs) : nullptr),
        table(ints(c.table)), lens(ints(c.lens)), L(int(c.L)), P(int(c.P)), Hkv(int(c.Hkv)), page(int(c.page)),
        d(int(c.d)), S(int(c.S)), M(int(c.M)), on(c.table->device()) {}
};

// (q, k_pages, v_pages, table, lens, window, sinks, scale) -> (o, lse)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  int window = 0, sinks;
  float scale;
  FA_IF(n == 8 && get_pages(a[1], a[2], false, c) && get_table(a[3], a[4], c) &&
        (a[5] == Py_None || get_int(a[5], window)) && get_int(a[6], sinks) && get_scale(a[7], c.d, scale));
  const Tensor* tq = cuda_tensor(a[0]);
  FA_IF(tq && tq->dim() == 3 && tq->size(0) == c.S && tq->size(1) > 0 && tq->size(1) % c.Hkv == 0 &&
        fits({tq->size(1)}));
  const at::ScalarType type = c.k->scalar_type();
  const int64_t stride = row_stride(tq, tq->size(1), c.d, type);
  FA_IF(stride > 0);
  const Raw r(c);
  const int H = int(tq->size(1));
  const size_t need = fa_decode_workspace_size(r.S, H, r.Hkv, r.d);
  FA_IF(need);
  const void* q = tq->data_ptr();
  Tensor o, lse;
  int status;
  {
    const NoGil no_gil;
    o = empty({r.S, H, r.d}, type, r.on);
    lse = empty({r.S, H}, at::kFloat, r.on);
    const Tensor ws = bytes(need, r.on);
    status = fa_decode(q, r.k, r.v, r.table, r.lens, o.data_ptr(), lse.data_ptr<float>(), ws.data_ptr(), need, r.S, H,
                       r.Hkv, r.d, r.P, r.page, r.M, stride, window, sinks, scale, c.elem, stream_of(r.on));
  }
  if (status) return not_ok("fa_decode", status);
  return tuple_of(o, lse);
  END_HANDLE_TH_ERRORS
}

// (k, v, k_pages, v_pages, table, lens, cu or None) -> True
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  FA_IF(n == 7 && get_pages(a[2], a[3], false, c) && get_table(a[4], a[5], c));
  const Tensor *tk = cuda_tensor(a[0]), *tv = cuda_tensor(a[1]);
  const at::ScalarType type = c.k->scalar_type();
  const int64_t ks = row_stride(tk, c.Hkv, c.d, type), vs = row_stride(tv, c.Hkv, c.d, type);
  FA_IF(ks > 0 && vs > 0 && tk->size(0) == tv->size(0) && tk->size(0) > 0 && fits({tk->size(0)}));
  const int32_t* cu = nullptr;
  if (a[6] != Py_None) {
    const Tensor* t = dense_int(a[6], 1);
    FA_IF(t && t->size(0) == c.S + 1);
    cu = ints(t);
  }
  const Raw r(c);
  const int T = int(tk->size(0));
  const void *k = tk->data_ptr(), *v = tv->data_ptr();
  int status;
  {
    const NoGil no_gil;
    status = fa_cache_append(k, v, r.k, r.v, r.table, r.lens, cu, T, r.S, r.Hkv, r.d, r.P, r.page, r.M, ks, vs,
                             stream_of(r.on));
  }
  if (status) return not_ok("fa_cache_append", status);
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

bool get_refs(PyObject* refs, Cache& c) {
  c.refs = dense_int(refs, 1);
  return c.refs && fits({c.refs->size(0)});
}

// (refs, table, lens, add, page) -> missing
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  int page;
  FA_IF(n == 5 && get_refs(a[0], c) && get_table(a[1], a[2], c) && get_int(a[4], page));
  const Tensor* tadd = dense_int(a[3], 1);
  FA_IF(tadd && tadd->size(0) == c.S);
  const Raw r(c);
  const int P = int(c.refs->size(0));
  const int32_t* add = ints(tadd);
  Tensor missing;
  int status;
  {
    const NoGil no_gil;
    missing = empty({1}, at::kInt, r.on);
    status = fa_cache_reserve(r.refs, r.table, r.lens, add, ints(&missing), r.S, P, page, r.M, stream_of(r.on));
  }
  if (status) return not_ok("fa_cache_reserve", status);
  return THPVariable_Wrap(missing);
  END_HANDLE_TH_ERRORS
}

// (k_pages, v_pages, refs, table, lens, src, dst) -> missing
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  FA_IF(n == 7 && get_pages(a[0], a[1], true, c) && get_refs(a[2], c) && get_table(a[3], a[4], c) &&
        c.refs->size(0) == c.P);
  const Tensor *tsrc = dense_int(a[5], 1), *tdst = dense_int(a[6], 1);
  FA_IF(tsrc && tdst && tsrc->size(0) == tdst->size(0) && fits({tsrc->size(0)}));
  const Raw r(c);
  const size_t need = fa_cache_workspace_size(r.S, r.P);
  FA_IF(need);
  const int F = int(tsrc->size(0));
  const int32_t *src = ints(tsrc), *dst = ints(tdst);
  Tensor missing;
  int status;
  {
    const NoGil no_gil;
    missing = empty({1}, at::kInt, r.on);
    const Tensor ws = bytes(need, r.on);
    status = fa_cache_fork(r.k, r.v, r.refs, r.table, r.lens, src, dst, ints(&missing), ws.data_ptr(), need, F, r.L,
                           r.S, r.Hkv, r.d, r.P, r.page, r.M, stream_of(r.on));
  }
  if (status) return not_ok("fa_cache_fork", status);
  return THPVariable_Wrap(missing);
  END_HANDLE_TH_ERRORS
}

// (refs, table, lens, seqs, page) -> True
PyObject* free_seqs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  int page;
  FA_IF(n == 5 && get_refs(a[0], c) && get_table(a[1], a[2], c) && get_int(a[4], page));
  const Tensor* tseqs = dense_int(a[3], 1);
  FA_IF(tseqs && fits({tseqs->size(0)}));
  const Raw r(c);
  const int F = int(tseqs->size(0)), P = int(c.refs->size(0));
  const int32_t* seqs = ints(tseqs);
  int status;
  {
    const NoGil no_gil;
    status = fa_cache_free(r.refs, r.table, r.lens, seqs, F, r.S, P, page, r.M, stream_of(r.on));
  }
  if (status) return not_ok("fa_cache_free", status);
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// (k_pages, v_pages, refs, table, lens) -> live
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Cache c;
  FA_IF(n == 5 && get_pages(a[0], a[1], true, c) && get_refs(a[2], c) && get_table(a[3], a[4], c) &&
        c.refs->size(0) == c.P);
  const Raw r(c);
  const size_t need = fa_cache_workspace_size(r.S, r.P);
  FA_IF(need);
  Tensor live;
  int status;
  {
    const NoGil no_gil;
    live = empty({1}, at::kInt, r.on);
    const Tensor ws = bytes(need, r.on);
    status = fa_cache_compact(r.k, r.v, r.refs, r.table, r.lens, ints(&live), ws.data_ptr(), need, r.L, r.S, r.Hkv, r.d,
                              r.P, r.page, r.M, stream_of(r.on));
  }
  if (status) return not_ok("fa_cache_compact", status);
  return THPVariable_Wrap(live);
  END_HANDLE_TH_ERRORS
}

#define FA_METHOD(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_METHOD("window_fwd", window_fwd), FA_METHOD("window_bwd", window_bwd),
                         FA_METHOD("decode", decode),         FA_METHOD("append", append),
                         FA_METHOD("reserve", reserve),       FA_METHOD("fork", fork),
                         FA_METHOD("free", free_seqs),        FA_METHOD("compact", compact),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fast", "The short way through the window and cache bindings.", -1,
                          methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__fast() { return PyModule_Create(&module_def); }
