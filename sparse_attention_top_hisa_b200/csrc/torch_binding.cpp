// Argument checks and calls of the entry points that run once per layer and decode step,
// for binding.py: what checking eight or nine tensors costs in Python (about 7 us of a call
// that takes the GPU as long) costs well under a microsecond here.  The functions take
// torch tensors positionally, check device, type, contiguity and shape, pass addresses and
// the stream to the C ABI and hand any status but HISA_OK to the callable that raises
// HisaError.  The entry points' addresses come from the loaded library (setup()).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <vector>

#include "hisa.h"

namespace {

struct Bad {};  // a Python exception is set

PyObject *g_raise = nullptr;  // raise(status, name)
decltype(&hisa_kv4_store) p_store = nullptr;
decltype(&hisa_kv4_load) p_load = nullptr;
decltype(&hisa_sparse_attention_kv4) p_attention = nullptr;
decltype(&hisa_token_weights) p_weights = nullptr;
decltype(&hisa_evict_select) p_select = nullptr;
decltype(&hisa_evict_rows) p_rows = nullptr;

[[noreturn]] void bad(const char *fmt, const char *a = "", const char *b = "") {
  PyErr_Format(PyExc_ValueError, fmt, a, b);
  throw Bad();
}

struct Args {
  PyObject *const *a;
  int dev = -1;  // of the call: the current device
  void *stream = nullptr;

  bool none(int i) const { return a[i] == Py_None; }

  // Tensor i, on the call's device (which the first one sets), of type t, contiguous and,
  // with cols >= 0, of the shape [*, cols].
  const at::Tensor &tensor(int i, const char *name, at::ScalarType t, int64_t cols = -1) {
    if (none(i)) bad("%s is required", name);
    if (!THPVariable_Check(a[i])) bad("%s must be a tensor", name);
    const at::Tensor &x = THPVariable_Unpack(a[i]);
    if (!x.is_cuda()) bad("%s must be a CUDA tensor", name);
    if (x.scalar_type() != t) bad("%s must be %s", name, c10::toString(t));
    if (!x.is_contiguous()) bad("%s must be contiguous", name);
    if (cols >= 0 && (x.dim() != 2 || x.size(1) != cols)) bad(cols == HISA_ATT_DIM ? "%s must have shape [*, 128]" : "%s must have shape [*, 16]", name);
    place(x, name);
    return x;
  }
  void place(const at::Tensor &x, const char *name) {
    const int d = x.get_device();
    if (dev < 0) {
      if (d != c10::cuda::current_device()) bad("%s must be on the current device", name);
      dev = d;
    } else if (d != dev) {
      bad("tensors must be on one device: %s is on another", name);
    }
  }
  int64_t number(int i) const {
    const long long v = PyLong_AsLongLong(a[i]);
    if (v == -1 && PyErr_Occurred()) throw Bad();
    return v;
  }
  int whole(int i) const {  // an int of the C ABI
    const int64_t v = number(i);
    if (v < INT32_MIN || v > INT32_MAX) bad("a size does not fit 32 bits");
    return (int)v;
  }
  bool given = false;  // the caller named a stream
  void on(int i) {     // the stream: None is the current one
    given = !none(i);
    stream = given ? PyLong_AsVoidPtr(a[i]) : (void *)c10::cuda::getCurrentCUDAStream(dev).stream();
    if (PyErr_Occurred()) throw Bad();
  }
  // A new tensor whose memory belongs to the call's stream: freed, it is not handed to
  // another stream's work while the call may still write it.
  at::Tensor fresh(at::IntArrayRef sizes, const at::TensorOptions &o) const {
    if (!given) return at::empty(sizes, o);
    c10::cuda::CUDAStreamGuard guard(
        c10::cuda::getStreamFromExternal((cudaStream_t)stream, (c10::DeviceIndex)dev));
    return at::empty(sizes, o);
  }
};

struct Items {  // of a Python sequence, held while they are looked at
  PyObject *s;
  explicit Items(PyObject *o) : s(PySequence_Fast(o, "src and dst must be sequences")) {
    if (!s) throw Bad();
  }
  ~Items() { Py_DECREF(s); }
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(s); }
  PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(s, i); }
};

bool overlap(const at::Tensor &x, const at::Tensor &y) {  // of contiguous tensors
  const uintptr_t a = (uintptr_t)x.data_ptr(), b = (uintptr_t)y.data_ptr();
  return x.nbytes() && y.nbytes() && a < b + y.nbytes() && b < a + x.nbytes();
}

template <typename T>
T *at_of(const at::Tensor &x) {
  return static_cast<T *>(x.data_ptr());
}

int rows_of(const at::Tensor &x) {
  if (x.size(0) > INT32_MAX) bad("a tensor has more than 2^31 - 1 rows");
  return (int)x.size(0);
}

// Number of sequences of the offsets and lengths, which have to agree on it.
int sequences(const at::Tensor *cu_q, const at::Tensor &cu_k, const at::Tensor *lens) {
  const int64_t s = cu_k.numel() - 1;
  if (s < 0 || s > INT32_MAX || (cu_q && cu_q->numel() != s + 1) || (lens && lens->numel() != s))
    bad("cu_seqlens_q, cu_seqlens_k and seqlens_k disagree on the sequences");
  return (int)s;
}

void check(hisa_status s, const char *name) {
  if (s == HISA_OK) return;
  PyObject *r = PyObject_CallFunction(g_raise, "is", (int)s, name);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, "the status was not raised");
  throw Bad();
}

void kv4_rows(Args &g, int i, const at::Tensor *&kv4, const at::Tensor *&scale) {
  kv4 = &g.tensor(i, "kv4", at::kByte, HISA_KV4_ROW_BYTES);
  scale = &g.tensor(i + 1, "kv4_scale", at::kByte, HISA_KV4_ROW_SCALES);
  if (kv4->size(0) != scale->size(0)) bad("kv4 and kv4_scale must have the same number of rows");
}

const int32_t *lengths(Args &g, int i, const at::Tensor *&x) {
  x = g.none(i) ? nullptr : &g.tensor(i, "seqlens_k", at::kInt);
  return x ? at_of<int32_t>(*x) : nullptr;
}

// k_new, v_new, cu_seqlens_q, cu_seqlens_k, seqlens_k, kv4, kv4_scale, stream
PyObject *kv4_store(Args g) {
  const at::Tensor *kv4, *scale, *lens;
  kv4_rows(g, 5, kv4, scale);
  const at::Tensor &k = g.tensor(0, "k_new", at::kBFloat16, HISA_ATT_DIM);
  const at::Tensor &v = g.tensor(1, "v_new", at::kBFloat16, HISA_ATT_DIM);
  const at::Tensor &cq = g.tensor(2, "cu_seqlens_q", at::kInt);
  const at::Tensor &ck = g.tensor(3, "cu_seqlens_k", at::kInt);
  const int32_t *n = lengths(g, 4, lens);
  const int s = sequences(&cq, ck, lens);
  if (k.size(0) != v.size(0)) bad("k_new and v_new must have the same shape");
  g.on(7);
  check(p_store(at_of<hisa_bf16>(k), at_of<hisa_bf16>(v), at_of<int32_t>(cq), at_of<int32_t>(ck),
                n, s, rows_of(k), at_of<uint8_t>(*kv4), at_of<uint8_t>(*scale), g.stream),
        "hisa_kv4_store");
  Py_RETURN_NONE;
}

// kv4, kv4_scale, cu_seqlens_q, cu_seqlens_k, seqlens_k, total_q, k_out, v_out, stream
PyObject *kv4_load(Args g) {
  const at::Tensor *kv4, *scale, *lens;
  kv4_rows(g, 0, kv4, scale);
  const at::Tensor &cq = g.tensor(2, "cu_seqlens_q", at::kInt);
  const at::Tensor &ck = g.tensor(3, "cu_seqlens_k", at::kInt);
  const int32_t *n = lengths(g, 4, lens);
  const int total_q = g.whole(5);
  const int s = sequences(&cq, ck, lens);
  if (total_q < 0) bad("total_q must not be negative");
  at::Tensor out[2];
  g.on(8);
  for (int i = 0; i < 2; i++) {
    if (g.none(6 + i))
      out[i] = g.fresh({total_q, HISA_ATT_DIM}, kv4->options().dtype(at::kBFloat16));
    else
      out[i] = g.tensor(6 + i, i ? "v_out" : "k_out", at::kBFloat16, HISA_ATT_DIM);
    if (out[i].size(0) != total_q) bad("k_out and v_out need one row per query row");
  }
  check(p_load(at_of<uint8_t>(*kv4), at_of<uint8_t>(*scale), at_of<int32_t>(cq),
               at_of<int32_t>(ck), n, s, total_q, at_of<hisa_bf16>(out[0]),
               at_of<hisa_bf16>(out[1]), g.stream),
        "hisa_kv4_load");
  PyObject *k = THPVariable_Wrap(out[0]), *v = THPVariable_Wrap(out[1]);
  PyObject *r = PyTuple_Pack(2, k, v);
  Py_DECREF(k);
  Py_DECREF(v);
  return r;
}

// The shapes of an attention's arguments, which have to fit one another.
struct AttShape {
  int total_q, heads, k;
};
AttShape att_shape(const at::Tensor &q, const at::Tensor &idx, const at::Tensor *lse,
                   const at::Tensor *weights, int64_t rows) {
  if (q.dim() != 3 || q.size(2) != HISA_ATT_DIM) bad("q_att must be [total_q, H, 128]");
  if (idx.dim() != 2 || idx.size(0) != q.size(0)) bad("topk_idx must be [total_q, k]");
  if (lse && (lse->dim() != 2 || lse->size(0) != q.size(0) || lse->size(1) != q.size(1)))
    bad("lse must be [total_q, H]");
  if (weights && weights->numel() != rows) bad("weights must hold one number per cache row");
  if (q.size(1) > INT32_MAX || idx.size(1) > INT32_MAX) bad("a size does not fit 32 bits");
  return {rows_of(q), (int)q.size(1), (int)idx.size(1)};
}

// q_att, kv4, kv4_scale, topk_idx, cu_seqlens_q, cu_seqlens_k, scale, out, lse, weights, stream
PyObject *attention_kv4(Args g) {
  const at::Tensor *kv4, *scale;
  const at::Tensor &q = g.tensor(0, "q_att", at::kBFloat16);
  kv4_rows(g, 1, kv4, scale);
  const at::Tensor &idx = g.tensor(3, "topk_idx", at::kInt);
  const at::Tensor &cq = g.tensor(4, "cu_seqlens_q", at::kInt);
  const at::Tensor &ck = g.tensor(5, "cu_seqlens_k", at::kInt);
  const double sc = PyFloat_AsDouble(g.a[6]);
  if (sc == -1.0 && PyErr_Occurred()) throw Bad();
  const at::Tensor *lse = g.none(8) ? nullptr : &g.tensor(8, "lse", at::kFloat);
  const at::Tensor *w = g.none(9) ? nullptr : &g.tensor(9, "weights", at::kLong);
  const AttShape s = att_shape(q, idx, lse, w, kv4->size(0));
  const int seqs = sequences(&cq, ck, nullptr);
  if (w && !lse) bad("weights need lse");
  g.on(10);
  at::Tensor made;
  if (g.none(7)) made = g.fresh(q.sizes(), q.options());
  const at::Tensor &out = g.none(7) ? made : g.tensor(7, "out", at::kBFloat16);
  if (out.sizes() != q.sizes()) bad("out must have the shape of q_att");
  check(p_attention(at_of<hisa_bf16>(q), at_of<uint8_t>(*kv4), at_of<uint8_t>(*scale),
                    at_of<int32_t>(idx), at_of<int32_t>(cq), at_of<int32_t>(ck), seqs, s.total_q,
                    s.heads, s.k, (float)sc, at_of<hisa_bf16>(out),
                    lse ? at_of<float>(*lse) : nullptr, w ? at_of<int64_t>(*w) : nullptr,
                    g.stream),
        "hisa_sparse_attention_kv4");
  if (g.none(7)) return THPVariable_Wrap(made);
  Py_INCREF(g.a[7]);
  return g.a[7];
}

// q_att, k_att, topk_idx, lse, cu_seqlens_q, cu_seqlens_k, scale, weights, stream
PyObject *token_weights(Args g) {
  const at::Tensor &q = g.tensor(0, "q_att", at::kBFloat16);
  const at::Tensor &k = g.tensor(1, "k_att", at::kBFloat16, HISA_ATT_DIM);
  const at::Tensor &idx = g.tensor(2, "topk_idx", at::kInt);
  const at::Tensor &lse = g.tensor(3, "lse", at::kFloat);
  const at::Tensor &cq = g.tensor(4, "cu_seqlens_q", at::kInt);
  const at::Tensor &ck = g.tensor(5, "cu_seqlens_k", at::kInt);
  const double sc = PyFloat_AsDouble(g.a[6]);
  if (sc == -1.0 && PyErr_Occurred()) throw Bad();
  const at::Tensor &w = g.tensor(7, "weights", at::kLong);
  const AttShape s = att_shape(q, idx, &lse, &w, k.size(0));
  const int seqs = sequences(&cq, ck, nullptr);
  g.on(8);
  check(p_weights(at_of<hisa_bf16>(q), at_of<hisa_bf16>(k), at_of<int32_t>(idx),
                  at_of<float>(lse), at_of<int32_t>(cq), at_of<int32_t>(ck), seqs, s.total_q,
                  s.heads, s.k, (float)sc, at_of<int64_t>(w), g.stream),
        "hisa_token_weights");
  Py_INCREF(g.a[7]);
  return g.a[7];
}

// weights, cu_seqlens_k, seqlens_k, keep, max_seqlen_k, n_sink, n_recent, kept, kept_len, stream
PyObject *evict_select(Args g) {
  const at::Tensor *lens;
  const at::Tensor &w = g.tensor(0, "weights", at::kLong);
  const at::Tensor &ck = g.tensor(1, "cu_seqlens_k", at::kInt);
  const int32_t *n = lengths(g, 2, lens);
  const at::Tensor &keep = g.tensor(3, "keep", at::kInt);
  const int s = sequences(nullptr, ck, lens);
  if (keep.numel() != s) bad("keep must hold one budget per sequence");
  at::Tensor kept, kept_len;
  const auto i32 = w.options().dtype(at::kInt);
  g.on(9);
  kept = g.none(7) ? g.fresh({w.numel()}, i32) : g.tensor(7, "kept", at::kInt);
  kept_len = g.none(8) ? g.fresh({s}, i32) : g.tensor(8, "kept_len", at::kInt);
  if (kept.numel() != w.numel() || kept_len.numel() != s)
    bad("kept must hold one number per cache row, kept_len one per sequence");
  for (const at::Tensor *in : {&w, &ck, &keep, lens})
    if (in && (overlap(kept, *in) || overlap(kept_len, *in)))
      bad("kept or kept_len overlaps an input");
  if (overlap(kept, kept_len)) bad("kept overlaps kept_len");
  check(p_select(at_of<int64_t>(w), at_of<int32_t>(ck), n, at_of<int32_t>(keep), s, g.whole(4),
                 g.whole(5), g.whole(6), at_of<int32_t>(kept), at_of<int32_t>(kept_len),
                 g.stream),
        "hisa_evict_select");
  PyObject *a = THPVariable_Wrap(kept), *b = THPVariable_Wrap(kept_len);
  PyObject *r = PyTuple_Pack(2, a, b);
  Py_DECREF(a);
  Py_DECREF(b);
  return r;
}

struct Span {
  uintptr_t from, to;
  bool dst;
};

// src, dst (sequences of tensors), cu_src, cu_dst, kept, kept_len, max_keep, stream
PyObject *evict_rows(Args g) {
  const at::Tensor &kept = g.tensor(4, "kept", at::kInt);
  const at::Tensor &kept_len = g.tensor(5, "kept_len", at::kInt);
  const at::Tensor &cs = g.tensor(2, "cu_src", at::kInt);
  const at::Tensor &cd = g.tensor(3, "cu_dst", at::kInt);
  const int s = sequences(&cd, cs, &kept_len);
  const Items src(g.a[0]), dst(g.a[1]);
  const Py_ssize_t n = src.size();
  if (dst.size() != n || n > HISA_MAX_ROW_ARRAYS) bad("src and dst must be as many arrays, at most 8");
  std::vector<Span> spans;
  hisa_rows rows[HISA_MAX_ROW_ARRAYS];
  auto span = [&](const at::Tensor &x, bool dst) {
    const uintptr_t p = (uintptr_t)x.data_ptr();
    spans.push_back({p, p + x.nbytes(), dst});
  };
  for (const at::Tensor *in : {&kept, &kept_len, &cs, &cd}) span(*in, false);
  for (Py_ssize_t i = 0; i < n; i++) {
    const at::Tensor *t[2];
    for (int d = 0; d < 2; d++) {
      PyObject *o = d ? dst[i] : src[i];
      const char *name = d ? "a destination" : "a source";
      if (!THPVariable_Check(o)) bad("%s must be a tensor", name);
      t[d] = &THPVariable_Unpack(o);
      if (!t[d]->is_cuda()) bad("%s must be a CUDA tensor", name);
      if (!t[d]->is_contiguous()) bad("row arrays must be contiguous: %s is not", name);
      g.place(*t[d], name);
    }
    const at::Tensor &a = *t[0], &b = *t[1];
    if (a.dim() < 1 || b.dim() < 1 || a.scalar_type() != b.scalar_type() ||
        a.sizes().slice(1) != b.sizes().slice(1))
      bad("a source and its destination must have rows of one type and shape");
    if (a.size(0) != kept.numel()) bad("kept must hold one number per source row");
    rows[i] = {a.data_ptr(), b.data_ptr(),
               a.size(0) ? (size_t)(a.nbytes() / a.size(0)) : (size_t)4};
    span(b, true);  // in place counts once
    if (a.data_ptr() != b.data_ptr() || a.nbytes() != b.nbytes()) span(a, false);
  }
  // in order of their starts, a span may touch none before it, unless both are sources
  std::sort(spans.begin(), spans.end(),
            [](const Span &x, const Span &y) { return x.from < y.from; });
  uintptr_t end = 0, end_dst = 0;
  for (const Span &x : spans) {
    if (x.from < (x.dst ? end : end_dst) && x.from < x.to)
      bad("a destination overlaps a source, kept or an offset, or two destinations overlap");
    end = std::max(end, x.to);
    if (x.dst) end_dst = std::max(end_dst, x.to);
  }
  g.on(7);
  check(p_rows(rows, (int)n, at_of<int32_t>(cs), at_of<int32_t>(cd), at_of<int32_t>(kept),
               at_of<int32_t>(kept_len), s, g.whole(6), g.stream),
        "hisa_evict_rows");
  Py_RETURN_NONE;
}

template <PyObject *(*F)(Args), int N>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
    return nullptr;
  }
  if (!g_raise) {
    PyErr_SetString(PyExc_RuntimeError, "setup() has not been called");
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    Args g;
    g.a = a;
    return F(g);
  } catch (const Bad &) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// raise, then the addresses of the six entry points in the order of the pointers above
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "7 arguments are wanted");
    return nullptr;
  }
  void *p[6];
  for (int i = 0; i < 6; i++) {
    p[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) return nullptr;
  }
  p_store = (decltype(p_store))p[0];
  p_load = (decltype(p_load))p[1];
  p_attention = (decltype(p_attention))p[2];
  p_weights = (decltype(p_weights))p[3];
  p_select = (decltype(p_select))p[4];
  p_rows = (decltype(p_rows))p[5];
  Py_INCREF(a[0]);
  Py_XDECREF(g_raise);
  g_raise = a[0];
  Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    ENTRY(kv4_store, 8),
    ENTRY(kv4_load, 9),
    ENTRY(attention_kv4, 11),
    ENTRY(token_weights, 9),
    ENTRY(evict_select, 10),
    ENTRY(evict_rows, 8),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hisa_torch", nullptr, -1, methods};

}  // namespace

// BUILT_FOR: the torch and Python whose headers the code above was compiled with; the caller
// compares before the first call.
PyMODINIT_FUNC PyInit__hisa_torch(void) {
  PyObject *m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "BUILT_FOR", HISA_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
