// Host side of the rotary and paged-attention calls: checks of the tensors, the
// argument block, the result and the call itself, in one step from Python.
//
// What bounds a call on a few tokens is the host: looking at eight or nine tensors
// from Python (type, shape, strides, pointer) and packing what was found took 10 of the
// 16 us between two calls, of which the GPU worked 4 to 15. A tensor takes some 30 ns
// here, a call 5 us in all (3 of them the launch): one token's cache write took 17.1 us among
// others without it and takes 5.0, the host's time; attention of one token over 1037 went from
// 22.5 to the GPU's own time (12.0 now).
//
// A function returns the call's result, or None for anything out of the ordinary: a
// tensor that does not fit, an argument of an unusual type, a refusal by the library.
// The caller then goes through the same arguments in Python, which says what is wrong
// (or makes the call). So nothing here raises, and nothing is decided here alone.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <limits>
#include <optional>

#include "kaio_qkv.h"

namespace {

int (*g_rope)(const kaio_rope_args*, void*);
int (*g_rope_append)(const kaio_rope_args*, void*);
int (*g_paged_attention)(const kaio_paged_attention_args*, void*);

// A tensor on a GPU, dense in its last dimension, without gradient tracking.
const at::Tensor* usable(PyObject* o, int rank) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.requires_grad() || t.dim() != rank) return nullptr;
  if (t.size(rank - 1) > 1 && t.stride(rank - 1) != 1) return nullptr;
  return &t;
}

const at::Tensor* usable(PyObject* o, at::ScalarType type, at::IntArrayRef sizes) {
  const at::Tensor* t = usable(o, static_cast<int>(sizes.size()));
  return t && t->scalar_type() == type && t->sizes() == sizes ? t : nullptr;
}

bool type_code(const at::Tensor& t, int32_t* code) {
  if (t.scalar_type() == at::kHalf) *code = KAIO_DTYPE_F16;
  else if (t.scalar_type() == at::kBFloat16) *code = KAIO_DTYPE_BF16;
  else return false;
  return true;
}

bool to_int(PyObject* o, int32_t* v) {
  if (!PyLong_Check(o)) return false;
  int over = 0;
  const long x = PyLong_AsLongAndOverflow(o, &over);
  if (over || x < std::numeric_limits<int32_t>::min() || x > std::numeric_limits<int32_t>::max()) return false;
  *v = static_cast<int32_t>(x);
  return true;
}

bool fits(int64_t n) { return n <= std::numeric_limits<int32_t>::max(); }

bool to_flag(PyObject* o, int32_t* v) {
  if (!PyBool_Check(o)) return false;
  *v = o == Py_True;
  return true;
}

// The stream given, or the current one of the tensor's device.
bool stream_of(PyObject* o, const at::Tensor& t, void** stream) {
  if (o == Py_None) {
    *stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
    return true;
  }
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) return false;
  *stream = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  return !PyErr_Occurred();
}

template <typename Args>
bool call(int (*entry)(const Args*, void*), const Args& args, void* stream) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = entry(&args, stream);
  Py_END_ALLOW_THREADS
  return status == KAIO_OK;
}

// positions [T] or [axes, T], inv_freq [R] and the pairs of each axis
bool rope_angles(kaio_rope_args* a, PyObject* positions, PyObject* inv_freq, PyObject* sections, int64_t tokens) {
  const at::Tensor* f = usable(inv_freq, 1);
  if (!f || f->scalar_type() != at::kFloat || !fits(f->size(0))) return false;
  a->pairs = static_cast<int32_t>(f->size(0));
  a->inv_freq = static_cast<const float*>(f->data_ptr());
  const at::Tensor* p = usable(positions, 1);
  int64_t axes = 1;
  if (!p) {
    p = usable(positions, 2);
    if (!p) return false;
    axes = p->size(0);
    a->positions_axis_stride = p->stride(0);
  }
  if (p->scalar_type() != at::kInt || p->size(p->dim() - 1) != tokens || axes > 4) return false;
  a->positions = static_cast<const int32_t*>(p->data_ptr());
  a->axes = static_cast<int32_t>(axes);
  if (sections == Py_None) {
    a->sections[0] = a->pairs;
    return axes == 1;
  }
  if (!PyTuple_Check(sections) && !PyList_Check(sections)) return false;
  if (PySequence_Fast_GET_SIZE(sections) != axes) return false;
  for (int i = 0; i < axes; ++i)
    if (!to_int(PySequence_Fast_GET_ITEM(sections, i), &a->sections[i])) return false;
  return true;
}

// A new result, which belongs to the stream that the kernel runs on (see kaio._empty).
at::Tensor new_tensor(at::IntArrayRef sizes, const at::TensorOptions& options, PyObject* given_stream, void* stream) {
  std::optional<c10::cuda::CUDAStreamGuard> on;
  if (given_stream != Py_None)
    on.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), options.device().index()));
  return at::empty(sizes, options);
}

// The result: the tensor given, or a new dense one like x.
const at::Tensor* result_like(PyObject* given, const at::Tensor& x, PyObject* given_stream, void* stream,
                              at::Tensor* made, int64_t* ts, int64_t* hs) {
  const at::Tensor* out;
  if (given == Py_None) {
    *made = new_tensor(x.sizes(), x.options(), given_stream, stream);
    *ts = x.size(1) * x.size(2);
    *hs = x.size(2);
    return made;
  }
  out = usable(given, x.scalar_type(), x.sizes());
  if (!out) return nullptr;
  *ts = out->stride(0);
  *hs = out->stride(1);
  return out;
}

PyObject* hand_back(PyObject* given, const at::Tensor& made) {
  return given == Py_None ? THPVariable_Wrap(made) : Py_NewRef(given);
}

// (x, positions, inv_freq, sections, interleaved, inverse, out, stream)
PyObject* rope(PyObject* const* v) {
  const at::Tensor* x = usable(v[0], 3);
  kaio_rope_args a{};
  a.struct_size = sizeof(a);
  if (!x || !type_code(*x, &a.dtype) || !fits(x->size(0)) || !fits(x->size(1)) || !fits(x->size(2))) return nullptr;
  a.tokens = static_cast<int32_t>(x->size(0)), a.heads = static_cast<int32_t>(x->size(1));
  a.dim = static_cast<int32_t>(x->size(2));
  a.q = x->data_ptr(), a.q_token_stride = x->stride(0), a.q_head_stride = x->stride(1);
  void* stream;
  if (!rope_angles(&a, v[1], v[2], v[3], x->size(0)) || !to_flag(v[4], &a.interleaved) || !to_flag(v[5], &a.inverse) ||
      !stream_of(v[7], *x, &stream))
    return nullptr;
  at::Tensor made;
  const at::Tensor* out = result_like(v[6], *x, v[7], stream, &made, &a.q_out_token_stride, &a.q_out_head_stride);
  if (!out) return nullptr;
  a.q_out = out->data_ptr();
  return call(g_rope, a, stream) ? hand_back(v[6], made) : nullptr;
}

// (q, k, v, positions, inv_freq, k_cache, v_cache, slots, sections, interleaved, q_out, stream)
PyObject* rope_append(PyObject* const* v) {
  const at::Tensor *q = usable(v[0], 3), *k = usable(v[1], 3), *kc = usable(v[5], 4);
  kaio_rope_args a{};
  a.struct_size = sizeof(a);
  if (!q || !k || !kc || !type_code(*q, &a.dtype)) return nullptr;
  const at::ScalarType type = q->scalar_type();
  const int64_t t = q->size(0), h = q->size(1), d = q->size(2), kh = k->size(1);
  if (!fits(t) || !fits(h) || !fits(d) || !fits(kh) || !fits(kc->size(0)) || !fits(kc->size(1))) return nullptr;
  const int64_t kv[3] = {t, kh, d}, cache[4] = {kc->size(0), kc->size(1), kh, d}, one[1] = {t};
  if (k->scalar_type() != type || k->sizes() != at::IntArrayRef(kv) || kc->scalar_type() != type ||
      kc->sizes() != at::IntArrayRef(cache))
    return nullptr;
  const at::Tensor *vv = usable(v[2], type, kv), *vc = usable(v[6], type, cache), *slots = usable(v[7], at::kInt, one);
  if (!vv || !vc || !slots) return nullptr;
  a.tokens = static_cast<int32_t>(t), a.heads = static_cast<int32_t>(h), a.kv_heads = static_cast<int32_t>(kh);
  a.dim = static_cast<int32_t>(d);
  a.num_pages = static_cast<int32_t>(cache[0]), a.page_size = static_cast<int32_t>(cache[1]);
  a.q = q->data_ptr(), a.k = k->data_ptr(), a.v = vv->data_ptr(), a.k_cache = kc->data_ptr(), a.v_cache = vc->data_ptr();
  a.slots = static_cast<const int32_t*>(slots->data_ptr());
  a.q_token_stride = q->stride(0), a.q_head_stride = q->stride(1);
  a.k_token_stride = k->stride(0), a.k_head_stride = k->stride(1);
  a.v_token_stride = vv->stride(0), a.v_head_stride = vv->stride(1);
  a.k_page_stride = kc->stride(0), a.k_slot_stride = kc->stride(1), a.k_cache_head_stride = kc->stride(2);
  a.v_page_stride = vc->stride(0), a.v_slot_stride = vc->stride(1), a.v_cache_head_stride = vc->stride(2);
  void* stream;
  if (!rope_angles(&a, v[3], v[4], v[8], t) || !to_flag(v[9], &a.interleaved) || !stream_of(v[11], *q, &stream)) return nullptr;
  at::Tensor made;
  const at::Tensor* out = result_like(v[10], *q, v[11], stream, &made, &a.q_out_token_stride, &a.q_out_head_stride);
  if (!out) return nullptr;
  a.q_out = out->data_ptr();
  return call(g_rope_append, a, stream) ? hand_back(v[10], made) : nullptr;
}

// (q, k_cache, v_cache, page_table, kv_lens, q_starts, max_new, scale, causal, window, sinks, workspace, out,
//  return_lse, lse, stream)
PyObject* paged_attention(PyObject* const* v) {
  const at::Tensor *q = usable(v[0], 3), *kc = usable(v[1], 4), *table = usable(v[3], 2), *lens = usable(v[4], 1);
  const at::Tensor* ws = usable(v[11], 1);
  kaio_paged_attention_args a{};
  a.struct_size = sizeof(a);
  if (!q || !kc || !table || !lens || !ws || !type_code(*q, &a.dtype)) return nullptr;
  const at::ScalarType type = q->scalar_type();
  const int64_t t = q->size(0), h = q->size(1), d = q->size(2), b = lens->size(0);
  const int64_t cache[4] = {kc->size(0), kc->size(1), kc->size(2), d}, lse_size[2] = {t, h}, starts_size[1] = {b + 1};
  if (!fits(t) || !fits(h) || !fits(d) || !fits(b) || !fits(cache[0]) || !fits(cache[1]) || !fits(cache[2]) ||
      !fits(table->size(1)))
    return nullptr;
  const at::Tensor* vc = usable(v[2], type, cache);
  if (!vc || kc->scalar_type() != type || kc->sizes() != at::IntArrayRef(cache) || lens->scalar_type() != at::kInt ||
      table->scalar_type() != at::kInt || table->size(0) != b || ws->scalar_type() != at::kByte)
    return nullptr;
  a.batch = static_cast<int32_t>(b), a.tokens = static_cast<int32_t>(t), a.heads = static_cast<int32_t>(h);
  a.kv_heads = static_cast<int32_t>(cache[2]), a.dim = static_cast<int32_t>(d);
  a.num_pages = static_cast<int32_t>(cache[0]), a.page_size = static_cast<int32_t>(cache[1]);
  a.max_pages = static_cast<int32_t>(table->size(1));
  a.q = q->data_ptr(), a.k_cache = kc->data_ptr(), a.v_cache = vc->data_ptr();
  a.page_table = static_cast<const int32_t*>(table->data_ptr()), a.kv_lens = static_cast<const int32_t*>(lens->data_ptr());
  a.workspace = ws->data_ptr(), a.workspace_bytes = static_cast<uint64_t>(ws->numel());
  a.q_token_stride = q->stride(0), a.q_head_stride = q->stride(1);
  a.k_page_stride = kc->stride(0), a.k_slot_stride = kc->stride(1), a.k_head_stride = kc->stride(2);
  a.v_page_stride = vc->stride(0), a.v_slot_stride = vc->stride(1), a.v_head_stride = vc->stride(2);
  a.table_stride = table->stride(0);
  a.max_new = 1;
  if (v[5] != Py_None) {
    const at::Tensor* starts = usable(v[5], at::kInt, starts_size);
    if (!starts) return nullptr;
    a.q_starts = static_cast<const int32_t*>(starts->data_ptr());
    a.max_new = a.tokens;
  }
  if (v[6] != Py_None && !to_int(v[6], &a.max_new)) return nullptr;
  if (v[7] == Py_None) a.scale = static_cast<float>(std::pow(static_cast<double>(d), -0.5));
  else if (PyFloat_Check(v[7])) a.scale = static_cast<float>(PyFloat_AS_DOUBLE(v[7]));
  else return nullptr;
  void* stream;
  if (!to_flag(v[8], &a.causal) || !to_int(v[9], &a.window) || !to_int(v[10], &a.sinks) || !PyBool_Check(v[13]) ||
      !stream_of(v[15], *q, &stream))
    return nullptr;
  at::Tensor made, made_lse;
  const at::Tensor* out = result_like(v[12], *q, v[15], stream, &made, &a.out_token_stride, &a.out_head_stride);
  if (!out) return nullptr;
  a.out = out->data_ptr();
  const bool wants_lse = v[13] == Py_True;
  if (v[14] != Py_None) {
    const at::Tensor* lse = usable(v[14], at::kFloat, lse_size);
    if (!lse || (t > 1 && lse->stride(0) != h)) return nullptr;
    a.lse = static_cast<float*>(lse->data_ptr());
  } else if (wants_lse) {
    made_lse = new_tensor(lse_size, q->options().dtype(at::kFloat), v[15], stream);
    a.lse = static_cast<float*>(made_lse.data_ptr());
  }
  if (!call(g_paged_attention, a, stream)) return nullptr;
  PyObject* first = hand_back(v[12], made);
  if (!wants_lse || !first) return first;
  PyObject* second = hand_back(v[14], made_lse);
  PyObject* both = second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_DECREF(first);
  Py_XDECREF(second);
  return both;
}

template <PyObject* (*kCall)(PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  PyObject* result = nullptr;
  try {
    if (n == kArgs) result = kCall(args);
  } catch (...) {
    result = nullptr;
  }
  if (result) return result;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// The library's entries, as addresses: kaio_rope, kaio_rope_append, kaio_paged_attention.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes three addresses");
    return nullptr;
  }
  void* at[3];
  for (int i = 0; i < 3; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_rope = reinterpret_cast<decltype(g_rope)>(at[0]);
  g_rope_append = reinterpret_cast<decltype(g_rope_append)>(at[1]);
  g_paged_attention = reinterpret_cast<decltype(g_paged_attention)>(at[2]);
  Py_RETURN_NONE;
}

template <typename F> PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef g_methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"rope", fast(entry<rope, 8>), METH_FASTCALL, nullptr},
    {"rope_append", fast(entry<rope_append, 12>), METH_FASTCALL, nullptr},
    {"paged_attention", fast(entry<paged_attention, 16>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&g_module); }
