// tensors.cpp — the serving operators on torch tensors: a CPython module that
// checks what a struct of addresses cannot show (types, shapes, strides,
// devices), fills the C ABI's argument structs, makes the outputs that the
// caller did not bring and enqueues on the caller's stream.
//
// A single-token operator takes a few microseconds on the device; marshalled
// attribute by attribute from Python, its call takes three times as long.
// The module holds no link to libmk.so: the binding hands it the functions'
// addresses and the exception class once (init).
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/mk.h"

namespace {

struct Refusal {
  int status;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refusal{MK_ERR_INVALID_ARG, what}; }

struct Abi {
  decltype(&mk_append_kv) append = nullptr;
  decltype(&mk_prompt_attention) prompt = nullptr;
  decltype(&mk_prompt_attention_workspace_bytes) prompt_bytes = nullptr;
  decltype(&mk_paged_attention) paged = nullptr;
  decltype(&mk_paged_attention_workspace_bytes) paged_bytes = nullptr;
  decltype(&mk_process_logits) logits = nullptr;
  decltype(&mk_last_error) last_error = nullptr;
  PyObject* error = nullptr;  // MkError(status, message)
} abi;

std::string shape_text(const at::Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

// the tensor behind an argument; nullptr for None
const at::Tensor* given(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = given(o, name);
  if (!t) refuse(std::string(name) + " is required");
  return *t;
}

int element_type(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MK_DTYPE_BF16;
    case at::kHalf: return MK_DTYPE_FP16;
    case at::kFloat: return MK_DTYPE_FP32;
    default: return -1;
  }
}

int as_int(int64_t v, const char* name) {
  if (v > 0x7fffffff) refuse(std::string(name) + ": a size above 2^31 - 1");
  return static_cast<int>(v);
}

// Address and strides of a [rows][heads][head_dim] tensor whose last dimension
// is dense (the stride of a dimension of size 1 is not used).
template <class P>
void rows(const char* name, const at::Tensor& t, int64_t n, int64_t heads, int64_t d, at::ScalarType type, P& p,
          long long& row_stride, long long& head_stride) {
  if (t.scalar_type() != type || t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != d)
    refuse(std::string(name) + " must be " + c10::toString(type) + " [" + std::to_string(n) + ", " + std::to_string(heads) +
           ", " + std::to_string(d) + "], not " + shape_text(t));
  if (d > 1 && t.stride(2) != 1) refuse(std::string(name) + ": the last dimension must be dense");
  p = t.data_ptr();
  row_stride = n > 1 ? t.stride(0) : 0;
  head_stride = heads > 1 ? t.stride(1) : 0;
}

// an output's rows must not lie on top of one another
void apart(const char* name, long long row_stride, long long head_stride, int64_t n, int64_t heads, int64_t d) {
  const bool wide_rows = row_stride >= head_stride;
  const long long outer = wide_rows ? row_stride : head_stride, inner = wide_rows ? head_stride : row_stride;
  const int64_t n_outer = wide_rows ? n : heads, n_inner = wide_rows ? heads : n;
  if ((n_inner > 1 && inner < d) || (n_outer > 1 && outer < (n_inner - 1) * inner + d))
    refuse(std::string(name) + ": its rows overlap");
}

// address of a dense array of n values; nullptr: not given
void* array(const char* name, const at::Tensor* t, at::ScalarType type, int64_t n) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    refuse(std::string(name) + " must be a dense " + c10::toString(type) + " [" + std::to_string(n) + "], not " + shape_text(*t));
  return t->data_ptr();
}

// [n][width] with dense rows (width < 0: any)
void* dense_rows(const char* name, const at::Tensor& t, at::ScalarType type, int64_t n, int64_t width, long long& stride) {
  if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != n || (width >= 0 && t.size(1) != width))
    refuse(std::string(name) + " must be " + c10::toString(type) + " [" + std::to_string(n) + ", " +
           (width < 0 ? "n" : std::to_string(width)) + "], not " + shape_text(t));
  if (t.size(1) > 1 && t.stride(1) != 1) refuse(std::string(name) + " must have dense rows");
  stride = n > 1 ? t.stride(0) : t.size(1);
  return t.data_ptr();
}

void pages(mk_kv_pages& p, const at::Tensor& k, const at::Tensor& v, const at::Tensor& table, int64_t batch) {
  const int type = element_type(k);
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || type < 0 || type == MK_DTYPE_FP32)
    refuse("k and v pages must both be bf16 or fp16 [n_pages][n_kv_heads][page_size][head_dim]");
  long long st[4];
  for (int i = 0; i < 4; ++i) {
    st[i] = k.size(i) > 1 ? k.stride(i) : (i == 3 ? 1 : 0);
    if (k.size(i) > 1 && v.stride(i) != k.stride(i)) refuse("k and v pages must have the same strides");
  }
  if (st[3] != 1) refuse("k and v pages must have a dense last dimension");
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != batch)
    refuse("page_table must be int32 [batch][width], not " + shape_text(table));
  if (table.size(1) > 1 && table.stride(1) != 1) refuse("page_table must have dense rows");
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  p.dtype = type;
  p.n_pages = as_int(k.size(0), "pages");
  p.n_kv_heads = as_int(k.size(1), "pages");
  p.page_size = as_int(k.size(2), "pages");
  p.head_dim = as_int(k.size(3), "pages");
  p.page_stride = st[0];
  p.head_stride = st[1];
  p.row_stride = st[2];
  p.page_table = static_cast<const int*>(table.data_ptr());
  p.table_width = as_int(table.size(1), "page_table");
  p.table_stride = as_int(batch > 1 ? table.stride(0) : table.size(1), "page_table");
}

float scale_of(PyObject* o) {
  if (o == Py_None) return 0.f;
  const double s = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw python_error();
  const float f = static_cast<float>(s);
  if (!(f > 0.f)) refuse("scale must be above 0 in fp32");  // (0 would stand for 1 / sqrt(head_dim))
  return f;
}

// Where a call runs: every tensor on one CUDA device, that device current, and
// the stream given (or the device's current one) current, so that outputs made
// here belong to it.
struct Place {
  c10::Device device;
  c10::cuda::OptionalCUDAStreamGuard guard;
  cudaStream_t raw = nullptr;

  Place(const at::Tensor& first, std::initializer_list<const at::Tensor*> others, PyObject* stream) : device(first.device()) {
    if (!device.is_cuda()) refuse("the tensors must be on a CUDA device");
    for (const at::Tensor* t : others)
      if (t && t->device() != device)
        refuse("a tensor " + shape_text(*t) + " is on " + t->device().str() + ", the others on " + device.str());
    if (stream == Py_None) {
      const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream(device.index());
      if (c10::cuda::current_device() != device.index()) guard.reset_stream(s);
      raw = s.stream();
      return;
    }
    long long part[3];
    const char* names[3] = {"stream_id", "device_index", "device_type"};
    for (int i = 0; i < 3; ++i) {
      PyObject* v = PyObject_GetAttrString(stream, names[i]);
      if (!v) {
        PyErr_Clear();
        refuse("stream must be a torch.cuda.Stream");
      }
      part[i] = PyLong_AsLongLong(v);
      Py_DECREF(v);
      if (PyErr_Occurred()) throw python_error();
    }
    const c10::Stream s = c10::Stream::unpack3(part[0], static_cast<c10::DeviceIndex>(part[1]), static_cast<c10::DeviceType>(part[2]));
    if (s.device() != device) refuse("the stream is on " + s.device().str() + ", the tensors on " + device.str());
    guard.reset_stream(s);
    raw = c10::cuda::CUDAStream(s).stream();
  }
};

void done(int status) {
  if (status != MK_OK) throw Refusal{status, abi.last_error()};
}

PyObject* result(PyObject* given_out, const at::Tensor& out) {
  if (given_out != Py_None) return Py_NewRef(given_out);
  return THPVariable_Wrap(out);
}

// ---------------------------------------------------------------- the operators (arguments in the binding's order)
// q, k, v, k_pages, v_pages, page_table, ctx_lens, cu_seqlens, rope_theta, q_out, status, stream
PyObject* append(PyObject* const* o) {
  const at::Tensor *q = given(o[0], "q"), &k = needed(o[1], "k"), &v = needed(o[2], "v"), &kp = needed(o[3], "k_pages"),
                   &vp = needed(o[4], "v_pages"), &table = needed(o[5], "page_table"), &ctx = needed(o[6], "ctx_lens"),
                   &cu = needed(o[7], "cu_seqlens"), *qo = given(o[9], "q_out"), *status = given(o[10], "status");
  mk_append_args a = {};
  const int64_t batch = ctx.numel();
  pages(a.pages, kp, vp, table, batch);
  if (k.dim() != 3) refuse("k must be [tokens][n_kv_heads][head_dim]");
  const int64_t n = k.size(0), d = kp.size(3);
  const at::ScalarType type = kp.scalar_type();
  a.batch = as_int(batch, "ctx_lens");
  a.n_tokens = as_int(n, "k");
  rows("k", k, n, kp.size(1), d, type, a.k, a.k_row_stride, a.k_head_stride);
  rows("v", v, n, kp.size(1), d, type, a.v, a.v_row_stride, a.v_head_stride);
  a.ctx_lens = static_cast<const int*>(array("ctx_lens", &ctx, at::kInt, batch));
  a.cu_seqlens = static_cast<const int*>(array("cu_seqlens", &cu, at::kInt, batch + 1));
  a.status = static_cast<int*>(array("status", status, at::kInt, 1));
  if (o[8] != Py_None) {
    a.rope_theta = PyFloat_AsDouble(o[8]);
    if (PyErr_Occurred()) throw python_error();
  }
  if (q) {
    if (q->dim() != 3) refuse("q must be [tokens][n_q_heads][head_dim]");
    a.n_q_heads = as_int(q->size(1), "q");
    rows("q", *q, n, q->size(1), d, type, a.q, a.q_row_stride, a.q_head_stride);
  } else if (qo) {
    refuse("q_out without q");
  }
  Place place(k, {q, &v, &kp, &vp, &table, &ctx, &cu, qo, status}, o[11]);
  at::Tensor out;
  if (q) {
    out = qo ? *qo : at::empty(q->sizes(), q->options());
    rows("q_out", out, n, q->size(1), d, type, a.q_out, a.qo_row_stride, a.qo_head_stride);
    apart("q_out", a.qo_row_stride, a.qo_head_stride, n, q->size(1), d);
  }
  done(abi.append(&a, place.raw));
  if (!q) Py_RETURN_NONE;
  return result(o[9], out);
}

// q, k, v, cu_q, cu_k, page_table, kv_lens, causal, scale, out, workspace, status, stream
PyObject* prompt(PyObject* const* o) {
  const at::Tensor &q = needed(o[0], "q"), &k = needed(o[1], "k"), &v = needed(o[2], "v"), &cu_q = needed(o[3], "cu_q"),
                   *cu_k = given(o[4], "cu_k"), *table = given(o[5], "page_table"), *lens = given(o[6], "kv_lens"),
                   *given_out = given(o[9], "out"), *given_ws = given(o[10], "workspace"), *status = given(o[11], "status");
  mk_prompt_args a = {};
  mk_kv_pages& p = a.pages;
  if (cu_q.numel() < 1) refuse("cu_q must be int32 [batch + 1]");
  const int64_t batch = cu_q.numel() - 1;
  if (table) {
    if (!lens || cu_k) refuse("paged keys take kv_lens, not cu_k");
    if (table->numel() == 0 && batch > 0) refuse("page_table names no pages");
    pages(p, k, v, *table, batch);
    a.kv_lens = static_cast<const int*>(array("kv_lens", lens, at::kInt, batch));
  } else {
    if (lens) refuse("packed keys take cu_k, not kv_lens");
    p.dtype = element_type(k);
    if (k.dim() != 3 || p.dtype < 0 || p.dtype == MK_DTYPE_FP32) refuse("k and v must both be bf16 or fp16 [tokens][n_kv_heads][head_dim]");
    long long row, head;
    rows("k", k, k.size(0), k.size(1), k.size(2), k.scalar_type(), p.k, p.row_stride, p.head_stride);
    rows("v", v, k.size(0), k.size(1), k.size(2), k.scalar_type(), p.v, row, head);
    if (row != p.row_stride || head != p.head_stride) refuse("k and v must have the same strides");
    p.n_pages = 1;
    p.page_size = as_int(k.size(0), "k");
    p.n_kv_heads = as_int(k.size(1), "k");
    p.head_dim = as_int(k.size(2), "k");
    a.cu_k = static_cast<const int*>(array("cu_k", cu_k ? cu_k : &cu_q, at::kInt, batch + 1));
  }
  if (q.dim() != 3) refuse("q must be [tokens][n_q_heads][head_dim]");
  const int64_t n = q.size(0), heads = q.size(1);
  a.batch = as_int(batch, "cu_q");
  a.n_tokens = as_int(n, "q");
  a.n_q_heads = as_int(heads, "q");
  a.causal = PyObject_IsTrue(o[7]);
  if (a.causal < 0) throw python_error();
  a.scale = scale_of(o[8]);
  rows("q", q, n, heads, p.head_dim, k.scalar_type(), a.q, a.q_row_stride, a.q_head_stride);
  a.cu_q = static_cast<const int*>(array("cu_q", &cu_q, at::kInt, batch + 1));
  a.status = static_cast<int*>(array("status", status, at::kInt, 1));
  if (given_ws && (given_ws->scalar_type() != at::kByte || !given_ws->is_contiguous())) refuse("workspace must be a dense uint8 tensor");
  Place place(q, {&k, &v, &cu_q, cu_k, table, lens, given_out, given_ws, status}, o[12]);
  const at::Tensor out = given_out ? *given_out : at::empty(q.sizes(), q.options());
  rows("out", out, n, heads, p.head_dim, q.scalar_type(), a.out, a.o_row_stride, a.o_head_stride);
  apart("out", a.o_row_stride, a.o_head_stride, n, heads, p.head_dim);
  at::Tensor ws;
  if (given_ws) {
    ws = *given_ws;
  } else {
    const size_t bytes = abi.prompt_bytes(a.batch, a.n_tokens, a.n_q_heads, p.n_kv_heads, p.head_dim,
                                          (long long)p.page_size * (table ? p.table_width : 1));
    if (bytes) ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
  }
  if (ws.defined()) {
    a.workspace = ws.data_ptr();
    a.workspace_bytes = static_cast<size_t>(ws.numel());
  }
  done(abi.prompt(&a, place.raw));
  return result(o[9], out);
}

// q, k_pages, v_pages, page_table, kv_lens, scale, out, workspace, status, stream
PyObject* paged(PyObject* const* o) {
  const at::Tensor &q = needed(o[0], "q"), &kp = needed(o[1], "k_pages"), &vp = needed(o[2], "v_pages"),
                   &table = needed(o[3], "page_table"), &lens = needed(o[4], "kv_lens"), *given_out = given(o[6], "out"),
                   *given_ws = given(o[7], "workspace"), *status = given(o[8], "status");
  if (q.dim() != 3) refuse("q must be [batch][n_q_heads][head_dim]");
  mk_paged_attn_args a = {};
  const int64_t n = q.size(0), heads = q.size(1);
  pages(a.pages, kp, vp, table, n);
  a.batch = as_int(n, "q");
  a.n_q_heads = as_int(heads, "q");
  a.scale = scale_of(o[5]);
  rows("q", q, n, heads, kp.size(3), kp.scalar_type(), a.q, a.q_row_stride, a.q_head_stride);
  a.kv_lens = static_cast<const int*>(array("kv_lens", &lens, at::kInt, n));
  a.status = static_cast<int*>(array("status", status, at::kInt, 1));
  if (given_ws && (given_ws->scalar_type() != at::kByte || !given_ws->is_contiguous())) refuse("workspace must be a dense uint8 tensor");
  Place place(q, {&kp, &vp, &table, &lens, given_out, given_ws, status}, o[9]);
  const at::Tensor out = given_out ? *given_out : at::empty(q.sizes(), q.options());
  rows("out", out, n, heads, kp.size(3), q.scalar_type(), a.out, a.o_row_stride, a.o_head_stride);
  apart("out", a.o_row_stride, a.o_head_stride, n, heads, kp.size(3));
  at::Tensor ws;
  if (given_ws) {
    ws = *given_ws;
  } else {
    ws = at::empty({static_cast<int64_t>(abi.paged_bytes(a.batch, a.n_q_heads, a.pages.n_kv_heads, a.pages.head_dim))},
                   q.options().dtype(at::kByte));
  }
  a.workspace = ws.data_ptr();
  a.workspace_bytes = static_cast<size_t>(ws.numel());
  done(abi.paged(&a, place.raw));
  return result(o[6], out);
}

// logits, history, history_lens, prompt_lens, repetition, frequency, presence, bias indptr, ids, values, mask, out,
// next_tokens, status, stream
PyObject* logits(PyObject* const* o) {
  const at::Tensor &x = needed(o[0], "logits"), *history = given(o[1], "history"), *lens = given(o[2], "history_lens"),
                   *prompts = given(o[3], "prompt_lens"), *rep = given(o[4], "repetition"), *freq = given(o[5], "frequency"),
                   *pres = given(o[6], "presence"), *indptr = given(o[7], "bias indptr"), *ids = given(o[8], "bias ids"),
                   *values = given(o[9], "bias values"), *mask = given(o[10], "mask"), *given_out = given(o[11], "out"),
                   *given_next = given(o[12], "next_tokens"), *status = given(o[13], "status");
  mk_logits_args a = {};
  a.dtype = element_type(x);
  if (a.dtype < 0 || x.dim() != 2) refuse("logits must be fp32, bf16 or fp16 [rows][vocab], not " + shape_text(x));
  const int64_t n = x.size(0), vocab = x.size(1);
  a.rows = as_int(n, "logits");
  a.vocab = as_int(vocab, "logits");
  a.logits = dense_rows("logits", x, x.scalar_type(), n, vocab, a.logits_stride);
  if (history) {
    a.history = static_cast<const int*>(dense_rows("history", *history, at::kInt, n, -1, a.history_stride));
    a.history_width = as_int(history->size(1), "history");
    const void *l = array("history_lens", lens, at::kInt, n), *p = array("prompt_lens", prompts, at::kInt, n),
               *r = array("repetition", rep, at::kFloat, n), *f = array("frequency", freq, at::kFloat, n),
               *s = array("presence", pres, at::kFloat, n);
    if (a.history) {  // (a history without columns has no address)
      a.history_lens = static_cast<const int*>(l);
      a.prompt_lens = static_cast<const int*>(p);
      a.repetition = static_cast<const float*>(r);
      a.frequency = static_cast<const float*>(f);
      a.presence = static_cast<const float*>(s);
    }
  } else if (lens || prompts || rep || freq || pres) {
    refuse("penalties and history lengths need a history");
  }
  if (indptr || ids || values) {
    if (!indptr || !ids || !values) refuse("bias must be (indptr, ids, values)");
    const int64_t count = ids->numel();
    const void *p = array("bias indptr", indptr, at::kInt, n + 1), *i = array("bias ids", ids, at::kInt, count),
               *v = array("bias values", values, at::kFloat, count);
    if (count) {
      a.bias_indptr = static_cast<const int*>(p);
      a.bias_ids = static_cast<const int*>(i);
      a.bias_values = static_cast<const float*>(v);
      a.bias_count = as_int(count, "bias");
    }
  }
  if (mask) {
    const int64_t m = mask->dim() == 2 && mask->size(0) == 1 ? 1 : n;
    long long stride = 0;
    a.mask = static_cast<const unsigned*>(dense_rows("mask", *mask, at::kInt, m, (vocab + 31) / 32, stride));
    a.mask_stride = m > 1 ? stride : 0;
  }
  a.status = static_cast<int*>(array("status", status, at::kInt, 1));
  Place place(x, {history, lens, prompts, rep, freq, pres, indptr, ids, values, mask, given_out, given_next, status}, o[14]);
  const at::Tensor out = given_out ? *given_out : at::empty({n, vocab}, x.options().dtype(at::kFloat));
  const at::Tensor next = given_next ? *given_next : at::empty({n}, x.options().dtype(at::kInt));
  a.out = static_cast<float*>(dense_rows("out", out, at::kFloat, n, vocab, a.out_stride));
  a.next_tokens = static_cast<int*>(array("next_tokens", &next, at::kInt, n));
  done(abi.logits(&a, place.raw));
  PyObject* pair = PyTuple_New(2);
  PyTuple_SET_ITEM(pair, 0, result(o[11], out));
  PyTuple_SET_ITEM(pair, 1, result(o[12], next));
  return pair;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, not %zd", N, n);
    return nullptr;
  }
  if (!abi.error) {
    PyErr_SetString(PyExc_RuntimeError, "init has not been called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refusal& r) {
    PyObject* e = PyObject_CallFunction(abi.error, "is", r.status, r.what.c_str());
    if (e) {
      PyErr_SetObject(abi.error, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// (MkError, addresses of mk_append_kv, mk_prompt_attention,
// mk_prompt_attention_workspace_bytes, mk_paged_attention,
// mk_paged_attention_workspace_bytes, mk_process_logits, mk_last_error)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* f[7];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "init takes the error class and seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  abi.append = reinterpret_cast<decltype(abi.append)>(f[0]);
  abi.prompt = reinterpret_cast<decltype(abi.prompt)>(f[1]);
  abi.prompt_bytes = reinterpret_cast<decltype(abi.prompt_bytes)>(f[2]);
  abi.paged = reinterpret_cast<decltype(abi.paged)>(f[3]);
  abi.paged_bytes = reinterpret_cast<decltype(abi.paged_bytes)>(f[4]);
  abi.logits = reinterpret_cast<decltype(abi.logits)>(f[5]);
  abi.last_error = reinterpret_cast<decltype(abi.last_error)>(f[6]);
  Py_XDECREF(abi.error);
  abi.error = Py_NewRef(args[0]);
  Py_RETURN_NONE;
}

#define MK_METHOD(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"init", MK_METHOD(init), METH_FASTCALL, nullptr},
    {"append_kv", MK_METHOD((call<append, 12>)), METH_FASTCALL, nullptr},
    {"prompt_attention", MK_METHOD((call<prompt, 13>)), METH_FASTCALL, nullptr},
    {"paged_attention", MK_METHOD((call<paged, 10>)), METH_FASTCALL, nullptr},
    {"process_logits", MK_METHOD((call<logits, 15>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
