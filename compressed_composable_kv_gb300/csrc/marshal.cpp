// Arguments of the paged calls and of the token log probabilities, from torch
// tensors to the C ABI: every tensor's type, shape, contiguity and device are
// checked, then the C function is called and its status returned.
//
// In Python the same checks take 6 to 10 us a call, as long as the kernels of a
// small decode step; here they take a few hundred nanoseconds.  The stream and
// the current device are the caller's business (binding.py).
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <vector>

#include "c2kv.h"

namespace {

struct Bad : std::runtime_error {
  using std::runtime_error::runtime_error;
};

struct Item {   // a new reference
  PyObject* o;
  ~Item() { Py_XDECREF(o); }
};

int64_t as_int(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Bad("");   // the Python error is set
  return v;
}

int32_t as_int32(PyObject* o, const char* name) {
  const int64_t v = as_int(o);
  if (v < INT32_MIN || v > INT32_MAX) throw Bad(std::string(name) + " is out of range");
  return (int32_t)v;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

std::string form(at::ScalarType type, at::IntArrayRef sizes) {
  std::string s = std::string(c10::toString(type)) + " (";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + ")";
}

void on_device(const at::Tensor& t, int64_t dev, const char* name) {
  if (!t.is_cuda() || t.get_device() != dev)
    throw Bad(std::string(name) + " must be on the current CUDA device, like the call's other tensors");
}

// The address of a contiguous tensor of this type and shape on device dev.
void* address(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t dev) {
  const at::Tensor& t = tensor(o, name);
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.scalar_type() != type || t.sizes() != want || !t.is_contiguous())
    throw Bad(std::string(name) + " must be a contiguous " + form(type, want) + " tensor, got " +
              form(t.scalar_type(), t.sizes()));
  on_device(t, dev, name);
  return t.data_ptr();
}

void* optional(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t dev) {
  return o == Py_None ? nullptr : address(o, name, type, shape, dev);
}

// A contiguous tensor of any type and shape on device dev: its bytes.
size_t bytes(PyObject* o, const char* name, int64_t dev, void** at) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_contiguous()) throw Bad(std::string(name) + " must be contiguous");
  on_device(t, dev, name);
  *at = t.data_ptr();
  return t.nbytes();
}

// Arguments 0-4 geometry, 5 device, then k8, v8, k_scale, v_scale, page_table.
constexpr int kPagesArgs = 11;
struct Pages {
  c2kv_geometry g;
  c2kv_pages8 pages;
  int64_t dev;
  const int32_t* table;
  int32_t max_pages;

  Pages(PyObject* const* a, int64_t batch) {
    g.n_layers = as_int32(a[0], "n_layers");
    g.n_q_heads = as_int32(a[1], "n_q_heads");
    g.n_kv_heads = as_int32(a[2], "n_kv_heads");
    g.head_dim = as_int32(a[3], "head_dim");
    g.rope_theta = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) throw Bad("");
    dev = as_int(a[5]);
    const at::Tensor& k8 = tensor(a[6], "k8");
    if (k8.dim() != 5) throw Bad("k8 must be [n_layers][n_pages][n_kv_heads][page][head_dim]");
    const int64_t n = k8.size(1), page = k8.size(3);
    const auto e4m3 = at::kFloat8_e4m3fn;
    pages.k = address(a[6], "k8", e4m3, {g.n_layers, n, g.n_kv_heads, page, g.head_dim}, dev);
    pages.v = address(a[7], "v8", e4m3, {g.n_layers, n, g.n_kv_heads, page, g.head_dim}, dev);
    pages.k_scale = (float*)address(a[8], "k_scale", at::kFloat, {g.n_layers, n, g.n_kv_heads}, dev);
    pages.v_scale = (float*)address(a[9], "v_scale", at::kFloat, {g.n_layers, n, g.n_kv_heads}, dev);
    if (n > INT32_MAX || page > INT32_MAX) throw Bad("k8 has too many pages");
    pages.n_pages = (int32_t)n;
    pages.page = (int32_t)page;
    const at::Tensor& t = tensor(a[10], "page_table");
    if (t.dim() != 2 || t.size(1) > INT32_MAX) throw Bad("page_table must be [batch][max_pages]");
    max_pages = (int32_t)t.size(1);
    table = (const int32_t*)address(a[10], "page_table", at::kInt, {batch, max_pages}, dev);
  }

  // A RoPE table of any type: its rows.
  int32_t rope_rows(PyObject* o, void** at) const {
    const size_t n = bytes(o, "rope_table", dev, at);
    const size_t row = (size_t)(g.head_dim > 1 ? g.head_dim / 2 : 1) * 16;
    return (int32_t)std::min<size_t>(n / row, INT32_MAX);
  }
};

PyObject* status(c2kv_status s) { return PyLong_FromLong(s); }

template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& f) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", have, want);
    return nullptr;
  }
  try {
    return f();
  } catch (const Bad& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// pages8_fill(pages..., k_caches, v_caches, cap, n_rows, layer_begin, layer_end, stream)
PyObject* pages8_fill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, kPagesArgs + 7, [&]() -> PyObject* {
    PyObject* const* r = a + kPagesArgs;
    const Py_ssize_t batch = PySequence_Size(r[0]);
    if (batch < 0 || PySequence_Size(r[1]) != batch || PySequence_Size(r[3]) != batch)
      throw Bad(PyErr_Occurred() ? "" : "k_caches, v_caches and n_rows need one entry per sequence");
    const Pages p(a, batch);
    const int32_t cap = as_int32(r[2], "cap");
    const int64_t need = (int64_t)p.g.n_layers * p.g.n_kv_heads * (cap > 0 ? cap : 0) * p.g.head_dim;
    std::vector<void*> at(2 * batch + 1);
    std::vector<int32_t> rows(batch + 1);
    for (int kv = 0; kv < 2; ++kv)
      for (Py_ssize_t b = 0; b < batch; ++b) {
        const Item item{PySequence_GetItem(r[kv], b)};
        if (!item.o) throw Bad("");
        const char* name = kv == 0 ? "k_caches" : "v_caches";
        const at::Tensor& t = tensor(item.o, name);
        if (t.scalar_type() != at::kBFloat16 || t.numel() < need || !t.is_contiguous())
          throw Bad(std::string(name) + "[" + std::to_string(b) + "] must be a contiguous bfloat16 tensor of at least " +
                    std::to_string(need) + " elements, got " + form(t.scalar_type(), t.sizes()));
        on_device(t, p.dev, name);
        at[kv * batch + b] = t.data_ptr();
      }
    for (Py_ssize_t b = 0; b < batch; ++b) {
      const Item item{PySequence_GetItem(r[3], b)};
      if (!item.o) throw Bad("");
      rows[b] = as_int32(item.o, "n_rows");
    }
    return status(c2kv_pages8_fill(&p.g, &p.pages, as_int32(r[4], "layer_begin"), as_int32(r[5], "layer_end"),
                                   (int32_t)batch, at.data(), at.data() + batch, cap, rows.data(), p.table,
                                   p.max_pages, (void*)as_int(r[6])));
  });
}

// pages8_append(pages..., layer, n_cached, n_new, k_new, v_new, rope_table, rope_row, stream)
PyObject* pages8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, kPagesArgs + 8, [&]() -> PyObject* {
    PyObject* const* r = a + kPagesArgs;
    const at::Tensor& k = tensor(r[3], "k_new");
    if (k.dim() != 4) throw Bad("k_new must be [batch][t_len][n_kv_heads][head_dim]");
    const int64_t batch = k.size(0), t_len = k.size(1);
    if (batch > INT32_MAX || t_len > INT32_MAX) throw Bad("k_new has too many tokens");
    const Pages p(a, batch);
    const int64_t h = p.g.n_kv_heads, d = p.g.head_dim;
    void* rope;
    const int32_t rows = p.rope_rows(r[5], &rope);
    return status(c2kv_pages8_append(
        &p.g, &p.pages, as_int32(r[0], "layer"), (int32_t)batch, (int32_t)t_len, p.table, p.max_pages,
        (const int32_t*)address(r[1], "n_cached_dev", at::kInt, {batch}, p.dev),
        (const int32_t*)optional(r[2], "n_new_dev", at::kInt, {batch}, p.dev),
        address(r[3], "k_new", at::kBFloat16, {batch, t_len, h, d}, p.dev),
        address(r[4], "v_new", at::kBFloat16, {batch, t_len, h, d}, p.dev), rope, rows,
        (const int32_t*)address(r[6], "rope_row_dev", at::kInt, {batch}, p.dev), (void*)as_int(r[7])));
  });
}

// attend_pages8(pages..., layer, n_cached, max_keys, q, k_new, v_new, rope_table, rope_row, out, workspace, flags, stream)
PyObject* attend_pages8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, kPagesArgs + 12, [&]() -> PyObject* {
    PyObject* const* r = a + kPagesArgs;
    const at::Tensor& q = tensor(r[3], "q");
    if (q.dim() != 3 || q.size(0) > INT32_MAX) throw Bad("q must be [batch][n_q_heads][head_dim]");
    const int64_t batch = q.size(0);
    const Pages p(a, batch);
    const int64_t hq = p.g.n_q_heads, h = p.g.n_kv_heads, d = p.g.head_dim;
    void *rope, *ws;
    const int32_t rows = p.rope_rows(r[6], &rope);
    const size_t ws_bytes = bytes(r[9], "workspace", p.dev, &ws);
    return status(c2kv_attend_pages8(
        &p.g, &p.pages, as_int32(r[0], "layer"), (int32_t)batch, p.table, p.max_pages,
        (const int32_t*)address(r[1], "n_cached_dev", at::kInt, {batch}, p.dev), as_int32(r[2], "max_keys"),
        address(r[3], "q", at::kBFloat16, {batch, hq, d}, p.dev),
        optional(r[4], "k_new", at::kBFloat16, {batch, h, d}, p.dev),
        optional(r[5], "v_new", at::kBFloat16, {batch, h, d}, p.dev), rope, rows,
        (const int32_t*)address(r[7], "rope_row_dev", at::kInt, {batch}, p.dev),
        address(r[8], "out", at::kBFloat16, {batch, hq, d}, p.dev), ws, ws_bytes, (uint32_t)as_int32(r[10], "flags"),
        (void*)as_int(r[11])));
  });
}

// token_logprobs(device, logits, tokens, top_k, logprob, entropy, top_ids, top_logprobs, stream)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int64_t dev = as_int(a[0]);
    const at::Tensor& x = tensor(a[1], "logits");
    if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1))
      throw Bad("logits must be [rows][vocab] with neighbouring logits of a row side by side");
    const bool f32 = x.scalar_type() == at::kFloat;
    if (!f32 && x.scalar_type() != at::kBFloat16)
      throw Bad("logits must be bfloat16 or float32, got " + form(x.scalar_type(), x.sizes()));
    on_device(x, dev, "logits");
    const int64_t rows = x.size(0), vocab = x.size(1), k = as_int(a[3]);
    if (rows > INT32_MAX || vocab > INT32_MAX || k < INT32_MIN || k > INT32_MAX) throw Bad("logits are too large");
    return status(c2kv_token_logprobs(
        x.data_ptr(), f32 ? C2KV_F32 : C2KV_BF16, (int32_t)rows, (int32_t)vocab,
        rows > 1 ? x.stride(0) : std::max(vocab, x.stride(0)),
        (const int32_t*)optional(a[2], "tokens", at::kInt, {rows}, dev), (int32_t)k,
        (float*)optional(a[4], "logprob", at::kFloat, {rows}, dev),
        (float*)optional(a[5], "entropy", at::kFloat, {rows}, dev),
        (int32_t*)optional(a[6], "top_ids", at::kInt, {rows, k}, dev),
        (float*)optional(a[7], "top_logprobs", at::kFloat, {rows, k}, dev), (void*)as_int(a[8])));
  });
}

PyMethodDef methods[] = {
    {"pages8_fill", (PyCFunction)(void (*)(void))pages8_fill, METH_FASTCALL, nullptr},
    {"pages8_append", (PyCFunction)(void (*)(void))pages8_append, METH_FASTCALL, nullptr},
    {"attend_pages8", (PyCFunction)(void (*)(void))attend_pages8, METH_FASTCALL, nullptr},
    {"token_logprobs", (PyCFunction)(void (*)(void))token_logprobs, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
