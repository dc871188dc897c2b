// The Python side of include/gqa_paged.h: turns tensors into the pointers, sizes
// and strides of the C functions and calls them.
//
// A step of drafted tokens is four calls, each of a few microseconds on the GPU.
// Marshalled in Python (some 60 attributes of tensors a call, and ctypes), such a
// step took 37 us on the host for 15 us of kernels.  Only marshalling and the
// checks of tensors are here; what the C functions check is left to them, and
// their status is returned.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/gqa_paged.h"

namespace {

using at::Tensor;
using at::IntArrayRef;

// The functions of the loaded library, by use().
struct {
  decltype(&gqa_rotary_apply) rotary_apply;
  decltype(&gqa_paged_append) paged_append;
  decltype(&gqa_tree_from_parents) tree_from_parents;
  decltype(&gqa_tree_workspace_size) tree_workspace_size;
  decltype(&gqa_tree_attn) tree_attn;
  decltype(&gqa_paged_keep) paged_keep;
} c_api;

[[noreturn]] void refuse(const std::string& why) { throw std::invalid_argument(why); }

// A Python exception is set already.
struct PythonError {};

// ------------------------------------------------------------- arguments
const Tensor* tensor_or_none(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %s", what, Py_TYPE(o)->tp_name);
    throw PythonError{};
  }
  return &THPVariable_Unpack(o);
}

const Tensor& tensor(PyObject* o, const char* what) {
  const Tensor* t = tensor_or_none(o, what);
  if (t == nullptr) refuse(std::string(what) + " must be a tensor");
  return *t;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}

int as_int(int64_t v, const char* what) {
  if (v < INT_MIN || v > INT_MAX) refuse(std::string(what) + " is out of range");
  return static_cast<int>(v);
}

int device_of(const Tensor& t, const char* what) {
  if (!t.is_cuda()) refuse(std::string(what) + " must be a CUDA tensor");
  return static_cast<int>(t.get_device());
}

bool on(const Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

std::string shape_text(IntArrayRef shape) {
  std::ostringstream s;
  s << shape;
  return s.str();
}

// The address of a contiguous tensor of this type and shape on the call's device.
void* whole(const Tensor& t, const char* what, int device, at::ScalarType type, IntArrayRef shape) {
  if (t.scalar_type() != type || t.sizes() != shape || !on(t, device) || !t.is_contiguous()) {
    std::ostringstream s;
    s << what << " must be contiguous " << at::toString(type) << " " << shape << " on the call's CUDA device";
    refuse(s.str());
  }
  return t.data_ptr();
}

int32_t* ints(const Tensor* t, const char* what, int device, IntArrayRef shape) {
  return t == nullptr ? nullptr : static_cast<int32_t*>(whole(*t, what, device, at::kInt, shape));
}

int32_t* ints(PyObject* o, const char* what, int device, IntArrayRef shape) {
  return ints(&tensor(o, what), what, device, shape);
}

int32_t* ints_or_none(PyObject* o, const char* what, int device, IntArrayRef shape) {
  return ints(tensor_or_none(o, what), what, device, shape);
}

int type_code(at::ScalarType t, bool fp32) {
  if (t == at::kBFloat16) return GQA_DTYPE_BF16;
  if (t == at::kHalf) return GQA_DTYPE_FP16;
  if (t == at::kFloat && fp32) return GQA_DTYPE_FP32;
  refuse(std::string("unsupported dtype ") + at::toString(t));
}

// Elements from token to token of t [..., tokens, heads, d]: dense heads, one
// stride for all tokens.
int64_t token_stride(const Tensor& t, const char* what) {
  const IntArrayRef sizes = t.sizes(), strides = t.strides();
  const size_t n = sizes.size();
  const int64_t heads = sizes[n - 2], d = sizes[n - 1];
  if ((d > 1 && strides[n - 1] != 1) || (heads > 1 && strides[n - 2] != d))
    refuse(std::string(what) + " must have dense heads");
  if (t.numel() == 0) return heads * d;  // no token is reached by any
  int64_t stride = -1, run = 1;  // from the last token dimension outwards
  for (size_t i = n - 2; i-- > 0;) {
    if (sizes[i] == 1) continue;
    if (stride < 0) stride = strides[i];
    else if (strides[i] != stride * run) refuse(std::string(what) + " must have one stride from token to token");
    run *= sizes[i];
  }
  return stride < 0 ? heads * d : stride;
}

gqa_rotary_t rotary(const Tensor& turns, int device, PyObject* interleaved, PyObject* inverse, PyObject* magnitude) {
  if (turns.scalar_type() != at::kLong || turns.dim() != 1 || !on(turns, device) || !turns.is_contiguous())
    refuse("turns (of rotary_turns) must be contiguous int64 [dim / 2] on the call's CUDA device");
  gqa_rotary_t r;
  r.dim = as_int(2 * turns.numel(), "dim");
  r.interleaved = truth(interleaved) ? 1 : 0;
  r.inverse = inverse != nullptr && truth(inverse) ? 1 : 0;
  r.magnitude = static_cast<float>(real(magnitude));
  return r;
}

// A batch and its caches [pages, page_size, kv_heads, d], of any strides but the
// last.
struct Paged {
  gqa_desc_t desc;
  gqa_pages_t pages;
  const int32_t* table;
};

Paged describe(int64_t batch, int64_t tokens, int64_t q_heads, int64_t d, at::ScalarType type, const Tensor& cache,
               const Tensor& table, int out_code, int device) {
  if (cache.dim() != 4 || cache.size(3) != d || cache.stride(3) != 1)
    refuse("the caches must be [pages, page_size, kv_heads, " + std::to_string(d) + "] with dense heads, not " +
           shape_text(cache.sizes()));
  if (cache.scalar_type() != type || !on(cache, device))
    refuse("the caches must be of the inputs' type and on their device");
  if (table.dim() != 2 || table.size(0) != batch || table.scalar_type() != at::kInt || !on(table, device) ||
      !table.is_contiguous())
    refuse("page_table must be contiguous int32 [" + std::to_string(batch) +
           ", pages of a sequence] on the call's CUDA device");
  Paged p;
  const int64_t size = cache.size(1);
  auto stride = [&](int i) { return cache.size(i) > 1 ? cache.stride(i) : d; };  // (of one element: not used)
  p.pages.num_pages = as_int(cache.size(0), "pages");
  p.pages.page_size = as_int(size, "page_size");
  p.pages.max_pages = as_int(table.size(1), "pages of a sequence");
  p.pages.page_stride = stride(0);
  p.pages.pos_stride = stride(1);
  p.pages.head_stride = stride(2);
  const int64_t most = table.size(1) * size;
  p.desc.batch = as_int(batch, "batch");
  p.desc.q_tokens = as_int(tokens, "tokens");
  p.desc.q_heads = as_int(q_heads, "q_heads");
  p.desc.kv_heads = as_int(cache.size(2), "kv_heads");
  p.desc.head_dim = as_int(d, "head_dim");
  p.desc.max_seqlen = static_cast<int>(most < (1 << 30) ? most : (1 << 30));
  p.desc.scale = 0.f;
  p.desc.causal = 0;
  p.desc.in_dtype = type_code(type, false);
  p.desc.out_dtype = out_code < 0 ? p.desc.in_dtype : out_code;
  p.desc.reduction = GQA_REDUCE_AUTO;
  p.table = static_cast<const int32_t*>(table.data_ptr());
  return p;
}

void alike(const Tensor& k_cache, const Tensor& v_cache) {
  if (v_cache.scalar_type() != k_cache.scalar_type() || v_cache.sizes() != k_cache.sizes() ||
      v_cache.strides() != k_cache.strides() || v_cache.device() != k_cache.device())
    refuse("the caches must be alike in type, shape and strides, and on one device");
}

// ------------------------------------------------------------------ calls
// f(stream) on `device`, without the interpreter's lock; its status.
template <typename F>
PyObject* launch(int device, PyObject* stream, const F& f) {
  void* raw = stream == Py_None ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(
                                      static_cast<c10::DeviceIndex>(device)).stream())
                                : reinterpret_cast<void*>(static_cast<uintptr_t>(integer(stream)));
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  gqa_status_t rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(raw);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

PyObject* rotary_apply(PyObject* const* a) {
  const Tensor &x = tensor(a[0], "x"), &positions = tensor(a[1], "positions"), &turns = tensor(a[2], "turns"),
               &out = tensor(a[3], "out");
  const int device = device_of(x, "x");
  const int64_t n = x.dim();
  if (n < 3 || out.scalar_type() != x.scalar_type() || out.sizes() != x.sizes() || !on(out, device))
    refuse("x must be [..., heads, d], and out of its type and shape and on its device");
  const int32_t* at = ints(&positions, "positions", device, x.sizes().slice(0, n - 2));
  const gqa_rotary_t rope = rotary(turns, device, a[4], a[5], a[6]);
  const int heads = as_int(x.size(n - 2), "heads"), d = as_int(x.size(n - 1), "head_dim");
  const int code = type_code(x.scalar_type(), true);
  const int64_t tokens = positions.numel(), from = token_stride(x, "x"), to = token_stride(out, "out");
  const void* src = x.data_ptr();
  void* dst = out.data_ptr();
  const uint64_t* table = static_cast<const uint64_t*>(turns.data_ptr());
  return launch(device, a[7], [&](void* s) {
    return c_api.rotary_apply(&rope, table, at, tokens, heads, d, code, src, from, dst, to, s);
  });
}

PyObject* paged_append(PyObject* const* a) {
  const Tensor *q = tensor_or_none(a[0], "q"), *q_out = tensor_or_none(a[3], "q_out"),
               *turns = tensor_or_none(a[10], "turns");
  const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &k_cache = tensor(a[4], "k_cache"),
               &v_cache = tensor(a[5], "v_cache"), &table = tensor(a[6], "page_table");
  const int device = device_of(k, "k");
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || !on(v, device))
    refuse("k and v must be [B, nq, kv_heads, d], of one type and device");
  if ((q == nullptr) != (q_out == nullptr)) refuse("q and q_out come together");
  if (q != nullptr && q->dim() != 4) refuse("q must be [B, nq, q_heads, d]");
  const int64_t B = k.size(0), nq = k.size(1), d = k.size(3), heads = q == nullptr ? k.size(2) : q->size(2);
  const Paged p = describe(B, nq, heads, d, k.scalar_type(), k_cache, table, -1, device);
  alike(k_cache, v_cache);
  if (k_cache.size(2) != k.size(2))
    refuse("k " + shape_text(k.sizes()) + " and cache " + shape_text(k_cache.sizes()) + " disagree");
  const int64_t batch[1] = {B}, tokens[2] = {B, nq}, rows[4] = {B, nq, heads, d};
  const int32_t* lens = ints(a[7], "seqlens", device, batch);
  const int32_t* news = ints_or_none(a[8], "new_lens", device, batch);
  const int32_t* positions = ints_or_none(a[9], "positions", device, tokens);
  const void *q_at = nullptr, *k_at = k.data_ptr(), *v_at = v.data_ptr();
  void* q_to = nullptr;
  int64_t q_stride = 0;
  if (q != nullptr) {
    if (q->sizes() != IntArrayRef(rows) || q->scalar_type() != k.scalar_type() || !on(*q, device))
      refuse("q must be [B, nq, q_heads, d], of k's type and on its device");
    q_to = whole(*q_out, "q_out", device, k.scalar_type(), rows);
    q_at = q->data_ptr();
    q_stride = token_stride(*q, "q");
  }
  gqa_rotary_t rope;
  const uint64_t* turn = nullptr;
  if (turns != nullptr) {
    rope = rotary(*turns, device, a[11], nullptr, a[12]);
    turn = static_cast<const uint64_t*>(turns->data_ptr());
  }
  const int64_t k_stride = token_stride(k, "k"), v_stride = token_stride(v, "v");
  void *kc = k_cache.data_ptr(), *vc = v_cache.data_ptr();
  return launch(device, a[13], [&](void* s) {
    return c_api.paged_append(&p.desc, &p.pages, turn == nullptr ? nullptr : &rope, turn, positions, q_at, q_stride, k_at,
                              k_stride, v_at, v_stride, q_to, kc, vc, p.table, lens, news, s);
  });
}

PyObject* tree_from_parents(PyObject* const* a) {
  const Tensor& parents = tensor(a[0], "parents");
  const int device = device_of(parents, "parents");
  if (parents.dim() != 2) refuse("parents must be [B, nq]");
  const int64_t B = parents.size(0), nq = parents.size(1);
  const int64_t batch[1] = {B}, tokens[2] = {B, nq}, bits[3] = {B, nq, (nq + 31) / 32};
  const int32_t* up = ints(&parents, "parents", device, tokens);
  const int32_t* lens = ints(a[1], "seqlens", device, batch);
  uint32_t* tree = reinterpret_cast<uint32_t*>(ints(a[2], "tree", device, bits));
  int32_t* positions = ints_or_none(a[3], "positions", device, tokens);
  const int32_t* news = ints_or_none(a[4], "new_lens", device, batch);
  const int b = as_int(B, "batch"), n = as_int(nq, "tokens"), most = as_int(integer(a[5]), "max_seqlen");
  return launch(device, a[6], [&](void* s) {
    return c_api.tree_from_parents(b, n, most, up, lens, news, tree, positions, s);
  });
}

PyObject* tree_workspace_size(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "k_cache"), &table = tensor(a[2], "page_table");
  const int device = device_of(q, "q");
  if (q.dim() != 4) refuse("q must be [B, nq, q_heads, d]");
  const Paged p = describe(q.size(0), q.size(1), q.size(2), q.size(3), q.scalar_type(), cache, table,
                           as_int(integer(a[3]), "out_dtype"), device);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  return PyLong_FromSize_t(c_api.tree_workspace_size(&p.desc, &p.pages));
}

PyObject* tree_attn(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k_cache = tensor(a[1], "k_cache"), &v_cache = tensor(a[2], "v_cache"),
               &table = tensor(a[3], "page_table"), &out = tensor(a[5], "out");
  const Tensor *lse = tensor_or_none(a[6], "lse"), *workspace = tensor_or_none(a[7], "workspace");
  const int device = device_of(q, "q");
  if (q.dim() != 4) refuse("q must be [B, nq, q_heads, d]");
  const int64_t B = q.size(0), nq = q.size(1), heads = q.size(2);
  Paged p = describe(B, nq, heads, q.size(3), q.scalar_type(), k_cache, table, type_code(out.scalar_type(), true), device);
  alike(k_cache, v_cache);
  p.desc.causal = truth(a[10]) ? 1 : 0;
  p.desc.scale = static_cast<float>(real(a[11]));
  const int64_t batch[1] = {B}, rows[3] = {B, nq, heads}, bits[3] = {B, nq, (nq + 31) / 32};
  const int32_t* lens = ints(a[4], "seqlens", device, batch);
  const int32_t* news = ints_or_none(a[8], "new_lens", device, batch);
  const uint32_t* tree = reinterpret_cast<const uint32_t*>(ints_or_none(a[9], "tree", device, bits));
  const void* q_at = whole(q, "q", device, q.scalar_type(), q.sizes());
  void* o = whole(out, "out", device, out.scalar_type(), q.sizes());
  float* l = lse == nullptr ? nullptr : static_cast<float*>(whole(*lse, "lse", device, at::kFloat, rows));
  void* ws = workspace == nullptr ? nullptr
                                  : whole(*workspace, "workspace", device, workspace->scalar_type(), workspace->sizes());
  const size_t ws_bytes = workspace == nullptr ? 0 : workspace->nbytes();
  const void *kc = k_cache.data_ptr(), *vc = v_cache.data_ptr();
  return launch(device, a[12], [&](void* s) {
    return c_api.tree_attn(&p.desc, &p.pages, q_at, kc, vc, p.table, lens, news, tree, o, l, ws, ws_bytes, s);
  });
}

PyObject* paged_keep(PyObject* const* a) {
  const Tensor &k_cache = tensor(a[0], "k_cache"), &v_cache = tensor(a[1], "v_cache"), &table = tensor(a[2], "page_table"),
               &path = tensor(a[4], "path");
  const int device = device_of(k_cache, "k_cache");
  if (path.dim() != 2 || k_cache.dim() != 4)
    refuse("path must be [B, n], and the caches [pages, page_size, kv_heads, d]");
  const int64_t B = path.size(0), batch[1] = {B};
  const Paged p = describe(B, integer(a[8]), k_cache.size(2), k_cache.size(3), k_cache.scalar_type(), k_cache, table, -1,
                           device);
  alike(k_cache, v_cache);
  const int32_t* lens = ints(a[3], "seqlens", device, batch);
  const int32_t* branch = ints(&path, "path", device, path.sizes());
  const int32_t* keep = ints(a[5], "keep_lens", device, batch);
  int32_t* lens_out = ints_or_none(a[6], "seqlens_out", device, batch);
  const int32_t* news = ints_or_none(a[7], "new_lens", device, batch);
  const int most = as_int(path.size(1), "path");
  void *kc = k_cache.data_ptr(), *vc = v_cache.data_ptr();
  return launch(device, a[9], [&](void* s) {
    return c_api.paged_keep(&p.desc, &p.pages, kc, vc, p.table, lens, news, branch, most, keep, lens_out, s);
  });
}

PyObject* stride_of(PyObject* const* a) {
  const Tensor& t = tensor(a[0], "tensor");
  if (t.dim() < 3) refuse("a tensor [..., heads, d]");
  return PyLong_FromLongLong(token_stride(t, "tensor"));
}

PyObject* use(PyObject* const* a) {
  auto at = [&](int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(integer(a[i]))); };
  c_api.rotary_apply = reinterpret_cast<decltype(c_api.rotary_apply)>(at(0));
  c_api.paged_append = reinterpret_cast<decltype(c_api.paged_append)>(at(1));
  c_api.tree_from_parents = reinterpret_cast<decltype(c_api.tree_from_parents)>(at(2));
  c_api.tree_workspace_size = reinterpret_cast<decltype(c_api.tree_workspace_size)>(at(3));
  c_api.tree_attn = reinterpret_cast<decltype(c_api.tree_attn)>(at(4));
  c_api.paged_keep = reinterpret_cast<decltype(c_api.paged_keep)>(at(5));
  Py_RETURN_NONE;
}

// N arguments by position; what is thrown becomes the Python exception.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are needed, not %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PythonError&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define GQA_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<&f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GQA_ENTRY(use, 6),
                         GQA_ENTRY(rotary_apply, 8),
                         GQA_ENTRY(paged_append, 14),
                         GQA_ENTRY(tree_from_parents, 7),
                         GQA_ENTRY(tree_workspace_size, 4),
                         GQA_ENTRY(tree_attn, 13),
                         GQA_ENTRY(paged_keep, 10),
                         GQA_ENTRY(stride_of, 1),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
