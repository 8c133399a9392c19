// Python module _qknorm_torch: torch tensors into the descriptors of
// libqknorm.so for the operators around headwise QK-Norm. Argument checks and
// marshalling only, in C++ because a decode step's kernels take a few
// microseconds: read attribute by attribute from Python, the tensors of one
// call cost more host time than its kernels take on the GPU (11 to 20 us of host
// time a call, 5 to 9 this way).
//
// Each call takes its arguments by position and ends in one call of the C ABI
// on the given stream, whose status it returns (0: done), or, with `keep`, in
// an object that holds the marshalled call and its tensors for launch().

#include <Python.h>

#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <string>
#include <vector>

#include "qknorm.h"

namespace {

struct Refused {
  PyObject* type;
  std::string text;
};

[[noreturn]] void refuse(const std::string& text) { throw Refused{PyExc_ValueError, text}; }
[[noreturn]] void refuse_type(const std::string& text) { throw Refused{PyExc_TypeError, text}; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

// A marshalled call: descriptors, and the tensors that their pointers lead to.
struct Call {
  enum Kind { ROPE, GRAD, APPEND, ATTEND } kind;
  qknorm_operand_t q{}, k{}, v{};
  qknorm_grad_operand_t gq{}, gk{};
  qknorm_rope_t rope{};
  bool has_q = true, has_rope = false;
  qknorm_cache_t cache{};
  qknorm_batch_t batch{};
  int64_t T = 0, head_dim = 0, gstride = 0, window = 0;
  int dtype = 0, causal = 0;
  float eps = 0.0f, scale = 0.0f;
  const int64_t* slots = nullptr;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  std::vector<at::Tensor> held;

  int run(void* stream) const {
    const qknorm_rope_t* r = has_rope ? &rope : nullptr;
    switch (kind) {
      case ROPE: return qknorm_headwise_rope(&q, &k, T, dtype, eps, head_dim, gstride, r, stream);
      case GRAD:
        return qknorm_headwise_rope_backward(&gq, &gk, T, dtype, eps, head_dim, gstride, r, ws, ws_bytes, stream);
      case APPEND:
        return qknorm_paged_append(has_q ? &q : nullptr, &k, &v, T, dtype, eps, head_dim, gstride, r, &cache, slots,
                                   stream);
      default:
        return qknorm_paged_attend(&q, T, dtype, &cache, head_dim, &batch, scale, causal, window, ws, ws_bytes,
                                   stream);
    }
  }
};

// ------------------------------------------------------------------ arguments
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse(std::string(name) + " is required");
  return *t;
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type(std::string(name) + " must be an integer");
  }
  return v;
}
double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type(std::string(name) + " must be a number");
  }
  return v;
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse_type(std::string(name) + " must be true or false");
  }
  return v != 0;
}

// ------------------------------------------------------------------- tensors
void on_device(const at::Tensor& t, const at::Tensor& ref, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a device tensor");
  if (t.get_device() != ref.get_device())
    refuse(std::string(name) + " is on device " + std::to_string(t.get_device()) + ", the rows on device " +
           std::to_string(ref.get_device()));
}

int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return QKNORM_F32;
    case at::kBFloat16: return QKNORM_BF16;
    case at::kFloat8_e4m3fn: return QKNORM_FP8_E4M3;
    default: refuse_type("unsupported dtype (bfloat16, float32 or float8_e4m3fn)");
  }
}

// Row stride of a 2-D tensor of rows with contiguous columns.
int64_t rows(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(std::string(name) + " must be 2-D [T, h], got " + shape_of(t));
  if (t.size(1) > 1 && t.stride(1) != 1) refuse(std::string(name) + " columns must be contiguous (stride(1) == 1)");
  if (!t.is_cuda()) refuse(std::string(name) + " must be a device tensor");
  // one-row (or empty) views can carry any stride(0); the row length is a valid one
  return t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}
int64_t like(const at::Tensor& y, const at::Tensor& x, const char* name) {
  if (y.sizes() != x.sizes() || y.scalar_type() != x.scalar_type())
    refuse(std::string(name) + " must have the rows' shape " + shape_of(x) + " and dtype, got " + shape_of(y));
  on_device(y, x, name);
  return rows(y, name);
}
int64_t same_tokens(const at::Tensor& a, const at::Tensor& b) {
  if (a.dim() != 2 || b.dim() != 2 || a.size(0) != b.size(0))
    refuse("the sides must be 2-D with the same number of rows, got " + shape_of(a) + " and " + shape_of(b));
  if (a.scalar_type() != b.scalar_type()) refuse_type("the sides must have the same dtype");
  if (a.device() != b.device()) refuse("the sides must be on the same device");
  return a.size(0);
}
template <class T>
T* vector(const at::Tensor& t, int64_t n, at::ScalarType type, const at::Tensor& ref, const char* name) {
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " vector of " + std::to_string(n) +
           ", got " + c10::toString(t.scalar_type()) + " " + shape_of(t));
  on_device(t, ref, name);
  return static_cast<T*>(t.data_ptr());
}

const void* gamma_of(Call& c, const at::Tensor* g, const at::Tensor& x, const char* name) {
  if (!g) return nullptr;
  const int64_t need = c.head_dim > 0 && c.gstride >= 0 ? (x.size(1) / c.head_dim - 1) * c.gstride + c.head_dim : 0;
  const at::ScalarType type = x.scalar_type() == at::kFloat8_e4m3fn ? at::kBFloat16 : x.scalar_type();
  if (g->dim() != 1 || g->size(0) < need || (g->size(0) > 1 && g->stride(0) != 1) || g->scalar_type() != type)
    refuse(std::string("gamma for ") + name + " must be contiguous, dtype " + c10::toString(type) + ", >= " +
           std::to_string(need) + " elements");
  on_device(*g, x, "gamma");
  c.held.push_back(*g);
  return g->data_ptr();
}

qknorm_operand_t side(Call& c, const at::Tensor& x, const at::Tensor* y, const at::Tensor* gamma, const char* name) {
  qknorm_operand_t o{};
  o.ld_x = rows(x, name);
  o.x = x.data_ptr();
  o.h = x.size(1);
  c.held.push_back(x);
  if (y) {
    o.ld_y = like(*y, x, "output rows");
    o.y = y->data_ptr();
    c.held.push_back(*y);
  }
  o.gamma = gamma_of(c, gamma, x, name);
  return o;
}

void rope_of(Call& c, PyObject* table, PyObject* positions, PyObject* interleaved, const at::Tensor& ref) {
  const at::Tensor* t = tensor(table, "cos_sin");
  if (!t) return;
  if (t->scalar_type() != at::kFloat || t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1))
    refuse("cos_sin must be a float32 table [n_positions, rot_dim] with contiguous rows");
  on_device(*t, ref, "cos_sin");
  const at::Tensor& p = needed(positions, "positions");
  c.has_rope = true;
  c.rope.cos_sin = static_cast<const float*>(t->data_ptr());
  c.rope.n_positions = t->size(0);
  c.rope.rot_dim = t->size(1);
  c.rope.ld = t->size(0) > 1 ? t->stride(0) : std::max(t->stride(0), t->size(1));
  c.rope.positions = vector<int64_t>(p, c.T, at::kLong, ref, "positions");
  c.rope.interleaved = truth(interleaved, "interleaved");
  c.held.push_back(*t);
  c.held.push_back(p);
}

// Strides of a cache's pages, heads and tokens. An axis of length one may carry
// any: what a packed axis would have is taken.
void strides_of(const at::Tensor& t, int64_t inner, int64_t (&s)[3]) {
  s[2] = t.size(2) == 1 ? inner : t.stride(2);
  s[1] = t.size(1) == 1 ? s[2] * t.size(2) : t.stride(1);
  s[0] = t.size(0) == 1 ? std::max(s[1] * t.size(1), s[2] * t.size(2)) : t.stride(0);
}

// A cache of [pages, heads, page_size, head_dim] tensors (any strides, a
// head's row contiguous), or of uint8 codes [.., head_dim / 2] with uint8
// scales [.., head_dim / 32].
void cache_of(Call& c, PyObject* pk, PyObject* pv, PyObject* pks, PyObject* pvs, const at::Tensor& ref) {
  const at::Tensor &k = needed(pk, "k_cache"), &v = needed(pv, "v_cache");
  const at::Tensor *ks = tensor(pks, "k_scales"), *vs = tensor(pvs, "v_scales");
  if (!ks != !vs) refuse("k_scales and v_scales go together");
  const bool four = ks != nullptr;
  const int64_t last = four ? c.head_dim / 2 : c.head_dim;
  const at::ScalarType type = four ? at::kByte : ref.scalar_type();
  for (const at::Tensor* t : {&k, &v}) {
    if (t->dim() != 4 || t->size(3) != last || t->scalar_type() != type || (last > 1 && t->stride(3) != 1))
      refuse("k_cache and v_cache must be " + std::string(c10::toString(type)) + " [pages, heads, page_size, " +
             std::to_string(last) + "] with a contiguous last axis, got " + c10::toString(t->scalar_type()) + " " +
             shape_of(*t));
    on_device(*t, ref, "the cache");
    c.held.push_back(*t);
  }
  int64_t s[3], sv[3];
  strides_of(k, last, s);
  strides_of(v, last, sv);
  if (k.sizes() != v.sizes() || !std::equal(s, s + 3, sv))
    refuse("k_cache and v_cache must have the same shape and strides");
  qknorm_cache_t& o = c.cache;
  o.format = four ? QKNORM_CACHE_MXFP4 : QKNORM_CACHE_ROWS;
  o.k = k.data_ptr();
  o.v = v.data_ptr();
  o.n_pages = k.size(0);
  o.heads = k.size(1);
  o.page_size = k.size(2);
  o.page_stride = s[0];
  o.head_stride = s[1];
  o.token_stride = s[2];
  if (!four) return;
  const int64_t blocks = c.head_dim / 32;
  for (const at::Tensor* t : {ks, vs}) {
    if (t->dim() != 4 || t->size(0) != o.n_pages || t->size(1) != o.heads || t->size(2) != o.page_size ||
        t->size(3) != blocks || t->scalar_type() != at::kByte || (blocks > 1 && t->stride(3) != 1) ||
        (o.page_size > 1 && t->stride(2) != blocks))
      refuse("k_scales and v_scales must be uint8 [pages, heads, page_size, " + std::to_string(blocks) +
             "], a head's tokens packed, got " + shape_of(*t));
    on_device(*t, ref, "the scales");
    c.held.push_back(*t);
  }
  strides_of(*ks, blocks, s);
  strides_of(*vs, blocks, sv);
  if (!std::equal(s, s + 3, sv)) refuse("k_scales and v_scales must have the same strides");
  o.k_scales = ks->data_ptr();
  o.v_scales = vs->data_ptr();
  o.scale_page_stride = s[0];
  o.scale_head_stride = s[1];
}

void workspace_of(Call& c, PyObject* given, size_t need, const at::Tensor& ref) {
  const at::Tensor* t = tensor(given, "workspace");
  if (!t) {
    if (!need) return;
    // from the caching allocator, on the device's current stream: the callers
    // that name another stream, or keep the call, pass memory of their own
    c.held.push_back(at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(ref.device())));
    t = &c.held.back();
  } else {
    if (!t->is_contiguous()) refuse("workspace must be contiguous");
    on_device(*t, ref, "workspace");
    c.held.push_back(*t);
  }
  c.ws = t->data_ptr();
  c.ws_bytes = (size_t)t->nbytes();
}

// ---------------------------------------------------------------------- calls
void make_rope(Call& c, PyObject* const* a) {
  const at::Tensor &q = needed(a[0], "q"), &k = needed(a[1], "k");
  c.kind = Call::ROPE;
  c.T = same_tokens(q, k);
  c.eps = (float)number(a[4], "eps");
  c.head_dim = integer(a[5], "head_dim");
  c.gstride = integer(a[9], "gamma_head_stride");
  const at::Tensor *oq = tensor(a[10], "out_q"), *ok = tensor(a[11], "out_k");
  c.q = side(c, q, oq ? oq : &q, &needed(a[2], "gamma_q"), "q");
  c.k = side(c, k, ok ? ok : &k, &needed(a[3], "gamma_k"), "k");
  rope_of(c, a[6], a[7], a[8], q);
  c.dtype = dtype_code(q);
}

qknorm_grad_operand_t grad_side(Call& c, const at::Tensor& x, PyObject* dy, PyObject* gamma, PyObject* dx,
                                PyObject* dgamma, const char* name) {
  qknorm_grad_operand_t o{};
  const at::Tensor &g = needed(gamma, "gamma"), &d = needed(dy, "dy"), &out = needed(dx, "dx");
  o.ld_x = rows(x, name);
  o.x = x.data_ptr();
  o.h = x.size(1);
  o.ld_dy = like(d, x, "dy");
  o.dy = d.data_ptr();
  o.ld_dx = like(out, x, "dx");
  o.dx = out.data_ptr();
  o.gamma = gamma_of(c, &g, x, name);
  const at::Tensor* w = tensor(dgamma, "dgamma");
  if (w) {
    if (w->scalar_type() != at::kFloat || w->sizes() != g.sizes() || (w->size(0) > 1 && w->stride(0) != 1))
      refuse("dgamma must be contiguous float32 " + shape_of(g));
    on_device(*w, x, "dgamma");
    o.dgamma = static_cast<float*>(w->data_ptr());
    c.held.push_back(*w);
  }
  c.held.push_back(x);
  c.held.push_back(d);
  c.held.push_back(out);
  return o;
}

void make_grad(Call& c, PyObject* const* a) {
  const at::Tensor &q = needed(a[2], "q"), &k = needed(a[3], "k");
  c.kind = Call::GRAD;
  c.T = same_tokens(q, k);
  c.eps = (float)number(a[6], "eps");
  c.head_dim = integer(a[7], "head_dim");
  c.gstride = integer(a[11], "gamma_head_stride");
  c.gq = grad_side(c, q, a[0], a[4], a[12], a[14], "q");
  c.gk = grad_side(c, k, a[1], a[5], a[13], a[15], "k");
  rope_of(c, a[8], a[9], a[10], q);
  c.dtype = dtype_code(q);
  size_t need = 0;
  if (c.gq.dgamma || c.gk.dgamma)
    need = qknorm_headwise_rope_backward_workspace(c.gq.h, c.gk.h, c.T, c.dtype, c.head_dim, c.gstride);
  workspace_of(c, a[16], need, q);
}

void make_append(Call& c, PyObject* const* a) {
  const at::Tensor* q = tensor(a[0], "q");
  const at::Tensor &k = needed(a[1], "k"), &v = needed(a[2], "v");
  c.kind = Call::APPEND;
  c.T = same_tokens(k, v);
  c.eps = (float)number(a[5], "eps");
  c.head_dim = integer(a[6], "head_dim");
  c.gstride = integer(a[15], "gamma_head_stride");
  c.has_q = q != nullptr;
  if (q) {
    same_tokens(*q, k);
    const at::Tensor* oq = tensor(a[16], "out_q");
    c.q = side(c, *q, oq ? oq : q, tensor(a[3], "gamma_q"), "q");
  }
  c.k = side(c, k, tensor(a[17], "out_k"), tensor(a[4], "gamma_k"), "k");
  c.v = side(c, v, tensor(a[18], "out_v"), nullptr, "v");
  cache_of(c, a[9], a[10], a[12], a[13], k);
  rope_of(c, a[7], a[8], a[14], k);
  const at::Tensor& s = needed(a[11], "slots");
  c.slots = vector<int64_t>(s, c.T, at::kLong, k, "slots");
  c.held.push_back(s);
  c.dtype = dtype_code(k);
}

void make_attend(Call& c, PyObject* const* a) {
  const at::Tensor &q = needed(a[0], "q"), &table = needed(a[5], "block_table"), &lens = needed(a[6], "seq_lens");
  const at::Tensor* cu = tensor(a[8], "cu_q");
  c.kind = Call::ATTEND;
  if (a[3] == Py_None || a[4] == Py_None) refuse("k_scales and v_scales are required: the cache is MXFP4");
  c.head_dim = integer(a[7], "head_dim");
  c.q = side(c, q, &needed(a[14], "out"), nullptr, "q");
  c.T = q.size(0);
  cache_of(c, a[1], a[2], a[3], a[4], q);
  if (table.dim() != 2 || table.scalar_type() != at::kInt || (table.size(1) > 1 && table.stride(1) != 1))
    refuse("block_table must be int32 [B, pages] with contiguous rows");
  on_device(table, q, "block_table");
  c.held.push_back(table);
  qknorm_batch_t& b = c.batch;
  b.B = table.size(0);
  b.table_pages = table.size(1);
  b.ld_table = b.B > 1 ? table.stride(0) : std::max(table.stride(0), b.table_pages);
  b.block_table = static_cast<const int32_t*>(table.data_ptr());
  b.seq_lens = vector<int32_t>(lens, b.B, at::kInt, q, "seq_lens");
  c.held.push_back(lens);
  if (cu) {
    b.cu_q = vector<int32_t>(*cu, b.B + 1, at::kInt, q, "cu_q");
    c.held.push_back(*cu);
  }
  const int64_t capacity = b.table_pages * c.cache.page_size;
  b.max_q = !cu ? 1 : a[12] == Py_None ? std::max<int64_t>(c.T, 1) : integer(a[12], "max_q");
  b.max_len = a[13] == Py_None ? capacity : std::min(integer(a[13], "max_len"), capacity);
  c.scale = a[9] == Py_None ? (c.head_dim > 0 ? (float)(1.0 / std::sqrt((double)c.head_dim)) : 0.0f)
                            : (float)number(a[9], "scale");
  c.causal = truth(a[10], "causal");
  c.window = a[11] == Py_None ? 0 : integer(a[11], "window");
  c.dtype = dtype_code(q);
  size_t need = 0;
  if (c.head_dim > 0 && c.cache.heads > 0)
    need = qknorm_paged_attend_workspace(c.T, c.q.h / c.head_dim, c.cache.heads, c.head_dim, b.B, b.max_q, b.max_len);
  workspace_of(c, a[15], need, q);
}

// --------------------------------------------------------------------- module
constexpr const char* kCapsule = "_qknorm_torch.call";
void drop(PyObject* o) { delete static_cast<Call*>(PyCapsule_GetPointer(o, kCapsule)); }

// N arguments of the call, then the stream (an integer handle) and `keep`.
template <void (*MAKE)(Call&, PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N + 2) return PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N + 2, n);
  try {
    auto call = std::make_unique<Call>();
    MAKE(*call, a);
    if (truth(a[N + 1], "keep")) {
      PyObject* o = PyCapsule_New(call.get(), kCapsule, drop);
      if (o) call.release();
      return o;
    }
    return PyLong_FromLong(call->run(reinterpret_cast<void*>((uintptr_t)integer(a[N], "stream"))));
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* launch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2) return PyErr_Format(PyExc_TypeError, "launch(call, stream)");
  const Call* c = static_cast<const Call*>(PyCapsule_GetPointer(a[0], kCapsule));
  if (!c) return nullptr;
  const long long s = PyLong_AsLongLong(a[1]);
  if (s == -1 && PyErr_Occurred()) return nullptr;
  return PyLong_FromLong(c->run(reinterpret_cast<void*>((uintptr_t)s)));
}

PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void*)entry<make_rope, 12>, METH_FASTCALL, nullptr},
    {"rope_backward", (PyCFunction)(void*)entry<make_grad, 17>, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void*)entry<make_append, 19>, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void*)entry<make_attend, 16>, METH_FASTCALL, nullptr},
    {"launch", (PyCFunction)(void*)launch, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qknorm_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__qknorm_torch() { return PyModule_Create(&module); }
