// Native marshalling of the cached speculative step's calls (smp_cache.h and
// smp_spec_verify_probs): torch tensors in, argument checks, one call of the
// C ABI on the current stream.  A step makes several of these calls, each a
// few microseconds of kernel, so the checks run here and not in Python.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "smp.h"
#include "smp_cache.h"

namespace {

PyObject* g_error = nullptr;   // SmpError

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

std::string shape_text(c10::IntArrayRef s) {
  std::string out = "[";
  for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
  return out + "]";
}

using Tensor = at::Tensor;

// The GPU of the call at hand: its first tensor's, which the others must share (-1: none seen yet).
thread_local int g_device = -1;

// The tensor of an argument, or nullptr for None.
const Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  const int device = t.device().index();
  if (g_device < 0) g_device = device;
  if (device != g_device)
    refuse("the tensors of a call must be on one GPU: " + std::string(name) + " is on cuda:" + std::to_string(device) +
           ", the first one on cuda:" + std::to_string(g_device));
  return &t;
}

const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = optional(o, name);
  if (!t) refuse(std::string(name) + " must be a torch tensor");
  return *t;
}

// A contiguous tensor of this type and shape (-1: any size).
void flat(const Tensor& t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
  bool ok = t.scalar_type() == type && size_t(t.dim()) == shape.size() && t.is_contiguous();
  if (ok) {
    size_t i = 0;
    for (const int64_t want : shape) {
      ok &= want < 0 || t.size(int64_t(i)) == want;
      ++i;
    }
  }
  if (!ok) {
    std::string want = "[";
    for (const int64_t s : shape) want += (want.size() > 1 ? ", " : "") + (s < 0 ? std::string("any") : std::to_string(s));
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + want + "], got " +
           c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
  }
}

void* at_of(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
void* at_of(const Tensor& t) { return t.data_ptr(); }

int32_t* status_of(PyObject* o) {
  const Tensor* t = optional(o, "status");
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->numel() < 1 || !t->is_contiguous()) refuse("status must be an int32 [1] tensor");
  return static_cast<int32_t*>(t->data_ptr());
}

int32_t small(int64_t n, const char* name) {
  if (n < 0 || n > 0x7FFFFFFF) refuse(std::string(name) + " is too large");
  return int32_t(n);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused("");
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return int32_t(v);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused("");
  return v;
}

// A torch.cuda.Stream's handle (an int), or None for the current stream of the call's GPU.
void* stream_of(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(g_device)).stream();
  return reinterpret_cast<void*>(uintptr_t(integer(o)));
}

// What every call takes last; with it all tensors have been seen, and their GPU is the current one for the launch.
struct Launch {
  int32_t* status;
  c10::cuda::OptionalCUDAGuard on;   // set where another GPU is current
  void* stream;
  Launch(PyObject* status_arg, PyObject* stream_arg) : status(status_of(status_arg)) {
    if (c10::cuda::current_device() != g_device) on.set_index(c10::DeviceIndex(g_device));
    stream = stream_of(stream_arg);
  }
};

smp_dtype dtype_of(const Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SMP_BF16;
  if (t.scalar_type() == at::kFloat) return SMP_F32;
  refuse(std::string(name) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
}

// The token stride of a [tokens, heads, dim] tensor whose heads are contiguous.
int64_t heads_of(const Tensor& t, const char* name, const Tensor* like = nullptr) {
  if (t.dim() != 3) refuse(std::string(name) + " must be [tokens, heads, dim]");
  dtype_of(t, name);
  if (like && (t.scalar_type() != like->scalar_type() || t.sizes() != like->sizes()))
    refuse(std::string(name) + " must have the type and shape " + shape_text(like->sizes()) + ", got " +
           c10::toString(t.scalar_type()) + " " + shape_text(t.sizes()));
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2), row = h * d;
  if ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d) || (n > 1 && t.stride(0) < row))
    refuse("the heads of " + std::string(name) + " must be contiguous and its tokens in order");
  return n > 1 ? t.stride(0) : row;
}

smp_cache cache_of(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("a cache is a tuple (k, v, k_scale, v_scale)");
  const Tensor& k = tensor(PyTuple_GET_ITEM(o, 0), "k");
  const Tensor& v = tensor(PyTuple_GET_ITEM(o, 1), "v");
  const Tensor& ks = tensor(PyTuple_GET_ITEM(o, 2), "k_scale");
  const Tensor& vs = tensor(PyTuple_GET_ITEM(o, 3), "v_scale");
  if (k.scalar_type() != at::kFloat8_e4m3fn && k.scalar_type() != at::kChar)
    refuse(std::string("cache codes must be float8_e4m3fn or int8, got ") + c10::toString(k.scalar_type()));
  if (k.dim() != 4) refuse("cache codes must be [blocks, kv_heads, block_size, head_dim]");
  const int64_t n = k.size(0), h = k.size(1), bs = k.size(2), d = k.size(3);
  flat(k, "k", k.scalar_type(), {n, h, bs, d});
  flat(v, "v", k.scalar_type(), {n, h, bs, d});
  flat(ks, "k_scale", at::kFloat, {n, h});
  flat(vs, "v_scale", at::kFloat, {n, h});
  smp_cache c;
  c.k = at_of(k), c.v = at_of(v);
  c.k_scale = static_cast<float*>(at_of(ks)), c.v_scale = static_cast<float*>(at_of(vs));
  c.num_blocks = small(n, "the number of blocks"), c.kv_heads = small(h, "kv_heads");
  c.block_size = small(bs, "block_size"), c.head_dim = small(d, "head_dim");
  c.type = k.scalar_type() == at::kChar ? SMP_CACHE_I8 : SMP_CACHE_E4M3;
  return c;
}

template <typename T>
T* ptr(const Tensor* t) {
  return static_cast<T*>(at_of(t));
}
template <typename T>
T* ptr(const Tensor& t) {
  return static_cast<T*>(at_of(t));
}

void check(smp_status s) {
  if (s == SMP_OK) return;
  std::string what = smp_status_string(s);
  if (s == SMP_ERR_CUDA) what += " (cudaError " + std::to_string(smp_last_cuda_error()) + ")";
  refuse(what);
}

// Runs `body` and turns its exceptions into Python's.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& body) {
  try {
    if (have != want) refuse("wrong number of arguments");
    g_device = -1;
    body();
    Py_RETURN_NONE;
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* py_set_error(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&] {
    Py_XINCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
  });
}

// lens, add, held, free_blocks, free_head, table, block_size, num_blocks, max_tokens, the seven outputs, status, stream
PyObject* py_block_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&] {
    const Tensor& lens = tensor(a[0], "lens");
    const Tensor& add = tensor(a[1], "add");
    const Tensor& held = tensor(a[2], "held");
    const Tensor& free_blocks = tensor(a[3], "free_blocks");
    const Tensor& head = tensor(a[4], "free_head");
    const Tensor& table = tensor(a[5], "block_table");
    const int32_t cap = integer32(a[8], "max_tokens");
    flat(lens, "lens", at::kInt, {-1});
    const int64_t b = lens.size(0);
    flat(add, "add", at::kInt, {b});
    flat(held, "held", at::kInt, {b});
    flat(free_blocks, "free_blocks", at::kInt, {-1});
    flat(head, "free_head", at::kInt, {1});
    flat(table, "block_table", at::kInt, {b, -1});
    static const char* const names[7] = {"out.lens",     "out.held",    "out.free_head", "out.start",
                                         "out.position", "out.request", "out.slot"};
    const int64_t sizes[7] = {b, b, 1, b + 1, cap, cap, cap};
    const Tensor* out[7];
    for (int i = 0; i < 7; ++i) {
      out[i] = &tensor(a[9 + i], names[i]);
      flat(*out[i], names[i], i == 6 ? at::kLong : at::kInt, {sizes[i]});
    }
    const Launch to(a[16], a[17]);
    check(smp_block_plan(ptr<int32_t>(lens), ptr<int32_t>(add), ptr<int32_t>(held), small(b, "batch"),
                         ptr<int32_t>(free_blocks), small(free_blocks.size(0), "free_blocks"), ptr<int32_t>(head),
                         ptr<int32_t>(table), small(table.size(1), "block_table"), integer32(a[6], "block_size"),
                         integer32(a[7], "num_blocks"), cap, ptr<int32_t>(out[0]), ptr<int32_t>(out[1]),
                         ptr<int32_t>(out[2]), ptr<int32_t>(out[3]), ptr<int32_t>(out[4]), ptr<int32_t>(out[5]),
                         ptr<int64_t>(out[6]), to.status, to.stream));
  });
}

// q, k, positions, table, q_weight, k_weight, eps, interleaved, out_q, out_k, status, stream
PyObject* py_qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const Tensor& q = tensor(a[0], "q");
    const Tensor* k = optional(a[1], "k");
    const Tensor& positions = tensor(a[2], "positions");
    const Tensor* table = optional(a[3], "table");
    const Tensor* qw = optional(a[4], "q_weight");
    const Tensor* kw = optional(a[5], "k_weight");
    const Tensor& oq = tensor(a[8], "out_q");
    const Tensor* ok = optional(a[9], "out_k");
    const int64_t qs = heads_of(q, "q"), oqs = heads_of(oq, "out_q", &q), t = q.size(0), d = q.size(2);
    int64_t ks = 0, oks = 0, hk = 0;
    if (k) {
      ks = heads_of(*k, "k");
      hk = k->size(1);
      if (k->size(0) != t || k->size(2) != d || k->scalar_type() != q.scalar_type())
        refuse("k must be [tokens, heads, dim] with the tokens, dim and type of q");
      if (!ok) refuse("out_k must be a torch tensor");
      oks = heads_of(*ok, "out_k", k);
    }
    flat(positions, "positions", at::kInt, {t});
    if (table) flat(*table, "table", at::kFloat, {-1, -1});
    if (qw) flat(*qw, "q_weight", at::kFloat, {d});
    if (kw) flat(*kw, "k_weight", at::kFloat, {d});
    const Launch to(a[10], a[11]);
    check(smp_qk_norm_rope(at_of(q), at_of(k), small(t, "tokens"), small(q.size(1), "heads"), small(hk, "heads"),
                           small(d, "dim"), qs, ks, dtype_of(q, "q"), ptr<float>(qw), ptr<float>(kw),
                           float(number(a[6])), ptr<float>(table), table ? small(table->size(0), "table") : 0,
                           table ? small(table->size(1), "table") : 0, integer32(a[7], "interleaved"),
                           ptr<int32_t>(positions), at_of(oq), k ? at_of(ok) : nullptr, oqs, oks, to.status, to.stream));
  });
}

// cache, k, v, slots, status, stream
PyObject* py_cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const smp_cache c = cache_of(a[0]);
    const Tensor& k = tensor(a[1], "k");
    const Tensor& v = tensor(a[2], "v");
    const Tensor& slots = tensor(a[3], "slots");
    const int64_t ks = heads_of(k, "k"), vs = heads_of(v, "v", &k), t = k.size(0);
    if (k.size(1) != c.kv_heads || k.size(2) != c.head_dim) refuse("k must be [tokens, kv_heads, head_dim] of the cache");
    flat(slots, "slots", at::kLong, {t});
    const Launch to(a[4], a[5]);
    check(smp_cache_append(&c, at_of(k), at_of(v), small(t, "tokens"), ks, vs, dtype_of(k, "k"), ptr<int64_t>(slots),
                           to.status, to.stream));
  });
}

// cache, q, start, lens, table, scale (None: head_dim^-0.5), window, out, lse, workspace, status, stream
PyObject* py_cache_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const smp_cache c = cache_of(a[0]);
    const Tensor& q = tensor(a[1], "q");
    const Tensor& start = tensor(a[2], "start");
    const Tensor& lens = tensor(a[3], "lens");
    const Tensor& table = tensor(a[4], "block_table");
    const Tensor& out = tensor(a[7], "out");
    const Tensor* lse = optional(a[8], "lse");
    const Tensor& work = tensor(a[9], "workspace");
    const int64_t qs = heads_of(q, "q"), os = heads_of(out, "out", &q), t = q.size(0), h = q.size(1);
    if (q.size(2) != c.head_dim) refuse("q must have the cache's head_dim");
    flat(lens, "lens", at::kInt, {-1});
    const int64_t b = lens.size(0);
    flat(start, "start", at::kInt, {b + 1});
    flat(table, "block_table", at::kInt, {b, -1});
    if (lse) flat(*lse, "lse", at::kFloat, {t, h});
    const double scale = a[5] == Py_None ? std::pow(double(c.head_dim > 0 ? c.head_dim : 1), -0.5) : number(a[5]);
    flat(work, "workspace", at::kByte, {-1});
    const Launch to(a[10], a[11]);
    check(smp_cache_attention(&c, at_of(q), small(t, "tokens"), small(h, "heads"), qs, dtype_of(q, "q"),
                              ptr<int32_t>(start), ptr<int32_t>(lens), small(b, "batch"), ptr<int32_t>(table),
                              small(table.size(1), "block_table"), float(scale), integer32(a[6], "window"),
                              at_of(out), os, ptr<float>(lse), to.status, at_of(work), size_t(work.numel()),
                              to.stream));
  });
}

// p, q, draft_ids, uniforms, noise, draft_lens, out_accepted, out_ids, status, stream
PyObject* py_spec_verify_probs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const Tensor& p = tensor(a[0], "p");
    const Tensor* q = optional(a[1], "q");
    const Tensor& ids = tensor(a[2], "draft_ids");
    const Tensor& uniforms = tensor(a[3], "uniforms");
    const Tensor& noise = tensor(a[4], "noise");
    const Tensor* lens = optional(a[5], "draft_lens");
    const Tensor& accepted = tensor(a[6], "out_accepted");
    const Tensor& out = tensor(a[7], "out_ids");
    if (p.dim() != 3 || p.size(1) < 1) refuse("p must be [batch, drafts + 1, vocab]");
    const int64_t b = p.size(0), k = p.size(1) - 1, v = p.size(2);
    const smp_dtype dtype = dtype_of(p, "p");
    flat(p, "p", p.scalar_type(), {b, k + 1, v});
    if (q) flat(*q, "q", p.scalar_type(), {b, k, v});
    flat(ids, "draft_ids", at::kInt, {b, k});
    flat(uniforms, "uniforms", at::kFloat, {b, k});
    flat(noise, "noise", at::kFloat, {b, v});
    if (lens) flat(*lens, "draft_lens", at::kInt, {b});
    flat(accepted, "out_accepted", at::kInt, {b});
    flat(out, "out_ids", at::kInt, {b, k + 1});
    const Launch to(a[8], a[9]);
    check(smp_spec_verify_probs(at_of(p), at_of(q), ptr<int32_t>(ids), ptr<int32_t>(lens), small(b, "batch"),
                                small(k, "drafts"), small(v, "vocab"), dtype, ptr<float>(uniforms), ptr<float>(noise),
                                ptr<int32_t>(accepted), ptr<int32_t>(out), to.status, to.stream));
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<py_set_error>("set_error"),
                           method<py_block_plan>("block_plan"),
                           method<py_qk_norm_rope>("qk_norm_rope"),
                           method<py_cache_append>("cache_append"),
                           method<py_cache_attention>("cache_attention"),
                           method<py_spec_verify_probs>("spec_verify_probs"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "smp_step_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_smp_step_binding(void) { return PyModule_Create(&g_module); }
