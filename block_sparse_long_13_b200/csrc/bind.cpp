// The calls of the 8-bit cache from Python: checks of the tensors, structures and the call itself without the interpreter.
//
// These calls serve single tokens, where thirteen tensors checked one by one in Python cost more than the kernels: one
// row over 32K keys took 16.6 us call after call instead of 12.3, of which the device needs 10.2; the smallest batch
// advance 12 instead of 5.0.  Each function returns the library's status, or None as soon as an argument is not
// exactly what the call wants; the Python function then looks for what is wrong, and names it.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "../../include/msa.h"

namespace {

decltype(&msa_attn_decode_fp8) g_decode;
decltype(&msa_attn_prefill_fp8) g_prefill;
decltype(&msa_qknorm_rope_insert_fp8) g_insert;
decltype(&msa_advance_batch) g_advance;

struct Misfit {};                                   // an argument that Python has to look at

enum Name { NUM_Q, NUM_KV, HEAD, IDX_HEADS, IDX_DIM, BLOCK, TOPK, SCALE, Q_START, CTX_LEN, PAGE_TABLE, TOTAL_Q, MAX_Q, PAGES,
            HANDLE, NAMES };
PyObject* g_name[NAMES];
const char* const kName[NAMES] = {"num_q_heads", "num_kv_heads", "head_dim", "idx_heads", "idx_dim", "block_size", "topk",
                                  "softmax_scale", "q_start", "ctx_len", "page_table", "total_q", "max_q_per_seq",
                                  "num_pages", "cuda_stream"};

struct Held {                                       // an attribute, held while it is looked at
  PyObject* o;
  Held(PyObject* from, Name n) : o(PyObject_GetAttr(from, g_name[n])) {
    if (!o) throw Misfit();
  }
  ~Held() { Py_DECREF(o); }
  Held(const Held&) = delete;
};

int32_t int_of(PyObject* o) {
  if (!PyLong_CheckExact(o)) throw Misfit();
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  if (over || v < INT32_MIN || v > INT32_MAX) throw Misfit();
  return static_cast<int32_t>(v);
}
int32_t int_of(PyObject* from, Name n) { return int_of(Held(from, n).o); }
float float_of(PyObject* o) {
  if (PyFloat_CheckExact(o)) return static_cast<float>(PyFloat_AS_DOUBLE(o));
  return static_cast<float>(int_of(o));
}

const at::Tensor& tensor_of(PyObject* o) {
  if (!THPVariable_CheckExact(o)) throw Misfit();
  return THPVariable_Unpack(o);
}

struct Checks {
  int device = -1;                                  // the current one
  void* pointer(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
    if (!t.is_cuda()) throw Misfit();
    if (device < 0) device = c10::cuda::current_device();
    if (t.get_device() != device || t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) throw Misfit();
    return t.data_ptr();
  }
  void* pointer(PyObject* o, at::ScalarType type, at::IntArrayRef shape) { return pointer(tensor_of(o), type, shape); }
  void* maybe(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : pointer(o, type, shape);
  }
  cudaStream_t stream(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    if (PyLong_CheckExact(o)) return handle(o);
    return handle(Held(o, HANDLE).o);
  }
  static cudaStream_t handle(PyObject* o) {
    if (!PyLong_CheckExact(o)) throw Misfit();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Misfit();
    return static_cast<cudaStream_t>(p);
  }
  msa_config_t config(PyObject* o) {
    msa_config_t c{};
    c.num_q_heads = int_of(o, NUM_Q);
    c.num_kv_heads = int_of(o, NUM_KV);
    c.head_dim = int_of(o, HEAD);
    c.idx_heads = int_of(o, IDX_HEADS);
    c.idx_dim = int_of(o, IDX_DIM);
    c.block_size = int_of(o, BLOCK);
    c.topk = int_of(o, TOPK);
    c.softmax_scale = float_of(Held(o, SCALE).o);
    return c;
  }
  msa_batch_t batch(PyObject* o) {
    msa_batch_t b{};
    const Held qs(o, Q_START), ctx(o, CTX_LEN), pages(o, PAGE_TABLE);
    const at::Tensor &n = tensor_of(ctx.o), &p = tensor_of(pages.o);
    if (n.dim() != 1 || p.dim() != 2 || n.size(0) >= INT32_MAX || p.size(1) > INT32_MAX) throw Misfit();
    b.num_seqs = static_cast<int32_t>(n.size(0));
    b.max_blocks_per_seq = static_cast<int32_t>(p.size(1));
    b.total_q = int_of(o, TOTAL_Q);
    b.max_q_per_seq = int_of(o, MAX_Q);
    b.num_pages = int_of(o, PAGES);
    b.q_start = static_cast<const int32_t*>(pointer(qs.o, at::kInt, {n.size(0) + 1}));
    b.ctx_len = static_cast<const int32_t*>(pointer(n, at::kInt, {n.size(0)}));
    b.page_table = static_cast<const int32_t*>(pointer(p, at::kInt, {n.size(0), p.size(1)}));
    return b;
  }
};

template <typename F>
PyObject* answer(F&& call) {
  try {
    return PyLong_FromLong(call());
  } catch (const Misfit&) {
  } catch (const std::exception&) {                 // torch's own: tensors without storage and the like
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

template <typename F>
long outside(F&& call) {                            // without the interpreter's lock, as ctypes does it
  long status;
  Py_BEGIN_ALLOW_THREADS
  status = call();
  Py_END_ALLOW_THREADS
  return status;
}

// attn(prefill, cfg, batch, q, k_cache, v_cache, k_scale, v_scale, block_idx, out, lse, workspace, stream)
PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer([&]() -> long {
    if (n != 13) throw Misfit();
    Checks c;
    const msa_config_t cfg = c.config(a[1]);
    const msa_batch_t b = c.batch(a[2]);
    const int64_t rows[] = {b.total_q, cfg.num_q_heads, cfg.head_dim};
    const int64_t cache[] = {b.num_pages, cfg.num_kv_heads, cfg.block_size, cfg.head_dim};
    const int64_t slots[] = {b.total_q, cfg.num_kv_heads, cfg.topk};
    const at::IntArrayRef r(rows), kv(cache);
    void* q = c.pointer(a[3], at::kBFloat16, r);
    void* k = c.pointer(a[4], at::kByte, kv);
    void* v = c.pointer(a[5], at::kByte, kv);
    void* ks = c.pointer(a[6], at::kFloat, kv.slice(0, 2));
    void* vs = c.pointer(a[7], at::kFloat, kv.slice(0, 2));
    void* idx = c.pointer(a[8], at::kInt, slots);
    void* out = c.pointer(a[9], at::kBFloat16, r);
    void* lse = c.maybe(a[10], at::kFloat, r.slice(0, 2));
    void* ws = nullptr;
    int64_t bytes = 0;
    if (a[11] != Py_None) {
      const at::Tensor& t = tensor_of(a[11]);
      bytes = t.numel();
      ws = c.pointer(t, at::kByte, {bytes});
    }
    const cudaStream_t s = c.stream(a[12]);
    const bool prefill = a[0] == Py_True;
    return outside([&] {
      return (prefill ? g_prefill : g_decode)(&cfg, &b, q, k, v, static_cast<const float*>(ks), static_cast<const float*>(vs),
                                              static_cast<const int32_t*>(idx), out, static_cast<float*>(lse), ws,
                                              static_cast<size_t>(bytes), s);
    });
  });
}

// insert(cfg, batch, q, k_new, v_new, q_norm_w, k_norm_w, q_out, k_cache, v_cache, k_scale, v_scale, rotary_dim, theta, eps,
// stream)
PyObject* insert(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer([&]() -> long {
    if (n != 16) throw Misfit();
    Checks c;
    const msa_config_t cfg = c.config(a[0]);
    const msa_batch_t b = c.batch(a[1]);
    const int64_t rows[] = {b.total_q, cfg.num_q_heads, cfg.head_dim}, fresh[] = {b.total_q, cfg.num_kv_heads, cfg.head_dim};
    const int64_t cache[] = {b.num_pages, cfg.num_kv_heads, cfg.block_size, cfg.head_dim};
    const at::IntArrayRef r(rows), f(fresh), kv(cache);
    void* q = c.pointer(a[2], at::kBFloat16, r);
    void* kn = c.pointer(a[3], at::kBFloat16, f);
    void* vn = c.pointer(a[4], at::kBFloat16, f);
    void* qw = c.pointer(a[5], at::kBFloat16, f.slice(2));
    void* kw = c.pointer(a[6], at::kBFloat16, f.slice(2));
    void* qo = c.pointer(a[7], at::kBFloat16, r);
    void* k = c.pointer(a[8], at::kByte, kv);
    void* v = c.pointer(a[9], at::kByte, kv);
    void* ks = c.pointer(a[10], at::kFloat, kv.slice(0, 2));
    void* vs = c.pointer(a[11], at::kFloat, kv.slice(0, 2));
    const int32_t rotary = int_of(a[12]);
    const float theta = float_of(a[13]), eps = float_of(a[14]);
    const cudaStream_t s = c.stream(a[15]);
    return outside([&] {
      return g_insert(&cfg, &b, q, kn, vn, qw, kw, qo, k, v, static_cast<float*>(ks), static_cast<float*>(vs), rotary, theta,
                      eps, s);
    });
  });
}

// advance(delta, ctx_len, page_table, free_ring, pool, ctx_len_out, pool_out, q_start, slot_map, block_size, stream)
PyObject* advance(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer([&]() -> long {
    if (n != 11) throw Misfit();
    Checks c;
    const at::Tensor &table = tensor_of(a[2]), &ring = tensor_of(a[3]);
    if (table.dim() != 2 || ring.dim() != 1) throw Misfit();
    const int64_t seqs = table.size(0), width = table.size(1), pages = ring.size(0);
    int64_t rows = 0;
    if (a[8] != Py_None) rows = tensor_of(a[8]).numel();
    if (seqs >= INT32_MAX || width > INT32_MAX || pages > INT32_MAX || rows > INT32_MAX) throw Misfit();
    auto ints = [&](PyObject* o, int64_t len) { return static_cast<int32_t*>(c.pointer(o, at::kInt, {len})); };
    const int32_t *delta = ints(a[0], seqs), *ctx = ints(a[1], seqs);
    int32_t* pt = static_cast<int32_t*>(c.pointer(table, at::kInt, {seqs, width}));
    int32_t *fr = ints(a[3], pages), *pool = ints(a[4], 4), *ctx_out = ints(a[5], seqs), *pool_out = ints(a[6], 4);
    int32_t* qs = ints(a[7], seqs + 1);
    int32_t* map = a[8] == Py_None ? nullptr : ints(a[8], rows);
    if (rows == 0) map = nullptr;
    const int32_t block = int_of(a[9]);
    const cudaStream_t s = c.stream(a[10]);
    return outside([&] {
      return g_advance(static_cast<int32_t>(seqs), static_cast<int32_t>(width), static_cast<int32_t>(pages), block, delta, ctx,
                       pt, fr, pool, ctx_out, pool_out, qs, map, static_cast<int32_t>(rows), s);
    });
  });
}

// setup(decode, prefill, insert, advance): the entry points of the loaded library
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "setup takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  g_decode = reinterpret_cast<decltype(g_decode)>(p[0]);
  g_prefill = reinterpret_cast<decltype(g_prefill)>(p[1]);
  g_insert = reinterpret_cast<decltype(g_insert)>(p[2]);
  g_advance = reinterpret_cast<decltype(g_advance)>(p[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)); }

PyMethodDef methods[] = {{"setup", fast<setup>(), METH_FASTCALL, nullptr},
                         {"attn", fast<attn>(), METH_FASTCALL, nullptr},
                         {"insert", fast<insert>(), METH_FASTCALL, nullptr},
                         {"advance", fast<advance>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
  for (int i = 0; i < NAMES; ++i)
    if (!(g_name[i] = PyUnicode_InternFromString(kName[i]))) return nullptr;
  return PyModule_Create(&module);
}
