// py_binding.cpp -- Python entry points of the calls that serve single tokens
// (the verification step and the sliding window): argument checks and
// marshalling in C++, because a call with the same checks in Python, through
// ctypes, took 15 to 17 us of host time (8 to 10 with the checks pared down;
// eleven tensors, four attribute reads each), more than the kernels behind
// them take, and takes 2.5 this way.  Each function checks dtypes, devices, shapes and
// strides, passes raw device pointers and the current CUDA stream to the
// exported C function of the same name and returns its status; a wrong
// argument raises TypeError or ValueError.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "pkv.h"

namespace {

constexpr int64_t kBlockSize = 16;
constexpr int64_t kHeadDim = 128;

// A Python exception has been set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}
[[noreturn]] void refuse(const char* name, const char* what) { raise(PyExc_ValueError, std::string(name) + " " + what); }

enum class Kind { kBf16, kI32, kI64, kF32, kBytes, kWords };

bool is_kind(at::ScalarType t, Kind k) {
  switch (k) {
    case Kind::kBf16: return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16;
    case Kind::kI32: return t == at::kInt;
    case Kind::kI64: return t == at::kLong;
    case Kind::kF32: return t == at::kFloat;
    case Kind::kBytes: return t == at::kByte || t == at::kChar;
    case Kind::kWords: return t == at::kLong || t == at::kUInt64;
  }
  return false;
}

const char* kind_name(Kind k) {
  switch (k) {
    case Kind::kBf16: return "must hold BF16 values (bfloat16 or 16-bit bit patterns)";
    case Kind::kI32: return "must hold int32 values";
    case Kind::kI64: return "must hold int64 values";
    case Kind::kF32: return "must hold float32 values";
    case Kind::kBytes: return "must hold bytes (uint8)";
    case Kind::kWords: return "must hold 64-bit words (int64 or uint64)";
  }
  return "";
}

// The arguments of one call, read in order.
class Call {
 public:
  Call(PyObject* const* args, Py_ssize_t n, Py_ssize_t expected) : args_(args) {
    if (n != expected) raise(PyExc_TypeError, "wrong number of arguments");
    device_ = c10::cuda::current_device();
  }
  int device() const { return device_; }

  bool none() {
    if (args_[at_] != Py_None) return false;
    ++at_;
    return true;
  }

  // A tensor of a kind on the current device; contiguous unless strided is asked for.
  const at::Tensor& tensor(const char* name, Kind kind, bool strided = false) {
    PyObject* o = args_[at_++];
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!is_kind(t.scalar_type(), kind)) raise(PyExc_TypeError, std::string(name) + " " + kind_name(kind));
    if (!t.is_cuda() || t.get_device() != device_ || (!strided && !t.is_contiguous()))
      refuse(name, "must be a contiguous tensor on the current CUDA device");
    return t;
  }
  const at::Tensor* optional(const char* name, Kind kind) { return none() ? nullptr : &tensor(name, kind); }

  // Scratch memory of any dtype.
  void workspace(void** p, size_t* bytes) {
    *p = nullptr;
    *bytes = 0;
    if (none()) return;
    PyObject* o = args_[at_++];
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "workspace must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device_ || !t.is_contiguous())
      refuse("workspace", "must be a contiguous tensor on the current CUDA device");
    *p = t.data_ptr();
    *bytes = t.nbytes();
  }

  int32_t i32(const char* name) {
    const long long v = PyLong_AsLongLong(args_[at_++]);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX) refuse(name, "does not fit into 32 bits");
    return static_cast<int32_t>(v);
  }
  void* address() {
    void* v = PyLong_AsVoidPtr(args_[at_++]);
    if (v == nullptr && PyErr_Occurred()) throw Raised{};
    return v;
  }
  float f32() {
    const double v = PyFloat_AsDouble(args_[at_++]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(v);
  }
  bool truth() {
    const int v = PyObject_IsTrue(args_[at_++]);
    if (v < 0) throw Raised{};
    return v != 0;
  }
  // A cudaStream_t as an integer, or None for the current stream.
  void* stream() {
    if (none()) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
    return address();
  }

 private:
  PyObject* const* args_;
  Py_ssize_t at_ = 0;
  int device_;
};

int32_t size32(const at::Tensor& t, int d, const char* name) {
  const int64_t v = t.size(d);
  if (v > INT32_MAX) refuse(name, "has a size beyond 32 bits");
  return static_cast<int32_t>(v);
}

bool shape_is(const at::Tensor& t, std::initializer_list<int64_t> want) { return t.sizes() == at::IntArrayRef(want); }

Kind pool_kind(int32_t format) { return format == PKV_KV_BF16 ? Kind::kBf16 : Kind::kBytes; }

pkv_cache_desc pool_desc(const at::Tensor& t, int32_t format, const char* name) {
  if (format == PKV_KV_Q8_0) {
    if (t.dim() != 3 || t.size(2) != PKV_Q8_TILE_BYTES) refuse(name, "must be [num_blocks][num_kv_heads][2176]");
    return {size32(t, 0, name), kBlockSize, size32(t, 1, name), kHeadDim};
  }
  if (format != PKV_KV_BF16 && format != PKV_KV_FP8_E4M3) raise(PyExc_ValueError, "unknown kv_format");
  if (t.dim() != 4) refuse(name, "must be [num_blocks][num_kv_heads][16][128]");
  return {size32(t, 0, name), size32(t, 2, name), size32(t, 1, name), size32(t, 3, name)};
}

// K and V pool of one format and shape.
pkv_cache_desc pools(Call& c, int32_t format, const at::Tensor** k, const at::Tensor** v) {
  *k = &c.tensor("k_cache", pool_kind(format));
  *v = &c.tensor("v_cache", pool_kind(format));
  const pkv_cache_desc d = pool_desc(**k, format, "k_cache");
  if ((*k)->sizes() != (*v)->sizes()) raise(PyExc_ValueError, "k_cache and v_cache differ in shape");
  return d;
}

// BF16 [tokens][heads][128] whose heads are contiguous: its token stride.
int64_t token_stride(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads) {
  if (!shape_is(t, {tokens, heads, kHeadDim})) refuse(name, "must be [num_tokens][heads][128]");
  if (tokens > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != kHeadDim)))
    refuse(name, "must have the heads of a token contiguous");
  return tokens > 1 ? t.stride(0) : heads * kHeadDim;
}

void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return PyLong_FromLong(static_cast<long>(f()));
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {  // torch's own errors
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
    return nullptr;
  }
}

// (q_out, kv_format, k_cache, v_cache, slot_mapping, q, k, v, positions,
//  rope_table, q_weight, k_weight, eps, interleaved, stream)
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> pkv_status {
    Call c(args, n, 15);
    const at::Tensor& q_out = c.tensor("q_out", Kind::kBf16);
    const int32_t format = c.i32("kv_format");
    const at::Tensor *kc, *vc;
    const pkv_cache_desc d = pools(c, format, &kc, &vc);
    const at::Tensor& slots = c.tensor("slot_mapping", Kind::kI64);
    const int64_t tokens = slots.numel();
    if (tokens > INT32_MAX) refuse("slot_mapping", "has a size beyond 32 bits");
    const at::Tensor& q = c.tensor("q", Kind::kBf16, true);
    const at::Tensor& k = c.tensor("k", Kind::kBf16, true);
    const at::Tensor& v = c.tensor("v", Kind::kBf16, true);
    if (q.dim() != 3) refuse("q", "must be [num_tokens][heads][128]");
    const int64_t qs = token_stride(q, "q", tokens, q.size(1));
    const int64_t ks = token_stride(k, "k", tokens, d.num_kv_heads);
    const int64_t vs = token_stride(v, "v", tokens, d.num_kv_heads);
    if (q_out.sizes() != q.sizes()) raise(PyExc_ValueError, "q_out and q differ in shape");
    const at::Tensor* pos = c.optional("positions", Kind::kI32);
    const at::Tensor* table = c.optional("rope_table", Kind::kF32);
    const at::Tensor* qw = c.optional("q_weight", Kind::kBf16);
    const at::Tensor* kw = c.optional("k_weight", Kind::kBf16);
    if ((qw != nullptr && qw->numel() != kHeadDim) || (kw != nullptr && kw->numel() != kHeadDim))
      raise(PyExc_ValueError, "q_weight and k_weight must have 128 values");
    int32_t rows = 0, rot = 0;
    if (table != nullptr) {
      if (table->dim() != 2 || pos == nullptr)
        raise(PyExc_ValueError, "rope_table must be [max_positions][rot_dim], with positions beside it");
      if (pos->numel() != tokens) raise(PyExc_ValueError, "positions must have one entry per token");
      rows = size32(*table, 0, "rope_table");
      rot = size32(*table, 1, "rope_table");
    }
    const float eps = c.f32();
    const bool interleaved = c.truth();
    return pkv_qk_norm_rope_append(q_out.data_ptr(), kc->data_ptr(), vc->data_ptr(), &d, format,
                                   static_cast<const int64_t*>(slots.data_ptr()), q.data_ptr(), qs, k.data_ptr(), ks,
                                   v.data_ptr(), vs, static_cast<int32_t>(q.size(1)), ptr(qw), ptr(kw), eps,
                                   static_cast<const float*>(ptr(table)), rows, rot, interleaved ? 1 : 0,
                                   table != nullptr ? static_cast<const int32_t*>(ptr(pos)) : nullptr,
                                   static_cast<int32_t>(tokens), c.stream());
  });
}

// What the two masked attention calls share.
struct Masked {
  const at::Tensor *out, *q, *k, *v, *tables, *lens;
  pkv_cache_desc desc;
  int32_t seqs, q_len, heads, max_blocks;
};

Masked masked(Call& c) {
  Masked m;
  m.out = &c.tensor("out", Kind::kBf16);
  m.q = &c.tensor("q", Kind::kBf16);
  m.desc = pools(c, PKV_KV_BF16, &m.k, &m.v);
  m.tables = &c.tensor("block_tables", Kind::kI32);
  m.lens = &c.tensor("context_lens", Kind::kI32);
  if (m.lens->numel() > INT32_MAX) refuse("context_lens", "has a size beyond 32 bits");
  m.seqs = static_cast<int32_t>(m.lens->numel());
  if (m.q->dim() != 4 || m.q->size(0) != m.seqs || m.q->size(3) != kHeadDim || m.out->sizes() != m.q->sizes())
    raise(PyExc_ValueError, "q and out must be [num_seqs][query tokens][num_q_heads][128]");
  if (m.tables->dim() != 2 || m.tables->size(0) != m.seqs)
    raise(PyExc_ValueError, "block_tables must be [num_seqs][max_blocks_per_seq]");
  m.q_len = size32(*m.q, 1, "q");
  m.heads = size32(*m.q, 2, "q");
  m.max_blocks = size32(*m.tables, 1, "block_tables");
  return m;
}

// (out, q, k_cache, v_cache, block_tables, context_lens, tree_mask, tree_lens,
//  scale, kv_blocks_per_split, workspace, stream)
PyObject* paged_attention_tree(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> pkv_status {
    Call c(args, n, 12);
    const Masked m = masked(c);
    const at::Tensor& mask = c.tensor("tree_mask", Kind::kWords);
    if (!shape_is(mask, {m.seqs, m.q_len, (int64_t{m.q_len} + 63) / 64}))
      raise(PyExc_ValueError, "tree_mask must be [num_seqs][tree_len][ceil(tree_len / 64)]");
    const at::Tensor* tree_lens = c.optional("tree_lens", Kind::kI32);
    if (tree_lens != nullptr && tree_lens->numel() != m.seqs)
      raise(PyExc_ValueError, "tree_lens must have one entry per request");
    const float scale = c.f32();
    const int32_t split = c.i32("kv_blocks_per_split");
    void* ws;
    size_t ws_bytes;
    c.workspace(&ws, &ws_bytes);
    return pkv_paged_attention_tree(m.out->data_ptr(), m.q->data_ptr(), m.k->data_ptr(), m.v->data_ptr(), &m.desc,
                                    static_cast<const int32_t*>(m.tables->data_ptr()), m.max_blocks,
                                    static_cast<const int32_t*>(m.lens->data_ptr()),
                                    static_cast<const int32_t*>(ptr(tree_lens)),
                                    static_cast<const uint64_t*>(mask.data_ptr()), m.seqs, m.q_len, m.heads, scale,
                                    split, ws, ws_bytes, c.stream());
  });
}

// (out, q, k_cache, v_cache, block_tables, context_lens, q_len, window,
//  num_sinks, scale, kv_blocks_per_split, workspace, stream)
PyObject* paged_attention_window(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> pkv_status {
    Call c(args, n, 13);
    const Masked m = masked(c);
    if (c.i32("q_len") != m.q_len) raise(PyExc_ValueError, "q and out must be [num_seqs][q_len][num_q_heads][128]");
    const int32_t window = c.i32("window");
    const int32_t sinks = c.i32("num_sinks");
    const float scale = c.f32();
    const int32_t split = c.i32("kv_blocks_per_split");
    void* ws;
    size_t ws_bytes;
    c.workspace(&ws, &ws_bytes);
    return pkv_paged_attention_window(m.out->data_ptr(), m.q->data_ptr(), m.k->data_ptr(), m.v->data_ptr(), &m.desc,
                                      static_cast<const int32_t*>(m.tables->data_ptr()), m.max_blocks,
                                      static_cast<const int32_t*>(m.lens->data_ptr()), m.seqs, m.q_len, m.heads,
                                      window, sinks, scale, split, ws, ws_bytes, c.stream());
  });
}

// (k pointer array, v pointer array, num_layers, num_blocks, num_kv_heads,
//  kv_format, pools' device, block_tables, context_lens, accepted,
//  num_accepted, tree_len, tree_lens, stream)
PyObject* kv_compact(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> pkv_status {
    Call c(args, n, 14);
    void* k = c.address();
    void* v = c.address();
    const int32_t layers = c.i32("num_layers");
    pkv_cache_desc d{};
    d.num_blocks = c.i32("num_blocks");
    d.block_size = kBlockSize;
    d.num_kv_heads = c.i32("num_kv_heads");
    d.head_dim = kHeadDim;
    const int32_t format = c.i32("kv_format");
    if (c.i32("device") != c.device()) raise(PyExc_ValueError, "the pools must be on the current CUDA device");
    const at::Tensor& tables = c.tensor("block_tables", Kind::kI32);
    const at::Tensor& lens = c.tensor("context_lens", Kind::kI32);
    const at::Tensor& accepted = c.tensor("accepted", Kind::kI32);
    const at::Tensor& num = c.tensor("num_accepted", Kind::kI32);
    const int32_t tree_len = c.i32("tree_len");
    const at::Tensor* tree_lens = c.optional("tree_lens", Kind::kI32);
    const int64_t seqs = lens.numel();
    if (seqs > INT32_MAX) refuse("context_lens", "has a size beyond 32 bits");
    if (tables.dim() != 2 || tables.size(0) != seqs)
      raise(PyExc_ValueError, "block_tables must be [num_seqs][max_blocks_per_seq]");
    if (accepted.dim() != 2 || accepted.size(0) != seqs || num.numel() != seqs)
      raise(PyExc_ValueError, "accepted must be [num_seqs][max_accepted] and num_accepted [num_seqs]");
    if (tree_lens != nullptr && tree_lens->numel() != seqs)
      raise(PyExc_ValueError, "tree_lens must have one entry per request");
    return pkv_kv_compact(static_cast<void* const*>(k), static_cast<void* const*>(v), layers, &d, format,
                          static_cast<const int32_t*>(tables.data_ptr()), size32(tables, 1, "block_tables"),
                          static_cast<const int32_t*>(lens.data_ptr()), static_cast<const int32_t*>(ptr(tree_lens)),
                          static_cast<int32_t>(seqs), tree_len, static_cast<const int32_t*>(accepted.data_ptr()),
                          static_cast<const int32_t*>(num.data_ptr()), size32(accepted, 1, "accepted"), c.stream());
  });
}

template <typename F>
constexpr PyCFunction fastcall(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef kMethods[] = {
    {"qk_norm_rope_append", fastcall(qk_norm_rope_append), METH_FASTCALL, nullptr},
    {"paged_attention_tree", fastcall(paged_attention_tree), METH_FASTCALL, nullptr},
    {"paged_attention_window", fastcall(paged_attention_window), METH_FASTCALL, nullptr},
    {"kv_compact", fastcall(kv_compact), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pkv_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_binding() { return PyModule_Create(&kModule); }
