// The Python side of the norm, rotation and 4-bit entries (include/pkv.h) as a CPython
// extension.
//
// A decode step's kernels take 2 - 5 us, and checking a dozen tensors and passing their
// addresses through ctypes takes the host 12 - 15; the same checks here take less than
// one.  Each function takes its arguments in order (None: not given), refuses tensors of
// another device, type, layout or shape with Python's ValueError / TypeError, makes the
// call on the cache's device and its current stream, and returns the entry's status.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "../../include/pkv.h"

namespace {

struct Raised {};  // a Python exception is set

[[noreturn]] void fail(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

std::string sizes(std::initializer_list<int64_t> want) {
  std::string s = "(";
  for (int64_t n : want) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
  return s + (want.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

int index_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda())
    fail(PyExc_ValueError, std::string(name) + " must be a CUDA tensor (the library has no CPU path)");
  return t.get_device();
}

void check_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> want,
                 const char* why = "") {
  if (t.sizes() != c10::IntArrayRef(want))
    fail(PyExc_ValueError, std::string(name) + " must be " + sizes(want) + why);
}

void check_place(const at::Tensor& t, const char* name, at::ScalarType type, int index) {
  if (!t.is_cuda() || t.get_device() != index)
    fail(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", the call on cuda:" +
                               std::to_string(index));
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                              c10::toString(t.scalar_type()));
}

// Address of a contiguous tensor.
void* address(const at::Tensor& t, const char* name, at::ScalarType type, int index) {
  check_place(t, name, type, index);
  if (!t.is_contiguous()) fail(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

void* address(PyObject* o, const char* name, at::ScalarType type, int index,
              std::initializer_list<int64_t> want, const char* why = "") {
  const at::Tensor& t = tensor(o, name);
  check_shape(t, name, want, why);
  return address(t, name, type, index);
}

int32_t* error_word(PyObject* o, int index) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "err");
  if (t.numel() < 1) fail(PyExc_ValueError, "err must hold one int32");
  return static_cast<int32_t*>(address(t, "err", at::kInt, index));
}

int32_t type_code(at::ScalarType type) {
  if (type == at::kFloat) return PKV_F32;
  if (type == at::kBFloat16) return PKV_BF16;
  fail(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(type) +
                            ": float32 or bfloat16");
}

int32_t int32_of(int64_t n, const char* name) {
  if (n < INT32_MIN || n > INT32_MAX) fail(PyExc_ValueError, std::string(name) + " is past 32 bits");
  return static_cast<int32_t>(n);
}

int32_t integer(PyObject* o, const char* name) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw Raised{};
  return int32_of(n, name);
}

float number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(x);
}

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Raised{};
  return r != 0;
}

// Rows [tokens, heads, head_dim], a token's heads together: address and token stride.
struct Rows {
  void* at;
  int64_t stride;
};

const at::Tensor& rows_tensor(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 3) fail(PyExc_ValueError, std::string(name) + " must be [tokens, heads, head_dim]");
  return t;
}

Rows rows(const at::Tensor& t, const char* name, at::ScalarType type, int index) {
  check_place(t, name, type, index);
  if ((t.size(2) > 1 && t.stride(2) != 1) || (t.size(1) > 1 && t.stride(1) != t.size(2)))
    fail(PyExc_ValueError, std::string(name) + ": a token's heads must be contiguous");
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2)};
}

Rows rows(PyObject* o, const char* name, at::ScalarType type, int index,
          std::initializer_list<int64_t> want) {
  const at::Tensor& t = rows_tensor(o, name);
  check_shape(t, name, want);
  return rows(t, name, type, index);
}

// Runs an entry on the device and its current stream.
template <typename F>
PyObject* call(int index, F entry) {
  pkv_status st;
  {
    const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(index));
    void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    Py_BEGIN_ALLOW_THREADS;
    st = entry(stream);
    Py_END_ALLOW_THREADS;
  }
  return PyLong_FromLong(st);
}

template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F body) {
  try {
    if (got != want)
      fail(PyExc_TypeError, std::string(name) + " takes " + std::to_string(want) + " arguments");
    return body();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// A 4-bit cache's six tensors, from args[0] on.
struct Cache {
  int index;
  pkv_pool_desc desc;
  void *k_pool, *v_pool, *k_groups, *v_groups;
  const float *k_scale, *v_scale;

  explicit Cache(PyObject* const* args) {
    const at::Tensor& kp = tensor(args[0], "k_pool");
    if (kp.dim() != 4) fail(PyExc_ValueError, "pool must be [num_blocks, n_kv, block_size, head_dim / 2]");
    const at::Tensor& vp = tensor(args[1], "v_pool");
    if (vp.sizes() != kp.sizes()) fail(PyExc_ValueError, "k_pool and v_pool must have the same shape");
    const int64_t nb = kp.size(0), nkv = kp.size(1), bs = kp.size(2), half = kp.size(3);
    if (half % 8 != 0) fail(PyExc_ValueError, "head_dim must be a multiple of 16");
    const at::Tensor* g[2] = {&tensor(args[2], "k_groups"), &tensor(args[3], "v_groups")};
    const at::Tensor* s[2] = {&tensor(args[4], "k_scale"), &tensor(args[5], "v_scale")};
    check_shape(*g[0], "k_groups", {nb, nkv, bs, half / 8}, ": one per 16 elements");
    check_shape(*g[1], "v_groups", {nb, nkv, bs, half / 8}, ": one per 16 elements");
    check_shape(*s[0], "k_scale", {nkv}, ": one per KV head");
    check_shape(*s[1], "v_scale", {nkv}, ": one per KV head");
    index = index_of(kp, "k_pool");
    k_pool = address(kp, "k_pool", at::kByte, index);
    v_pool = address(vp, "v_pool", at::kByte, index);
    k_groups = address(*g[0], "k_groups", at::kFloat8_e4m3fn, index);
    v_groups = address(*g[1], "v_groups", at::kFloat8_e4m3fn, index);
    k_scale = static_cast<const float*>(address(*s[0], "k_scale", at::kFloat, index));
    v_scale = static_cast<const float*>(address(*s[1], "v_scale", at::kFloat, index));
    desc = pkv_pool_desc{int32_of(nb, "num_blocks"), int32_of(bs, "block_size"), int32_of(nkv, "n_kv"),
                         int32_of(2 * half, "head_dim"), PKV_FP4_E2M1};
  }
};

// A batch's tables and lengths.
struct Batch {
  const int32_t *tables, *lens;
  int32_t num_seqs, width;

  Batch(PyObject* bt, PyObject* sl, int index) {
    const at::Tensor& t = tensor(bt, "block_tables");
    if (t.dim() != 2) fail(PyExc_ValueError, "block_tables must be [num_seqs, max_blocks_per_seq]");
    num_seqs = int32_of(t.size(0), "num_seqs");
    width = int32_of(t.size(1), "max_blocks_per_seq");
    tables = static_cast<const int32_t*>(address(t, "block_tables", at::kInt, index));
    lens = static_cast<const int32_t*>(
        address(sl, "seq_lens", at::kInt, index, {t.size(0)}, ": one per row of block_tables"));
  }
};

// What a norm and rotation takes: args[0] cos_sin, args[1] positions; weights, eps and
// interleaved from more[0] on.
pkv_norm_rope_desc norm_rope(PyObject* const* args, PyObject* const* more, int64_t tokens,
                             int64_t head_dim, at::ScalarType type, int index) {
  pkv_norm_rope_desc d{};
  const at::Tensor& cs = tensor(args[0], "cos_sin");
  if (cs.dim() != 2) fail(PyExc_ValueError, "cos_sin must be [num_positions, rot_dim]");
  d.cos_sin = static_cast<const float*>(address(cs, "cos_sin", at::kFloat, index));
  d.num_positions = int32_of(cs.size(0), "num_positions");
  d.rot_dim = int32_of(cs.size(1), "rot_dim");
  d.positions = static_cast<const int32_t*>(
      address(args[1], "positions", at::kInt, index, {tokens}, ": one per token"));
  if (more[0] != Py_None) d.q_weight = address(more[0], "q_weight", type, index, {head_dim});
  if (more[1] != Py_None) d.k_weight = address(more[1], "k_weight", type, index, {head_dim});
  d.eps = number(more[2]);
  d.interleaved = truth(more[3]);
  return d;
}

const int64_t* slot_mapping(PyObject* o, int64_t tokens, int index) {
  return static_cast<const int64_t*>(
      address(o, "slot_mapping", at::kLong, index, {tokens}, ": one entry per token"));
}

// (q, k, cos_sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out, err)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope", n, 11, [&] {
    const at::Tensor& q = rows_tensor(a[0], "q");
    const int index = index_of(q, "q");
    const at::ScalarType type = q.scalar_type();
    const int64_t T = q.size(0), H = q.size(1), hd = q.size(2);
    const at::Tensor& k = rows_tensor(a[1], "k");
    if (k.size(0) != T || k.size(2) != hd)
      fail(PyExc_ValueError, "k must be [T, n_kv, head_dim] with q's tokens and head_dim");
    const int64_t nkv = k.size(1);
    const Rows qr = rows(q, "q", type, index), kr = rows(k, "k", type, index);
    const pkv_norm_rope_desc d = norm_rope(a + 2, a + 4, T, hd, type, index);
    const Rows qo = rows(a[8], "q_out", type, index, {T, H, hd});
    const Rows ko = rows(a[9], "k_out", type, index, {T, nkv, hd});
    int32_t* err = error_word(a[10], index);
    const int32_t code = type_code(type), tokens = int32_of(T, "T"), heads = int32_of(H, "n_heads");
    const int32_t kv = int32_of(nkv, "n_kv"), dim = int32_of(hd, "head_dim");
    return call(index, [&](void* stream) {
      return pkv_qk_norm_rope(qr.at, qr.stride, kr.at, kr.stride, code, tokens, heads, kv, dim, &d,
                              qo.at, qo.stride, ko.at, ko.stride, err, stream);
    });
  });
}

// (q, k, v, cos_sin, positions, slot_mapping, k_pool, v_pool, q_weight, k_weight, eps,
//  interleaved, q_out, err)
PyObject* qk_norm_rope_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope_write", n, 14, [&] {
    const at::Tensor& kp = tensor(a[6], "k_pool");
    if (kp.dim() != 4) fail(PyExc_ValueError, "pool must be [num_blocks, block_size, n_kv, head_dim]");
    const at::Tensor& vp = tensor(a[7], "v_pool");
    if (vp.sizes() != kp.sizes()) fail(PyExc_ValueError, "k_pool and v_pool must have the same shape");
    const int index = index_of(kp, "k_pool");
    const at::ScalarType type = kp.scalar_type();
    const pkv_pool_desc desc{int32_of(kp.size(0), "num_blocks"), int32_of(kp.size(1), "block_size"),
                             int32_of(kp.size(2), "n_kv"), int32_of(kp.size(3), "head_dim"),
                             type_code(type)};
    void *k_pool = address(kp, "k_pool", type, index), *v_pool = address(vp, "v_pool", type, index);
    const at::Tensor& q = rows_tensor(a[0], "q");
    const int64_t T = q.size(0), H = q.size(1), hd = kp.size(3), nkv = kp.size(2);
    if (q.size(2) != hd)
      fail(PyExc_ValueError, "q must be [T, n_heads, head_dim] with the pool's head_dim");
    const Rows qr = rows(q, "q", type, index), kr = rows(a[1], "k", type, index, {T, nkv, hd});
    const Rows vr = rows(a[2], "v", type, index, {T, nkv, hd});
    const pkv_norm_rope_desc d = norm_rope(a + 3, a + 8, T, hd, type, index);
    const int64_t* slots = slot_mapping(a[5], T, index);
    const Rows qo = rows(a[12], "q_out", type, index, {T, H, hd});
    int32_t* err = error_word(a[13], index);
    const int32_t tokens = int32_of(T, "T"), heads = int32_of(H, "n_heads");
    return call(index, [&](void* stream) {
      return pkv_qk_norm_rope_write(qr.at, qr.stride, kr.at, kr.stride, vr.at, vr.stride, tokens,
                                    heads, &d, qo.at, qo.stride, slots, k_pool, v_pool, &desc, err,
                                    stream);
    });
  });
}

// (q, k, v, cos_sin, positions, slot_mapping, the cache's six, q_weight, k_weight, eps,
//  interleaved, q_out, err)
PyObject* qk_norm_rope_write_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope_write_fp4", n, 18, [&] {
    const Cache c(a + 6);
    const at::Tensor& q = rows_tensor(a[0], "q");
    const at::ScalarType type = q.scalar_type();
    const int64_t T = q.size(0), H = q.size(1), hd = c.desc.head_dim, nkv = c.desc.n_kv;
    if (q.size(2) != hd)
      fail(PyExc_ValueError, "q must be [T, n_heads, head_dim] with the pool's head_dim");
    const Rows qr = rows(q, "q", type, c.index), kr = rows(a[1], "k", type, c.index, {T, nkv, hd});
    const Rows vr = rows(a[2], "v", type, c.index, {T, nkv, hd});
    const pkv_norm_rope_desc d = norm_rope(a + 3, a + 12, T, hd, type, c.index);
    const int64_t* slots = slot_mapping(a[5], T, c.index);
    const Rows qo = rows(a[16], "q_out", type, c.index, {T, H, hd});
    int32_t* err = error_word(a[17], c.index);
    const int32_t code = type_code(type), tokens = int32_of(T, "T"), heads = int32_of(H, "n_heads");
    return call(c.index, [&](void* stream) {
      return pkv_qk_norm_rope_write_fp4(qr.at, qr.stride, kr.at, kr.stride, vr.at, vr.stride, code,
                                        tokens, heads, &d, qo.at, qo.stride, slots, c.k_pool, c.v_pool,
                                        c.k_groups, c.v_groups, c.k_scale, c.v_scale, &c.desc, err,
                                        stream);
    });
  });
}

// (k, v, slot_mapping, the cache's six, err)
PyObject* kv_write_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_write_fp4", n, 10, [&] {
    const Cache c(a + 3);
    const at::Tensor& k = rows_tensor(a[0], "k");
    const at::ScalarType type = k.scalar_type();
    const int64_t T = k.size(0), hd = c.desc.head_dim, nkv = c.desc.n_kv;
    check_shape(k, "k", {T, nkv, hd});
    const Rows kr = rows(k, "k", type, c.index), vr = rows(a[1], "v", type, c.index, {T, nkv, hd});
    const int64_t* slots = slot_mapping(a[2], T, c.index);
    int32_t* err = error_word(a[9], c.index);
    const int32_t code = type_code(type), tokens = int32_of(T, "T");
    return call(c.index, [&](void* stream) {
      return pkv_kv_write_fp4(kr.at, kr.stride, vr.at, vr.stride, code, slots, tokens, c.k_pool,
                              c.v_pool, c.k_groups, c.v_groups, c.k_scale, c.v_scale, &c.desc, err,
                              stream);
    });
  });
}

// (the cache's six, block_tables, seq_lens, cu_seq_lens, total_tokens, k_out, v_out, err)
PyObject* kv_gather_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_gather_fp4", n, 13, [&] {
    const Cache c(a);
    const Batch b(a[6], a[7], c.index);
    const int32_t* cu = static_cast<const int32_t*>(
        address(a[8], "cu_seq_lens", at::kInt, c.index, {int64_t(b.num_seqs) + 1}));
    const int32_t total = integer(a[9], "total_tokens");
    const at::ScalarType type = tensor(a[10], "k_out").scalar_type();
    const int32_t code = type_code(type);
    void* k_out = address(a[10], "k_out", type, c.index, {total, c.desc.n_kv, c.desc.head_dim});
    void* v_out = address(a[11], "v_out", type, c.index, {total, c.desc.n_kv, c.desc.head_dim});
    int32_t* err = error_word(a[12], c.index);
    return call(c.index, [&](void* stream) {
      return pkv_kv_gather_fp4(c.k_pool, c.v_pool, c.k_groups, c.v_groups, c.k_scale, c.v_scale,
                               &c.desc, b.tables, b.width, b.lens, cu, b.num_seqs, total, code, k_out,
                               v_out, err, stream);
    });
  });
}

// Queries and outputs of an attention call: [rows, n_heads, head_dim] of one type.
struct Attention {
  const void* q;
  void* out;
  int32_t code, rows, heads;

  Attention(PyObject* qo, PyObject* oo, const Cache& c) {
    const at::Tensor& t = tensor(qo, "q");
    if (t.dim() != 3 || t.size(2) != c.desc.head_dim)
      fail(PyExc_ValueError, "q must be [rows, n_heads, head_dim] with the pool's head_dim");
    const at::ScalarType type = t.scalar_type();
    code = type_code(type);
    rows = int32_of(t.size(0), "rows");
    heads = int32_of(t.size(1), "n_heads");
    q = address(t, "q", type, c.index);
    out = address(oo, "out", type, c.index, {t.size(0), t.size(1), t.size(2)});
  }
};

// (q, the cache's six, block_tables, seq_lens, scale, max_seq_len, out, workspace, max_ctas,
//  err)
PyObject* paged_attention_decode_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention_decode_fp4", n, 15, [&] {
    const Cache c(a + 1);
    const Batch b(a[7], a[8], c.index);
    const Attention t(a[0], a[11], c);
    if (t.rows != b.num_seqs) fail(PyExc_ValueError, "q must have one row per sequence");
    const float scale = number(a[9]);
    const int32_t most = integer(a[10], "max_seq_len"), ctas = integer(a[13], "max_ctas");
    const at::Tensor& ws = tensor(a[12], "workspace");
    void* at = address(ws, "workspace", ws.scalar_type(), c.index);
    const size_t bytes = ws.nbytes();
    int32_t* err = error_word(a[14], c.index);
    return call(c.index, [&](void* stream) {
      return pkv_paged_attention_decode_fp4(t.q, t.code, b.num_seqs, t.heads, c.k_pool, c.v_pool,
                                            c.k_groups, c.v_groups, c.k_scale, c.v_scale, &c.desc,
                                            b.tables, b.width, b.lens, most, scale, ctas, t.out, at,
                                            bytes, err, stream);
    });
  });
}

// (q, cu_q_lens, the cache's six, block_tables, seq_lens, scale, max_q_len, max_seq_len, out,
//  err)
PyObject* paged_attention_prefill_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention_prefill_fp4", n, 15, [&] {
    const Cache c(a + 2);
    const Batch b(a[8], a[9], c.index);
    const Attention t(a[0], a[13], c);
    const int32_t* cu = static_cast<const int32_t*>(
        address(a[1], "cu_q_lens", at::kInt, c.index, {int64_t(b.num_seqs) + 1}));
    const float scale = number(a[10]);
    const int32_t most_q = integer(a[11], "max_q_len"), most = integer(a[12], "max_seq_len");
    int32_t* err = error_word(a[14], c.index);
    return call(c.index, [&](void* stream) {
      return pkv_paged_attention_prefill_fp4(t.q, t.code, cu, b.num_seqs, t.rows, most_q, t.heads,
                                             c.k_pool, c.v_pool, c.k_groups, c.v_groups, c.k_scale,
                                             c.v_scale, &c.desc, b.tables, b.width, b.lens, most, scale,
                                             t.out, err, stream);
    });
  });
}

#define PKV_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {PKV_METHOD(qk_norm_rope),
                         PKV_METHOD(qk_norm_rope_write),
                         PKV_METHOD(qk_norm_rope_write_fp4),
                         PKV_METHOD(kv_write_fp4),
                         PKV_METHOD(kv_gather_fp4),
                         PKV_METHOD(paged_attention_decode_fp4),
                         PKV_METHOD(paged_attention_prefill_fp4),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

// Tensors are read through the layouts of the PyTorch that this was compiled against, so
// another one is refused.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  PyObject* text = version ? PyObject_Str(version) : nullptr;
  const char* found = text ? PyUnicode_AsUTF8(text) : nullptr;
  PyObject* m = nullptr;
  if (found != nullptr) {
    if (std::string(found) == PKV_TORCH_VERSION)
      m = PyModule_Create(&module);
    else
      PyErr_Format(PyExc_ImportError, "built for PyTorch %s, this is %s", PKV_TORCH_VERSION, found);
  }
  Py_XDECREF(text);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return m;
}
