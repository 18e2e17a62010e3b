// marshal.cpp -- Python marshalling of the calls that a server makes once per layer or per
// token (rotary append, paged attention, commit, quantisers, e4m3 logits), as a CPython
// module.  At decoding sizes the kernels take 2 to 4 us, and the same calls through ctypes
// spent 8 to 11 us on the host; here it is the checks, one pointer per tensor and the launch.
//
// Every function takes the arguments of its namesake in binding.py in order and returns the
// library's status.  Tensors are dense device tensors of the current device (or None) of the
// types and dimensions that the shape says (neighbouring dimensions may be merged or split);
// the structures are the ctypes ones of binding.py.  The library is reached by the addresses
// that bind() is given, so this module links to nothing of it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>

#include "../../include/eagle_verify.h"

namespace {

// raised as ValueError
struct BadArgument : std::exception {
  const char* text;
  explicit BadArgument(const char* t) : text(t) {}
  const char* what() const noexcept override { return text; }
};
struct PythonError {};  // a Python exception is set

struct Entry {
  decltype(&eagle_rope_append) rope_append;
  decltype(&eagle_tree_attention_paged) tree_attention_paged;
  decltype(&eagle_commit_accepted_paged) commit_accepted_paged;
  decltype(&eagle_quantize_rows) quantize_rows;
  decltype(&eagle_quantize_blocks) quantize_blocks;
  decltype(&eagle_lm_head_logits_scaled) lm_head_logits_scaled;
} g_entry = {};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw BadArgument("library arguments are device tensors");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw BadArgument("library arguments are device tensors");
  if (t.get_device() != c10::cuda::current_device()) throw BadArgument("library arguments are on the current device");
  return t;
}

using Dims = std::initializer_list<int64_t>;

// Whether a dense tensor of as many elements (at least one) holds them in the order of an
// array `want`: its dimensions are those, some neighbours of either side merged into one.  With
// dimensions swapped ([B, heads, N, D] for [B, N, heads, D]) both sides have a boundary inside
// a stretch that has no common one.
bool same_order(const at::Tensor& t, Dims want) {
  // products of the last dimensions, from 1 to the number of elements
  int64_t i = t.dim(), have = 1, need = 1;
  const int64_t* w = want.end();
  bool inner_have = false, inner_need = false;
  auto next_have = [&] {
    const int64_t before = have;
    while (i > 0 && have == before) have *= t.size(--i);
  };
  auto next_need = [&] {
    const int64_t before = need;
    while (w != want.begin() && need == before) need *= *--w;
  };
  for (const int64_t numel = t.numel(); have != numel || need != numel;) {
    if (have == need) {
      inner_have = inner_need = false;
      next_have();
      next_need();
    } else if (have < need) {
      inner_have = true;
      next_have();
    } else {
      inner_need = true;
      next_need();
    }
    if (inner_have && inner_need) return false;
  }
  return true;
}

// A dense tensor's memory, if it is that array of that type; None is a null pointer.
template <typename T = void>
T* ptr(PyObject* o, Dims dims, at::ScalarType type) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  if (!t.is_contiguous()) throw BadArgument("library arguments are contiguous tensors");
  int64_t numel = 1;
  for (const int64_t d : dims) numel *= d;
  if (t.numel() != numel || t.scalar_type() != type)
    throw BadArgument("a tensor does not have the size or the type that the shape says");
  if (numel > 0 && !same_order(t, dims)) throw BadArgument("a tensor does not have the dimensions that the shape says");
  return static_cast<T*>(t.data_ptr());
}
int32_t* ints(PyObject* o, Dims dims) { return ptr<int32_t>(o, dims, at::kInt); }
float* floats(PyObject* o, Dims dims) { return ptr<float>(o, dims, at::kFloat); }
// e4m3 values, or their bytes
void* bytes(PyObject* o, Dims dims) {
  const bool raw = THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kByte;
  return ptr(o, dims, raw ? at::kByte : at::kFloat8_e4m3fn);
}

// [R, heads, D] whose rows may be strided parts of a wider array.
struct Rows {
  void* p = nullptr;
  int64_t stride = 0;
};
Rows token_rows(PyObject* o, int64_t rows, int64_t heads, int64_t d, at::ScalarType type) {
  Rows r;
  if (o == Py_None) return r;
  const at::Tensor& t = tensor(o);
  if (t.dim() != 3 || t.size(0) != rows || t.size(1) != heads || t.size(2) != d || t.scalar_type() != type)
    throw BadArgument("token rows are [R, heads, D] of the shape's heads and type");
  if (rows > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d)))
    throw BadArgument("token rows are [R, heads, D] with dense heads");
  r.p = t.data_ptr();
  r.stride = rows > 1 ? t.stride(0) : heads * d;
  return r;
}

// A ctypes structure; None is a null pointer.
template <typename T>
struct Struct {
  Py_buffer view{};
  const T* p = nullptr;
  explicit Struct(PyObject* o) {
    if (o == Py_None) return;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw PythonError{};
    if (view.len != static_cast<Py_ssize_t>(sizeof(T))) {
      PyBuffer_Release(&view);
      throw BadArgument("a structure of binding.py is expected");
    }
    p = static_cast<const T*>(view.buf);
  }
  ~Struct() {
    if (p != nullptr) PyBuffer_Release(&view);
  }
  Struct(const Struct&) = delete;
  Struct& operator=(const Struct&) = delete;
};

// None is torch's current stream; else a handle or a torch stream.
void* stream(PyObject* o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  if (PyLong_Check(o)) {
    void* s = PyLong_AsVoidPtr(o);
    if (s == nullptr && PyErr_Occurred()) throw PythonError{};
    return s;
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (h == nullptr) throw PythonError{};
  void* s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (s == nullptr && PyErr_Occurred()) throw PythonError{};
  return s;
}

int32_t integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < INT32_MIN || v > INT32_MAX) throw BadArgument("a 32-bit integer is expected");
  return static_cast<int32_t>(v);
}

// What the shape says of the cache.  Its numbers are the library's to refuse; here they only
// size tensors.
struct Sizes {
  int64_t B, N, Hq, Hkv, D, H, pages, page_size, max_pages;
  at::ScalarType type;
  Sizes(const eagle_shape_t* s, const eagle_pages_t* pg) {
    if (s == nullptr) throw BadArgument("a shape is expected");
    B = s->batch;
    N = s->num_nodes;
    Hq = s->num_q_heads;
    Hkv = s->num_kv_heads;
    D = s->head_dim;
    H = s->hidden;
    pages = pg == nullptr ? 0 : pg->num_pages;
    page_size = pg == nullptr ? 0 : pg->page_size;
    max_pages = pg == nullptr ? 0 : pg->max_pages;
    type = s->dtype == EAGLE_DTYPE_BF16 ? at::kBFloat16 : at::kFloat;
  }
  void* pool(PyObject* o) const { return ptr(o, {pages, Hkv, page_size, D}, type); }
  int32_t* table(PyObject* o) const { return ints(o, {B, max_pages}); }
  void* nodes(PyObject* o, int64_t heads) const { return ptr(o, {B, N, heads, D}, type); }
};

int32_t dtype(const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return EAGLE_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return EAGLE_DTYPE_F32;
  throw BadArgument("fp32 or bf16 is expected");
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (g_entry.rope_append == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const PythonError&) {
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

using Args = PyObject* const*;

PyObject* bind(PyObject*, Args a, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "six addresses are expected");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  g_entry.rope_append = reinterpret_cast<decltype(g_entry.rope_append)>(p[0]);
  g_entry.tree_attention_paged = reinterpret_cast<decltype(g_entry.tree_attention_paged)>(p[1]);
  g_entry.commit_accepted_paged = reinterpret_cast<decltype(g_entry.commit_accepted_paged)>(p[2]);
  g_entry.quantize_rows = reinterpret_cast<decltype(g_entry.quantize_rows)>(p[3]);
  g_entry.quantize_blocks = reinterpret_cast<decltype(g_entry.quantize_blocks)>(p[4]);
  g_entry.lm_head_logits_scaled = reinterpret_cast<decltype(g_entry.lm_head_logits_scaled)>(p[5]);
  Py_RETURN_NONE;
}

// shape, pages, q, k, v, positions, seq_ids, cos_sin, k_pages, v_pages, page_table, q_out,
// k_out, interleaved, stream
PyObject* rope_append(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const Struct<eagle_shape_t> shape(a[0]);
    const Struct<eagle_pages_t> pages(a[1]);
    const Sizes z(shape.p, pages.p);
    const at::Tensor& pos = tensor(a[5]);
    if (pos.dim() != 1 || pos.size(0) > INT32_MAX) throw BadArgument("positions are [R]");
    const int64_t R = pos.size(0);
    const Rows q = token_rows(a[2], R, z.Hq, z.D, z.type), k = token_rows(a[3], R, z.Hkv, z.D, z.type),
               v = token_rows(a[4], R, z.Hkv, z.D, z.type);
    eagle_rope_t rope{0, 0, 0};
    if (a[7] != Py_None) {
      const at::Tensor& cs = tensor(a[7]);
      if (cs.dim() != 2 || cs.size(0) > INT32_MAX || cs.size(1) > INT32_MAX)
        throw BadArgument("cos_sin is [table_len, rotary_dim]");
      rope.table_len = static_cast<int32_t>(cs.size(0));
      rope.rotary_dim = static_cast<int32_t>(cs.size(1));
      const int truth = PyObject_IsTrue(a[13]);
      if (truth < 0) throw PythonError{};
      rope.interleaved = truth;
    }
    return g_entry.rope_append(
        shape.p, pages.p, &rope, static_cast<int32_t>(R), q.p, q.stride, k.p, k.stride, v.p, v.stride, ints(a[5], {R}),
        ints(a[6], {R}), floats(a[7], {rope.table_len, rope.rotary_dim}), z.pool(a[8]), z.pool(a[9]), z.table(a[10]),
        ptr(a[11], {R, z.Hq, z.D}, z.type), ptr(a[12], {R, z.Hkv, z.D}, z.type), stream(a[14]));
  });
}

// shape, pages, q, k_pages, v_pages, page_table, prefix_lens, shared_len, k_tree, v_tree,
// parents, out, workspace, stream
PyObject* tree_attention_paged(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const Struct<eagle_shape_t> shape(a[0]);
    const Struct<eagle_pages_t> pages(a[1]);
    const Sizes z(shape.p, pages.p);
    int64_t space = 0;
    if (a[12] != Py_None) space = tensor(a[12]).numel();
    return g_entry.tree_attention_paged(
        shape.p, pages.p, z.nodes(a[2], z.Hq), z.pool(a[3]), z.pool(a[4]), z.table(a[5]), ints(a[6], {z.B}),
        integer(a[7]), z.nodes(a[8], z.Hkv), z.nodes(a[9], z.Hkv), ints(a[10], {z.B, z.N}), z.nodes(a[11], z.Hq),
        ptr(a[12], {space}, at::kByte), static_cast<size_t>(space), stream(a[13]));
  });
}

// shape, pages, k_pages, v_pages, page_table, prefix_lens, k_tree, v_tree, hidden, parents,
// accepted_nodes, accept_len, new_prefix_lens, feat, stream
PyObject* commit_accepted_paged(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const Struct<eagle_shape_t> shape(a[0]);
    const Struct<eagle_pages_t> pages(a[1]);
    const Sizes z(shape.p, pages.p);
    return g_entry.commit_accepted_paged(
        shape.p, pages.p, z.pool(a[2]), z.pool(a[3]), z.table(a[4]), ints(a[5], {z.B}), z.nodes(a[6], z.Hkv),
        z.nodes(a[7], z.Hkv), ptr(a[8], {z.B, z.N, z.H}, z.type), ints(a[9], {z.B, z.N}), ints(a[10], {z.B, z.N}),
        ints(a[11], {z.B}), ints(a[12], {z.B}), ptr(a[13], {z.B, z.N, z.H}, z.type), stream(a[14]));
  });
}

void matrix(const at::Tensor& t) {
  if (t.dim() != 2 || t.size(0) > INT32_MAX - 127 || t.size(1) > INT32_MAX - 127) throw BadArgument("matrices are 2-D");
}
bool is(PyObject* o, int64_t rows, int64_t cols) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
}

// x, x_out, scales, stream
PyObject* quantize_rows(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const at::Tensor& x = tensor(a[0]);
    matrix(x);
    const int64_t R = x.size(0), H = x.size(1);
    if (!is(a[1], R, H) || !is(a[2], (H + 127) / 128, (R + 3) / 4 * 4))
      throw BadArgument("x_out is [R, H] and scales [ceil(H / 128), R rounded up to 4]");
    return g_entry.quantize_rows(static_cast<int32_t>(R), static_cast<int32_t>(H), dtype(x),
                                 ptr(a[0], {R, H}, x.scalar_type()), bytes(a[1], {R, H}),
                                 floats(a[2], {(H + 127) / 128, (R + 3) / 4 * 4}), stream(a[3]));
  });
}

// w, w_out, scales, stream
PyObject* quantize_blocks(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    const at::Tensor& w = tensor(a[0]);
    matrix(w);
    const int64_t V = w.size(0), H = w.size(1);
    if (!is(a[1], V, H) || !is(a[2], (V + 127) / 128, (H + 127) / 128))
      throw BadArgument("w_out is [V, H] and scales [ceil(V / 128), ceil(H / 128)]");
    return g_entry.quantize_blocks(static_cast<int32_t>(V), static_cast<int32_t>(H), dtype(w),
                                   ptr(a[0], {V, H}, w.scalar_type()), bytes(a[1], {V, H}),
                                   floats(a[2], {(V + 127) / 128, (H + 127) / 128}), stream(a[3]));
  });
}

// x, x_scales, w, w_scales, logits, stream
PyObject* lm_head_logits_scaled(PyObject*, Args a, Py_ssize_t n) {
  return guarded(n, 6, [&] {
    const at::Tensor& x = tensor(a[0]);
    const at::Tensor& w = tensor(a[2]);
    matrix(x);
    matrix(w);
    const int64_t R = x.size(0), H = x.size(1), V = w.size(0), KB = (H + 127) / 128;
    if (w.size(1) != H || !is(a[1], KB, (R + 3) / 4 * 4) || !is(a[3], (V + 127) / 128, KB) || !is(a[4], R, V))
      throw BadArgument(
          "operands are x [R, H], x_scales [KB, R rounded up to 4], w [V, H], "
          "w_scales [ceil(V / 128), KB] and logits [R, V]");
    return g_entry.lm_head_logits_scaled(static_cast<int32_t>(R), static_cast<int32_t>(H), static_cast<int32_t>(V),
                                         bytes(a[0], {R, H}), floats(a[1], {KB, (R + 3) / 4 * 4}), bytes(a[2], {V, H}),
                                         floats(a[3], {(V + 127) / 128, KB}), floats(a[4], {R, V}), stream(a[5]));
  });
}

template <PyObject* (*F)(PyObject*, Args, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<bind>("bind"),
                           method<rope_append>("rope_append"),
                           method<tree_attention_paged>("tree_attention_paged"),
                           method<commit_accepted_paged>("commit_accepted_paged"),
                           method<quantize_rows>("quantize_rows"),
                           method<quantize_blocks>("quantize_blocks"),
                           method<lm_head_logits_scaled>("lm_head_logits_scaled"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
