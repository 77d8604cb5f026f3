// Python entry of the calls that fill the paged cache, and of those for beams and
// encoder states: argument checks and the call into libvg, natively.  These calls are made once per layer or step, for a
// single token too, where checking ten tensors in Python costs more than the
// kernel (a tensor attribute costs 50 ns there, a tensor with all its checks 20 ns here).
//
// Each function takes its arguments in the order of the binding in vg.py, raises
// ValueError for tensors of the wrong type, shape or place, and returns the
// library's status.  The call runs on the given stream, or the current stream of
// the tensors' device, with that device current.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/vg.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(const char* name, const char* what) {
  throw std::invalid_argument(std::string(name) + ": " + what);
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "a tensor is needed");
  return THPVariable_Unpack(o);
}

// The device of a call: that of its first tensor, which the others share.
struct Device {
  int index = -1;
  // False where t is not on a GPU.
  bool has(const Tensor& t, const char* name) {
    if (!t.is_cuda()) return false;
    const int i = t.get_device();
    if (index < 0) index = i;
    if (i != index) refuse(name, "is on another device than the call's other tensors");
    return true;
  }
};

int32_t* int32s(Device& dev, const Tensor& t, int64_t n, const char* name) {
  if (t.scalar_type() != at::kInt || !dev.has(t, name) || !t.is_contiguous() || t.numel() != n)
    refuse(name, ("a contiguous int32 GPU tensor of " + std::to_string(n) + " elements is needed").c_str());
  return static_cast<int32_t*>(t.data_ptr());
}

int32_t* flag(Device& dev, PyObject* o) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "error_flag");
  if (t.numel() < 1) refuse("error_flag", "an int32 GPU tensor is needed");
  return int32s(dev, t, t.numel(), "error_flag");
}

int as_int(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX) refuse(name, "does not fit 32 bits");
  return static_cast<int>(v);
}

int as_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(name, "an integer is needed");
  }
  return as_int(static_cast<int64_t>(v), name);
}

// Rows [tokens][heads][head_dim] of 16 bits whose heads are contiguous in a token.
struct Rows {
  void* base;
  int tokens, heads, dim;
  int64_t stride;  // elements between tokens
};

Rows rows(Device& dev, PyObject* o, const char* name, at::ScalarType type = at::kBFloat16) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !dev.has(t, name) || t.dim() != 3)
    refuse(name, type == at::kHalf ? "a float16 GPU tensor [tokens][heads][head_dim] is needed"
                                   : "a bfloat16 GPU tensor [tokens][heads][head_dim] is needed");
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
  if (n > 0 && d > 0 && (t.stride(2) != 1 || (h > 1 && t.stride(1) != d)))
    refuse(name, "the heads of a token have to be contiguous");
  return {t.data_ptr(), as_int(n, name), as_int(h, name), as_int(d, name), n > 1 ? t.stride(0) : h * d};
}

vg_paged_kv paged_kv(Device& dev, PyObject* ko, PyObject* vo, PyObject* to) {
  const Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages"), &t = tensor(to, "page_table");
  if (k.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16 || !dev.has(k, "cache") ||
      !dev.has(v, "cache") || k.dim() != 4 || k.sizes() != v.sizes() || !k.is_contiguous() || !v.is_contiguous())
    refuse("cache", "contiguous bfloat16 GPU pools [pages][heads][16][head_dim] are needed");
  if (t.dim() != 2) refuse("page_table", "[batch][max_pages] is needed");
  vg_paged_kv kv;
  kv.k_pages = k.data_ptr();
  kv.v_pages = v.data_ptr();
  kv.page_table = int32s(dev, t, t.numel(), "page_table");
  kv.num_pages = as_int(k.size(0), "cache");
  kv.page_size = as_int(k.size(2), "cache");
  kv.max_pages_per_seq = as_int(t.size(1), "page_table");
  kv.num_kv_heads = as_int(k.size(1), "cache");
  kv.head_dim = as_int(k.size(3), "cache");
  return kv;
}

// The device of a call, made current, and its stream (None: the current one).
struct Place {
  c10::cuda::CUDAGuard guard;
  cudaStream_t stream;
  Place(const Device& dev, PyObject* raw) : guard(static_cast<c10::DeviceIndex>(dev.index)) {
    if (raw == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream().stream();
    } else {
      stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
      if (!stream && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("stream", "a stream's integer is needed");
      }
    }
  }
};

// Other threads of Python run during the library's call: a full launch queue makes
// it wait, perhaps for a host callback that needs the interpreter.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// No C++ exception leaves for Python's C code.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// page_table, num_pages, cached_lens, new_lens, cu_tokens, kv_lens, positions,
// slots, owned, free_pages, free_count, error_flag, stream
PyObject* step_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int {
    Device dev;
    const Tensor& table = tensor(a[0], "page_table");
    if (table.dim() != 2) refuse("page_table", "[batch][max_pages] is needed");
    const int64_t B = table.size(0);
    const Tensor& pos = tensor(a[6], "positions");
    const int64_t T = pos.numel();
    int32_t *owned = nullptr, *pages = nullptr, *count = nullptr;
    int room = 0;
    if (a[8] != Py_None || a[9] != Py_None || a[10] != Py_None) {
      if (a[8] == Py_None || a[9] == Py_None || a[10] == Py_None)
        refuse("owned, free_pages and free_count", "are given together");
      const Tensor& list = tensor(a[9], "free_pages");
      room = as_int(list.numel(), "free_pages");
      owned = int32s(dev, tensor(a[8], "owned"), B, "owned");
      pages = int32s(dev, list, room, "free_pages");
      count = int32s(dev, tensor(a[10], "free_count"), 1, "free_count");
    }
    int32_t* tab = int32s(dev, table, table.numel(), "page_table");
    const int32_t* cached = int32s(dev, tensor(a[2], "cached_lens"), B, "cached_lens");
    const int32_t* fresh = int32s(dev, tensor(a[3], "new_lens"), B, "new_lens");
    int32_t* cu = int32s(dev, tensor(a[4], "cu_tokens"), B + 1, "cu_tokens");
    int32_t* lens = int32s(dev, tensor(a[5], "kv_lens"), B, "kv_lens");
    int32_t* positions = int32s(dev, pos, T, "positions");
    int32_t* slots = int32s(dev, tensor(a[7], "slots"), T, "slots");
    int32_t* err = flag(dev, a[11]);
    const int num_pages = as_int(a[1], "num_pages"), batch = as_int(B, "page_table");
    const int width = as_int(table.size(1), "page_table"), tokens = as_int(T, "positions");
    Place at(dev, a[12]);
    Unlocked free;
    return vg_step_tables(cached, fresh, batch, tab, width,
                          num_pages, owned, pages, room, count, tokens, cu, lens,
                          positions, slots, err, at.stream);
  });
}

// k_pages, v_pages, page_table, q, k, v, slots, q_out, positions, inv_freq,
// freq_axis, interleaved, error_flag, stream
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> int {
    Device dev;
    const vg_paged_kv kv = paged_kv(dev, a[0], a[1], a[2]);
    const Rows k = rows(dev, a[4], "k"), v = rows(dev, a[5], "v");
    if (k.tokens != v.tokens || k.heads != v.heads || k.dim != v.dim || k.heads != kv.num_kv_heads ||
        k.dim != kv.head_dim)
      refuse("k, v", "do not match each other or the cache");
    Rows q = {}, out = {};
    if (a[3] != Py_None) {
      q = rows(dev, a[3], "q");
      out = a[7] == Py_None ? q : rows(dev, a[7], "q_out");
      if (q.tokens != k.tokens || q.dim != k.dim || out.tokens != k.tokens || out.heads != q.heads ||
          out.dim != q.dim)
        refuse("q, q_out", "do not match each other or k");
    }
    const int32_t *positions = nullptr, *axis = nullptr;
    const float* freq = nullptr;
    int axes = 0, half = 0;
    int64_t pos_stride = 0;
    if (a[9] != Py_None) {
      const Tensor& f = tensor(a[9], "inv_freq");
      if (f.scalar_type() != at::kFloat || !dev.has(f, "inv_freq") || !f.is_contiguous())
        refuse("inv_freq", "a contiguous float32 GPU tensor is needed");
      if (a[8] == Py_None) refuse("positions", "are needed with inv_freq");
      const Tensor& pos = tensor(a[8], "positions");
      if (pos.scalar_type() != at::kInt || !dev.has(pos, "positions") || pos.dim() < 1 || pos.dim() > 2 ||
          pos.size(-1) != k.tokens || (k.tokens > 1 && pos.stride(-1) != 1))
        refuse("positions", "int32 [tokens] or [axes][tokens] on the GPU is needed");
      axes = pos.dim() == 1 ? 1 : as_int(pos.size(0), "positions");
      pos_stride = axes == 1 ? k.tokens : pos.stride(0);
      half = as_int(f.numel(), "inv_freq");
      positions = static_cast<const int32_t*>(pos.data_ptr());
      freq = static_cast<const float*>(f.data_ptr());
      if (a[10] != Py_None) axis = int32s(dev, tensor(a[10], "freq_axis"), half, "freq_axis");
    }
    const int32_t* slots = int32s(dev, tensor(a[6], "slots"), k.tokens, "slots");
    int32_t* err = flag(dev, a[12]);
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) {
      PyErr_Clear();
      refuse("interleaved", "true or false is needed");
    }
    Place at(dev, a[13]);
    Unlocked free;
    return vg_rope_append(&kv, q.base, q.stride, k.base, k.stride, v.base, v.stride, out.base, out.stride,
                          k.tokens, q.heads, positions, pos_stride, axes, freq, axis, 2 * half,
                          interleaved, slots, err, at.stream);
  });
}

// k_pages, v_pages, page_table, q, cu_q, kv_lens, softmax_scale, out, lse,
// workspace, error_flag, stream
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    Device dev;
    const vg_paged_kv kv = paged_kv(dev, a[0], a[1], a[2]);
    const Rows q = rows(dev, a[3], "q"), out = rows(dev, a[7], "out");
    if (q.tokens != out.tokens || q.heads != out.heads || q.dim != out.dim || q.dim != kv.head_dim)
      refuse("out", "it or the cache does not match q");
    const Tensor& lens = tensor(a[5], "kv_lens");
    const int64_t B = lens.numel();
    if (tensor(a[2], "page_table").size(0) != B) refuse("page_table", "has another batch size");
    const int32_t* kv_lens = int32s(dev, lens, B, "kv_lens");
    const int32_t* cu_q = int32s(dev, tensor(a[4], "cu_q"), B + 1, "cu_q");
    float* lse = nullptr;
    if (a[8] != Py_None) {
      const Tensor& t = tensor(a[8], "lse");
      if (t.scalar_type() != at::kFloat || !dev.has(t, "lse") || !t.is_contiguous() ||
          t.numel() != (int64_t)q.tokens * q.heads)
        refuse("lse", "a contiguous float32 GPU tensor [tokens][heads] is needed");
      lse = static_cast<float*>(t.data_ptr());
    }
    const int batch = as_int(B, "kv_lens");
    const Tensor& ws = tensor(a[9], "workspace");
    if (!dev.has(ws, "workspace") || !ws.is_contiguous()) refuse("workspace", "a contiguous GPU tensor is needed");
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("softmax_scale", "a number is needed");
    }
    int32_t* err = flag(dev, a[10]);
    Place at(dev, a[11]);
    Unlocked free;
    return vg_chunk_attention(&kv, q.base, q.stride, cu_q, kv_lens, batch, q.tokens,
                              q.heads, static_cast<float>(scale), out.base, out.stride, lse, ws.data_ptr(),
                              ws.nbytes(), err, at.stream);
  });
}

// Marks of one byte each: a contiguous bool or uint8 tensor of n elements, or None.
uint8_t* marks(Device& dev, PyObject* o, int64_t n, const char* name) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, name);
  if ((t.scalar_type() != at::kBool && t.scalar_type() != at::kByte) || !dev.has(t, name) || !t.is_contiguous() ||
      t.numel() != n)
    refuse(name, ("a contiguous bool or uint8 GPU tensor of " + std::to_string(n) + " elements is needed").c_str());
  return static_cast<uint8_t*>(t.data_ptr());
}

float* floats(Device& dev, const Tensor& t, int64_t n, const char* name) {
  if (t.scalar_type() != at::kFloat || !dev.has(t, name) || !t.is_contiguous() || t.numel() != n)
    refuse(name, ("a contiguous float32 GPU tensor of " + std::to_string(n) + " elements is needed").c_str());
  return static_cast<float*>(t.data_ptr());
}

const Tensor& workspace(Device& dev, PyObject* o) {
  const Tensor& t = tensor(o, "workspace");
  if (!dev.has(t, "workspace") || !t.is_contiguous()) refuse("workspace", "a contiguous GPU tensor is needed");
  return t;
}

// q, k, v, cu_q, state_starts, state_lens, softmax_scale, out, mask, lse,
// workspace, error_flag, stream
PyObject* cross_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int {
    Device dev;
    const at::ScalarType type = tensor(a[0], "q").scalar_type() == at::kHalf ? at::kHalf : at::kBFloat16;
    const Rows q = rows(dev, a[0], "q", type), k = rows(dev, a[1], "k", type), v = rows(dev, a[2], "v", type);
    const Rows out = rows(dev, a[7], "out", type);
    if (q.tokens != out.tokens || q.heads != out.heads || q.dim != out.dim) refuse("out", "does not match q");
    if (k.tokens != v.tokens || k.heads != v.heads || k.dim != v.dim || k.dim != q.dim)
      refuse("k, v", "do not match each other or q");
    const Tensor& lens = tensor(a[5], "state_lens");
    const int64_t E = lens.numel();
    const int32_t* state_lens = int32s(dev, lens, E, "state_lens");
    const int32_t* state_starts = int32s(dev, tensor(a[4], "state_starts"), E, "state_starts");
    const int32_t* cu_q = int32s(dev, tensor(a[3], "cu_q"), E + 1, "cu_q");
    const uint8_t* mask = marks(dev, a[8], k.tokens, "mask");
    float* lse = a[9] == Py_None ? nullptr : floats(dev, tensor(a[9], "lse"), (int64_t)q.tokens * q.heads, "lse");
    const int batch = as_int(E, "state_lens");
    const Tensor& ws = workspace(dev, a[10]);
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("softmax_scale", "a number is needed");
    }
    int32_t* err = flag(dev, a[11]);
    Place at(dev, a[12]);
    Unlocked free;
    return vg_cross_attention(q.base, q.stride, k.base, k.stride, v.base, v.stride,
                              type == at::kHalf ? VG_TYPE_FP16 : VG_TYPE_BF16, cu_q, state_starts, state_lens, mask,
                              batch, q.tokens, k.tokens, q.heads, k.heads, q.dim, static_cast<float>(scale), out.base,
                              out.stride, lse, ws.data_ptr(), ws.nbytes(), err, at.stream);
  });
}

// logits, scores, ended, end_token, out_scores, out_tokens, out_parents,
// out_ended, workspace, error_flag, stream
PyObject* beam_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> int {
    Device dev;
    const Tensor &x = tensor(a[0], "logits"), &s = tensor(a[1], "scores"), &o = tensor(a[4], "out_scores");
    const at::ScalarType t = x.scalar_type();
    if ((t != at::kFloat && t != at::kBFloat16 && t != at::kHalf) || !dev.has(x, "logits") || x.dim() != 2 ||
        (x.size(1) > 1 && x.stride(1) != 1))
      refuse("logits", "a float32, bfloat16 or float16 GPU tensor [batch * beams][vocab] is needed, rows contiguous");
    if (s.dim() != 2 || o.dim() != 2 || s.size(0) != o.size(0) || s.numel() != x.size(0))
      refuse("scores, out_scores", "[batch][beams] and [batch][num_out] are needed, a row of logits for every beam");
    const int64_t B = s.size(0), W = s.size(1), K = o.size(1);
    const float* scores = floats(dev, s, B * W, "scores");
    const uint8_t* ended = marks(dev, a[2], B * W, "ended");
    float* out_scores = floats(dev, o, B * K, "out_scores");
    int32_t* tokens = int32s(dev, tensor(a[5], "out_tokens"), B * K, "out_tokens");
    int32_t* parents = int32s(dev, tensor(a[6], "out_parents"), B * K, "out_parents");
    uint8_t* out_ended = marks(dev, a[7], B * K, "out_ended");
    const Tensor& ws = workspace(dev, a[8]);
    int32_t* err = flag(dev, a[9]);
    const long long end = PyLong_AsLongLong(a[3]);
    if ((end == -1 && PyErr_Occurred()) || end < INT32_MIN || end > INT32_MAX) {
      PyErr_Clear();
      refuse("end_token", "an integer of 32 bits is needed");
    }
    const int batch = as_int(B, "scores"), beams = as_int(W, "scores"), vocab = as_int(x.size(1), "logits");
    const int out = as_int(K, "out_scores");
    const int type = t == at::kFloat ? VG_TYPE_FP32 : t == at::kBFloat16 ? VG_TYPE_BF16 : VG_TYPE_FP16;
    Place at(dev, a[10]);
    Unlocked free;
    return vg_beam_select(x.data_ptr(), type, x.size(0) > 1 ? x.stride(0) : vocab, scores, ended,
                          static_cast<int>(end), batch, beams, vocab, out, out_scores, tokens, parents, out_ended,
                          ws.data_ptr(), ws.nbytes(), err, at.stream);
  });
}

// page_table, num_pages, parents, lens, owned, free_pages, free_count, copies,
// error_flag, stream
PyObject* beam_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    Device dev;
    const Tensor &table = tensor(a[0], "page_table"), &par = tensor(a[2], "parents"), &list = tensor(a[5], "free_pages");
    if (table.dim() != 2) refuse("page_table", "[batch * beams][max_pages] is needed");
    if (par.dim() != 2) refuse("parents", "[batch][beams] is needed");
    const int64_t R = table.size(0);
    int32_t* tab = int32s(dev, table, table.numel(), "page_table");
    const int32_t* parents = int32s(dev, par, R, "parents");
    int32_t* lens = int32s(dev, tensor(a[3], "lens"), R, "lens");
    int32_t* owned = int32s(dev, tensor(a[4], "owned"), R, "owned");
    int32_t* pages = int32s(dev, list, list.numel(), "free_pages");
    int32_t* count = int32s(dev, tensor(a[6], "free_count"), 1, "free_count");
    int32_t* copies = int32s(dev, tensor(a[7], "copies"), 3 * R, "copies");
    int32_t* err = flag(dev, a[8]);
    const int num_pages = as_int(a[1], "num_pages"), width = as_int(table.size(1), "page_table");
    const int batch = as_int(par.size(0), "parents"), beams = as_int(par.size(1), "parents");
    const int room = as_int(list.numel(), "free_pages");
    Place at(dev, a[9]);
    Unlocked free;
    return vg_beam_tables(parents, batch, beams, lens, tab, width, num_pages, owned, pages, room, count, copies, err,
                          at.stream);
  });
}

// lists of k_pages and of v_pages, copies, error_flag, stream
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> int {
    Device dev;
    if (!PyList_Check(a[0]) || !PyList_Check(a[1]) || PyList_GET_SIZE(a[0]) != PyList_GET_SIZE(a[1]) ||
        PyList_GET_SIZE(a[0]) == 0)
      refuse("kv", "a cache, or a list of them, is needed");
    const Py_ssize_t layers = PyList_GET_SIZE(a[0]);
    const Tensor& like = tensor(PyList_GET_ITEM(a[0], 0), "k_pages");
    std::vector<void*> pools[2];
    for (int v = 0; v < 2; ++v)
      for (Py_ssize_t i = 0; i < layers; ++i) {
        const Tensor& t = tensor(PyList_GET_ITEM(a[v], i), v ? "v_pages" : "k_pages");
        if (t.scalar_type() != at::kBFloat16 || !dev.has(t, "cache") || t.dim() != 4 || t.size(2) != 16 ||
            !t.is_contiguous() || t.sizes() != like.sizes())
          refuse("cache", "contiguous bfloat16 GPU pools [pages][heads][16][head_dim] of one shape are needed");
        pools[v].push_back(t.data_ptr());
      }
    const Tensor& c = tensor(a[2], "copies");
    if (c.dim() != 2 || c.size(1) != 3) refuse("copies", "[copies][3] is needed");
    const int32_t* copies = int32s(dev, c, c.numel(), "copies");
    int32_t* err = flag(dev, a[3]);
    const int num = as_int(c.size(0), "copies"), pages = as_int(like.size(0), "cache");
    const int heads = as_int(like.size(1), "cache"), dim = as_int(like.size(3), "cache");
    Place at(dev, a[4]);
    Unlocked free;
    return vg_copy_pages(pools[0].data(), pools[1].data(), static_cast<int>(layers), pages, heads, dim, copies, num,
                         err, at.stream);
  });
}

PyMethodDef methods[] = {
    {"step_tables", (PyCFunction)(void (*)(void))step_tables, METH_FASTCALL, "see vg.step_tables"},
    {"rope_append", (PyCFunction)(void (*)(void))rope_append, METH_FASTCALL, "see vg.rope_append"},
    {"chunk_attention", (PyCFunction)(void (*)(void))chunk_attention, METH_FASTCALL, "see vg.chunk_attention"},
    {"cross_attention", (PyCFunction)(void (*)(void))cross_attention, METH_FASTCALL, "see vg.cross_attention"},
    {"beam_select", (PyCFunction)(void (*)(void))beam_select, METH_FASTCALL, "see vg.beam_select"},
    {"beam_tables", (PyCFunction)(void (*)(void))beam_tables, METH_FASTCALL, "see vg.beam_tables"},
    {"copy_pages", (PyCFunction)(void (*)(void))copy_pages, METH_FASTCALL, "see vg.copy_pages"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "vg_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_vg_binding(void) { return PyModule_Create(&module); }
