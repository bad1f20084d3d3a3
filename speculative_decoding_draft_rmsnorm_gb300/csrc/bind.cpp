// bind.cpp -- the argument marshalling of decode.py's calls, as a CPython module over PyTorch tensors.
//
// A decode step makes a handful of these calls, each a few microseconds of GPU time; checked and marshalled in
// Python and ctypes one cost 22 us of host time on the Arm host (6 of them the call itself), here about 6.
// Nothing is computed here: every function checks its tensors, allocates the outputs and the workspace that were
// not given, calls the C entry point on the current stream of the tensors' device, and counts what it wrote as changed. A function returns its
// outputs, or the C entry point's status where that is not 0; wrong arguments raise TypeError or ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <string>
#include <vector>

#include "../../include/dflash.h"

namespace {

struct Raised {};  // a Python error is set

template <typename... A>
[[noreturn]] void raise(PyObject* type, const char* format, A... args) {
  PyErr_Format(type, format, args...);
  throw Raised{};
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// Where a call runs: the device of its first tensor.
struct Place {
  c10::Device device;
  explicit Place(const at::Tensor& first) : device(first.device()) {
    if (!device.is_cuda()) raise(PyExc_ValueError, "tensors must live on a CUDA device");
  }
  cudaStream_t stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    // past the dispatcher: 0.7 us instead of 1.5
    return at::Tensor(at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                type, std::nullopt));
  }

  // A contiguous tensor in bytes [at, ..) of another's storage.
  static at::Tensor slice(const at::Tensor& whole, int64_t at, at::IntArrayRef shape, at::ScalarType type) {
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                            c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    return t;
  }

  // The address of a tensor of that type on this device.
  void* plain(const char* name, const at::Tensor& t, at::ScalarType type, bool contiguous = true) const {
    if (t.scalar_type() != type)
      raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.device() != device)
      raise(PyExc_ValueError, "%s is on %s, the call's tensors are on %s", name, t.device().str().c_str(), device.str().c_str());
    if (contiguous && !t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
  }
  // The same with a shape; null for None.
  void* address(const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef shape, bool contiguous = true) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    void* p = plain(name, t, type, contiguous);
    if (t.sizes() != shape)
      raise(PyExc_ValueError, "%s has shape %s, expected %s", name, text(t.sizes()).c_str(), text(shape).c_str());
    return p;
  }
};

void rows(const at::Tensor& t, const char* name, int64_t dims) {
  if (t.dim() != dims) raise(PyExc_ValueError, "%s must have %d dimensions, got %d", name, static_cast<int>(dims), static_cast<int>(t.dim()));
  if (t.size(-1) > 1 && t.stride(-1) != 1) raise(PyExc_ValueError, "%s: the last dimension must be contiguous", name);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, "%s does not fit in 32 bits", name);
  return static_cast<int>(v);
}
int dim32(int64_t v, const char* name) {
  if (v > INT32_MAX) raise(PyExc_ValueError, "%s is too large", name);
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// The workspace given, or new memory of `need` bytes, which belongs to the current stream and is free for what
// follows on it when the call returns.
struct Scratch {
  c10::DataPtr own;
  void* p = nullptr;
  size_t bytes = 0;
};
template <typename Need>
bool scratch(const Place& at, PyObject* o, Need need, Scratch* s) {
  if (o == Py_None) {
    const size_t n = need();
    if (n == 0) return false;
    s->own = c10::cuda::CUDACachingAllocator::get()->allocate(n);
    s->p = s->own.get();
    s->bytes = n;
  } else {
    const at::Tensor& t = tensor(o, "workspace");
    s->p = at.plain("workspace", t, at::kByte);
    s->bytes = t.nbytes();
  }
  return true;
}

// The call, without the interpreter's lock, on the current stream of the place.
template <typename F>
int run(const Place& at, F call) {
  struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  };
  const cudaStream_t stream = at.stream();
  Unlocked unlocked;
  return call(stream);
}

// Tensors that a call wrote (None: nothing): what autograd keeps of them for a backward pass is out of date.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(std::initializer_list<PyObject*> list) {
  for (PyObject* o : list)
    if (THPVariable_Check(o)) written(THPVariable_Unpack(o));
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
// The object given, or the tensor made in its place.
PyObject* given(PyObject* o, const at::Tensor& made) {
  if (o != Py_None) return Py_NewRef(o);
  return made.defined() ? wrap(made) : Py_NewRef(Py_None);
}

struct Buffer : Py_buffer {
  explicit Buffer(PyObject* o, int flags = PyBUF_C_CONTIGUOUS) {
    if (PyObject_GetBuffer(o, this, flags) != 0) throw Raised{};
  }
  ~Buffer() { PyBuffer_Release(this); }
};

// A small table of whole numbers in 0 .. 255 from a buffer of any integer type.
std::vector<uint8_t> small_table(PyObject* o, const char* name) {
  const Buffer b(o, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT);
  const std::string type = b.format ? b.format : "B";
  if (type.size() != 1 || !std::strchr("bBhHiIlLqQ", type[0])) raise(PyExc_TypeError, "%s must hold integers", name);
  const bool sign = std::strchr("bhilq", type[0]) != nullptr;
  std::vector<uint8_t> out(static_cast<size_t>(b.len / b.itemsize));
  for (size_t i = 0; i < out.size(); ++i) {
    uint64_t x = 0;  // little-endian
    std::memcpy(&x, static_cast<const char*>(b.buf) + i * b.itemsize, static_cast<size_t>(b.itemsize));
    if (x > 255 || (sign && b.itemsize == 1 && x > 127)) raise(PyExc_ValueError, "%s: entry %d is out of range", name, static_cast<int>(i));
    out[i] = static_cast<uint8_t>(x);
  }
  return out;
}

// q, positions, inv_freq (buffer of doubles), k, v, q_out, k_out, v_out, slot, amplitude, interleaved, inverse, status
// and with several axes: the axis of every pair (buffer of integers)
template <bool AXES>
PyObject* rotary_any(PyObject* const* a) {
  struct Part {
    const void* src = nullptr;
    void* dst = nullptr;
    int64_t tok = 0, head = 0, out_tok = 0, out_head = 0, heads = 0;
  } q, k, v;
  PyObject *oq = a[0], *ok = a[3], *ov = a[4], *slot = a[8];
  if (oq == Py_None && ok == Py_None) raise(PyExc_ValueError, "pass q, k or both");
  const bool has_q = oq != Py_None, has_k = ok != Py_None, has_v = ov != Py_None;
  const at::Tensor& first = tensor(has_q ? oq : ok, has_q ? "q" : "k");
  const Place at(first);
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  const at::ScalarType type = first.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) raise(PyExc_TypeError, "rotary takes bfloat16 or float32, got %s", c10::toString(type));
  if (has_v != (a[7] != Py_None)) raise(PyExc_ValueError, "pass v and v_out together");
  if (has_v && !has_k) raise(PyExc_ValueError, "v needs k");
  const bool slots = slot != Py_None;
  if (slots && (!has_k || a[6] == Py_None)) raise(PyExc_ValueError, "slot needs k and k_out");
  rows(first, has_q ? "q" : "k", 3);
  const int64_t n = first.size(0), dh = first.size(2);
  int64_t capacity = n;
  at::Tensor new_q, new_k;
  if (has_q) {
    if (a[5] == Py_None) new_q = at.empty(first.sizes(), type);
    const at::Tensor& out = a[5] == Py_None ? new_q : tensor(a[5], "q_out");
    rows(out, "q_out", 3);
    if (out.sizes() != first.sizes()) raise(PyExc_ValueError, "q_out has shape %s, expected %s", text(out.sizes()).c_str(), text(first.sizes()).c_str());
    q = Part{first.data_ptr(), at.plain("q_out", out, type, false), first.stride(0), first.stride(1), out.stride(0), out.stride(1), first.size(1)};
  }
  auto store = [&](const at::Tensor& t, const char* name, const at::Tensor& like) {
    at::Tensor s = t;
    if (t.dim() == 4) {
      if (!t.is_contiguous()) raise(PyExc_ValueError, "%s: pools must be contiguous", name);
      s = t.view({t.size(0) * t.size(1), t.size(2), t.size(3)});
    }
    rows(s, name, 3);
    if (s.size(1) != like.size(1) || s.size(2) != dh || (!slots && s.size(0) != n))
      raise(PyExc_ValueError, "%s must be [%s, Hkv, Dh]", name, slots ? "capacity" : "n");
    return s;
  };
  if (has_k) {
    const at::Tensor& t = tensor(ok, "k");
    rows(t, "k", 3);
    if (t.size(0) != n || t.size(2) != dh) raise(PyExc_ValueError, "k must be [n, Hkv, Dh] like q");
    if (a[6] == Py_None) new_k = at.empty(t.sizes(), type);
    const at::Tensor out = store(a[6] == Py_None ? new_k : tensor(a[6], "k_out"), "k_out", t);
    capacity = out.size(0);
    k = Part{at.plain("k", t, type, false), at.plain("k_out", out, type, false), t.stride(0), t.stride(1), out.stride(0), out.stride(1), t.size(1)};
    if (has_v) {
      const at::Tensor& x = tensor(ov, "v");
      rows(x, "v", 3);
      if (x.sizes() != t.sizes()) raise(PyExc_ValueError, "v has shape %s, expected %s", text(x.sizes()).c_str(), text(t.sizes()).c_str());
      const at::Tensor vo = store(tensor(a[7], "v_out"), "v_out", t);
      if (vo.size(0) != capacity) raise(PyExc_ValueError, "v_out must have as many rows as k_out");
      v = Part{at.plain("v", x, type, false), at.plain("v_out", vo, type, false), x.stride(0), x.stride(1), vo.stride(0), vo.stride(1), 0};
    }
  }
  const int32_t* pos;
  int64_t axis_stride = 0;
  int axes = 0;
  std::vector<uint8_t> pair_axis;
  if constexpr (AXES) {
    const at::Tensor& p = tensor(a[1], "positions");
    if (p.dim() != 2 || p.size(1) != n) raise(PyExc_ValueError, "positions must be [axes, n], got %s", text(p.sizes()).c_str());
    pos = static_cast<const int32_t*>(at.plain("positions", p, at::kInt, false));
    if (n > 1 && p.stride(1) != 1) raise(PyExc_ValueError, "positions: those of an axis must be contiguous");
    axes = dim32(p.size(0), "axes"), axis_stride = axes > 1 ? p.stride(0) : n;
    pair_axis = small_table(a[13], "axes");
  } else {
    pos = static_cast<const int32_t*>(at.address("positions", a[1], at::kInt, {n}));
  }
  const auto* slot_p = static_cast<const int32_t*>(at.address("slot", slot, at::kInt, {n}));
  auto* status = static_cast<int32_t*>(at.address("status", a[12], at::kInt, {1}));
  const double amplitude = number(a[9]);
  const int inter = truth(a[10]), inverse = truth(a[11]);
  const int hq = dim32(q.heads, "Hq"), hkv = dim32(k.heads, "Hkv"), d = dim32(dh, "Dh");
  const Buffer freq(a[2]);
  const int rotary_dim = static_cast<int>(2 * (freq.len / static_cast<Py_ssize_t>(sizeof(double))));
  if (AXES && pair_axis.size() * 2 != static_cast<size_t>(rotary_dim))
    raise(PyExc_ValueError, "axes has %d entries, inv_freq %d", static_cast<int>(pair_axis.size()), rotary_dim / 2);
  if (c10::GradMode::is_enabled())
    for (int i : {0, 3, 4, 5, 6, 7})
      if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad())
        raise(PyExc_ValueError, "rotary records no gradient: call it under torch.no_grad() or with detached tensors "
                                "(inverse=True gives the gradient of the inputs)");
  const int rc = run(at, [&](cudaStream_t stream) {
    const auto* f = static_cast<const double*>(freq.buf);
    const int dtype = type == at::kFloat ? DFLASH_OUT_F32 : DFLASH_OUT_BF16;
    if constexpr (AXES)
      return dflash_rotary_axes(q.src, q.tok, q.head, q.dst, q.out_tok, q.out_head, hq, k.src, k.tok, k.head, k.dst, k.out_tok, k.out_head,
                                hkv, v.src, v.tok, v.head, v.dst, v.out_tok, v.out_head, pos, axis_stride, axes, pair_axis.data(), slot_p, n,
                                capacity, d, rotary_dim, f, amplitude, inter, inverse, dtype, status, stream);
    return dflash_rotary(q.src, q.tok, q.head, q.dst, q.out_tok, q.out_head, hq, k.src, k.tok, k.head, k.dst, k.out_tok, k.out_head, hkv,
                         v.src, v.tok, v.head, v.dst, v.out_tok, v.out_head, pos, slot_p, n, capacity, d, rotary_dim, f, amplitude, inter,
                         inverse, dtype, status, stream);
  });
  if (rc) return PyLong_FromLong(rc);
  if (has_q) written({a[5]});
  if (has_k) written({a[6], a[7]});
  written({a[12]});
  return Py_BuildValue("(NN)", has_q ? given(a[5], new_q) : Py_NewRef(Py_None), has_k ? given(a[6], new_k) : Py_NewRef(Py_None));
}

PyObject* rotary(PyObject* const* a) { return rotary_any<false>(a); }
PyObject* rotary_axes(PyObject* const* a) { return rotary_any<true>(a); }

// x, weight, residual, out dtype (None: x's), group_size, eps, out, residual_out, scales, status
PyObject* rms_norm(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight");
  const Place at(x);
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  rows(x, "x", 2);
  const at::ScalarType type = x.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) raise(PyExc_TypeError, "rms_norm takes bfloat16 or float32, got %s", c10::toString(type));
  if (w.scalar_type() != at::kBFloat16 && w.scalar_type() != at::kFloat)
    raise(PyExc_TypeError, "weight must be bfloat16 or float32, got %s", c10::toString(w.scalar_type()));
  const int64_t n = x.size(0), d = x.size(1);
  const auto code = [](at::ScalarType t) { return t == at::kFloat ? DFLASH_OUT_F32 : DFLASH_OUT_BF16; };
  const int dtype = code(type), out_dtype = a[3] == Py_None ? dtype : small(a[3], "out_dtype");
  const bool eight = out_dtype == DFLASH_OUT_E4M3;
  if (!eight && out_dtype != dtype) raise(PyExc_ValueError, "out_dtype must be OUT_E4M3 or the input's type");
  const at::ScalarType out_type = eight ? at::kFloat8_e4m3fn : type;
  const int group = small(a[4], "group_size"), width = dim32(d, "d");
  const float eps = static_cast<float>(number(a[5]));
  auto* status = static_cast<int32_t*>(at.address("status", a[9], at::kInt, {1}));
  const void* pw = at.address("weight", a[1], w.scalar_type(), {d});
  struct Matrix {
    at::Tensor t;
    void* p = nullptr;
    int64_t stride = 0;
  };
  auto matrix = [&](const char* name, PyObject* o, at::ScalarType t) {  // [n, d] that was given
    const at::Tensor& m = tensor(o, name);
    rows(m, name, 2);
    if (m.sizes() != x.sizes()) raise(PyExc_ValueError, "%s has shape %s, expected %s", name, text(m.sizes()).c_str(), text(x.sizes()).c_str());
    void* p = at.plain(name, m, t, false);
    return Matrix{m, p, m.stride(0)};
  };
  auto made = [&](const char* name, PyObject* o, at::ScalarType t) {
    if (o != Py_None) return matrix(name, o, t);
    at::Tensor m = at.empty(x.sizes(), t);
    return Matrix{m, m.data_ptr(), d};
  };
  if (a[2] == Py_None && a[7] != Py_None) raise(PyExc_ValueError, "residual_out needs a residual");
  if (!eight && a[8] != Py_None) raise(PyExc_ValueError, "scales need out_dtype=OUT_E4M3");
  if (group < 0 || group % 16) raise(PyExc_ValueError, "group_size must be 0 or a multiple of 16");
  if (group && !eight) raise(PyExc_ValueError, "group_size needs out_dtype=OUT_E4M3");
  if (c10::GradMode::is_enabled())
    for (int i : {0, 1, 2, 6, 7})
      if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i]).requires_grad())
        raise(PyExc_ValueError, "rms_norm records no gradient: call it under torch.no_grad() or with detached tensors");
  Matrix r, ro;
  if (a[2] != Py_None) r = matrix("residual", a[2], type), ro = made("residual_out", a[7], type);
  const Matrix out = made("out", a[6], out_type);
  at::Tensor new_scales;
  float* scales = nullptr;
  if (eight) {
    if (a[8] == Py_None) {
      if (group) new_scales = at.empty({n, (d + group - 1) / group}, at::kFloat);
      else new_scales = at.empty({n, 1}, at::kFloat);
      scales = static_cast<float*>(new_scales.data_ptr());
    } else {
      scales = static_cast<float*>(at.address("scales", a[8], at::kFloat, {n, group ? (d + group - 1) / group : 1}));
    }
  }
  const int rc = run(at, [&](cudaStream_t stream) {
    return dflash_rms_norm(x.data_ptr(), x.stride(0), r.p, r.stride, pw, ro.p, ro.stride, out.p, out.stride, scales, n, width, dtype,
                           code(w.scalar_type()), out_dtype, group, eps, status, stream);
  });
  if (rc) return PyLong_FromLong(rc);
  written({a[6], a[7], a[8], a[9]});
  return Py_BuildValue("(NNN)", given(a[6], out.t), given(a[7], ro.t), given(a[8], new_scales));
}

// block_table, seq_lens, group_start_loc, page_size, out, status
PyObject* shared_prefixes(PyObject* const* a) {
  const at::Tensor &table = tensor(a[0], "block_table"), &starts = tensor(a[2], "group_start_loc");
  const Place at(table);
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  if (table.dim() != 2 || starts.dim() != 1 || starts.size(0) < 1)
    raise(PyExc_ValueError, "block_table must be [N, max_pages] and group_start_loc [groups + 1]");
  const int n = dim32(table.size(0), "N"), width = dim32(table.size(1), "max_pages"), groups = dim32(starts.size(0) - 1, "groups");
  if (n && width > 1 && table.stride(1) != 1) raise(PyExc_ValueError, "block_table: a row must be contiguous");
  const auto* pt = static_cast<const int32_t*>(at.plain("block_table", table, at::kInt, false));
  tensor(a[1], "seq_lens");
  const auto* pl = static_cast<const int32_t*>(at.address("seq_lens", a[1], at::kInt, {n}));
  const auto* ps = static_cast<const int32_t*>(at.plain("group_start_loc", starts, at::kInt));
  const int page = small(a[3], "page_size");
  auto* status = static_cast<int32_t*>(at.address("status", a[5], at::kInt, {1}));
  at::Tensor made;
  if (a[4] == Py_None) made = at.empty({groups}, at::kInt);
  auto* out = static_cast<int32_t*>(made.defined() ? made.data_ptr() : at.address("out", a[4], at::kInt, {groups}));
  const int rc = run(at, [&](cudaStream_t stream) {
    return dflash_shared_prefixes(pt, n > 1 ? table.stride(0) : width, pl, ps, n, groups, width, page, out, status, stream);
  });
  if (rc) return PyLong_FromLong(rc);
  written({a[4], a[5]});
  return given(a[4], made);
}

// q, k_pool, v_pool, block_table, seq_lens, max_ctx_len, out, lse, return_lse, workspace, scale, window, out_dtype, status
// and of a call that shares prefixes: group_start_loc, prefix_lens, flags
template <bool SHARED>
PyObject* decode_attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q");
  const Place at(q);
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  rows(q, "q", 3);
  const at::Tensor &kp = tensor(a[1], "k_pool"), &table = tensor(a[3], "block_table");
  if (kp.dim() != 4 || table.dim() != 2) raise(PyExc_ValueError, "k_pool must be [num_pages, page_size, Hkv, Dh] and block_table [N, max_pages]");
  const int n = dim32(q.size(0), "N"), hq = dim32(q.size(1), "Hq"), dh = dim32(q.size(2), "Dh");
  const int page = dim32(kp.size(1), "page_size"), hkv = dim32(kp.size(2), "Hkv"), width = dim32(table.size(1), "max_pages");
  if (kp.size(3) != dh) raise(PyExc_ValueError, "q has head_dim %d, the pools %d", dh, static_cast<int>(kp.size(3)));
  if (hq > 1 && n && q.stride(1) != dh) raise(PyExc_ValueError, "q: the heads of a sequence must be contiguous");
  if (width > 1 && table.stride(1) != 1) raise(PyExc_ValueError, "block_table: a row must be contiguous");
  const int dtype = small(a[12], "out_dtype");
  if (dtype != DFLASH_OUT_BF16 && dtype != DFLASH_OUT_F32) raise(PyExc_ValueError, "out_dtype must be OUT_BF16 or OUT_F32");
  const at::ScalarType type = dtype == DFLASH_OUT_F32 ? at::kFloat : at::kBFloat16;
  const auto* pq = static_cast<const dflash_bf16*>(at.plain("q", q, at::kBFloat16, false));
  const auto* pk = static_cast<const dflash_bf16*>(at.plain("k_pool", kp, at::kBFloat16));
  const auto* pv = static_cast<const dflash_bf16*>(at.address("v_pool", a[2], at::kBFloat16, kp.sizes()));
  const auto* pt = static_cast<const int32_t*>(at.address("block_table", a[3], at::kInt, {n, width}, false));
  const auto* pl = static_cast<const int32_t*>(at.address("seq_lens", a[4], at::kInt, {n}));
  auto* status = static_cast<int32_t*>(at.address("status", a[13], at::kInt, {1}));
  const int longest = small(a[5], "max_ctx_len"), window = small(a[11], "window");
  const float scale = static_cast<float>(number(a[10]));
  const int32_t *starts = nullptr, *prefixes = nullptr;
  int groups = 0, flags = 0;
  if constexpr (SHARED) {
    flags = small(a[16], "flags");
    const at::Tensor& t = tensor(a[14], "group_start_loc");
    if (t.dim() != 1 || t.size(0) < 1) raise(PyExc_ValueError, "group_start_loc must be [groups + 1]");
    groups = dim32(t.size(0) - 1, "groups");
    starts = static_cast<const int32_t*>(at.plain("group_start_loc", t, at::kInt));
    tensor(a[15], "prefix_lens");
    prefixes = static_cast<const int32_t*>(at.address("prefix_lens", a[15], at::kInt, {groups}));
  }
  at::Tensor new_out, new_lse;
  if (a[6] == Py_None) new_out = at.empty(q.sizes(), type);
  if (a[7] == Py_None && truth(a[8])) new_lse = at.empty({n, hq}, at::kFloat);
  void* out = a[6] == Py_None ? new_out.data_ptr() : at.address("out", a[6], type, q.sizes());
  auto* lse = static_cast<float*>(new_lse.defined() ? new_lse.data_ptr() : at.address("lse", a[7], at::kFloat, {n, hq}));
  Scratch ws;
  const auto need = [&] {
    return SHARED ? dflash_shared_workspace_size(n, groups, hq, hkv, dh, longest, window)
                  : dflash_decode_workspace_size(n, hq, hkv, dh, longest, window);
  };
  if (!scratch(at, a[9], need, &ws))
    return PyLong_FromLong(DFLASH_ERR_INVALID_ARG);
  const int rc = run(at, [&](cudaStream_t stream) {
    const int64_t q_stride = n > 1 ? q.stride(0) : static_cast<int64_t>(hq) * dh, table_stride = n > 1 ? table.stride(0) : width;
    if constexpr (SHARED)
      return dflash_decode_attention_shared(pq, q_stride, pk, pv, pt, table_stride, pl, starts, prefixes, n, groups, hq, hkv, dh, kp.size(0), page,
                                            width, longest, scale, window, dtype, out, lse, ws.p, ws.bytes, flags, status, stream);
    return dflash_decode_attention_paged(pq, q_stride, pk, pv, pt, table_stride, pl, n, hq, hkv, dh, kp.size(0), page, width, longest, scale,
                                         window, dtype, out, lse, ws.p, ws.bytes, status, stream);
  });
  if (rc) return PyLong_FromLong(rc);
  written({a[6], a[7], a[9], a[13]});
  if (!lse && !(a[7] != Py_None || new_lse.defined())) return given(a[6], new_out);
  return Py_BuildValue("(NN)", given(a[6], new_out), given(a[7], new_lse));
}
PyObject* decode_attention_paged(PyObject* const* a) { return decode_attention<false>(a); }
PyObject* decode_attention_shared(PyObject* const* a) { return decode_attention<true>(a); }

// logits, scores, beams_out (None: as many as in), finished, eos, scores out, tokens out, parents out, finished out, workspace
PyObject* beam_select(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const Place at(x);
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  rows(x, "logits", 3);
  const at::ScalarType type = x.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) raise(PyExc_TypeError, "logits must be bfloat16 or float32, got %s", c10::toString(type));
  const int dtype = type == at::kFloat ? DFLASH_OUT_F32 : DFLASH_OUT_BF16;
  const int n = dim32(x.size(0), "N"), w = dim32(x.size(1), "beams"), vocab = dim32(x.size(2), "vocab");
  const int k = a[2] == Py_None ? w : small(a[2], "beams_out"), eos = small(a[4], "eos");
  const auto* scores = static_cast<const float*>(at.address("scores", a[1], at::kFloat, {n, w}));
  const auto* finished = static_cast<const uint8_t*>(at.address("finished", a[3], at::kBool, {n, w}));
  if (k <= 0) raise(PyExc_ValueError, "beams_out must be positive");
  static const char* const names[4] = {"scores", "tokens", "parents", "finished"};
  static const at::ScalarType types[4] = {at::kFloat, at::kInt, at::kInt, at::kBool};
  // outputs that were not given lie side by side in one allocation
  const int64_t each = (static_cast<int64_t>(n) * k * 4 + 15) / 16 * 16;
  at::Tensor made[4], whole;
  void* out[4];
  for (int i = 0; i < 4; ++i) {
    if (a[5 + i] == Py_None) {
      if (!whole.defined()) whole = at.empty({4 * each}, at::kByte);
      made[i] = Place::slice(whole, i * each, {n, k}, types[i]);
      out[i] = made[i].data_ptr();
    } else {
      out[i] = at.address(names[i], a[5 + i], types[i], {n, k});
    }
  }
  Scratch ws;
  if (!scratch(at, a[9], [&] { return dflash_beam_workspace_size(n, w, k, vocab, dtype); }, &ws))
    return PyLong_FromLong(DFLASH_ERR_INVALID_ARG);
  const int rc = run(at, [&](cudaStream_t stream) {
    return dflash_beam_select(x.data_ptr(), x.stride(0), x.stride(1), scores, finished, n, w, k, vocab, eos, dtype, static_cast<float*>(out[0]),
                              static_cast<int32_t*>(out[1]), static_cast<int32_t*>(out[2]), static_cast<uint8_t*>(out[3]), ws.p, ws.bytes,
                              stream);
  });
  if (rc) return PyLong_FromLong(rc);
  written({a[5], a[6], a[7], a[8], a[9]});
  return Py_BuildValue("(NNNN)", given(a[5], made[0]), given(a[6], made[1]), given(a[7], made[2]), given(a[8], made[3]));
}

struct Table {
  int rows, width;
  int64_t stride, pages;
  int32_t *table, *refs;
  Table(const Place& at, PyObject* t, PyObject* r) {
    const at::Tensor &x = tensor(t, "block_table"), &y = tensor(r, "page_refs");
    if (x.dim() != 2 || y.dim() != 1) raise(PyExc_ValueError, "block_table must be [N, max_pages] and page_refs [num_pages]");
    rows = dim32(x.size(0), "N"), width = dim32(x.size(1), "max_pages");
    if (width > 1 && x.stride(1) != 1) raise(PyExc_ValueError, "block_table: a row must be contiguous");
    if (rows > 1 && x.stride(0) < width) raise(PyExc_ValueError, "block_table: rows must not overlap");
    stride = rows > 1 ? x.stride(0) : width;
    pages = y.size(0);
    table = static_cast<int32_t*>(at.plain("block_table", x, at::kInt, false));
    refs = static_cast<int32_t*>(at.plain("page_refs", y, at::kInt));
  }
};

struct Pools {
  std::vector<void*> p;
  std::vector<at::Tensor> tensors;
  int64_t bytes = 0, page = -1;
  Pools(const Place& at, PyObject* list, int64_t pages) {
    PyObject* seq = PySequence_Fast(list, "pools must be a list of tensors");
    if (!seq) throw Raised{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    PyObject** items = PySequence_Fast_ITEMS(seq);
    const char* bad = nullptr;
    for (Py_ssize_t i = 0; i < n && !bad; ++i) {
      if (!THPVariable_Check(items[i])) {
        bad = "pools must be a list of tensors";
        break;
      }
      const at::Tensor& t = THPVariable_Unpack(items[i]);
      if (t.device() != at.device || !t.is_contiguous() || t.dim() < 2 || t.size(0) != pages)
        bad = "pools must be contiguous [num_pages, page_size, ...] tensors on the call's device";
      else {
        const int64_t b = pages ? static_cast<int64_t>(t.nbytes()) / pages : 0;
        if (i && (b != bytes || t.size(1) != page)) bad = "all pools must have pages of the same size";
        bytes = b, page = t.size(1);
        p.push_back(t.data_ptr());
        tensors.push_back(t);
      }
    }
    Py_DECREF(seq);
    if (bad) raise(PyExc_ValueError, "%s", bad);
  }
};

// parent, seq_lens, block_table, page_refs, status
PyObject* fork_pages(PyObject* const* a) {
  const Place at(tensor(a[2], "block_table"));
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  const Table t(at, a[2], a[3]);
  const at::Tensor& parent = tensor(a[0], "parent");
  if (parent.numel() != t.rows) raise(PyExc_ValueError, "parent has %d entries, expected %d", static_cast<int>(parent.numel()), t.rows);
  const auto* pp = static_cast<const int32_t*>(at.plain("parent", parent, at::kInt));
  auto* lens = static_cast<int32_t*>(at.address("seq_lens", a[1], at::kInt, {t.rows}));
  auto* status = static_cast<int32_t*>(at.address("status", a[4], at::kInt, {1}));
  const int rc = run(at, [&](cudaStream_t stream) { return dflash_fork_pages(pp, lens, t.table, t.stride, t.refs, t.rows, t.width, t.pages, status, stream); });
  if (rc) return PyLong_FromLong(rc);
  written({a[1], a[2], a[3], a[4]});
  Py_RETURN_NONE;
}

// new_start_loc, seq_lens, block_table, page_refs, pools, num_new, page_size, advance, slots, positions, workspace, status
PyObject* reserve_pages(PyObject* const* a) {
  const Place at(tensor(a[2], "block_table"));
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  const Table t(at, a[2], a[3]);
  const Pools pools(at, a[4], t.pages);
  int64_t page = pools.page;
  if (a[6] != Py_None) {
    const int64_t asked = integer(a[6]);
    if (page >= 0 && asked != page) raise(PyExc_ValueError, "page_size is not the pools'");
    page = asked;
  } else if (page < 0) {
    raise(PyExc_ValueError, "page_size is needed without pools");
  }
  const int64_t num_new = integer(a[5]);
  if (num_new < 0) raise(PyExc_ValueError, "num_new must be >= 0");
  const auto* starts = static_cast<const int32_t*>(at.address("new_start_loc", a[0], at::kInt, {t.rows + 1}));
  auto* lens = static_cast<int32_t*>(at.address("seq_lens", a[1], at::kInt, {t.rows}));
  auto* status = static_cast<int32_t*>(at.address("status", a[11], at::kInt, {1}));
  at::Tensor new_slots, new_pos;
  if (a[8] == Py_None) new_slots = at.empty({num_new}, at::kInt);
  if (a[9] == Py_None) new_pos = at.empty({num_new}, at::kInt);
  auto* slots = static_cast<int32_t*>(new_slots.defined() ? new_slots.data_ptr() : at.address("slots", a[8], at::kInt, {num_new}));
  auto* pos = static_cast<int32_t*>(new_pos.defined() ? new_pos.data_ptr() : at.address("positions", a[9], at::kInt, {num_new}));
  const int advance = truth(a[7]), page32 = dim32(page, "page_size");
  Scratch ws;
  if (!scratch(at, a[10], [&] { return dflash_pages_workspace_size(t.rows, t.pages); }, &ws)) return PyLong_FromLong(DFLASH_ERR_INVALID_ARG);
  const int rc = run(at, [&](cudaStream_t stream) {
    return dflash_reserve_pages(starts, lens, t.table, t.stride, t.refs, pools.p.data(), static_cast<int>(pools.p.size()), pools.bytes, t.rows,
                                num_new, t.width, page32, t.pages, advance, slots, pos, ws.p, ws.bytes, status, stream);
  });
  if (rc) return PyLong_FromLong(rc);
  written({a[1], a[2], a[3], a[8], a[9], a[10], a[11]});
  for (const at::Tensor& x : pools.tensors) written(x);
  return Py_BuildValue("(NN)", given(a[8], new_slots), given(a[9], new_pos));
}

// block_table, page_refs, pools, used, workspace, status
PyObject* compact_pages(PyObject* const* a) {
  const Place at(tensor(a[0], "block_table"));
  const c10::cuda::OptionalCUDAGuard guard(at.device);
  const Table t(at, a[0], a[1]);
  const Pools pools(at, a[2], t.pages);
  auto* status = static_cast<int32_t*>(at.address("status", a[5], at::kInt, {1}));
  at::Tensor made;
  if (a[3] == Py_None) made = at.empty({1}, at::kInt);
  auto* used = static_cast<int32_t*>(made.defined() ? made.data_ptr() : at.address("used", a[3], at::kInt, {1}));
  Scratch ws;
  if (!scratch(at, a[4], [&] { return dflash_pages_workspace_size(t.rows, t.pages); }, &ws)) return PyLong_FromLong(DFLASH_ERR_INVALID_ARG);
  const int rc = run(at, [&](cudaStream_t stream) {
    return dflash_compact_pages(t.table, t.stride, t.refs, pools.p.data(), static_cast<int>(pools.p.size()), pools.bytes, t.rows, t.width,
                                t.pages, used, ws.p, ws.bytes, status, stream);
  });
  if (rc) return PyLong_FromLong(rc);
  written({a[0], a[1], a[3], a[4], a[5]});
  for (const at::Tensor& x : pools.tensors) written(x);
  return given(a[3], made);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %d", N, static_cast<int>(n));
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name, n) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(rotary, 13),       ENTRY(decode_attention_paged, 14), ENTRY(beam_select, 10), ENTRY(fork_pages, 5),
                         ENTRY(reserve_pages, 12), ENTRY(compact_pages, 6),           ENTRY(rotary_axes, 14), ENTRY(rms_norm, 10),
                         ENTRY(shared_prefixes, 6), ENTRY(decode_attention_shared, 17), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_decode_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_bind() { return PyModule_Create(&module_def); }
