// Python calls of the appends, of the 4-bit cache and of the prefill over
// quantized caches, as an extension module.
//
// The binding marshals: it checks types, shapes, layouts and devices, takes
// addresses and the current stream, and calls the C ABI.  For a decode step of
// a few tokens that costs more than the kernel when every look at a tensor is a
// Python attribute (11.7 us a call of the append with its dozen tensors, of
// which 2 us are the launch), so these entry points do it on the tensors' own
// objects.  Nothing is computed here, and nothing is kept between calls.
//
// Every function takes its arguments by position (ops.py has the keywords and
// the documentation) and returns the library's status; a wrong type raises
// TypeError, a wrong shape, layout or device ValueError.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <string>

#include "../../include/pa.h"

namespace {

// A Python exception is set.
struct Raised {};

[[noreturn]] void raise(PyObject* kind, const std::string& what) {
  PyErr_SetString(kind, what.c_str());
  throw Raised{};
}

const char* kNoTensor = " must be a tensor";

// The arguments of one call, in order.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n, Py_ssize_t want) : a_(a) {
    if (n != want) raise(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
    dev_ = c10::cuda::current_device();
  }
  // a tensor (nullptr for None), on any device and of any layout
  const at::Tensor* any(const char* name, bool optional = false) {
    PyObject* o = a_[i_++];
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + kNoTensor);
    return &THPVariable_Unpack(o);
  }
  void here(const at::Tensor& t, const char* name) const {
    if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (t.get_device() != dev_)
      raise(PyExc_ValueError, std::string(name) + " must be on the current device, cuda:" +
                                  std::to_string((int)dev_));
  }
  // a contiguous tensor on the current device
  const at::Tensor* flat(const char* name, bool optional = false) {
    const at::Tensor* t = any(name, optional);
    if (t) {
      here(*t, name);
      if (!t->is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    }
    return t;
  }
  const at::Tensor* flat(const char* name, at::ScalarType dtype, const char* says) {
    const at::Tensor* t = flat(name);
    if (t->scalar_type() != dtype)
      raise(PyExc_TypeError, std::string(name) + " must be " + says);
    return t;
  }
  double number() {
    const double x = PyFloat_AsDouble(a_[i_++]);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return x;
  }
  long integer() {
    const long x = PyLong_AsLong(a_[i_++]);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_OverflowError, "an argument exceeds 32 bits");
    return x;
  }
  bool truth() {
    const int x = PyObject_IsTrue(a_[i_++]);
    if (x < 0) throw Raised{};
    return x != 0;
  }
  pa_stream stream() const { return c10::cuda::getCurrentCUDAStream(dev_).stream(); }

 private:
  PyObject* const* a_;
  Py_ssize_t i_ = 0;
  c10::DeviceIndex dev_ = 0;
};

void* at_(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// PA_F16 or PA_BF16
int code16(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kHalf) return PA_F16;
  if (t.scalar_type() == at::kBFloat16) return PA_BF16;
  raise(PyExc_TypeError, std::string(name) + " must be float16 or bfloat16");
}

struct Pools {
  const at::Tensor *k, *v;
  int64_t blocks;
  int B, H, D, code;
};

// k_cache, v_cache: 16-bit or E4M3 pools [num_blocks, B, H_kv, D], or 4-bit pools
// [num_blocks, H_kv, B, 9 D / 16]
Pools pools(Args& a, bool only4) {
  Pools p;
  p.k = a.flat("k_cache");
  p.v = a.flat("v_cache");
  if (p.k->dim() != 4 || p.v->sizes() != p.k->sizes() || p.v->scalar_type() != p.k->scalar_type())
    raise(PyExc_ValueError, "k_cache and v_cache must share one shape of four dimensions");
  const auto s = p.k->sizes();
  const at::ScalarType dtype = p.k->scalar_type();
  p.blocks = s[0];
  if (s[1] > INT32_MAX || s[2] > INT32_MAX || s[3] > INT32_MAX)
    raise(PyExc_ValueError, "a pool's dimension exceeds 32 bits");
  const bool four = dtype == at::kByte && (s[3] == 36 || s[3] == 72);
  if (only4 && dtype != at::kByte)
    raise(PyExc_TypeError, "4-bit pools must be uint8 tensors of codes and scales");
  if (only4 && !four)
    raise(PyExc_ValueError, "4-bit pools must be [num_blocks, H_kv, B, 9 D / 16], D 64 or 128");
  if (four) {
    p.H = (int)s[1];
    p.B = (int)s[2];
    p.D = (int)s[3] / 9 * 16;
    p.code = PA_FP4_E2M1;
  } else {
    p.B = (int)s[1];
    p.H = (int)s[2];
    p.D = (int)s[3];
    p.code = dtype == at::kByte ? PA_FP8_E4M3 : code16(*p.k, "k_cache");
  }
  return p;
}

// block_tables, token_seq, token_pos
struct Tokens {
  const at::Tensor *bt, *seq, *pos;
  int64_t n;
  int seqs, stride;
};
Tokens tokens(Args& a) {
  Tokens t;
  t.bt = a.flat("block_tables", at::kInt, "int32");
  t.seq = a.flat("token_seq", at::kInt, "int32");
  t.pos = a.flat("token_pos", at::kInt, "int32");
  if (t.bt->dim() != 2 || t.bt->size(0) > INT32_MAX || t.bt->size(1) > INT32_MAX)
    raise(PyExc_ValueError, "block_tables must be [num_seqs, stride]");
  t.n = t.seq->numel();
  if (t.pos->numel() != t.n)
    raise(PyExc_ValueError, "token_seq and token_pos differ in length");
  t.seqs = (int)t.bt->size(0);
  t.stride = (int)t.bt->size(1);
  return t;
}

const at::Tensor* slots_out(Args& a, int64_t n) {
  const at::Tensor* t = a.flat("slot_mapping", true);
  if (t && (t->scalar_type() != at::kLong || t->numel() != n))
    raise(PyExc_ValueError, "slot_mapping must be int64 [num_tokens]");
  return t;
}

const at::Tensor* err_word(Args& a) {
  const at::Tensor* t = a.flat("err", true);
  if (t && (t->scalar_type() != at::kInt || t->numel() < 1))
    raise(PyExc_ValueError, "err must be an int32 CUDA tensor");
  return t;
}

// [n, heads, D] with a token's heads contiguous; returns the elements between tokens
int64_t token_rows(const Args& a, const at::Tensor& t, const char* name, int64_t n, int64_t heads,
                   int64_t D, at::ScalarType dtype) {
  a.here(t, name);
  if (t.scalar_type() != dtype) raise(PyExc_TypeError, "q, k and v must share a dtype");
  if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != D)
    raise(PyExc_ValueError, std::string(name) + " must be [num_tokens, heads, head_dim]");
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D))
    raise(PyExc_ValueError, std::string("the heads of a token must be contiguous in ") + name);
  return n > 1 ? t.stride(0) : heads * D;
}

// k, v [n, H, D], contiguous, of one 16-bit dtype; its code
int kv_rows(const at::Tensor& k, const at::Tensor& v, int64_t n, const Pools& p) {
  if (k.dim() != 3 || k.size(0) != n || k.size(1) != p.H || k.size(2) != p.D ||
      v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
    raise(PyExc_ValueError, "k and v must be [num_tokens, H_kv, D] of one dtype");
  return code16(k, "k");
}

// (q, k, v, cos_sin, [axis_of, rot_pos,] block_tables, token_seq, token_pos,
//  k_cache, v_cache, interleaved, q_norm, k_norm, eps, k_scale, v_scale, q_out,
//  slot_mapping, err)
template <bool kAxes>
int append_rope(Args& a) {
  const at::Tensor *q = a.any("q", true), *k = a.any("k"), *v = a.any("v");
  const at::Tensor* cs = a.flat("cos_sin", !kAxes);
  const at::Tensor *axis_of = nullptr, *rot_pos = nullptr;
  if constexpr (kAxes) {
    axis_of = a.flat("axis_of", at::kByte, "uint8");
    rot_pos = a.flat("rot_pos", at::kInt, "int32");
  }
  const Tokens t = tokens(a);
  const Pools p = pools(a, false);
  const bool interleaved = a.truth();
  const at::Tensor *qn = a.flat("q_norm", true), *kn = a.flat("k_norm", true);
  const double eps = a.number(), k_scale = a.number(), v_scale = a.number();
  const at::Tensor* q_out = a.any("q_out", true);
  const at::Tensor* slots = slots_out(a, t.n);
  const at::Tensor* err = err_word(a);
  const at::ScalarType dtype = k->scalar_type();
  const int code = code16(*k, "k");
  if (p.code != code && p.code != PA_FP8_E4M3 && p.code != PA_FP4_E2M1)
    raise(PyExc_TypeError, "the pools must be of k's dtype, or uint8");
  const int64_t ks = token_rows(a, *k, "k", t.n, p.H, p.D, dtype);
  const int64_t vs = token_rows(a, *v, "v", t.n, p.H, p.D, dtype);
  int64_t Hq = 0, qs = 0, rot = 0, max_pos = 0;
  if (q) {
    if (q->dim() != 3) raise(PyExc_ValueError, "q must be [num_tokens, Hq, D]");
    Hq = q->size(1);
    qs = token_rows(a, *q, "q", t.n, Hq, p.D, dtype);
    if (!q_out) raise(PyExc_ValueError, "q without q_out");
    a.here(*q_out, "q_out");
    if (q_out->sizes() != q->sizes() || q_out->scalar_type() != dtype || !q_out->is_contiguous())
      raise(PyExc_ValueError, "q_out must be [num_tokens, Hq, D] of q's dtype, contiguous");
  } else if (q_out) {
    raise(PyExc_ValueError, "q_out without q");
  }
  if (cs) {
    if (cs->scalar_type() != at::kFloat || cs->dim() != 2)
      raise(PyExc_TypeError, "cos_sin must be float32 [max_pos, rotary_dim]");
    max_pos = cs->size(0);
    rot = cs->size(1);
  }
  for (const at::Tensor* g : {qn, kn})
    if (g && (g->scalar_type() != dtype || g->dim() != 1 || g->size(0) != p.D))
      raise(PyExc_ValueError, "q_norm and k_norm must be [D] of k's dtype");
  if (Hq > INT32_MAX || rot > INT32_MAX || max_pos > INT32_MAX)
    raise(PyExc_ValueError, "a dimension exceeds 32 bits");
  if constexpr (kAxes) {
    if (axis_of->numel() != rot / 2)
      raise(PyExc_ValueError, "axis_of must be [rotary_dim / 2]");
    if (rot_pos->dim() != 2 || rot_pos->size(1) != t.n || rot_pos->size(0) < 1 ||
        rot_pos->size(0) > 4)
      raise(PyExc_ValueError, "rot_pos must be [num_axes, num_tokens], 1 to 4 axes");
    return pa_append_rope_axes(
        at_(q), qs, at_(k), ks, at_(v), vs, code, static_cast<const float*>(at_(cs)), (int)rot,
        (int)max_pos, static_cast<const uint8_t*>(at_(axis_of)),
        static_cast<const int32_t*>(at_(rot_pos)), (int)rot_pos->size(0), interleaved ? 1 : 0,
        at_(qn), at_(kn), (float)eps, static_cast<const int32_t*>(at_(t.bt)), t.stride, t.seqs,
        static_cast<const int32_t*>(at_(t.seq)), static_cast<const int32_t*>(at_(t.pos)), t.n,
        at_(q_out), at_(p.k), at_(p.v), p.blocks, p.B, (int)Hq, p.H, p.D, p.code, (float)k_scale,
        (float)v_scale, static_cast<int64_t*>(at_(slots)), static_cast<int32_t*>(at_(err)),
        a.stream());
  }
  return pa_append_rope(
      at_(q), qs, at_(k), ks, at_(v), vs, code, static_cast<const float*>(at_(cs)), (int)rot,
      (int)max_pos, interleaved ? 1 : 0, at_(qn), at_(kn), (float)eps,
      static_cast<const int32_t*>(at_(t.bt)), t.stride, t.seqs,
      static_cast<const int32_t*>(at_(t.seq)), static_cast<const int32_t*>(at_(t.pos)), t.n,
      at_(q_out), at_(p.k), at_(p.v), p.blocks, p.B, (int)Hq, p.H, p.D, p.code, (float)k_scale,
      (float)v_scale, static_cast<int64_t*>(at_(slots)), static_cast<int32_t*>(at_(err)),
      a.stream());
}

// (k, v, slot_mapping, k_cache, v_cache, k_scale, v_scale, err)
int cache_write_fp4(Args& a) {
  const at::Tensor *k = a.flat("k"), *v = a.flat("v");
  const at::Tensor* slots = a.flat("slot_mapping", at::kLong, "int64");
  const Pools p = pools(a, true);
  const double k_scale = a.number(), v_scale = a.number();
  const at::Tensor* err = err_word(a);
  const int64_t n = slots->numel();
  const int code = kv_rows(*k, *v, n, p);
  return pa_cache_write_fp4(at_(k), at_(v), code, static_cast<const int64_t*>(at_(slots)), n,
                            at_(p.k), at_(p.v), p.blocks, p.B, p.H, p.D, (float)k_scale,
                            (float)v_scale, static_cast<int32_t*>(at_(err)), a.stream());
}

// (k, v, block_tables, token_seq, token_pos, k_cache, v_cache, k_scale, v_scale,
//  slot_mapping, err)
int cache_write_fp4_mapped(Args& a) {
  const at::Tensor *k = a.flat("k"), *v = a.flat("v");
  const Tokens t = tokens(a);
  const Pools p = pools(a, true);
  const double k_scale = a.number(), v_scale = a.number();
  const at::Tensor* slots = slots_out(a, t.n);
  const at::Tensor* err = err_word(a);
  const int code = kv_rows(*k, *v, t.n, p);
  return pa_cache_write_fp4_mapped(
      at_(k), at_(v), code, static_cast<const int32_t*>(at_(t.bt)), t.stride, t.seqs,
      static_cast<const int32_t*>(at_(t.seq)), static_cast<const int32_t*>(at_(t.pos)), t.n,
      at_(p.k), at_(p.v), p.blocks, p.B, p.H, p.D, (float)k_scale, (float)v_scale,
      static_cast<int64_t*>(at_(slots)), static_cast<int32_t*>(at_(err)), a.stream());
}

// (slot_mapping, k_cache, v_cache, k_scale, v_scale, k_out, v_out, err)
int cache_read_fp4(Args& a) {
  const at::Tensor* slots = a.flat("slot_mapping", at::kLong, "int64");
  const Pools p = pools(a, true);
  const double k_scale = a.number(), v_scale = a.number();
  const at::Tensor *k = a.flat("k_out"), *v = a.flat("v_out");
  const at::Tensor* err = err_word(a);
  const int64_t n = slots->numel();
  const int code = kv_rows(*k, *v, n, p);
  return pa_cache_read_fp4(static_cast<const int64_t*>(at_(slots)), n, at_(p.k), at_(p.v),
                           p.blocks, p.B, p.H, p.D, (float)k_scale, (float)v_scale, at_(k), at_(v),
                           code, static_cast<int32_t*>(at_(err)), a.stream());
}

// (q, k_cache, v_cache, block_tables, seq_lens, scale, k_scale, v_scale, window,
//  out, workspace, flags, num_ctas, err)
int decode_fp4(Args& a) {
  const at::Tensor* q = a.flat("q");
  const Pools p = pools(a, true);
  const at::Tensor* bt = a.flat("block_tables", at::kInt, "int32");
  const at::Tensor* lens = a.flat("seq_lens", at::kInt, "int32");
  const double scale = a.number(), k_scale = a.number(), v_scale = a.number();
  const long window = a.integer();
  const at::Tensor *out = a.flat("out"), *ws = a.flat("workspace");
  const long flags = a.integer(), num_ctas = a.integer();
  const at::Tensor* err = err_word(a);
  const int code = code16(*q, "q");
  if (q->dim() != 3 || q->size(2) != p.D || q->size(0) > INT32_MAX || q->size(1) > INT32_MAX)
    raise(PyExc_ValueError, "q must be [N, Hq, D]");
  const int64_t N = q->size(0);
  if (bt->dim() != 2 || bt->size(0) != N || lens->numel() != N || bt->size(1) > INT32_MAX)
    raise(PyExc_ValueError, "block_tables must be [N, stride] and seq_lens [N]");
  if (out->sizes() != q->sizes() || out->scalar_type() != q->scalar_type())
    raise(PyExc_ValueError, "out must be [N, Hq, D] of q's dtype");
  return pa_decode_fp4(at_(q), at_(p.k), at_(p.v), static_cast<const int32_t*>(at_(bt)),
                       (int)bt->size(1), static_cast<const int32_t*>(at_(lens)), (int)N,
                       (int)q->size(1), p.H, p.D, p.B, p.blocks, code, (float)scale,
                       (float)k_scale, (float)v_scale, (int)window, at_(out), at_(ws),
                       (size_t)ws->numel() * ws->element_size(), (int)flags, (int)num_ctas,
                       static_cast<int32_t*>(at_(err)), a.stream());
}

// (q, k_cache, v_cache, block_tables, seq_lens, query_start, scale, k_scale,
//  v_scale, window, out, workspace, err)
template <bool kFour>
int prefill_quant(Args& a) {
  const at::Tensor* q = a.flat("q");
  const Pools p = pools(a, kFour);
  if (!kFour && p.code != PA_FP8_E4M3)
    raise(PyExc_TypeError, "E4M3 pools must be uint8 tensors of codes [num_blocks, B, H_kv, D]");
  const at::Tensor* bt = a.flat("block_tables", at::kInt, "int32");
  const at::Tensor* lens = a.flat("seq_lens", at::kInt, "int32");
  const at::Tensor* start = a.flat("query_start", at::kInt, "int32");
  const double scale = a.number(), k_scale = a.number(), v_scale = a.number();
  const long window = a.integer();
  const at::Tensor *out = a.flat("out"), *ws = a.flat("workspace");
  const at::Tensor* err = err_word(a);
  const int code = code16(*q, "q");
  if (q->dim() != 3 || q->size(2) != p.D || q->size(1) > INT32_MAX)
    raise(PyExc_ValueError, "q must be [total_q, Hq, D]");
  const int64_t N = lens->numel();
  if (N > INT32_MAX || start->numel() != N + 1 || bt->dim() != 2 || bt->size(0) != N ||
      bt->size(1) > INT32_MAX)
    raise(PyExc_ValueError, "query_start must be [N + 1], block_tables [N, stride], seq_lens [N]");
  if (out->sizes() != q->sizes() || out->scalar_type() != q->scalar_type())
    raise(PyExc_ValueError, "out must be [total_q, Hq, D] of q's dtype");
  return (kFour ? pa_prefill_fp4 : pa_prefill_fp8)(
      at_(q), at_(p.k), at_(p.v), static_cast<const int32_t*>(at_(bt)), (int)bt->size(1),
      static_cast<const int32_t*>(at_(lens)), static_cast<const int32_t*>(at_(start)), (int)N,
      q->size(0), (int)q->size(1), p.H, p.D, p.B, p.blocks, code, (float)scale, (float)k_scale,
      (float)v_scale, (int)window, at_(out), at_(ws), (size_t)ws->numel() * ws->element_size(),
      static_cast<int32_t*>(at_(err)), a.stream());
}

// No C++ exception leaves a call.
template <int (*kCall)(Args&), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    Args a(args, n, kArgs);
    return PyLong_FromLong(kCall(a));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <int (*kCall)(Args&), int kArgs>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&entry<kCall, kArgs>));
}

PyMethodDef methods[] = {
    {"append_rope", fast<append_rope<false>, 18>(), METH_FASTCALL, nullptr},
    {"append_rope_axes", fast<append_rope<true>, 20>(), METH_FASTCALL, nullptr},
    {"cache_write_fp4", fast<cache_write_fp4, 8>(), METH_FASTCALL, nullptr},
    {"cache_write_fp4_mapped", fast<cache_write_fp4_mapped, 11>(), METH_FASTCALL, nullptr},
    {"cache_read_fp4", fast<cache_read_fp4, 8>(), METH_FASTCALL, nullptr},
    {"decode_fp4", fast<decode_fp4, 14>(), METH_FASTCALL, nullptr},
    {"prefill_fp8", fast<prefill_quant<false>, 13>(), METH_FASTCALL, nullptr},
    {"prefill_fp4", fast<prefill_quant<true>, 13>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pa_call",
                      "Marshalling of the appends', the 4-bit cache's and the quantized prefill's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pa_call(void) { return PyModule_Create(&module); }
