// The binding of the position and serving calls, as a Python module (_calls).  A single token's kernels
// run for a few microseconds; checking tensors, making outputs and converting 20 to 30 arguments in
// Python took longer, so these calls do it here (calls one after the other: append B64 H32/8 17.7 us ->
// 6.3, norm and rotation B2 N128 H12 21.1 -> 8.5, its gradient 38.7 -> 16 to 20, decode B1 H16 C512 21.9 -> 10.6).  serving.py
// holds the public functions and their documentation, and this file their checks: the same
// refusals (ValueError, TypeError, RaError), then the C ABI call on torch's current stream of the
// tensors' device, with the interpreter free.  Host code only; it holds no state.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <limits>
#include <sstream>
#include <string>
#include <vector>

#include "raattn.h"

namespace {

using at::Tensor;

struct Refusal {   // becomes a Python exception; type nullptr: one is set already
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

// ---- arguments ---------------------------------------------------------------------------------
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
const Tensor* optional_tensor(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
int integer(PyObject* o) {
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Refusal{nullptr, ""};
  const long long v = PyLong_AsLongLong(i);
  Py_DECREF(i);
  if (PyErr_Occurred()) throw Refusal{nullptr, ""};
  if (v < std::numeric_limits<int>::min() || v > std::numeric_limits<int>::max())
    throw Refusal{PyExc_OverflowError, "a size is beyond int32"};
  return static_cast<int>(v);
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw Refusal{nullptr, ""};
  return static_cast<float>(v);
}
int size32(int64_t n) {
  if (n > std::numeric_limits<int>::max()) throw Refusal{PyExc_OverflowError, "a size is beyond int32"};
  return static_cast<int>(n);
}
ra_dtype_t dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return RA_F32;
  if (t.scalar_type() == at::kBFloat16) return RA_BF16;
  throw Refusal{PyExc_TypeError,
                std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + ": libraattn takes float32 or bfloat16"};
}
void check(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType dtype, const at::Device& device) {
  if (t.scalar_type() == dtype && t.sizes() == shape && t.device() == device && t.is_contiguous()) return;
  std::ostringstream s;
  s << name << " must be a contiguous " << c10::toString(dtype) << " tensor of shape " << shape << " on " << device;
  refuse(s.str());
}
void* address(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
// at::empty; without its dispatch, 0.35 us less each, where nothing would see that (page_write B64 5.55 us a call -> 4.85,
// page_compact 10.2 -> 8.8, norm and rotation 7.2 -> 6.2): under a dispatch mode, and where torch fills what it allocates, it is
// called as it stands.
Tensor make(at::IntArrayRef shape, at::ScalarType dtype, const at::Device& device) {
  const at::Context& context = at::globalContext();
  if (c10::impl::dispatch_mode_enabled() || (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory()))
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
  return Tensor(at::detail::empty_cuda(shape, dtype, device, c10::nullopt));
}

// f(stream) on the current stream of `device`, which is the current one meanwhile.
template <typename F>
ra_status_t on_stream(const at::Device& device, F f) {
  const c10::cuda::CUDAGuard guard(device);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  ra_status_t code;
  Py_BEGIN_ALLOW_THREADS code = f(stream);
  Py_END_ALLOW_THREADS return code;
}
void check_status(const char* call, ra_status_t code) {   // the package's RaError
  if (code == RA_OK) return;
  PyObject* package = PyImport_ImportModule("rational_softmax_attention_gb300");
  PyObject* r = package ? PyObject_CallMethod(package, "_check", "si", call, static_cast<int>(code)) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(package);
  throw Refusal{nullptr, ""};
}
PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw Refusal{nullptr, ""};
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = Py_None;
    if (t.defined()) o = THPVariable_Wrap(t);
    else Py_INCREF(o);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// ---- norm and rotation --------------------------------------------------------------------------
constexpr int kLead = 13;   // arguments that the forward, the append and the backward share

// The kernels read a tensor's values alone, so a tangent that it carries would be lost without a word.
void refuse_tangents(PyObject* const* a, std::initializer_list<int> which) {
  for (const int i : which)
    if (THPVariable_Check(a[i]) && THPVariable_Unpack(a[i])._fw_grad(0).defined())
      throw Refusal{PyExc_NotImplementedError, "forward-mode derivatives of ra_qk_norm_rope are not supported"};
}

struct NormRope {
  Tensor qkv, positions;
  const Tensor *qw, *qb, *kw, *kb, *frequencies;
  int64_t row, token, pos_axis = 0, pos_batch = 0;
  ra_norm_t norm;
  float eps;
  std::vector<int32_t> sections;
  int interleaved, B, N, Hq, Hkv, D;
  ra_dtype_t code;
  at::Device device{at::kCPU};
  at::ScalarType dtype;

  // qkv, num_heads, num_kv_heads, norm, q_weight, q_bias, k_weight, k_bias, eps, frequencies, sections, positions,
  // interleaved
  explicit NormRope(PyObject* const* a) : qkv(tensor(a[0], "qkv")) {
    if (qkv.dim() != 3 || !qkv.is_cuda())
      refuse("qkv must be a CUDA tensor [B, N, (num_heads + 2 num_kv_heads) * head_dim]");
    dtype = qkv.scalar_type();
    device = qkv.device();
    code = dtype_code(qkv);
    Hq = integer(a[1]);
    Hkv = a[2] == Py_None ? Hq : integer(a[2]);
    B = size32(qkv.size(0));
    N = size32(qkv.size(1));
    const int64_t width = qkv.size(2), heads = static_cast<int64_t>(Hq) + 2 * static_cast<int64_t>(Hkv);
    if (Hq < 1 || Hkv < 1 || width < 1 || width % heads)
      refuse("qkv must be [B, N, (num_heads + 2 num_kv_heads) * head_dim]");
    D = size32(width / heads);
    if (B < 1 || N < 1) refuse("qkv must hold at least one token");
    const int64_t mask = code == RA_BF16 ? 7 : 3;
    if (qkv.stride(2) != 1 || qkv.stride(0) & mask || qkv.stride(1) & mask ||
        reinterpret_cast<uintptr_t>(qkv.data_ptr()) & 15)
      qkv = qkv.clone(at::MemoryFormat::Contiguous);
    row = qkv.stride(0);
    token = qkv.stride(1);
    if (!PyUnicode_Check(a[3])) refuse("norm must be 'none', 'layer' or 'rms'");
    if (!PyUnicode_CompareWithASCIIString(a[3], "layer")) norm = RA_NORM_LAYER;
    else if (!PyUnicode_CompareWithASCIIString(a[3], "rms")) norm = RA_NORM_RMS;
    else if (!PyUnicode_CompareWithASCIIString(a[3], "none")) norm = RA_NORM_NONE;
    else refuse("norm must be 'none', 'layer' or 'rms'");
    qw = optional_tensor(a[4], "q_weight");
    qb = optional_tensor(a[5], "q_bias");
    kw = optional_tensor(a[6], "k_weight");
    kb = optional_tensor(a[7], "k_bias");
    if (norm == RA_NORM_NONE) {
      if (qw || qb || kw || kb) refuse("norm='none' takes no weights and no biases");
    } else {
      if (!qw || !kw) refuse("q_weight and k_weight are required with a norm");
      check("q_weight", *qw, {D}, dtype, device);
      check("k_weight", *kw, {D}, dtype, device);
      if (norm == RA_NORM_RMS && (qb || kb)) refuse("norm='rms' takes no biases");
      if (qb) check("q_bias", *qb, {D}, dtype, device);
      if (kb) check("k_bias", *kb, {D}, dtype, device);
    }
    eps = number(a[8]);
    frequencies = optional_tensor(a[9], "frequencies");
    const Tensor* pos = optional_tensor(a[11], "positions");
    read_sections(a[10]);
    if (!sections.empty()) {
      if (!frequencies || !pos) refuse("sections need frequencies and positions");
      int64_t pairs = 0;
      for (const int32_t s : sections) pairs += s;
      check("frequencies", *frequencies, {pairs}, at::kDouble, device);
      read_positions(*pos);
    } else if (frequencies || pos) {
      refuse("frequencies and positions need sections");
    }
    const int truth = PyObject_IsTrue(a[12]);
    if (truth < 0) throw Refusal{nullptr, ""};
    interleaved = truth;
  }

  void read_sections(PyObject* o) {
    if (o == Py_None) return;
    PyObject* seq = PySequence_Fast(o, "sections must be a sequence of pair counts");
    if (!seq) throw Refusal{nullptr, ""};
    int64_t pairs = 0;
    bool good = true;
    try {
      for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i) {
        sections.push_back(integer(PySequence_Fast_GET_ITEM(seq, i)));
        good = good && sections.back() >= 1;
        pairs += sections.back();
      }
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
    Py_DECREF(seq);
    if (!good || 2 * pairs > D) refuse("sections must be positive pair counts with 2 * sum(sections) <= head_dim");
  }

  void read_positions(const Tensor& given) {
    positions = given;
    if (positions.scalar_type() == at::kLong) positions = positions.to(at::kInt);
    else if (positions.scalar_type() != at::kInt) refuse("positions must be an int32 or int64 tensor");
    const int64_t d = positions.dim(), axes = static_cast<int64_t>(sections.size());
    if (positions.device() != device || d < 1 || d > 3 || positions.size(-1) != N ||
        (d > 1 && positions.size(-2) != 1 && positions.size(-2) != B) ||
        (d > 2 && positions.size(0) != 1 && positions.size(0) != axes))
      refuse("positions must be [N], [B, N] or [axes, B, N] on qkv's device, or broadcast to it");
    if (positions.stride(-1) != 1 && N > 1) positions = positions.clone(at::MemoryFormat::Contiguous);
    if (d > 1 && positions.size(-2) > 1) pos_batch = positions.stride(-2);
    if (d > 2 && positions.size(0) > 1) pos_axis = positions.stride(0);
  }

  ra_status_t forward(void* q, void* k, void* v, const Tensor* start, const Tensor* count, int capacity) const {
    return on_stream(device, [&](cudaStream_t st) {
      return ra_qk_norm_rope_fwd(qkv.data_ptr(), row, token, address(qw), address(qb), address(kw), address(kb), norm, eps,
                                 static_cast<const double*>(address(frequencies)), ints(positions), pos_axis, pos_batch,
                                 sections.data(), axes(), interleaved, q, k, v, static_cast<const int32_t*>(address(start)),
                                 static_cast<const int32_t*>(address(count)), capacity, B, N, Hq, Hkv, D, code, st);
    });
  }
  ra_status_t backward(const Tensor& dq, const Tensor& dk, const Tensor& dv, const Tensor& dqkv, const Tensor& dparams,
                       const Tensor& workspace) const {
    return on_stream(device, [&](cudaStream_t st) {
      return ra_qk_norm_rope_bwd(qkv.data_ptr(), row, token, address(qw), address(qb), address(kw), address(kb), norm, eps,
                                 static_cast<const double*>(address(frequencies)), ints(positions), pos_axis, pos_batch,
                                 sections.data(), axes(), interleaved, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                 dqkv.data_ptr(), dparams.defined() ? static_cast<float*>(dparams.data_ptr()) : nullptr,
                                 workspace.defined() ? workspace.data_ptr() : nullptr, B, N, Hq, Hkv, D, code, st);
    });
  }
  int axes() const { return static_cast<int>(sections.size()); }
  static const int32_t* ints(const Tensor& t) { return t.defined() ? static_cast<const int32_t*>(t.data_ptr()) : nullptr; }
};

PyObject* norm_rope(PyObject* const* a) {
  refuse_tangents(a, {0, 4, 5, 6, 7});   // qkv, the weights and biases
  const NormRope s(a);
  const Tensor q = make({s.B, s.Hq, s.N, s.D}, s.dtype, s.device), k = make({s.B, s.Hkv, s.N, s.D}, s.dtype, s.device),
               v = make({s.B, s.Hkv, s.N, s.D}, s.dtype, s.device);
  check_status("ra_qk_norm_rope_fwd", s.forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), nullptr, nullptr, 0));
  return tuple({q, k, v});
}

// .., dq, dk, dv
PyObject* norm_rope_backward(PyObject* const* a) {
  refuse_tangents(a, {0, 4, 5, 6, 7, kLead, kLead + 1, kLead + 2});
  const NormRope s(a);
  const Tensor &dq = tensor(a[kLead], "dq"), &dk = tensor(a[kLead + 1], "dk"), &dv = tensor(a[kLead + 2], "dv");
  check("dq", dq, {s.B, s.Hq, s.N, s.D}, s.dtype, s.device);
  check("dk", dk, {s.B, s.Hkv, s.N, s.D}, s.dtype, s.device);
  check("dv", dv, {s.B, s.Hkv, s.N, s.D}, s.dtype, s.device);
  const Tensor dqkv = make(s.qkv.sizes(), s.dtype, s.device);
  Tensor dparams, workspace, dqw, dqb, dkw, dkb;
  if (s.norm != RA_NORM_NONE) {
    dparams = make({4, s.D}, at::kFloat, s.device);
    workspace = make({static_cast<int64_t>(ra_qk_norm_rope_bwd_workspace_size(s.D)) + 16}, at::kByte, s.device);
  }
  check_status("ra_qk_norm_rope_bwd", s.backward(dq, dk, dv, dqkv, dparams, workspace));
  if (dparams.defined()) {
    dqw = dparams.select(0, 0);
    if (s.qb) dqb = dparams.select(0, 1);
    dkw = dparams.select(0, 2);
    if (s.kb) dkb = dparams.select(0, 3);
  }
  return tuple({dqkv, dqw, dqb, dkw, dkb});
}

// .., k, v, length, count
PyObject* cache_append(PyObject* const* a) {
  const NormRope s(a);
  const Tensor &k = tensor(a[kLead], "k"), &v = tensor(a[kLead + 1], "v"), &length = tensor(a[kLead + 2], "length");
  const Tensor* count = optional_tensor(a[kLead + 3], "count");
  if (k.dim() != 4 || k.size(2) < 1) refuse("the cache must be [B, num_kv_heads, C, head_dim] with C >= 1");
  const int C = size32(k.size(2));
  check("k", k, {s.B, s.Hkv, C, s.D}, s.dtype, s.device);
  check("v", v, {s.B, s.Hkv, C, s.D}, s.dtype, s.device);
  check("length", length, {s.B}, at::kInt, s.device);
  if (count) check("count", *count, {s.B}, at::kInt, s.device);
  const Tensor q = make({s.B, s.Hq, s.N, s.D}, s.dtype, s.device);
  check_status("ra_qk_norm_rope_fwd", s.forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), &length, count, C));
  return THPVariable_Wrap(q);
}

// ---- decode -------------------------------------------------------------------------------------
// q, k, v, length, prefix_k, prefix_v, scale, weight
PyObject* attention_decode(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  if (q.dim() != 3 || k.dim() != 4) refuse("q must be [B, H, D] and the cache [B, H_kv, C, D]");
  if (!q.is_cuda() || !q.is_contiguous()) refuse("q must be a contiguous CUDA tensor (there is no CPU path)");
  const Tensor &v = tensor(a[2], "v"), &length = tensor(a[3], "length");
  const Tensor *pk = optional_tensor(a[4], "prefix_k"), *pv = optional_tensor(a[5], "prefix_v"),
               *weight = optional_tensor(a[7], "weight");
  const at::ScalarType dtype = q.scalar_type();
  const at::Device device = q.device();
  const ra_dtype_t code = dtype_code(q);
  const int B = size32(q.size(0)), Hq = size32(q.size(1)), D = size32(q.size(2)), Hkv = size32(k.size(1)),
            C = size32(k.size(2));
  check("k", k, {B, Hkv, C, D}, dtype, device);
  check("v", v, {B, Hkv, C, D}, dtype, device);
  check("length", length, {B}, at::kInt, device);
  if (B < 1 || Hkv < 1 || C < 1 || Hq < 1 || D < 1 || Hq % Hkv)
    refuse("the number of query heads must be a multiple of the key heads', and no size 0");
  int P = 0;
  if (!pk != !pv) refuse("prefix_k and prefix_v come together");
  if (pk) {
    P = pk->dim() == 3 ? size32(pk->size(1)) : -1;
    check("prefix_k", *pk, {Hkv, P, D}, dtype, device);
    check("prefix_v", *pv, {Hkv, P, D}, dtype, device);
    if (P == 0) pk = pv = nullptr;
  }
  if (weight) check("weight", *weight, {B, Hkv, C}, at::kFloat, device);
  const float scale = a[6] == Py_None ? 0.0f : number(a[6]);
  const Tensor o = make({B, Hq, D}, dtype, device);
  const Tensor ws = make({static_cast<int64_t>(ra_attention_decode_workspace_size(B, Hq, Hkv, C, P, D, code)) + 16},
                         at::kByte, device);
  check_status("ra_attention_decode", on_stream(device, [&](cudaStream_t st) {
                 return ra_attention_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            static_cast<const int32_t*>(length.data_ptr()), address(pk), address(pv),
                                            o.data_ptr(), static_cast<float*>(address(weight)), ws.data_ptr(), B, Hq, Hkv, C,
                                            P, D, scale, code, st);
               }));
  return THPVariable_Wrap(o);
}

// ---- eviction -----------------------------------------------------------------------------------
// k, v, weight, length, keep, recent, out
PyObject* cache_evict(PyObject* const* a) {
  const Tensor& k = tensor(a[0], "k");
  if (k.dim() != 4) refuse("the cache must be [B, H_kv, C, D]");
  if (!k.is_cuda() || !k.is_contiguous()) refuse("k must be a contiguous CUDA tensor (there is no CPU path)");
  const Tensor &v = tensor(a[1], "v"), &weight = tensor(a[2], "weight"), &length = tensor(a[3], "length");
  const int keep = integer(a[4]), recent = integer(a[5]);
  const at::ScalarType dtype = k.scalar_type();
  const at::Device device = k.device();
  const ra_dtype_t code = dtype_code(k);
  const int B = size32(k.size(0)), Hkv = size32(k.size(1)), C = size32(k.size(2)), D = size32(k.size(3));
  if (B < 1 || Hkv < 1 || C < 1 || D < 1 || keep < 1 || recent < 0 || recent > keep)
    refuse("keep must be at least 1, recent between 0 and keep, and no size 0");
  check("v", v, {B, Hkv, C, D}, dtype, device);
  check("weight", weight, {B, Hkv, C}, at::kFloat, device);
  check("length", length, {B}, at::kInt, device);
  Tensor ko, vo, wo;
  if (a[6] == Py_None) {
    const at::TensorOptions options = at::TensorOptions().dtype(dtype).device(device);
    ko = at::zeros({B, Hkv, keep, D}, options);
    vo = at::zeros({B, Hkv, keep, D}, options);
    wo = at::zeros({B, Hkv, keep}, options.dtype(at::kFloat));
  } else {
    if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 3) refuse("out must be (k, v, weight)");
    ko = tensor(PyTuple_GET_ITEM(a[6], 0), "out[0]");
    vo = tensor(PyTuple_GET_ITEM(a[6], 1), "out[1]");
    wo = tensor(PyTuple_GET_ITEM(a[6], 2), "out[2]");
  }
  const int Co = ko.dim() == 4 ? size32(ko.size(2)) : 0;
  if (Co < keep) refuse("out must have room for `keep` entries");
  check("out[0]", ko, {B, Hkv, Co, D}, dtype, device);
  check("out[1]", vo, {B, Hkv, Co, D}, dtype, device);
  check("out[2]", wo, {B, Hkv, Co}, at::kFloat, device);
  const Tensor new_length = make({B}, at::kInt, device), index = make({B, Hkv, keep}, at::kInt, device);
  check_status("ra_cache_evict", on_stream(device, [&](cudaStream_t st) {
                 return ra_cache_evict(k.data_ptr(), v.data_ptr(), static_cast<const float*>(weight.data_ptr()),
                                       static_cast<const int32_t*>(length.data_ptr()), ko.data_ptr(), vo.data_ptr(),
                                       static_cast<float*>(wo.data_ptr()), static_cast<int32_t*>(new_length.data_ptr()),
                                       static_cast<int32_t*>(index.data_ptr()), B, Hkv, C, Co, D, keep, recent, code, st);
               }));
  return tuple({ko, vo, wo, new_length, index});
}

// ---- pages in 4 bits ----------------------------------------------------------------------------
// uint8 [pages, H_kv, 2, page, row]: a layer's slice of a larger tensor will do, pages may lie apart.
struct Pool {
  const Tensor* t;
  int pages, Hkv, page, D;
  int64_t stride, bytes;   // from page to page; of a page

  Pool(PyObject* o, const char* name) : t(&tensor(o, name)) {
    std::ostringstream s;
    if (t->dim() != 5 || t->scalar_type() != at::kByte || !t->is_cuda() || t->size(2) != 2 ||
        (t->size(4) != 36 && t->size(4) != 72)) {
      s << name << " must be a CUDA uint8 tensor [pages, num_kv_heads, 2, page_size, head_dim / 2 + head_dim / 16], head_dim 64 or 128";
      refuse(s.str());
    }
    pages = size32(t->size(0));
    Hkv = size32(t->size(1));
    page = size32(t->size(3));
    D = t->size(4) == 36 ? 64 : 128;
    if (pages < 1 || Hkv < 1 || (page != 16 && page != 32 && page != 64 && page != 128 && page != 256)) {
      s << name << " must have pages of 16, 32, 64, 128 or 256 tokens, and no size 0";
      refuse(s.str());
    }
    const int64_t part = t->size(3) * t->size(4);
    bytes = 2 * Hkv * part;
    stride = pages > 1 ? t->stride(0) : bytes;
    if (t->stride(4) != 1 || t->stride(3) != t->size(4) || t->stride(2) != part || (Hkv > 1 && t->stride(1) != 2 * part) ||
        stride < bytes || stride % 16 || reinterpret_cast<uintptr_t>(t->data_ptr()) & 15) {
      s << name << " must hold each page without gaps, pages a multiple of 16 bytes apart, at a 16-byte address";
      refuse(s.str());
    }
  }
  at::Device device() const { return t->device(); }
  void* data() const { return t->data_ptr(); }
};
// int32 [B, M] on the pool's device
const Tensor& table_of(PyObject* o, const at::Device& device) {
  const Tensor& t = tensor(o, "table");
  if (t.dim() != 2 || t.size(0) < 1 || t.size(1) < 1) refuse("table must be [sequences, pages], and no size 0");
  check("table", t, {t.size(0), t.size(1)}, at::kInt, device);
  size32(t.size(0));
  size32(t.size(1));
  return t;
}
const int32_t* ints(const Tensor* t) { return static_cast<const int32_t*>(address(t)); }
int32_t* ints(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
const Tensor* per_sequence(PyObject* o, const char* name, int B, const at::Device& device) {
  const Tensor* t = optional_tensor(o, name);
  if (t) check(name, *t, {B}, at::kInt, device);
  return t;
}
Tensor rows_for(const Tensor& x, int vec) {   // as the kernel reads them, whatever view of another tensor they are
  if (x.stride(3) != 1 || x.stride(0) % vec || x.stride(1) % vec || x.stride(2) % vec ||
      reinterpret_cast<uintptr_t>(x.data_ptr()) & 15)
    return x.clone(at::MemoryFormat::Contiguous);
  return x;
}

// k, v, pool, table, start, count, held
PyObject* page_write(PyObject* const* a) {
  const Tensor &k0 = tensor(a[0], "k"), &v0 = tensor(a[1], "v");
  const Pool pool(a[2], "pool");
  const Tensor& table = table_of(a[3], pool.device());
  const int B = size32(table.size(0)), M = size32(table.size(1));
  const ra_dtype_t code = dtype_code(k0);
  if (k0.dim() != 4 || k0.size(2) < 1) refuse("k must be [B, num_kv_heads, N, head_dim] with N >= 1");
  const int N = size32(k0.size(2));
  for (const Tensor* t : {&k0, &v0})
    if (t->sizes() != at::IntArrayRef({B, pool.Hkv, N, pool.D}) || t->scalar_type() != k0.scalar_type() || t->device() != pool.device()) {
      std::ostringstream s;
      s << "k and v must be [B, num_kv_heads, N, head_dim] = " << at::IntArrayRef({B, pool.Hkv, N, pool.D})
        << " of one dtype on the pool's device";
      refuse(s.str());
    }
  const Tensor *start = per_sequence(a[4], "start", B, pool.device()), *count = per_sequence(a[5], "count", B, pool.device());
  const int truth = PyObject_IsTrue(a[6]);
  if (truth < 0) throw Refusal{nullptr, ""};
  const int vec = code == RA_BF16 ? 8 : 4;
  const Tensor k = rows_for(k0, vec), v = rows_for(v0, vec);
  Tensor kh, vh;
  if (truth) {
    kh = make({B, pool.Hkv, N, pool.D}, k.scalar_type(), pool.device());
    vh = make({B, pool.Hkv, N, pool.D}, k.scalar_type(), pool.device());
  }
  const int64_t ks[3] = {k.stride(0), k.stride(1), k.stride(2)}, vs[3] = {v.stride(0), v.stride(1), v.stride(2)};
  check_status("ra_page_write", on_stream(pool.device(), [&](cudaStream_t st) {
                 return ra_page_write(k.data_ptr(), v.data_ptr(), ks, vs, pool.data(), pool.stride, ints(table), ints(start),
                                      ints(count), truth ? kh.data_ptr() : nullptr, truth ? vh.data_ptr() : nullptr, B, N,
                                      pool.Hkv, pool.D, pool.pages, pool.page, M, code, st);
               }));
  if (truth) return tuple({kh, vh});
  Py_RETURN_NONE;
}

// pool, table, length, tokens, start, dtype (a code)
PyObject* page_read(PyObject* const* a) {
  const Pool pool(a[0], "pool");
  const Tensor& table = table_of(a[1], pool.device());
  const int B = size32(table.size(0)), M = size32(table.size(1)), N = integer(a[3]);
  const Tensor *length = per_sequence(a[2], "length", B, pool.device()), *start = per_sequence(a[4], "start", B, pool.device());
  if (N < 1) refuse("tokens must be at least 1");
  const ra_dtype_t code = integer(a[5]) == RA_BF16 ? RA_BF16 : RA_F32;
  const at::ScalarType dtype = code == RA_BF16 ? at::kBFloat16 : at::kFloat;
  const Tensor k = make({B, pool.Hkv, N, pool.D}, dtype, pool.device()), v = make({B, pool.Hkv, N, pool.D}, dtype, pool.device());
  check_status("ra_page_read", on_stream(pool.device(), [&](cudaStream_t st) {
                 return ra_page_read(pool.data(), pool.stride, ints(table), ints(start), ints(length), k.data_ptr(), v.data_ptr(),
                                     B, N, pool.Hkv, pool.D, pool.pages, pool.page, M, code, st);
               }));
  return tuple({k, v});
}

// q, pool, table, length, scale
PyObject* attention_decode_paged(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  if (q.dim() != 3) refuse("q must be [B, H, D]");
  if (!q.is_cuda() || !q.is_contiguous()) refuse("q must be a contiguous CUDA tensor (there is no CPU path)");
  const Pool pool(a[1], "pool");
  const Tensor& table = table_of(a[2], pool.device());
  const ra_dtype_t code = dtype_code(q);
  const int B = size32(table.size(0)), M = size32(table.size(1)), Hq = size32(q.size(1));
  if (q.device() != pool.device() || q.size(0) != B || q.size(2) != pool.D || Hq < 1 || Hq % pool.Hkv)
    refuse("q must be [B, H, head_dim] on the pool's device, with H a multiple of the key heads, B as in the table");
  const Tensor& length = tensor(a[3], "length");
  check("length", length, {B}, at::kInt, pool.device());
  const float scale = a[4] == Py_None ? 0.0f : number(a[4]);
  // an address that the kernels cannot read as it is
  const Tensor in = reinterpret_cast<uintptr_t>(q.data_ptr()) & 15 ? q.clone(at::MemoryFormat::Contiguous) : q;
  const Tensor o = make({B, Hq, pool.D}, q.scalar_type(), pool.device());
  const Tensor ws = make({static_cast<int64_t>(ra_attention_decode_paged_workspace_size(B, Hq, pool.Hkv, M, pool.page, pool.D)) + 16},
                         at::kByte, pool.device());
  check_status("ra_attention_decode_paged", on_stream(pool.device(), [&](cudaStream_t st) {
                 return ra_attention_decode_paged(in.data_ptr(), pool.data(), pool.stride, ints(table), ints(length), o.data_ptr(),
                                                  ws.data_ptr(), B, Hq, pool.Hkv, pool.D, pool.pages, pool.page, M, scale, code, st);
               }));
  return THPVariable_Wrap(o);
}

// table, length, uses, parent
PyObject* page_fork(PyObject* const* a) {
  const Tensor& first = tensor(a[0], "table");
  if (!first.is_cuda()) refuse("table must be a CUDA tensor (there is no CPU path)");
  const at::Device device = first.device();
  const Tensor &table = table_of(a[0], device), &length = tensor(a[1], "length"), &uses = tensor(a[2], "uses"),
               &parent = tensor(a[3], "parent");
  const int B = size32(table.size(0)), M = size32(table.size(1));
  if (uses.dim() != 1 || uses.size(0) < 1) refuse("uses must be [pages]");
  check("length", length, {B}, at::kInt, device);
  check("uses", uses, {uses.size(0)}, at::kInt, device);
  check("parent", parent, {B}, at::kInt, device);
  const int pages = size32(uses.size(0));
  check_status("ra_page_fork", on_stream(device, [&](cudaStream_t st) {
                 return ra_page_fork(ints(table), ints(length), ints(uses), ints(parent), B, M, pages, st);
               }));
  Py_RETURN_NONE;
}

// pool, table, length, uses, tokens, count
PyObject* page_reserve(PyObject* const* a) {
  const Pool pool(a[0], "pool");
  const at::Device device = pool.device();
  const Tensor &table = table_of(a[1], device), &length = tensor(a[2], "length"), &uses = tensor(a[3], "uses");
  const int B = size32(table.size(0)), M = size32(table.size(1)), tokens = integer(a[4]);
  check("length", length, {B}, at::kInt, device);
  check("uses", uses, {pool.pages}, at::kInt, device);
  const Tensor* count = per_sequence(a[5], "count", B, device);
  if (tokens < 1) refuse("tokens must be at least 1");
  const Tensor granted = make({B}, at::kInt, device);
  const Tensor ws = make({static_cast<int64_t>(ra_page_reserve_workspace_size(B, tokens, pool.page)) + 16}, at::kByte, device);
  check_status("ra_page_reserve", on_stream(device, [&](cudaStream_t st) {
                 return ra_page_reserve(pool.data(), pool.stride, pool.bytes, ints(table), ints(length), ints(uses), ints(count),
                                        ints(granted), ws.data_ptr(), B, M, tokens, pool.pages, pool.page, st);
               }));
  return THPVariable_Wrap(granted);
}

// pool, table, uses, out
PyObject* page_compact(PyObject* const* a) {
  const Pool pool(a[0], "pool"), out(a[3], "out");
  const at::Device device = pool.device();
  const Tensor &table = table_of(a[1], device), &uses = tensor(a[2], "uses");
  const int B = size32(table.size(0)), M = size32(table.size(1));
  check("uses", uses, {pool.pages}, at::kInt, device);
  if (out.device() != device || out.Hkv != pool.Hkv || out.page != pool.page || out.D != pool.D)
    refuse("out must be a pool of the same heads, pages' size and head_dim on the same device");
  const char *p0 = static_cast<const char*>(pool.data()), *p1 = p0 + (pool.pages - 1) * pool.stride + pool.bytes;
  const char *o0 = static_cast<const char*>(out.data()), *o1 = o0 + (out.pages - 1) * out.stride + out.bytes;
  // slices of one tensor may interleave (layers); what must not happen is that a page of one lies in a page of the other
  const int64_t apart = ((o0 - p0) % pool.stride + pool.stride) % pool.stride;
  const bool interleaved = pool.stride == out.stride && apart >= pool.bytes && apart + pool.bytes <= pool.stride;
  if (o0 < p1 && p0 < o1 && !interleaved) refuse("out must not share memory with pool");
  const Tensor table_out = make({B, M}, at::kInt, device), uses_out = make({out.pages}, at::kInt, device), live = make({1}, at::kInt, device);
  const Tensor ws = make({static_cast<int64_t>(ra_page_compact_workspace_size(pool.pages)) + 16}, at::kByte, device);
  check_status("ra_page_compact", on_stream(device, [&](cudaStream_t st) {
                 return ra_page_compact(pool.data(), pool.stride, ints(table), ints(uses), out.data(), out.stride, ints(table_out),
                                        ints(uses_out), ints(live), ws.data_ptr(), pool.bytes, B, M, pool.pages, out.pages, st);
               }));
  return tuple({table_out, uses_out, live});
}

template <PyObject* (*F)(PyObject* const*), int COUNT>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != COUNT) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %d expected", n, COUNT);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refusal& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int COUNT>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, COUNT>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<norm_rope, kLead>("norm_rope"),
                         method<norm_rope_backward, kLead + 3>("norm_rope_backward"),
                         method<cache_append, kLead + 4>("cache_append"),
                         method<attention_decode, 8>("attention_decode"),
                         method<cache_evict, 7>("cache_evict"),
                         method<page_write, 7>("page_write"),
                         method<page_read, 6>("page_read"),
                         method<attention_decode_paged, 5>("attention_decode_paged"),
                         method<page_fork, 4>("page_fork"),
                         method<page_reserve, 6>("page_reserve"),
                         method<page_compact, 4>("page_compact"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
