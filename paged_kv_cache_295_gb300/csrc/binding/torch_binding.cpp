// Python entry points of the block-scaled cache, of windowed attention and of the step around
// the cache (slots, rotary positions, packed prompts), taking torch tensors (module _pkv_torch).  A serving loop makes these calls once per
// layer and step, where the checks and the marshalling of ten tensors in Python cost
// more than the kernel; here they take about a microsecond.  Each function checks its
// arguments, makes the tensors' device current, allocates what the caller did not
// give, and makes one call of include/pagedkv.h on the current stream.
//
// A refused argument raises ValueError; a pkv_status other than PKV_OK is returned as
// an int, which the package turns into its own exception.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <stdexcept>
#include <string>
#include <utility>

#include "pagedkv.h"

namespace {

using at::Tensor;

struct Refusal : std::runtime_error {   // becomes ValueError
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string& why) { throw Refusal(why); }

std::string show(const Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] of " + std::string(c10::toString(t.scalar_type()));
}

// A tensor argument; None gives an undefined one where that is allowed.
const Tensor& tensor(PyObject* o, const char* name, bool optional = false) {
  static const Tensor none;
  if (optional && o == Py_None) return none;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}

float real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
}

int32_t code_of(at::ScalarType t) {   // pkv_dtype
  switch (t) {
    case at::kFloat: return PKV_F32;
    case at::kBFloat16: return PKV_BF16;
    case at::kByte:
    case at::kFloat8_e4m3fn: return PKV_FP8_E4M3;
    case at::kChar: return PKV_INT8;
    default: refuse("unsupported dtype " + std::string(c10::toString(t)));
  }
}
bool is_codes(int32_t code) { return code == PKV_FP8_E4M3 || code == PKV_INT8; }

void want(const Tensor& t, const char* name, std::initializer_list<int64_t> shape,
          std::initializer_list<at::ScalarType> types) {
  bool ok = t.sizes() == at::IntArrayRef(shape), typed = false;
  for (at::ScalarType s : types) typed = typed || t.scalar_type() == s;
  if (ok && typed) return;
  std::string s = std::string(name) + " must be [";
  int i = 0;
  for (int64_t n : shape) s += (i++ ? ", " : "") + std::to_string(n);
  s += "] of";
  i = 0;
  for (at::ScalarType ty : types) s += std::string(i++ ? " or " : " ") + c10::toString(ty);
  refuse(s + ", got " + show(t));
}

// The device pointer of a contiguous tensor on `dev`; null for an undefined one.
void* ptr(const Tensor& t, const char* name, const at::Device& dev) {
  if (!t.defined()) return nullptr;
  if (t.device() != dev)
    refuse(std::string(name) + " is on " + t.device().str() + ", the call on " + dev.str());
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t.data_ptr();
}
template <typename T>
T* ptr_as(const Tensor& t, const char* name, const at::Device& dev) {
  return static_cast<T*>(ptr(t, name, dev));
}

at::Device cuda_device(const Tensor& t) {
  if (!t.is_cuda()) refuse("CUDA tensors are needed (no CPU path)");
  return t.device();
}

pkv_stream_t stream_of(const at::Device& dev) {
  return reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

struct Cache {
  int64_t blocks;
  int32_t block_size, heads, dim, code;
};
Cache cache_of(const Tensor& k, const Tensor& v) {
  if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
    refuse("k_cache and v_cache must be alike, [num_blocks, block_size, num_kv_heads, head_dim]; got " +
           show(k) + " and " + show(v));
  for (int i = 1; i < 4; ++i)
    if (k.size(i) > INT32_MAX) refuse("a cache dimension is out of range");
  return {k.size(0), static_cast<int32_t>(k.size(1)), static_cast<int32_t>(k.size(2)),
          static_cast<int32_t>(k.size(3)), code_of(k.scalar_type())};
}

int32_t count32(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + " has too many rows");
  return static_cast<int32_t>(n);
}

int32_t tables_width(const Tensor& bt, int64_t seqs) {
  if (bt.dim() != 2 || bt.size(0) != seqs || bt.scalar_type() != at::kInt)
    refuse("block_tables must be Int [" + std::to_string(seqs) + ", max_blocks], got " + show(bt));
  return count32(bt.size(1), "block_tables");
}

// Floats between the scales of two blocks; 0 for one scale per head ([heads], or any shape of as
// many elements).
int64_t scale_stride(const Tensor& ks, const Tensor& vs, const Cache& c) {
  if (!ks.defined() || !vs.defined()) refuse("an 8-bit cache needs k_scale and v_scale");
  auto stride = [&](const Tensor& t) -> int64_t {   // -1: neither form
    if (t.scalar_type() != at::kFloat) return -1;
    if (t.dim() == 2 && t.size(0) == c.blocks && t.size(1) >= c.heads) return t.size(1);
    return t.numel() == c.heads ? 0 : -1;
  };
  if (stride(ks) < 0 || stride(vs) != stride(ks))
    refuse("k_scale and v_scale must be Float [" + std::to_string(c.heads) + "] or [" +
           std::to_string(c.blocks) + ", >= " + std::to_string(c.heads) + "], both alike, got " +
           show(ks) + " and " + show(vs));
  return stride(ks);
}

at::ScalarType out_type(PyObject* dtype, const Tensor& out, at::ScalarType otherwise) {
  if (dtype != Py_None) {
    if (!THPDtype_Check(dtype)) refuse("out_dtype must be a torch.dtype");
    const at::ScalarType t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    if (out.defined() && out.scalar_type() != t)
      refuse("the output is " + std::string(c10::toString(out.scalar_type())) + ", out_dtype " +
             c10::toString(t));
    return t;
  }
  return out.defined() ? out.scalar_type() : otherwise;
}

// The status word: an int32 on the device, or None.
const Tensor& status_word(PyObject* o) {
  const Tensor& t = tensor(o, "device_status", true);
  if (t.defined() && (t.scalar_type() != at::kInt || t.numel() < 1))
    refuse("device_status must be Int with at least one element, got " + show(t));
  return t;
}

void arity(Py_ssize_t n, Py_ssize_t wanted) {
  if (n != wanted) refuse("wrong number of arguments");
}

PyObject* status(pkv_status s) { return PyLong_FromLong(s); }

// quantize_and_cache(k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables,
//                    context_lens, query_start, max_query_len, device_status) -> status
PyObject* do_quantize(PyObject* const* a, Py_ssize_t na) {
  arity(na, 11);
  const Tensor &kn = tensor(a[0], "k_new"), &vn = tensor(a[1], "v_new"), &kc = tensor(a[2], "k_cache"),
               &vc = tensor(a[3], "v_cache"), &ks = tensor(a[4], "k_scales"),
               &vs = tensor(a[5], "v_scales"), &bt = tensor(a[6], "block_tables"),
               &cl = tensor(a[7], "context_lens"), &qs = tensor(a[8], "query_start", true),
               &st = status_word(a[10]);
  const int32_t max_query = integer32(a[9], "max_query_len");
  const Cache c = cache_of(kc, vc);
  if (kn.dim() != 3 || cl.dim() != 1) refuse("k_new must be [T, heads, dim] and context_lens [S]");
  const int64_t T = kn.size(0), S = cl.size(0);
  want(kn, "k_new", {T, c.heads, c.dim}, {at::kFloat, at::kBFloat16});
  want(vn, "v_new", {T, c.heads, c.dim}, {kn.scalar_type()});
  want(cl, "context_lens", {S}, {at::kInt});
  const int32_t mb = tables_width(bt, S);
  if (qs.defined()) want(qs, "query_start", {S + 1}, {at::kInt});
  const int64_t stride = scale_stride(ks, vs, c);
  if (stride == 0) refuse("k_scales and v_scales must be [num_blocks, >= num_kv_heads]");
  const at::Device dev = cuda_device(kn);
  const c10::cuda::CUDAGuard guard(dev);
  const void *knp = ptr(kn, "k_new", dev), *vnp = ptr(vn, "v_new", dev);
  const int32_t *qsp = ptr_as<int32_t>(qs, "query_start", dev), *btp = ptr_as<int32_t>(bt, "block_tables", dev),
                *clp = ptr_as<int32_t>(cl, "context_lens", dev);
  void *kcp = ptr(kc, "k_cache", dev), *vcp = ptr(vc, "v_cache", dev);
  float *ksp = ptr_as<float>(ks, "k_scales", dev), *vsp = ptr_as<float>(vs, "v_scales", dev);
  int32_t* stp = ptr_as<int32_t>(st, "device_status", dev);
  const int32_t src = code_of(kn.scalar_type()), t32 = count32(T, "k_new"), s32 = count32(S, "context_lens");
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = quantize_and_cache(knp, vnp, qsp, btp, clp, kcp, vcp, ksp, vsp, s32, t32, max_query, c.heads, c.dim,
                         c.block_size, c.blocks, mb, stride, src, c.code, stp, stream);
  Py_END_ALLOW_THREADS
  return status(r);
}

// gather_cache(k_cache, v_cache, block_tables, row_start, num_rows, max_rows, first_pos, k_scale,
//              v_scale, out_dtype, k_out, v_out, device_status) -> (k, v) or status
PyObject* do_gather(PyObject* const* a, Py_ssize_t na) {
  arity(na, 13);
  const Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache"),
               &bt = tensor(a[2], "block_tables"), &rs = tensor(a[3], "row_start"),
               &fp = tensor(a[6], "first_pos", true), &st = status_word(a[12]);
  const int64_t rows = integer32(a[4], "num_rows");
  const int32_t max_rows = integer32(a[5], "max_rows");
  const Cache c = cache_of(kc, vc);
  const bool codes = is_codes(c.code);
  const Tensor none, &ks = codes ? tensor(a[7], "k_scale", true) : none,
                     &vs = codes ? tensor(a[8], "v_scale", true) : none;
  Tensor ko = tensor(a[10], "k_out", true), vo = tensor(a[11], "v_out", true);
  if (bt.dim() != 2) refuse("block_tables must be [S, max_blocks]");
  const int64_t S = bt.size(0);
  const int32_t mb = tables_width(bt, S);
  want(rs, "row_start", {S + 1}, {at::kInt});
  if (fp.defined()) want(fp, "first_pos", {S}, {at::kInt});
  const int64_t stride = codes ? scale_stride(ks, vs, c) : 0;
  if (rows < 0) refuse("num_rows is negative");
  const at::ScalarType type = out_type(a[9], ko, at::kBFloat16);
  const int32_t out = code_of(type);
  const at::Device dev = cuda_device(kc);
  const c10::cuda::CUDAGuard guard(dev);
  if (!ko.defined()) ko = at::empty({rows, c.heads, c.dim}, kc.options().dtype(type));
  if (!vo.defined()) vo = at::empty({rows, c.heads, c.dim}, kc.options().dtype(type));
  want(ko, "k_out", {rows, c.heads, c.dim}, {type});
  want(vo, "v_out", {rows, c.heads, c.dim}, {type});
  const void *kcp = ptr(kc, "k_cache", dev), *vcp = ptr(vc, "v_cache", dev);
  const int32_t *btp = ptr_as<int32_t>(bt, "block_tables", dev), *rsp = ptr_as<int32_t>(rs, "row_start", dev),
                *fpp = ptr_as<int32_t>(fp, "first_pos", dev);
  const float *ksp = ptr_as<float>(ks, "k_scale", dev), *vsp = ptr_as<float>(vs, "v_scale", dev);
  void *kop = ptr(ko, "k_out", dev), *vop = ptr(vo, "v_out", dev);
  int32_t* stp = ptr_as<int32_t>(st, "device_status", dev);
  const int32_t s32 = count32(S, "block_tables");
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = gather_cache(kcp, vcp, btp, rsp, fpp, s32, static_cast<int32_t>(rows), max_rows, c.heads, c.dim,
                   c.block_size, c.blocks, mb, c.code, ksp, vsp, stride, out, kop, vop, stp, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  PyObject *k = THPVariable_Wrap(std::move(ko)), *v = THPVariable_Wrap(std::move(vo));
  PyObject* both = k && v ? PyTuple_Pack(2, k, v) : nullptr;
  Py_XDECREF(k);
  Py_XDECREF(v);
  return both;
}

// What the two attention calls have in common.
struct Attention {
  const Tensor &q, &kc, &vc, &bt, &cl;
  Cache c;
  int64_t T, S;
  int32_t q_heads, mb, q_code;
  int64_t stride;
  Attention(PyObject* oq, PyObject* okc, PyObject* ovc, PyObject* obt, PyObject* ocl, const Tensor& ks,
            const Tensor& vs)
      : q(tensor(oq, "q")), kc(tensor(okc, "k_cache")), vc(tensor(ovc, "v_cache")),
        bt(tensor(obt, "block_tables")), cl(tensor(ocl, "context_lens")), c(cache_of(kc, vc)) {
    if (q.dim() != 3 || cl.dim() != 1) refuse("q must be [T, heads, dim] and context_lens [S]");
    T = q.size(0);
    S = cl.size(0);
    q_heads = count32(q.size(1), "q");
    want(q, "q", {T, q.size(1), c.dim}, {at::kFloat, at::kBFloat16});
    want(cl, "context_lens", {S}, {at::kInt});
    mb = tables_width(bt, S);
    q_code = code_of(q.scalar_type());
    stride = is_codes(c.code) ? scale_stride(ks, vs, c) : 0;
    count32(T, "q");
    count32(S, "context_lens");
  }
};

Tensor attention_out(const Attention& at_, Tensor out, PyObject* dtype) {
  const at::ScalarType type = out_type(dtype, out, at::kFloat);
  if (type != at::kFloat && type != at::kBFloat16) refuse("the output must be Float or BFloat16");
  if (!out.defined()) out = at::empty(at_.q.sizes(), at_.q.options().dtype(type));
  want(out, "out", {at_.T, at_.q_heads, at_.c.dim}, {type});
  return out;
}

// decode_window(q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, out,
//               k_scale, v_scale, workspace, partition, device_status, window, sinks, out_dtype)
//   -> out or status
PyObject* do_decode(PyObject* const* a, Py_ssize_t na) {
  arity(na, 16);
  Tensor ks = tensor(a[8], "k_scale", true), vs = tensor(a[9], "v_scale", true);
  const Attention p(a[0], a[1], a[2], a[3], a[4], ks, vs);
  if (!is_codes(p.c.code)) ks = vs = Tensor();
  if (p.T != p.S)
    refuse("q must hold one row per sequence: " + std::to_string(p.T) + " rows, " + std::to_string(p.S) +
           " contexts");
  const float scale = real(a[5], "scale");
  const int32_t max_ctx = integer32(a[6], "max_context_len"), part = integer32(a[11], "partition"),
                window = integer32(a[13], "window"), sinks = integer32(a[14], "sinks");
  const Tensor& st = status_word(a[12]);
  const at::Device dev = cuda_device(p.q);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out = attention_out(p, tensor(a[7], "out", true), a[15]), ws = tensor(a[10], "workspace", true);
  const size_t need = paged_attention_window_call_bytes(static_cast<int32_t>(p.S), p.q_heads, p.c.heads,
                                                        p.c.dim, max_ctx, part, window, sinks, p.c.code);
  if (need > (ws.defined() ? ws.nbytes() : 0))
    ws = at::empty({static_cast<int64_t>(need)}, p.q.options().dtype(at::kByte));
  const void *q = ptr(p.q, "q", dev), *kc = ptr(p.kc, "k_cache", dev), *vc = ptr(p.vc, "v_cache", dev);
  const int32_t *bt = ptr_as<int32_t>(p.bt, "block_tables", dev),
                *cl = ptr_as<int32_t>(p.cl, "context_lens", dev);
  const float *ksp = ptr_as<float>(ks, "k_scale", dev), *vsp = ptr_as<float>(vs, "v_scale", dev);
  void *op = ptr(out, "out", dev), *wp = ptr(ws, "workspace", dev);
  int32_t* stp = ptr_as<int32_t>(st, "device_status", dev);
  const size_t ws_bytes = ws.defined() ? ws.nbytes() : 0;
  const int32_t type = code_of(out.scalar_type());
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = paged_attention_decode_window(q, kc, vc, bt, cl, static_cast<int32_t>(p.S), p.q_heads, p.c.heads,
                                    p.c.dim, p.c.block_size, p.c.blocks, p.mb, max_ctx, scale, p.q_code,
                                    p.c.code, ksp, vsp, p.stride, window, sinks, type, op, wp, ws_bytes,
                                    part, stp, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  return THPVariable_Wrap(std::move(out));
}

// prefill_window(q, query_start, k_cache, v_cache, block_tables, context_lens, scale, max_query_len,
//                max_context_len, causal, out, k_scale, v_scale, device_status, window, sinks,
//                out_dtype) -> out or status
PyObject* do_prefill(PyObject* const* a, Py_ssize_t na) {
  arity(na, 17);
  Tensor ks = tensor(a[11], "k_scale", true), vs = tensor(a[12], "v_scale", true);
  const Attention p(a[0], a[2], a[3], a[4], a[5], ks, vs);
  if (!is_codes(p.c.code)) ks = vs = Tensor();
  const Tensor &qs = tensor(a[1], "query_start"), &st = status_word(a[13]);
  want(qs, "query_start", {p.S + 1}, {at::kInt});
  const float scale = real(a[6], "scale");
  const int32_t max_query = integer32(a[7], "max_query_len"), max_ctx = integer32(a[8], "max_context_len"),
                window = integer32(a[14], "window"), sinks = integer32(a[15], "sinks");
  const int causal = PyObject_IsTrue(a[9]);
  if (causal < 0) {
    PyErr_Clear();
    refuse("causal must be a truth value");
  }
  const at::Device dev = cuda_device(p.q);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out = attention_out(p, tensor(a[10], "out", true), a[16]);
  const void *q = ptr(p.q, "q", dev), *kc = ptr(p.kc, "k_cache", dev), *vc = ptr(p.vc, "v_cache", dev);
  const int32_t *qsp = ptr_as<int32_t>(qs, "query_start", dev),
                *bt = ptr_as<int32_t>(p.bt, "block_tables", dev),
                *cl = ptr_as<int32_t>(p.cl, "context_lens", dev);
  const float *ksp = ptr_as<float>(ks, "k_scale", dev), *vsp = ptr_as<float>(vs, "v_scale", dev);
  void* op = ptr(out, "out", dev);
  int32_t* stp = ptr_as<int32_t>(st, "device_status", dev);
  const int32_t type = code_of(out.scalar_type());
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = paged_attention_prefill_window(q, qsp, kc, vc, bt, cl, static_cast<int32_t>(p.S),
                                     static_cast<int32_t>(p.T), max_query, p.q_heads, p.c.heads, p.c.dim,
                                     p.c.block_size, p.c.blocks, p.mb, max_ctx, scale, causal, p.q_code,
                                     p.c.code, ksp, vsp, p.stride, window, sinks, type, op, stp, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  return THPVariable_Wrap(std::move(out));
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a truth value");
  }
  return v != 0;
}

// The device pointer of a tensor of this type and shape, allocated where it was not given.
template <typename T>
T* made(Tensor& t, const char* name, std::initializer_list<int64_t> shape, at::ScalarType type,
        const at::Device& dev) {
  if (!t.defined()) t = at::empty(at::IntArrayRef(shape), at::TensorOptions().dtype(type).device(dev));
  want(t, name, shape, {type});
  return ptr_as<T>(t, name, dev);
}

PyObject* wrapped(Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}
// A tuple of tensors (None for an undefined one).
template <size_t N>
PyObject* tuple_of(Tensor (&ts)[N]) {
  PyObject* out = PyTuple_New(N);
  if (!out) return nullptr;
  for (size_t i = 0; i < N; ++i) {
    PyObject* o = wrapped(std::move(ts[i]));
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i, o);
  }
  return out;
}

// slots_from_lengths(block_tables, context_lens, new_lens, free_blocks, num_blocks, block_size,
//                    num_tokens, free_start, row_per_sequence, first_block_held, slot_mapping,
//                    positions, query_start, context_out, free_next, device_status)
//   -> (slot_mapping, positions, query_start, context_out, free_next) or status
PyObject* do_slots(PyObject* const* a, Py_ssize_t na) {
  arity(na, 16);
  const Tensor &bt = tensor(a[0], "block_tables"), &cl = tensor(a[1], "context_lens"),
               &nl = tensor(a[2], "new_lens", true), &fb = tensor(a[3], "free_blocks"),
               &fs = tensor(a[7], "free_start", true), &st = status_word(a[15]);
  const int64_t blocks = integer(a[4], "num_blocks");
  const int32_t block = integer32(a[5], "block_size");
  const bool per_row = truth(a[8], "row_per_sequence"), held = truth(a[9], "first_block_held");
  if (cl.dim() != 1) refuse("context_lens must be [S]");
  const int64_t S = cl.size(0);
  const int64_t T = a[6] == Py_None && per_row ? S : integer32(a[6], "num_tokens");
  if (T < 0) refuse("num_tokens is negative");
  want(cl, "context_lens", {S}, {at::kInt});
  if (nl.defined()) want(nl, "new_lens", {S}, {at::kInt});
  if (fb.dim() != 1) refuse("free_blocks must be [F]");
  want(fb, "free_blocks", {fb.size(0)}, {at::kInt});
  if (fs.defined()) want(fs, "free_start", {1}, {at::kInt});
  const int32_t mb = tables_width(bt, S), s32 = count32(S, "context_lens"), f32 = count32(fb.size(0), "free_blocks");
  const at::Device dev = cuda_device(cl);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out[5] = {tensor(a[10], "slot_mapping", true), tensor(a[11], "positions", true),
                   tensor(a[12], "query_start", true), tensor(a[13], "context_out", true),
                   tensor(a[14], "free_next", true)};
  int64_t* slots = made<int64_t>(out[0], "slot_mapping", {T}, at::kLong, dev);
  int32_t* pos = made<int32_t>(out[1], "positions", {T}, at::kInt, dev);
  if (per_row && out[2].defined()) refuse("query_start is not written with row_per_sequence");
  int32_t* qs = per_row ? nullptr : made<int32_t>(out[2], "query_start", {S + 1}, at::kInt, dev);
  int32_t* co = made<int32_t>(out[3], "context_out", {S}, at::kInt, dev);
  int32_t* fn = made<int32_t>(out[4], "free_next", {1}, at::kInt, dev);
  int32_t *btp = ptr_as<int32_t>(bt, "block_tables", dev), *stp = ptr_as<int32_t>(st, "device_status", dev);
  const int32_t *clp = ptr_as<int32_t>(cl, "context_lens", dev), *nlp = ptr_as<int32_t>(nl, "new_lens", dev),
                *fbp = ptr_as<int32_t>(fb, "free_blocks", dev), *fsp = ptr_as<int32_t>(fs, "free_start", dev);
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = slots_from_lengths(btp, clp, nlp, fbp, fsp, s32, static_cast<int32_t>(T), f32, blocks, block, mb, per_row,
                         held, slots, pos, qs, co, fn, stp, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  return tuple_of(out);
}

// Rows [T, heads, dim] whose elements lie side by side; any strides between rows and heads.
void want_rows(const Tensor& t, const char* name, int64_t rows, int64_t heads, int64_t dim,
               at::ScalarType type, const at::Device& dev, bool written = false) {
  want(t, name, {rows, heads, dim}, {type});
  if (t.device() != dev) refuse(std::string(name) + " is on " + t.device().str() + ", the call on " + dev.str());
  if (t.numel() == 0) return;
  if (dim > 1 && t.stride(2) != 1) refuse(std::string(name) + " must have its last dimension contiguous");
  if (!written) return;
  const int inner = t.size(0) > 1 && (t.size(1) <= 1 || t.stride(0) < t.stride(1)) ? 0 : 1, outer = 1 - inner;
  const int64_t span = t.size(inner) > 1 ? (t.size(inner) - 1) * t.stride(inner) + dim : dim;
  if ((t.size(inner) > 1 && t.stride(inner) < dim) || (t.size(outer) > 1 && t.stride(outer) < span))
    refuse(std::string(name) + " must not overlap itself");
}

// What rotary_and_cache takes beside q, k, v and the outputs.
struct RotaryTensors {
  PyObject* const* plan;   // (turns, axis, rotary_dim, num_axes, adjacent, scale)
  const Tensor &pos, &turns, &axis, &slots, &kc, &vc, &ks, &vs;
  // positions, plan, slot_mapping, k_cache, v_cache, k_scale, v_scale
  explicit RotaryTensors(PyObject* const* a)
      : plan(items(a[1])), pos(tensor(a[0], "positions")), turns(tensor(plan[0], "turns")),
        axis(tensor(plan[1], "axis", true)), slots(tensor(a[2], "slot_mapping", true)),
        kc(tensor(a[3], "k_cache", true)), vc(tensor(a[4], "v_cache", true)), ks(tensor(a[5], "k_scale", true)),
        vs(tensor(a[6], "v_scale", true)) {}
  static PyObject* const* items(PyObject* plan) {
    if (!PyTuple_Check(plan) || PyTuple_GET_SIZE(plan) != 6) refuse("rotary must be a Rotary's plan");
    return &PyTuple_GET_ITEM(plan, 0);
  }
};

// The call's arguments, checked; outputs that are not given are allocated on the current device.
pkv_rotary_args rotary_args(const Tensor& q, const Tensor& k, const Tensor& v, const RotaryTensors& x, Tensor (&out)[2],
                            bool keep_k, const Tensor& st) {
  const auto &[plan, pos, turns, axis, slots, kc, vc, ks, vs] = x;
  const bool cached = kc.defined();
  pkv_rotary_args p{};
  p.rotary_dim = integer32(plan[2], "rotary_dim");
  p.num_axes = integer32(plan[3], "num_axes");
  p.adjacent = truth(plan[4], "adjacent");
  p.scale = real(plan[5], "scale");
  if (k.dim() != 3 || (q.defined() && q.dim() != 3)) refuse("q and k must be [T, heads, dim]");
  const int64_t T = k.size(0), hkv = k.size(1), dim = k.size(2), hq = q.defined() ? q.size(1) : 0;
  const at::ScalarType type = k.scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) refuse("k must be Float or BFloat16, got " + show(k));
  if (hq > (1 << 20) || hkv > (1 << 20) || dim > (1 << 20)) refuse("too many heads or dims");
  const at::Device dev = cuda_device(k);
  want_rows(k, "k", T, hkv, dim, type, dev);
  if (q.defined()) {
    want_rows(q, "q", T, hq, dim, type, dev);
    if (!out[0].defined()) out[0] = at::empty({T, hq, dim}, q.options());
    want_rows(out[0], "q_out", T, hq, dim, type, dev, true);
  } else if (out[0].defined()) {
    refuse("q_out without q");
  }
  if (!out[1].defined() && (keep_k || !cached)) out[1] = at::empty({T, hkv, dim}, k.options());
  if (out[1].defined()) want_rows(out[1], "k_out", T, hkv, dim, type, dev, true);
  if (p.rotary_dim < 0 || p.rotary_dim % 2 != 0 || p.rotary_dim > dim)
    refuse("rotary_dim must be even and at most " + std::to_string(dim));
  want(turns, "turns", {p.rotary_dim / 2}, {at::kLong});
  if (axis.defined()) want(axis, "axis", {p.rotary_dim / 2}, {at::kInt});
  if (p.num_axes == 1 && pos.dim() == 1)
    want(pos, "positions", {T}, {at::kInt});
  else
    want(pos, "positions", {p.num_axes, T}, {at::kInt});
  if (cached) {
    const Cache c = cache_of(kc, vc);
    if (c.heads != hkv || c.dim != dim)
      refuse("the caches must be [num_blocks, block_size, " + std::to_string(hkv) + ", " + std::to_string(dim) +
             "], got " + show(kc));
    if (!v.defined()) refuse("v must be a tensor");
    if (!slots.defined()) refuse("slot_mapping must be a tensor");
    want_rows(v, "v", T, hkv, dim, type, dev);
    want(slots, "slot_mapping", {T}, {at::kLong});
    if (is_codes(c.code)) {
      if (scale_stride(ks, vs, c) != 0)
        refuse("rotary_and_cache takes one scale per head, not scales per block");
      p.k_scale = ptr_as<float>(ks, "k_scale", dev);
      p.v_scale = ptr_as<float>(vs, "v_scale", dev);
    }
    p.slot_mapping = ptr_as<int64_t>(slots, "slot_mapping", dev);
    p.k_cache = ptr(kc, "k_cache", dev);
    p.v_cache = ptr(vc, "v_cache", dev);
    p.block_size = c.block_size;
    p.num_blocks = c.blocks;
    p.cache_dtype = c.code;
    p.v = v.data_ptr();
    p.v_token_stride = v.stride(0);
    p.v_head_stride = v.stride(1);
  } else if (vc.defined()) {
    refuse("v_cache without k_cache");
  }
  p.k = k.data_ptr();
  p.k_token_stride = k.stride(0);
  p.k_head_stride = k.stride(1);
  if (q.defined()) {
    p.q = q.data_ptr();
    p.q_token_stride = q.stride(0);
    p.q_head_stride = q.stride(1);
    p.q_out = out[0].data_ptr();
    p.q_out_token_stride = out[0].stride(0);
    p.q_out_head_stride = out[0].stride(1);
  }
  if (out[1].defined()) {
    p.k_out = out[1].data_ptr();
    p.k_out_token_stride = out[1].stride(0);
    p.k_out_head_stride = out[1].stride(1);
  }
  p.num_tokens = count32(T, "k");
  p.num_q_heads = static_cast<int32_t>(hq);
  p.num_kv_heads = static_cast<int32_t>(hkv);
  p.head_dim = static_cast<int32_t>(dim);
  p.src_dtype = code_of(type);
  p.turns = reinterpret_cast<const uint64_t*>(ptr_as<int64_t>(turns, "turns", dev));
  p.axis = ptr_as<int32_t>(axis, "axis", dev);
  p.positions = ptr_as<int32_t>(pos, "positions", dev);
  p.device_status = ptr_as<int32_t>(st, "device_status", dev);
  return p;
}

// rotary_and_cache(q, k, v, positions, plan, slot_mapping, k_cache, v_cache, k_scale, v_scale, q_out, k_out,
//                  keep_k, device_status) -> (q_out, k_out) or status
PyObject* do_rotary(PyObject* const* a, Py_ssize_t na) {
  arity(na, 14);
  const Tensor &q = tensor(a[0], "q", true), &k = tensor(a[1], "k"), &v = tensor(a[2], "v", true),
               &st = status_word(a[13]);
  const RotaryTensors x(a + 3);
  Tensor out[2] = {tensor(a[10], "q_out", true), tensor(a[11], "k_out", true)};
  const bool keep_k = truth(a[12], "keep_k");
  const at::Device dev = cuda_device(k);
  const c10::cuda::CUDAGuard guard(dev);
  const pkv_rotary_args p = rotary_args(q, k, v, x, out, keep_k, st);
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = rotary_and_cache(&p, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  return tuple_of(out);
}

// The arguments of packed_attention_prefill over these rows, checked; `a`: query_start, scale, key_start, causal,
// window, sinks, weight_parts, context_lens, out, out_dtype, device_status.  `out` is allocated on the current
// device where it is not given.
pkv_packed_prefill_args packed_args(const Tensor& q, const Tensor& k, const Tensor& v, PyObject* const* a, Tensor& out) {
  const Tensor &qs = tensor(a[0], "query_start"), &ks = tensor(a[2], "key_start", true),
               &cl = tensor(a[7], "context_lens", true), &st = status_word(a[10]);
  if (q.dim() != 3 || k.dim() != 3) refuse("q, k and v must be [T, heads, dim]");
  if (qs.dim() != 1 || qs.size(0) < 1) refuse("query_start must be [S + 1]");
  const int64_t T = q.size(0), hq = q.size(1), dim = q.size(2), N = k.size(0), hkv = k.size(1), S = qs.size(0) - 1;
  if (hq > (1 << 20) || hkv > (1 << 20) || dim > (1 << 20)) refuse("too many heads or dims");
  pkv_packed_prefill_args p{};
  p.scale = real(a[1], "scale");
  p.causal = truth(a[3], "causal");
  p.window = integer32(a[4], "window");
  p.sinks = integer32(a[5], "sinks");
  p.weight_parts = integer32(a[6], "weight_parts");
  if (p.weight_parts < 1) refuse("weight_parts must be 1 or 2");
  const at::Device dev = cuda_device(q);
  want_rows(q, "q", T, hq, dim, at::kBFloat16, dev);
  want_rows(k, "k", N, hkv, dim, at::kBFloat16, dev);
  want_rows(v, "v", N, hkv, dim, at::kBFloat16, dev);
  want(qs, "query_start", {S + 1}, {at::kInt});
  if (ks.defined())
    want(ks, "key_start", {S + 1}, {at::kInt});
  else if (N != T)
    refuse("k must have as many rows as q, or key_start be given");
  for (const auto& x : {std::make_pair(&q, "q"), std::make_pair(&k, "k"), std::make_pair(&v, "v")})
    for (int i = 0; i < 2; ++i)
      if (x.first->numel() > 0 && x.first->size(i) > 1 && (x.first->stride(i) <= 0 || x.first->stride(i) % 8 != 0))
        refuse(std::string(x.second) + " must have strides that are multiples of 8 elements");
  out = tensor(a[8], "out", true);
  const at::ScalarType type = out_type(a[9], out, at::kFloat);
  if (type != at::kFloat && type != at::kBFloat16) refuse("the output must be Float or BFloat16");
  if (!out.defined()) out = at::empty({T, hq, dim}, q.options().dtype(type));
  want(out, "out", {T, hq, dim}, {type});
  p.out = ptr(out, "out", dev);
  p.q = q.data_ptr(), p.k = k.data_ptr(), p.v = v.data_ptr();
  p.q_token_stride = q.stride(0), p.q_head_stride = q.stride(1);
  p.k_token_stride = k.stride(0), p.k_head_stride = k.stride(1);
  p.v_token_stride = v.stride(0), p.v_head_stride = v.stride(1);
  p.query_start = ptr_as<int32_t>(qs, "query_start", dev);
  p.key_start = ptr_as<int32_t>(ks, "key_start", dev);
  if (cl.defined()) want(cl, "context_lens", {S}, {at::kInt});
  p.context_lens = ptr_as<int32_t>(cl, "context_lens", dev);
  p.num_seqs = count32(S, "query_start");
  p.num_tokens = count32(T, "q");
  p.num_keys = count32(N, "k");
  p.num_q_heads = static_cast<int32_t>(hq);
  p.num_kv_heads = static_cast<int32_t>(hkv);
  p.head_dim = static_cast<int32_t>(dim);
  p.q_dtype = p.kv_dtype = PKV_BF16;
  p.out_dtype = code_of(type);
  p.device_status = ptr_as<int32_t>(st, "device_status", dev);
  return p;
}

// packed_prefill(q, k, v, query_start, scale, key_start, causal, window, sinks, weight_parts, context_lens, out,
//                out_dtype, device_status) -> out or status
PyObject* do_packed(PyObject* const* a, Py_ssize_t na) {
  arity(na, 14);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const at::Device dev = cuda_device(q);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor out;
  const pkv_packed_prefill_args p = packed_args(q, k, v, a + 3, out);
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = packed_attention_prefill(&p, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  return THPVariable_Wrap(std::move(out));
}

// prompt(q, k, v, positions, plan, slot_mapping, k_cache, v_cache, k_scale, v_scale, query_start, ... as packed_prefill)
//   -> out or status: rotary_and_cache, then packed_attention_prefill over the turned rows.  What the second
// refuses is refused before the first writes anything.
PyObject* do_prompt(PyObject* const* a, Py_ssize_t na) {
  arity(na, 21);
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &st = status_word(a[20]);
  const RotaryTensors x(a + 3);
  const at::Device dev = cuda_device(k);
  const c10::cuda::CUDAGuard guard(dev);
  Tensor turned[2], out;
  const pkv_rotary_args rp = rotary_args(q, k, v, x, turned, true, st);
  const pkv_packed_prefill_args pp = packed_args(turned[0], turned[1], v, a + 10, out);
  const pkv_stream_t stream = stream_of(dev);
  pkv_status r;
  Py_BEGIN_ALLOW_THREADS
  r = packed_attention_prefill_check(&pp);
  if (r == PKV_OK) r = rotary_and_cache(&rp, stream);
  if (r == PKV_OK) r = packed_attention_prefill(&pp, stream);
  Py_END_ALLOW_THREADS
  if (r != PKV_OK) return status(r);
  return THPVariable_Wrap(std::move(out));
}

// No C++ exception leaves an entry point.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t na) {
  HANDLE_TH_ERRORS
  try {
    return F(a, na);
  } catch (const Refusal& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"quantize_and_cache", reinterpret_cast<PyCFunction>(entry<do_quantize>), METH_FASTCALL, nullptr},
    {"gather_cache", reinterpret_cast<PyCFunction>(entry<do_gather>), METH_FASTCALL, nullptr},
    {"decode_window", reinterpret_cast<PyCFunction>(entry<do_decode>), METH_FASTCALL, nullptr},
    {"prefill_window", reinterpret_cast<PyCFunction>(entry<do_prefill>), METH_FASTCALL, nullptr},
    {"slots_from_lengths", reinterpret_cast<PyCFunction>(entry<do_slots>), METH_FASTCALL, nullptr},
    {"rotary_and_cache", reinterpret_cast<PyCFunction>(entry<do_rotary>), METH_FASTCALL, nullptr},
    {"packed_prefill", reinterpret_cast<PyCFunction>(entry<do_packed>), METH_FASTCALL, nullptr},
    {"prompt", reinterpret_cast<PyCFunction>(entry<do_prompt>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&kModule); }
