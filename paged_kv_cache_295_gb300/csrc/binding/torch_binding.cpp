// Python entry points of the block-scaled cache and of windowed attention, taking
// torch tensors (module _pkv_torch).  A serving loop makes these calls once per
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
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_pkv_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_torch() { return PyModule_Create(&kModule); }
