// Calls of the C ABI straight from torch tensors, for the high-level Python
// functions: the same checks, allocations and entry points as the ctypes
// binding, at a tenth of its host time (reading a tensor's strides and
// pointer, allocating and converting arguments from Python cost 15 to 70 us a
// call, more than the kernels of small calls).  The module holds no kernels
// and links nothing of libbsm.so: bind() receives the addresses of the loaded
// library's functions.  Without this module the ctypes binding serves alone.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <map>
#include <string>
#include <utility>

#include "bsm.h"

namespace {

// ------------------------------------------------------- the bound library
decltype(&bsm_mask_info_bytes) f_mask_info_bytes;
decltype(&bsm_build_mask_info) f_build_mask_info;
decltype(&bsm_splash_fwd_mod) f_splash_fwd_mod;
decltype(&bsm_splash_bwd_mod) f_splash_bwd_mod;
decltype(&bsm_kv_append) f_kv_append;
decltype(&bsm_paged_attention) f_paged_attention;
size_t fwd_workspace_bytes, paged_workspace_bytes;
decltype(&bsm_splash_bwd_workspace_bytes) f_bwd_workspace_bytes;
decltype(&bsm_splash_bwd_mod_workspace_bytes) f_bwd_mod_workspace_bytes;
PyObject* on_status;  // Python callable that raises for a status

// A Python exception is set.
struct Raised {};

[[noreturn]] void value_error(const std::string& msg) {
  PyErr_SetString(PyExc_ValueError, msg.c_str());
  throw Raised{};
}

// Runs a function body; C++ exceptions become Python ones.
template <class F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type =
        torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type != nullptr) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

void check_status(bsm_status s) {
  if (s == BSM_OK) return;
  PyObject* r = PyObject_CallFunction(on_status, "i", static_cast<int>(s));
  if (r != nullptr) {  // it always raises
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, "libbsm call failed");
  }
  throw Raised{};
}

// ---------------------------------------------------------------- arguments
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}

// An undefined tensor for None.
at::Tensor tensor_or_none(PyObject* o, const char* name) {
  return o == Py_None ? at::Tensor() : tensor(o, name);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

int32_t int32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error("integer out of range");
  return static_cast<int32_t>(v);
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

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  throw Raised{};
}

// ------------------------------------------------------------------- views
bsm_tensor view(const at::Tensor& t) {
  if (t.dim() != 4 || t.stride(3) != 1)
    value_error(
        "tensors must be 4-D [B, H, S, D] views with a contiguous head "
        "dimension");
  bsm_tensor v;
  v.data = const_cast<void*>(t.const_data_ptr());
  for (int i = 0; i < 3; ++i) v.strides[i] = t.stride(i);
  return v;
}

template <class T>
T* data(const at::Tensor& t) {
  return t.defined() ? static_cast<T*>(const_cast<void*>(t.const_data_ptr()))
                     : nullptr;
}

size_t bytes_of(const at::Tensor& t) {
  return t.defined() ? static_cast<size_t>(t.nbytes()) : 0;
}

std::string device_name(const at::Device& d) { return d.str(); }

bsm_score_mod score_mod(double softcap, const at::Tensor& slopes, int64_t H,
                        const at::Device& dev) {
  if (slopes.defined() &&
      (slopes.scalar_type() != at::kFloat || slopes.dim() != 1 ||
       slopes.size(0) != H || !slopes.is_contiguous() ||
       slopes.device() != dev))
    value_error("alibi_slopes must be a contiguous float32 tensor [" +
                std::to_string(H) + "] on " + device_name(dev));
  bsm_score_mod m;
  m.softcap = static_cast<float>(softcap);
  m.alibi_slopes = data<const float>(slopes);
  return m;
}

// bf16, or its bits under a 16-bit integer type.
bool bf16_bits(const at::Tensor& t) {
  const at::ScalarType s = t.scalar_type();
  return s == at::kBFloat16 || s == at::kShort || s == at::kUInt16;
}

// Whether t holds the first `sizes` (a larger buffer may serve).
bool covers(const at::Tensor& t, at::IntArrayRef sizes) {
  if (t.dim() != static_cast<int64_t>(sizes.size())) return false;
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) < sizes[i]) return false;
  return true;
}

// The operands of a forward or backward: bf16 tensors of one CUDA device that
// hold what the pointers will be read with (k's heads and length).
void check_operands(const at::Tensor& q, const at::Tensor& k,
                    const at::Tensor& v) {
  const at::Device dev = q.device();
  if (!dev.is_cuda()) value_error("q must be a CUDA tensor");
  const std::pair<const char*, const at::Tensor&> all[3] = {
      {"q", q}, {"k", k}, {"v", v}};
  for (const auto& [name, t] : all) {
    if (t.dim() != 4 || t.stride(3) != 1)
      value_error(
          "tensors must be 4-D [B, H, S, D] views with a contiguous head "
          "dimension");
    if (!bf16_bits(t) || t.device() != dev)
      value_error(std::string(name) + " must be a bfloat16 tensor on " +
                  device_name(dev));
  }
  const int64_t need[4] = {q.size(0), k.size(1), k.size(2), q.size(3)};
  if (!covers(k, need) || !covers(v, need))
    value_error("k and v must be [B, H_kv, Skv, D] for q's B and D");
}

// A tensor with the shape and device of `like` (bf16).
void check_like(const at::Tensor& t, const at::Tensor& like, const char* name) {
  if (t.defined() && (!bf16_bits(t) || !covers(t, like.sizes()) ||
                      t.device() != like.device()))
    value_error(std::string(name) + " must be a bfloat16 tensor of q's shape "
                                    "and device");
}

void check_lse(const at::Tensor& t, const at::Tensor& q) {
  if (t.defined() &&
      (t.scalar_type() != at::kFloat ||
       t.numel() < q.size(0) * q.size(1) * q.size(2) || !t.is_contiguous() ||
       t.device() != q.device()))
    value_error("lse must be a contiguous float32 tensor of B H Sq elements "
                "or more on q's device");
}

void check_id_size(const at::Tensor& t, int64_t n, const char* name) {
  if (t.defined() &&
      ((t.scalar_type() != at::kInt && t.scalar_type() != at::kUInt32) ||
       t.numel() < n || !t.is_contiguous()))
    value_error(std::string(name) + " must be a contiguous int32 tensor of " +
                std::to_string(n) + " elements or more");
}

void check_ids(const at::Tensor& t, int64_t B, int64_t S,
               const at::Device& dev, const char* name) {
  if (t.defined() &&
      ((t.scalar_type() != at::kInt && t.scalar_type() != at::kUInt32) ||
       t.numel() < B * S || !t.is_contiguous() || t.device() != dev))
    value_error(std::string(name) + " must be a contiguous int32 tensor of "
                                    "B S elements or more on " + device_name(dev));
}

// Makes the tensors' device current for a call, and gives the stream: the
// one asked for (an integer handle) or that device's current one.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream = nullptr;
  OnDevice(const at::Device& dev, PyObject* handle) {
    if (dev.is_cuda()) {
      if (dev.index() != c10::cuda::current_device()) guard.set_device(dev);
      if (handle == Py_None) {
        stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
        return;
      }
    }
    if (handle != Py_None)
      stream = reinterpret_cast<void*>(static_cast<intptr_t>(integer(handle)));
  }
};

at::Tensor empty_on(at::IntArrayRef size, at::ScalarType type,
                    const at::Device& dev) {
  return at::empty(size, at::TensorOptions().dtype(type).device(dev));
}

// Scratch memory: one per (kind, device, stream), as calls on one stream run
// in order; while the stream is being captured a new one from the graph's
// memory, as two graphs captured on one stream may run at once.  The map is
// never destroyed (its tensors would outlive CUDA at the process's end).
at::Tensor workspace(int kind, size_t bytes, const at::Device& dev,
                     void* stream) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  if (dev.is_cuda() &&
      (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &st) !=
           cudaSuccess ||
       st != cudaStreamCaptureStatusNone)) {
    (void)cudaGetLastError();
    return empty_on({static_cast<int64_t>(bytes)}, at::kByte, dev);
  }
  using Key = std::pair<std::pair<int, int>, void*>;
  static auto* kept = new std::map<Key, at::Tensor>();
  at::Tensor& t = (*kept)[Key({kind, dev.index()}, stream)];
  if (!t.defined())
    t = empty_on({static_cast<int64_t>(bytes)}, at::kByte, dev);
  return t;
}

// ---------------------------------------------------------------- functions

// build_mask_info(struct address, flags, window, q_seg, kv_seg, B, Sq, Skv,
// block_q, block_kv, device index or None, dense_bits, stream) -> buffer, or
// None where the sizes are refused
PyObject* py_build_mask_info(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 13);
    auto* info = reinterpret_cast<bsm_mask_info*>(
        static_cast<intptr_t>(integer(a[0])));
    const at::Tensor qs = tensor_or_none(a[3], "q_segment_ids");
    const at::Tensor ks = tensor_or_none(a[4], "kv_segment_ids");
    const at::Tensor bits = tensor_or_none(a[11], "dense_bits");
    bsm_mask_spec spec = {};
    spec.flags = static_cast<uint32_t>(integer(a[1]));
    spec.window = int32(a[2]);
    if (bits.defined()) {
      if (bits.dim() != 2 || bits.stride(1) != 1 || bits.element_size() != 4)
        value_error(
            "dense_bits must be a [Sq, W] 32-bit tensor with contiguous rows");
      spec.dense_bits = data<const uint32_t>(bits);
      spec.dense_row_words = bits.stride(0);
    }
    int32_t s[5];  // B, Sq, Skv, block_q, block_kv
    for (int i = 0; i < 5; ++i) s[i] = int32(a[5 + i]);
    const size_t bytes =
        f_mask_info_bytes(&spec, s[0], s[1], s[2], s[3], s[4]);
    if (bytes == 0) Py_RETURN_NONE;
    // what the kernels will read
    if (spec.flags & BSM_MASK_SEGMENT) {
      check_id_size(qs, int64_t{s[0]} * s[1], "q_segment_ids");
      check_id_size(ks, int64_t{s[0]} * s[2], "kv_segment_ids");
    }
    if ((spec.flags & BSM_MASK_DENSE) && bits.defined() &&
        (bits.size(0) < s[1] || bits.size(1) < (int64_t{s[2]} + 31) / 32))
      value_error("dense_bits must have Sq rows of ceil(Skv / 32) words");
    if ((qs.defined() && !qs.device().is_cuda()) ||
        (ks.defined() && !ks.device().is_cuda()) ||
        (bits.defined() && !bits.device().is_cuda()))
      value_error("segment ids and dense_bits must be CUDA tensors");
    const at::Device dev(at::kCUDA,
                         static_cast<c10::DeviceIndex>(
                             a[10] == Py_None ? c10::cuda::current_device()
                                              : integer(a[10])));
    for (const at::Tensor* t : {&qs, &ks, &bits})
      if (t->defined() && t->device() != dev)
        value_error("segment ids and dense_bits must be on " +
                    device_name(dev));
    OnDevice on(dev, a[12]);
    at::Tensor buf =
        empty_on({static_cast<int64_t>(bytes)}, at::kByte, dev);
    check_status(f_build_mask_info(
        &spec, data<const int32_t>(qs), data<const int32_t>(ks), s[0], s[1],
        s[2], s[3], s[4], buf.mutable_data_ptr(), bytes, info, on.stream));
    return THPVariable_Wrap(std::move(buf));
  });
}

// splash_fwd(q, k, v, struct address, q_seg, kv_seg, scale, score, softcap,
// slopes, out, lse, want_lse, stream) -> (out, lse)
PyObject* py_splash_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 14);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"),
                     &v = tensor(a[2], "v");
    check_operands(q, k, v);
    const bsm_tensor qv = view(q), kv = view(k), vv = view(v);
    const at::Tensor qs = tensor_or_none(a[4], "q_segment_ids");
    const at::Tensor ks = tensor_or_none(a[5], "kv_segment_ids");
    const at::Device dev = q.device();
    check_ids(qs, q.size(0), q.size(2), dev, "q_segment_ids");
    check_ids(ks, q.size(0), k.size(2), dev, "kv_segment_ids");
    const int64_t B = q.size(0), H = q.size(1), Sq = q.size(2), D = q.size(3);
    const bsm_score_mod mod =
        score_mod(number(a[8]), tensor_or_none(a[9], "alibi_slopes"), H, dev);
    OnDevice on(dev, a[13]);
    at::Tensor out = tensor_or_none(a[10], "out");
    check_like(out, q, "out");
    if (!out.defined()) out = empty_on({B, H, Sq, D}, at::kBFloat16, dev);
    const bool want_lse = truth(a[12]);
    at::Tensor lse = want_lse ? tensor_or_none(a[11], "lse") : at::Tensor();
    check_lse(lse, q);
    if (want_lse && !lse.defined())
      lse = empty_on({B, H, Sq}, at::kFloat, dev);
    const bsm_tensor ov = view(out);
    const at::Tensor ws = workspace(0, fwd_workspace_bytes, dev, on.stream);
    check_status(f_splash_fwd_mod(
        qv.data, kv.data, vv.data, qv.strides, kv.strides, vv.strides,
        ov.strides, static_cast<int32_t>(B), static_cast<int32_t>(H),
        static_cast<int32_t>(k.size(1)), static_cast<int32_t>(Sq),
        static_cast<int32_t>(k.size(2)), static_cast<int32_t>(D),
        reinterpret_cast<const bsm_mask_info*>(
            static_cast<intptr_t>(integer(a[3]))),
        data<const int32_t>(qs), data<const int32_t>(ks),
        static_cast<float>(number(a[6])), int32(a[7]), &mod, ov.data,
        data<float>(lse), data<void>(ws), bytes_of(ws), on.stream));
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
    if (lse.defined()) {
      PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(lse)));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 1, Py_None);
    }
    return r;
  });
}

// splash_bwd(q, k, v, out, lse, dout, struct address, q_seg, kv_seg, scale,
// score, softcap, slopes, stream) -> (dq, dk, dv)
PyObject* py_splash_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 14);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"),
                     &v = tensor(a[2], "v"), &dout = tensor(a[5], "dout");
    const at::Tensor out = tensor_or_none(a[3], "out");
    const at::Tensor lse = tensor_or_none(a[4], "lse");
    check_operands(q, k, v);
    check_like(out, q, "out");
    check_like(dout, q, "dout");
    check_lse(lse, q);
    const bsm_tensor qv = view(q), kv = view(k), vv = view(v), dv = view(dout);
    bsm_tensor ov = {};
    if (out.defined()) ov = view(out);
    const at::Tensor qs = tensor_or_none(a[7], "q_segment_ids");
    const at::Tensor ks = tensor_or_none(a[8], "kv_segment_ids");
    const at::Device dev = q.device();
    check_ids(qs, q.size(0), q.size(2), dev, "q_segment_ids");
    check_ids(ks, q.size(0), k.size(2), dev, "kv_segment_ids");
    const int32_t score = int32(a[10]);
    const int32_t B = static_cast<int32_t>(q.size(0));
    const int32_t H = static_cast<int32_t>(q.size(1));
    const int32_t Sq = static_cast<int32_t>(q.size(2));
    const bsm_score_mod mod =
        score_mod(number(a[11]), tensor_or_none(a[12], "alibi_slopes"), H, dev);
    OnDevice on(dev, a[13]);
    at::Tensor g[3] = {at::empty_like(q), at::empty_like(k), at::empty_like(v)};
    const bsm_tensor gv[3] = {view(g[0]), view(g[1]), view(g[2])};
    const bool modified = mod.softcap != 0.f || mod.alibi_slopes != nullptr;
    const size_t need =
        modified ? f_bwd_mod_workspace_bytes(
                       B, H, static_cast<int32_t>(k.size(1)), Sq,
                       static_cast<int32_t>(k.size(2)),
                       static_cast<int32_t>(q.size(3)))
                 : f_bwd_workspace_bytes(B, H, Sq, score);
    at::Tensor ws;
    if (need > 0) ws = empty_on({static_cast<int64_t>(need)}, at::kByte, dev);
    check_status(f_splash_bwd_mod(
        &qv, &kv, &vv, out.defined() ? &ov : nullptr, data<const float>(lse),
        &dv, B, H, static_cast<int32_t>(k.size(1)), Sq,
        static_cast<int32_t>(k.size(2)), static_cast<int32_t>(q.size(3)),
        reinterpret_cast<const bsm_mask_info*>(
            static_cast<intptr_t>(integer(a[6]))),
        data<const int32_t>(qs), data<const int32_t>(ks),
        static_cast<float>(number(a[9])), score, &mod, &gv[0], &gv[1], &gv[2],
        data<void>(ws), bytes_of(ws), on.stream));
    PyObject* r = PyTuple_New(3);
    for (int i = 0; i < 3; ++i)
      PyTuple_SET_ITEM(r, i, THPVariable_Wrap(std::move(g[i])));
    return r;
  });
}

// check_cache(k_pages, v_pages, k_scale, v_scale)
PyObject* py_check_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 4);
    const at::Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages"),
                     &ks = tensor(a[2], "k_scale"),
                     &vs = tensor(a[3], "v_scale");
    for (const at::Tensor* t : {&k, &v})
      if (t->scalar_type() != at::kFloat8_e4m3fn || t->dim() != 4 ||
          t->sizes() != k.sizes() || !t->is_contiguous() ||
          t->device() != k.device())
        value_error(
            "k_pages and v_pages must be contiguous float8_e4m3fn tensors of "
            "one shape [num_pages, H_kv, page_size, D] on one device");
    for (const at::Tensor* t : {&ks, &vs})
      if (t->scalar_type() != at::kFloat || t->dim() != 2 ||
          t->size(0) != k.size(0) || t->size(1) != k.size(1) ||
          !t->is_contiguous() || t->device() != k.device())
        value_error(
            "k_scale and v_scale must be contiguous float32 tensors "
            "[num_pages, H_kv] beside the pages");
    Py_RETURN_NONE;
  });
}

// The cache's four tensors, which KVCache has checked.
bsm_kv_cache cache_of(PyObject* const* a) {
  const at::Tensor& k = tensor(a[0], "k_pages");
  bsm_kv_cache c;
  c.k = data<void>(k);
  c.v = data<void>(tensor(a[1], "v_pages"));
  c.k_scale = data<float>(tensor(a[2], "k_scale"));
  c.v_scale = data<float>(tensor(a[3], "v_scale"));
  c.num_pages = static_cast<int32_t>(k.size(0));
  c.H_kv = static_cast<int32_t>(k.size(1));
  c.page_size = static_cast<int32_t>(k.size(2));
  c.D = static_cast<int32_t>(k.size(3));
  return c;
}

void check_table(const at::Device& dev, const at::Tensor& table, int64_t B,
                 const at::Tensor& lens, const at::Tensor& n_new) {
  if (table.scalar_type() != at::kInt || table.dim() != 2 ||
      table.size(0) != B || table.device() != dev ||
      (table.size(1) > 1 && table.stride(1) != 1))
    value_error(
        "page_table must be an int32 tensor [B, max_pages] with contiguous "
        "rows, beside the cache");
  const std::pair<const char*, const at::Tensor&> ints[2] = {{"lens", lens},
                                                             {"n_new", n_new}};
  for (const auto& [name, t] : ints)
    if (t.defined() &&
        (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != B ||
         !t.is_contiguous() || t.device() != dev))
      value_error(std::string(name) +
                  " must be a contiguous int32 tensor [B] beside the cache");
}

bsm_tensor token_view(const at::Tensor& t, int64_t B, int64_t heads, int64_t T,
                      int64_t D, const at::Device& dev, const char* name) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 4 || t.size(0) != B ||
      t.size(1) != heads || t.size(2) != T || t.size(3) != D ||
      t.device() != dev || t.stride(3) != 1)
    value_error(std::string(name) + " must be a bfloat16 tensor [" +
                std::to_string(B) + ", " + std::to_string(heads) + ", " +
                std::to_string(T) + ", " + std::to_string(D) +
                "] with a contiguous head dimension, beside the cache");
  return view(t);
}

// kv_append(k_pages, v_pages, k_scale, v_scale, page_table, lens, k_new,
// v_new, n_new, stream)
PyObject* py_kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 10);
    const bsm_kv_cache c = cache_of(a);
    const at::Device dev = tensor(a[0], "k_pages").device();
    const at::Tensor &table = tensor(a[4], "page_table"),
                     &lens = tensor(a[5], "lens"),
                     &k_new = tensor(a[6], "k_new"),
                     &v_new = tensor(a[7], "v_new");
    const at::Tensor n_new = tensor_or_none(a[8], "n_new");
    if (k_new.dim() != 4) value_error("k_new must be [B, H_kv, T, D]");
    const int64_t B = k_new.size(0), T = k_new.size(2);
    check_table(dev, table, B, lens, n_new);
    const bsm_tensor kt = token_view(k_new, B, c.H_kv, T, c.D, dev, "k_new");
    const bsm_tensor vt = token_view(v_new, B, c.H_kv, T, c.D, dev, "v_new");
    if (!dev.is_cuda()) value_error("the cache must be on a CUDA device");
    OnDevice on(dev, a[9]);
    check_status(f_kv_append(&c, data<const int32_t>(table), table.stride(0),
                             static_cast<int32_t>(table.size(1)),
                             data<const int32_t>(lens),
                             data<const int32_t>(n_new), &kt, &vt,
                             static_cast<int32_t>(B), static_cast<int32_t>(T),
                             on.stream));
    Py_RETURN_NONE;
  });
}

// paged_attention(k_pages, v_pages, k_scale, v_scale, page_table, lens, q,
// scale or None, window, softcap, slopes, out, lse, want_lse, stream) ->
// (out, lse)
PyObject* py_paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 15);
    const bsm_kv_cache c = cache_of(a);
    const at::Device dev = tensor(a[0], "k_pages").device();
    const at::Tensor &table = tensor(a[4], "page_table"),
                     &lens = tensor(a[5], "lens"), &q = tensor(a[6], "q");
    if (q.dim() != 4) value_error("q must be [B, H, T, D]");
    const int64_t B = q.size(0), H = q.size(1), T = q.size(2);
    check_table(dev, table, B, lens, at::Tensor());
    const bsm_tensor qt = token_view(q, B, H, T, c.D, dev, "q");
    OnDevice on(dev, a[14]);
    at::Tensor out = tensor_or_none(a[11], "out");
    if (!out.defined()) out = empty_on({B, H, T, c.D}, at::kBFloat16, dev);
    const bsm_tensor ot = token_view(out, B, H, T, c.D, dev, "out");
    const bool want_lse = truth(a[13]);
    at::Tensor lse = want_lse ? tensor_or_none(a[12], "lse") : at::Tensor();
    if (want_lse && !lse.defined()) lse = empty_on({B, H, T}, at::kFloat, dev);
    if (lse.defined() &&
        (lse.scalar_type() != at::kFloat || lse.dim() != 3 ||
         lse.size(0) != B || lse.size(1) != H || lse.size(2) != T ||
         lse.device() != dev || !lse.is_contiguous()))
      value_error(
          "lse must be a contiguous float32 tensor [B, H, T] beside the "
          "cache");
    const bsm_score_mod mod = score_mod(
        number(a[9]), tensor_or_none(a[10], "alibi_slopes"), H, dev);
    if (!dev.is_cuda()) value_error("the cache must be on a CUDA device");
    const float scale = static_cast<float>(
        a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.D))
                        : number(a[7]));
    const at::Tensor ws = workspace(1, paged_workspace_bytes, dev, on.stream);
    check_status(f_paged_attention(
        &qt, &c, data<const int32_t>(table), table.stride(0),
        static_cast<int32_t>(table.size(1)), data<const int32_t>(lens),
        static_cast<int32_t>(B), static_cast<int32_t>(H),
        static_cast<int32_t>(T), scale, int32(a[8]), &mod, &ot,
        data<float>(lse), data<void>(ws), bytes_of(ws), on.stream));
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
    if (lse.defined()) {
      PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(lse)));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 1, Py_None);
    }
    return r;
  });
}

// bind(status callable, {name: address})
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    expect(n, 2);
    auto at_name = [&](const char* name) {
      PyObject* o = PyDict_GetItemString(a[1], name);  // borrowed
      if (o == nullptr) {
        PyErr_Format(PyExc_KeyError, "%s", name);
        throw Raised{};
      }
      return reinterpret_cast<void*>(static_cast<intptr_t>(integer(o)));
    };
    auto set = [&](auto& f, const char* name) {
      f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(at_name(name));
    };
    set(f_mask_info_bytes, "bsm_mask_info_bytes");
    set(f_build_mask_info, "bsm_build_mask_info");
    set(f_splash_fwd_mod, "bsm_splash_fwd_mod");
    set(f_splash_bwd_mod, "bsm_splash_bwd_mod");
    set(f_bwd_workspace_bytes, "bsm_splash_bwd_workspace_bytes");
    set(f_bwd_mod_workspace_bytes, "bsm_splash_bwd_mod_workspace_bytes");
    set(f_kv_append, "bsm_kv_append");
    set(f_paged_attention, "bsm_paged_attention");
    decltype(&bsm_splash_fwd_workspace_bytes) f0;
    decltype(&bsm_paged_attention_workspace_bytes) f1;
    set(f0, "bsm_splash_fwd_workspace_bytes");
    set(f1, "bsm_paged_attention_workspace_bytes");
    fwd_workspace_bytes = f0();
    paged_workspace_bytes = f1();
    Py_INCREF(a[0]);
    Py_XSETREF(on_status, a[0]);
    Py_RETURN_NONE;
  });
}

#define FAST(name) \
  {#name, reinterpret_cast<PyCFunction>(py_##name), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),       FAST(build_mask_info),
                         FAST(splash_fwd), FAST(splash_bwd),
                         FAST(kv_append),  FAST(paged_attention),
                         FAST(check_cache),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bsm_torch", nullptr, -1,
                      methods};

}  // namespace

PyMODINIT_FUNC PyInit__bsm_torch(void) { return PyModule_Create(&module); }
