// qsa_torch.cpp -- the layer operators' torch-facing calls (layer.py) as a CPython extension:
// checks of the tensors, allocation of missing outputs and workspaces, and the call of the C
// entry point (include/qsa_layer.h) on torch's current stream.  A call of one small kernel
// costs its host time: through ctypes these calls took 13 us (four tensors) to 27 us (eleven)
// on a 2.7 GHz Xeon, most of it in reading the tensors' fields one Python call at a time.
// Nothing is computed here and nothing is kept between calls.
//
// Every function takes its arguments by position, as layer.py passes them, and returns its
// result, or the status of the C call as an int when that is not QSA_OK.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/CUDAContext.h>

#include <cmath>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "qsa_layer.h"

namespace {

using at::ScalarType;
using at::Tensor;
constexpr auto kBF16 = ScalarType::BFloat16;
constexpr auto kF32 = ScalarType::Float;
constexpr auto kI32 = ScalarType::Int;
constexpr auto kI8 = ScalarType::Char;
constexpr auto kU8 = ScalarType::Byte;
constexpr auto kE4M3 = ScalarType::Float8_e4m3fn;

struct Raised {};  // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised{};
}

const char* dtype_name(ScalarType t) {
  switch (t) {
    case kBF16: return "torch.bfloat16";
    case kF32: return "torch.float32";
    case kI32: return "torch.int32";
    case kI8: return "torch.int8";
    case kU8: return "torch.uint8";
    case kE4M3: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    throw Raised{};
  }
  return THPVariable_Unpack(o);
}
const Tensor* maybe(const char* name, PyObject* o) { return o == Py_None ? nullptr : &tensor(name, o); }

int64_t whole(const char* name, PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int32_t whole32(const char* name, PyObject* o) {
  const int64_t v = whole(name, o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is beyond 32 bits");
  return int32_t(v);
}
int32_t size32(const char* name, int64_t v) {
  if (v > INT32_MAX) refuse(std::string(name) + " is beyond 32 bits");
  return int32_t(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return float(v);
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// type and device, contiguous in the last dimension, and (a non-empty `shape`) sizes
void check(const char* name, const Tensor& t, ScalarType dtype, at::Device device,
           std::initializer_list<int64_t> shape, bool any_shape = false) {
  if (t.device() != device)
    refuse(std::string(name) + " must live on " + device.str() + ", got " + t.device().str());
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + " must be " + dtype_name(dtype) + ", got " + dtype_name(t.scalar_type()));
  if (!any_shape && !(t.sizes() == at::IntArrayRef(shape)))
    refuse(std::string(name) + " must be " + shape_text(at::IntArrayRef(shape)) + ", got " + shape_text(t.sizes()));
  if (t.dim() > 0 && t.size(-1) > 1 && t.stride(-1) != 1)
    refuse(std::string(name) + " must be contiguous in its last dimension");
}
void check_dims(const char* name, const Tensor& t, ScalarType dtype, at::Device device, int64_t dims) {
  if (t.dim() != dims) refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions");
  check(name, t, dtype, device, {}, true);
}

at::Device cuda_device(const char* what, const Tensor& t) {
  if (!t.is_cuda()) refuse(std::string(what) + " runs on CUDA tensors only");
  return t.device();
}

uint32_t* err_ptr(PyObject* o, at::Device device) {
  const Tensor* t = maybe("err_word", o);
  if (t == nullptr) return nullptr;
  if (t->device() != device || t->element_size() != 4 || t->numel() < 1)
    refuse("err_word must be a 4-byte integer tensor on " + device.str());
  return static_cast<uint32_t*>(t->data_ptr());
}

// The stride of a dimension, 0 where it is never taken (a tensor's views may give it any value).
int64_t pitch(const Tensor& t, int d) { return t.size(d) > 1 ? t.stride(d) : 0; }
int64_t pitch(const Tensor* t, int d) { return t == nullptr ? 0 : pitch(*t, d); }

void* ptr(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
const int32_t* ptr32(const Tensor* t) { return static_cast<const int32_t*>(ptr(t)); }

Tensor empty(std::initializer_list<int64_t> shape, ScalarType dtype, at::Device device) {
  return at::detail::empty_cuda(at::IntArrayRef(shape), dtype, device, std::nullopt);
}

void* stream_of(at::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

PyObject* status(qsa_status_t st) { return PyLong_FromLong(long(st)); }

// Python errors and C++ exceptions both leave as Python errors.
template <class F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, F&& body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", name, want, n);
    return nullptr;
  }
  try {
    return body();
  } catch (const Raised&) {
    return nullptr;
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// q, positions, inv_freq, k, v, q_weight, k_weight, eps, weight_offset, sections, interleaved,
// rope_scale, q_out, k_cache, v_cache, slots, k_scale, v_scale, err_word -> (q_out, keys | None)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope", n, 19, [&]() -> PyObject* {
    const Tensor& q = tensor("q", a[0]);
    const at::Device device = cuda_device("qk_norm_rope", q);
    check_dims("q", q, kBF16, device, 3);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    const Tensor& inv_freq = tensor("inv_freq", a[2]);
    check_dims("inv_freq", inv_freq, kF32, device, 1);
    const int64_t rot = 2 * inv_freq.size(0);
    const Tensor& pos = tensor("positions", a[1]);
    const int64_t axes = pos.dim() == 1 ? 1 : pos.size(0);
    if (pos.dim() == 1) check("positions", pos, kI32, device, {T});
    else check("positions", pos, kI32, device, {axes, T});
    int32_t sections[QSA_MAX_ROPE_AXES] = {0};
    const bool has_sections = a[9] != Py_None;
    if (!has_sections && axes != 1) refuse("positions of several axes need sections");
    if (has_sections) {
      PyObject* seq = PySequence_Fast(a[9], "sections must be a sequence of integers");
      if (seq == nullptr) throw Raised{};
      const Py_ssize_t m = PySequence_Fast_GET_SIZE(seq);
      bool bad = m != axes;
      for (Py_ssize_t i = 0; i < m && i < QSA_MAX_ROPE_AXES && !bad; ++i) {
        const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
        if ((v == -1 && PyErr_Occurred()) || v < INT32_MIN || v > INT32_MAX) {
          Py_DECREF(seq);
          if (!PyErr_Occurred()) refuse("sections are beyond 32 bits");
          throw Raised{};
        }
        sections[i] = int32_t(v);
      }
      Py_DECREF(seq);
      if (bad) refuse("one section per axis of positions");
    }
    const Tensor *k = maybe("k", a[3]), *v = maybe("v", a[4]), *k_cache = maybe("k_cache", a[13]),
                 *v_cache = maybe("v_cache", a[14]), *slots = maybe("slots", a[15]);
    int64_t Hkv = 0;
    if (k != nullptr) {
      if (k->dim() != 3) refuse("k must be [T, Hkv, D]");
      Hkv = k->size(1);
      check("k", *k, kBF16, device, {T, Hkv, D});
    } else if (v != nullptr || k_cache != nullptr || v_cache != nullptr) {
      refuse("v, k_cache and v_cache need k");
    }
    if (v != nullptr) check("v", *v, kBF16, device, {T, Hkv, D});
    const Tensor *qw = maybe("q_weight", a[5]), *kw = maybe("k_weight", a[6]);
    if (qw != nullptr) check("q_weight", *qw, kBF16, device, {D});
    if (kw != nullptr) check("k_weight", *kw, kBF16, device, {D});
    const bool fp8 = k_cache != nullptr && k_cache->scalar_type() == kE4M3;
    int64_t rows = T;
    if (k_cache != nullptr) {
      if (k_cache->dim() != 3) refuse("k_cache must be [S, Hkv, D]");
      rows = k_cache->size(0);
      check("k_cache", *k_cache, fp8 ? kE4M3 : kBF16, device, {rows, Hkv, D});
    }
    if ((v == nullptr) != (v_cache == nullptr)) refuse("v and v_cache come together");
    if (v_cache != nullptr) {
      if (k_cache == nullptr) refuse("v_cache needs k_cache");
      check("v_cache", *v_cache, fp8 ? kE4M3 : kBF16, device, {rows, Hkv, D});
    }
    if (slots != nullptr) {
      if (k_cache == nullptr) refuse("slots need k_cache");
      check("slots", *slots, kI32, device, {T});
    }
    uint32_t* err = err_ptr(a[18], device);
    const int interleaved = PyObject_IsTrue(a[10]);
    if (interleaved < 0) throw Raised{};
    const float eps = real(a[7]), offset = real(a[8]), rope_scale = real(a[11]), ks = real(a[16]), vs = real(a[17]);
    const c10::cuda::OptionalCUDAGuard guard(device);
    const Tensor* given = maybe("q_out", a[12]);
    if (given != nullptr) check("q_out", *given, kBF16, device, {T, Hq, D});
    const Tensor q_out = given != nullptr ? *given : empty({T, Hq, D}, kBF16, device);
    Tensor k_out;
    if (k != nullptr && k_cache == nullptr) k_out = empty({T, Hkv, D}, kBF16, device);
    const Tensor* k_dst = k_cache != nullptr ? k_cache : k != nullptr ? &k_out : nullptr;
    const qsa_status_t st = qsa_qk_norm_rope(
        q.data_ptr(), pitch(q, 0), pitch(q, 1), ptr(k), pitch(k, 0), pitch(k, 1), ptr(v), pitch(v, 0), pitch(v, 1),
        ptr(qw), ptr(kw), offset, eps, ptr32(&pos), axes > 1 ? pitch(pos, 0) : 0,
        static_cast<const float*>(inv_freq.data_ptr()), size32("inv_freq", rot), interleaved,
        has_sections ? sections : nullptr, size32("positions", axes), rope_scale, size32("T", T), size32("Hq", Hq),
        size32("Hkv", Hkv), size32("D", D), q_out.data_ptr(), pitch(q_out, 0), pitch(q_out, 1), ptr(k_dst),
        pitch(k_dst, 0), pitch(k_dst, 1), ptr(v_cache), pitch(v_cache, 0), pitch(v_cache, 1), ptr32(slots), rows,
        fp8 ? 1 : 0, ks, vs, err, stream_of(device));
    if (st != QSA_OK) return status(st);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) throw Raised{};
    if (given != nullptr) {
      Py_INCREF(a[12]);
      PyTuple_SET_ITEM(r, 0, a[12]);
    } else {
      PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(q_out));
    }
    if (k_out.defined()) {
      PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(k_out));
    } else {
      Py_INCREF(Py_None);
      PyTuple_SET_ITEM(r, 1, Py_None);
    }
    return r;
  });
}

// keys, blocks, codes, scales, block, err_word -> 0
PyObject* pack_index_keys(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("pack_index_keys", n, 6, [&]() -> PyObject* {
    const Tensor& keys = tensor("keys", a[0]);
    const at::Device device = cuda_device("pack_index_keys", keys);
    check_dims("keys", keys, kBF16, device, 2);
    const int64_t S = keys.size(0), Di = keys.size(1);
    const int32_t block = whole32("block", a[4]);
    if (block < 1) refuse("block must be positive");
    const Tensor &blocks = tensor("blocks", a[1]), &codes = tensor("codes", a[2]), &scales = tensor("scales", a[3]);
    check_dims("blocks", blocks, kI32, device, 1);
    check("codes", codes, kI8, device, {S / block, Di});
    check("scales", scales, kF32, device, {S / block});
    uint32_t* err = err_ptr(a[5], device);
    const c10::cuda::OptionalCUDAGuard guard(device);
    return status(qsa_pack_index_keys(keys.data_ptr(), pitch(keys, 0), ptr32(&blocks), size32("blocks", blocks.size(0)),
                                      block, size32("Di", Di), S, static_cast<int8_t*>(codes.data_ptr()),
                                      pitch(codes, 0), static_cast<float*>(scales.data_ptr()), err, stream_of(device)));
  });
}

// q, weight, codes, scales, page_table, seq_lens, top_blocks, page_size, block, cu_q, sink_blocks,
// local_blocks, slot_idx, width, workspace, err_word -> (slot_idx, width)
PyObject* select_slots(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("select_slots", n, 16, [&]() -> PyObject* {
    const Tensor& q = tensor("q", a[0]);
    const at::Device device = cuda_device("select_slots", q);
    check_dims("q", q, kBF16, device, 3);
    const int64_t Tq = q.size(0), Hi = q.size(1), Di = q.size(2);
    const Tensor &weight = tensor("weight", a[1]), &codes = tensor("codes", a[2]), &scales = tensor("scales", a[3]),
                 &table = tensor("page_table", a[4]), &lens = tensor("seq_lens", a[5]);
    check("weight", weight, kF32, device, {Tq, Hi});
    check_dims("codes", codes, kI8, device, 2);
    if (codes.size(1) != Di) refuse("codes must be [blocks, Di]");
    check("scales", scales, kF32, device, {codes.size(0)});
    if (table.dim() != 2) refuse("page_table must be [B, P]");
    check("page_table", table, kI32, device, {}, true);
    const int64_t B = table.size(0), P = table.size(1);
    check("seq_lens", lens, kI32, device, {B});
    const Tensor* cu = maybe("cu_q", a[9]);
    if (cu != nullptr) check("cu_q", *cu, kI32, device, {B + 1});
    uint32_t* err = err_ptr(a[15], device);
    const int32_t top = whole32("top_blocks", a[6]), page = whole32("page_size", a[7]), block = whole32("block", a[8]),
                  sink = whole32("sink_blocks", a[10]), local = whole32("local_blocks", a[11]);
    if (block < 1 || page < 1 || page % block != 0) refuse("page_size must be a positive multiple of block");
    const int32_t tq = size32("Tq", Tq), b = size32("B", B), p = size32("P", P), hi = size32("Hi", Hi),
                  di = size32("Di", Di);
    size_t need = qsa_select_slots_workspace_bytes(tq, b, p, page, hi, di, block);
    if (need == SIZE_MAX) need = 0;  // sizes that the call below refuses
    const int64_t W = int64_t(top < 0 ? 0 : top) * block + block - 1;
    if (W > int64_t(QSA_MAX_TOP_BLOCKS) * 17) refuse("top_blocks is too large");
    const c10::cuda::OptionalCUDAGuard guard(device);
    const Tensor *given_idx = maybe("slot_idx", a[12]), *given_width = maybe("width", a[13]),
                 *given_work = maybe("workspace", a[14]);
    if (given_idx != nullptr) check("slot_idx", *given_idx, kI32, device, {Tq, W});
    if (given_width != nullptr) check("width", *given_width, kI32, device, {Tq});
    if (given_work != nullptr) check_dims("workspace", *given_work, kU8, device, 1);
    const Tensor idx = given_idx != nullptr ? *given_idx : empty({Tq, W}, kI32, device);
    const Tensor width = given_width != nullptr ? *given_width : empty({Tq}, kI32, device);
    const Tensor work = given_work != nullptr ? *given_work : empty({int64_t(need)}, kU8, device);
    const qsa_status_t st = qsa_select_slots(
        q.data_ptr(), pitch(q, 0), pitch(q, 1), static_cast<const float*>(weight.data_ptr()), pitch(weight, 0),
        static_cast<const int8_t*>(codes.data_ptr()), pitch(codes, 0), static_cast<const float*>(scales.data_ptr()),
        ptr32(&table), pitch(table, 0), ptr32(&lens), ptr32(cu), tq, b, p, codes.size(0) / (page / block), page, hi, di,
        block, top, sink, local, static_cast<int32_t*>(idx.data_ptr()), pitch(idx, 0),
        static_cast<int32_t*>(width.data_ptr()), work.data_ptr(), size_t(work.numel()), err, stream_of(device));
    if (st != QSA_OK) return status(st);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) throw Raised{};
    const auto put = [&](int i, PyObject* given, const Tensor& t) {
      if (given != Py_None) Py_INCREF(given);
      PyTuple_SET_ITEM(r, i, given != Py_None ? given : THPVariable_Wrap(t));
    };
    put(0, a[12], idx);
    put(1, a[13], width);
    return r;
  });
}

// q, k_cache, v_cache, page_table, seq_lens, page_size, scale, k_scale, v_scale, out, lse, blocks,
// workspace, err_word -> out
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_decode", n, 14, [&]() -> PyObject* {
    const Tensor& q = tensor("q", a[0]);
    const at::Device device = cuda_device("paged_decode", q);
    check_dims("q", q, kBF16, device, 3);
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const Tensor &k = tensor("k_cache", a[1]), &v = tensor("v_cache", a[2]), &table = tensor("page_table", a[3]),
                 &lens = tensor("seq_lens", a[4]);
    if (k.dim() != 3) refuse("k_cache must be [S, Hkv, D]");
    const bool fp8 = k.scalar_type() == kE4M3;
    const int64_t S = k.size(0), Hkv = k.size(1);
    check("k_cache", k, fp8 ? kE4M3 : kBF16, device, {S, Hkv, D});
    check("v_cache", v, fp8 ? kE4M3 : kBF16, device, {S, Hkv, D});
    if (table.dim() != 2 || table.size(0) != B) refuse("page_table must be [B, P]");
    check("page_table", table, kI32, device, {}, true);
    const int64_t P = table.size(1);
    check("seq_lens", lens, kI32, device, {B});
    uint32_t* err = err_ptr(a[13], device);
    const Tensor* lse = maybe("lse", a[10]);
    if (lse != nullptr) {
      check("lse", *lse, kF32, device, {B, Hq});
      if (!lse->is_contiguous()) refuse("lse must be contiguous");
    }
    const int32_t page = whole32("page_size", a[5]), request = whole32("blocks", a[11]);
    if (page < 1) refuse("page_size must be positive");
    const float scale = a[6] == Py_None ? float(1.0 / std::sqrt(double(D))) : real(a[6]);
    const float ks = real(a[7]), vs = real(a[8]);
    const c10::cuda::OptionalCUDAGuard guard(device);
    const int32_t b = size32("B", B), hq = size32("Hq", Hq), hkv = size32("Hkv", Hkv), d = size32("D", D),
                  p = size32("P", P);
    size_t need = 0;
    const int32_t blocks = qsa_paged_decode_plan(
        b, hq, hkv, d, p, page, fp8 ? 1 : 0, at::cuda::getCurrentDeviceProperties()->multiProcessorCount, request, &need);
    if (blocks < 0) return PyLong_FromLong(-blocks);
    const Tensor *given = maybe("out", a[9]), *given_work = maybe("workspace", a[12]);
    if (given != nullptr) check("out", *given, kBF16, device, {B, Hq, D});
    if (given_work != nullptr) check_dims("workspace", *given_work, kU8, device, 1);
    const Tensor out = given != nullptr ? *given : empty({B, Hq, D}, kBF16, device);
    const Tensor work = given_work != nullptr ? *given_work : need > 0 ? empty({int64_t(need)}, kU8, device) : Tensor();
    const qsa_status_t st = qsa_paged_decode(
        q.data_ptr(), pitch(q, 0), pitch(q, 1), k.data_ptr(), pitch(k, 0), pitch(k, 1), v.data_ptr(), pitch(v, 0),
        pitch(v, 1), ptr32(&table), pitch(table, 0), ptr32(&lens), b, hq, hkv, d, p, S / page, page, scale, fp8 ? 1 : 0,
        ks, vs, out.data_ptr(), pitch(out, 0), pitch(out, 1), static_cast<float*>(ptr(lse)), blocks,
        work.defined() ? work.data_ptr() : nullptr, work.defined() ? size_t(work.numel()) : 0, err, stream_of(device));
    if (st != QSA_OK) return status(st);
    if (given != nullptr) {
      Py_INCREF(a[9]);
      return a[9];
    }
    return THPVariable_Wrap(out);
  });
}

#define QSA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {QSA_METHOD(qk_norm_rope), QSA_METHOD(pack_index_keys), QSA_METHOD(select_slots),
                          QSA_METHOD(paged_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_layer_ext", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer_ext() { return PyModule_Create(&kModule); }
