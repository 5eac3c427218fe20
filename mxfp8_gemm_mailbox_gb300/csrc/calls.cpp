// The calls of a decode step that cost the host as much as the GPU, as a
// Python module over the C ABI: checks of dtypes, shapes, devices and strides,
// the output on the call's stream, the call without the interpreter's lock.
// (Made of Python attributes and ctypes, the same took 5 to 8 us of a 2 to 9 us
// kernel's call on a Grace core.)
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/ScalarTypeToTypeMeta.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <string>
#include <vector>

#include "mxfp8_mailbox.h"

namespace {

constexpr int64_t kRope = MXFP8_LATENT_ROPE;

[[noreturn]] void refuse(PyObject* kind, const std::string& text) {
  PyErr_SetString(kind, text.c_str());
  throw python_error();
}
std::string text_of(at::IntArrayRef shape) {
  std::string s = "[";
  for (size_t i = 0; i < shape.size(); ++i)
    s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + "]";
}
const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    default: return c10::toString(t);
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    refuse(PyExc_TypeError,
           std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
int gpu_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

// t is dtype, shape, contiguous and on the device.
void expect(const at::Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape,
            int device) {
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must be " + name_of(dtype) + ", got " +
                                name_of(t.scalar_type()));
  if (t.sizes() != shape)
    refuse(PyExc_ValueError,
           std::string(name) + " must be " + text_of(shape) + ", got " + text_of(t.sizes()));
  if (device < 0 || gpu_of(t) != device || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor on device " +
                                 std::to_string(std::max(device, 0)));
}
int on_current_device(const at::Tensor& t, const char* name) {
  const int device = gpu_of(t);
  if (device < 0)
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor");
  const int current = c10::cuda::current_device();
  if (device != current)
    refuse(PyExc_ValueError, std::string(name) + " is on device " + std::to_string(device) +
                                 ", the current device is " + std::to_string(current));
  return device;
}
// A matrix of one-byte codes [rows >= min_rows][cols]; returns rows.
int64_t codes(const at::Tensor& t, const char* name, int64_t cols, int64_t min_rows) {
  if (t.element_size() != 1)
    refuse(PyExc_TypeError, std::string(name) + " must hold one-byte codes (uint8 / float8), got " +
                                name_of(t.scalar_type()));
  if (t.dim() != 2 || t.size(1) != cols || t.size(0) < min_rows)
    refuse(PyExc_ValueError, std::string(name) + " must be [rows >= " + std::to_string(min_rows) +
                                 "][" + std::to_string(cols) + "], got " + text_of(t.sizes()));
  if (!t.is_cuda() || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor");
  return t.size(0);
}
// A matrix of two-byte values [rows >= min_rows][cols].
void halves(const at::Tensor& t, const char* name, int64_t cols, int64_t min_rows) {
  if (t.element_size() != 2)
    refuse(PyExc_TypeError, std::string(name) +
                                " must hold two-byte values (bfloat16 / int16), got " +
                                name_of(t.scalar_type()));
  if (t.dim() != 2 || t.size(1) != cols || t.size(0) < min_rows)
    refuse(PyExc_ValueError, std::string(name) + " must be [rows >= " + std::to_string(min_rows) +
                                 "][" + std::to_string(cols) + "], got " + text_of(t.sizes()));
  if (!t.is_cuda() || !t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be a contiguous CUDA tensor");
}
// New memory of the current stream, as torch's own outputs have it, without its
// dispatcher (1 us of a call on a Grace core).  The device is the current one.
c10::Storage new_storage(int64_t bytes) {
  c10::Allocator* const allocator = c10::cuda::CUDACachingAllocator::get();
  const auto size = static_cast<size_t>(bytes);
  return c10::Storage(c10::Storage::use_byte_size_t(), size, allocator->allocate(size), allocator,
                      /*resizable=*/true);
}
// A contiguous tensor at a place of a storage (in elements).
at::Tensor tensor_of(c10::Storage storage, int64_t at, at::IntArrayRef shape,
                     at::ScalarType dtype) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
      c10::scalarTypeToTypeMeta(dtype));
  c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  impl->set_sizes_contiguous(shape);
  impl->set_storage_offset(at);
  return t;
}
// Torch makes it where there is more to do than to take memory: an object of another device;
// a size below zero, which it refuses; its deterministic mode, where it fills the memory (rows
// that a call leaves as they were hold NaN or a type's largest, the same every time).
at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType dtype, int device) {
  const at::Context& context = at::globalContext();
  bool plain = device == c10::cuda::current_device() &&
               !(context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory());
  int64_t bytes = static_cast<int64_t>(c10::elementSize(dtype));
  for (const int64_t n : shape) {
    plain = plain && n >= 0;
    bytes *= n;
  }
  if (!plain)
    return at::empty(shape,
                     at::TensorOptions().dtype(dtype).device(at::Device(at::kCUDA, device)));
  return tensor_of(new_storage(bytes), 0, shape, dtype);
}
void* handle_of(PyObject* s) {
  THPObjectPtr handle(PyObject_GetAttrString(s, "cuda_stream"));
  if (!handle) {
    PyErr_Clear();
    handle = THPObjectPtr(PyNumber_Long(s));
    if (!handle) throw python_error();
  }
  void* p = PyLong_AsVoidPtr(handle.get());
  if (PyErr_Occurred()) throw python_error();
  return p;
}
// A call's stream, which is torch's current one while this lives: an output made
// here is that stream's memory.  (From the current stream's, it could be a block
// that work queued there still reads, and on its release be given to work there
// before the kernel has written it.)
class CallStream {
 public:
  CallStream(PyObject* s, int device) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device);
    handle_ = current.stream();
    if (s == Py_None) return;
    handle_ = static_cast<cudaStream_t>(handle_of(s));
    if (handle_ == current.stream()) return;
    // (Torch's default stream is the legacy one; its numbers of streams hold odd
    // values for others than handles.)
    guard_.reset_stream(handle_ == nullptr || handle_ == cudaStreamLegacy
                            ? c10::cuda::getDefaultCUDAStream(device)
                            : c10::cuda::getStreamFromExternal(handle_, device));
  }
  operator void*() const { return handle_; }

 private:
  cudaStream_t handle_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}
// `call` without the interpreter's lock: a launch blocks where the GPU's queue is
// full, and what would empty it may be another thread's to issue.
template <typename Call>
mxfp8_status unlocked(Call&& call) {
  PyThreadState* const state = PyEval_SaveThread();
  const mxfp8_status status = call();
  PyEval_RestoreThread(state);
  return status;
}
// What the package raises for a status that is not OK.
void check(mxfp8_status status, const char* where) {
  if (status == MXFP8_OK) return;
  THPObjectPtr module(PyImport_ImportModule("mxfp8_gemm_mailbox_gb300._lib"));
  if (module)
    THPObjectPtr(PyObject_CallMethod(module.get(), "check", "is", static_cast<int>(status), where));
  throw python_error();
}
void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want)
    refuse(PyExc_TypeError, "takes " + std::to_string(want) + " arguments, got " +
                                std::to_string(got));
}
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}
// A matrix a head.
const at::Tensor& matrices(PyObject* o) {
  const at::Tensor& w = tensor(o, "w");
  if (w.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError, std::string("w must be bfloat16, got ") + name_of(w.scalar_type()));
  if (w.dim() != 3)
    refuse(PyExc_ValueError, "w must be [heads][outputs][inputs], got " + text_of(w.sizes()));
  on_current_device(w, "w");
  if (!w.is_contiguous()) refuse(PyExc_ValueError, "w must be a contiguous CUDA tensor");
  return w;
}
int32_t rows_of(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) refuse(PyExc_ValueError, std::string(name) + " must be [rows][heads][...]");
  return static_cast<int32_t>(t.size(0));
}

// (q_nope, q_rope, w, out | None, stream | None) -> out
PyObject* latent_query(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const at::Tensor& w = matrices(args[2]);
  const int64_t heads = w.size(0), latent = w.size(1), nope = w.size(2);
  const int device = gpu_of(w);
  const at::Tensor &q = tensor(args[0], "q_nope"), &rope = tensor(args[1], "q_rope");
  const int32_t rows = rows_of(q, "q_nope");
  expect(q, "q_nope", at::kBFloat16, {rows, heads, nope}, device);
  expect(rope, "q_rope", at::kBFloat16, {rows, heads, kRope}, device);
  const CallStream stream(args[4], device);
  at::Tensor out;
  if (args[3] == Py_None) {
    out = new_tensor({rows, heads, latent + kRope}, at::kBFloat16, device);
  } else {
    out = tensor(args[3], "out");
    expect(out, "out", at::kBFloat16, {rows, heads, latent + kRope}, device);
  }
  const void *const qp = q.data_ptr(), *const rp = rope.data_ptr(), *const wp = w.data_ptr();
  void* const op = out.data_ptr();
  check(unlocked([&] {
          return mxfp8_latent_query(qp, rp, wp, op, rows, static_cast<int32_t>(heads),
                                    static_cast<int32_t>(nope), static_cast<int32_t>(latent),
                                    stream);
        }),
        "mxfp8_latent_query");
  return args[3] == Py_None ? THPVariable_Wrap(std::move(out)) : given(args[3]);
  END_HANDLE_TH_ERRORS
}

// (o, w, x | None, x_scale | None, stream | None) -> (x, x_scale)
PyObject* latent_values(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const at::Tensor& w = matrices(args[1]);
  const int64_t heads = w.size(0), value = w.size(1), latent = w.size(2), k = heads * value;
  const int device = gpu_of(w);
  const at::Tensor& o = tensor(args[0], "o");
  const int32_t rows = rows_of(o, "o");
  expect(o, "o", at::kBFloat16, {rows, heads, latent}, device);
  const CallStream stream(args[4], device);
  auto result = [&](PyObject* t, const char* name, at::ScalarType dtype, int64_t cols) {
    if (t == Py_None) return new_tensor({rows, cols}, dtype, device);
    const at::Tensor& x = tensor(t, name);
    codes(x, name, cols, rows);
    expect(x, name, x.scalar_type(), {rows, cols}, device);
    return x;
  };
  at::Tensor x = result(args[2], "x", at::kFloat8_e4m3fn, k);
  at::Tensor scale = result(args[3], "x_scale", at::kFloat8_e8m0fnu, k / 32);
  const void *const op = o.data_ptr(), *const wp = w.data_ptr();
  void *const xp = x.data_ptr(), *const sp = scale.data_ptr();
  check(unlocked([&] {
          return mxfp8_latent_values(op, wp, xp, sp, rows, static_cast<int32_t>(heads),
                                     static_cast<int32_t>(latent), static_cast<int32_t>(value),
                                     stream);
        }),
        "mxfp8_latent_values");
  THPObjectPtr a(args[2] == Py_None ? THPVariable_Wrap(std::move(x)) : given(args[2]));
  THPObjectPtr b(args[3] == Py_None ? THPVariable_Wrap(std::move(scale)) : given(args[3]));
  if (!a || !b) throw python_error();
  return PyTuple_Pack(2, a.get(), b.get());
  END_HANDLE_TH_ERRORS
}

// (heads, latent, workspace, its bytes, flags, q, cache, page_table, lengths, row_begin, scale,
//  tree | None, out | None, stream | None) -> out; workspace and flags are tensors.
PyObject* latent_attend(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 14);
  const int64_t heads = integer(args[0]), latent = integer(args[1]), width = latent + kRope;
  const at::Tensor& workspace = tensor(args[2], "workspace");
  const at::Tensor &q = tensor(args[5], "q"), &cache = tensor(args[6], "cache");
  const at::Tensor &table = tensor(args[7], "page_table"), &lengths = tensor(args[8], "lengths");
  const at::Tensor& begin = tensor(args[9], "row_begin");
  if (q.dim() != 3 || q.size(1) != heads || q.size(2) != width)
    refuse(PyExc_ValueError, "q must be [rows][" + std::to_string(heads) + "][" +
                                 std::to_string(width) + "], got " + text_of(q.sizes()));
  const int device = on_current_device(q, "q");
  if (gpu_of(workspace) != device)
    refuse(PyExc_ValueError, "q is on device " + std::to_string(device) +
                                 ", this object's workspace is not");
  const int64_t rows = q.size(0);
  expect(q, "q", at::kBFloat16, {rows, heads, width}, device);
  if (cache.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError,
           std::string("cache must be bfloat16, got ") + name_of(cache.scalar_type()));
  if (cache.dim() != 3 || cache.size(2) != width)
    refuse(PyExc_ValueError, "cache must be [pages][page_size][" + std::to_string(width) +
                                 "], got " + text_of(cache.sizes()));
  if (gpu_of(cache) != device || cache.stride(2) != 1)
    refuse(PyExc_ValueError, "cache must be a CUDA tensor on device " + std::to_string(device) +
                                 " with contiguous tokens");
  if (table.dim() != 2)
    refuse(PyExc_ValueError,
           "page_table must be [requests][width], got " + text_of(table.sizes()));
  const int64_t requests = table.size(0), limit = INT32_MAX;
  expect(table, "page_table", at::kInt, table.sizes(), device);
  expect(lengths, "lengths", at::kInt, {requests}, device);
  expect(begin, "row_begin", at::kInt, {requests + 1}, device);
  const void* masks = nullptr;
  if (args[11] != Py_None) {
    const at::Tensor& tree = tensor(args[11], "tree");
    expect(tree, "tree", at::kLong, {rows}, device);
    masks = tree.data_ptr();
  }
  if (rows > limit || requests > limit || cache.size(0) > limit || cache.size(1) > limit ||
      table.size(1) > limit)
    refuse(PyExc_ValueError, "a size is past 2^31 - 1");
  const CallStream stream(args[13], device);
  at::Tensor out;
  if (args[12] == Py_None) {
    out = new_tensor({rows, heads, latent}, at::kBFloat16, device);
  } else {
    out = tensor(args[12], "out");
    expect(out, "out", at::kBFloat16, {rows, heads, latent}, device);
  }
  const double scale = PyFloat_AsDouble(args[10]);
  if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  const mxfp8_latent_desc desc = {static_cast<int32_t>(heads),
                                  static_cast<int32_t>(latent),
                                  static_cast<int32_t>(rows),
                                  static_cast<int32_t>(requests),
                                  static_cast<int32_t>(cache.size(1)),
                                  static_cast<int32_t>(cache.size(0)),
                                  static_cast<int32_t>(table.size(1)),
                                  static_cast<float>(scale),
                                  cache.stride(1),
                                  cache.stride(0)};
  const void *const qp = q.data_ptr(), *const kp = cache.data_ptr();
  const auto *const tp = static_cast<const int32_t*>(table.data_ptr()),
             *const lp = static_cast<const int32_t*>(lengths.data_ptr()),
             *const bp = static_cast<const int32_t*>(begin.data_ptr());
  void *const op = out.data_ptr(), *const sp = workspace.data_ptr();
  const auto bytes = static_cast<size_t>(integer(args[3]));
  auto* const flags = static_cast<int32_t*>(tensor(args[4], "flags").data_ptr());
  check(unlocked([&] {
          return mxfp8_latent_attend(&desc, qp, kp, tp, lp, bp, static_cast<const int64_t*>(masks),
                                     op, sp, bytes, flags, stream);
        }),
        "mxfp8_latent_attend");
  return args[12] == Py_None ? THPVariable_Wrap(std::move(out)) : given(args[12]);
  END_HANDLE_TH_ERRORS
}

// (handle, n, k, adapters' descriptor, workspace, its bytes, x, x_scale, which, alpha | None,
//  c | None, stream | None) -> c; the handle and the descriptor as addresses, the workspace, which
//  is where the adapters are, a tensor.
PyObject* run_adapted(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 12);
  const int64_t outputs = integer(args[1]), k = integer(args[2]);
  const at::Tensor &x = tensor(args[6], "x"), &scale = tensor(args[7], "x_scale");
  const at::Tensor& which = tensor(args[8], "which");
  const void *alpha = nullptr;
  void* c = nullptr;
  if (args[9] != Py_None) {
    const at::Tensor& t = tensor(args[9], "alpha");
    if (t.scalar_type() != at::kFloat || !t.is_cuda())
      refuse(PyExc_TypeError, "alpha must be a float32 CUDA tensor");
    if (t.numel() != 1)
      refuse(PyExc_ValueError, "alpha must hold one number, got " + text_of(t.sizes()));
    alpha = t.data_ptr();
  }
  const int64_t m = codes(x, "x", k, 0);
  codes(scale, "x_scale", k / 32, m);
  const int device = on_current_device(x, "x");
  const at::Tensor& workspace = tensor(args[4], "workspace");
  if (gpu_of(workspace) != device)
    refuse(PyExc_ValueError, "x is on device " + std::to_string(device) + ", the adapters are not");
  if (args[10] != Py_None) {
    const at::Tensor& t = tensor(args[10], "c");
    halves(t, "c", outputs, m);
    c = t.data_ptr();
  }
  if (which.scalar_type() != at::kInt || which.dim() != 1 || which.size(0) < m)
    refuse(PyExc_ValueError, "which must be int32 [>= " + std::to_string(m) + "], got " +
                                 name_of(which.scalar_type()) + " " + text_of(which.sizes()));
  if (!which.is_cuda() || !which.is_contiguous())
    refuse(PyExc_ValueError, "which must be a contiguous CUDA tensor");
  for (const int i : {7, 8, 9, 10})
    if (args[i] != Py_None && gpu_of(THPVariable_Unpack(args[i])) != device)
      refuse(PyExc_ValueError, std::string(i == 7   ? "x_scale"
                                           : i == 8 ? "which"
                                           : i == 9 ? "alpha"
                                                    : "c") +
                                   " must be on device " + std::to_string(device));
  const CallStream stream(args[11], device);
  auto* const gemm = static_cast<mxfp8_publish_gemm*>(address(args[0]));
  const auto* const adapters = static_cast<const mxfp8_adapters*>(address(args[3]));
  void* const space = workspace.data_ptr();
  const auto bytes = static_cast<size_t>(integer(args[5]));
  const void *const xp = x.data_ptr(), *const sp = scale.data_ptr();
  const auto* const ip = static_cast<const int32_t*>(which.data_ptr());
  check(unlocked([&] {
          return mxfp8_publish_gemm_run_adapted(
              gemm, xp, sp, static_cast<int32_t>(std::min<int64_t>(m, INT32_MAX)),
              static_cast<const float*>(alpha), adapters, ip, space, bytes, c, stream);
        }),
        "mxfp8_publish_gemm_run_adapted");
  return given(args[10]);
  END_HANDLE_TH_ERRORS
}

// (words, state, capacity, n, m, out | None, timeout_ns, stream | None) -> out; words and state
// are tensors.
PyObject* mailbox_consume(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  arguments(count, 8);
  const at::Tensor &words = tensor(args[0], "words"), &state = tensor(args[1], "state");
  const int64_t capacity = integer(args[2]), n = integer(args[3]), m = integer(args[4]);
  if (m < INT32_MIN || m > INT32_MAX) refuse(PyExc_ValueError, "m is past 32 bits");
  const CallStream stream(args[7], c10::cuda::current_device());
  at::Tensor out;
  if (args[5] == Py_None) {
    out = new_tensor({m, n}, at::kBFloat16, gpu_of(words));
  } else {
    out = tensor(args[5], "out");
    halves(out, "out", n, m);
  }
  const uint64_t timeout = PyLong_AsUnsignedLongLongMask(args[6]);  // -1: no limit
  if (PyErr_Occurred()) throw python_error();
  void *const wp = words.data_ptr(), *const op = out.data_ptr();
  auto* const sp = static_cast<int32_t*>(state.data_ptr());
  check(unlocked([&] {
          return ::mailbox_consume(wp, sp, static_cast<int32_t>(capacity), static_cast<int32_t>(n),
                                   static_cast<int32_t>(m), op, timeout, stream);
        }),
        "mailbox_consume");
  return args[5] == Py_None ? THPVariable_Wrap(std::move(out)) : given(args[5]);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ a layer of routed experts

// MXFP8_BF16, _FP16 or _FP32.
int32_t type_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MXFP8_BF16;
    case at::kHalf: return MXFP8_FP16;
    case at::kFloat: return MXFP8_FP32;
    default:
      refuse(PyExc_TypeError, std::string(name) + " must be bfloat16, float16 or float32, got " +
                                  name_of(t.scalar_type()));
  }
}
// A matrix whose rows are contiguous and may be strided; returns the stride.
int64_t strided_rows(const at::Tensor& t, const char* name, const char* shape) {
  if (t.dim() != 2)
    refuse(PyExc_ValueError, std::string(name) + " must be " + shape + ", got " + text_of(t.sizes()));
  if (!t.is_cuda() || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor with contiguous rows");
  return t.stride(0);
}
int32_t narrowed(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, std::string(what) + " is past 2^31 - 1");
  return static_cast<int32_t>(v);
}
int32_t* flags_of(PyObject* o, int device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "flags");
  expect(t, "flags", at::kInt, {1}, device);
  return static_cast<int32_t*>(t.data_ptr());
}
// What a format is called, as a number.
int32_t format_of(PyObject* o, bool none_is_bf16) {
  if (none_is_bf16 && o == Py_None) return MXFP8_FORMAT_BF16;
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "mxfp8") == 0) return MXFP8_FORMAT_MXFP8;
    if (PyUnicode_CompareWithASCIIString(o, "mxfp4") == 0) return MXFP8_FORMAT_MXFP4;
  }
  refuse(PyExc_ValueError, none_is_bf16 ? "format must be None, \"mxfp8\" or \"mxfp4\""
                                        : "format must be \"mxfp8\" or \"mxfp4\"");
}
// One-byte codes of exactly this shape, contiguous, on the device.
void exact_codes(const at::Tensor& t, const char* name, at::IntArrayRef shape, int device) {
  if (t.element_size() != 1)
    refuse(PyExc_TypeError, std::string(name) + " must hold one-byte codes (uint8 / float8), got " +
                                name_of(t.scalar_type()));
  expect(t, name, t.scalar_type(), shape, device);
}

// (logits, k, normalize, stream | None) -> (weight, expert, slot, row, begin)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const at::Tensor& logits = tensor(args[0], "logits");
  const int32_t type = type_of(logits, "logits");
  const int64_t stride = strided_rows(logits, "logits", "[tokens][experts]");
  const int device = on_current_device(logits, "logits");
  const int64_t tokens = logits.size(0), experts = logits.size(1), k = integer(args[1]);
  const int normalize = PyObject_IsTrue(args[2]);
  if (normalize < 0) throw python_error();
  // Sizes that no output could be made for; the others the library refuses.
  if (k < 1 || k > MXFP8_MAX_CHOICES || k > experts)
    refuse(PyExc_ValueError, "k must be in 1..min(experts, " + std::to_string(MXFP8_MAX_CHOICES) +
                                 "), got " + std::to_string(k) + " of " + std::to_string(experts));
  if (tokens > INT32_MAX / k) refuse(PyExc_ValueError, "tokens x k must be below 2^31");
  const CallStream stream(args[3], device);
  const auto space = static_cast<int64_t>(
      mxfp8_route_workspace_bytes(tokens, narrowed(experts, "the number of experts")));
  // All five in one piece of memory, and the workspace behind them, each on a boundary of
  // 16 bytes (places in words of 4).
  const auto rounded = [](int64_t words) { return (words + 3) / 4 * 4; };
  const int64_t each = rounded(tokens * k), begins = rounded(experts + 1);
  c10::Storage memory = new_storage(4 * (4 * each + begins) + space);
  auto* const ep = static_cast<int32_t*>(memory.mutable_data()) + each;
  auto* const wp = reinterpret_cast<float*>(ep - each);
  int32_t *const sp = ep + each, *const rp = sp + each, *const bp = rp + each;
  void* const space_p = space ? bp + begins : nullptr;
  const void* const lp = logits.data_ptr();
  check(unlocked([&] {
          return mxfp8_route(lp, type, stride, tokens, static_cast<int32_t>(experts),
                             static_cast<int32_t>(k), normalize, wp, ep, sp, rp, bp, space_p,
                             static_cast<size_t>(space), stream);
        }),
        "mxfp8_route");
  PyObject* out = PyTuple_New(5);
  if (!out) throw python_error();
  PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(tensor_of(memory, 0, {tokens, k}, at::kFloat)));
  PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(tensor_of(memory, each, {tokens, k}, at::kInt)));
  PyTuple_SET_ITEM(out, 2, THPVariable_Wrap(tensor_of(memory, 2 * each, {tokens, k}, at::kInt)));
  PyTuple_SET_ITEM(out, 3, THPVariable_Wrap(tensor_of(memory, 3 * each, {tokens * k}, at::kInt)));
  PyTuple_SET_ITEM(out, 4, THPVariable_Wrap(tensor_of(memory, 4 * each, {experts + 1}, at::kInt)));
  return out;
  END_HANDLE_TH_ERRORS
}

// (x, format, rows | None, codes | None, scale | None, flags | None, stream | None) -> (codes,
// scale)
PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const at::Tensor& x = tensor(args[0], "x");
  const int32_t type = type_of(x, "x"), format = format_of(args[1], false);
  if (x.dim() < 1) refuse(PyExc_ValueError, "x must be [...][K], got " + text_of(x.sizes()));
  const int device = on_current_device(x, "x");
  const int64_t k = x.size(-1);
  if (k < 32 || k % 32)
    refuse(PyExc_ValueError, "K must be a positive multiple of 32, got " + std::to_string(k));
  int64_t x_rows = 1, stride = k;
  if (x.dim() == 2) {
    stride = strided_rows(x, "x", "[rows][K]");
    x_rows = x.size(0);
  } else {
    if (!x.is_contiguous())
      refuse(PyExc_ValueError, "x of other than two axes must be contiguous");
    x_rows = x.numel() / k;
  }
  std::vector<int64_t> shape(x.sizes().begin(), x.sizes().end());
  const int32_t* index = nullptr;
  int64_t out_rows = x_rows;
  if (args[2] != Py_None) {
    const at::Tensor& rows = tensor(args[2], "rows");
    if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [rows][K] to be indexed");
    if (rows.dim() != 1)
      refuse(PyExc_ValueError, "rows must have one axis, got " + text_of(rows.sizes()));
    expect(rows, "rows", at::kInt, rows.sizes(), device);
    shape[0] = out_rows = rows.size(0);
    index = static_cast<const int32_t*>(rows.data_ptr());
    // (An empty tensor has no address, and without one every row would be taken.)
    if (out_rows == 0) index = reinterpret_cast<const int32_t*>(uintptr_t{4});
  }
  int32_t* const flags = flags_of(args[5], device);
  const CallStream stream(args[6], device);
  const bool wide = format == MXFP8_FORMAT_MXFP8;
  const auto result = [&](PyObject* t, const char* name, at::ScalarType dtype, int64_t last) {
    shape.back() = last;
    if (t == Py_None) return new_tensor(shape, dtype, device);
    exact_codes(tensor(t, name), name, shape, device);
    return tensor(t, name);
  };
  at::Tensor codes = result(args[3], "codes", wide ? at::kFloat8_e4m3fn : at::kByte,
                            wide ? k : k / 2);
  at::Tensor scale = result(args[4], "scale", at::kFloat8_e8m0fnu, k / 32);
  const int32_t k32 = narrowed(k, "K");
  const void* const xp = x.data_ptr();
  void *const cp = codes.data_ptr(), *const sp = scale.data_ptr();
  check(unlocked([&] {
          return mxfp8_quantize(xp, type, stride, x_rows, k32, index, out_rows, format, cp, sp, flags,
                                stream);
        }),
        "mxfp8_quantize");
  THPObjectPtr a(args[3] == Py_None ? THPVariable_Wrap(std::move(codes)) : given(args[3]));
  THPObjectPtr b(args[4] == Py_None ? THPVariable_Wrap(std::move(scale)) : given(args[4]));
  if (!a || !b) throw python_error();
  return PyTuple_Pack(2, a.get(), b.get());
  END_HANDLE_TH_ERRORS
}

// (codes, scale, type as a number, stream | None) -> values
PyObject* dequantize(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const at::Tensor &codes = tensor(args[0], "codes"), &scale = tensor(args[1], "scale");
  if (scale.dim() < 1)
    refuse(PyExc_ValueError, "scale must be [...][K / 32], got " + text_of(scale.sizes()));
  const int device = on_current_device(scale, "scale");
  exact_codes(scale, "scale", scale.sizes(), device);
  const int64_t k = scale.size(-1) * 32;
  if (k == 0) refuse(PyExc_ValueError, "K must be a positive multiple of 32, got 0");
  const bool wide = codes.dim() == scale.dim() && codes.size(-1) == k;
  std::vector<int64_t> shape(scale.sizes().begin(), scale.sizes().end());
  shape.back() = wide ? k : k / 2;
  exact_codes(codes, "codes", shape, device);
  shape.back() = k;
  const int32_t type = static_cast<int32_t>(integer(args[2]));
  const CallStream stream(args[3], device);
  at::Tensor out = new_tensor(
      shape, type == MXFP8_BF16 ? at::kBFloat16 : type == MXFP8_FP16 ? at::kHalf : at::kFloat,
      device);
  const void *const cp = codes.data_ptr(), *const sp = scale.data_ptr();
  void* const op = out.data_ptr();
  const int64_t rows = scale.numel() / (k / 32);
  const int32_t k32 = narrowed(k, "K");
  check(unlocked([&] {
          return mxfp8_dequantize(cp, sp, rows, k32,
                                  wide ? MXFP8_FORMAT_MXFP8 : MXFP8_FORMAT_MXFP4, type, op, stream);
        }),
        "mxfp8_dequantize");
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// (experts, n, k, gated, w_format, w, laid scales, workspace, flags, x, x_scale, begin | None,
//  format | None, out | None, out_scale | None, stream | None) -> out or (out, out_scale)
PyObject* expert_product(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  arguments(count, 16);
  mxfp8_expert_desc desc{};
  desc.experts = static_cast<int32_t>(integer(args[0]));
  desc.n = static_cast<int32_t>(integer(args[1]));
  desc.k = static_cast<int32_t>(integer(args[2]));
  desc.gated = static_cast<int32_t>(integer(args[3]));
  desc.w_format = static_cast<int32_t>(integer(args[4]));
  const at::Tensor &w = tensor(args[5], "w"), &laid = tensor(args[6], "laid");
  const at::Tensor& workspace = tensor(args[7], "workspace");
  const at::Tensor &x = tensor(args[9], "x"), &x_scale = tensor(args[10], "x_scale");
  const int64_t n = desc.n, k = desc.k;
  const int device = on_current_device(x, "x");
  if (gpu_of(w) != device)
    refuse(PyExc_ValueError,
           "x is on device " + std::to_string(device) + ", this object's matrices are not");
  if (x.dim() != 2 || (x.size(1) != k && x.size(1) != k / 2))
    refuse(PyExc_ValueError, "x must be [rows][" + std::to_string(k) + "] (MXFP8) or [rows][" +
                                 std::to_string(k / 2) + "] (MXFP4), got " + text_of(x.sizes()));
  const int64_t rows = x.size(0);
  exact_codes(x, "x", x.sizes(), device);
  exact_codes(x_scale, "x_scale", {rows, k / 32}, device);
  desc.x_format = x.size(1) == k ? MXFP8_FORMAT_MXFP8 : MXFP8_FORMAT_MXFP4;
  desc.out_format = format_of(args[12], true);
  desc.rows = narrowed(rows, "the number of rows");
  const int32_t* begin = nullptr;
  if (args[11] != Py_None) {
    const at::Tensor& b = tensor(args[11], "begin");
    expect(b, "begin", at::kInt, {desc.experts + 1}, device);
    begin = static_cast<const int32_t*>(b.data_ptr());
  }
  int32_t* const flags = flags_of(args[8], device);
  const bool codes = desc.out_format != MXFP8_FORMAT_BF16;
  if (codes && n % 32)
    refuse(PyExc_ValueError, "N must be a multiple of 32 to be rounded to blocks, got " +
                                 std::to_string(n));
  if (!codes && args[14] != Py_None) refuse(PyExc_ValueError, "out_scale goes with a format");
  const CallStream stream(args[15], device);
  const int64_t width = desc.out_format == MXFP8_FORMAT_MXFP4 ? n / 2 : n;
  at::Tensor out, scale;
  if (args[13] == Py_None) {
    out = new_tensor({rows, width},
                     desc.out_format == MXFP8_FORMAT_BF16    ? at::kBFloat16
                     : desc.out_format == MXFP8_FORMAT_MXFP8 ? at::kFloat8_e4m3fn
                                                             : at::kByte,
                     device);
  } else {
    out = tensor(args[13], "out");
    if (codes)
      exact_codes(out, "out", {rows, width}, device);
    else
      expect(out, "out", at::kBFloat16, {rows, width}, device);
  }
  if (codes) {
    if (args[14] == Py_None) {
      scale = new_tensor({rows, n / 32}, at::kFloat8_e8m0fnu, device);
    } else {
      scale = tensor(args[14], "out_scale");
      exact_codes(scale, "out_scale", {rows, n / 32}, device);
    }
  }
  const void *const wp = w.data_ptr(), *const lp = laid.data_ptr(), *const xp = x.data_ptr(),
                    *const sp = x_scale.data_ptr();
  void *const op = out.data_ptr(), *const tp = codes ? scale.data_ptr() : nullptr,
              *const space = workspace.data_ptr();
  const auto bytes = static_cast<size_t>(workspace.numel());
  check(unlocked([&] {
          return mxfp8_expert_product(&desc, wp, lp, xp, sp, begin, op, tp, space, bytes, flags, stream);
        }),
        "mxfp8_expert_product");
  THPObjectPtr a(args[13] == Py_None ? THPVariable_Wrap(std::move(out)) : given(args[13]));
  if (!a) throw python_error();
  if (!codes) return a.release();
  THPObjectPtr b(args[14] == Py_None ? THPVariable_Wrap(std::move(scale)) : given(args[14]));
  if (!b) throw python_error();
  return PyTuple_Pack(2, a.get(), b.get());
  END_HANDLE_TH_ERRORS
}

// (y, weight, slot, add | None, out | None, flags | None, stream | None) -> out
PyObject* combine(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  arguments(count, 7);
  const at::Tensor &y = tensor(args[0], "y"), &weight = tensor(args[1], "weight");
  const at::Tensor& slot = tensor(args[2], "slot");
  if (y.scalar_type() != at::kBFloat16)
    refuse(PyExc_TypeError, std::string("y must be bfloat16, got ") + name_of(y.scalar_type()));
  const int64_t stride = strided_rows(y, "y", "[rows][N]");
  const int device = on_current_device(y, "y");
  const int64_t n = y.size(1);
  if (slot.dim() != 2)
    refuse(PyExc_ValueError, "slot must be [tokens][k], got " + text_of(slot.sizes()));
  const int64_t tokens = slot.size(0), k = slot.size(1);
  expect(slot, "slot", at::kInt, {tokens, k}, device);
  expect(weight, "weight", at::kFloat, {tokens, k}, device);
  const void* add = nullptr;
  if (args[3] != Py_None) {
    const at::Tensor& t = tensor(args[3], "add");
    expect(t, "add", at::kBFloat16, {tokens, n}, device);
    add = t.data_ptr();
  }
  int32_t* const flags = flags_of(args[5], device);
  const CallStream stream(args[6], device);
  at::Tensor out;
  if (args[4] == Py_None) {
    out = new_tensor({tokens, n}, at::kBFloat16, device);
  } else {
    out = tensor(args[4], "out");
    expect(out, "out", at::kBFloat16, {tokens, n}, device);
  }
  const int32_t slots = narrowed(y.size(0), "the number of rows"), k32 = narrowed(k, "k"),
                n32 = narrowed(n, "N");
  const void* const yp = y.data_ptr();
  const auto* const wp = static_cast<const float*>(weight.data_ptr());
  const auto* const sp = static_cast<const int32_t*>(slot.data_ptr());
  void* const op = out.data_ptr();
  check(unlocked([&] {
          return mxfp8_combine(yp, stride, slots, wp, sp, tokens, k32, n32, add, op, flags, stream);
        }),
        "mxfp8_combine");
  return args[4] == Py_None ? THPVariable_Wrap(std::move(out)) : given(args[4]);
  END_HANDLE_TH_ERRORS
}

PyCFunction fast(PyObject* (*call)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call));
}
PyMethodDef methods[] = {{"latent_query", fast(latent_query), METH_FASTCALL, nullptr},
                         {"latent_values", fast(latent_values), METH_FASTCALL, nullptr},
                         {"latent_attend", fast(latent_attend), METH_FASTCALL, nullptr},
                         {"run_adapted", fast(run_adapted), METH_FASTCALL, nullptr},
                         {"mailbox_consume", fast(mailbox_consume), METH_FASTCALL, nullptr},
                         {"route", fast(route), METH_FASTCALL, nullptr},
                         {"quantize", fast(quantize), METH_FASTCALL, nullptr},
                         {"dequantize", fast(dequantize), METH_FASTCALL, nullptr},
                         {"expert_product", fast(expert_product), METH_FASTCALL, nullptr},
                         {"combine", fast(combine), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
