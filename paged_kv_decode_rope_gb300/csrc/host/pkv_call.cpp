// pkv_call.cpp -- the Python side of the calls that a serving step makes: the
// checks of their tensors and the call of the C ABI (include/pkv.h), as a
// CPython module.
//
// On a small step these calls last 2 to 4 us on the GPU. Reading shapes, types
// and pointers off ten tensors in Python and passing them through ctypes took
// 8 to 11 us, so the host set the pace; here a call takes about 3 us, most of it
// the launch. Refusals are worded as everywhere in the binding. The library's
// entry points come from its ctypes handle (bind), so that this module needs
// nothing of CUDA but torch's current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "../../../include/pkv.h"

namespace {

struct {
  decltype(&paged_tables_build) tables;
  decltype(&paged_rope_append) rope;
  decltype(&paged_gqa_decode_scored) decode;
  decltype(&paged_gqa_prefill_scored) prefill;
  decltype(&token_logprobs) logprobs;
} g_lib;

constexpr int64_t kAny = -1;

// A refused argument: a Python exception is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const std::string& why) {
  PyErr_SetString(kind, why.c_str());
  throw Refused();
}

std::string dims(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + (s[i] == kAny ? std::string("*") : std::to_string(s[i]));
  return r + "]";
}

const char* type_name(at::ScalarType t) {
  return t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32" : t == at::kBFloat16 ? "torch.bfloat16"
                                                                                              : "torch.uint8";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

void check_shape(const at::Tensor& t, std::initializer_list<int64_t> want, const char* name) {
  const at::IntArrayRef got = t.sizes(), w(want);
  bool same = got.size() == w.size();
  for (size_t i = 0; same && i < w.size(); ++i) same = w[i] == kAny || w[i] == got[i];
  if (!same) refuse(PyExc_ValueError, std::string(name) + " must have shape " + dims(w) + ", got " + dims(got));
}

void check_cuda(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
}

// The tensor, of this shape.
const at::Tensor& sized(PyObject* o, std::initializer_list<int64_t> want, const char* name) {
  const at::Tensor& t = tensor(o, name);
  check_shape(t, want, name);
  return t;
}

// The pointer of a contiguous CUDA tensor of this type and shape.
void* pointer(const at::Tensor& t, at::ScalarType type, const char* name) {
  check_cuda(t, name);
  if (t.scalar_type() != type)
    refuse(PyExc_ValueError, std::string(name) + " must be " + type_name(type) + ", got " + toString(t.scalar_type()));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}
void* pointer(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> want, const char* name) {
  return pointer(sized(o, want, name), type, name);
}
template <typename T>
T* ints(PyObject* o, std::initializer_list<int64_t> want, const char* name) {
  return static_cast<T*>(pointer(o, at::kInt, want, name));
}
// The same, or null for None.
void* optional(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> want, const char* name) {
  return o == Py_None ? nullptr : pointer(o, type, want, name);
}

// PKV_BF16 or PKV_F32.
int type_of(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return PKV_BF16;
  if (t.scalar_type() == at::kFloat) return PKV_F32;
  refuse(PyExc_ValueError,
         std::string(name) + " must be bfloat16 or float32, got " + toString(t.scalar_type()));
}

int size_of(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too large");
  return static_cast<int>(n);
}

long long number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int integer(PyObject* o, const char* name) {
  const long long v = number(o);
  if (v > INT32_MAX || v < INT32_MIN) refuse(PyExc_ValueError, std::string(name) + " is too large");
  return static_cast<int>(v);
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return static_cast<float>(v);
}
pkv_pool_t* pool_of(PyObject* o) { return reinterpret_cast<pkv_pool_t*>(number(o)); }

// The stream given (a torch stream or a cudaStream_t as a number), or torch's
// current one on the tensor's device.
void* stream_of(PyObject* o, const at::Tensor& t, const char* name) {
  check_cuda(t, name);
  if (o == Py_None) return at::cuda::getCurrentCUDAStream(t.get_device()).stream();
  if (PyLong_Check(o)) return reinterpret_cast<void*>(number(o));
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) throw Refused();
  const long long v = PyLong_AsLongLong(raw);
  Py_DECREF(raw);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return reinterpret_cast<void*>(v);
}

// The device of the call's CUDA tensors, -1 if it has none (what is no CUDA
// tensor is refused by name where it is read).
int device_of(PyObject* const* a, Py_ssize_t n) {
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (a[i] == Py_None || PyLong_Check(a[i]) || PyFloat_Check(a[i]) || !THPVariable_Check(a[i])) continue;
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_cuda()) continue;
    const int d = t.get_device();
    if (device >= 0 && d != device)
      refuse(PyExc_ValueError, "all tensors must be on one device, got cuda:" + std::to_string(device) + " and cuda:" +
                                   std::to_string(d));
    device = d;
  }
  return device;
}

// Every function takes exactly `count` positional arguments and returns the
// library's result, called with the tensors' device current. No C++ exception
// leaves it.
template <Py_ssize_t count, typename F>
PyObject* call(PyObject* const* a, Py_ssize_t n, F body) {
  try {
    if (n != count) refuse(PyExc_TypeError, "expected " + std::to_string(count) + " arguments");
    const int device = device_of(a, n);
    c10::cuda::OptionalCUDAGuard guard;
    if (device >= 0) guard.set_index(static_cast<c10::DeviceIndex>(device));
    return PyLong_FromLong(body(a));
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

constexpr int64_t D = PKV_HEAD_DIM;

PyObject* tables_build(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call<12>(a, n, [](PyObject* const* a) {
    const at::Tensor& free_pages = sized(a[3], {kAny}, "free_pages");
    const at::Tensor& tables = sized(a[6], {kAny, kAny, kAny}, "block_tables");
    const at::Tensor& positions = sized(a[9], {kAny}, "positions");
    const int64_t layers = tables.size(0), batch = tables.size(1), blocks = tables.size(2), tokens = positions.size(0);
    return g_lib.tables(
        pool_of(a[0]), ints<const int32_t>(a[1], {batch}, "start_pos"), ints<const int32_t>(a[2], {batch}, "new_tokens"),
        size_of(batch, "batch"), size_of(layers, "layers"),
        static_cast<const int32_t*>(pointer(free_pages, at::kInt, "free_pages")), size_of(free_pages.size(0), "free_pages"),
        ints<const int32_t>(a[4], {1}, "free_head"), ints<int32_t>(a[5], {1}, "free_head_out"),
        static_cast<int32_t*>(pointer(tables, at::kInt, "block_tables")), size_of(blocks, "max_blocks"),
        ints<int32_t>(a[7], {batch + 1}, "cu_tokens"), ints<int32_t>(a[8], {batch}, "seq_lens"),
        static_cast<int32_t*>(pointer(positions, at::kInt, "positions")),
        ints<int32_t>(a[10], {layers, tokens}, "slot_map"), size_of(tokens, "capacity"), stream_of(a[11], tables, "block_tables"));
  });
}

// bf16 [tokens][heads][64] whose heads are contiguous, at any token stride.
struct Rows {
  const void* data;
  long long stride;
};
Rows rows_of(const at::Tensor& t, const char* name) {
  check_cuda(t, name);
  if (t.scalar_type() != at::kBFloat16)
    refuse(PyExc_ValueError, std::string(name) + " must be torch.bfloat16, got " + toString(t.scalar_type()));
  const int64_t tokens = t.size(0), heads = t.size(1);
  if (tokens > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D)))
    refuse(PyExc_ValueError, std::string(name) + " must have contiguous heads");
  return {t.data_ptr(), tokens > 1 ? t.stride(0) : heads * D};
}

PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call<12>(a, n, [](PyObject* const* a) {
    const int64_t hkv = number(a[1]);
    const at::Tensor& q = sized(a[2], {kAny, kAny, D}, "q");
    const int64_t tokens = q.size(0), hq = q.size(1);
    const Rows qr = rows_of(q, "q"), kr = rows_of(sized(a[3], {tokens, hkv, D}, "k"), "k"),
               vr = rows_of(sized(a[4], {tokens, hkv, D}, "v"), "v");
    const at::Tensor& table = sized(a[8], {kAny}, "rope_table");
    return g_lib.rope(pool_of(a[0]), qr.data, qr.stride, kr.data, kr.stride, vr.data, vr.stride,
                      static_cast<float*>(pointer(a[5], at::kFloat, {tokens, hq, D}, "q_rot")),
                      ints<const int32_t>(a[6], {tokens}, "slot_map"), ints<const int32_t>(a[7], {tokens}, "positions"),
                      size_of(tokens, "tokens"), size_of(hq, "heads"), pointer(table, at::kByte, "rope_table"),
                      size_of(table.size(0) / static_cast<int64_t>(PKV_ROPE_TABLE_BYTES(1)), "rope_table"),
                      integer(a[9], "rot_dim"), truth(a[10]), stream_of(a[11], q, "q"));
  });
}

pkv_scoring_t scoring(PyObject* scale, PyObject* softcap, PyObject* slopes, PyObject* window, int64_t hq) {
  pkv_scoring_t s;
  s.scale = real(scale);
  s.softcap = real(softcap);
  s.alibi_slopes = static_cast<const float*>(optional(slopes, at::kFloat, {hq}, "alibi_slopes"));
  s.window = integer(window, "window");
  return s;
}

PyObject* decode_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call<12>(a, n, [](PyObject* const* a) {
    const at::Tensor& q = sized(a[1], {kAny, kAny, D}, "q_rot");
    const int64_t batch = q.size(0), hq = q.size(1);
    const at::Tensor& out = sized(a[2], {batch, hq, D}, "out");
    const at::Tensor& tables = sized(a[3], {batch, kAny}, "block_tables");
    const at::Tensor& ws = sized(a[6], {kAny}, "workspace");
    const int type = type_of(out, "out");
    const pkv_scoring_t s = scoring(a[5], a[7], a[8], a[9], hq);
    return g_lib.decode(pool_of(a[0]), static_cast<const float*>(pointer(q, at::kFloat, "q_rot")),
                        pointer(out, out.scalar_type(), "out"), type,
                        static_cast<const int32_t*>(pointer(tables, at::kInt, "block_tables")),
                        size_of(tables.size(1), "max_blocks"), ints<const int32_t>(a[4], {batch}, "seq_lens"),
                        static_cast<const int32_t*>(optional(a[10], at::kInt, {batch}, "first_keys")),
                        size_of(batch, "batch"), size_of(hq, "heads"), &s, pointer(ws, at::kByte, "workspace"),
                        static_cast<size_t>(ws.size(0)), stream_of(a[11], q, "q_rot"));
  });
}

PyObject* prefill_scored(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call<14>(a, n, [](PyObject* const* a) {
    const at::Tensor& q = sized(a[1], {kAny, kAny, D}, "q_rot");
    const int64_t total = q.size(0), hq = q.size(1);
    const at::Tensor& out = sized(a[2], {total, hq, D}, "out");
    const at::Tensor& tables = sized(a[3], {kAny, kAny}, "block_tables");
    const int64_t batch = tables.size(0);
    const at::Tensor& ws = sized(a[7], {kAny}, "workspace");
    const int type = type_of(out, "out");
    const pkv_scoring_t s = scoring(a[6], a[8], a[9], a[10], hq);
    return g_lib.prefill(pool_of(a[0]), static_cast<const float*>(pointer(q, at::kFloat, "q_rot")),
                         pointer(out, out.scalar_type(), "out"), type,
                         static_cast<const int32_t*>(pointer(tables, at::kInt, "block_tables")),
                         size_of(tables.size(1), "max_blocks"), ints<const int32_t>(a[4], {batch + 1}, "cu_tokens"),
                         ints<const int32_t>(a[5], {batch}, "start_pos"),
                         static_cast<const int32_t*>(optional(a[11], at::kInt, {batch}, "prefix_lens")),
                         static_cast<const int32_t*>(optional(a[12], at::kInt, {total}, "doc_starts")),
                         size_of(batch, "batch"), size_of(total, "tokens"), size_of(hq, "heads"), &s,
                         pointer(ws, at::kByte, "workspace"), static_cast<size_t>(ws.size(0)), stream_of(a[13], q, "q_rot"));
  });
}

PyObject* logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call<9>(a, n, [](PyObject* const* a) {
    const at::Tensor& x = sized(a[0], {kAny, kAny}, "logits");
    check_cuda(x, "logits");
    const int64_t rows = x.size(0), vocab = x.size(1);
    if (vocab > 1 && x.stride(1) != 1) refuse(PyExc_ValueError, "logits must have contiguous rows");
    const int type = type_of(x, "logits");
    const int64_t top = a[4] == Py_None ? 0 : sized(a[4], {rows, kAny}, "top_ids").size(1);
    const at::Tensor& ws = sized(a[6], {kAny}, "workspace");
    return g_lib.logprobs(x.data_ptr(), type, rows > 1 ? x.stride(0) : vocab, size_of(rows, "rows"),
                          size_of(vocab, "vocab"), real(a[7]),
                          static_cast<const int32_t*>(optional(a[1], at::kInt, {rows}, "targets")), size_of(top, "top"),
                          static_cast<float*>(optional(a[2], at::kFloat, {rows}, "logprobs")),
                          static_cast<float*>(optional(a[3], at::kFloat, {rows}, "entropy")),
                          static_cast<int32_t*>(optional(a[4], at::kInt, {rows, top}, "top_ids")),
                          static_cast<float*>(optional(a[5], at::kFloat, {rows, top}, "top_logprobs")),
                          pointer(ws, at::kByte, "workspace"), static_cast<size_t>(ws.size(0)), stream_of(a[8], x, "logits"));
  });
}

// bind(address, ...): the library's entry points, in g_lib's order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call<5>(a, n, [](PyObject* const* a) {
    g_lib.tables = reinterpret_cast<decltype(g_lib.tables)>(number(a[0]));
    g_lib.rope = reinterpret_cast<decltype(g_lib.rope)>(number(a[1]));
    g_lib.decode = reinterpret_cast<decltype(g_lib.decode)>(number(a[2]));
    g_lib.prefill = reinterpret_cast<decltype(g_lib.prefill)>(number(a[3]));
    g_lib.logprobs = reinterpret_cast<decltype(g_lib.logprobs)>(number(a[4]));
    return 0;
  });
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<bind>("bind"),
                           method<tables_build>("paged_tables_build"),
                           method<rope_append>("paged_rope_append"),
                           method<decode_scored>("paged_gqa_decode_scored"),
                           method<prefill_scored>("paged_gqa_prefill_scored"),
                           method<logprobs>("token_logprobs"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pkv_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkv_call() { return PyModule_Create(&g_module); }
