// decode_calls.cpp -- the usual calls of _decode.py, made without Python in
// between: a decoding step's kernels take a few microseconds, checking and
// marshalling a call in Python takes up to fifteen.
//
// Every function here takes the tensors of one call on the current device and
// stream, with nothing given but the inputs.  It makes the call and returns
// its outputs (or the library's error status as an int) if the arguments are as
// they usually are; else it returns None and has done nothing, and _decode.py
// goes through the call step by step and says what is wrong with it.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <map>
#include <utility>
#include <vector>

#include "../../include/topk_b200.h"

namespace {

// Entry points of the CUDA library, set by bind().
struct Entries {
  decltype(&paged_attention) attend;
  decltype(&paged_attention_workspace_bytes) attend_bytes;
  decltype(&cache_write) write;
  decltype(&cache_read) read;
  decltype(&topk_beam) beam;
  decltype(&topk_beam_bf16) beam_bf16;
  decltype(&topk_beam_workspace_bytes) beam_bytes;
  decltype(&beam_reorder) reorder;
} g_lib = {};

struct NotUsual {};

void usual(bool ok) {
  if (!ok) throw NotUsual{};
}

const at::Tensor& tensor(PyObject* o) {
  usual(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

const at::Tensor& on(PyObject* o, int dev, at::ScalarType type, int64_t dims) {
  const at::Tensor& t = tensor(o);
  usual(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.dim() == dims &&
        t.layout() == at::kStrided);
  return t;
}

// The device of `t`, which has to be the current one.
int current_device_of(const at::Tensor& t) {
  usual(t.is_cuda() && t.get_device() == c10::cuda::current_device());
  return t.get_device();
}

at::Tensor empty_on(int dev, at::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<at::DeviceIndex>(dev)), std::nullopt);
}

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(const_cast<void*>(t.const_data_ptr()));
}

topk_cache cache_of(PyObject* data_obj, PyObject* scale_obj, int dev) {
  const at::Tensor& t = tensor(data_obj);
  topk_cache c{};
  c.type = t.scalar_type() == at::kFloat8_e4m3fn ? TOPK_CACHE_E4M3 : TOPK_CACHE_BF16;
  usual(c.type == TOPK_CACHE_E4M3 || t.scalar_type() == at::kBFloat16);
  usual(t.is_cuda() && t.get_device() == dev && t.dim() == 4 && t.layout() == at::kStrided && t.stride(3) == 1);
  usual(t.size(1) <= INT32_MAX && t.size(2) <= INT32_MAX && t.size(3) <= INT32_MAX);
  c.data = data<void>(t);
  c.pages = t.size(0);
  c.kv_heads = static_cast<int>(t.size(1));
  c.page_size = static_cast<int>(t.size(2));
  c.d = static_cast<int>(t.size(3));
  c.page_stride = t.stride(0);
  c.head_stride = t.stride(1);
  c.token_stride = t.stride(2);
  if (c.type == TOPK_CACHE_BF16) {
    usual(scale_obj == Py_None);
    return c;
  }
  const at::Tensor& s = on(scale_obj, dev, at::kFloat, 3);
  usual(s.size(0) == t.size(0) && s.size(1) == t.size(1) && s.size(2) == t.size(2));
  c.scale = data<float>(s);
  c.scale_page_stride = s.stride(0);
  c.scale_head_stride = s.stride(1);
  c.scale_token_stride = s.stride(2);
  return c;
}

bool alike(const topk_cache& a, const topk_cache& b) {
  return a.type == b.type && a.pages == b.pages && a.kv_heads == b.kv_heads && a.page_size == b.page_size && a.d == b.d;
}

struct Table {
  const int32_t* table;
  const int32_t* lens;
  int64_t stride;
  int width;
};

Table table_of(PyObject* table_obj, PyObject* lens_obj, int64_t batch, int dev) {
  const at::Tensor& t = on(table_obj, dev, at::kInt, 2);
  const at::Tensor& l = on(lens_obj, dev, at::kInt, 1);
  usual(t.size(0) == batch && t.size(1) > 0 && t.size(1) <= INT32_MAX && (t.size(1) == 1 || t.stride(1) == 1));
  usual(l.size(0) == batch && l.is_contiguous());
  return Table{data<int32_t>(t), data<int32_t>(l), t.stride(0), static_cast<int>(t.size(1))};
}

// The attention's workspace, one per (device, stream), as _decode.py keeps for
// its own calls (threads may share a stream: a call is one launch, so theirs
// follow one another).  The caller holds it until its launch, while another
// thread may put a larger one in its place.  Under stream capture a call gets
// one from the graph's memory: not usual.
at::Tensor workspace(size_t bytes, int dev, cudaStream_t stream, const at::Tensor& like) {
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  usual(cudaStreamIsCapturing(stream, &capture) == cudaSuccess && capture == cudaStreamCaptureStatusNone);
  static auto* kept = new std::map<std::pair<int, cudaStream_t>, at::Tensor>();  // outlives the CUDA context
  at::Tensor& ws = (*kept)[{dev, stream}];
  if (!ws.defined() || static_cast<size_t>(ws.numel()) < bytes)
    ws = at::zeros({static_cast<int64_t>(bytes)}, like.options().dtype(at::kByte));
  return ws;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

template <typename F>
int without_gil(F&& f) {
  PyThreadState* state = PyEval_SaveThread();
  const int st = f();
  PyEval_RestoreThread(state);
  return st;
}

// Runs a call's body; whatever is not usual there, exceptions included, is None.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t want, F&& body) {
  if (given != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return body();
  } catch (const NotUsual&) {
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (q, k_cache, v_cache, block_table, seq_lens, k_scale, v_scale, positions, scale, return_lse)
PyObject* call_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0]);
    const int dev = current_device_of(q);
    usual(q.scalar_type() == at::kBFloat16 && q.dim() == 3 && q.layout() == at::kStrided && q.stride(2) == 1);
    const int64_t batch = q.size(0), heads = q.size(1), d = q.size(2);
    usual(heads == 1 || q.stride(1) == d);
    const topk_cache k = cache_of(a[1], a[5], dev), v = cache_of(a[2], a[6], dev);
    usual(alike(k, v) && k.d == d && k.kv_heads > 0 && heads > 0 && heads <= INT32_MAX && heads % k.kv_heads == 0);
    const Table t = table_of(a[3], a[4], batch, dev);
    const int32_t* positions = nullptr;
    int64_t lists = 0, c = 0;
    if (a[7] != Py_None) {
      const at::Tensor& p = on(a[7], dev, at::kInt, 3);
      lists = p.size(1);
      c = p.size(2);
      usual(p.is_contiguous() && p.size(0) == batch && lists > 0 && c > 0 && c <= INT32_MAX &&
            lists % k.kv_heads == 0 && heads % lists == 0);
      positions = data<int32_t>(p);
    }
    double scale;
    if (a[8] == Py_None) {
      scale = 1.0 / std::sqrt(static_cast<double>(d));
    } else {
      usual(PyFloat_Check(a[8]));
      scale = PyFloat_AS_DOUBLE(a[8]);
    }
    const int truth = PyObject_IsTrue(a[9]);
    usual(truth >= 0);
    const bool with_lse = truth != 0;
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    const at::Tensor ws = workspace(g_lib.attend_bytes(1, 1, 0, static_cast<int>(d)), dev, stream, q);
    at::Tensor out = empty_on(dev, {batch, heads, d}, at::kBFloat16);
    at::Tensor lse;
    if (with_lse) lse = empty_on(dev, {batch, heads}, at::kFloat);
    const int st = without_gil([&] {
      return g_lib.attend(data<uint16_t>(q), q.stride(0), batch, static_cast<int>(heads), &k, &v, t.table, t.stride,
                          t.width, t.lens, positions, static_cast<int>(lists), static_cast<int>(c),
                          static_cast<float>(scale), data<uint16_t>(out), with_lse ? data<float>(lse) : nullptr,
                          data<void>(ws), static_cast<size_t>(ws.numel()), stream);
    });
    if (st != TOPK_OK) return status(st);
    if (!with_lse) return THPVariable_Wrap(std::move(out));
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(out)), THPVariable_Wrap(std::move(lse)));
  });
}

// (k, v, k_cache, v_cache, slots, k_scale, v_scale) -> 0
PyObject* call_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor& k = tensor(a[0]);
    const int dev = current_device_of(k);
    on(a[0], dev, at::kBFloat16, 3);
    const at::Tensor& v = on(a[1], dev, at::kBFloat16, 3);
    const topk_cache kc = cache_of(a[2], a[5], dev), vc = cache_of(a[3], a[6], dev);
    const at::Tensor& slots = on(a[4], dev, at::kLong, 1);
    usual(alike(kc, vc) && k.sizes() == v.sizes() && k.stride(2) == 1 && v.stride(2) == 1 &&
          k.size(1) == kc.kv_heads && k.size(2) == kc.d && slots.size(0) == k.size(0) && slots.is_contiguous());
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    return status(without_gil([&] {
      return g_lib.write(data<uint16_t>(k), k.stride(0), k.stride(1), data<uint16_t>(v), v.stride(0), v.stride(1),
                         k.size(0), &kc, &vc, data<int64_t>(slots), stream);
    }));
  });
}

// (cache, block_table, seq_lens, n, scale)
PyObject* call_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor& t = tensor(a[0]);
    const int dev = current_device_of(t);
    const topk_cache c = cache_of(a[0], a[4], dev);
    const int64_t batch = tensor(a[2]).numel();
    const Table tab = table_of(a[1], a[2], batch, dev);
    usual(PyLong_Check(a[3]));
    const long long len = PyLong_AsLongLong(a[3]);
    usual(len > 0 && len <= INT32_MAX);
    at::Tensor out = empty_on(dev, {batch, c.kv_heads, len, c.d}, at::kBFloat16);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    const int st = without_gil([&] {
      return g_lib.read(&c, tab.table, tab.stride, tab.width, tab.lens, batch, len, data<uint16_t>(out), stream);
    });
    return st != TOPK_OK ? status(st) : THPVariable_Wrap(std::move(out));
  });
}

// (logits, beam_scores, k)
PyObject* call_beam(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0]);
    const int dev = current_device_of(x);
    const bool bf16 = x.scalar_type() == at::kBFloat16;
    usual((bf16 || x.scalar_type() == at::kFloat) && x.dim() == 3 && x.layout() == at::kStrided && x.is_contiguous());
    const at::Tensor& s = on(a[1], dev, at::kFloat, 2);
    const int64_t batch = x.size(0), beams = x.size(1), len = x.size(2);
    usual(s.is_contiguous() && s.size(0) == batch && s.size(1) == beams && beams <= TOPK_BEAM_MAX && PyLong_Check(a[2]));
    const long long k = PyLong_AsLongLong(a[2]);
    usual(k > 0 && k <= TOPK_BEAM_MAX);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    const size_t bytes = g_lib.beam_bytes(batch, static_cast<int>(beams), len, static_cast<int>(k));
    usual(bytes > 0);
    // Scratch of its own: between the call's launches another thread's may follow on the same stream.
    const at::Tensor ws = empty_on(dev, {static_cast<int64_t>(bytes)}, at::kByte);
    at::Tensor score = empty_on(dev, {batch, k}, at::kFloat);
    at::Tensor parent = empty_on(dev, {batch, k}, at::kInt);
    at::Tensor token = empty_on(dev, {batch, k}, at::kInt);
    const int st = without_gil([&] {
      float* o = data<float>(score);
      int32_t *p = data<int32_t>(parent), *t = data<int32_t>(token);
      void* w = data<void>(ws);
      const size_t wb = static_cast<size_t>(ws.numel());
      return bf16 ? g_lib.beam_bf16(data<uint16_t>(x), data<float>(s), batch, static_cast<int>(beams), len,
                                    static_cast<int>(k), o, p, t, w, wb, stream)
                  : g_lib.beam(data<float>(x), data<float>(s), batch, static_cast<int>(beams), len, static_cast<int>(k),
                               o, p, t, w, wb, stream);
    });
    if (st != TOPK_OK) return status(st);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(score)), THPVariable_Wrap(std::move(parent)),
                         THPVariable_Wrap(std::move(token)));
  });
}

// (states: list or tuple of tensors, parents) -> list
PyObject* call_reorder(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    const at::Tensor& parents = tensor(a[1]);
    const int dev = current_device_of(parents);
    on(a[1], dev, at::kInt, 2);
    usual(parents.is_contiguous() && (PyList_Check(a[0]) || PyTuple_Check(a[0])));
    const Py_ssize_t m = PySequence_Fast_GET_SIZE(a[0]);
    usual(m > 0 && m <= 256);
    PyObject** items = PySequence_Fast_ITEMS(a[0]);
    const int64_t batch = parents.size(0), k = parents.size(1);
    std::vector<const void*> src(m);
    std::vector<void*> dst(m);
    std::vector<int64_t> bytes(m), shape;
    std::vector<at::Tensor> out(m);
    int64_t beams = 0;
    for (Py_ssize_t i = 0; i < m; ++i) {
      const at::Tensor& t = tensor(items[i]);
      usual(t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided && t.dim() >= 2 && t.is_contiguous() &&
            !t.is_conj() && !t.is_neg() && t.numel() > 0 && t.size(0) == batch && (i == 0 || t.size(1) == beams) && t.size(1) <= INT32_MAX);
      beams = t.size(1);
      shape.assign(t.sizes().begin(), t.sizes().end());
      shape[1] = k;
      out[i] = empty_on(dev, shape, t.scalar_type());
      src[i] = t.const_data_ptr();
      dst[i] = data<void>(out[i]);
      bytes[i] = t.numel() / (batch * beams) * t.element_size();
    }
    usual(k > 0 && k <= INT32_MAX);
    const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    const int st = without_gil([&] {
      return g_lib.reorder(src.data(), dst.data(), bytes.data(), static_cast<int>(m), batch, static_cast<int>(beams),
                           static_cast<int>(k), data<int32_t>(parents), stream);
    });
    if (st != TOPK_OK) return status(st);
    PyObject* list = PyList_New(m);
    if (!list) return nullptr;
    for (Py_ssize_t i = 0; i < m; ++i) PyList_SET_ITEM(list, i, THPVariable_Wrap(std::move(out[i])));
    return list;
  });
}

// bind(address, ...): the library's entry points in the order of Entries.
PyObject* call_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_lib.attend = reinterpret_cast<decltype(g_lib.attend)>(p[0]);
  g_lib.attend_bytes = reinterpret_cast<decltype(g_lib.attend_bytes)>(p[1]);
  g_lib.write = reinterpret_cast<decltype(g_lib.write)>(p[2]);
  g_lib.read = reinterpret_cast<decltype(g_lib.read)>(p[3]);
  g_lib.beam = reinterpret_cast<decltype(g_lib.beam)>(p[4]);
  g_lib.beam_bf16 = reinterpret_cast<decltype(g_lib.beam_bf16)>(p[5]);
  g_lib.beam_bytes = reinterpret_cast<decltype(g_lib.beam_bytes)>(p[6]);
  g_lib.reorder = reinterpret_cast<decltype(g_lib.reorder)>(p[7]);
  Py_RETURN_NONE;
}

PyMethodDef g_methods[7] = {};  // filled at import, the last one empty

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_decode_calls", "Usual calls of the decoding step's operators.", -1,
                        g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode_calls() {
  auto fast = [](PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
  };
  g_methods[0] = {"bind", fast(call_bind), METH_FASTCALL, "Entry points of the CUDA library."};
  g_methods[1] = {"paged_attention", fast(call_attention), METH_FASTCALL, nullptr};
  g_methods[2] = {"cache_write", fast(call_write), METH_FASTCALL, nullptr};
  g_methods[3] = {"cache_read", fast(call_read), METH_FASTCALL, nullptr};
  g_methods[4] = {"topk_beam", fast(call_beam), METH_FASTCALL, nullptr};
  g_methods[5] = {"beam_reorder", fast(call_reorder), METH_FASTCALL, nullptr};
  return PyModule_Create(&g_module);
}
