// Argument marshalling of the operators around the layer and of those over the paged cache for Python (module
// _marshal).
//
// These calls come several times per layer on batches down to one token, where the host's time is
// the call's time.  Tensors are looked at through PyTorch's C++ interface instead of attribute by
// attribute in Python, which takes the Python side of a call from 5-9 us to about 2.  Nothing is
// computed here: shapes, types, devices and strides are checked (ValueError names the argument and
// what it was), results that the caller does not bring are allocated, and the C ABI is called with
// raw pointers and the stream.  A nonzero status of the C call is returned as an int, which the
// Python side turns into its exception.
#include "../../include/moe_lora.h"

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <sstream>
#include <string>

namespace {

using at::ScalarType;
using at::Tensor;

// The C ABI's entry points, handed over by the Python side from the library that it has loaded.
decltype(&moe_lora_select_experts) g_select = nullptr;
decltype(&moe_lora_linear) g_linear = nullptr;
decltype(&moe_lora_linear_workspace_size) g_linear_workspace = nullptr;
decltype(&moe_lora_qk_norm_rope) g_qk = nullptr;
decltype(&moe_lora_device) g_device = nullptr;
decltype(&moe_lora_page_tables) g_page_tables = nullptr;
decltype(&moe_lora_cache_write) g_cache_write = nullptr;
decltype(&moe_lora_attention) g_attention = nullptr;
decltype(&moe_lora_attention_workspace_size) g_attention_workspace = nullptr;

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(const std::string& msg) {
  PyErr_SetString(PyExc_ValueError, msg.c_str());
  throw Refused();
}
[[noreturn]] void refuse(const Tensor& t, const char* name, const std::string& want) {
  std::ostringstream s;
  s << name << " must be " << want << ", got " << t.scalar_type() << " " << t.sizes() << " strides " << t.strides()
    << " on " << t.device();
  refuse(s.str());
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int int32(PyObject* o) {
  const long v = integer(o);
  if (v != static_cast<int>(v)) refuse("an integer argument does not fit 32 bits");
  return static_cast<int>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}
int size(int64_t v, const char* name) {
  if (v > 0x7fffffff) refuse(std::string(name) + " has a dimension past 2^31");
  return static_cast<int>(v);
}

std::string on(const at::Device& d) { return " on " + d.str(); }

const void* dense_vector(const Tensor& t, int64_t n, at::Device dev, const char* name) {
  if (t.dim() != 1 || t.size(0) != n || t.device() != dev || !t.is_contiguous())
    refuse(t, name, "a dense [" + std::to_string(n) + "] tensor" + on(dev));
  return t.data_ptr();
}
const void* vector_of(PyObject* o, ScalarType type, int64_t n, at::Device dev, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type) refuse(t, name, std::string("of type ") + c10::toString(type));
  return dense_vector(t, n, dev, name);
}
void* dense_out(const Tensor& t, int64_t rows, int64_t cols, ScalarType type, at::Device dev, const char* name) {
  if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.device() != dev ||
      !t.is_contiguous())
    refuse(t, name, std::string("a contiguous ") + c10::toString(type) + " [" + std::to_string(rows) + ", " +
                        std::to_string(cols) + "] tensor" + on(dev));
  return t.data_ptr();
}
// [rows, cols] with adjacent columns; the row stride
int64_t rows_of(const Tensor& t, const char* name) {
  if (t.size(1) > 1 && t.stride(1) != 1) refuse(t, name, "a tensor with adjacent columns");
  return t.stride(0);
}
moe_lora_stream stream_of(PyObject* o, at::Device dev) {
  if (o == Py_None) return reinterpret_cast<moe_lora_stream>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Refused();
  return static_cast<moe_lora_stream>(p);
}
// The handle of a call on tensors of `dev` (null: a closed one, which the C call refuses).
moe_lora_handle* handle_of(PyObject* o, at::Device dev) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Refused();
  moe_lora_handle* h = static_cast<moe_lora_handle*>(p);
  int own = 0;
  if (g_device(h, &own) == MOE_LORA_OK && own != dev.index())
    refuse("the tensors are" + on(dev) + ", the handle is on cuda:" + std::to_string(own));
  return h;
}
// Memory for a call on `stream` (None: the current one) comes from that stream's: whatever the block held
// before was used there, so the call's kernels cannot run into it.
// (at::empty would come to the same through PyTorch's dispatcher)
Tensor allocate(at::IntArrayRef sizes, ScalarType type, at::Device dev, PyObject* stream) {
  if (stream == Py_None) return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
  const c10::cuda::CUDAStreamGuard on_it(
      c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(PyLong_AsVoidPtr(stream)), dev.index()));
  return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}
// A result of such a call goes to a caller on the current stream, whose uses a reuse of its memory waits for.
void handed_over(const Tensor& t, PyObject* stream, at::Device dev) {
  if (stream != Py_None && t.defined()) t.record_stream(c10::cuda::getCurrentCUDAStream(dev.index()).unwrap());
}

// A call's small results come from one allocation (select, two results: 3.9 -> 3.55 us of the host; results
// past 1 MB in all have their own, so that keeping one does not keep the others' memory).
struct Results {
  static constexpr int64_t kTogether = 1 << 20;
  at::Device dev;
  PyObject* stream;
  int64_t bytes = 0, at = 0;
  Tensor block;
  Results(at::Device d, PyObject* s) : dev(d), stream(s) {}
  static int64_t size_of(at::IntArrayRef sizes, ScalarType type) {
    int64_t n = static_cast<int64_t>(c10::elementSize(type));
    for (int64_t s : sizes) n *= s;
    return (n + 255) / 256 * 256;
  }
  void expect(at::IntArrayRef sizes, ScalarType type) { bytes += size_of(sizes, type); }   // each, first
  Tensor make(at::IntArrayRef sizes, ScalarType type) {
    if (bytes > kTogether) return allocate(sizes, type, dev, stream);
    if (!block.defined()) block = allocate({bytes}, ScalarType::Byte, dev, stream);
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(),
                                                        c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    at += size_of(sizes, type);
    return t;
  }
};

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
    throw Refused();
  }
}

// Runs f, turning C++ exceptions into Python ones.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* kIds;
PyObject* kWeights;
PyObject* kPacked;

// (handle, logits, top_k, scoring, bias, n_group, topk_group, group_score, renormalize, factor, packed, outputs, stream)
PyObject* select_experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 13);
    const Tensor& z = tensor(a[1], "logits");
    const ScalarType type = z.scalar_type();
    if (z.dim() != 2 || !z.is_cuda() || (type != ScalarType::Float && type != ScalarType::BFloat16))
      refuse(z, "logits", "a bf16 or float32 CUDA tensor [T, E]");
    const at::Device dev = z.device();
    moe_lora_handle* h = handle_of(a[0], dev);
    const int64_t T = z.size(0), E = z.size(1), row = rows_of(z, "logits");
    moe_lora_select_args p;
    p.logits = z.data_ptr();
    p.logits_stride = T > 1 ? row : E;
    p.T = size(T, "logits");
    p.E = size(E, "logits");
    p.top_k = int32(a[2]);
    p.logits_f32 = type == ScalarType::Float;
    p.scoring = int32(a[3]);
    p.bias = a[4] == Py_None ? nullptr : static_cast<const float*>(vector_of(a[4], ScalarType::Float, E, dev, "bias"));
    p.n_group = int32(a[5]);
    p.topk_group = int32(a[6]);
    p.group_score = int32(a[7]);
    p.renormalize = truth(a[8]);
    p.routed_scaling_factor = static_cast<float>(number(a[9]));
    const bool packed = truth(a[10]);
    if (p.top_k < 1 || p.top_k > E) return PyLong_FromLong(MOE_LORA_ERR_INVALID_ARG);   // before [T, top_k] is allocated
    const int64_t k = p.top_k;
    PyObject* o = a[11];
    const bool given = o != Py_None;
    if (given && !PyDict_Check(o)) refuse("outputs must be a dict");
    if (given) Py_INCREF(o);
    else if ((o = PyDict_New()) == nullptr) throw Refused();
    auto brought = [&](PyObject* key) -> PyObject* {
      PyObject* have = given ? PyDict_GetItem(o, key) : nullptr;
      return have == Py_None ? nullptr : have;
    };
    Results results(dev, a[12]);
    if (brought(kIds) == nullptr) results.expect({T, k}, ScalarType::Int);
    if (brought(kWeights) == nullptr) results.expect({T, k}, ScalarType::Float);
    if (packed && brought(kPacked) == nullptr) results.expect({T, k}, ScalarType::Int);
    auto output = [&](PyObject* key, ScalarType t, const char* name, bool wanted) -> void* {
      if (PyObject* have = brought(key)) return dense_out(tensor(have, name), T, k, t, dev, name);
      if (!wanted) return nullptr;
      Tensor made = results.make({T, k}, t);
      void* at = made.data_ptr();
      handed_over(made, a[12], dev);
      PyObject* w = THPVariable_Wrap(std::move(made));
      if (w == nullptr) throw Refused();
      const int bad = PyDict_SetItem(o, key, w);
      Py_DECREF(w);
      if (bad) throw Refused();
      return at;
    };
    int st;
    try {
      p.topk_ids = static_cast<int32_t*>(output(kIds, ScalarType::Int, "topk_ids", true));
      p.topk_weights = static_cast<float*>(output(kWeights, ScalarType::Float, "topk_weights", true));
      p.packed_topk_ids = static_cast<int32_t*>(output(kPacked, ScalarType::Int, "packed_topk_ids", packed));
      st = g_select(h, &p, stream_of(a[12], dev));
    } catch (...) {
      Py_DECREF(o);
      throw;
    }
    if (st != 0) {
      Py_DECREF(o);
      return PyLong_FromLong(st);
    }
    return o;
  });
}

// The adapters of a projection, as moe_lora_linear_adapters stacked them (a capsule).  Callers never see the
// stack's tensor, so calls on other streams than its own are recorded on it here.
struct Adapters {
  int S = 0, N = 0, K = 0, device = 0;
  Tensor packed;
  cudaStream_t stream = nullptr;   // whose memory it is
  const void* address = nullptr;
  int32_t ranks[64] = {};
  float scalings[64] = {};
};
constexpr const char* kAdapters = "moe_lora.adapters";

// (packed, S, N, K, ranks, scalings, stream that packed is the memory of)
PyObject* adapters(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 7);
    const Tensor& t = tensor(a[0], "packed");
    Adapters* d = new Adapters();
    try {
      d->S = int32(a[1]);
      d->N = int32(a[2]);
      d->K = int32(a[3]);
      d->device = t.device().index();
      d->packed = t;
      d->stream = reinterpret_cast<cudaStream_t>(stream_of(a[6], t.device()));
      d->address = t.data_ptr();
      if (d->S < 1 || d->S > 64 || !PyList_Check(a[4]) || !PyList_Check(a[5]) || PyList_Size(a[4]) != d->S ||
          PyList_Size(a[5]) != d->S)
        refuse("ranks and scalings must be lists of S <= 64 values");
      for (int s = 0; s < d->S; ++s) {
        d->ranks[s] = int32(PyList_GetItem(a[4], s));
        d->scalings[s] = static_cast<float>(number(PyList_GetItem(a[5], s)));
      }
    } catch (...) {
      delete d;
      throw;
    }
    PyObject* c = PyCapsule_New(d, kAdapters, [](PyObject* o) {
      delete static_cast<Adapters*>(PyCapsule_GetPointer(o, kAdapters));
    });
    if (c == nullptr) delete d;
    return c;
  });
}

// (handle, x, w, adapters or None, slot_idx, bias, out, out is float32, workspace, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 10);
    const Tensor& x = tensor(a[1], "x");
    if (x.dim() != 2 || !x.is_cuda() || x.scalar_type() != ScalarType::BFloat16)
      refuse(x, "x", "a bf16 CUDA tensor [T, K]");
    const at::Device dev = x.device();
    moe_lora_handle* h = handle_of(a[0], dev);
    const int64_t T = x.size(0), K = x.size(1);
    const Tensor& w = tensor(a[2], "w");
    if (w.dim() != 2 || w.scalar_type() != ScalarType::BFloat16 || w.device() != dev || w.size(1) != K)
      refuse(w, "w", "a bf16 [N, " + std::to_string(K) + "] tensor" + on(dev));
    const int64_t N = w.size(0);
    moe_lora_linear_args p;
    p.x = static_cast<const moe_lora_bf16*>(x.data_ptr());
    p.w = static_cast<const moe_lora_bf16*>(w.data_ptr());
    p.x_stride = rows_of(x, "x");
    p.w_stride = rows_of(w, "w");
    p.T = size(T, "x");
    p.N = size(N, "w");
    p.K = size(K, "x");
    p.bias = a[5] == Py_None ? nullptr : static_cast<const float*>(vector_of(a[5], ScalarType::Float, N, dev, "bias"));
    p.S = 0;
    p.adapters = nullptr;
    p.slot_idx = nullptr;
    p.h_ranks = nullptr;
    p.h_scalings = nullptr;
    const Adapters* used = nullptr;
    if (a[3] != Py_None) {
      const Adapters* d = used = static_cast<const Adapters*>(PyCapsule_GetPointer(a[3], kAdapters));
      if (d == nullptr) throw Refused();
      if (d->N != N || d->K != K || d->device != dev.index())
        refuse("the adapters are for a [" + std::to_string(d->N) + ", " + std::to_string(d->K) + "] projection on cuda:" +
               std::to_string(d->device) + ", w is [" + std::to_string(N) + ", " + std::to_string(K) + "]" + on(dev));
      if (a[4] == Py_None) refuse("slot_idx [T] is required with adapters");
      p.S = d->S;
      p.adapters = d->address;
      p.h_ranks = d->ranks;
      p.h_scalings = d->scalings;
      p.slot_idx = static_cast<const int32_t*>(vector_of(a[4], ScalarType::Int, T, dev, "slot_idx"));
    }
    Tensor made;
    const Tensor* out;
    if (a[6] == Py_None) {
      made = allocate({T, N}, truth(a[7]) ? ScalarType::Float : ScalarType::BFloat16, dev, a[9]);
      out = &made;
      p.y_stride = N;
    } else {
      out = &tensor(a[6], "out");
      if ((out->scalar_type() != ScalarType::BFloat16 && out->scalar_type() != ScalarType::Float) || out->dim() != 2 ||
          out->size(0) != T || out->size(1) != N || out->device() != dev)
        refuse(*out, "out", "a bf16 or float32 [" + std::to_string(T) + ", " + std::to_string(N) + "] tensor" + on(dev));
      p.y_stride = rows_of(*out, "out");
    }
    p.y = out->data_ptr();
    p.y_f32 = out->scalar_type() == ScalarType::Float;
    Tensor scratch;
    const Tensor* ws;
    if (a[8] == Py_None) {
      size_t bytes = 0;
      const int st = g_linear_workspace(p.T, p.S, p.h_ranks, &bytes);
      if (st != 0) return PyLong_FromLong(st);
      scratch = allocate({static_cast<int64_t>(bytes)}, ScalarType::Byte, dev, a[9]);
      ws = &scratch;
    } else {
      ws = &tensor(a[8], "workspace");
      if (ws->scalar_type() != ScalarType::Byte || ws->device() != dev || !ws->is_contiguous())
        refuse(*ws, "workspace", "a contiguous uint8 tensor" + on(dev));
    }
    handed_over(made, a[9], dev);
    const moe_lora_stream stream = stream_of(a[9], dev);
    if (used != nullptr && stream != used->stream)
      used->packed.record_stream(c10::cuda::getStreamFromExternal(stream, dev.index()).unwrap());
    const int st = g_linear(h, &p, ws->data_ptr(), static_cast<size_t>(ws->numel()), stream);
    if (st != 0) return PyLong_FromLong(st);
    if (a[6] == Py_None) return THPVariable_Wrap(std::move(made));
    Py_INCREF(a[6]);
    return a[6];
  });
}

// [T, H, D] heads with adjacent values
const Tensor& heads(PyObject* o, int64_t T, int64_t H, int64_t D, at::Device dev, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != ScalarType::BFloat16 || t.dim() != 3 || t.size(0) != T || (H >= 0 && t.size(1) != H) ||
      t.size(2) != D || t.device() != dev || (D > 1 && t.stride(2) != 1))
    refuse(t, name, "a bf16 [" + std::to_string(T) + ", heads, " + std::to_string(D) + "] tensor with adjacent head values" +
                        on(dev));
  return t;
}

// (handle, q, k, q_weight, k_weight, cos_sin, positions, eps, interleaved, q_out, k_out, workspace, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 13);
    const Tensor& q = tensor(a[1], "q");
    if (q.dim() != 3 || !q.is_cuda()) refuse(q, "q", "a bf16 CUDA tensor [T, heads, D]");
    const at::Device dev = q.device();
    moe_lora_handle* h = handle_of(a[0], dev);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    heads(a[1], T, Hq, D, dev, "q");
    const Tensor& k = heads(a[2], T, -1, D, dev, "k");
    const int64_t Hk = k.size(1);
    const Tensor& table = tensor(a[5], "cos_sin");
    if (table.dim() != 2 || table.scalar_type() != ScalarType::Float || table.device() != dev)
      refuse(table, "cos_sin", "a float32 [positions, R] tensor" + on(dev));
    const Tensor& wq = tensor(a[3], "q_weight");
    const ScalarType wt = wq.scalar_type();
    if (wt != ScalarType::BFloat16 && wt != ScalarType::Float) refuse(wq, "q_weight", "bf16 or float32");
    const Tensor& pos = tensor(a[6], "positions");
    const ScalarType pt = pos.scalar_type();
    if (pt != ScalarType::Int && pt != ScalarType::Long) refuse(pos, "positions", "int32 or int64");
    moe_lora_qk_args p;
    p.q = static_cast<const moe_lora_bf16*>(q.data_ptr());
    p.k = static_cast<const moe_lora_bf16*>(k.data_ptr());
    p.q_stride_t = q.stride(0);
    p.q_stride_h = q.stride(1);
    p.k_stride_t = k.stride(0);
    p.k_stride_h = k.stride(1);
    p.q_weight = dense_vector(wq, D, dev, "q_weight");
    p.k_weight = vector_of(a[4], wt, D, dev, "k_weight");
    p.cos_sin = static_cast<const float*>(table.data_ptr());
    p.cos_sin_stride = rows_of(table, "cos_sin");
    p.positions = dense_vector(pos, T, dev, "positions");
    p.T = size(T, "q");
    p.q_heads = size(Hq, "q");
    p.k_heads = size(Hk, "k");
    p.head_dim = size(D, "q");
    p.rotary_dim = size(table.size(1), "cos_sin");
    p.num_positions = size(table.size(0), "cos_sin");
    p.weight_f32 = wt == ScalarType::Float;
    p.positions_i64 = pt == ScalarType::Long;
    p.eps = static_cast<float>(number(a[7]));
    p.interleaved = truth(a[8]);
    Tensor made[2];
    Results results(dev, a[12]);
    if (a[9] == Py_None) results.expect({T, Hq, D}, ScalarType::BFloat16);
    if (a[10] == Py_None) results.expect({T, Hk, D}, ScalarType::BFloat16);
    auto output = [&](PyObject* o, int64_t H, Tensor& mine, const char* name, moe_lora_bf16*& at, int64_t& st, int64_t& sh) {
      if (o == Py_None) mine = results.make({T, H, D}, ScalarType::BFloat16);
      const Tensor& t = o == Py_None ? mine : heads(o, T, H, D, dev, name);
      at = static_cast<moe_lora_bf16*>(t.data_ptr());
      st = t.stride(0);
      sh = t.stride(1);
    };
    output(a[9], Hq, made[0], "q_out", p.q_out, p.q_out_stride_t, p.q_out_stride_h);
    output(a[10], Hk, made[1], "k_out", p.k_out, p.k_out_stride_t, p.k_out_stride_h);
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[11] != Py_None) {
      const Tensor& t = tensor(a[11], "workspace");
      if (t.scalar_type() != ScalarType::Byte || t.device() != dev || !t.is_contiguous())
        refuse(t, "workspace", "a contiguous uint8 tensor" + on(dev));
      ws = t.data_ptr();
      ws_bytes = static_cast<size_t>(t.numel());
    }
    for (const Tensor& t : made) handed_over(t, a[12], dev);
    const int st = g_qk(h, &p, ws, ws_bytes, stream_of(a[12], dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) throw Refused();
    for (int i = 0; i < 2; ++i) {
      PyObject* o = a[9 + i];
      if (o == Py_None) o = THPVariable_Wrap(std::move(made[i]));
      else Py_INCREF(o);
      if (o == nullptr) {
        Py_DECREF(r);
        throw Refused();
      }
      PyTuple_SET_ITEM(r, i, o);
    }
    return r;
  });
}

// An optional status word, or more, of the caller's.
void* workspace_of(PyObject* o, at::Device dev, size_t& bytes) {
  bytes = 0;
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "workspace");
  if (t.scalar_type() != ScalarType::Byte || t.device() != dev || !t.is_contiguous())
    refuse(t, "workspace", "a contiguous uint8 tensor" + on(dev));
  bytes = static_cast<size_t>(t.numel());
  return t.data_ptr();
}
const int32_t* lengths(PyObject* o, int64_t n, at::Device dev, const char* name) {
  return static_cast<const int32_t*>(vector_of(o, ScalarType::Int, n, dev, name));
}
// [B, width] int32 rows
const Tensor& block_tables(PyObject* o) {
  const Tensor& t = tensor(o, "block_tables");
  if (t.dim() != 2 || !t.is_cuda() || t.scalar_type() != ScalarType::Int) refuse(t, "block_tables", "an int32 CUDA tensor [B, width]");
  rows_of(t, "block_tables");
  return t;
}
// [pages, heads, page size, D] with adjacent head values
const Tensor& cache_of(PyObject* o, int64_t heads, int64_t D, at::Device dev, const Tensor* like, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != ScalarType::BFloat16 || t.dim() != 4 || (heads >= 0 && t.size(1) != heads) || t.size(3) != D ||
      t.device() != dev || (D > 1 && t.stride(3) != 1) || (like != nullptr && t.sizes() != like->sizes()))
    refuse(t, name, "a bf16 [pages, heads, page size, " + std::to_string(D) + "] tensor with adjacent head values" + on(dev) +
                        (like != nullptr ? ", of the sizes of k_cache" : ""));
  return t;
}

PyObject* kKvLens;
PyObject* kQueryOffsets;
PyObject* kSlotMap;
PyObject* kPositions;
PyObject* kTaken;

// (handle, block_tables, cached_lens, new_lens, page_size, free_pages, taken, num_tokens, outputs, workspace, stream)
PyObject* page_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 11);
    const Tensor& table = block_tables(a[1]);
    const at::Device dev = table.device();
    moe_lora_handle* h = handle_of(a[0], dev);
    const int64_t B = table.size(0);
    moe_lora_page_tables_args p;
    p.block_tables = static_cast<int32_t*>(table.data_ptr());
    p.table_stride = B > 1 ? table.stride(0) : table.size(1);
    p.B = size(B, "block_tables");
    p.table_width = size(table.size(1), "block_tables");
    p.cached_lens = lengths(a[2], B, dev, "cached_lens");
    p.new_lens = lengths(a[3], B, dev, "new_lens");
    p.page_size = int32(a[4]);
    const Tensor& free_pages = tensor(a[5], "free_pages");
    if (free_pages.dim() != 1) refuse(free_pages, "free_pages", "a dense int32 vector" + on(dev));
    p.num_free = size(free_pages.size(0), "free_pages");
    p.free_pages = lengths(a[5], p.num_free, dev, "free_pages");
    p.taken = lengths(a[6], 1, dev, "taken");
    p.T = int32(a[7]);
    if (p.T < 0) return PyLong_FromLong(MOE_LORA_ERR_INVALID_ARG);
    PyObject* o = a[8];
    const bool given = o != Py_None;
    if (given && !PyDict_Check(o)) refuse("outputs must be a dict");
    if (given) Py_INCREF(o);
    else if ((o = PyDict_New()) == nullptr) throw Refused();
    int st;
    try {
      const struct {
        PyObject* key;
        const char* name;
        int64_t n;
        int32_t** at;
      } outs[5] = {{kKvLens, "kv_lens", B, &p.kv_lens},
                   {kQueryOffsets, "query_offsets", B + 1, &p.query_offsets},
                   {kSlotMap, "slot_map", p.T, &p.slot_map},
                   {kPositions, "positions", p.T, &p.positions},
                   {kTaken, "taken", 1, &p.taken_out}};
      Results results(dev, a[10]);
      bool have[5];
      for (int i = 0; i < 5; ++i) {
        PyObject* v = given ? PyDict_GetItem(o, outs[i].key) : nullptr;
        have[i] = v != nullptr && v != Py_None;
        if (have[i]) *outs[i].at = const_cast<int32_t*>(lengths(v, outs[i].n, dev, outs[i].name));
        else results.expect({outs[i].n}, ScalarType::Int);
      }
      for (int i = 0; i < 5; ++i) {
        if (have[i]) continue;
        Tensor made = results.make({outs[i].n}, ScalarType::Int);
        *outs[i].at = static_cast<int32_t*>(made.data_ptr());
        handed_over(made, a[10], dev);
        PyObject* w = THPVariable_Wrap(std::move(made));
        if (w == nullptr) throw Refused();
        const int bad = PyDict_SetItem(o, outs[i].key, w);
        Py_DECREF(w);
        if (bad) throw Refused();
      }
      size_t bytes;
      void* ws = workspace_of(a[9], dev, bytes);
      st = g_page_tables(h, &p, ws, bytes, stream_of(a[10], dev));
    } catch (...) {
      Py_DECREF(o);
      throw;
    }
    if (st != 0) {
      Py_DECREF(o);
      return PyLong_FromLong(st);
    }
    return o;
  });
}

// (handle, k, v, k_cache, v_cache, slot_map, workspace, stream)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 8);
    const Tensor& k = tensor(a[1], "k");
    if (k.dim() != 3 || !k.is_cuda()) refuse(k, "k", "a bf16 CUDA tensor [T, heads, D]");
    const at::Device dev = k.device();
    moe_lora_handle* h = handle_of(a[0], dev);
    const int64_t T = k.size(0), H = k.size(1), D = k.size(2);
    heads(a[1], T, H, D, dev, "k");
    const Tensor& v = heads(a[2], T, H, D, dev, "v");
    const Tensor& kc = cache_of(a[3], H, D, dev, nullptr, "k_cache");
    const Tensor& vc = cache_of(a[4], H, D, dev, &kc, "v_cache");
    moe_lora_cache_write_args p;
    p.k = static_cast<const moe_lora_bf16*>(k.data_ptr());
    p.v = static_cast<const moe_lora_bf16*>(v.data_ptr());
    p.k_cache = static_cast<moe_lora_bf16*>(kc.data_ptr());
    p.v_cache = static_cast<moe_lora_bf16*>(vc.data_ptr());
    p.slot_map = lengths(a[5], T, dev, "slot_map");
    p.k_stride_t = k.stride(0);
    p.k_stride_h = k.stride(1);
    p.v_stride_t = v.stride(0);
    p.v_stride_h = v.stride(1);
    p.k_stride_page = kc.stride(0);
    p.k_stride_head = kc.stride(1);
    p.k_stride_token = kc.stride(2);
    p.v_stride_page = vc.stride(0);
    p.v_stride_head = vc.stride(1);
    p.v_stride_token = vc.stride(2);
    p.T = size(T, "k");
    p.heads = size(H, "k");
    p.head_dim = size(D, "k");
    p.num_pages = size(kc.size(0), "k_cache");
    p.page_size = size(kc.size(2), "k_cache");
    size_t bytes;
    void* ws = workspace_of(a[6], dev, bytes);
    return PyLong_FromLong(g_cache_write(h, &p, ws, bytes, stream_of(a[7], dev)));
  });
}

// (handle, q, k_cache, v_cache, block_tables, kv_lens, query_offsets, max_query_len, scale, shared_len, out, lse or
//  whether it is wanted, workspace, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 14);
    const Tensor& q = tensor(a[1], "q");
    if (q.dim() != 3 || !q.is_cuda()) refuse(q, "q", "a bf16 CUDA tensor [T, heads, D]");
    const at::Device dev = q.device();
    moe_lora_handle* h = handle_of(a[0], dev);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    heads(a[1], T, Hq, D, dev, "q");
    const Tensor& kc = cache_of(a[2], -1, D, dev, nullptr, "k_cache");
    const Tensor& vc = cache_of(a[3], -1, D, dev, &kc, "v_cache");
    const Tensor& table = block_tables(a[4]);
    if (table.device() != dev) refuse(table, "block_tables", "a tensor" + on(dev));
    const int64_t B = table.size(0);
    moe_lora_attention_args p;
    p.q = static_cast<const moe_lora_bf16*>(q.data_ptr());
    p.k_cache = static_cast<const moe_lora_bf16*>(kc.data_ptr());
    p.v_cache = static_cast<const moe_lora_bf16*>(vc.data_ptr());
    p.block_tables = static_cast<const int32_t*>(table.data_ptr());
    p.table_stride = B > 1 ? table.stride(0) : table.size(1);
    p.kv_lens = lengths(a[5], B, dev, "kv_lens");
    if (a[6] == Py_None && T != B)
      refuse("without query_offsets q has a row for each of the " + std::to_string(B) + " requests, got " + std::to_string(T));
    p.query_offsets = a[6] == Py_None ? nullptr : lengths(a[6], B + 1, dev, "query_offsets");
    p.T = size(T, "q");
    p.B = size(B, "block_tables");
    p.q_heads = size(Hq, "q");
    p.k_heads = size(kc.size(1), "k_cache");
    if (p.k_heads < 1 || p.q_heads % p.k_heads != 0)
      refuse("the heads of q, " + std::to_string(Hq) + ", must be a multiple of those of k_cache, " + std::to_string(p.k_heads));
    p.head_dim = size(D, "q");
    p.num_pages = size(kc.size(0), "k_cache");
    p.page_size = size(kc.size(2), "k_cache");
    p.table_width = size(table.size(1), "block_tables");
    p.max_query_len = a[7] == Py_None ? (a[6] == Py_None ? 1 : p.T) : int32(a[7]);
    p.scale = a[8] == Py_None ? 1.0f / std::sqrt(static_cast<float>(D)) : static_cast<float>(number(a[8]));
    p.shared_len = int32(a[9]);
    p.q_stride_t = q.stride(0);
    p.q_stride_h = q.stride(1);
    p.k_stride_page = kc.stride(0);
    p.k_stride_head = kc.stride(1);
    p.k_stride_token = kc.stride(2);
    p.v_stride_page = vc.stride(0);
    p.v_stride_head = vc.stride(1);
    p.v_stride_token = vc.stride(2);
    const bool lse_given = THPVariable_Check(a[11]), with_lse = lse_given || truth(a[11]);
    Tensor made[2];
    Results results(dev, a[13]);
    if (a[10] == Py_None) results.expect({T, Hq, D}, ScalarType::BFloat16);
    if (with_lse && !lse_given) results.expect({T, Hq}, ScalarType::Float);
    if (a[10] == Py_None) made[0] = results.make({T, Hq, D}, ScalarType::BFloat16);
    const Tensor& out = a[10] == Py_None ? made[0] : heads(a[10], T, Hq, D, dev, "out");
    p.out = static_cast<moe_lora_bf16*>(out.data_ptr());
    p.out_stride_t = out.stride(0);
    p.out_stride_h = out.stride(1);
    p.lse = nullptr;
    if (lse_given) {
      p.lse = static_cast<float*>(dense_out(tensor(a[11], "lse"), T, Hq, ScalarType::Float, dev, "lse"));
    } else if (with_lse) {
      made[1] = results.make({T, Hq}, ScalarType::Float);
      p.lse = static_cast<float*>(made[1].data_ptr());
    }
    size_t bytes;
    void* ws = workspace_of(a[12], dev, bytes);
    Tensor scratch;
    if (ws == nullptr) {
      const int st = g_attention_workspace(p.T, p.q_heads, p.k_heads, p.head_dim, &bytes);
      if (st != 0) return PyLong_FromLong(st);
      scratch = allocate({static_cast<int64_t>(bytes)}, ScalarType::Byte, dev, a[13]);
      ws = scratch.data_ptr();
    }
    for (const Tensor& t : made) handed_over(t, a[13], dev);
    const int st = g_attention(h, &p, ws, bytes, stream_of(a[13], dev));
    if (st != 0) return PyLong_FromLong(st);
    PyObject* o = a[10];
    if (o == Py_None) {
      if ((o = THPVariable_Wrap(std::move(made[0]))) == nullptr) throw Refused();
    } else {
      Py_INCREF(o);
    }
    if (!with_lse) return o;
    PyObject* e = a[11];
    if (lse_given) Py_INCREF(e);
    else if ((e = THPVariable_Wrap(std::move(made[1]))) == nullptr) {
      Py_DECREF(o);
      throw Refused();
    }
    PyObject* r = PyTuple_Pack(2, o, e);
    Py_DECREF(o);
    Py_DECREF(e);
    if (r == nullptr) throw Refused();
    return r;
  });
}

// (addresses of select_experts, linear, linear_workspace_size, qk_norm_rope, device, page_tables, cache_write,
//  attention, attention_workspace_size)
PyObject* entry_points(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 9);
    void* at[9];
    for (int i = 0; i < 9; ++i)
      if ((at[i] = PyLong_AsVoidPtr(a[i])) == nullptr) refuse("an entry point is missing");
    g_select = reinterpret_cast<decltype(g_select)>(at[0]);
    g_linear = reinterpret_cast<decltype(g_linear)>(at[1]);
    g_linear_workspace = reinterpret_cast<decltype(g_linear_workspace)>(at[2]);
    g_qk = reinterpret_cast<decltype(g_qk)>(at[3]);
    g_device = reinterpret_cast<decltype(g_device)>(at[4]);
    g_page_tables = reinterpret_cast<decltype(g_page_tables)>(at[5]);
    g_cache_write = reinterpret_cast<decltype(g_cache_write)>(at[6]);
    g_attention = reinterpret_cast<decltype(g_attention)>(at[7]);
    g_attention_workspace = reinterpret_cast<decltype(g_attention_workspace)>(at[8]);
    Py_RETURN_NONE;
  });
}

#define ML_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ML_METHOD(select_experts), ML_METHOD(adapters),     ML_METHOD(linear),
                          ML_METHOD(qk_norm_rope),   ML_METHOD(page_tables),  ML_METHOD(cache_write),
                          ML_METHOD(attention),      ML_METHOD(entry_points), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  kIds = PyUnicode_InternFromString("topk_ids");
  kWeights = PyUnicode_InternFromString("topk_weights");
  kPacked = PyUnicode_InternFromString("packed_topk_ids");
  kKvLens = PyUnicode_InternFromString("kv_lens");
  kQueryOffsets = PyUnicode_InternFromString("query_offsets");
  kSlotMap = PyUnicode_InternFromString("slot_map");
  kPositions = PyUnicode_InternFromString("positions");
  kTaken = PyUnicode_InternFromString("taken");
  return PyModule_Create(&kModule);
}
