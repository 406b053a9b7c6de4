// The ordinary calls of include/flce_ops.h, flce_embed.h and flce_blocks.h from Python, without ctypes: reads the tensors,
// allocates the outputs (and the workspace) on the current stream and enqueues the call.
//
// A kernel of a decoding step takes a few microseconds; marshalling its arguments through
// Python and ctypes takes 25 to 30. Each function here serves the plain form of a call (no
// preallocated outputs, workspace, status word or stream given). Where an argument is not of
// the expected kind, or the library refuses the call, it returns None without having
// enqueued anything, and the caller goes on to the general form in _ops_binding.py, which
// says what is wrong. A CUDA error may come after a launch, so it is raised here and not tried
// again.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstdint>
#include <exception>
#include <vector>

#include "../../include/flce_blocks.h"
#include "../../include/flce_embed.h"
#include "../../include/flce_ops.h"

namespace {

using at::Tensor;

struct Refused {};

// A tensor argument; null for None.
const Tensor* tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused{};
  return &THPVariable_Unpack(o);
}

const Tensor& required(PyObject* o, int device) {
  const Tensor* t = tensor(o);
  if (t == nullptr || !t->is_cuda() || t->get_device() != device) throw Refused{};
  return *t;
}

int dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return FLCE_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return FLCE_DTYPE_BF16;
  throw Refused{};
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{};
  }
  return v;
}

int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  if (v != static_cast<int32_t>(v)) throw Refused{};
  return static_cast<int32_t>(v);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{};
  }
  return v;
}

void check(bool ok) {
  if (!ok) throw Refused{};
}

struct Failed {
  const char* where;
};

// The library's answer to call `where`: only what it refuses has enqueued nothing.
void check(int rc, const char* where) {
  if (rc == FLCE_ERR_CUDA) throw Failed{where};
  check(rc == FLCE_OK);
}

PyObject* error_type = nullptr;   // FLCEError

// Allocations and launches of one call: the current device and its current stream.
struct Here {
  int device;
  void* stream;
  Here() {
    if (c10::cuda::device_count() == 0) throw Refused{};
    device = c10::cuda::current_device();
    stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  }
  Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                  std::nullopt);
  }
};

// int32 [N] tokens, or null.
const int32_t* tokens_of(PyObject* o, int64_t N, int device) {
  if (o == Py_None) return nullptr;
  const Tensor& t = required(o, device);
  check(t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == N && t.is_contiguous());
  return t.const_data_ptr<int32_t>();
}

// fp32 [N], or null.
const float* vector_of(PyObject* o, int64_t N, int device) {
  if (o == Py_None) return nullptr;
  const Tensor& t = required(o, device);
  check(t.scalar_type() == at::kFloat && t.dim() == 1 && t.size(0) == N && t.is_contiguous());
  return t.const_data_ptr<float>();
}

// [N, V] with unit column stride: its row stride.
int64_t rows_of(const Tensor& t) {
  check(t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1));
  const int64_t ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
  check(ld >= t.size(1));
  return ld;
}

flce_logprob_options options(PyObject* ignore_index, int64_t top_k, PyObject* temperature,
                             int dw_dtype = FLCE_DTYPE_F32) {
  flce_logprob_options o;
  flce_default_logprob_options(&o);
  o.ignore_index = integer32(ignore_index);
  o.top_k = static_cast<int32_t>(top_k);
  o.temperature = static_cast<float>(number(temperature));
  o.dw_dtype = dw_dtype;
  return o;
}

// New reference to a tuple of tensors; undefined ones are None.
PyObject* tuple(std::initializer_list<Tensor> tensors) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (r == nullptr) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : tensors) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (o == nullptr) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Runs f with C++ exceptions turned into None (a refusal) or a Python error.
template <typename F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F&& f) {
  if (nargs != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
    Py_RETURN_NONE;
  } catch (const Failed& f) {
    if (error_type == nullptr) {
      PyErr_SetString(PyExc_RuntimeError, f.where);
      return nullptr;
    }
    PyObject* const error = PyObject_CallFunction(error_type, "is", FLCE_ERR_CUDA, f.where);
    if (error != nullptr) {
      PyErr_SetObject(error_type, error);
      Py_DECREF(error);
    }
    return nullptr;
  } catch (...) {   // out of memory and the like, as PyTorch's own types
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

#define FUNCTION(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)

struct LogprobOutputs {
  Tensor logprob, entropy, lse, top_logprob, top_id;
  LogprobOutputs(const Here& h, int64_t N, int64_t top_k)
      : logprob(h.empty({N}, at::kFloat)), entropy(h.empty({N}, at::kFloat)), lse(h.empty({N}, at::kFloat)) {
    if (top_k > 0) {
      top_logprob = h.empty({N, top_k}, at::kFloat);
      top_id = h.empty({N, top_k}, at::kInt);
    }
  }
  float* top_lp() const { return top_id.defined() ? top_logprob.data_ptr<float>() : nullptr; }
  int32_t* ids() const { return top_id.defined() ? top_id.data_ptr<int32_t>() : nullptr; }
  PyObject* tuple() const { return ::tuple({logprob, entropy, lse, top_logprob, top_id}); }
};

// (logits, tokens, top_k, temperature, ignore_index)
FUNCTION(token_logprobs) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Here h;
    const Tensor& z = required(a[0], h.device);
    const int dtype = dtype_of(z);
    const int64_t ld = rows_of(z), N = z.size(0), V = z.size(1), k = integer(a[2]);
    check(k >= 0 && k <= FLCE_MAX_TOP_K);
    const int32_t* y = tokens_of(a[1], N, h.device);
    const flce_logprob_options o = options(a[4], k, a[3]);
    const LogprobOutputs out(h, N, k);
    check(flce_token_logprobs(z.const_data_ptr(), dtype, ld, y, N, V, &o, out.logprob.data_ptr<float>(),
                              out.entropy.data_ptr<float>(), out.lse.data_ptr<float>(), out.top_lp(),
                              out.ids(), nullptr, h.stream), "flce_token_logprobs");
    return out.tuple();
  });
}

// (logits, tokens, logprob, entropy, lse, dlogprob, dentropy, dlse, temperature, ignore_index)
FUNCTION(token_logprobs_backward) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Here h;
    const Tensor& z = required(a[0], h.device);
    const int dtype = dtype_of(z);
    const int64_t ld = rows_of(z), N = z.size(0), V = z.size(1);
    const int32_t* y = tokens_of(a[1], N, h.device);
    const float* v[6];
    for (int i = 0; i < 6; ++i) v[i] = vector_of(a[2 + i], N, h.device);
    const flce_logprob_options o = options(a[9], 0, a[8]);
    // rows that start relative to 16 bytes as the logits' do (the first one too), however far
    // apart those are
    const int64_t elt = static_cast<int64_t>(z.element_size()), dld = V + (ld - V) % (16 / elt);
    const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(z.const_data_ptr()) & 15u) / elt;
    const Tensor g = h.empty({N > 0 ? off + (N - 1) * dld + V : 0}, z.scalar_type());
    g.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef({N, V}), at::IntArrayRef({dld, 1}),
                                                   N > 0 ? off : 0);
    check(flce_token_logprobs_backward(z.const_data_ptr(), dtype, ld, y, N, V, &o, v[0], v[1], v[2], v[3],
                                       v[4], v[5], g.data_ptr(), dld, h.stream),
          "flce_token_logprobs_backward");
    return THPVariable_Wrap(g);
  });
}

struct Linear {
  const Tensor& H;
  const Tensor& W;
  int64_t N, D, V;
  Linear(PyObject* h, PyObject* w, int device) : H(required(h, device)), W(required(w, device)) {
    check(H.scalar_type() == at::kBFloat16 && W.scalar_type() == at::kBFloat16 && H.dim() == 2 &&
          W.dim() == 2 && H.size(1) == W.size(1) && H.is_contiguous() && W.is_contiguous());
    N = H.size(0);
    D = H.size(1);
    V = W.size(0);
  }
  const uint16_t* h() const { return static_cast<const uint16_t*>(H.const_data_ptr()); }
  const uint16_t* w() const { return static_cast<const uint16_t*>(W.const_data_ptr()); }
  Tensor workspace(const Here& here, const flce_logprob_options& o, int backward, size_t* bytes) const {
    check(flce_linear_logprobs_workspace_size(N, D, V, &o, backward, bytes),
          "flce_linear_logprobs_workspace_size");
    return here.empty({static_cast<int64_t>(*bytes < 16 ? 16 : *bytes)}, at::kByte);
  }
};

// (H, W, tokens, top_k, temperature, ignore_index)
FUNCTION(linear_token_logprobs) {
  return guarded(n, 6, [&]() -> PyObject* {
    const Here h;
    const Linear p(a[0], a[1], h.device);
    const int64_t k = integer(a[3]);
    check(k >= 0 && k <= FLCE_MAX_TOP_K);
    const int32_t* y = tokens_of(a[2], p.N, h.device);
    const flce_logprob_options o = options(a[5], k, a[4]);
    const LogprobOutputs out(h, p.N, k);
    size_t bytes = 0;
    const Tensor ws = p.workspace(h, o, 0, &bytes);
    check(flce_linear_token_logprobs(p.h(), p.w(), y, p.N, p.D, p.V, &o, out.logprob.data_ptr<float>(),
                                     out.entropy.data_ptr<float>(), out.lse.data_ptr<float>(), out.top_lp(),
                                     out.ids(), ws.data_ptr(), bytes, nullptr, h.stream),
          "flce_linear_token_logprobs");
    return out.tuple();
  });
}

// (H, W, tokens, logprob, entropy, lse, dlogprob, dentropy, dlse, temperature, ignore_index,
//  need_dh, need_dw, dw_dtype)
FUNCTION(linear_token_logprobs_backward) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Here h;
    const Linear p(a[0], a[1], h.device);
    const int32_t* y = tokens_of(a[2], p.N, h.device);
    const float* v[6];
    for (int i = 0; i < 6; ++i) v[i] = vector_of(a[3 + i], p.N, h.device);
    const int dw_dtype = static_cast<int>(integer(a[13]));
    const flce_logprob_options o = options(a[10], 0, a[9], dw_dtype);
    Tensor dH, dW;
    if (integer(a[11])) dH = h.empty({p.N, p.D}, at::kBFloat16);
    if (integer(a[12])) dW = h.empty({p.V, p.D}, dw_dtype == FLCE_DTYPE_BF16 ? at::kBFloat16 : at::kFloat);
    size_t bytes = 0;
    const Tensor ws = p.workspace(h, o, 1, &bytes);
    check(flce_linear_token_logprobs_backward(
              p.h(), p.w(), y, p.N, p.D, p.V, &o, v[0], v[1], v[2], v[3], v[4], v[5],
              dH.defined() ? static_cast<uint16_t*>(dH.data_ptr()) : nullptr,
              dW.defined() ? dW.data_ptr() : nullptr, ws.data_ptr(), bytes, nullptr, h.stream),
          "flce_linear_token_logprobs_backward");
    return tuple({dH, dW});
  });
}

// x [..., D] as rows of unit column stride.
struct NormRows {
  int64_t N, D, ld;
  explicit NormRows(const Tensor& x) {
    check(x.dim() >= 1 && x.numel() > 0);
    D = x.size(-1);
    N = x.numel() / D;
    if (x.dim() == 2) {
      ld = rows_of(x);
    } else {
      check(x.is_contiguous());
      ld = D;
    }
  }
};

const void* param_of(PyObject* o, int64_t D, int device, int* code) {
  if (o == Py_None) return nullptr;
  const Tensor& t = required(o, device);
  check(t.dim() == 1 && t.size(0) == D && t.is_contiguous());
  const int c = dtype_of(t);
  check(*code < 0 || *code == c);
  *code = c;
  return t.const_data_ptr();
}

// (x, weight, bias, eps)
FUNCTION(layer_norm) {
  return guarded(n, 4, [&]() -> PyObject* {
    const Here h;
    const Tensor& x = required(a[0], h.device);
    const int dtype = dtype_of(x);
    const NormRows r(x);
    int wcode = -1;
    const void* w = param_of(a[1], r.D, h.device, &wcode);
    const void* b = param_of(a[2], r.D, h.device, &wcode);
    const Tensor y = h.empty(x.sizes(), x.scalar_type());
    const Tensor mean = h.empty({r.N}, at::kFloat), rstd = h.empty({r.N}, at::kFloat);
    check(flce_layer_norm(x.const_data_ptr(), dtype, r.ld, w, b, wcode < 0 ? FLCE_DTYPE_F32 : wcode, r.N,
                          r.D, static_cast<float>(number(a[3])), y.data_ptr(), r.D,
                          mean.data_ptr<float>(), rstd.data_ptr<float>(), h.stream), "flce_layer_norm");
    return tuple({y, mean, rstd});
  });
}

// (dy, x, weight, mean, rstd, need_dx, need_dweight, need_dbias)
FUNCTION(layer_norm_backward) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Here h;
    const Tensor &dy = required(a[0], h.device), &x = required(a[1], h.device);
    const int dtype = dtype_of(x);
    check(dy.scalar_type() == x.scalar_type() && dy.sizes() == x.sizes());
    const NormRows r(x), g(dy);
    int wcode = -1;
    const void* w = param_of(a[2], r.D, h.device, &wcode);
    const float *mean = vector_of(a[3], r.N, h.device), *rstd = vector_of(a[4], r.N, h.device);
    const at::ScalarType wtype = wcode == FLCE_DTYPE_BF16 ? at::kBFloat16 : at::kFloat;
    Tensor dx, dw, db, ws;
    if (integer(a[5])) dx = h.empty(x.sizes(), x.scalar_type());
    if (integer(a[6])) dw = h.empty({r.D}, wtype);
    if (integer(a[7])) db = h.empty({r.D}, wtype);
    size_t bytes = 0;
    if (dw.defined() || db.defined()) {
      check(flce_layer_norm_workspace_size(r.N, r.D, &bytes), "flce_layer_norm_workspace_size");
      ws = h.empty({static_cast<int64_t>(bytes < 16 ? 16 : bytes)}, at::kByte);
    }
    auto at_of = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    check(flce_layer_norm_backward(dy.const_data_ptr(), g.ld, x.const_data_ptr(), dtype, r.ld, w,
                                   wcode < 0 ? FLCE_DTYPE_F32 : wcode, mean, rstd, r.N, r.D, at_of(dx),
                                   r.D, at_of(dw), at_of(db), at_of(ws), bytes, h.stream),
          "flce_layer_norm_backward");
    return tuple({dx, dw, db});
  });
}

// (grads: list, outs: list or None, max_norm); outs may be grads. Contiguous tensors only.
FUNCTION(clip_grads) {
  return guarded(n, 3, [&]() -> PyObject* {
    const Here h;
    check(PyList_CheckExact(a[0]) && (a[1] == Py_None || PyList_CheckExact(a[1])));
    const Py_ssize_t count = PyList_GET_SIZE(a[0]);
    check(a[1] == Py_None || PyList_GET_SIZE(a[1]) == count);
    std::vector<const void*> src(static_cast<size_t>(count));
    std::vector<void*> dst(static_cast<size_t>(a[1] == Py_None ? 0 : count));
    std::vector<int64_t> numel(static_cast<size_t>(count));
    std::vector<int32_t> codes(static_cast<size_t>(count));
    for (Py_ssize_t i = 0; i < count; ++i) {
      const Tensor& g = required(PyList_GET_ITEM(a[0], i), h.device);
      check(g.is_contiguous());
      const size_t k = static_cast<size_t>(i);
      src[k] = g.const_data_ptr();
      numel[k] = g.numel();
      codes[k] = dtype_of(g);
      if (a[1] != Py_None) {
        const Tensor& o = required(PyList_GET_ITEM(a[1], i), h.device);
        check(o.scalar_type() == g.scalar_type() && o.sizes() == g.sizes() && o.is_contiguous());
        dst[k] = o.data_ptr();
      }
    }
    size_t bytes = 0;
    check(flce_clip_grads_workspace_size(count, &bytes), "flce_clip_grads_workspace_size");
    const Tensor norm = h.empty({1}, at::kFloat);
    const Tensor ws = h.empty({static_cast<int64_t>(bytes)}, at::kByte);
    check(flce_clip_grads(src.data(), a[1] == Py_None ? nullptr : dst.data(), numel.data(), codes.data(),
                          count, static_cast<float>(number(a[2])), norm.data_ptr<float>(), ws.data_ptr(),
                          bytes, h.stream), "flce_clip_grads");
    return THPVariable_Wrap(norm);
  });
}

// A torch.dtype, or `none` for None.
at::ScalarType type_of(PyObject* o, at::ScalarType none) {
  if (o == Py_None) return none;
  check(THPDtype_Check(o));
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int code_of(at::ScalarType t) {
  if (t == at::kFloat) return FLCE_DTYPE_F32;
  if (t == at::kBFloat16) return FLCE_DTYPE_BF16;
  throw Refused{};
}

// int32 tokens of any shape, dense.
const Tensor& ids_of(PyObject* o, int device) {
  const Tensor& t = required(o, device);
  check(t.scalar_type() == at::kInt && t.is_contiguous());
  return t;
}

// (weight, tokens, scale, ignore_index, dtype)
FUNCTION(embedding) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Here h;
    const Tensor &w = required(a[0], h.device), &ids = ids_of(a[1], h.device);
    const int wcode = dtype_of(w);
    const int64_t ldw = rows_of(w), D = w.size(1);
    const at::ScalarType type = type_of(a[4], w.scalar_type());
    const int code = code_of(type);
    std::vector<int64_t> shape(ids.sizes().begin(), ids.sizes().end());
    shape.push_back(D);
    const float scale = static_cast<float>(number(a[2]));
    const int32_t ignore = integer32(a[3]);
    const Tensor y = h.empty(shape, type);
    check(flce_embedding(w.const_data_ptr(), wcode, ldw, ids.const_data_ptr<int32_t>(), ids.numel(), w.size(0),
                         D, scale, ignore, y.data_ptr(), code, D, nullptr, h.stream), "flce_embedding");
    return THPVariable_Wrap(y);
  });
}

// (dy, tokens, rows, scale, ignore_index, dtype)
FUNCTION(embedding_backward) {
  return guarded(n, 6, [&]() -> PyObject* {
    const Here h;
    const Tensor &dy = required(a[0], h.device), &ids = ids_of(a[1], h.device);
    const int dtype = dtype_of(dy);
    check(dy.dim() == ids.dim() + 1 && dy.sizes().slice(0, dy.dim() - 1) == ids.sizes());
    const NormRows r(dy);
    const int64_t rows = integer(a[2]);
    const at::ScalarType type = type_of(a[5], dy.scalar_type());
    const int code = code_of(type);
    const float scale = static_cast<float>(number(a[3]));
    const int32_t ignore = integer32(a[4]);
    size_t bytes = 0;
    check(flce_embedding_backward_workspace_size(r.N, rows, r.D, &bytes), "flce_embedding_backward_workspace_size");
    const Tensor dW = h.empty({rows, r.D}, type);
    const Tensor ws = h.empty({static_cast<int64_t>(bytes < 16 ? 16 : bytes)}, at::kByte);
    check(flce_embedding_backward(dy.const_data_ptr(), dtype, r.ld, ids.const_data_ptr<int32_t>(), r.N, rows, r.D,
                                  scale, ignore, dW.data_ptr(), code, r.D, 0, ws.data_ptr(), bytes, h.stream),
          "flce_embedding_backward");
    return THPVariable_Wrap(dW);
  });
}

int64_t record_of(int64_t D) {
  int64_t bytes = 0;
  check(flce_packed_row_bytes(D, &bytes), "flce_packed_row_bytes");
  return bytes;
}

// (x): the records
FUNCTION(pack_e4m3) {
  return guarded(n, 1, [&]() -> PyObject* {
    const Here h;
    const Tensor& x = required(a[0], h.device);
    const int dtype = dtype_of(x);
    const NormRows r(x);
    const Tensor data = h.empty({r.N, record_of(r.D)}, at::kByte);
    check(flce_pack_e4m3(x.const_data_ptr(), dtype, r.ld, r.N, r.D, static_cast<uint8_t*>(data.data_ptr()),
                         h.stream), "flce_pack_e4m3");
    return THPVariable_Wrap(data);
  });
}

// Records of a shape (a tuple): rows and D.
struct Records {
  std::vector<int64_t> shape;
  int64_t N = 1, D;
  const uint8_t* data;
  Records(PyObject* o, PyObject* size, int device) {
    check(PyTuple_Check(size) && PyTuple_GET_SIZE(size) >= 1);
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(size); ++i) shape.push_back(integer(PyTuple_GET_ITEM(size, i)));
    D = shape.back();
    for (size_t i = 0; i + 1 < shape.size(); ++i) N *= shape[i];
    const Tensor& t = required(o, device);
    check(t.scalar_type() == at::kByte && t.dim() == 2 && t.size(0) == N && t.size(1) == record_of(D) &&
          t.is_contiguous());
    data = static_cast<const uint8_t*>(t.const_data_ptr());
  }
};

// (records, shape, dtype)
FUNCTION(unpack_e4m3) {
  return guarded(n, 3, [&]() -> PyObject* {
    const Here h;
    const Records r(a[0], a[1], h.device);
    const at::ScalarType type = type_of(a[2], at::kFloat);
    const int code = code_of(type);
    const Tensor x = h.empty(r.shape, type);
    check(flce_unpack_e4m3(r.data, r.N, r.D, x.data_ptr(), code, r.D, h.stream), "flce_unpack_e4m3");
    return THPVariable_Wrap(x);
  });
}

// (x, weight, bias, eps)
FUNCTION(layer_norm_packed) {
  return guarded(n, 4, [&]() -> PyObject* {
    const Here h;
    const Tensor& x = required(a[0], h.device);
    const int dtype = dtype_of(x);
    const NormRows r(x);
    int wcode = -1;
    const void* w = param_of(a[1], r.D, h.device, &wcode);
    const void* b = param_of(a[2], r.D, h.device, &wcode);
    const float eps = static_cast<float>(number(a[3]));
    const Tensor data = h.empty({r.N, record_of(r.D)}, at::kByte);
    const Tensor y = h.empty(x.sizes(), x.scalar_type());
    const Tensor mean = h.empty({r.N}, at::kFloat), rstd = h.empty({r.N}, at::kFloat);
    check(flce_layer_norm_packed(x.const_data_ptr(), dtype, r.ld, w, b, wcode < 0 ? FLCE_DTYPE_F32 : wcode, r.N,
                                 r.D, eps, y.data_ptr(), r.D, mean.data_ptr<float>(), rstd.data_ptr<float>(),
                                 static_cast<uint8_t*>(data.data_ptr()), h.stream), "flce_layer_norm_packed");
    return tuple({y, mean, rstd, data});
  });
}

// (dy, records, shape, weight, mean, rstd, need_dx, need_dweight, need_dbias)
FUNCTION(layer_norm_packed_backward) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Here h;
    const Tensor& dy = required(a[0], h.device);
    const int dtype = dtype_of(dy);
    const Records x(a[1], a[2], h.device);
    check(dy.sizes() == at::IntArrayRef(x.shape));
    const NormRows g(dy);
    int wcode = -1;
    const void* w = param_of(a[3], g.D, h.device, &wcode);
    const float *mean = vector_of(a[4], g.N, h.device), *rstd = vector_of(a[5], g.N, h.device);
    const at::ScalarType wtype = wcode == FLCE_DTYPE_BF16 ? at::kBFloat16 : at::kFloat;
    Tensor dx, dw, db, ws;
    if (integer(a[6])) dx = h.empty(dy.sizes(), dy.scalar_type());
    if (integer(a[7])) dw = h.empty({g.D}, wtype);
    if (integer(a[8])) db = h.empty({g.D}, wtype);
    size_t bytes = 0;
    if (dw.defined() || db.defined()) {
      check(flce_layer_norm_workspace_size(g.N, g.D, &bytes), "flce_layer_norm_workspace_size");
      ws = h.empty({static_cast<int64_t>(bytes < 16 ? 16 : bytes)}, at::kByte);
    }
    auto at_of = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    check(flce_layer_norm_packed_backward(dy.const_data_ptr(), dtype, g.ld, x.data, w,
                                          wcode < 0 ? FLCE_DTYPE_F32 : wcode, mean, rstd, g.N, g.D, at_of(dx),
                                          g.D, at_of(dw), at_of(db), at_of(ws), bytes, h.stream),
          "flce_layer_norm_packed_backward");
    return tuple({dx, dw, db});
  });
}

// (x, format): codes, scales, row scales
FUNCTION(quantize_fp4) {
  return guarded(n, 2, [&]() -> PyObject* {
    const Here h;
    const Tensor& x = required(a[0], h.device);
    const int dtype = dtype_of(x);
    const NormRows r(x);
    const int32_t format = integer32(a[1]);
    int64_t row = 0;
    size_t size = 0;
    check(flce_fp4_sizes(r.N, r.D, format, &row, &size), "flce_fp4_sizes");
    const Tensor codes = h.empty({r.N, row}, at::kByte), scales = h.empty({static_cast<int64_t>(size)}, at::kByte);
    Tensor rows;
    if (format == FLCE_FP4_NV) rows = h.empty({r.N}, at::kFloat);
    check(flce_quantize_fp4(x.const_data_ptr(), dtype, r.ld, r.N, r.D, format,
                            static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()),
                            rows.defined() ? rows.data_ptr<float>() : nullptr, h.stream), "flce_quantize_fp4");
    return tuple({codes, scales, rows});
  });
}

// A 4-bit matrix: codes, scales, row scales and shape.
struct Fp4 {
  std::vector<int64_t> shape;
  int64_t N = 1, D;
  const uint8_t *codes, *scales;
  const float* rows;
  Fp4(PyObject* const* a, int32_t format, int device) {
    check(PyTuple_Check(a[3]) && PyTuple_GET_SIZE(a[3]) >= 1);
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[3]); ++i) shape.push_back(integer(PyTuple_GET_ITEM(a[3], i)));
    D = shape.back();
    for (size_t i = 0; i + 1 < shape.size(); ++i) N *= shape[i];
    int64_t row = 0;
    size_t size = 0;
    check(flce_fp4_sizes(N, D, format, &row, &size), "flce_fp4_sizes");
    auto bytes = [&](PyObject* o, at::IntArrayRef want) {
      const Tensor& t = required(o, device);
      check(t.scalar_type() == at::kByte && t.sizes() == want && t.is_contiguous());
      return static_cast<const uint8_t*>(t.const_data_ptr());
    };
    codes = bytes(a[0], {N, row});
    scales = bytes(a[1], {static_cast<int64_t>(size)});
    rows = format == FLCE_FP4_NV ? vector_of(a[2], N, device) : nullptr;
  }
};

// (codes, scales, row scales, shape, format, dtype)
FUNCTION(dequantize_fp4) {
  return guarded(n, 6, [&]() -> PyObject* {
    const Here h;
    const int32_t format = integer32(a[4]);
    const Fp4 m(a, format, h.device);
    const at::ScalarType type = type_of(a[5], at::kFloat);
    const int code = code_of(type);
    const Tensor x = h.empty(m.shape, type);
    check(flce_dequantize_fp4(m.codes, m.scales, m.rows, m.N, m.D, format, x.data_ptr(), code, m.D, h.stream),
          "flce_dequantize_fp4");
    return THPVariable_Wrap(x);
  });
}

// (h: codes, scales, row scales, shape, w: the same, format, dtype)
FUNCTION(linear_fp4) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Here h;
    const int32_t format = integer32(a[8]);
    const Fp4 H(a, format, h.device), W(a + 4, format, h.device);
    check(W.shape.size() == 2 && W.D == H.D);
    const at::ScalarType type = type_of(a[9], at::kBFloat16);
    const int code = code_of(type);
    std::vector<int64_t> shape(H.shape);
    shape.back() = W.N;
    const Tensor y = h.empty(shape, type);
    check(flce_linear_fp4(H.codes, H.scales, H.rows, W.codes, W.scales, W.rows, H.N, H.D, W.N, format, y.data_ptr(),
                          code, W.N, 0, nullptr, h.stream), "flce_linear_fp4");
    return THPVariable_Wrap(y);
  });
}

// (FLCEError): the type of the errors raised here.
FUNCTION(set_error_type) {
  return guarded(n, 1, [&]() -> PyObject* {
    Py_INCREF(a[0]);
    Py_XSETREF(error_type, a[0]);
    Py_RETURN_NONE;
  });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(token_logprobs),        METHOD(token_logprobs_backward),
                         METHOD(linear_token_logprobs), METHOD(linear_token_logprobs_backward),
                         METHOD(layer_norm),            METHOD(layer_norm_backward),
                         METHOD(clip_grads),            METHOD(set_error_type),
                         METHOD(embedding),             METHOD(embedding_backward),
                         METHOD(pack_e4m3),             METHOD(unpack_e4m3),
                         METHOD(layer_norm_packed),     METHOD(layer_norm_packed_backward),
                         METHOD(quantize_fp4),          METHOD(dequantize_fp4),
                         METHOD(linear_fp4),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_flce_ops", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__flce_ops() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) {
    Py_DECREF(m);
    m = nullptr;
  }
  return m;
}
