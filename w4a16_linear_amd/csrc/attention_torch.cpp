// The attention side's calls on torch tensors, as a CPython extension
// (w4a16_linear_amd/_attention.so): the tensor checks, the outputs' allocation
// and the marshalling of attention.py in C++.  A call of one new token is a few
// microseconds of GPU time, less than Python needs to look at its tensors:
// through ctypes rotary, cache write and attention took 11.5, 13.4 and 20.8 us of
// host time a call, of which the launches are 3, 3 and 6.
//
// Nothing here computes; every call ends in libopq (include/opq_attention.h).
#include <ATen/MemoryOverlap.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <vector>

#include "opq_attention.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // opq.OpqError

// The library launches on the current device: make it the tensors' one.
struct OnDevice {
  c10::DeviceIndex old, dev;
  explicit OnDevice(const Tensor& t) : old(c10::hip::current_device()), dev(t.device().index()) {
    if (old != dev) c10::hip::set_device(dev);
  }
  ~OnDevice() {
    if (old != dev) c10::hip::set_device(old);
  }
  void* stream() const { return c10::hip::getCurrentHIPStream(dev).stream(); }
};

const Tensor& tensor_of(PyObject* o, const char* name) {
  TORCH_CHECK_VALUE(THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(), name,
                    " must be a CUDA (HIP) tensor");
  return THPVariable_Unpack(o);
}

// These calls compute outside autograd: a result that ought to carry a gradient would
// come back without one, and nothing would say so.
const Tensor& plain(const Tensor& t, const char* name) {
  TORCH_CHECK(!(t.requires_grad() && at::GradMode::is_enabled()), name,
              " requires grad, which this call does not follow (apply_rotary turns positions "
              "under autograd): detach it, or call under torch.no_grad()");
  return t;
}
// A tensor whose memory this call writes: autograd learns of it, as of every in-place
// operation, should it have saved the old values.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A dense tensor of a known type and shape.
void* dense(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape,
            c10::Device dev) {
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.sizes() == shape && t.is_contiguous(), name,
                    " must be contiguous with shape ", shape, ", got ", t.sizes());
  TORCH_CHECK_VALUE(t.device() == dev, name, " must be on ", dev, ", got ", t.device());
  return t.data_ptr();
}
void* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape,
            c10::Device dev) {
  return dense(tensor_of(o, name), name, type, shape, dev);
}

// A tensor whose last dimension is dense; its other strides are free.
const Tensor& rows(PyObject* o, const char* name, int64_t ndim) {
  const Tensor& t = tensor_of(o, name);
  TORCH_CHECK_VALUE(t.dim() == ndim && (t.size(-1) <= 1 || t.stride(-1) == 1), name, " must be ",
                    ndim, "-d with a dense last dimension");
  return plain(t, name);
}

int dtype_of(at::ScalarType t, const char* what) {
  TORCH_CHECK_VALUE(t == at::kFloat || t == at::kBFloat16, what,
                    " must be float32 or bfloat16, got ", t);
  return t == at::kFloat ? OPQ_F32 : OPQ_BF16;
}

void check(const char* fn, int status) {
  if (status == OPQ_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "sis", fn, status, opq_status_str(status));
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

int64_t int_of(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double double_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// ------------------------------------------------------------------ rotary

// x, positions, table, layout, sections or None, out or None, backward
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor& x = rows(a[0], "x", 3);
  const int dtype = dtype_of(x.scalar_type(), "x");
  const int64_t tokens = x.size(0), heads = x.size(1), dim = x.size(2);
  const Tensor& table = tensor_of(a[2], "table");
  TORCH_CHECK_VALUE(table.dim() == 3, "table must be [length, pairs, 2]");
  const int64_t pairs = table.size(1), length = table.size(0);
  const void* pt = dense(plain(table, "table"), "table", at::kFloat, {length, pairs, 2}, x.device());
  std::vector<int32_t> sections;
  if (a[4] == Py_None) {
    sections.push_back((int32_t)pairs);
  } else {
    PyObject* seq = PySequence_Fast(a[4], "sections must be a sequence");
    if (!seq) throw python_error();
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
    for (Py_ssize_t i = 0; i < count; ++i) {
      const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
      if (v == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw python_error();
      }
      sections.push_back(v < 0 || v > 0x7FFFFFFF ? -1 : (int32_t)v);
    }
    Py_DECREF(seq);
  }
  const int64_t axes = (int64_t)sections.size();
  const Tensor& pos = tensor_of(a[1], "positions");
  const void* pp = pos.dim() == 1 && axes == 1
                       ? dense(pos, "positions", at::kInt, {tokens}, x.device())
                       : dense(pos, "positions", at::kInt, {tokens, axes}, x.device());
  const OnDevice on(x);
  Tensor out;
  if (a[5] == Py_None) {
    out = at::empty({tokens, heads, dim}, x.options());
  } else {
    out = rows(a[5], "out", 3);
    // several threads would write an element, in any order
    TORCH_CHECK_VALUE(at::has_internal_overlap(out) != at::MemOverlap::Yes,
                      "out must not be expanded: its rows would be the same memory");
    TORCH_CHECK_VALUE(out.sizes() == x.sizes() && out.scalar_type() == x.scalar_type() &&
                          out.device() == x.device(),
                      "out must be ", x.scalar_type(), " of shape ", x.sizes(), " on ", x.device());
  }
  check("opq_rotary",
        opq_rotary(x.data_ptr(), dtype, tokens, heads, dim, x.stride(0), x.stride(1),
                   static_cast<const int32_t*>(pp), axes, sections.data(),
                   static_cast<const float*>(pt), length, 2 * pairs, (int)int_of(a[3]),
                   (int)int_of(a[6]), out.data_ptr(), out.stride(0), out.stride(1), on.stream()));
  if (a[5] != Py_None) {
    written(out);
    Py_INCREF(a[5]);
    return a[5];
  }
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------- cache

struct Cache {
  opq_cache c;
  c10::Device dev = c10::Device(c10::kCPU);
};

// PagedCache: (fmt, alpha, k, k_sign, k_scale, v, v_sign, v_scale)
Cache cache_of(PyObject* o) {
  TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 8, "cache must be a PagedCache");
  auto item = [&](int i) { return PyTuple_GET_ITEM(o, i); };
  Cache r;
  std::memset(&r.c, 0, sizeof r.c);
  const char* fmt = PyUnicode_Check(item(0)) ? PyUnicode_AsUTF8(item(0)) : nullptr;
  at::ScalarType type = at::kBFloat16;
  r.c.format = -1;
  if (fmt && !std::strcmp(fmt, "bf16")) r.c.format = OPQ_CACHE_BF16;
  if (fmt && !std::strcmp(fmt, "fp8")) r.c.format = OPQ_CACHE_FP8, type = at::kFloat8_e4m3fn;
  if (fmt && !std::strcmp(fmt, "opq4")) r.c.format = OPQ_CACHE_OPQ4, type = at::kInt;
  TORCH_CHECK_VALUE(r.c.format >= 0, "fmt must be 'bf16', 'fp8' or 'opq4'");
  const Tensor& k = tensor_of(item(2), "k");
  TORCH_CHECK_VALUE(k.dim() == 4, "cache codes must be [pages, heads, page, ...]");
  r.dev = k.device();
  r.c.alpha = (float)double_of(item(1));
  r.c.pages = k.size(0);
  r.c.heads = k.size(1);
  r.c.page = k.size(2);
  r.c.dim = k.size(3);
  const at::IntArrayRef shape = k.sizes();
  r.c.k = dense(k, "k", type, shape, r.dev);
  r.c.v = dense(item(5), "v", type, shape, r.dev);
  if (r.c.format == OPQ_CACHE_OPQ4) {
    r.c.dim *= 8;
    const int64_t signs[4] = {r.c.pages, r.c.heads, r.c.page, r.c.dim / 32};
    r.c.k_sign = static_cast<uint32_t*>(dense(item(3), "k_sign", at::kInt, signs, r.dev));
    r.c.v_sign = static_cast<uint32_t*>(dense(item(6), "v_sign", at::kInt, signs, r.dev));
  }
  r.c.k_scale = static_cast<float*>(dense(item(4), "k_scale", at::kFloat, shape.slice(0, 3), r.dev));
  r.c.v_scale = static_cast<float*>(dense(item(7), "v_scale", at::kFloat, shape.slice(0, 3), r.dev));
  return r;
}

void cache_written(PyObject* o) {
  for (int i = 2; i < 8; ++i)
    if (THPVariable_Check(PyTuple_GET_ITEM(o, i))) written(THPVariable_Unpack(PyTuple_GET_ITEM(o, i)));
}

// cache, k, v, slots
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Cache r = cache_of(a[0]);
  const Tensor& k = rows(a[1], "k", 3);
  const Tensor& v = rows(a[2], "v", 3);
  const int dtype = dtype_of(k.scalar_type(), "k");
  TORCH_CHECK_VALUE(v.scalar_type() == k.scalar_type(), "k and v must have one type, got ",
                    k.scalar_type(), " and ", v.scalar_type());
  TORCH_CHECK_VALUE(k.sizes() == v.sizes() && k.size(1) == r.c.heads && k.size(2) == r.c.dim,
                    "k and v must be [tokens, ", r.c.heads, ", ", r.c.dim, "], got ", k.sizes(),
                    " and ", v.sizes());
  TORCH_CHECK_VALUE(k.device() == r.dev && v.device() == r.dev, "k and v must be on ", r.dev);
  const int64_t tokens = k.size(0);
  const void* slots = dense(a[3], "slots", at::kInt, {tokens}, r.dev);
  const OnDevice on(k);
  check("opq_cache_write",
        opq_cache_write(&r.c, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                        v.stride(1), dtype, tokens, static_cast<const int32_t*>(slots),
                        on.stream()));
  cache_written(a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// cache, slots, bfloat16 results?, k_out or None, v_out or None
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 5);
  const Cache r = cache_of(a[0]);
  const Tensor& slots = tensor_of(a[1], "slots");
  TORCH_CHECK_VALUE(slots.dim() == 1, "slots must be [tokens]");
  const int64_t tokens = slots.size(0);
  const void* ps = dense(slots, "slots", at::kInt, {tokens}, r.dev);
  const bool bf16 = int_of(a[2]) != 0;
  const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
  const int64_t shape[3] = {tokens, r.c.heads, r.c.dim};
  const OnDevice on(slots);
  Tensor out[2];
  void* p[2];
  for (int i = 0; i < 2; ++i) {
    if (a[3 + i] == Py_None) out[i] = at::empty(shape, slots.options().dtype(type));
    else out[i] = plain(tensor_of(a[3 + i], "out"), "out");
    p[i] = dense(out[i], "out", type, shape, r.dev);
  }
  const size_t bytes = out[0].nbytes();
  TORCH_CHECK_VALUE(bytes == 0 || static_cast<char*>(p[0]) + bytes <= p[1] ||
                        static_cast<char*>(p[1]) + bytes <= p[0],
                    "the two of out must not share memory");
  check("opq_cache_read", opq_cache_read(&r.c, tokens, static_cast<const int32_t*>(ps), p[0], p[1],
                                         bf16 ? OPQ_BF16 : OPQ_F32, on.stream()));
  for (const Tensor& t : out) written(t);
  PyObject* k = THPVariable_Wrap(std::move(out[0]));
  PyObject* v = THPVariable_Wrap(std::move(out[1]));
  PyObject* both = k && v ? PyTuple_Pack(2, k, v) : nullptr;
  Py_XDECREF(k);
  Py_XDECREF(v);
  return both;
  END_HANDLE_TH_ERRORS
}

// cache, src, dst
PyObject* cache_move(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 3);
  const Cache r = cache_of(a[0]);
  const Tensor& src = tensor_of(a[1], "src");
  TORCH_CHECK_VALUE(src.dim() == 2, "src must be [batch, count]");
  const int64_t batch = src.size(0), count = src.size(1);
  const void* ps = dense(src, "src", at::kInt, {batch, count}, r.dev);
  const void* pd = dense(a[2], "dst", at::kInt, {batch, count}, r.dev);
  const OnDevice on(src);
  check("opq_cache_move", opq_cache_move(&r.c, batch, count, static_cast<const int32_t*>(ps),
                                         static_cast<const int32_t*>(pd), on.stream()));
  cache_written(a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// --------------------------------------------------------------- attention

// q, cache, page_table, lens, mask|None, counts|None, scale|None, max_len|None, out|None,
// return_lse, workspace|None
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 11);
  const Cache r = cache_of(a[1]);
  const Tensor& q = rows(a[0], "q", 4);
  TORCH_CHECK_VALUE(q.scalar_type() == at::kBFloat16, "q must be bfloat16, got ", q.scalar_type());
  TORCH_CHECK_VALUE(q.device() == r.dev, "q must be on ", r.dev, ", got ", q.device());
  const int64_t batch = q.size(0), draft = q.size(1), heads = q.size(2), dim = q.size(3);
  TORCH_CHECK_VALUE(dim == r.c.dim && r.c.heads > 0 && heads % r.c.heads == 0, "q has ", heads,
                    " heads of ", dim, ", the cache ", r.c.heads, " of ", r.c.dim);
  const Tensor& table = tensor_of(a[2], "page_table");
  TORCH_CHECK_VALUE(table.dim() == 2, "page_table must be [batch, max_pages]");
  const int64_t max_pages = table.size(1);
  const void* pt = dense(table, "page_table", at::kInt, {batch, max_pages}, r.dev);
  const void* lens = dense(a[3], "lens", at::kInt, {batch}, r.dev);
  const void* mask = nullptr;
  int64_t mask_batch = 0;
  if (a[4] != Py_None) {
    const Tensor& m = tensor_of(a[4], "mask");
    const int64_t words = (draft + 31) / 32;
    if (m.dim() == 3) {
      mask = dense(m, "mask", at::kInt, {batch, draft, words}, r.dev);
      mask_batch = draft * words;
    } else {
      mask = dense(m, "mask", at::kInt, {draft, words}, r.dev);
    }
  }
  const void* counts =
      a[5] == Py_None ? nullptr : dense(a[5], "counts", at::kInt, {batch}, r.dev);
  const float scale =
      a[6] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)double_of(a[6]);
  const int64_t room = max_pages * r.c.page - draft;
  const int64_t max_len = a[7] == Py_None ? (room > 0 ? room : 0) : int_of(a[7]);
  const OnDevice on(q);
  const int64_t shape[4] = {batch, draft, heads, dim};
  Tensor out =
      a[8] == Py_None ? at::empty(shape, q.options()) : plain(tensor_of(a[8], "out"), "out");
  void* po = dense(out, "out", at::kBFloat16, shape, r.dev);
  Tensor lse;
  if (int_of(a[9])) lse = at::empty({batch, draft, heads}, q.options().dtype(at::kFloat));
  size_t bytes =
      opq_cache_attention_workspace_bytes(batch, draft, heads, r.c.heads, dim, max_len);
  Tensor ws;
  if (a[10] != Py_None) {
    ws = tensor_of(a[10], "workspace");
    TORCH_CHECK_VALUE(ws.is_contiguous() && ws.device() == r.dev,
                      "workspace must be a contiguous tensor on ", r.dev);
    bytes = (size_t)ws.numel() * ws.element_size();
  } else if (bytes) {
    ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
  }
  check("opq_cache_attention",
        opq_cache_attention(
            &r.c, static_cast<const uint16_t*>(q.data_ptr()), batch, draft, heads, q.stride(0),
            q.stride(1), q.stride(2), static_cast<const int32_t*>(pt), max_pages,
            static_cast<const int32_t*>(lens), static_cast<const int32_t*>(counts), max_len,
            static_cast<const uint32_t*>(mask), mask_batch, scale, static_cast<uint16_t*>(po),
            lse.defined() ? lse.data_ptr<float>() : nullptr,
            ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? bytes : 0, on.stream()));
  PyObject* first = nullptr;
  if (a[8] == Py_None) {
    first = THPVariable_Wrap(std::move(out));
  } else {
    written(out);
    first = a[8];
    Py_INCREF(first);
  }
  if (!lse.defined() || !first) return first;
  PyObject* second = THPVariable_Wrap(std::move(lse));
  PyObject* both = second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_DECREF(first);
  Py_XDECREF(second);
  return both;
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef kMethods[] = {{"rotary", FAST(rotary), METH_FASTCALL, nullptr},
                          {"cache_write", FAST(cache_write), METH_FASTCALL, nullptr},
                          {"cache_read", FAST(cache_read), METH_FASTCALL, nullptr},
                          {"cache_move", FAST(cache_move), METH_FASTCALL, nullptr},
                          {"attention", FAST(attention), METH_FASTCALL, nullptr},
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention() { return PyModule_Create(&kModule); }
