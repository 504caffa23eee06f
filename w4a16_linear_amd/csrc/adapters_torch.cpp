// The adapters' calls on torch tensors: checks, outputs and marshalling of adapters.py
// in C++, for the reason attention_torch.cpp gives (a call for a few tokens is a few
// microseconds).  Nothing here computes; every call ends in libopq (include/opq_adapters.h).
#include "opq_adapters.h"
#include "torch_common.hpp"

namespace opq_torch {
namespace {

struct Stack {
  opq_lowrank a;
  Tensor down;
};

// Adapters: (down, up, scale)
Stack stack_of(PyObject* o) {
  TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 3, "adapters must be Adapters(down, up, scale)");
  Stack s;
  const Tensor& down = plain(tensor_of(PyTuple_GET_ITEM(o, 0), "down"), "down");
  const Tensor& up = plain(tensor_of(PyTuple_GET_ITEM(o, 1), "up"), "up");
  const Tensor& scale = plain(tensor_of(PyTuple_GET_ITEM(o, 2), "scale"), "scale");
  TORCH_CHECK_VALUE(down.dim() == 3 && up.dim() == 3, "down and up must be [adapters, rank, in] and [adapters, rank, out]");
  s.a.count = down.size(0);
  s.a.rank = down.size(1);
  s.a.k = down.size(2);
  s.a.n = up.size(2);
  const c10::Device dev = down.device();
  s.a.down = static_cast<const uint16_t*>(dense(down, "down", at::kBFloat16, down.sizes(), dev));
  s.a.up = static_cast<const uint16_t*>(dense(up, "up", at::kBFloat16, {s.a.count, s.a.rank, s.a.n}, dev));
  s.a.scale = static_cast<const float*>(dense(scale, "scale", at::kFloat, {s.a.count}, dev));
  s.down = down;
  return s;
}

// [m, width] with dense rows
const Tensor& matrix(PyObject* o, const char* name, int64_t m, int64_t width, c10::Device dev) {
  const Tensor& t = rows(o, name, 2);
  TORCH_CHECK_VALUE((m < 0 || t.size(0) == m) && t.size(1) == width, name, " must be [", m < 0 ? t.size(0) : m,
                    ", ", width, "], got ", t.sizes());
  TORCH_CHECK_VALUE(t.device() == dev, name, " must be on ", dev, ", got ", t.device());
  return t;
}

// A row's stride: one row has none of its own.
int64_t stride_of(const Tensor& t) { return t.size(0) <= 1 ? (t.size(1) + 7) / 8 * 8 : t.stride(0); }

// Whether writing rows of `out` could change what is read from `in`: they share bytes and are
// neither the same rows nor columns of one matrix that lie apart.
bool mixed_up(const Tensor& out, const Tensor& in, bool same_allowed) {
  if (out.numel() == 0 || in.numel() == 0) return false;
  const int64_t eo = out.element_size(), ei = in.element_size();
  const char* po = static_cast<const char*>(out.data_ptr());
  const char* pi = static_cast<const char*>(in.data_ptr());
  const int64_t so = out.size(0) <= 1 ? 0 : out.stride(0) * eo, si = in.size(0) <= 1 ? 0 : in.stride(0) * ei;
  const int64_t wo = out.size(1) * eo, wi = in.size(1) * ei;
  if (po + (out.size(0) - 1) * so + wo <= pi || pi + (in.size(0) - 1) * si + wi <= po) return false;
  if (same_allowed && po == pi && so == si && eo == ei) return false;
  if (so != si || so == 0) return true;
  const int64_t off = ((pi - po) % so + so) % so;
  return !(off >= wo && off + wi <= so);
}

void separate(const Tensor& out, const char* name, const Tensor& in, const char* other, bool same_allowed) {
  TORCH_CHECK_VALUE(!mixed_up(out, in, same_allowed), name, " must not share memory with ", other,
                    same_allowed ? ", unless it is the same rows" : "");
}

const int32_t* index_of(PyObject* o, int64_t m, c10::Device dev) {
  return static_cast<const int32_t*>(dense(o, "index", at::kInt, {m}, dev));
}

}  // namespace

// y or None, x, adapters, index, out or None, out as bfloat16? (without out and y's type),
// workspace or None
PyObject* lowrank_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Stack s = stack_of(a[2]);
  const c10::Device dev = s.down.device();
  const Tensor& x = matrix(a[1], "x", -1, s.a.k, dev);
  TORCH_CHECK_VALUE(x.scalar_type() == at::kBFloat16, "x must be bfloat16, got ", x.scalar_type());
  const int64_t m = x.size(0);
  const int32_t* index = index_of(a[3], m, dev);
  Tensor y;
  if (a[0] != Py_None) y = matrix(a[0], "y", m, s.a.n, dev);
  const int y_dtype = y.defined() ? dtype_of(y.scalar_type(), "y") : OPQ_F32;
  const OnDevice on(x);
  Tensor out;
  if (a[4] == Py_None) {
    out = fresh({m, s.a.n}, int_of(a[5]) ? at::kBFloat16 : at::kFloat, x);
  } else {
    out = matrix(a[4], "out", m, s.a.n, dev);
    TORCH_CHECK_VALUE(at::has_internal_overlap(out) != at::MemOverlap::Yes, "out must not be expanded");
    separate(out, "out", x, "x", false);
    if (y.defined()) separate(out, "out", y, "y", true);
  }
  const int out_dtype = dtype_of(out.scalar_type(), "out");
  size_t bytes = opq_lowrank_workspace_bytes(m, s.a.k, s.a.n, s.a.rank);
  const Tensor ws = workspace_of(a[6], &bytes, x);
  check("opq_lowrank_add",
        opq_lowrank_add(&s.a, static_cast<const uint16_t*>(x.data_ptr()), stride_of(x), index, m,
                        y.defined() ? y.data_ptr() : nullptr, y.defined() ? stride_of(y) : 0, y_dtype,
                        out.data_ptr(), stride_of(out), out_dtype, ws.defined() ? ws.data_ptr() : nullptr,
                        ws.defined() ? bytes : 0, on.stream()));
  if (a[4] != Py_None) {
    written(out);
    Py_INCREF(a[4]);
    return a[4];
  }
  return THPVariable_Wrap(std::move(out));
  END_HANDLE_TH_ERRORS
}

// dy, x, adapters, index, dx or None, out or None, dx as bfloat16?, gradients as bfloat16?,
// input's gradient wanted?, adapters' gradients wanted?, workspace or None
// -> (dx or None, d_down or None, d_up or None)
PyObject* lowrank_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 11);
  const Stack s = stack_of(a[2]);
  const c10::Device dev = s.down.device();
  const Tensor& dy = matrix(a[0], "dy", -1, s.a.n, dev);
  const int64_t m = dy.size(0);
  const Tensor& x = matrix(a[1], "x", m, s.a.k, dev);
  TORCH_CHECK_VALUE(dy.scalar_type() == at::kBFloat16 && x.scalar_type() == at::kBFloat16,
                    "dy and x must be bfloat16, got ", dy.scalar_type(), " and ", x.scalar_type());
  const int32_t* index = index_of(a[3], m, dev);
  Tensor dx;
  if (a[4] != Py_None) dx = matrix(a[4], "dx", m, s.a.k, dev);
  const bool want_dx = int_of(a[8]) != 0, want = int_of(a[9]) != 0;
  const OnDevice on(dy);
  Tensor out;
  if (want_dx) {
    if (a[5] == Py_None) {
      const at::ScalarType type = dx.defined() ? dx.scalar_type() : int_of(a[6]) ? at::kBFloat16 : at::kFloat;
      out = fresh({m, s.a.k}, type, dy);
    } else {
      out = matrix(a[5], "out", m, s.a.k, dev);
      TORCH_CHECK_VALUE(at::has_internal_overlap(out) != at::MemOverlap::Yes, "out must not be expanded");
      TORCH_CHECK_VALUE(!dx.defined() || dx.scalar_type() == out.scalar_type(), "out and dx must have one type, got ",
                        out.scalar_type(), " and ", dx.defined() ? dx.scalar_type() : out.scalar_type());
      separate(out, "out", x, "x", false);
      separate(out, "out", dy, "dy", false);
      if (dx.defined()) separate(out, "out", dx, "dx", true);
    }
  }
  const int dx_dtype = want_dx ? dtype_of(out.scalar_type(), "dx") : OPQ_F32;
  const bool bf16 = int_of(a[7]) != 0;
  Tensor down, up;
  if (want) {
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
    down = fresh({s.a.count, s.a.rank, s.a.k}, type, dy);
    up = fresh({s.a.count, s.a.rank, s.a.n}, type, dy);
  }
  size_t bytes = opq_lowrank_backward_workspace_bytes(m, s.a.k, s.a.n, s.a.rank, s.a.count);
  const Tensor ws = workspace_of(a[10], &bytes, dy);
  check("opq_lowrank_backward",
        opq_lowrank_backward(&s.a, static_cast<const uint16_t*>(dy.data_ptr()), stride_of(dy),
                             static_cast<const uint16_t*>(x.data_ptr()), stride_of(x), index, m,
                             dx.defined() ? dx.data_ptr() : nullptr, dx.defined() ? stride_of(dx) : 0, dx_dtype,
                             want_dx ? out.data_ptr() : nullptr, want_dx ? stride_of(out) : 0,
                             want ? down.data_ptr() : nullptr, want ? up.data_ptr() : nullptr,
                             bf16 ? OPQ_BF16 : OPQ_F32, ws.defined() ? ws.data_ptr() : nullptr,
                             ws.defined() ? bytes : 0, on.stream()));
  PyObject* r[3] = {nullptr, nullptr, nullptr};
  if (want_dx && a[5] != Py_None) {
    written(out);
    Py_INCREF(a[5]);
    r[0] = a[5];
  } else if (want_dx) {
    r[0] = THPVariable_Wrap(std::move(out));
  } else {
    Py_INCREF(Py_None);
    r[0] = Py_None;
  }
  for (int i = 0; i < 2; ++i) {
    if (want) {
      r[1 + i] = THPVariable_Wrap(std::move(i ? up : down));
    } else {
      Py_INCREF(Py_None);
      r[1 + i] = Py_None;
    }
  }
  PyObject* all = r[0] && r[1] && r[2] ? PyTuple_Pack(3, r[0], r[1], r[2]) : nullptr;
  for (PyObject* o : r) Py_XDECREF(o);
  return all;
  END_HANDLE_TH_ERRORS
}

}  // namespace opq_torch
