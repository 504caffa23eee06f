// The attention side's calls on torch tensors, as a CPython extension
// (w4a16_linear_amd/_attention.so): the tensor checks, the outputs' allocation
// and the marshalling of attention.py in C++.  A call of one new token is a few
// microseconds of GPU time, less than Python needs to look at its tensors:
// through ctypes rotary, cache write and attention took 11.5, 13.4 and 20.8 us of
// host time a call, of which the launches are 3, 3 and 6.
//
// Nothing here computes; every call ends in libopq (include/opq_attention.h).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "opq_attention.h"
#include "torch_common.hpp"

namespace opq_torch {

PyObject* g_error = nullptr;

}  // namespace opq_torch

namespace {

using namespace opq_torch;

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

// cache, src, dst
PyObject* cache_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 3);
  const Cache r = cache_of(a[0]);
  const Tensor& src = tensor_of(a[1], "src");
  TORCH_CHECK_VALUE(src.dim() == 1, "src must be [count]");
  const int64_t count = src.size(0);
  const void* ps = dense(src, "src", at::kInt, {count}, r.dev);
  const void* pd = dense(a[2], "dst", at::kInt, {count}, r.dev);
  const OnDevice on(src);
  check("opq_cache_copy_pages",
        opq_cache_copy_pages(&r.c, count, static_cast<const int32_t*>(ps),
                             static_cast<const int32_t*>(pd), on.stream()));
  cache_written(a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------- pages

// The tuple of results: tensors made here, or (where given) objects passed in.
template <size_t N>
PyObject* tuple_of(Tensor (&t)[N], PyObject* const (&given)[N]) {
  PyObject* all = PyTuple_New(N);
  for (size_t i = 0; all && i < N; ++i) {
    PyObject* o = given[i];
    if (o) {
      Py_INCREF(o);
      written(t[i]);
    } else {
      o = THPVariable_Wrap(std::move(t[i]));
    }
    if (!o) Py_CLEAR(all);
    else PyTuple_SET_ITEM(all, i, o);
  }
  return all;
}

const Tensor& page_table_of(PyObject* o) {
  const Tensor& t = tensor_of(o, "page_table");
  TORCH_CHECK_VALUE(t.dim() == 2, "page_table must be [rows, columns]");
  dense(t, "page_table", at::kInt, t.sizes(), t.device());
  return t;
}

int32_t* ints(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// Two dense tensors that share bytes.
bool share(const Tensor& a, const Tensor& b) {
  const char* pa = static_cast<const char*>(a.data_ptr());
  const char* pb = static_cast<const char*>(b.data_ptr());
  return a.nbytes() && b.nbytes() && pa < pb + b.nbytes() && pb < pa + a.nbytes();
}

// page_table, lens, pages, page, out or None, workspace or None -> (table, missing)
PyObject* pages_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Tensor& table = page_table_of(a[0]);
  const int64_t rows = table.size(0), columns = table.size(1), pages = int_of(a[2]);
  const Tensor& lens = tensor_of(a[1], "lens");
  const void* pl = dense(lens, "lens", at::kInt, {rows}, table.device());
  const OnDevice on(table);
  Tensor t[2];
  PyObject* given[2] = {nullptr, nullptr};
  if (a[4] == Py_None) {
    t[0] = fresh(table.sizes(), at::kInt, table);
  } else {
    t[0] = tensor_of(given[0] = a[4], "out");
    dense(t[0], "out", at::kInt, table.sizes(), table.device());
    TORCH_CHECK_VALUE(t[0].data_ptr() == table.data_ptr() || !share(t[0], table),
                      "out must be page_table itself or share no memory with it");
    TORCH_CHECK_VALUE(!share(t[0], lens), "out must not share memory with lens");
  }
  t[1] = fresh({1}, at::kInt, table);
  size_t bytes = opq_pages_workspace_bytes(rows, pages);
  const Tensor ws = workspace_of(a[5], &bytes, table);
  check("opq_pages_resize",
        opq_pages_resize(ints(table), static_cast<const int32_t*>(pl), rows, columns, pages,
                         int_of(a[3]), ints(t[0]), ints(t[1]), ws.defined() ? ws.data_ptr() : nullptr,
                         ws.defined() ? bytes : 0, on.stream()));
  return tuple_of(t, given);
  END_HANDLE_TH_ERRORS
}

// page_table, lens, parents, pages, page, out or None, workspace or None
// -> (table, lens, src, dst, missing)
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor& table = page_table_of(a[0]);
  const int64_t rows = table.size(0), columns = table.size(1), pages = int_of(a[3]);
  const Tensor& lens = tensor_of(a[1], "lens");
  const void* pl = dense(lens, "lens", at::kInt, {rows}, table.device());
  const Tensor& parents = tensor_of(a[2], "parents");
  TORCH_CHECK_VALUE(parents.dim() == 1, "parents must be [new rows]");
  const int64_t made = parents.size(0);
  const void* pp = dense(parents, "parents", at::kInt, {made}, table.device());
  const OnDevice on(table);
  Tensor t[5];
  PyObject* given[5] = {};
  if (a[5] == Py_None) {
    t[0] = fresh({made, columns}, at::kInt, table);
  } else {
    t[0] = tensor_of(given[0] = a[5], "out");
    dense(t[0], "out", at::kInt, {made, columns}, table.device());
    TORCH_CHECK_VALUE(!share(t[0], table) && !share(t[0], lens) && !share(t[0], parents),
                      "out must not share memory with page_table, lens or parents: rows are copied from rows");
  }
  for (int i = 1; i < 4; ++i) t[i] = fresh({made}, at::kInt, table);
  t[4] = fresh({1}, at::kInt, table);
  size_t bytes = opq_pages_workspace_bytes(made, pages);
  const Tensor ws = workspace_of(a[6], &bytes, table);
  check("opq_pages_fork",
        opq_pages_fork(ints(table), static_cast<const int32_t*>(pl), rows, columns,
                       static_cast<const int32_t*>(pp), made, pages, int_of(a[4]), ints(t[0]),
                       ints(t[1]), ints(t[2]), ints(t[3]), ints(t[4]),
                       ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? bytes : 0, on.stream()));
  return tuple_of(t, given);
  END_HANDLE_TH_ERRORS
}

// page_table, pages, out or None, workspace or None -> (table, src, dst, used)
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor& table = page_table_of(a[0]);
  const int64_t rows = table.size(0), columns = table.size(1), pages = int_of(a[1]);
  const OnDevice on(table);
  Tensor t[4];
  PyObject* given[4] = {};
  if (a[2] == Py_None) {
    t[0] = fresh(table.sizes(), at::kInt, table);
  } else {
    t[0] = tensor_of(given[0] = a[2], "out");
    dense(t[0], "out", at::kInt, table.sizes(), table.device());
    TORCH_CHECK_VALUE(t[0].data_ptr() == table.data_ptr() || !share(t[0], table),
                      "out must be page_table itself or share no memory with it");
  }
  const int64_t moves = std::max<int64_t>(0, std::min(pages / 2, rows * columns));
  t[1] = fresh({moves}, at::kInt, table);
  t[2] = fresh({moves}, at::kInt, table);
  t[3] = fresh({1}, at::kInt, table);
  size_t bytes = opq_pages_workspace_bytes(rows, pages);
  const Tensor ws = workspace_of(a[3], &bytes, table);
  check("opq_pages_compact",
        opq_pages_compact(ints(table), rows, columns, pages, ints(t[0]), ints(t[1]), ints(t[2]),
                          ints(t[3]), ws.defined() ? ws.data_ptr() : nullptr,
                          ws.defined() ? bytes : 0, on.stream()));
  return tuple_of(t, given);
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ drafts

// probs, tokens, uniforms, draft_probs or None, parents or None, counts or None, workspace or None
// -> (kept, count, next)
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor& p = rows(a[0], "probs", 3);
  const int dtype = dtype_of(p.scalar_type(), "probs");
  const int64_t batch = p.size(0), draft = p.size(1), vocab = p.size(2);
  const c10::Device dev = p.device();
  const void* tokens = dense(a[1], "tokens", at::kInt, {batch, draft}, dev);
  const Tensor& u = plain(tensor_of(a[2], "uniforms"), "uniforms");
  const void* uniforms = dense(u, "uniforms", at::kFloat, {batch, draft}, dev);
  Tensor q;
  if (a[3] != Py_None) {
    q = rows(a[3], "draft_probs", 3);
    TORCH_CHECK_VALUE(q.size(0) == batch && q.size(1) == draft - 1 && q.size(2) == vocab,
                      "draft_probs must be [", batch, ", ", draft - 1, ", ", vocab, "], got ", q.sizes());
    TORCH_CHECK_VALUE(q.scalar_type() == p.scalar_type(), "draft_probs must be ", p.scalar_type(), " as probs, got ",
                      q.scalar_type());
    TORCH_CHECK_VALUE(q.device() == dev, "draft_probs must be on ", dev, ", got ", q.device());
    TORCH_CHECK_VALUE(a[4] == Py_None, "draft_probs go with a chain, not with parents");
  }
  const void* parents = a[4] == Py_None ? nullptr : dense(a[4], "parents", at::kInt, {batch, draft}, dev);
  const void* counts = a[5] == Py_None ? nullptr : dense(a[5], "counts", at::kInt, {batch}, dev);
  const OnDevice on(p);
  Tensor t[3] = {fresh({batch, draft}, at::kInt, p), fresh({batch}, at::kInt, p), fresh({batch}, at::kInt, p)};
  size_t bytes = opq_verify_drafts_workspace_bytes(batch, vocab);
  const Tensor ws = workspace_of(a[6], &bytes, p);
  // a draft of one token has no draft probabilities to point to
  const bool drawn = q.defined() && q.numel() > 0;
  check("opq_verify_drafts",
        opq_verify_drafts(p.data_ptr(), dtype, batch, draft, vocab, p.stride(0), p.stride(1),
                          static_cast<const int32_t*>(tokens), static_cast<const float*>(uniforms),
                          drawn ? q.data_ptr() : nullptr, drawn ? q.stride(0) : 0, drawn ? q.stride(1) : 0,
                          static_cast<const int32_t*>(parents), static_cast<const int32_t*>(counts), ints(t[0]),
                          ints(t[1]), ints(t[2]), ws.defined() ? ws.data_ptr() : nullptr,
                          ws.defined() ? bytes : 0, on.stream()));
  PyObject* none[3] = {};
  return tuple_of(t, none);
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
                          {"cache_copy_pages", FAST(cache_copy_pages), METH_FASTCALL, nullptr},
                          {"pages_resize", FAST(pages_resize), METH_FASTCALL, nullptr},
                          {"pages_fork", FAST(pages_fork), METH_FASTCALL, nullptr},
                          {"pages_compact", FAST(pages_compact), METH_FASTCALL, nullptr},
                          {"verify_drafts", FAST(verify_drafts), METH_FASTCALL, nullptr},
                          {"attention", FAST(attention), METH_FASTCALL, nullptr},
                          {"lowrank_add", FAST(lowrank_add), METH_FASTCALL, nullptr},
                          {"lowrank_backward", FAST(lowrank_backward), METH_FASTCALL, nullptr},
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention() { return PyModule_Create(&kModule); }
