// The C ABI of the adapters (include/opq_adapters.h): argument checks in the
// documented order, host tables, then the launches on the caller's stream.
#include "opq_adapters.h"

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "adapters_internal.hpp"
#include "opq_internal.hpp"

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 22;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxElements = int64_t(1) << 39;
constexpr int64_t kMaxLinear = 65536;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned4(const void* p) { return aligned(p, 4); }
bool aligned16(const void* p) { return aligned(p, 16); }
bool dtype_ok(int d) { return d == OPQ_F32 || d == OPQ_BF16; }
int hip_status(hipError_t e) { return e == hipSuccess ? OPQ_OK : OPQ_ERR_HIP; }

bool sizes_ok(int64_t m, int64_t k, int64_t n, int64_t rank) {
  return m >= 0 && k >= 8 && k % 8 == 0 && n >= 8 && n % 8 == 0 && rank >= 8 && rank <= 128 &&
         rank % 8 == 0;
}
// Rows of an output must not overlap; an input's may be the same.
bool in_stride_ok(int64_t s, int64_t width) { return s == 0 || s >= width; }
bool sizes_supported(int64_t m, int64_t k, int64_t n) {
  return m <= kMaxTokens && k <= kMaxWidth && n <= kMaxWidth;
}
bool within(int64_t m, int64_t stride) { return m == 0 || stride <= kMaxElements / m; }

}  // namespace

extern "C" {

size_t opq_lowrank_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank) {
  if (!sizes_ok(m, k, n, rank) || !sizes_supported(m, k, n) || m == 0) return 0;
  return opq::lowrank_workspace_bytes(m, k, n, rank);
}

int opq_lowrank_add(const opq_lowrank* adapters, const uint16_t* x, int64_t x_stride,
                    const int32_t* index, int64_t m, const void* y, int64_t y_stride, int y_dtype,
                    void* out, int64_t out_stride, int out_dtype, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!adapters) return OPQ_ERR_NULL;
  const opq_lowrank& a = *adapters;
  if ((a.count > 0 && (!a.down || !a.up || !a.scale)) || (m > 0 && (!x || !index || !out)))
    return OPQ_ERR_NULL;
  if (!sizes_ok(m, a.k, a.n, a.rank) || a.count < 0 || !in_stride_ok(x_stride, a.k) ||
      (y && !in_stride_ok(y_stride, a.n)) || out_stride < a.n)
    return OPQ_ERR_SHAPE;
  if (!aligned16(a.down) || !aligned16(a.up) || !aligned4(a.scale) || !aligned16(x) ||
      !aligned4(index) || !aligned16(y) || !aligned16(out) || !aligned16(workspace) ||
      x_stride % 8 || (y && y_stride % 8) || out_stride % 8)
    return OPQ_ERR_ALIGN;
  if ((y && !dtype_ok(y_dtype)) || !dtype_ok(out_dtype)) return OPQ_ERR_DTYPE;
  const size_t need = opq_lowrank_workspace_bytes(m, a.k, a.n, a.rank);
  if (workspace_bytes < need || (need > 0 && !workspace)) return OPQ_ERR_WORKSPACE;
  if (!sizes_supported(m, a.k, a.n) || a.count > (int64_t(1) << 30) || !within(m, x_stride) ||
      (y && !within(m, y_stride)) || !within(m, out_stride))
    return OPQ_ERR_UNSUPPORTED;
  if (m > 0 && y == out && ((m > 1 && y_stride != out_stride) || y_dtype != out_dtype)) return OPQ_ERR_UNSUPPORTED;
  if (m == 0) return OPQ_OK;
  opq::LowrankAdd c{};
  c.a = a;
  c.x = x;
  c.x_stride = x_stride;
  c.index = index;
  c.m = m;
  c.y = y;
  c.y_stride = y_stride;
  c.y_bf16 = y && y_dtype == OPQ_BF16;
  c.out = out;
  c.out_stride = out_stride;
  c.out_bf16 = out_dtype == OPQ_BF16;
  c.workspace = workspace;
  return hip_status(opq::launch_lowrank_add(c, static_cast<hipStream_t>(stream)));
}

size_t opq_lowrank_backward_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank,
                                            int64_t count) {
  if (!sizes_ok(m, k, n, rank) || !sizes_supported(m, k, n) || count < 0 || count > opq::kMaxTrained)
    return 0;
  return opq::lowrank_backward_workspace_bytes(m, k, n, rank, count);
}

int opq_lowrank_backward(const opq_lowrank* adapters, const uint16_t* dy, int64_t dy_stride,
                         const uint16_t* x, int64_t x_stride, const int32_t* index, int64_t m,
                         const void* dx, int64_t dx_stride, int dx_dtype, void* dx_out,
                         int64_t dx_out_stride, void* d_down, void* d_up, int grad_dtype,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!adapters) return OPQ_ERR_NULL;
  const opq_lowrank& a = *adapters;
  if ((a.count > 0 && (!a.down || !a.up || !a.scale || !d_down != !d_up)) ||
      (m > 0 && (!dy || !x || !index)))
    return OPQ_ERR_NULL;
  if (!sizes_ok(m, a.k, a.n, a.rank) || a.count < 0 || !in_stride_ok(dy_stride, a.n) ||
      !in_stride_ok(x_stride, a.k) || (dx && !in_stride_ok(dx_stride, a.k)) ||
      (dx_out && dx_out_stride < a.k))
    return OPQ_ERR_SHAPE;
  if (!aligned16(a.down) || !aligned16(a.up) || !aligned4(a.scale) || !aligned16(dy) ||
      !aligned16(x) || !aligned4(index) || !aligned16(dx) || !aligned16(dx_out) ||
      !aligned16(d_down) || !aligned16(d_up) || !aligned16(workspace) || dy_stride % 8 ||
      x_stride % 8 || (dx && dx_stride % 8) || (dx_out && dx_out_stride % 8))
    return OPQ_ERR_ALIGN;
  if ((dx_out && !dtype_ok(dx_dtype)) || (d_down && !dtype_ok(grad_dtype))) return OPQ_ERR_DTYPE;
  const size_t need = opq_lowrank_backward_workspace_bytes(m, a.k, a.n, a.rank, a.count);
  if (workspace_bytes < need || (need > 0 && !workspace)) return OPQ_ERR_WORKSPACE;
  if (!sizes_supported(m, a.k, a.n) || a.count > opq::kMaxTrained || !within(m, dy_stride) ||
      !within(m, x_stride) || (dx && !within(m, dx_stride)) || (dx_out && !within(m, dx_out_stride)))
    return OPQ_ERR_UNSUPPORTED;
  if (m > 1 && dx_out && dx == dx_out && dx_stride != dx_out_stride) return OPQ_ERR_UNSUPPORTED;
  if ((m == 0 || !dx_out) && (a.count == 0 || !d_down)) return OPQ_OK;
  opq::LowrankBackward c{};
  c.a = a;
  c.dy = dy;
  c.dy_stride = dy_stride;
  c.x = x;
  c.x_stride = x_stride;
  c.index = index;
  c.m = m;
  c.dx = dx;
  c.dx_stride = dx_stride;
  c.dx_bf16 = dx_dtype == OPQ_BF16;
  c.dx_out = m > 0 ? dx_out : nullptr;
  c.dx_out_stride = dx_out_stride;
  c.d_down = a.count > 0 ? d_down : nullptr;
  c.d_up = a.count > 0 ? d_up : nullptr;
  c.grad_bf16 = grad_dtype == OPQ_BF16;
  c.workspace = workspace;
  return hip_status(opq::launch_lowrank_backward(c, static_cast<hipStream_t>(stream)));
}

// ---------------------------------------------------------- projection's gradient

namespace {

// The workspace's parts, for 4-bit codes or for those of other widths: W' transposed ([k][ld]) at
// its beginning and, for other widths, W' as it is dequantized, neither where few tokens take
// 4-bit codes as they are; dy with rows of ld where its own are shorter than what is read; sums
// that are split.  Sizes are whole MiB, one at least.
struct BackwardSpace {
  int64_t ld;
  size_t padded, part, plain, bytes;
};
BackwardSpace backward_space(int64_t m, int64_t n, int64_t k, bool codes) {
  constexpr size_t kMiB = size_t(1) << 20;
  const opq::BackwardShort few = opq::backward_short_plan(m, n, k);
  const bool direct = codes && few.taken;
  BackwardSpace s;
  s.ld = n % 32 ? (n + 63) / 64 * 64 : n;  // padded rows: whole steps of the product
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~size_t(255);
    return here;
  };
  take(direct ? 0 : (size_t)k * s.ld * 2);
  s.padded = take((direct ? n % 8 != 0 : n < s.ld) ? (size_t)m * s.ld * 2 : 0);
  s.part = take(direct ? few.part_bytes : opq::linear_dense_part_bytes(m, k, s.ld));
  s.plain = take(codes ? 0 : (size_t)n * k * 2);
  s.bytes = std::max(kMiB, (at + kMiB - 1) & ~(kMiB - 1));
  return s;
}

bool backward_sizes_ok(int64_t m, int64_t n, int64_t k) {
  return m > 0 && n > 0 && k > 0 && k % 32 == 0 && m <= kMaxTokens && n <= kMaxLinear && k <= kMaxLinear;
}

}  // namespace

size_t opq_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (!backward_sizes_ok(m, n, k)) return 0;
  return std::max(backward_space(m, n, k, true).bytes, backward_space(m, n, k, false).bytes);
}

size_t opq_linear_backward_codes_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return backward_sizes_ok(m, n, k) ? backward_space(m, n, k, true).bytes : 0;
}

// The checks of one storage form; `more` its own about shapes and types.
static int backward_checks(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                           const void* scale, int64_t m, int64_t n, int64_t k, float alpha,
                           bool more_shape_ok, bool codes, const void* dx, int dx_dtype,
                           const void* workspace, size_t workspace_bytes) {
  if ((m > 0 && n > 0 && !dy) || (n > 0 && k > 0 && (!packed || !sign || !scale)) ||
      (m > 0 && k > 0 && !dx))
    return OPQ_ERR_NULL;
  if (m < 0 || n < 0 || k < 0 || k % 32 || !more_shape_ok) return OPQ_ERR_SHAPE;
  if (!(std::isfinite(alpha) && alpha > 0.0f)) return OPQ_ERR_ALPHA;
  if (!aligned16(dy) || !aligned16(packed) || !aligned16(sign) || !aligned16(scale) ||
      !aligned16(dx) || !aligned16(workspace))
    return OPQ_ERR_ALIGN;
  if (!dtype_ok(dx_dtype)) return OPQ_ERR_DTYPE;
  const size_t need = codes ? opq_linear_backward_codes_workspace_bytes(m, n, k)
                            : opq_linear_backward_workspace_bytes(m, n, k);
  if (workspace_bytes < need || (need > 0 && !workspace)) return OPQ_ERR_WORKSPACE;
  if (m > kMaxTokens || n > kMaxLinear || k > kMaxLinear) return OPQ_ERR_UNSUPPORTED;
  return OPQ_OK;
}

// dy with rows as the kernels read them: its own, or copied to rows of ld.
static int backward_rows(const uint16_t** dy, int64_t* ldy, int64_t m, int64_t n, const BackwardSpace& s,
                         char* ws, hipStream_t st) {
  *ldy = n;
  if (n == s.ld) return OPQ_OK;
  uint16_t* padded = reinterpret_cast<uint16_t*>(ws + s.padded);
  const int e = hip_status(opq::launch_pad_rows(*dy, m, n, padded, s.ld, st));
  *dy = padded;
  *ldy = s.ld;
  return e;
}

// The product, with W' transposed at the workspace's beginning (n > 0).
static int backward_product(const uint16_t* dy, int64_t m, int64_t n, int64_t k, void* dx, int dx_dtype,
                            const BackwardSpace& s, char* ws, hipStream_t st) {
  int64_t ldy;
  const int e = backward_rows(&dy, &ldy, m, n, s, ws, st);
  if (e != OPQ_OK) return e;
  float* part = opq::linear_dense_part_bytes(m, k, s.ld) ? reinterpret_cast<float*>(ws + s.part) : nullptr;
  return hip_status(opq::launch_linear_dense(dy, reinterpret_cast<const uint16_t*>(ws), nullptr, m, k, s.ld, dx,
                                             dx_dtype == OPQ_BF16, part, st));
}

// 4-bit codes, one max a row or a group (gs > 0), n > 0.
static int backward_codes(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                          const float* scale, const uint16_t* scale16, int64_t m, int64_t n, int64_t k,
                          int gs, const opq::Levels& lv, void* dx, int dx_dtype, char* ws, hipStream_t st) {
  const BackwardSpace s = backward_space(m, n, k, true);
  if (opq::backward_short_plan(m, n, k).taken) {
    int64_t ldy = n;
    const int e = n % 8 ? backward_rows(&dy, &ldy, m, n, s, ws, st) : OPQ_OK;
    if (e != OPQ_OK) return e;
    return hip_status(opq::launch_backward_short(dy, ldy, packed, sign, scale, scale16, m, n, k, gs, lv, dx,
                                                 dx_dtype == OPQ_BF16, reinterpret_cast<float*>(ws + s.part), st));
  }
  const int e = hip_status(opq::launch_dequantize_transposed(packed, sign, scale, scale16, n, k, gs, lv,
                                                             reinterpret_cast<uint16_t*>(ws), s.ld, st));
  if (e != OPQ_OK) return e;
  return backward_product(dy, m, n, k, dx, dx_dtype, s, ws, st);
}

// No rows of weights: sums of nothing.
static int no_rows(int64_t m, int64_t k, void* dx, int dx_dtype, hipStream_t st) {
  return hip_status(opq::launch_linear_dense(nullptr, nullptr, nullptr, m, k, 0, dx, dx_dtype == OPQ_BF16, nullptr, st));
}

int opq_linear_backward(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                        const float* scale, int64_t m, int64_t n, int64_t k, float alpha, void* dx,
                        int dx_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int e = backward_checks(dy, packed, sign, scale, m, n, k, alpha, true, true, dx, dx_dtype, workspace,
                          workspace_bytes);
  if (e != OPQ_OK || m == 0 || k == 0) return e;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (n == 0) return no_rows(m, k, dx, dx_dtype, st);
  opq::Levels lv;
  opq::levels(alpha, lv.g);
  return backward_codes(dy, packed, sign, scale, nullptr, m, n, k, 0, lv, dx, dx_dtype,
                        static_cast<char*>(workspace), st);
}

int opq_linear_backward_bits(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                             const float* scale, int64_t m, int64_t n, int64_t k, int bits,
                             float alpha, void* dx, int dx_dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int e = backward_checks(dy, packed, sign, scale, m, n, k, alpha, bits >= 3 && bits <= 6, bits == 4, dx,
                          dx_dtype, workspace, workspace_bytes);
  if (e != OPQ_OK || m == 0 || k == 0) return e;
  if (bits == 4)
    return opq_linear_backward(dy, packed, sign, scale, m, n, k, alpha, dx, dx_dtype, workspace,
                               workspace_bytes, stream);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (n == 0) return no_rows(m, k, dx, dx_dtype, st);
  char* ws = static_cast<char*>(workspace);
  const BackwardSpace s = backward_space(m, n, k, false);
  uint16_t* w = reinterpret_cast<uint16_t*>(ws + s.plain);
  e = opq_dequantize_bits(packed, sign, scale, n, k, bits, alpha, w, stream);
  if (e != OPQ_OK) return e;
  e = hip_status(opq::launch_transpose(w, n, k, reinterpret_cast<uint16_t*>(ws), s.ld, st));
  if (e != OPQ_OK) return e;
  return backward_product(dy, m, n, k, dx, dx_dtype, s, ws, st);
}

int opq_linear_backward_grouped(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                                const uint16_t* scale16, int64_t m, int64_t n, int64_t k,
                                int64_t group, float alpha, void* dx, int dx_dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const bool group_ok = (group == 32 || group == 64 || group == 128 || group == 256) && k % group == 0;
  int e = backward_checks(dy, packed, sign, scale16, m, n, k, alpha, group_ok, true, dx, dx_dtype,
                          workspace, workspace_bytes);
  if (e != OPQ_OK || m == 0 || k == 0) return e;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (n == 0) return no_rows(m, k, dx, dx_dtype, st);
  opq::DecisionPoints dp;
  if (!opq::decision_points(alpha, dp.t)) return OPQ_ERR_ALPHA;
  opq::Levels lv;
  opq::levels(alpha, lv.g);
  if (!opq::grouped_supported(dp, lv)) return OPQ_ERR_UNSUPPORTED;
  return backward_codes(dy, packed, sign, nullptr, scale16, m, n, k, (int)group, lv, dx, dx_dtype,
                        static_cast<char*>(workspace), st);
}

}  // extern "C"
