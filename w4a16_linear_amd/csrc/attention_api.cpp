// The C ABI of the attention side (include/opq_attention.h): argument checks
// in the documented order, host tables, then the launches on the caller's stream.
#include "opq_attention.h"

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "attention_internal.hpp"
#include "opq_internal.hpp"

namespace {

constexpr double kPi = 3.14159265358979323846;
constexpr int64_t kMaxElements = int64_t(1) << 39;
constexpr int64_t kMaxInt = 0x7FFFFFFF;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned4(const void* p) { return aligned(p, 4); }
bool aligned16(const void* p) { return aligned(p, 16); }
int hip_status(hipError_t e) { return e == hipSuccess ? OPQ_OK : OPQ_ERR_HIP; }
bool dtype_ok(int d) { return d == OPQ_F32 || d == OPQ_BF16; }

// a * b * c within `most`, for a, b, c >= 0
bool product_within(int64_t a, int64_t b, int64_t c, int64_t most) {
  if (a == 0 || b == 0 || c == 0) return true;
  return a <= most && b <= most / a && c <= most / (a * b);
}

// nearest bfloat16 (ties to even) of a level in [0, 1], from binary64 in one rounding
uint32_t bf16_of_level(double g) {
  if (!(g > 0.0)) return 0u;
  int e;
  const double f = std::frexp(g, &e);                 // g = f 2^e, f in [0.5, 1)
  if (e < -125) return 0u;                            // below the smallest normal bfloat16
  const double k = std::nearbyint(std::ldexp(f, 8));  // 128 .. 256, ties to even
  const float r = (float)std::ldexp(k, e - 8);
  uint32_t b;
  std::memcpy(&b, &r, 4);
  return b >> 16;
}

opq::LevelPlanes level_planes(float alpha) {
  opq::LevelPlanes p{};
  double g[16];
  opq::levels(alpha, g);
  for (int q = 0; q < 16; ++q) {
    const uint32_t e = bf16_of_level(g[q]);
    p.lo[q >> 2] |= (e & 0xFFu) << (8 * (q & 3));
    p.hi[q >> 2] |= (e >> 8) << (8 * (q & 3));
  }
  return p;
}

bool page_ok(int64_t page) { return page >= 16 && (page & (page - 1)) == 0; }

// The parts of a cache's checks, in the header's order.
bool cache_null(const opq_cache* c) {
  if (!c) return true;
  const bool some = c->pages > 0 && c->heads > 0 && c->page > 0;
  if (some && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return true;
  return some && c->format == OPQ_CACHE_OPQ4 && (!c->k_sign || !c->v_sign);
}
bool cache_shape_ok(const opq_cache& c) {
  return c.pages >= 0 && c.heads > 0 && page_ok(c.page) &&
         (c.dim == 64 || c.dim == 128 || c.dim == 256);
}
bool cache_alpha_ok(const opq_cache& c) {
  return c.format != OPQ_CACHE_OPQ4 || (c.alpha >= 0.05f && c.alpha <= 60.0f);
}
bool cache_aligned(const opq_cache& c) {
  return aligned16(c.k) && aligned16(c.v) && aligned16(c.k_scale) && aligned16(c.v_scale) &&
         aligned16(c.k_sign) && aligned16(c.v_sign);
}
bool format_ok(int f) { return f == OPQ_CACHE_BF16 || f == OPQ_CACHE_FP8 || f == OPQ_CACHE_OPQ4; }
bool cache_supported(const opq_cache& c) {
  return product_within(c.pages, c.page, 1, kMaxInt) && c.heads <= 65535;
}

}  // namespace

extern "C" {

int opq_rotary_frequencies(int64_t rot, double base, int scaling, double factor,
                           double original_len, double beta_fast, double beta_slow, double* out_f,
                           double* out_amplitude) {
  if (!out_f || !out_amplitude) return OPQ_ERR_NULL;
  if (rot < 2 || rot > 1024 || rot % 2) return OPQ_ERR_SHAPE;
  if (!std::isfinite(base) || base <= 1.0) return OPQ_ERR_ALPHA;
  const bool scaled = scaling != OPQ_ROPE_NONE;
  if (scaled && (!std::isfinite(factor) || factor < 1.0)) return OPQ_ERR_ALPHA;
  const bool yarn = scaling == OPQ_ROPE_YARN;
  if (yarn && !(std::isfinite(original_len) && original_len > 0.0 && std::isfinite(beta_fast) &&
                beta_slow >= 0.0 && beta_fast > beta_slow))
    return OPQ_ERR_ALPHA;
  if (scaling < OPQ_ROPE_NONE || scaling > OPQ_ROPE_YARN) return OPQ_ERR_DTYPE;
  if (scaling == OPQ_ROPE_NTK && rot > 2)
    base *= std::pow(factor, (double)rot / (double)(rot - 2));
  for (int64_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * (double)i / (double)rot);
    if (scaling == OPQ_ROPE_LINEAR) f /= factor;
    if (yarn) {
      const double turns = original_len * f / (2.0 * kPi);
      double keep = (turns - beta_slow) / (beta_fast - beta_slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      f = keep * f + (1.0 - keep) * f / factor;
    }
    out_f[i] = f;
  }
  *out_amplitude = yarn ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return OPQ_OK;
}

int opq_rotary_table(const double* freq, int64_t pairs, int64_t len, double amplitude,
                     float* table, void* stream) {
  if (!freq || (len > 0 && !table)) return OPQ_ERR_NULL;
  if (pairs < 1 || pairs > 512 || len < 0) return OPQ_ERR_SHAPE;
  if (!aligned16(freq) || !aligned16(table)) return OPQ_ERR_ALIGN;
  if (!product_within(len, pairs, 1, kMaxElements)) return OPQ_ERR_UNSUPPORTED;
  if (len == 0) return OPQ_OK;
  return hip_status(opq::launch_rotary_table(freq, pairs, len, amplitude, table,
                                             static_cast<hipStream_t>(stream)));
}

int opq_rotary(const void* x, int dtype, int64_t tokens, int64_t heads, int64_t dim,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
               int64_t axes, const int32_t* sections, const float* table, int64_t table_len,
               int64_t rot, int layout, int backward, void* out, int64_t out_token_stride,
               int64_t out_head_stride, void* stream) {
  const bool some = tokens > 0 && heads > 0;
  if (!sections || (some && (!x || !out || !positions || (table_len > 0 && !table))))
    return OPQ_ERR_NULL;
  if (tokens < 0 || heads < 0 || dim < 1 || dim > 65536 || rot < 2 || rot > dim || rot > 1024 ||
      rot % 2 || axes < 1 || axes > opq::kMaxAxes || table_len < 0)
    return OPQ_ERR_SHAPE;
  opq::RotaryArgs a{};
  int64_t end = 0;
  for (int64_t i = 0; i < axes; ++i) {
    if (sections[i] < 1) return OPQ_ERR_SHAPE;
    end += sections[i];
    a.end[i] = (int)(end < kMaxInt ? end : kMaxInt);
  }
  if (end != rot / 2) return OPQ_ERR_SHAPE;
  const uintptr_t element = dtype == OPQ_F32 ? 4 : 2;
  if (!aligned(x, element) || !aligned(out, element) || !aligned4(positions) || !aligned16(table))
    return OPQ_ERR_ALIGN;
  if (!dtype_ok(dtype) || (layout != OPQ_ROTARY_HALF && layout != OPQ_ROTARY_INTERLEAVED))
    return OPQ_ERR_DTYPE;
  if (!product_within(heads, dim, 1, int64_t(1) << 30) ||
      !product_within(tokens, heads, dim, kMaxElements))
    return OPQ_ERR_UNSUPPORTED;
  if (!some) return OPQ_OK;
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.table = table;
  a.x_token = x_token_stride;
  a.x_head = x_head_stride;
  a.out_token = out_token_stride;
  a.out_head = out_head_stride;
  a.tokens = tokens;
  a.table_len = table_len;
  a.heads = (int)heads;
  a.dim = (int)dim;
  a.rot = (int)rot;
  a.axes = (int)axes;
  a.turn = backward ? -1.0f : 1.0f;
  return hip_status(opq::launch_rotary(a, dtype == OPQ_BF16, layout == OPQ_ROTARY_INTERLEAVED,
                                       static_cast<hipStream_t>(stream)));
}

int opq_cache_write(const opq_cache* cache, const void* k, int64_t k_token_stride,
                    int64_t k_head_stride, const void* v, int64_t v_token_stride,
                    int64_t v_head_stride, int dtype, int64_t tokens, const int32_t* slots,
                    void* stream) {
  if (cache_null(cache) || (tokens > 0 && (!k || !v || !slots))) return OPQ_ERR_NULL;
  const opq_cache& c = *cache;
  if (!cache_shape_ok(c) || tokens < 0) return OPQ_ERR_SHAPE;
  if (!cache_alpha_ok(c)) return OPQ_ERR_ALPHA;
  const uintptr_t element = dtype == OPQ_F32 ? 4 : 2;
  if (!cache_aligned(c) || !aligned(k, element) || !aligned(v, element) || !aligned4(slots))
    return OPQ_ERR_ALIGN;
  if (!dtype_ok(dtype) || !format_ok(c.format)) return OPQ_ERR_DTYPE;
  if (!cache_supported(c) || !product_within(tokens, c.heads, 1, kMaxInt))
    return OPQ_ERR_UNSUPPORTED;
  if (tokens == 0 || c.pages == 0) return OPQ_OK;
  opq::CacheCodes cc{};
  if (c.format == OPQ_CACHE_OPQ4) {
    if (!opq::decision_points(c.alpha, cc.t)) return OPQ_ERR_ALPHA;
    cc.alpha = c.alpha;
    // Error of 15 u^alpha through log2 and exp2 in binary32: at most about
    // 8e-6 + 8e-6 alpha (an ulp each of log2, its product with alpha, exp2 and the
    // final sum, 3 ulps of |x| fl(1/m)).  The guard is three times that: it decides
    // how many elements take the slow way (5 % of the waves for alpha = 0.73).
    cc.guard = 3e-5f + 2.5e-5f * c.alpha;
  }
  const opq::CacheRows side[2] = {{k, k_token_stride, k_head_stride, c.k, c.k_sign, c.k_scale},
                                  {v, v_token_stride, v_head_stride, c.v, c.v_sign, c.v_scale}};
  return hip_status(opq::launch_cache_write(side, c, dtype == OPQ_BF16, tokens, slots, cc,
                                            static_cast<hipStream_t>(stream)));
}

int opq_cache_read(const opq_cache* cache, int64_t tokens, const int32_t* slots, void* k_out,
                   void* v_out, int dtype, void* stream) {
  if (cache_null(cache) || (tokens > 0 && (!k_out || !v_out || !slots))) return OPQ_ERR_NULL;
  const opq_cache& c = *cache;
  if (!cache_shape_ok(c) || tokens < 0) return OPQ_ERR_SHAPE;
  if (!cache_alpha_ok(c)) return OPQ_ERR_ALPHA;
  if (!cache_aligned(c) || !aligned16(k_out) || !aligned16(v_out) || !aligned4(slots))
    return OPQ_ERR_ALIGN;
  if (!dtype_ok(dtype) || !format_ok(c.format)) return OPQ_ERR_DTYPE;
  if (!cache_supported(c) || !product_within(tokens, c.heads, 1, kMaxInt))
    return OPQ_ERR_UNSUPPORTED;
  if (tokens == 0) return OPQ_OK;
  opq::LevelPlanes lp{};
  if (c.format == OPQ_CACHE_OPQ4) lp = level_planes(c.alpha);
  const opq::CacheRows side[2] = {{k_out, 0, 0, c.k, c.k_sign, c.k_scale},
                                  {v_out, 0, 0, c.v, c.v_sign, c.v_scale}};
  return hip_status(opq::launch_cache_read(side, c, dtype == OPQ_BF16, tokens, slots, lp,
                                           static_cast<hipStream_t>(stream)));
}

int opq_cache_move(const opq_cache* cache, int64_t batch, int64_t count, const int32_t* src,
                   const int32_t* dst, void* stream) {
  if (cache_null(cache) || (batch > 0 && count > 0 && (!src || !dst))) return OPQ_ERR_NULL;
  const opq_cache& c = *cache;
  if (!cache_shape_ok(c) || batch < 0 || count < 0) return OPQ_ERR_SHAPE;
  if (!cache_alpha_ok(c)) return OPQ_ERR_ALPHA;
  if (!cache_aligned(c) || !aligned4(src) || !aligned4(dst)) return OPQ_ERR_ALIGN;
  if (!format_ok(c.format)) return OPQ_ERR_DTYPE;
  if (!cache_supported(c) || batch > 65535 || count > opq::kMaxMoves ||
      !product_within(batch, c.heads, 2, int64_t(1) << 23))
    return OPQ_ERR_UNSUPPORTED;
  if (batch == 0 || count == 0 || c.pages == 0) return OPQ_OK;
  const bool signs = c.format == OPQ_CACHE_OPQ4;
  const opq::CacheRows side[2] = {{nullptr, 0, 0, c.k, signs ? c.k_sign : nullptr, c.k_scale},
                                  {nullptr, 0, 0, c.v, signs ? c.v_sign : nullptr, c.v_scale}};
  return hip_status(opq::launch_cache_move(side, c, batch, count, src, dst,
                                           static_cast<hipStream_t>(stream)));
}

int opq_cache_copy_pages(const opq_cache* cache, int64_t count, const int32_t* src,
                         const int32_t* dst, void* stream) {
  if (cache_null(cache) || (count > 0 && (!src || !dst))) return OPQ_ERR_NULL;
  const opq_cache& c = *cache;
  if (!cache_shape_ok(c) || count < 0) return OPQ_ERR_SHAPE;
  if (!cache_alpha_ok(c)) return OPQ_ERR_ALPHA;
  if (!cache_aligned(c) || !aligned4(src) || !aligned4(dst)) return OPQ_ERR_ALIGN;
  if (!format_ok(c.format)) return OPQ_ERR_DTYPE;
  if (!cache_supported(c) || count > opq::kMaxPages) return OPQ_ERR_UNSUPPORTED;
  if (count == 0 || c.pages == 0) return OPQ_OK;
  const bool signs = c.format == OPQ_CACHE_OPQ4;
  const opq::CacheRows side[2] = {{nullptr, 0, 0, c.k, signs ? c.k_sign : nullptr, c.k_scale},
                                  {nullptr, 0, 0, c.v, signs ? c.v_sign : nullptr, c.v_scale}};
  return hip_status(opq::launch_cache_copy_pages(side, c, count, src, dst,
                                                 static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------------ pages

constexpr int64_t kMaxPageRows = int64_t(1) << 20;
constexpr int64_t kMaxEntries = int64_t(1) << 28;

size_t opq_pages_workspace_bytes(int64_t rows, int64_t pages) {
  if (rows < 0 || rows > kMaxPageRows || pages < 1 || pages > opq::kMaxPages) return 0;
  return opq::pages_workspace_bytes(rows, pages);
}

// What the three calls check alike, once their pointers are known not to be NULL.
static int pages_checks(int64_t rows, int64_t new_rows, int64_t columns, int64_t pages,
                        const void* workspace, size_t workspace_bytes) {
  const size_t need = opq_pages_workspace_bytes(new_rows, pages);
  if (workspace_bytes < need || (need > 0 && !workspace)) return OPQ_ERR_WORKSPACE;
  if (rows > kMaxPageRows || new_rows > kMaxPageRows || pages > opq::kMaxPages ||
      !product_within(rows, columns, 1, kMaxEntries) ||
      !product_within(new_rows, columns, 1, kMaxEntries))
    return OPQ_ERR_UNSUPPORTED;
  return OPQ_OK;
}

int opq_pages_resize(const int32_t* table, const int32_t* lens, int64_t rows, int64_t columns,
                     int64_t pages, int64_t page, int32_t* out, int32_t* missing, void* workspace,
                     size_t workspace_bytes, void* stream) {
  if (!missing || (rows > 0 && !lens) || (rows > 0 && columns > 0 && (!table || !out)))
    return OPQ_ERR_NULL;
  if (rows < 0 || columns < 0 || pages < 1 || !page_ok(page)) return OPQ_ERR_SHAPE;
  if (!aligned4(table) || !aligned4(lens) || !aligned4(out) || !aligned4(missing) ||
      !aligned16(workspace))
    return OPQ_ERR_ALIGN;
  const int e = pages_checks(rows, rows, columns, pages, workspace, workspace_bytes);
  if (e != OPQ_OK) return e;
  if (page > kMaxInt) return OPQ_ERR_UNSUPPORTED;
  opq::PagesArgs a{};
  a.table = table;
  a.lens = lens;
  a.out = out;
  a.result = missing;
  a.rows = a.new_rows = (int)rows;
  a.columns = (int)columns;
  a.pages = (int)pages;
  a.page = (int)page;
  a.workspace = static_cast<char*>(workspace);
  return hip_status(opq::launch_pages(opq::PagesCall::kResize, a, static_cast<hipStream_t>(stream)));
}

int opq_pages_fork(const int32_t* table, const int32_t* lens, int64_t rows, int64_t columns,
                   const int32_t* parents, int64_t new_rows, int64_t pages, int64_t page,
                   int32_t* out, int32_t* out_lens, int32_t* src, int32_t* dst, int32_t* missing,
                   void* workspace, size_t workspace_bytes, void* stream) {
  if (!missing || (rows > 0 && !lens) || (rows > 0 && columns > 0 && !table) ||
      (new_rows > 0 && (!parents || !out_lens || !src || !dst)) ||
      (new_rows > 0 && columns > 0 && !out))
    return OPQ_ERR_NULL;
  if (rows < 0 || new_rows < 0 || columns < 0 || pages < 1 || !page_ok(page)) return OPQ_ERR_SHAPE;
  if (!aligned4(table) || !aligned4(lens) || !aligned4(parents) || !aligned4(out) ||
      !aligned4(out_lens) || !aligned4(src) || !aligned4(dst) || !aligned4(missing) ||
      !aligned16(workspace))
    return OPQ_ERR_ALIGN;
  const int e = pages_checks(rows, new_rows, columns, pages, workspace, workspace_bytes);
  if (e != OPQ_OK) return e;
  if (page > kMaxInt) return OPQ_ERR_UNSUPPORTED;
  opq::PagesArgs a{};
  a.table = table;
  a.lens = lens;
  a.parents = parents;
  a.out = out;
  a.out_lens = out_lens;
  a.src = src;
  a.dst = dst;
  a.result = missing;
  a.rows = (int)rows;
  a.new_rows = (int)new_rows;
  a.columns = (int)columns;
  a.pages = (int)pages;
  a.page = (int)page;
  a.workspace = static_cast<char*>(workspace);
  return hip_status(opq::launch_pages(opq::PagesCall::kFork, a, static_cast<hipStream_t>(stream)));
}

int opq_pages_compact(const int32_t* table, int64_t rows, int64_t columns, int64_t pages,
                      int32_t* out, int32_t* src, int32_t* dst, int32_t* used, void* workspace,
                      size_t workspace_bytes, void* stream) {
  const bool some = rows > 0 && columns > 0;
  if (!used || (some && (!table || !out)) || (some && pages > 1 && (!src || !dst)))
    return OPQ_ERR_NULL;
  if (rows < 0 || columns < 0 || pages < 1) return OPQ_ERR_SHAPE;
  if (!aligned4(table) || !aligned4(out) || !aligned4(src) || !aligned4(dst) || !aligned4(used) ||
      !aligned16(workspace))
    return OPQ_ERR_ALIGN;
  const int e = pages_checks(rows, rows, columns, pages, workspace, workspace_bytes);
  if (e != OPQ_OK) return e;
  opq::PagesArgs a{};
  a.table = table;
  a.out = out;
  a.src = src;
  a.dst = dst;
  a.result = used;
  a.rows = a.new_rows = (int)rows;
  a.columns = (int)columns;
  a.pages = (int)pages;
  a.page = 16;  // lengths do not matter here
  const int64_t entries = rows * columns;
  a.moves = (int)(entries < pages / 2 ? entries : pages / 2);
  a.workspace = static_cast<char*>(workspace);
  return hip_status(opq::launch_pages(opq::PagesCall::kCompact, a, static_cast<hipStream_t>(stream)));
}

// ----------------------------------------------------------------------- drafts

size_t opq_verify_drafts_workspace_bytes(int64_t batch, int64_t vocab) {
  if (batch < 1 || batch > 65535 || vocab < 1 || vocab > (int64_t(1) << 22)) return 0;
  return opq::verify_workspace_bytes(batch, vocab);
}

int opq_verify_drafts(const void* probs, int dtype, int64_t batch, int64_t draft, int64_t vocab,
                      int64_t batch_stride, int64_t token_stride, const int32_t* tokens,
                      const float* uniforms, const void* draft_probs, int64_t q_batch_stride,
                      int64_t q_token_stride, const int32_t* parents, const int32_t* counts,
                      int32_t* kept, int32_t* count, int32_t* next, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (batch > 0 && (!probs || !tokens || !uniforms || !kept || !count || !next)) return OPQ_ERR_NULL;
  if (batch < 0 || draft < 1 || vocab < 1 || batch_stride < 0 || token_stride < 0 ||
      (draft_probs && (q_batch_stride < 0 || q_token_stride < 0)))
    return OPQ_ERR_SHAPE;
  const uintptr_t element = dtype == OPQ_F32 ? 4 : 2;
  if (!aligned(probs, element) || !aligned(draft_probs, element) || !aligned4(tokens) ||
      !aligned4(uniforms) || !aligned4(parents) || !aligned4(counts) || !aligned4(kept) ||
      !aligned4(count) || !aligned4(next) || !aligned16(workspace))
    return OPQ_ERR_ALIGN;
  if (!dtype_ok(dtype)) return OPQ_ERR_DTYPE;
  const size_t need = opq_verify_drafts_workspace_bytes(batch, vocab);
  if (workspace_bytes < need || (need > 0 && !workspace)) return OPQ_ERR_WORKSPACE;
  if (batch > 65535 || draft > 1024 || vocab > (int64_t(1) << 22) || (draft_probs && parents) ||
      !product_within(batch, batch_stride, 1, kMaxElements) ||
      !product_within(draft, token_stride, 1, kMaxElements) ||
      (draft_probs && (!product_within(batch, q_batch_stride, 1, kMaxElements) ||
                       !product_within(draft, q_token_stride, 1, kMaxElements))))
    return OPQ_ERR_UNSUPPORTED;
  if (batch == 0) return OPQ_OK;
  opq::VerifyArgs a{};
  a.p = probs;
  a.q = draft_probs;
  a.tokens = tokens;
  a.uniforms = uniforms;
  a.parents = parents;
  a.counts = counts;
  a.kept = kept;
  a.count = count;
  a.next = next;
  a.p_batch = batch_stride;
  a.p_token = token_stride;
  a.q_batch = q_batch_stride;
  a.q_token = q_token_stride;
  a.batch = (int)batch;
  a.draft = (int)draft;
  a.vocab = (int)vocab;
  a.workspace = workspace;
  return hip_status(opq::launch_verify(a, dtype == OPQ_BF16, static_cast<hipStream_t>(stream)));
}

static bool attention_shape_ok(int64_t batch, int64_t draft, int64_t heads, int64_t kv_heads,
                               int64_t dim, int64_t max_len) {
  return batch >= 0 && draft >= 0 && heads > 0 && kv_heads > 0 && heads % kv_heads == 0 &&
         max_len >= 0 && (dim == 64 || dim == 128 || dim == 256);
}
static bool attention_supported(int64_t batch, int64_t draft, int64_t heads, int64_t max_len) {
  return batch <= 65535 && draft <= 65536 && heads <= 65535 && max_len <= kMaxInt &&
         product_within(batch, draft, heads, int64_t(1) << 22);
}

size_t opq_cache_attention_workspace_bytes(int64_t batch, int64_t draft, int64_t heads,
                                           int64_t kv_heads, int64_t dim, int64_t max_len) {
  if (!attention_shape_ok(batch, draft, heads, kv_heads, dim, max_len) || batch == 0 ||
      draft == 0 || !attention_supported(batch, draft, heads, max_len))
    return 0;
  return opq::attention_plan(batch, draft, heads, kv_heads, dim, max_len).workspace;
}

int opq_cache_attention(const opq_cache* cache, const uint16_t* q, int64_t batch, int64_t draft,
                        int64_t heads, int64_t q_batch_stride, int64_t q_token_stride,
                        int64_t q_head_stride, const int32_t* page_table, int64_t max_pages,
                        const int32_t* lens, const int32_t* counts, int64_t max_len,
                        const uint32_t* mask, int64_t mask_batch_stride, float scale,
                        uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream) {
  const bool some = batch > 0 && draft > 0;
  if (cache_null(cache) || (some && (!q || !lens || !out || (max_pages > 0 && !page_table))))
    return OPQ_ERR_NULL;
  const opq_cache& c = *cache;
  if (!cache_shape_ok(c) || !attention_shape_ok(batch, draft, heads, c.heads, c.dim, max_len) ||
      max_pages < 0 || max_len > kMaxInt || max_pages > kMaxInt / c.page ||
      max_len > max_pages * c.page || mask_batch_stride < 0)
    return OPQ_ERR_SHAPE;
  if (!cache_alpha_ok(c) || !std::isfinite(scale)) return OPQ_ERR_ALPHA;
  if (!cache_aligned(c) || !aligned16(q) || !aligned4(page_table) || !aligned4(lens) ||
      !aligned4(counts) || !aligned4(mask) || !aligned16(out) || !aligned4(lse) ||
      !aligned16(workspace) || q_batch_stride % 8 || q_token_stride % 8 || q_head_stride % 8)
    return OPQ_ERR_ALIGN;
  if (!format_ok(c.format)) return OPQ_ERR_DTYPE;
  const size_t need =
      opq_cache_attention_workspace_bytes(batch, draft, heads, c.heads, c.dim, max_len);
  if (workspace_bytes < need || (need > 0 && !workspace)) return OPQ_ERR_WORKSPACE;
  if (!cache_supported(c) || !attention_supported(batch, draft, heads, max_len))
    return OPQ_ERR_UNSUPPORTED;
  if (!some) return OPQ_OK;
  const opq::AttentionPlan plan =
      opq::attention_plan(batch, draft, heads, c.heads, c.dim, max_len);
  opq::AttentionArgs a{};
  a.q = q;
  a.q_batch = q_batch_stride;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.k = static_cast<const char*>(c.k);
  a.k_sign = c.k_sign;
  a.k_scale = c.k_scale;
  a.v = static_cast<const char*>(c.v);
  a.v_sign = c.v_sign;
  a.v_scale = c.v_scale;
  a.page_table = page_table;
  a.lens = lens;
  a.counts = counts;
  a.mask = mask;
  a.mask_batch = mask_batch_stride;
  a.mask_words = (draft + 31) / 32;
  a.max_pages = max_pages;
  // no pages, no keys: nothing of an empty cache may be read
  a.capacity = c.pages > 0 ? max_pages * c.page : 0;
  a.chunk = plan.chunk;
  a.pages = (uint32_t)c.pages;
  while ((int64_t(1) << a.page_shift) < c.page) ++a.page_shift;
  a.batch = (int)batch;
  a.draft = (int)draft;
  a.heads = (int)heads;
  a.kv_heads = (int)c.heads;
  a.share = (int)(heads / c.heads);
  a.rows = (int)(draft * (heads / c.heads));
  a.splits = plan.splits;
  a.groups = plan.groups;
  a.group_rows = plan.group_rows;
  a.scale_log2 = (float)(std::fabs((double)scale) * 1.4426950408889634);
  a.q_flip = scale < 0.0f ? 0x80008000u : 0u;
  a.out = out;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  const int64_t rows = (int64_t)plan.splits * batch * c.heads * a.rows;
  a.part_ml = plan.splits > 1 ? a.part_o + rows * c.dim : nullptr;
  if (c.format == OPQ_CACHE_OPQ4) a.lp = level_planes(c.alpha);
  return hip_status(opq::launch_attention(a, c.format, (int)c.dim, plan.tiles,
                                          static_cast<hipStream_t>(stream)));
}

}  // extern "C"
