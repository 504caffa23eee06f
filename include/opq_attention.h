/*
 * libopq, attention side: what a quantized transformer runs between its
 * quantized QKV projection and its quantized output projection.
 *   opq_rotary            rotary positions on queries and keys (and its backward pass);
 *   opq_cache_write/read  a paged key/value cache, quantized as it is written;
 *   opq_cache_attention   attention of one token, or of a tree of drafted
 *                         tokens, per sequence, straight from the cache's codes.
 *
 * The conventions of opq.h hold (status codes, order of the argument checks,
 * streams, nothing allocated or synchronised, nothing enqueued on an error),
 * with these additions:
 *   - strides are counted in elements; the last dimension is dense;
 *   - queries, keys and values may be cut from a fused projection: their token
 *     and head strides are free (also 0), and the pointers of opq_rotary and
 *     opq_cache_write need only their element's alignment (16-byte aligned
 *     ones run wider loads).  Index arrays, masks and lse are 4-byte aligned
 *     (they may start inside a longer array), every other array 16-byte;
 *   - indexes that kernels read from device memory (positions, slots, page
 *     ids, lengths) are checked against their arrays inside the kernels: what
 *     an invalid one does is stated at the call, and no access leaves an array.
 */
#ifndef OPQ_ATTENTION_H
#define OPQ_ATTENTION_H

#include "opq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary */

typedef enum { OPQ_ROTARY_HALF = 0, OPQ_ROTARY_INTERLEAVED = 1 } opq_rotary_layout;
typedef enum {
  OPQ_ROPE_NONE = 0,   /* f_i = base^(-2i/rot) */
  OPQ_ROPE_LINEAR = 1, /* f_i / factor: positions interpolated */
  OPQ_ROPE_NTK = 2,    /* base * factor^(rot/(rot-2)) in place of base */
  OPQ_ROPE_YARN = 3    /* by parts: below */
} opq_rope_scaling;

/*
 * Frequencies of rotary positions, in radians per position.  Host only.
 *   rot      dimensions that are turned, even, 2..1024; pair i = 0..rot/2-1
 *   base     > 1;  factor >= 1 (the context is `factor` times as long);
 *   OPQ_ROPE_YARN: a pair that turns r = original_len f_i / 2 pi times over the
 *            original context keeps f_i for r >= beta_fast, gets f_i / factor
 *            for r <= beta_slow, and a mixture linear in r in between;
 *            0 <= beta_slow < beta_fast, original_len > 0
 *   out_f    host, rot/2 doubles
 *   out_amplitude  host, 1 double: 0.1 ln(factor) + 1 for OPQ_ROPE_YARN, else 1:
 *            what cos and sin are multiplied by
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE (rot), OPQ_ERR_DTYPE (unknown scaling),
 * OPQ_ERR_ALPHA (any other parameter out of its range, or not finite).
 */
int opq_rotary_frequencies(int64_t rot, double base, int scaling, double factor,
                           double original_len, double beta_fast, double beta_slow,
                           double* out_f, double* out_amplitude);

/*
 * The table opq_rotary reads: table[p][i] = amplitude * (cos p f_i, sin p f_i)
 * in float32, p = 0..len-1, computed in double (the angle is reduced in turns,
 * so long contexts lose nothing).
 *   freq   device, [pairs] double;  table  device out, [len][pairs][2] float32
 *   pairs  1..512
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALIGN, OPQ_ERR_UNSUPPORTED
 * (len * pairs past 2^39), OPQ_ERR_HIP.
 */
int opq_rotary_table(const double* freq, int64_t pairs, int64_t len, double amplitude,
                     float* table, void* stream);

/*
 * Rotary positions.  A pair (a, b) of a head becomes (a c - b s, a s + b c)
 * with (c, s) = table[p][i], computed in float32 and rounded once; with
 * backward != 0 it becomes (a c + b s, b c - a s): applied to the gradient of the
 * output that is the gradient of x.  Pair i is (x[i], x[i + rot/2]) for
 * OPQ_ROTARY_HALF and (x[2i], x[2i+1]) for OPQ_ROTARY_INTERLEAVED; dimensions
 * rot..dim-1 are copied.
 *   x        device, [tokens][heads][dim] of dtype (OPQ_F32 or OPQ_BF16)
 *   positions device, [tokens][axes] int32; sections: host, [axes] int32 > 0
 *            with sum rot/2: the first sections[0] pairs take their position
 *            from axis 0, the next sections[1] from axis 1, and so on (axes 1..4;
 *            text has one axis, image tokens often three)
 *   table    device, [table_len][rot/2][2] float32.  A position outside
 *            0..table_len-1 turns its pairs into NaN
 *   out      device out, as x with its own strides (token and head rows of
 *            out must not overlap each other); out == x with equal strides
 *            works in place
 * dim 1..65536, rot even, 2..min(dim, 1024).
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALIGN, OPQ_ERR_DTYPE (dtype or
 * layout), OPQ_ERR_UNSUPPORTED (tokens * heads * dim past 2^39), OPQ_ERR_HIP.
 */
int opq_rotary(const void* x, int dtype, int64_t tokens, int64_t heads, int64_t dim,
               int64_t x_token_stride, int64_t x_head_stride, const int32_t* positions,
               int64_t axes, const int32_t* sections, const float* table, int64_t table_len,
               int64_t rot, int layout, int backward, void* out, int64_t out_token_stride,
               int64_t out_head_stride, void* stream);

/* ------------------------------------------------------------------- cache */

typedef enum {
  OPQ_CACHE_BF16 = 0, /* codes: bfloat16 [dim];  value = code * scale, scale 1 */
  OPQ_CACHE_FP8 = 1,  /* codes: OCP e4m3 bytes [dim];  scale s = max|x| / 448,
                         code = e4m3(x / s), value = code * s */
  OPQ_CACHE_OPQ4 = 2  /* codes and signs as opq_quantize packs a row of k = dim:
                         [dim/8] and [dim/32] uint32, scale m = max|x|;
                         value = +-L_q m with L_q = bfloat16(G_q) */
} opq_cache_format;

/*
 * A paged cache of keys and values: one row per (page, head, offset in the
 * page) holds the `dim` values of one token and head, as codes and one float32
 * scale; slot = page id * page + offset names a token's place.
 *   k, v              device, codes: [pages][heads][page][dim code bytes]
 *   k_sign, v_sign    device, [pages][heads][page][dim/32] uint32
 *                     (OPQ_CACHE_OPQ4; NULL otherwise)
 *   k_scale, v_scale  device, [pages][heads][page] float32
 *   page  tokens of a page: a power of two, 16 or more;  dim  64, 128 or 256
 *   alpha of OPQ_CACHE_OPQ4, 0.05..60 (others ignore it): the same for every
 *         call on one cache
 * Quotients are binary32 (nearest even); rounding to codes is to nearest (e4m3
 * and bfloat16: ties to even; OPQ: halves up, as opq_quantize).  In the two
 * quantized formats a row whose max is below 2^-100 gets scale 0 and codes 0.
 * A row with a NaN or an infinity (for OPQ_CACHE_BF16: after rounding to
 * bfloat16) gets scale NaN and codes 0, so every value of it reads as NaN: no
 * code is ever a NaN, and a token that a mask hides cannot leak one.  (Rows that were
 * never written hold what the memory held: start a cache as zeros, or write every token
 * that a sequence's length and draft cover, hidden ones too.)
 */
typedef struct {
  void* k;
  uint32_t* k_sign;
  float* k_scale;
  void* v;
  uint32_t* v_sign;
  float* v_scale;
  int64_t pages, heads, page, dim;
  int format;
  float alpha;
} opq_cache;

/*
 * Quantize keys and values of `tokens` tokens into their slots.
 *   k, v   device, [tokens][heads][dim] of dtype (OPQ_F32 or OPQ_BF16)
 *   slots  device, [tokens] int32.  A slot outside 0..pages*page-1 (such as -1
 *          for padding) writes nothing.  Equal slots in one call leave an
 *          unspecified mixture of their rows
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALPHA, OPQ_ERR_ALIGN,
 * OPQ_ERR_DTYPE (dtype or format), OPQ_ERR_UNSUPPORTED (pages * page past
 * 2^31 - 1, or tokens * heads past 2^31 - 1), OPQ_ERR_HIP.
 */
int opq_cache_write(const opq_cache* cache, const void* k, int64_t k_token_stride,
                    int64_t k_head_stride, const void* v, int64_t v_token_stride,
                    int64_t v_head_stride, int dtype, int64_t tokens, const int32_t* slots,
                    void* stream);

/*
 * Read rows back: k_out, v_out device out, dense [tokens][heads][dim] of dtype
 * (OPQ_F32: the value itself; OPQ_BF16: rounded to nearest even).  A slot
 * outside 0..pages*page-1 gives zeros.  Errors as opq_cache_write.
 */
int opq_cache_read(const opq_cache* cache, int64_t tokens, const int32_t* slots, void* k_out,
                   void* v_out, int dtype, void* stream);

/*
 * Move rows of a cache, codes and scales as they are: token src[b][i] to slot
 * dst[b][i], for every head, of keys and values.  What a verified tree of drafted
 * tokens needs: the accepted ones move up to the slots right after the cached
 * tokens.  Within a sequence b every row is read before any is written, so
 * slots may be sources and destinations at once (but each at most once a
 * destination); sequences of one call must not share slots.  A pair with a slot
 * outside 0..pages*page-1 (such as -1) moves nothing.
 *   src, dst  device, [batch][count] int32;  count 0..128; batch up to 65535 and
 *             batch * heads up to 2^22
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALPHA, OPQ_ERR_ALIGN,
 * OPQ_ERR_DTYPE, OPQ_ERR_UNSUPPORTED (count or batch past their limits), OPQ_ERR_HIP.
 */
int opq_cache_move(const opq_cache* cache, int64_t batch, int64_t count, const int32_t* src,
                   const int32_t* dst, void* stream);

/* --------------------------------------------------------------- attention */

/*
 * Bytes of device workspace opq_cache_attention needs (0: none, the pointer
 * may be NULL).  It holds the partial results of keys split over workgroups
 * and depends on these arguments alone.
 */
size_t opq_cache_attention_workspace_bytes(int64_t batch, int64_t draft, int64_t heads,
                                           int64_t kv_heads, int64_t dim, int64_t max_len);

/*
 * Attention of `draft` tokens per sequence over its cached ones.  The keys
 * and values of the drafted tokens are in the cache already, right after the
 * lens[b] tokens before them: token j of sequence b (cached or drafted) sits in
 * page page_table[b][j / page] at offset j % page.  Drafted token t sees every
 * one of the first lens[b] tokens, and drafted token j exactly when bit j % 32
 * of mask[b][t][j / 32] is set (mask NULL: when j <= t, a chain).  Query head
 * h reads kv head h / (heads / kv_heads).
 *   out[b][t][h] = sum_j p_j v_j,  p = softmax_j(scale q . k_j),
 *   lse[b][t][h] = ln sum_j exp(scale q . k_j)
 * A row that sees nothing gets out 0 and lse -infinity.
 *   q     device, [batch][draft][heads][dim] bfloat16, strides in elements,
 *         multiples of 8; 16-byte aligned
 *   page_table  device, [batch][max_pages] int32; entries past a sequence's
 *         tokens are not used.  A page id outside the cache makes its tokens' keys
 *         and values NaN
 *   lens  device, [batch] int32; counts: device, [batch] int32 or NULL: how many of
 *         the drafted tokens count (rows past it get out 0 and lse -infinity).
 *         Both are clamped: to 0 below, and lens + counts to max_pages * page
 *   max_len  an upper bound of lens that the host knows (at most max_pages *
 *         page): it sizes the split of the work.  A sequence longer than it is
 *         still computed in full
 *   mask  device, [batch][draft][ceil(draft/32)] uint32 or NULL;
 *         mask_batch_stride in words (0: one mask for every sequence)
 *   out   device out, dense [batch][draft][heads][dim] bfloat16
 *   lse   device out, dense [batch][draft][heads] float32, or NULL
 *   workspace  at least opq_cache_attention_workspace_bytes(...) bytes, no
 *         initialisation; calls that may overlap need their own
 * Scores, the softmax's maximum and sum, and the accumulators are float32.  Scores may
 * be as large as float32 holds; two that differ by less than its spacing there may come
 * out equal, or that spacing apart.  The
 * accumulators are divided by the weights' sum at the end, and weights are at
 * most 1: values of up to 2^127 divided by the number of keys cannot overflow.
 * For the matrix product with the codes the weights p v_scale are rounded to
 * bfloat16 (with up to 16 query rows a kv head, and for dim 256, on bf16 and fp8
 * caches: to twice its bits).  Results do not depend on timing and repeat bit for
 * bit.
 * heads a multiple of kv_heads; batch * draft * heads up to 2^22, batch and heads
 * up to 65535, draft up to 65536 (OPQ_ERR_UNSUPPORTED past them).
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALPHA (also scale not finite),
 * OPQ_ERR_ALIGN, OPQ_ERR_DTYPE, OPQ_ERR_WORKSPACE, OPQ_ERR_UNSUPPORTED, OPQ_ERR_HIP.
 */
int opq_cache_attention(const opq_cache* cache, const uint16_t* q, int64_t batch, int64_t draft,
                        int64_t heads, int64_t q_batch_stride, int64_t q_token_stride,
                        int64_t q_head_stride, const int32_t* page_table, int64_t max_pages,
                        const int32_t* lens, const int32_t* counts, int64_t max_len,
                        const uint32_t* mask, int64_t mask_batch_stride, float scale,
                        uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OPQ_ATTENTION_H */
