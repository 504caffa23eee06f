/*
 * libopq, attention side: what a quantized transformer runs between its
 * quantized QKV projection and its quantized output projection.
 *   opq_rotary            rotary positions on queries and keys (and its backward pass);
 *   opq_cache_write/read  a paged key/value cache, quantized as it is written;
 *   opq_cache_attention   attention of one token, or of a tree of drafted
 *                         tokens, per sequence, straight from the cache's codes;
 *   opq_pages_*           the cache's pages forked, taken, freed, drawn together;
 *   opq_verify_drafts     drafted tokens verified against the target's probabilities.
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

/* ------------------------------------------------------------------- pages */

/*
 * Pages of a cache, forked, taken, freed and drawn together.  A page table,
 * int32 [rows][columns], names the pages that hold each row's tokens, in order; an
 * entry outside 0..pages-1 (such as -1) names none.  A page that no entry of the
 * table names is free: the table is all the state there is, and what is freed is freed by
 * no longer naming it.  One table names the same pages in the caches of every layer.
 *   table, lens, parents  device;  every output: device out, int32, dense
 *   pages  1..2^20;  page  tokens of a page, a power of two, 16 or more;
 *   rows * columns up to 2^28, rows up to 2^20
 *   workspace  at least opq_pages_workspace_bytes(rows of the new table, pages)
 *          bytes, no initialisation; calls that may overlap need their own
 * Lengths are clamped to 0..columns * page.  Free pages are taken lowest first, so
 * results are the same from call to call.  Errors of the three: OPQ_ERR_NULL,
 * OPQ_ERR_SHAPE, OPQ_ERR_ALIGN, OPQ_ERR_WORKSPACE, OPQ_ERR_UNSUPPORTED, OPQ_ERR_HIP.
 */
size_t opq_pages_workspace_bytes(int64_t rows, int64_t pages);

/*
 * Rows resized: row i keeps the entries of its first lens[i] tokens (those of the rest
 * become -1: their pages are freed unless other rows name them) and takes free
 * pages, row by row, for the entries it lacks.
 *   lens     [rows] int32, the tokens each row shall have room for
 *   out      [rows][columns]; may be table
 *   missing  [1]: entries left -1 because no page was free (all of them come after
 *            those that got one)
 */
int opq_pages_resize(const int32_t* table, const int32_t* lens, int64_t rows, int64_t columns,
                     int64_t pages, int64_t page, int32_t* out, int32_t* missing, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Rows forked, reordered, dropped: row i of the new table is a copy of row
 * parents[i] as far as its lens[parents[i]] tokens go (beams after a step, samples of one
 * prompt; a parent outside 0..rows-1: an empty row).  Rows share full pages.  A
 * last page that is partly filled, so will be written on, stays with the
 * first new row that ends in it, unless a row names it as a full page; every other row that
 * ends in it gets a free page instead, and a pair for opq_cache_copy_pages (of each cache).
 *   parents  [new_rows] int32
 *   out      [new_rows][columns]; must not overlap table
 *   out_lens [new_rows]: the rows' tokens
 *   src, dst [new_rows]: page dst[i] is to become a copy of page src[i]; -1: none
 *   missing  [1]: rows that lack their last page (-1) because none was free
 */
int opq_pages_fork(const int32_t* table, const int32_t* lens, int64_t rows, int64_t columns,
                   const int32_t* parents, int64_t new_rows, int64_t pages, int64_t page,
                   int32_t* out, int32_t* out_lens, int32_t* src, int32_t* dst, int32_t* missing,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Pages drawn together: with U pages in use, the k-th used page (by id) past the first U
 * ids moves to the k-th free page of them.
 *   out       [rows][columns], the table after the move; may be table
 *   src, dst  [moves], moves = min(pages / 2, rows * columns): the pairs for
 *             opq_cache_copy_pages, -1 behind the last
 *   used      [1]: U
 */
int opq_pages_compact(const int32_t* table, int64_t rows, int64_t columns, int64_t pages,
                      int32_t* out, int32_t* src, int32_t* dst, int32_t* used, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * Whole pages copied, keys and values of every head, codes and scales as they are: page
 * src[i] to page dst[i].  A pair with a page outside 0..pages-1 (such as -1) copies
 * nothing.  No page may be a destination twice, or a source and a destination: what such
 * a page holds afterwards is unspecified.
 *   src, dst  device, [count] int32;  count up to 2^20
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALPHA, OPQ_ERR_ALIGN, OPQ_ERR_DTYPE,
 * OPQ_ERR_UNSUPPORTED, OPQ_ERR_HIP.
 */
int opq_cache_copy_pages(const opq_cache* cache, int64_t count, const int32_t* src,
                         const int32_t* dst, void* stream);

/* ------------------------------------------------------------------ drafts */

/* Bytes of device workspace opq_verify_drafts needs. */
size_t opq_verify_drafts_workspace_bytes(int64_t batch, int64_t vocab);

/*
 * Drafted tokens verified against the target model's probabilities, with given random
 * numbers: the tokens that come out are distributed as the target's own.  Of a
 * sequence's `draft` tokens the first is certain (the last one decided, whose
 * row gives what follows it); the others hang under their parents.  From node 0 on, the
 * node's children are tested in the order of their indexes; the first kept one is
 * the next node.  With p the probabilities of the node, x the child's token, u its random
 * number:
 *   - with draft_probs (a chain drawn from a draft model, q the probabilities x was
 *     drawn from): kept if u q(x) < p(x);
 *   - without (a tree or chain of candidates): kept if u Z < p(x), Z = 1 less the
 *     p of the node's children tested before; a sibling's token again counts p = 0.
 * Nothing with p(x) = 0 is kept.  At the last node `next` is drawn with the
 * first token's number u0 from weights w: p; max(p - q, 0) if a token drawn from q was
 * refused; p without the tested children's tokens for candidates.  It is the
 * lowest token i with w_i > 0 whose w_0 + ... + w_i exceeds u0 times the sum of all, the
 * last with w_i > 0 if rounding leaves none, -1 if every weight is 0.
 *   probs    device, [batch][draft][vocab] of dtype (OPQ_F32 or OPQ_BF16): row t
 *            after token t
 *   tokens   device, [batch][draft] int32; one outside 0..vocab-1 has p = 0
 *   uniforms device, [batch][draft] float32 in [0, 1)
 *   draft_probs  device, [batch][draft-1][vocab] of dtype, row t - 1 of token t; or NULL
 *   parents  device, [batch][draft] int32 or NULL (a chain: t - 1), not both this
 *            and draft_probs.  A token whose parent is not an earlier one is never kept
 *   counts   device, [batch] int32 or NULL: how many of the draft count (0: the
 *            sequence gets kept -1, count 0 and next -1)
 *   kept     device out, [batch][draft] int32: indexes of the kept tokens in order, 0
 *            first, then -1;  count, next  device out, [batch] int32
 * Rows of probabilities have free strides (in elements, not negative; vocab is dense) and need
 * only their element's alignment; the int32 and float32 arrays are dense and 4-byte
 * aligned, the workspace 16-byte.  A probability that is negative, infinite or NaN counts
 * as 0.  Products, Z and sums are in float64; sums in a fixed order.
 * draft 1..1024, vocab 1..2^22, batch up to 65535 (OPQ_ERR_UNSUPPORTED past them, and for
 * draft_probs with parents).
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALIGN, OPQ_ERR_DTYPE,
 * OPQ_ERR_WORKSPACE, OPQ_ERR_UNSUPPORTED, OPQ_ERR_HIP.
 */
int opq_verify_drafts(const void* probs, int dtype, int64_t batch, int64_t draft, int64_t vocab,
                      int64_t batch_stride, int64_t token_stride, const int32_t* tokens,
                      const float* uniforms, const void* draft_probs, int64_t q_batch_stride,
                      int64_t q_token_stride, const int32_t* parents, const int32_t* counts,
                      int32_t* kept, int32_t* count, int32_t* next, void* workspace,
                      size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OPQ_ATTENTION_H */
