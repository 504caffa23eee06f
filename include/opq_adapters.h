/*
 * libopq, adapters: what tunes and personalises a projection whose weights are
 * stored codes.
 *   opq_lowrank_add       low-rank adapters of many requests at once, added to
 *                         the outputs of one shared projection;
 *   opq_lowrank_backward  their gradients;
 *   opq_linear_backward*  the gradient of a quantized projection's input.
 *
 * The conventions of opq.h hold (status codes, order of the argument checks,
 * streams, nothing allocated or synchronised, nothing enqueued on an error),
 * with these additions:
 *   - matrices of tokens have a row stride, counted in elements and a multiple
 *     of 8; their rows do not overlap (inputs may also repeat: stride 0).
 *     Every array is 16-byte aligned, but index and scale, which are 4-byte
 *     aligned (they may start inside a longer array);
 *   - index is read on the device and checked in the kernels: what an entry
 *     that names no adapter does is stated below, and no access leaves an array.
 */
#ifndef OPQ_ADAPTERS_H
#define OPQ_ADAPTERS_H

#include "opq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A stack of adapters of one projection [k -> n]:
 *   down   device, [count][rank][k] bfloat16: D_i
 *   up     device, [count][rank][n] bfloat16: U_i (of an adapter kept as a layer
 *          rank -> n with weight [n][rank]: that weight transposed)
 *   scale  device, [count] float32: s_i
 * rank a multiple of 8, 8..128 (smaller ranks: rows of zeros); k and n multiples of 8.
 */
typedef struct {
  const uint16_t* down;
  const uint16_t* up;
  const float* scale;
  int64_t count, rank, k, n;
} opq_lowrank;

/* Bytes of device workspace opq_lowrank_add needs for m tokens. */
size_t opq_lowrank_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank);

/*
 * out[t] = y[t] + s_i U_i^T (D_i x[t]),  i = index[t].
 *   x      device, [m][k] bfloat16
 *   index  device, [m] int32.  A token whose entry is outside 0..count-1 (such as
 *          -1) uses no adapter: its out is its y
 *   y      device, [m][n] of y_dtype (OPQ_F32 or OPQ_BF16), or NULL: zeros
 *   out    device out, [m][n] of out_dtype; it may be y itself (same type and stride)
 *   workspace  at least opq_lowrank_workspace_bytes(m, k, n, rank) bytes, no
 *          initialisation; calls that may overlap need their own
 * Products of bfloat16 are summed in float32.  For the second product s_i D_i x is
 * taken in three bfloat16 parts (24 bits, all of a float32); the sum with y is float32,
 * rounded once: a bfloat16 out is the float32 one rounded.  Infinities and NaN come out
 * where the formula has them.  A token's result
 * does not depend on the other tokens of the call, whose number sets in how many pieces
 * sums over k are taken; results repeat bit for bit.
 * m up to 2^22, k and n up to 2^20, m * k and m * n up to 2^39 with their strides,
 * count up to 2^30 (OPQ_ERR_UNSUPPORTED past them, and for y itself as out with another
 * type or stride).  out must not overlap the other inputs.
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALIGN, OPQ_ERR_DTYPE,
 * OPQ_ERR_WORKSPACE, OPQ_ERR_UNSUPPORTED, OPQ_ERR_HIP.
 */
int opq_lowrank_add(const opq_lowrank* adapters, const uint16_t* x, int64_t x_stride,
                    const int32_t* index, int64_t m, const void* y, int64_t y_stride, int y_dtype,
                    void* out, int64_t out_stride, int out_dtype, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Bytes of device workspace opq_lowrank_backward needs. */
size_t opq_lowrank_backward_workspace_bytes(int64_t m, int64_t k, int64_t n, int64_t rank,
                                            int64_t count);

/*
 * The gradients of opq_lowrank_add from dy, the gradient of out (the gradient of y is dy):
 *   h_t = s_i D_i x_t,  e_t = s_i U_i dy_t  (i = index[t]),
 *   dx_out[t] = dx[t] + D_i^T e_t          (dx NULL: zeros),
 *   d_down[i] = sum over its tokens of e_t x_t^T,  d_up[i] = ... of h_t dy_t^T,
 * an adapter without tokens gets zeros.  Tokens without an adapter: dx_out = dx.
 *   dy      device, [m][n] bfloat16
 *   dx      device, [m][k] of dx_dtype or NULL; dx_out device out, of the same type,
 *           may be dx itself (same stride); NULL: not wanted
 *   d_down, d_up  device out, dense [count][rank][k], [count][rank][n] of grad_dtype;
 *           both NULL: not wanted
 *   workspace  as for opq_lowrank_add
 * Roundings as opq_lowrank_add: e and h enter their products with all their 24 bits;
 * sums are float32 and in a fixed order.
 * Limits as opq_lowrank_add, and count up to 1024.  Errors as opq_lowrank_add.
 */
int opq_lowrank_backward(const opq_lowrank* adapters, const uint16_t* dy, int64_t dy_stride,
                         const uint16_t* x, int64_t x_stride, const int32_t* index, int64_t m,
                         const void* dx, int64_t dx_stride, int dx_dtype, void* dx_out,
                         int64_t dx_out_stride, void* d_down, void* d_up, int grad_dtype,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * dx = dy W': the gradient of the input of y = x W'^T, with W' [n][k] the bfloat16
 * values opq_dequantize* writes.  Up to 512 tokens of 4-bit codes are multiplied as
 * the codes are decoded; otherwise W' goes transposed into the workspace, then a dense
 * product makes dx.  Both are bf16 matrix-core products with float32 sums.
 *   dy     device, [m][n] bfloat16, dense;  dx  device out, [m][k] of dx_dtype, dense;
 *          it must not overlap the inputs
 *   workspace  at least opq_linear_backward_workspace_bytes(m, n, k) bytes, or for 4-bit codes
 *          opq_linear_backward_codes_workspace_bytes(m, n, k), which are never more (both are
 *          whole MiB); no initialisation; calls that may overlap need their own
 * The other arguments as in opq_linear, opq_linear_bits and opq_linear_grouped; n up to
 * 65536 (the sums of more rows are those of blocks of them, added), k up to 65536 and a multiple of 32, m up to 2^22, m * n and m * k up to 2^39.
 * Errors: OPQ_ERR_NULL, OPQ_ERR_SHAPE, OPQ_ERR_ALPHA, OPQ_ERR_ALIGN, OPQ_ERR_DTYPE,
 * OPQ_ERR_WORKSPACE, OPQ_ERR_UNSUPPORTED, OPQ_ERR_HIP.
 */
size_t opq_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k);
size_t opq_linear_backward_codes_workspace_bytes(int64_t m, int64_t n, int64_t k);
int opq_linear_backward(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                        const float* scale, int64_t m, int64_t n, int64_t k, float alpha, void* dx,
                        int dx_dtype, void* workspace, size_t workspace_bytes, void* stream);
int opq_linear_backward_bits(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                             const float* scale, int64_t m, int64_t n, int64_t k, int bits,
                             float alpha, void* dx, int dx_dtype, void* workspace,
                             size_t workspace_bytes, void* stream);
int opq_linear_backward_grouped(const uint16_t* dy, const uint32_t* packed, const uint32_t* sign,
                                const uint16_t* scale16, int64_t m, int64_t n, int64_t k,
                                int64_t group, float alpha, void* dx, int dx_dtype,
                                void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* OPQ_ADAPTERS_H */
