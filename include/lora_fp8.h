/*
 * lora_fp8.h -- C ABI of the 8-bit part of a fine-tuning step: products with frozen weights in 8 bits, and the MLP
 * activation that checkpoints the fine-tuning rows in 8 bits.
 *
 * The fine-tuning adapter sits on a layer's attention projections ("DeltaServe: Host-Agnostic Co-Serving of
 * Inference and Fine-Tuning for LLMs", section 4.1); the MLP's projections carry none, but the whole batch runs
 * through them in the forward and the fine-tuning rows' gradient in the backward.  Which intermediates are kept for
 * that backward trades memory for recomputation (section 3.2, activation capture); here the MLP keeps gate|up of the
 * fine-tuning rows in 8 bits, half of what 16 bits take.
 *
 * 8-bit format.  Codes are e4m3 (1 sign, 4 exponent, 3 mantissa bits, largest value 448, no infinity); a value is its
 * code times the float32 scale of its block:
 *   rows     x [T,K]: a block is 128 consecutive columns of one row (the last one may be shorter);
 *            scales [T, ceil(K/128)].
 *   weights  W [N,K]: a block is 128 x 128 (the last ones may be smaller); scales [ceil(N/128), ceil(K/128)].
 * The functions here choose the smallest power of two s with max|block| <= 448 s (and at least 2^-108), so that
 * x / s is exact and a code is one rounding (to nearest, ties to even) of the value.  A block that holds an infinity
 * or a NaN gets the scale NaN: all its values are NaN.  The products accept any scales.
 *
 * The conventions of lora_mixed.h hold: device pointers unless marked HOST; the caller owns every buffer; everything
 * is validated on the host, and a call that returns an error has launched and written nothing; work is enqueued on
 * `stream` and nothing is waited for.  All matrices are row-major with unit column stride; ld_* is the distance of
 * two rows in elements.  A size of zero rows is valid and launches nothing.  Limits: K, I <= 2^22, T <= 2^31 -
 * 1025, and for lora_fp8_linear T x N <= 2^44 (LORA_ERR_LIMIT).
 */
#ifndef LORA_FP8_H
#define LORA_FP8_H

#include "lora_mixed.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_FP8_BLOCK 128

/* x [T,K] (element type dt, ld_x) -> codes [T,K] (ld_codes) and scales [T, ceil(K/128)] (contiguous).
 * K a multiple of 16; x and codes 16-byte aligned, ld_x * element size and ld_codes multiples of 16 bytes
 * (LORA_ERR_ALIGNMENT). */
int lora_fp8_quantize(int32_t T, int32_t K, lora_dtype_t dt, const void* x, int64_t ld_x, void* codes,
                      int64_t ld_codes, float* scales, void* stream);

/* W [N,K] (element type dt, ld_w) -> codes [N,K] (contiguous) and scales [ceil(N/128), ceil(K/128)].  Done once for a
 * frozen weight.  K a multiple of 16, N <= 65535 * 128; alignment as lora_fp8_quantize. */
int lora_fp8_quantize_weight(int32_t N, int32_t K, lora_dtype_t dt, const void* W, int64_t ld_w, void* codes,
                             float* scales, void* stream);

/* Bytes of device workspace that lora_fp8_linear needs for these sizes: x quantized on the way (x_fp8 = 0), the
 * status word and partial sums.  Returns 0 and sets lora_last_error on invalid sizes. */
size_t lora_fp8_workspace_size(int32_t T, int32_t K, int32_t N, int32_t x_fp8);

/* y [T,N] (bf16, ld_y) = x W^T for a weight in 8 bits:
 *     y[t,n] = sum_b sx[t,b] sw[n/128,b] sum_{k in block b} qx[t,k] qw[n,k]
 * with float32 sums, rounded to bf16 once.
 *   x_scales NULL:     x [T,K] in element type dt; it is quantized as lora_fp8_quantize does.
 *   x_scales non-NULL: x holds codes, x_scales [T, ceil(K/128)] (contiguous) their scales; dt is ignored.
 *   w [N,K] codes (contiguous), w_scales [ceil(N/128), ceil(K/128)].
 * The gradient of the input is the same call on the transposed weight's codes (K and N exchanged, scales
 * transposed).  K a multiple of 16, N a multiple of 8; x, w and y 16-byte aligned, ld_x * element size and ld_y * 2
 * multiples of 16 bytes.  workspace: 256-byte aligned, >= lora_fp8_workspace_size bytes; its status word is read by
 * lora_workspace_status (a call of zero rows leaves it as it was).  Sums are taken in a fixed order: repeated calls
 * give identical bits. */
int lora_fp8_linear(int32_t T, int32_t K, int32_t N, lora_dtype_t dt, const void* x, int64_t ld_x,
                    const float* x_scales, const void* w, const float* w_scales, void* y, int64_t ld_y,
                    void* workspace, size_t ws_bytes, void* stream);

/* Rows of the checkpoint of a segment table: the tokens of its is_train segments.  Negative LORA_ERR_* on a bad
 * table. */
int64_t lora_checkpoint_rows(int32_t T, const lora_segment_t* segs /* HOST */, int32_t n_segs);

/* h [T,I] = silu(gate) * up, gate|up = gu [T, 2 I] (element type dt, ld_gu): gate in columns [0,I), up in [I,2I).
 *   h_scales NULL:     h in element type dt (ld_h).
 *   h_scales non-NULL: h in 8 bits, codes [T,I] (ld_h) and scales [T, ceil(I/128)]: the input of the next product.
 * ck_codes non-NULL: gate|up of the rows of is_train segments is kept in 8 bits, segment after segment in increasing
 * start order: ck_codes [R, 2 I] and ck_scales [R, 2 ceil(I/128)], R = lora_checkpoint_rows, both contiguous; gate's
 * blocks first, then up's (each half starts a block of its own).  segs: the batch's table (as lora_mixed_forward's:
 * it covers [0,T) once; at most 48 fine-tuning segments; adapter ids are not read); with ck_codes NULL it may be NULL.
 * I a multiple of 8; gu and h 16-byte aligned, row distances multiples of 16 bytes; ck_codes 16-byte aligned. */
int lora_swiglu_forward(int32_t T, int32_t I, lora_dtype_t dt, const void* gu, int64_t ld_gu,
                        const lora_segment_t* segs /* HOST */, int32_t n_segs, void* h, int64_t ld_h, float* h_scales,
                        void* ck_codes, float* ck_scales, void* stream);

/* The backward from the checkpoint: with g, u the checkpoint's values and sig = 1 / (1 + e^-g),
 *     dgate = dh u sig (1 + g (1 - sig)),     dup = dh g sig
 *   dh [R,I] (element type dt, ld_dh): the gradient of h for the checkpoint's rows, in its order.
 *   dgu_scales NULL:     dgu [R, 2 I] in element type dt (ld_dgu).
 *   dgu_scales non-NULL: dgu in 8 bits, codes [R, 2 I] (ld_dgu) and scales [R, 2 I / 128], the input of the product
 *                        with the transposed gate|up weight; I then a multiple of 128.
 * Alignment as lora_swiglu_forward. */
int lora_swiglu_backward(int32_t R, int32_t I, lora_dtype_t dt, const void* ck_codes, const float* ck_scales,
                         const void* dh, int64_t ld_dh, void* dgu, int64_t ld_dgu, float* dgu_scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_FP8_H */
