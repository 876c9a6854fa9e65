/*
 * lora_attention.h -- C ABI of the attention side of a co-served step: from the fused q|k|v projection of the mixed batch
 * to the input of the output projection.
 *
 * The adapters sit on a layer's attention projections ("DeltaServe: Host-Agnostic Co-Serving of Inference and
 * Fine-Tuning for LLMs", section 4.1).  Between them, every row's query and key heads are normalised and turned by the
 * row's position; keys and values of served rows go into a paged cache; a decode row attends over its sequence's cache;
 * and the fine-tuning rows' gradient comes back through the rotation and the norm.
 *
 * Rotary positions.  A head's row x [D] is normalised (where a weight w [D] is given) and its first R elements turned:
 *     n = x w / sqrt(mean(x^2) + eps)
 * (a row whose squares add up past float32's range counts as infinitely long: n = 0; squares below 2^-126 lose digits, which
 * shows where eps is no larger than they)
 *     pair i < R/2:  a = n[i], b = n[i + R/2]   (interleaved: n[2i], n[2i+1])
 *     y_a = a cos t - b sin t,  y_b = b cos t + a sin t,   t = 2 pi position turns_i
 * turns_i is the pair's frequency in turns a position, as a whole number of 2^-64 turns (an angular frequency f, base^
 * (-2i/R) for instance, is f / 2 pi turns).  position * turns_i is taken modulo one turn exactly, in 64-bit whole numbers,
 * for positions of any size; then it is cut to a whole number of 2^-32 turns and goes on in float32.  What the given turns
 * are off their frequency counts position times: p 2^-65 turns for the nearest whole numbers.
 *
 * Paged cache.  Keys and values lie in pages of page_size rows for each of n_heads heads.  Element (page, head, row, d)
 * is at page * page_stride + head * head_stride + row * row_stride + d, so a page may be [heads, rows, D] or
 * [rows, heads, D], and keys and values may share a buffer.  Its element type is bf16, or 8 bits: e4m3 codes with one
 * float32 scale for each head's row, k_scales and v_scales at page * scale_page_stride + head * scale_head_stride +
 * row * scale_row_stride.  A value is its code times its row's scale.  The functions here choose the smallest power of two
 * that brings the row within 448, e4m3's largest value (and at least 2^-108), as the 8-bit rows of lora_fp8.h; a row that
 * holds an infinity or a NaN gets the scale NaN.  lora_cache_read accepts any scales,
 * lora_decode_attention any that are not negative (a negative value scale gives NaN).
 * The place of a row is its slot, page * page_size + row in the page.
 *
 * The conventions of lora_mixed.h hold: device pointers unless marked HOST; the caller owns every buffer; everything
 * that the host can see is validated before anything is launched, and a call that returns an error has launched and
 * written nothing; work is enqueued on `stream` and nothing is waited for.  What only the device can see (positions,
 * slots, page tables, lengths) is checked there: no access leaves a buffer.  Matrices are row-major with unit column
 * stride; ld_* is the distance of two rows in elements.  Zero rows are valid and launch nothing.
 *
 * Limits (LORA_ERR_LIMIT): D a multiple of 16, at most 256; R a multiple of 16, at most D; at most 1024 heads in all;
 * T and B <= 2^31 - 1025.  Data, weights and caches 16-byte aligned, their row distances and strides multiples of 16 bytes
 * (LORA_ERR_ALIGNMENT).
 */
#ifndef LORA_ATTENTION_H
#define LORA_ATTENTION_H

#include "lora_mixed.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a cache */
enum { LORA_CACHE_BF16 = 0, LORA_CACHE_E4M3 = 1 };

typedef struct lora_cache {
    void* k;                 /* device; element (0, 0, 0, 0) */
    void* v;
    float* k_scales;         /* device; NULL unless 8 bits */
    float* v_scales;
    int64_t page_stride;     /* elements; k and v alike */
    int64_t head_stride;
    int64_t row_stride;
    int64_t scale_page_stride;
    int64_t scale_head_stride;
    int64_t scale_row_stride;
    int32_t n_pages;
    int32_t n_heads;
    int32_t page_size;
    int32_t head_dim;
    int32_t dtype;           /* LORA_CACHE_* */
} lora_cache_t;

typedef struct lora_rotary {
    const int64_t* turns;    /* device [R/2]; NULL where R is 0 (no rotation) */
    const void* q_weight;    /* device [D], element type of the call; NULL: queries are not normalised */
    const void* k_weight;    /* the same for keys */
    int32_t n_heads;         /* query heads */
    int32_t n_kv_heads;      /* key heads */
    int32_t head_dim;        /* D */
    int32_t rot_dim;         /* R */
    int32_t interleaved;     /* nonzero: neighbours are pairs */
    float eps;
} lora_rotary_t;

/* x [T, (n_heads + n_kv_heads) D] (element type dt, ld_x): query heads, then key heads, for instance the first columns of
 * a fused q|k|v.  positions [T].
 *   cache NULL:     out [T, (n_heads + n_kv_heads) D] (element type dt, ld_out) gets queries and keys.
 *   cache non-NULL: keys, and the values v [T, n_kv_heads D] (element type dt, ld_v), go to the cache's slots [T]; out
 *                   gets the queries [T, n_heads D], and with keep_keys the keys after them.  A row whose slot lies
 *                   outside the cache (-1, for instance) is not written to it.  No two rows of a call may have the same
 *                   slot: that slot would hold a mixture of the two.
 * The cached rows are rounded once, from the 32-bit result.  out may be x itself (same ld): the results then take the
 * rows' place. */
int lora_rotary_forward(int32_t T, lora_dtype_t dt, const lora_rotary_t* rotary /* HOST */, const void* x, int64_t ld_x,
                        const int64_t* positions, void* out, int64_t ld_out, const void* v, int64_t ld_v,
                        const lora_cache_t* cache /* HOST */, const int64_t* slots, int32_t keep_keys, void* stream);

/* Bytes of workspace that lora_rotary_backward needs for the weights' gradients.  Returns 0 and sets lora_last_error on
 * invalid sizes. */
size_t lora_rotary_workspace_size(int32_t T, const lora_rotary_t* rotary /* HOST */);

/* The gradient of x from dout [T, (n_heads + n_kv_heads) D] (element type dt, ld_dout), the gradient of queries and keys:
 * with g = dout turned back, and r = 1 / sqrt(mean(x^2) + eps),
 *     dw = sum over rows and heads of g x r          dx = r (w g - x r^2 mean(w g x))
 *   x [T, (n_heads + n_kv_heads) D] (ld_x): the forward's input; NULL where neither weight is given.
 *   dx (element type dt, ld_dx): may be dout itself (same ld).
 *   dq_weight, dk_weight [D] float32 (4-byte aligned): written where non-NULL; they need their weight, and a workspace
 *   (16-byte aligned, >= lora_rotary_workspace_size bytes).  Sums are float32 in a fixed order: repeated calls give identical
 *   bits. */
int lora_rotary_backward(int32_t T, lora_dtype_t dt, const lora_rotary_t* rotary /* HOST */, const void* x, int64_t ld_x,
                         const int64_t* positions, const void* dout, int64_t ld_dout, void* dx, int64_t ld_dx,
                         float* dq_weight, float* dk_weight, void* workspace, size_t ws_bytes, void* stream);

/* k and v [T, n_heads D] (element type dt, ld_k, ld_v) to the cache's slots [T]; as lora_rotary_forward's keys and
 * values, without the norm and the rotation. */
int lora_cache_write(int32_t T, lora_dtype_t dt, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                     const lora_cache_t* cache /* HOST */, const int64_t* slots, void* stream);

/* The cached rows of slots [T] as k and v [T, n_heads D] (element type dt, ld_k, ld_v).  A slot outside the cache gives a
 * row of zeros; slots may repeat. */
int lora_cache_read(int32_t T, lora_dtype_t dt, const lora_cache_t* cache /* HOST */, const int64_t* slots, void* k,
                    int64_t ld_k, void* v, int64_t ld_v, void* stream);

/* Bytes of device workspace that lora_decode_attention needs on the current device for heads of these sizes, whatever the
 * number of sequences and their lengths.  Returns 0 and sets lora_last_error on invalid sizes. */
size_t lora_decode_workspace_size(int32_t n_heads, const lora_cache_t* cache /* HOST */);

/* Attention of one new token of each of B sequences over its cached rows (its own among them).  With n = n_heads / the
 * cache's heads, head h of sequence b attends with the cache's head h / n, over the rows j of [max(0, L_b - window), L_b)
 * (window 0: [0, L_b)), row j in page table[b, j / page_size]:
 *     s_j = scale q.k_j       (softcap c > 0: c tanh(s_j / c); scale / c and c log2(e), without a cap scale log2(e), must
 *                             be finite in float32)
 *     out = sum_j e^s_j v_j / sum_j e^s_j,   lse = log sum_j e^s_j
 *   q, out [B, n_heads D] (bf16, ld_q, ld_out); out may be q itself (same ld: another one is refused), and overlaps q in no
 *   other way.   lse [B, n_heads] float32 or NULL.   lengths [B], table [B, ld_table]: they stay as they are until the call's
 *   kernel has run (they are read more than once).
 * Products are of 16-bit numbers (8-bit codes exactly; a probability as two of them, 2^-16 of it off at most), sums and
 * statistics in 32 bits, in an order that depends on the lengths of the call's sequences only: repeated calls give
 * identical bits.
 * A length of zero or less gives out = 0 and lse = -infinity.  A sequence that is longer than its table's row, or one of
 * whose pages lies outside the cache, gives NaN; nothing outside the cache is read.  Rows outside the range, and table
 * entries past it, are not read.  An infinite element of a value row in the range gives an infinity or NaN there, and so do
 * finite ones where the sum before its division, of up to 2^8 e^(s_j - max s) |v_j|, passes float32's range (never while the
 * elements are below 2^88).  Queries are bf16, as the cache holds 16 bits at most: a float32 layer rounds its own.
 * n_heads a multiple of the cache's heads; the cache's last row at most 2^32 units from its first, of the largest power of
 * two that divides page_stride and row_stride in bytes (LORA_ERR_LIMIT).
 *   workspace: 256-byte aligned, >= lora_decode_workspace_size bytes, its first LORA_DECODE_COUNTER_BYTES zero before its first
 *   use; every call leaves them zero.  Calls that share a workspace must not overlap on the GPU. */
#define LORA_DECODE_COUNTER_BYTES 8192
int lora_decode_attention(int32_t B, int32_t n_heads, const void* q, int64_t ld_q, const lora_cache_t* cache /* HOST */,
                          const int32_t* table, int64_t ld_table, int32_t table_width, const int32_t* lengths,
                          int32_t window, float scale, float softcap, void* out, int64_t ld_out, float* lse,
                          void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_ATTENTION_H */
