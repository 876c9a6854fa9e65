// cache.h -- the paged key-value cache (include/lora_attention.h) on the device, and host checks that its entry points
// share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "decode_split.h"
#include "fp8.h"
#include "lora_attention.h"

namespace lora {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxHeads = 1024;

// A cache as kernels take it: strides in bytes (scales: in elements)
struct CacheView {
    char *k, *v;
    float *ks, *vs;
    int64_t page_stride, head_stride, row_stride;
    int64_t s_page, s_head, s_row;
    int64_t slots;           // n_pages * page_size
    int32_t n_pages, page_size;
    PageDivision pages;
};

// Where a slot's row lies in head 0, in bytes and in scales; the slot is inside the cache
struct RowPlace {
    int64_t row = 0, scale = 0;
    __device__ __forceinline__ RowPlace() {}
    __device__ __forceinline__ RowPlace(const CacheView& c, int64_t slot) {
        const int64_t page = (slot >> 31) == 0 ? (int64_t)c.pages.page_of((uint32_t)slot) : slot / c.page_size;
        const int64_t r = slot - page * c.page_size;
        row = page * c.page_stride + r * c.row_stride;
        scale = page * c.s_page + r * c.s_row;
    }
};

// --------------------------------------------------------------------------------------------------------- host
inline int check_cache(const char* fn, const lora_cache_t* c, CacheView* out) {
    const std::string f(fn);
    if (!c) return refuse(LORA_ERR_INVALID_ARG, f + ": cache is NULL");
    if (c->dtype != LORA_CACHE_BF16 && c->dtype != LORA_CACHE_E4M3)
        return refuse(LORA_ERR_DTYPE, f + ": unknown element type of the cache");
    if (c->n_pages < 0 || c->page_size < 1 || c->n_heads < 1)
        return refuse(LORA_ERR_INVALID_ARG, f + ": a cache has pages of at least one row and one head");
    if (c->head_dim < 16 || c->head_dim > kMaxHeadDim || c->head_dim % 16 != 0 || c->n_heads > kMaxHeads)
        return refuse(LORA_ERR_LIMIT, f + ": a head's size must be a multiple of 16, at most 256; at most 1024 heads");
    const bool e4m3 = c->dtype == LORA_CACHE_E4M3;
    const int64_t e = e4m3 ? 1 : 2;
    if (c->n_pages > 0) {
        if (!c->k || !c->v || (e4m3 && (!c->k_scales || !c->v_scales)))
            return refuse(LORA_ERR_INVALID_ARG, f + ": the cache's keys, values or scales are NULL");
        if (!is_aligned(c->k, 16) || !is_aligned(c->v, 16) || (c->page_stride * e) % 16 || (c->head_stride * e) % 16 ||
            (c->row_stride * e) % 16)
            return refuse(LORA_ERR_ALIGNMENT, f + ": the cache must be 16-byte aligned, its strides multiples of 16 bytes");
        if (e4m3 && (!is_aligned(c->k_scales, 4) || !is_aligned(c->v_scales, 4)))
            return refuse(LORA_ERR_ALIGNMENT, f + ": the cache's scales must be aligned to an element");
        if (c->page_stride < 0 || c->head_stride < 0 || c->row_stride < 0 || c->scale_page_stride < 0 ||
            c->scale_head_stride < 0 || c->scale_row_stride < 0)
            return refuse(LORA_ERR_INVALID_ARG, f + ": the cache's strides must not be negative");
    }
    out->k = static_cast<char*>(c->k);
    out->v = static_cast<char*>(c->v);
    out->ks = c->k_scales;
    out->vs = c->v_scales;
    out->page_stride = c->page_stride * e;
    out->head_stride = c->head_stride * e;
    out->row_stride = c->row_stride * e;
    out->s_page = c->scale_page_stride;
    out->s_head = c->scale_head_stride;
    out->s_row = c->scale_row_stride;
    out->n_pages = c->n_pages;
    out->page_size = c->page_size;
    out->slots = (int64_t)c->n_pages * c->page_size;
    out->pages = page_division((uint32_t)c->page_size);
    return LORA_OK;
}

}  // namespace lora
