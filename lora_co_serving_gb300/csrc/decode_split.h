// decode_split.h -- the index arithmetic of the attention over the paged cache, for the device and for host tests: the rows
// that a sequence attends over, their pages, and the split of all sequences' tiles over the CTAs.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define LORA_HD __host__ __device__ __forceinline__
#else
#define LORA_HD inline
#endif

namespace lora {

// n / d for n < 2^31, as a product: (n mul / 2^32 + n) / 2^shift
struct PageDivision {
    uint32_t mul, shift;
    LORA_HD uint32_t page_of(uint32_t n) const {
#ifdef __CUDA_ARCH__
        return (__umulhi(mul, n) + n) >> shift;
#else
        return ((uint32_t)(((uint64_t)mul * n) >> 32) + n) >> shift;
#endif
    }
};
inline PageDivision page_division(uint32_t d) {      // 1 <= d < 2^31
    PageDivision p{0, 0};
    while ((1ull << p.shift) < d) ++p.shift;
    p.mul = (uint32_t)((((1ull << p.shift) - d) << 32) / d + 1);
    return p;
}

// Rows [start, end) that a sequence of `length` rows attends over; window 0: all of them.  poisoned: the sequence is longer
// than its table's row of `width` pages; it then has one row at least, so that its NaN is written.
struct Range {
    int32_t start, end;
    bool poisoned;
    LORA_HD Range(int32_t length, int32_t window, int32_t width, int32_t page_size) {
        const int32_t n = length > 0 ? length : 0;
        const int64_t most = (int64_t)width * page_size;
        poisoned = n > most;
        end = poisoned ? (int32_t)most : n;
        start = window > 0 && window < n ? n - window : 0;
        if (poisoned && start >= end) start = end - 1;
    }
    LORA_HD int32_t tiles(int32_t rows) const {
        return end > start ? (int32_t)(((uint32_t)(end - start) + (uint32_t)rows - 1) / (uint32_t)rows) : 0;
    }
};

// a / b; most numbers here have 32 bits, whose division takes a fraction of the other's time
LORA_HD int64_t quotient(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// What the i-th of `of` takes of n, [first, last)
struct Share {
    int32_t first, last;
    LORA_HD Share(int32_t n, int32_t i, int32_t of) {
        const int64_t per = ((int64_t)n + of - 1) / of, from = i * per;
        first = (int32_t)(from < n ? from : n);
        last = (int32_t)(from + per < n ? from + per : n);
    }
};

// `tiles` in one line, in equal pieces: CTA c takes [first_tile(c), first_tile(c + 1)).  ctas <= tiles.
struct Line {
    int64_t tiles, ctas;
    LORA_HD int64_t first_tile(int64_t c) const { return quotient(c * tiles, ctas); }
    LORA_HD int64_t owner(int64_t p) const { return quotient((p + 1) * ctas - 1, tiles); }
};

}  // namespace lora
