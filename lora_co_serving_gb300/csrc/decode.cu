// decode.cu -- attention of one new token of each sequence over the paged cache (include/lora_attention.h).
//
// What bounds it: each cached element is used by the n query heads of its group only, 4 n operations for 2 bytes (or one).
// The cache's bytes bound the call at any matrix rate above some 100 TFLOP/s, so the products are small register-to-
// register MMAs (m16n8k16) whose operands come straight from global memory: rows of scores are queries, columns cached
// tokens.  Both products can take the cache as it lies, without a way through shared memory:
//   scores  the sum over a head's elements may be taken in any order, so a lane's 16 bytes of a key row are its share of
//           the B operand of two MMAs (four in 8 bits), if the query's elements are taken in the same order;
//   output  B needs a pair of tokens of one element in a register: a lane loads the same 16 bytes of a pair's two value
//           rows and interleaves them; which element is which output column is free, too.
// Work is counted in tiles of 64 tokens of one sequence and one cache head.  All tiles of a call form one line, and each
// CTA takes an equal piece of it, whatever the lengths are; a CTA's warps take 16 tokens of a tile each, with a running
// maximum and sum of their own.  A sequence and head whose tiles lie in several CTAs is joined by the last of them to
// arrive, in the order of the tiles.
#include <algorithm>
#include <type_traits>

#include "cache.h"
#include "decode_split.h"
#include "tc_prims.h"

namespace lora {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kWarpTokens = 16;
constexpr int kTileTokens = kWarps * kWarpTokens;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// A running maximum is raised only when a score exceeds it by a factor of 2^kSlack: probabilities stay below that.
constexpr float kSlack = 8.f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_fast(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c += a b for bf16 (kHalf: fp16) operands, m16n8k16
template <bool kHalf>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (kHalf)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
            "%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
            "%2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// two numbers in 16 bits, and what that rounding leaves in 16 bits more
template <bool kHalf>
__device__ __forceinline__ void split(float a, float b, uint32_t& hi, uint32_t& lo) {
    if constexpr (kHalf) {
        hi = pack_half(a, b);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        lo = pack_half(a - f.x, b - f.y);
    } else {
        hi = pack_bf16(a, b);
        lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
    }
}
// two e4m3 codes (the low 16 bits) as fp16, exactly
__device__ __forceinline__ uint32_t codes_to_half(uint32_t q) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)q, __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

struct Decode {
    const __nv_bfloat16* q;
    int64_t ld_q;
    __nv_bfloat16* out;
    int64_t ld_out;
    float* lse;
    const int32_t* table;
    int64_t ld_table;
    const int32_t* lengths;
    CacheView cache;
    int32_t B, n_heads, kv_heads, D;
    int32_t group;           // query heads of a cache head
    int32_t parts, rows;     // a group is taken in `parts` of up to `rows` (<= 8 or 16) query heads
    int32_t table_width, window;
    PageDivision pages;
    float scale, softcap;
    int32_t* counters;
    float* ws;
};

__device__ __forceinline__ Range range_of(const Decode& a, int32_t b) {
    return Range(a.lengths[b], a.window, a.table_width, a.cache.page_size);
}

// A warp's 16 tokens: where each token's row lies, one token a lane (and once more in lanes 16 to 31)
struct Rows {
    int64_t at;              // bytes from head 0 of the cache; -1: no token, or no page
    float scale;             // 8 bits: the token's key scale (lanes 16 to 31: value scale)
};

template <bool kE4m3, int kD, int kRows>
struct Warp {
    static constexpr int kKeyLoads = kE4m3 ? kD / 64 : kD / 32;            // 16-byte pieces of a key row in a lane
    static constexpr int kValueLoads = kE4m3 ? (kD + 127) / 128 : kD / 64; // pieces of a value row
    static constexpr bool kNarrow = kE4m3 && kD == 64;                     // value pieces of 8 bytes
    static constexpr int kOut = kD / 8;                                    // column tiles of the output
    static constexpr int kPerPiece = kE4m3 && !kNarrow ? 16 : 8;           // elements of a value piece

    uint4 key[2][kKeyLoads];
    uint4 value[4][kValueLoads];
    float o[kOut][4];

    __device__ __forceinline__ void load_keys(const char* base, int64_t at, int D) {
        const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t off = __shfl_sync(0xffffffffu, at, 8 * j + g);
#pragma unroll
            for (int i = 0; i < kKeyLoads; ++i) {
                const int byte = 64 * i + 16 * c;
                key[j][i] = off >= 0 && byte < (kE4m3 ? D : 2 * D) ? *reinterpret_cast<const uint4*>(base + off + byte)
                                                                  : make_uint4(0, 0, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void load_values(const char* base, int64_t at, int D) {
        const int lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t off = __shfl_sync(0xffffffffu, at, 8 * (j / 2) + 2 * c + j % 2);
#pragma unroll
            for (int i = 0; i < kValueLoads; ++i) {
                value[j][i] = make_uint4(0, 0, 0, 0);
                if constexpr (kNarrow) {
                    if (off >= 0 && 8 * g < D) {
                        const uint2 w = *reinterpret_cast<const uint2*>(base + off + 8 * g);
                        value[j][i].x = w.x;
                        value[j][i].y = w.y;
                    }
                } else {
                    const int byte = 128 * i + 16 * g;
                    if (off >= 0 && byte < (kE4m3 ? D : 2 * D))
                        value[j][i] = *reinterpret_cast<const uint4*>(base + off + byte);
                }
            }
        }
    }
    // s[j]: products of this lane's queries (rows g, g + 8) with tokens 8 j + 2 c and the next one
    template <class Query>
    __device__ __forceinline__ void scores(const Query& q, float (&s)[2][4]) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
        for (int i = 0; i < kKeyLoads; ++i)
#pragma unroll
            for (int m = 0; m < (kE4m3 ? 4 : 2); ++m)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w[4] = {key[j][i].x, key[j][i].y, key[j][i].z, key[j][i].w};
                    const int k = i * (kE4m3 ? 4 : 2) + m;
                    const uint32_t b0 = kE4m3 ? codes_to_half(w[m]) : w[2 * m % 4];
                    const uint32_t b1 = kE4m3 ? codes_to_half(w[m] >> 16) : w[(2 * m + 1) % 4];
                    mma<kE4m3>(s[j], q.lo[2 * k], kRows > 8 ? q.hi[2 * k] : 0u, q.lo[2 * k + 1],
                               kRows > 8 ? q.hi[2 * k + 1] : 0u, b0, b1);
                }
    }
    // o += p v.  p[j]: as scores.  Probabilities go in as a number of 16 bits and one for the rest of it.  With up to 8
    // queries the rest takes the place of rows 8 to 15.
    __device__ __forceinline__ void accumulate(const float (&p)[2][4]) {
        uint32_t hi[2][2], lo[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            split<kE4m3>(p[j][0], p[j][1], hi[j][0], lo[j][0]);
            if constexpr (kRows > 8) split<kE4m3>(p[j][2], p[j][3], hi[j][1], lo[j][1]);
        }
#pragma unroll
        for (int i = 0; i < kValueLoads; ++i)
#pragma unroll
            for (int e = 0; e < kPerPiece; ++e) {
                uint32_t b[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t u[4] = {value[2 * j][i].x, value[2 * j][i].y, value[2 * j][i].z, value[2 * j][i].w};
                    const uint32_t w[4] = {value[2 * j + 1][i].x, value[2 * j + 1][i].y, value[2 * j + 1][i].z,
                                           value[2 * j + 1][i].w};
                    if constexpr (kE4m3) {
                        const uint32_t x = __byte_perm(u[e / 4], w[e / 4], e % 4 < 2 ? 0x5140 : 0x7362);
                        b[j] = codes_to_half(e % 2 ? x >> 16 : x);
                    } else {
                        b[j] = __byte_perm(u[e / 2 % 4], w[e / 2 % 4], e % 2 ? 0x7632 : 0x5410);
                    }
                }
                float(&t)[4] = o[i * kPerPiece + e];
                if constexpr (kRows > 8) {
                    mma<kE4m3>(t, hi[0][0], hi[0][1], hi[1][0], hi[1][1], b[0], b[1]);
                    mma<kE4m3>(t, lo[0][0], lo[0][1], lo[1][0], lo[1][1], b[0], b[1]);
                } else {
                    mma<kE4m3>(t, hi[0][0], lo[0][0], hi[1][0], lo[1][0], b[0], b[1]);
                }
            }
    }
    // element of a head that o[t][e] belongs to (e = 0, 1 of row g; 2, 3 of row g + 8)
    static __device__ __forceinline__ int element(int t, int e) {
        const int c = threadIdx.x % 4;
        return (t / kPerPiece) * 8 * kPerPiece + (2 * c + (e & 1)) * kPerPiece + t % kPerPiece;
    }
};

// A group's queries as A operands, in the order of elements that Warp::scores takes; 8-bit caches: as fp16, scaled by a
// power of two that brings the largest element to 2^14, so that what 16 bits of bf16 hold stays exact over 31 binades
template <bool kE4m3, int kD, int kRows>
struct Query {
    static constexpr int kRegs = kD / 8;
    uint32_t lo[kRegs], hi[kRows > 8 ? kRegs : 1];
    float unit[2];           // what a product of rows g, g + 8 has to be multiplied by

    __device__ __forceinline__ void load_row(const __nv_bfloat16* row, bool in, int D, uint32_t* to, float* unit_) {
        const int c = threadIdx.x % 4;
        constexpr int kPieces = kD / 32;
        uint4 w[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            // 8-bit keys: a lane's 16 elements are two of these pieces
            const int at = kE4m3 ? 64 * (i / 2) + 16 * c + 8 * (i % 2) : 32 * i + 8 * c;
            w[i] = in && at < D ? *reinterpret_cast<const uint4*>(row + at) : make_uint4(0, 0, 0, 0);
        }
        float inv = 1.f;
        *unit_ = 1.f;
        if constexpr (kE4m3) {
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                Row8Bf16 r;
                r.q = w[i];
                a = max(a, r.abs_max());
            }
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
            const int e = min(max((int)(a >> 23) - 127, -112), 127);
            inv = a >= 0x7F800000u ? NAN : __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            *unit_ = a >= 0x7F800000u ? NAN : __uint_as_float((uint32_t)(127 - 14 + e) << 23);
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                to[4 * i + k] = kE4m3 ? pack_half(__uint_as_float(u[k] << 16) * inv, __uint_as_float(u[k] & 0xFFFF0000u) * inv)
                                      : u[k];
        }
    }
    __device__ __forceinline__ void load(const Decode& a, int b, int head0, int rows) {
        const int g = threadIdx.x % 32 / 4;
        const __nv_bfloat16* q = a.q + b * a.ld_q + (int64_t)head0 * a.D;
        load_row(q + g * a.D, g < rows, a.D, lo, &unit[0]);
        if constexpr (kRows > 8) load_row(q + (g + 8) * a.D, g + 8 < rows, a.D, hi, &unit[1]);
    }
};

// Running maximum and sum of a row of scores.  With a scale for each value row (8 bits), the numerators e^s * scale have
// a maximum of their own, in log2: what a large scale does to it leaves the sum alone.
struct Stats {
    float m, l, top;
};

template <bool kE4m3, int kD, int kRows, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) decode_kernel(const Decode a) {
    extern __shared__ __align__(16) float smem[];
    __shared__ int32_t sh_seq;
    __shared__ int64_t sh_before;
    __shared__ int64_t warp_sum[kWarps];
    __shared__ float sh_m[kWarps][kRows], sh_l[kWarps][kRows];
    __shared__ int32_t sh_last;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, c = lane % 4;
    grid_dep_launch();
    grid_dep_wait();

    // ---- this CTA's piece of the line of tiles: [p0, p1) of W, and the sequence that p0 lies in
    const int heads = a.kv_heads * a.parts;           // lines of tiles of one sequence
    const int per = (a.B + kThreads - 1) / kThreads;  // sequences of a thread
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += range_of(a, b).tiles(kTileTokens);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int64_t W = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += warp_sum[w];
        W += warp_sum[w];
    }
    W *= heads;
    const Line all{W, min((int64_t)gridDim.x, W)};
    const int64_t p0 = blockIdx.x < all.ctas ? all.first_tile(blockIdx.x) : W;
    const int64_t p1 = blockIdx.x < all.ctas ? all.first_tile(blockIdx.x + 1) : W;
    if (p0 < p1 && (upto - mine) * heads <= p0 && p0 < upto * heads) {
        int64_t before = upto - mine;
        int b = b0;
        for (;; ++b) {
            const int n = range_of(a, b).tiles(kTileTokens);
            if (p0 < (before + n) * heads) break;
            before += n;
        }
        sh_seq = b;
        sh_before = before * heads;
    }
    // sequences without rows: no tile, so the CTAs share them out
    for (int b = blockIdx.x * kWarps + warp; b < a.B; b += gridDim.x * kWarps) {
        if (range_of(a, b).tiles(kTileTokens) > 0) continue;
        for (int i = lane; i < a.n_heads * a.D / 8; i += 32)
            reinterpret_cast<uint4*>(a.out + b * a.ld_out)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = lane; i < a.n_heads; i += 32) a.lse[(int64_t)b * a.n_heads + i] = -INFINITY;
    }
    __syncthreads();
    if (p0 >= p1) return;
    int b = sh_seq;
    int64_t before = sh_before;

    int64_t p = p0;
    while (p < p1) {
        // ---- the next item: a sequence and a line of its tiles
        const Range range = range_of(a, b);
        const int n_tiles = range.tiles(kTileTokens);
        if (p >= before + (int64_t)n_tiles * heads) {
            before += (int64_t)n_tiles * heads;
            ++b;
            continue;
        }
        const int line = (int)((p - before) / n_tiles);      // a cache head, or a part of its group
        const int64_t i0 = before + (int64_t)line * n_tiles, i1 = i0 + n_tiles;
        const int kv = line / a.parts, part = line % a.parts;
        const int head0 = kv * a.group + part * a.rows, rows = min(a.rows, a.group - part * a.rows);
        const int t0 = (int)(p - i0), t1 = (int)(min(p1, i1) - i0);
        const char* kbase = a.cache.k + kv * a.cache.head_stride;
        const char* vbase = a.cache.v + kv * a.cache.head_stride;
        const int32_t* table = a.table + b * a.ld_table;

        Warp<kE4m3, kD, kRows> w;
        Query<kE4m3, kD, kRows> q;
        Stats st[kRows > 8 ? 2 : 1];
        for (auto& x : st) x = Stats{-INFINITY, 0.f, -INFINITY};
#pragma unroll
        for (int t = 0; t < kD / 8; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) w.o[t][e] = 0.f;
        bool bad = range.poisoned;

        // this warp's first token of tile t, and the page of this lane's (-1: a negative one, -2: no such token)
        auto token = [&](int t) { return (uint32_t)range.start + (uint32_t)t * kTileTokens + warp * kWarpTokens; };
        auto page_at = [&](int t) -> int32_t {
            const uint32_t tok = token(t) + lane % 16;
            return t < t1 && tok < (uint32_t)range.end ? max(table[a.pages.page_of(tok)], -1) : -2;
        };
        auto rows_at = [&](int t, int32_t page) -> Rows {
            Rows r{-1, 0.f};
            if (page == -2) return r;
            if (page == -1 || page >= a.cache.n_pages) {
                bad = true;
                return r;
            }
            const uint32_t tok = token(t) + lane % 16;
            const int64_t row = tok - a.pages.page_of(tok) * (uint32_t)a.cache.page_size;
            r.at = page * a.cache.page_stride + row * a.cache.row_stride;
            if (kE4m3)
                r.scale = (lane < 16 ? a.cache.ks : a.cache.vs)[page * a.cache.s_page + row * a.cache.s_row +
                                                               kv * a.cache.s_head];
            return r;
        };
        int32_t page = page_at(t0);
        Rows now = rows_at(t0, page);
        page = page_at(t0 + 1);
        w.load_keys(kbase, now.at, a.D);
        w.load_values(vbase, now.at, a.D);
        q.load(a, b, head0, rows);
        for (int t = t0; t < t1; ++t) {
            const Rows next = rows_at(t + 1, page);
            page = page_at(t + 2);
            float s[2][4];
            w.scores(q, s);
            if (t + 1 < t1) w.load_keys(kbase, next.at, a.D);
            // scores in log2, -infinity where there is no token
            const uint32_t tok = token(t) + 2 * c;
            float top[2][4], vs[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool in = tok + 8 * j + e < (uint32_t)range.end;
                    float ks = 1.f;
                    if (kE4m3) {
                        ks = __shfl_sync(0xffffffffu, now.scale, 8 * j + 2 * c + e);
                        vs[j][e] = __shfl_sync(0xffffffffu, now.scale, 16 + 8 * j + 2 * c + e);
                    }
#pragma unroll
                    for (int h = 0; h < (kRows > 8 ? 2 : 1); ++h) {
                        float& x = s[j][2 * h + e];
                        if (kE4m3) x *= ks * q.unit[h];
                        x *= a.scale;
                        if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                        x = in ? x * kLog2e : -INFINITY;
                        if (kE4m3) top[j][2 * h + e] = x + log2_fast(fabsf(vs[j][e]));
                    }
                }
            bool raise = false;
            float to[kRows > 8 ? 2 : 1][2];
#pragma unroll
            for (int h = 0; h < (kRows > 8 ? 2 : 1); ++h) {
                float m = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                to[h][0] = m;
                if (kE4m3) {
                    float u = fmaxf(fmaxf(top[0][2 * h], top[0][2 * h + 1]), fmaxf(top[1][2 * h], top[1][2 * h + 1]));
                    u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 1));
                    u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, 2));
                    to[h][1] = u;
                    raise |= u > st[h].top + kSlack;
                }
                raise |= m > st[h].m + kSlack;
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int h = 0; h < (kRows > 8 ? 2 : 1); ++h) {
                    const float m = fmaxf(st[h].m, to[h][0]);
                    const float fl = st[h].m == m ? 1.f : exp2_fast(st[h].m - m);
                    st[h].l *= fl;
                    st[h].m = m;
                    float fo = fl;
                    if (kE4m3) {
                        const float u = fmaxf(st[h].top, to[h][1]);
                        fo = st[h].top == u ? 1.f : exp2_fast(st[h].top - u);
                        st[h].top = u;
                    }
                    // rows 8 to 15 belong to the same queries where there are up to 8
#pragma unroll
                    for (int i = 0; i < kD / 8; ++i)
#pragma unroll
                        for (int e = 0; e < (kRows > 8 ? 2 : 4); ++e) w.o[i][2 * h + e] *= fo;
                }
            }
#pragma unroll
            for (int h = 0; h < (kRows > 8 ? 2 : 1); ++h) {
                const float m = st[h].m == -INFINITY ? 0.f : st[h].m;
                const float u = st[h].top == -INFINITY ? 0.f : st[h].top;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& x = s[j][2 * h + e];
                        const float pr = exp2_fast(x - m);
                        st[h].l += pr;
                        // 2^7 (2^15 with the slack) is the largest numerator: what is lost below 2^-24 is 2^-31 of it
                        x = kE4m3 ? copysignf(exp2_fast(top[j][2 * h + e] - u + 7.f), vs[j][e]) : pr;
                        if (kE4m3 && pr != pr) x = pr;
                    }
            }
            w.accumulate(s);
            if (t + 1 < t1) w.load_values(vbase, next.at, a.D);
            now = next;
        }
        bad = __any_sync(0xffffffffu, bad);

        // ---- the warps' rows together: m and l of each, then the elements
        float* so = smem;        // [kWarps][kRows][kD]
#pragma unroll
        for (int h = 0; h < (kRows > 8 ? 2 : 1); ++h) {
            float l = st[h].l;
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (bad) l = NAN;
            const int row = g + 8 * h;
            if (c == 0) {
                sh_m[warp][row] = st[h].m;
                sh_l[warp][row] = l;
            }
            float unit = 1.f;
            if (kE4m3) unit = st[h].top == -INFINITY ? 1.f : exp2_fast(st[h].top - 7.f - st[h].m);
#pragma unroll
            for (int i = 0; i < kD / 8; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    so[(warp * kRows + row) * kD + w.element(i, e)] =
                        (kRows > 8 ? w.o[i][2 * h + e] : w.o[i][e] + w.o[i][2 + e]) * unit;
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == n_tiles;
        const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
        constexpr int kSlot = kRows * (kD + 2);
        for (int i = tid; i < rows * (kD / 4); i += kThreads) {
            const int row = i / (kD / 4), d = i % (kD / 4) * 4;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) m = fmaxf(m, sh_m[k][row]);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float f = sh_m[k][row] == m ? 1.f : exp2_fast(sh_m[k][row] - m);
                const float4 x = *reinterpret_cast<const float4*>(so + (k * kRows + row) * kD + d);
                l = fmaf(sh_l[k][row], f, l);
                o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y); o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
            }
            if (!whole) {
                float* to = a.ws + (int64_t)slot * kSlot;
                if (d == 0) {
                    to[2 * row] = m;
                    to[2 * row + 1] = l;
                }
                *reinterpret_cast<float4*>(to + 2 * kRows + row * kD + d) = o;
            } else if (d < a.D) {
                const float r = 1.f / l;
                *reinterpret_cast<uint2*>(a.out + b * a.ld_out + (int64_t)(head0 + row) * a.D + d) =
                    make_uint2(pack_bf16(o.x * r, o.y * r), pack_bf16(o.z * r, o.w * r));
                if (d == 0 && a.lse) a.lse[(int64_t)b * a.n_heads + head0 + row] = (m + log2f(l)) * kLn2;
            }
        }
        if (!whole) {
            // ---- joined by the last CTA of the item to arrive, in the order of the CTAs
            const int first = (int)all.owner(i0), last = (int)all.owner(i1 - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) sh_last = atomicAdd(a.counters + first, 1) == last - first;
            __syncthreads();
            if (sh_last) {
                __threadfence();
                if (tid == 0) a.counters[first] = 0;
                for (int i = tid; i < rows * (kD / 4); i += kThreads) {
                    const int row = i / (kD / 4), d = i % (kD / 4) * 4;
                    float m = -INFINITY, l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k = first; k <= last; ++k)
                        m = fmaxf(m, a.ws[(int64_t)(2 * k + (k == first)) * kSlot + 2 * row]);
                    for (int k = first; k <= last; ++k) {
                        const float* from = a.ws + (int64_t)(2 * k + (k == first)) * kSlot;
                        const float f = from[2 * row] == m ? 1.f : exp2_fast(from[2 * row] - m);
                        const float4 x = *reinterpret_cast<const float4*>(from + 2 * kRows + row * kD + d);
                        l = fmaf(from[2 * row + 1], f, l);
                        o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y); o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
                    }
                    if (d >= a.D) continue;
                    const float r = 1.f / l;
                    *reinterpret_cast<uint2*>(a.out + b * a.ld_out + (int64_t)(head0 + row) * a.D + d) =
                        make_uint2(pack_bf16(o.x * r, o.y * r), pack_bf16(o.z * r, o.w * r));
                    if (d == 0 && a.lse) a.lse[(int64_t)b * a.n_heads + head0 + row] = (m + log2f(l)) * kLn2;
                }
            }
        }
        __syncthreads();
        p = min(p1, i1);
    }
}

// ---------------------------------------------------------------------------------------------------------- host
constexpr size_t kCounterBytes = LORA_DECODE_COUNTER_BYTES;

// CTAs on an SM: as many as the registers of a lane's pieces and sums leave room for
constexpr int ctas_of(bool e4m3, int kD, int kRows) { return kD == 256 ? 2 : kRows > 8 ? (e4m3 ? 3 : 2) : (e4m3 ? 4 : 3); }

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

template <class Go>
auto by_shape(bool e4m3, int D, int rows, Go go) {
    auto with_rows = [&](auto t, auto d) {
        return rows <= 8 ? go(t, d, std::integral_constant<int, 8>()) : go(t, d, std::integral_constant<int, 16>());
    };
    auto with_size = [&](auto t) {
        return D <= 64 ? with_rows(t, std::integral_constant<int, 64>())
                       : D <= 128 ? with_rows(t, std::integral_constant<int, 128>())
                                  : with_rows(t, std::integral_constant<int, 256>());
    };
    return e4m3 ? with_size(std::true_type()) : with_size(std::false_type());
}

// Query heads of a group that are taken together
int rows_of(int group) {
    const int parts = (group + 15) / 16;
    return (group + parts - 1) / parts;
}

struct Shape {
    int grid;
    size_t bytes;
};
Shape shape_of(bool e4m3, int D, int group) {
    return by_shape(e4m3, D, rows_of(group), [&](auto t, auto d, auto r) {
        const int grid = std::min<int>(sm_count() * ctas_of(decltype(t)::value, decltype(d)::value, decltype(r)::value),
                                       kCounterBytes / sizeof(int32_t));
        return Shape{grid, kCounterBytes + (size_t)grid * 2 * decltype(r)::value * (decltype(d)::value + 2) * sizeof(float)};
    });
}

int check_heads(const char* fn, int32_t n_heads, const lora_cache_t* cache) {
    if (n_heads < 1 || n_heads % cache->n_heads != 0)
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": n_heads must be a multiple of the cache's heads");
    if (n_heads > kMaxHeads) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 1024 heads");
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" size_t lora_decode_workspace_size(int32_t n_heads, const lora_cache_t* cache) {
    const int64_t n = guarded([&]() -> int64_t {
        const char* fn = "lora_decode_workspace_size";
        CacheView view;
        if (check_cache(fn, cache, &view) != LORA_OK || check_heads(fn, n_heads, cache) != LORA_OK) return 0;
        const Shape s = shape_of(cache->dtype == LORA_CACHE_E4M3, cache->head_dim, n_heads / cache->n_heads);
        if (s.grid == 0) {
            refuse(LORA_ERR_CUDA, std::string(fn) + ": no CUDA device");
            return 0;
        }
        return (int64_t)s.bytes;
    });
    return n > 0 ? (size_t)n : 0;
}

extern "C" int lora_decode_attention(int32_t B, int32_t n_heads, const void* q, int64_t ld_q, const lora_cache_t* cache,
                                     const int32_t* table, int64_t ld_table, int32_t table_width, const int32_t* lengths,
                                     int32_t window, float scale, float softcap, void* out, int64_t ld_out, float* lse,
                                     void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_decode_attention";
        Decode a = {};
        int rc = check_cache(fn, cache, &a.cache);
        if (rc != LORA_OK) return rc;
        if ((rc = check_heads(fn, n_heads, cache)) != LORA_OK) return rc;
        if (B < 0 || window < 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": B and window must be >= 0");
        if (!(fabsf(scale) < INFINITY) || !(softcap >= 0.f && softcap < INFINITY))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": scale must be finite, softcap finite and >= 0");
        if (B == 0) return LORA_OK;
        const int64_t cols = (int64_t)n_heads * cache->head_dim;
        if ((rc = check_matrix(fn, "q", q, cols, ld_q, 2)) != LORA_OK) return rc;
        if ((rc = check_matrix(fn, "out", out, cols, ld_out, 2)) != LORA_OK) return rc;
        if (!table || !lengths) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": table or lengths is NULL");
        if (table_width < 1 || ld_table < table_width)
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": rows of table are empty or overlap");
        if (!is_aligned(table, 4) || !is_aligned(lengths, 4) || (lse && !is_aligned(lse, 4)))
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": table, lengths and lse must be 4-byte aligned");
        const bool e4m3 = cache->dtype == LORA_CACHE_E4M3;
        a.group = n_heads / cache->n_heads;
        const Shape shape = shape_of(e4m3, cache->head_dim, a.group);
        if (shape.grid == 0) return refuse(LORA_ERR_CUDA, std::string(fn) + ": no CUDA device");
        if (!workspace || !is_aligned(workspace, 256) || ws_bytes < shape.bytes)
            return refuse(LORA_ERR_WORKSPACE, std::string(fn) + ": workspace missing, too small or not 256-byte aligned");
        a.q = static_cast<const __nv_bfloat16*>(q); a.ld_q = ld_q;
        a.out = static_cast<__nv_bfloat16*>(out); a.ld_out = ld_out; a.lse = lse;
        a.table = table; a.ld_table = ld_table; a.table_width = table_width; a.lengths = lengths;
        a.B = B; a.n_heads = n_heads; a.kv_heads = cache->n_heads; a.D = cache->head_dim;
        a.rows = rows_of(a.group);
        a.parts = (a.group + a.rows - 1) / a.rows;
        a.window = window; a.scale = scale; a.softcap = softcap;
        a.pages = page_division((uint32_t)cache->page_size);
        a.counters = static_cast<int32_t*>(workspace);
        a.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return enqueued(fn, by_shape(e4m3, a.D, a.rows, [&](auto t, auto kd, auto r) -> cudaError_t {
            constexpr bool kE4m3 = decltype(t)::value;
            constexpr int kD = decltype(kd)::value, kRows = decltype(r)::value;
            const auto kernel = decode_kernel<kE4m3, kD, kRows, ctas_of(kE4m3, kD, kRows)>;
            constexpr size_t smem = sizeof(float) * kWarps * kRows * kD;
            if (smem > 48 * 1024) {
                const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
                if (e != cudaSuccess) return e;
            }
            return launch_pdl(kernel, dim3((unsigned)shape.grid), dim3(kThreads), smem, st, a);
        }));
    });
}
