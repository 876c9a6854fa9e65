// decode.cu -- attention of one new token of each sequence over the paged cache (include/lora_attention.h).
//
// What bounds it: each cached element is used by the n query heads of its group only, 4 n operations for 2 bytes (or one).
// The cache's bytes bound the call at any matrix rate above some 100 TFLOP/s, so the products are small MMAs of a warp
// (m16n8k16): the cache's side has the 16 rows, up to 8 query heads the 8 columns.  Both take the cache as it lies, with
// no exchange between lanes:
//   scores  rows are tokens.  The sum over a head's elements may be taken in any order, so a lane's 16 bytes of a key row
//           are its share of two MMAs, if the query's elements are taken in the same order;
//   output  rows are elements, the sum goes over tokens, a pair of them in a register: a lane takes the same 16 bytes of a
//           pair's two value rows and interleaves them.  Which element is which row is free, too.  The probabilities, whose
//           tokens are rows, are turned around by the transposing move of 8 x 8 numbers.
// Every warp copies its rows into shared memory two steps ahead of their use, asynchronously, 512 neighbouring bytes at a
// time, and reads them back as its lanes need them: a barrier within the warp is all that it takes.  (Lanes that copied
// their own pieces, 64 bytes of 8 rows at a time, needed one and a half times the requests to L2: 236 us instead of 187
// for 64 x 8192 tokens in bf16.)
// Work is counted in tiles of 32 to 128 tokens of one sequence and one cache head.  All tiles of a call form one line, and
// each CTA takes an equal piece of it, whatever the lengths are; a CTA's warps take 16 or 32 tokens of a tile each, with a
// running maximum and sum of their own, and the copies run on from one sequence into the next.  A sequence and head whose
// tiles lie in several CTAs is joined by the last of them to arrive, in the order of the tiles.
#include <algorithm>
#include <type_traits>

#include "cache.h"
#include "decode_split.h"
#include "tc_prims.h"

namespace lora {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 912;        // of a launch, which the counters have room for; 152 SMs hold 456 (ctas_of)
constexpr int kJoined = 18;          // parts of an item that are joined in one stage
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
// An asynchronous copy of kBytes to shared memory; where `in` is false, zeros
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from, bool in) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(kBytes), "r"(in ? kBytes : 0)
                     : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most kPending of the thread's latest groups are under way
template <int kPending>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// the transpose of 8 x 8 numbers of 16 bits: row lane / 4, columns 2 (lane % 4) and the next
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
// four e4m3 codes as two pairs of fp16, exactly
__device__ __forceinline__ void codes_to_half(uint32_t q, uint32_t& low, uint32_t& high) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(low), "=r"(high)
        : "r"(q));
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
    uint32_t unit, page_units, row_units;      // bytes that divide the cache's strides; the strides in these units
    float scale, softcap;
    int32_t* counters;
    float* ws;
};

__device__ __forceinline__ Range range_of(const Decode& a, int32_t b) {
    return Range(a.lengths[b], a.window, a.table_width, a.cache.page_size);
}

// Shapes of a kernel for cache heads of up to kD elements and kRows query heads at a time.  A warp holds kPart elements of
// each row: 128 at most, so that its sums and its share of the queries stay in registers; heads of 256 are taken by two
// warps, which add up their scores.
template <bool kE4m3_, int kD_, int kRows_>
struct Shapes {
    static constexpr bool kE4m3 = kE4m3_;
    static constexpr int kD = kD_, kRows = kRows_;
    static constexpr int kSplit = kD > 128 ? 2 : 1, kPart = kD / kSplit;
    static constexpr int kTeams = kWarps / kSplit;                         // groups of warps with tokens of their own
    static constexpr int kBytes = kPart * (kE4m3 ? 1 : 2);                 // of a row in a warp
    static constexpr int kTokens = kBytes > 128 ? 16 : 32;                 // of a warp's step: 8 KB of keys and values
    static constexpr int kTile = kTeams * kTokens;
    static constexpr int kMmas = kTokens / 16;                             // MMAs' worth of tokens in a step
    static constexpr int kKeyLoads = kBytes / 64;                          // 16-byte pieces of a key row in a lane
    static constexpr int kPieceBytes = kBytes == 64 ? 8 : 16;              // a lane's piece of a value row
    static constexpr int kValueLoads = kBytes == 64 ? 1 : kBytes / 128;    // such pieces
    static constexpr int kPerPiece = kE4m3 ? kPieceBytes : kPieceBytes / 2;   // elements of one
    static constexpr int kOut = kPart / 16;                                // MMAs' worth of elements of the output
    static constexpr int kCols = kRows / 8;                                // MMAs' worth of queries
    // shared memory of a warp: two steps' keys, values and scales; after an item's last step its place holds the item's
    // sums, [kRows][kPart]
    static constexpr int kKeyBytes = kTokens * kBytes, kStepBytes = 2 * kKeyBytes;
    static_assert(kRows * kPart * 4 <= kStepBytes, "a warp's sums fit a step's place");
    static constexpr int kScaleBytes = kE4m3 ? 2 * 32 * 4 : 0;
    static constexpr int kWarpBytes = 2 * (kStepBytes + kScaleBytes);
    static constexpr int kExchangeFloats = kSplit > 1 ? 2 * kCols * kMmas * 4 * 32 : 0;      // a warp's scores, twice
    static constexpr int kSmem = kWarps * (kWarpBytes + 4 * kExchangeFloats);
    static constexpr int kSlot = kRows * (kD + 2);                         // floats of a part of an item: m, l; sums
};

template <class S>
struct Warp {
    float o[S::kOut][S::kCols][4];

    // Copies of a step's rows, [kTokens][kBytes] of keys, then of values.  rows: where the row of token `lane` of the step
    // lies, in units of a.unit bytes, from `keys`; bytes: of a row.  Pieces of 16 bytes lie in an order of their own in each
    // row, so that the lanes that read them at once (rows g, pieces c of the keys; rows 2 c, pieces g of the values) fall on
    // different banks.
    static constexpr int kAcross = S::kBytes / 16;                         // pieces of a row
    static __device__ __forceinline__ void copy(uint32_t to, const char* keys, int64_t to_values, uint32_t rows, uint32_t unit,
                                                int bytes) {
        const int lane = threadIdx.x % 32, row0 = lane / kAcross, col = lane % kAcross;
        const bool in = 16 * col < bytes;
        const int at_k = (col ^ (kAcross >= 8 ? 4 * (row0 & 1) : 0)) * 16 + row0 * S::kBytes;
        const int at_v = (col ^ (kAcross >= 8 ? row0 & 6 : (row0 >> 1) & 3)) * 16 + row0 * S::kBytes;
#pragma unroll
        for (int k = 0; k < S::kKeyBytes / 512; ++k) {
            const uint32_t at = __shfl_sync(0xffffffffu, rows, k * (32 / kAcross) + row0);
            const char* from = keys + (uint64_t)(in ? at : 0) * unit + 16 * col;      // not read where !in
            copy_async<16>(to + 512 * k + at_k, from, in);
            const int turn = kAcross >= 8 ? k * (32 / kAcross) & 6 : 0;
            copy_async<16>(to + S::kKeyBytes + 512 * k + (at_v ^ (16 * turn)), from + to_values, in);
        }
    }
    // the 16 bytes 4 i + c of the key row of token 8 j + g
    static __device__ __forceinline__ uint4 key(const char* at, int j, int i) {
        const int g = threadIdx.x % 32 / 4, c = threadIdx.x % 4;
        const int off = g * S::kBytes + ((kAcross >= 8 ? 4 * (g & 1) : 0) + c) * 16;
        return *reinterpret_cast<const uint4*>(at + 8 * j * S::kBytes + (off ^ (64 * i)));
    }
    // piece 8 i + g of the value row of token 8 (j / 2) + 2 c + j % 2
    static __device__ __forceinline__ uint4 value(const char* at, int j, int i) {
        const int g = threadIdx.x % 32 / 4, c = threadIdx.x % 4;
        const char* row = at + (8 * (j / 2) + j % 2 + 2 * c) * S::kBytes;
        if constexpr (S::kPieceBytes == 16) return *reinterpret_cast<const uint4*>(row + 128 * i + (g ^ (2 * c)) * 16);
        const uint2 v = *reinterpret_cast<const uint2*>(row + ((g / 2) ^ c) * 16 + g % 2 * 8);
        return make_uint4(v.x, v.y, 0, 0);
    }
    // s[n][m][2 h + f]: the product of token 16 m + 8 h + g with query 8 n + 2 c + f
    template <class Query>
    static __device__ __forceinline__ void scores(const char* keys, const Query& q, float (&s)[S::kCols][S::kMmas][4]) {
#pragma unroll
        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
            for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][m][e] = 0.f;
#pragma unroll
        for (int i = 0; i < S::kKeyLoads; ++i)
#pragma unroll
            for (int m = 0; m < S::kMmas; ++m) {
                const uint4 x = key(keys, 2 * m, i), y = key(keys, 2 * m + 1, i);
                const uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
                constexpr int kSums = S::kE4m3 ? 4 : 2;
#pragma unroll
                for (int k = 0; k < kSums; ++k) {
                    uint32_t v[4];
                    if constexpr (S::kE4m3) {
                        codes_to_half(u[k], v[0], v[2]);
                        codes_to_half(w[k], v[1], v[3]);
                    } else {
                        v[0] = u[2 * k]; v[1] = w[2 * k]; v[2] = u[2 * k + 1]; v[3] = w[2 * k + 1];
                    }
                    const int at = 2 * (i * kSums + k);
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n)
                        mma<S::kE4m3>(s[n][m], v[0], v[1], v[2], v[3], q.reg[n][at], q.reg[n][at + 1]);
                }
            }
    }
    // o += v p, p as scores gives them.  A probability goes in as a number of 16 bits and one for the rest of it.  bf16's 8
    // bits alone would double the square of what rounding the output costs; fp16's 11, beside 8-bit values, make an output now
    // and then a neighbour of the nearest number (64 x 4096 tokens of 16 heads in e4m3 96 us instead of 99, 256 x 2048 of 8
    // heads for 64 110 instead of 114).
    __device__ __forceinline__ void accumulate(const char* values, const float (&p)[S::kCols][S::kMmas][4]) {
        uint32_t hi[S::kCols][S::kMmas][2], lo[S::kCols][S::kMmas][2];
#pragma unroll
        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
            for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = p[n][m][2 * h], y = p[n][m][2 * h + 1];
                    if constexpr (S::kE4m3) {
                        const uint32_t v = pack_half(x, y);
                        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&v));
                        hi[n][m][h] = transposed(v);
                        lo[n][m][h] = transposed(pack_half(x - r.x, y - r.y));
                    } else {
                        const uint32_t v = pack_bf16(x, y);
                        hi[n][m][h] = transposed(v);
                        lo[n][m][h] =
                            transposed(pack_bf16(x - __uint_as_float(v << 16), y - __uint_as_float(v & 0xFFFF0000u)));
                    }
                }
#pragma unroll
        for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
            for (int i = 0; i < S::kValueLoads; ++i) {
                uint32_t v[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 x = value(values, 4 * m + j, i);
                    v[j][0] = x.x; v[j][1] = x.y; v[j][2] = x.z; v[j][3] = x.w;
                }
#pragma unroll
                for (int e = 0; e < S::kPerPiece / 2; ++e) {       // elements 2 e and 2 e + 1 of the piece
                    uint32_t a[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (S::kE4m3) {
                            const uint32_t z = __byte_perm(v[2 * h][e / 2], v[2 * h + 1][e / 2], e % 2 ? 0x7362 : 0x5140);
                            codes_to_half(z, a[2 * h], a[2 * h + 1]);
                        } else {
                            a[2 * h] = __byte_perm(v[2 * h][e], v[2 * h + 1][e], 0x5410);
                            a[2 * h + 1] = __byte_perm(v[2 * h][e], v[2 * h + 1][e], 0x7632);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n) {
                        float(&t)[4] = o[i * S::kPerPiece / 2 + e][n];
                        mma<S::kE4m3>(t, a[0], a[1], a[2], a[3], hi[n][m][0], hi[n][m][1]);
                        mma<S::kE4m3>(t, a[0], a[1], a[2], a[3], lo[n][m][0], lo[n][m][1]);
                    }
                }
            }
    }
    // Where four neighbouring sums of a row, from `element`, lie among a warp's staged sums; turned about by the row, so that
    // lanes of different rows fall on different banks
    static __device__ __forceinline__ int staged(int row, int element) {
        return row * S::kPart + ((element / 4) ^ (row & 7)) * 4;
    }
    // this lane's sums of query row 8 n + 2 c + f, times `by`
    __device__ __forceinline__ void stage(float* to, int n, int f, float by) const {
        const int g = threadIdx.x % 32 / 4, row = 8 * n + 2 * (threadIdx.x % 4) + f;
        constexpr int kHalf = S::kPerPiece / 2;
#pragma unroll
        for (int t = 0; t < S::kOut; t += 2)
            *reinterpret_cast<float4*>(to + staged(row, (t / kHalf * 8 + g) * S::kPerPiece + t % kHalf * 2)) =
                make_float4(o[t][n][f] * by, o[t][n][2 + f] * by, o[t + 1][n][f] * by, o[t + 1][n][2 + f] * by);
    }
};

// A group's queries as B operands, in the order of elements that Warp::scores takes; 8-bit caches: as fp16, scaled by a
// power of two that brings the largest element to between 2^14 and 2^15, so that what bf16 holds stays exact down to 2^-31
// of it.  (The MMAs that take e4m3 convert to fp16 themselves, and again for each call: with one number for a probability,
// queries split into two e4m3 numbers took 135 us instead of 110 for 256 x 2048 tokens.)
template <class S>
struct Query {
    uint32_t reg[S::kCols][S::kPart / 8];
    float unit[S::kCols];    // what a product of query 8 n + g has to be multiplied by

    // the rows as they are, from this warp's first element on; then the operands
    uint4 raw[S::kCols][S::kPart / 32];
    __device__ __forceinline__ void fetch(const Decode& a, int b, int head0, int rows, int first) {
        const int g = threadIdx.x % 32 / 4, c = threadIdx.x % 4;
        const __nv_bfloat16* q = a.q + b * a.ld_q + (int64_t)head0 * a.D + first;
#pragma unroll
        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
            for (int i = 0; i < S::kPart / 32; ++i) {
                // 8-bit keys: a lane's 16 elements are two of these pieces
                const int at = S::kE4m3 ? 64 * (i / 2) + 16 * c + 8 * (i % 2) : 32 * i + 8 * c;
                raw[n][i] = g + 8 * n < rows && at < a.D - first
                                ? *reinterpret_cast<const uint4*>(q + (g + 8 * n) * a.D + at)
                                : make_uint4(0, 0, 0, 0);
            }
    }
    __device__ __forceinline__ void convert() {
#pragma unroll
        for (int n = 0; n < S::kCols; ++n) convert_row(raw[n], reg[n], &unit[n]);
    }
    __device__ __forceinline__ void convert_row(const uint4 (&w)[S::kPart / 32], uint32_t* to, float* unit_) {
        constexpr int kPieces = S::kPart / 32;
        float inv = 1.f;
        *unit_ = 1.f;
        if constexpr (S::kE4m3) {
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
                to[4 * i + k] = S::kE4m3
                                    ? pack_half(__uint_as_float(u[k] << 16) * inv, __uint_as_float(u[k] & 0xFFFF0000u) * inv)
                                    : u[k];
        }
    }
};

// Running maximum m and sum l of a row of scores, in log2.  With a scale for each value row (8 bits) the numerators
// e^s * scale have a maximum of their own: what a large scale does to it leaves the sum alone.
struct Stats {
    float m, l, top;
};

// Sums of one row and four elements over parts that are relative to maxima of their own
struct Joined {
    float m, l;
    float4 o;
    __device__ __forceinline__ void add(float f, float pl, float4 x) {
        l = fmaf(pl, f, l);
        o.x = fmaf(x.x, f, o.x); o.y = fmaf(x.y, f, o.y); o.z = fmaf(x.z, f, o.z); o.w = fmaf(x.w, f, o.w);
    }
    static __device__ __forceinline__ float weight(float from, float to) { return from == to ? 1.f : exp2_fast(from - to); }
};
// parts k = 0 .. n - 1, at(k): [kRows] pairs of m and l, then [kRows, kD] sums.  Eight are loaded at a time.
template <class S, class At>
__device__ __forceinline__ Joined join_parts(int n, int row, int d, At at) {
    Joined r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    constexpr int kAhead = 8;
    for (int k0 = 0; k0 < n; k0 += kAhead) {
        float2 ml[kAhead];
        float4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float* from = at(min(k0 + k, n - 1));
            ml[k] = __ldcg(reinterpret_cast<const float2*>(from + 2 * row));      // other CTAs' writes: not from L1
            x[k] = __ldcg(reinterpret_cast<const float4*>(from + 2 * S::kRows + row * S::kD + d));
        }
        float m = r.m;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) m = fmaxf(m, ml[k].x);
        const float f = Joined::weight(r.m, m);
        r.m = m;
        r.l *= f;
        r.o.x *= f; r.o.y *= f; r.o.z *= f; r.o.w *= f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (k0 + k < n) r.add(Joined::weight(ml[k].x, m), ml[k].y, x[k]);
    }
    return r;
}

// A tile of the line: tile t of one of the lines of sequence b.  A line belongs to a cache head, or a part of its group.
template <class S>
struct Cursor {
    int32_t b, line, t, n_tiles;
    uint32_t start, end;
    bool poisoned;
    __device__ __forceinline__ void enter(const Decode& a) {
        const Range r = range_of(a, b);
        start = r.start;
        end = r.end;
        poisoned = r.poisoned;
        n_tiles = r.tiles(S::kTile);
    }
    // the next tile; the next line's first one; there is one
    __device__ __forceinline__ void next(const Decode& a) {
        if (++t == n_tiles) next_line(a);
    }
    __device__ __forceinline__ void next_line(const Decode& a) {
        t = 0;
        if (++line < a.kv_heads * a.parts) return;
        line = 0;
        do {
            ++b;
            enter(a);
        } while (n_tiles == 0);
    }
};

template <class S, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) decode_kernel(const Decode a) {
    extern __shared__ __align__(128) char smem[];
    __shared__ int32_t sh_seq;
    __shared__ int64_t sh_before;
    __shared__ int64_t warp_sum[kWarps];
    __shared__ float sh_m[S::kTeams][S::kRows], sh_l[S::kTeams][S::kRows];
    __shared__ int32_t sh_last;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, g = lane / 4, c = lane % 4;
    const int team = warp / S::kSplit, side = warp % S::kSplit;
    grid_dep_launch();
    grid_dep_wait();

    // ---- this CTA's piece of the line of tiles, [p0, p1), and the sequence that p0 lies in
    const int heads = a.kv_heads * a.parts;           // lines of tiles of one sequence
    const Share share(a.B, tid, kThreads);            // sequences of a thread
    int64_t mine = 0;
    for (int b = share.first; b < share.last; ++b) mine += range_of(a, b).tiles(S::kTile);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += warp_sum[w];
        total += warp_sum[w];
    }
    total *= heads;
    const Line all{total, min((int64_t)gridDim.x, total)};
    const int64_t p0 = blockIdx.x < all.ctas ? all.first_tile(blockIdx.x) : total;
    const int64_t p1 = blockIdx.x < all.ctas ? all.first_tile(blockIdx.x + 1) : total;
    if (p0 < p1 && (upto - mine) * heads <= p0 && p0 < upto * heads) {
        int64_t before = upto - mine;
        int b = share.first;
        for (;; ++b) {
            const int n = range_of(a, b).tiles(S::kTile);
            if (p0 < (before + n) * heads) break;
            before += n;
        }
        sh_seq = b;
        sh_before = before * heads;
    }
    // sequences without rows have no tile, so the CTAs share them out
    for (uint32_t b = blockIdx.x * kWarps + warp; b < (uint32_t)a.B; b += gridDim.x * kWarps) {
        if (range_of(a, b).tiles(S::kTile) > 0) continue;
        for (int i = lane; i < a.n_heads * a.D / 8; i += 32)
            reinterpret_cast<uint4*>(a.out + b * a.ld_out)[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int i = lane; i < a.n_heads; i += 32) a.lse[(int64_t)b * a.n_heads + i] = -INFINITY;
    }
    __syncthreads();
    if (p0 >= p1) return;

    // ---- the copies, two tiles ahead: `ahead` is the tile to be copied next, whose pages are on their way
    const int first = side * S::kPart;                // this warp's elements of a row
    const int bytes = (a.D - first) * (S::kE4m3 ? 1 : 2);
    char* const mine_at = smem + warp * S::kWarpBytes;
    const uint32_t mine_u32 = smem_u32(mine_at);
    Cursor<S> at;
    at.b = sh_seq;
    at.enter(a);
    at.line = (int)quotient(p0 - sh_before, at.n_tiles);
    at.t = (int)(p0 - sh_before - (int64_t)at.line * at.n_tiles);
    Cursor<S> ahead = at;
    int64_t to_copy = p1 - p0, to_do = p1 - p0;
    int32_t page = 0, following = 0;
    uint32_t bad_steps = 0;                           // bit i: step i's tile has a page outside the cache
    auto token = [&](const Cursor<S>& x) { return x.start + (uint32_t)x.t * S::kTile + team * S::kTokens; };
    // Lanes past the last token take that token's row once more: their scores become -infinity, and 0 times a value of the
    // range adds nothing.
    auto my_token = [&](const Cursor<S>& x) { return min(token(x) + lane % S::kTokens, x.end - 1); };
    auto page_of = [&](const Cursor<S>& x) { return a.table[x.b * a.ld_table + a.cache.pages.page_of(my_token(x))]; };
    auto copy = [&](int step, bool following_known = false) {
        if (to_copy > 0) {
            // a page outside the cache is taken as its first; the result becomes NaN
            const bool bad = (uint32_t)page >= (uint32_t)a.cache.n_pages;
            if (bad) page = 0;
            bad_steps = (bad_steps & ~(1u << step)) | (__any_sync(0xffffffffu, bad) ? 1u << step : 0);
            if (token(ahead) < ahead.end && a.cache.n_pages > 0) {
                const int kv = ahead.line / a.parts;
                const uint32_t tok = my_token(ahead);
                const uint32_t row = tok - a.cache.pages.page_of(tok) * (uint32_t)a.cache.page_size;
                Warp<S>::copy(mine_u32 + step * S::kStepBytes,
                              a.cache.k + kv * a.cache.head_stride + first * (S::kE4m3 ? 1 : 2), a.cache.v - a.cache.k,
                              (uint32_t)page * a.page_units + row * a.row_units, a.unit, bytes);
                if (S::kE4m3) {
                    const int64_t z = page * a.cache.s_page + row * a.cache.s_row + kv * a.cache.s_head;
                    const uint32_t sc = mine_u32 + 2 * S::kStepBytes + step * S::kScaleBytes + lane * 4;
                    copy_async<4>(sc, a.cache.ks + z, true);
                    copy_async<4>(sc + 128, a.cache.vs + z, true);
                }
            }
            if (--to_copy > 0) {
                ahead.next(a);
                page = following_known ? following : page_of(ahead);
            }
        }
        copies_commit();
    };
    // the first two tiles' pages are read at once
    page = page_of(ahead);
    if (to_copy > 1) {
        Cursor<S> second = ahead;
        second.next(a);
        following = page_of(second);
    }
    copy(0, true);
    copy(1);

    Query<S> q;
    auto fetch_queries = [&]() {
        const int kv = at.line / a.parts, part = at.line % a.parts;
        q.fetch(a, at.b, kv * a.group + part * a.rows, min(a.rows, a.group - part * a.rows), first);
    };
    fetch_queries();
    int step = 0;
    int64_t p = p0;
    while (to_do > 0) {
        // ---- the next item: a sequence and a line of its tiles
        const int b = at.b, n_tiles = at.n_tiles, t0 = at.t, t1 = (int)min((int64_t)n_tiles, t0 + to_do);
        const int64_t i0 = p - t0, i1 = i0 + n_tiles;
        const int kv = at.line / a.parts, part = at.line % a.parts;
        const int head0 = kv * a.group + part * a.rows, n_rows = min(a.rows, a.group - part * a.rows);
        Warp<S> w;
        Stats st[S::kCols][2];       // of queries 8 n + 2 c + f
#pragma unroll
        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
            for (int f = 0; f < 2; ++f) st[n][f] = Stats{-INFINITY, 0.f, -INFINITY};
#pragma unroll
        for (int t = 0; t < S::kOut; ++t)
#pragma unroll
            for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) w.o[t][n][e] = 0.f;
        bool bad = at.poisoned;
        q.convert();
        // what a score is multiplied by: its query's unit, the scale, and the change to powers of two
        float factor[S::kCols][2], unit[S::kCols][2];
#pragma unroll
        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                unit[n][f] = __shfl_sync(0xffffffffu, q.unit[n], 4 * (2 * c + f));
                factor[n][f] = (S::kSplit > 1 ? 1.f : unit[n][f]) * (a.softcap > 0.f ? a.scale / a.softcap : a.scale * kLog2e);
            }
        for (;; ++at.t, step ^= 1) {
            const bool last = at.t + 1 == t1;            // the next step's copies then wait: its place takes the item's sums
            const uint32_t tok = token(at);
            bad |= (bad_steps >> step) & 1;
            const char* keys = mine_at + step * S::kStepBytes;
            if (tok < at.end && a.cache.n_pages > 0) {
                copies_wait<1>();
                __syncwarp();
                float s[S::kCols][S::kMmas][4];
                Warp<S>::scores(keys, q, s);
                float ks[S::kMmas][2], lv[S::kMmas][2] = {};       // key scales; log2 of value scales
                if constexpr (S::kE4m3) {
                    const float* sc = reinterpret_cast<const float*>(mine_at + 2 * S::kStepBytes + step * S::kScaleBytes);
#pragma unroll
                    for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ks[m][h] = sc[16 * m + 8 * h + g];
                            lv[m][h] = log2_fast(sc[32 + 16 * m + 8 * h + g]);
                        }
                }
                if constexpr (S::kSplit > 1) {
                    // both warps of a team add the two halves in one order
                    float* const exchange = reinterpret_cast<float*>(smem + kWarps * S::kWarpBytes);
                    auto place = [&](int of, int i, int e) -> float& {
                        return exchange[(2 * team + of) * S::kExchangeFloats +
                                        ((step * S::kMmas * S::kCols + i) * 4 + e) * 32 + lane];
                    };
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                        for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e) place(side, n * S::kMmas + m, e) = s[n][m][e] * unit[n][e % 2];
                    asm volatile("bar.sync %0, 64;" ::"r"(team + 1) : "memory");
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                        for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                s[n][m][e] = place(0, n * S::kMmas + m, e) + place(1, n * S::kMmas + m, e);
                }
                // scores in log2, -infinity where there is no token
#pragma unroll
                for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                float& x = s[n][m][2 * h + f];
                                x *= S::kE4m3 ? ks[m][h] * factor[n][f] : factor[n][f];
                            }
                if (a.softcap > 0.f) {
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                        for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[n][m][e] = a.softcap * kLog2e * tanhf(s[n][m][e]);
                }
                if (tok + S::kTokens > at.end) {
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                        for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (tok + 16 * m + 8 * (e / 2) + g >= at.end) s[n][m][e] = -INFINITY;
                }
                bool raise = false;
#pragma unroll
                for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float most = s[n][0][f], top = most + lv[0][0];
#pragma unroll
                        for (int i = 1; i < 2 * S::kMmas; ++i) {
                            most = fmaxf(most, s[n][i / 2][2 * (i % 2) + f]);
                            if (S::kE4m3) top = fmaxf(top, s[n][i / 2][2 * (i % 2) + f] + lv[i / 2][i % 2]);
                        }
                        raise |= most > st[n][f].m + kSlack;
                        if (S::kE4m3) raise |= top > st[n][f].top + kSlack;
                    }
                if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                    for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            Stats& r = st[n][f];
                            float most = r.m, top = r.top;
#pragma unroll
                            for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    most = fmaxf(most, s[n][m][2 * h + f]);
                                    if (S::kE4m3) top = fmaxf(top, s[n][m][2 * h + f] + lv[m][h]);
                                }
#pragma unroll
                            for (int d = 4; d < 32; d *= 2) {
                                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                                if (S::kE4m3) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            }
                            float by = Joined::weight(r.m, most);
                            r.l *= by;
                            if (S::kE4m3) by = Joined::weight(r.top, top);
                            r.m = most;
                            r.top = top;
#pragma unroll
                            for (int i = 0; i < S::kOut; ++i) {
                                w.o[i][n][f] *= by;
                                w.o[i][n][2 + f] *= by;
                            }
                        }
                }
#pragma unroll
                for (int n = 0; n < S::kCols; ++n)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const float less = st[n][f].m == -INFINITY ? 0.f : st[n][f].m;
                        // 2^7 (2^15 with the slack) is the largest numerator in 8 bits: what its two fp16 numbers lose below
                        // 2^-24 is 2^-31 of it
                        const float top = st[n][f].top == -INFINITY ? -7.f : st[n][f].top - 7.f;
#pragma unroll
                        for (int m = 0; m < S::kMmas; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float& x = s[n][m][2 * h + f];
                                const float pr = exp2_fast(x - less);
                                st[n][f].l += pr;
                                x = S::kE4m3 ? exp2_fast(x + lv[m][h] - top) : pr;
                            }
                    }
                w.accumulate(keys + S::kKeyBytes, s);
                __syncwarp();       // the next copies take the place of what was read
            }
            if (last) break;
            copy(step);
        }
        bad = __any_sync(0xffffffffu, bad);

        // ---- the warps' rows together: m and l of each, then the elements
#pragma unroll
        for (int n = 0; n < S::kCols; ++n)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const Stats& r = st[n][f];
                float l = r.l;
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
                if (bad) l = NAN;
                const int row = 8 * n + 2 * c + f;
                if (g == 0 && side == 0) {
                    sh_m[team][row] = r.m;
                    sh_l[team][row] = l;
                }
                const float by = !S::kE4m3 || r.top == -INFINITY ? 1.f : exp2_fast(r.top - 7.f - r.m);
                w.stage(reinterpret_cast<float*>(mine_at + step * S::kStepBytes), n, f, by);
            }
        to_do -= t1 - t0;
        p += t1 - t0;
        if (to_do > 0) {             // the next item's queries come while this one is joined
            at.next_line(a);
            fetch_queries();
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == n_tiles;
        auto slot = [&](int cta, bool begins) { return a.ws + (int64_t)(2 * cta + (begins ? 1 : 0)) * S::kSlot; };
        auto write_out = [&](int row, int d, const Joined& r) {
            if (d >= a.D) return;
            const float f = 1.f / r.l;
            *reinterpret_cast<uint2*>(a.out + b * a.ld_out + (int64_t)(head0 + row) * a.D + d) =
                make_uint2(pack_bf16(r.o.x * f, r.o.y * f), pack_bf16(r.o.z * f, r.o.w * f));
            if (d == 0 && a.lse) a.lse[(int64_t)b * a.n_heads + head0 + row] = (r.m + log2f(r.l)) * kLn2;
        };
        auto write_part = [&](float* to, int row, int d, const Joined& r) {
            if (d == 0) *reinterpret_cast<float2*>(to + 2 * row) = make_float2(r.m, r.l);
            *reinterpret_cast<float4*>(to + 2 * S::kRows + row * S::kD + d) = r.o;
        };
        for (int i = tid; i < n_rows * (S::kD / 4); i += kThreads) {
            const int row = i / (S::kD / 4), d = i % (S::kD / 4) * 4;
            Joined r{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < S::kTeams; ++k) r.m = fmaxf(r.m, sh_m[k][row]);
#pragma unroll
            for (int k = 0; k < S::kTeams; ++k)
                r.add(Joined::weight(sh_m[k][row], r.m), sh_l[k][row],
                      *reinterpret_cast<const float4*>(
                          reinterpret_cast<const float*>(smem + (k * S::kSplit + d / S::kPart) * S::kWarpBytes +
                                                         step * S::kStepBytes) +
                          Warp<S>::staged(row, d % S::kPart)));
            if (whole) write_out(row, d, r);
            else write_part(slot(blockIdx.x, t0 == 0), row, d, r);
        }
        if (!whole) {
            // ---- the item's parts, in the order of its CTAs, are joined by the last CTA to arrive.  Where there are many,
            // those of each eight neighbouring CTAs are, and what they leave by the last eight to be done: a second stage
            // costs as much as ten parts more.
            const int c0 = (int)all.owner(i0), c1 = (int)all.owner(i1 - 1), eight = blockIdx.x / 8;
            const bool only = c1 - c0 < kJoined;
            const int e0 = only ? c0 : max(c0, 8 * eight), e1 = only ? c1 : min(c1, 8 * eight + 7);
            auto part_of = [&](int cta) { return slot(cta, cta == c0); };
            // the barriers order the CTA's writes before its one thread's release, and its acquire before the CTA's reads
            auto arrive = [&](int counter, int expected) -> bool {
                __syncthreads();
                if (tid == 0) {
                    int before;
                    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                                 : "=r"(before)
                                 : "l"(a.counters + counter)
                                 : "memory");
                    if (before == expected - 1) a.counters[counter] = 0;
                    sh_last = before == expected - 1;
                }
                __syncthreads();
                return sh_last;
            };
            // the first eight of an item count at its first CTA, the others, which begin with it, at their own number
            if (arrive(e0 == c0 ? c0 : kMaxCtas + eight, e1 - e0 + 1)) {
                const int n = c1 / 8 - c0 / 8 + 1;
                for (int i = tid; i < n_rows * (S::kD / 4); i += kThreads) {
                    const int row = i / (S::kD / 4), d = i % (S::kD / 4) * 4;
                    const Joined r = join_parts<S>(e1 - e0 + 1, row, d, [&](int k) { return part_of(e0 + k); });
                    if (only) write_out(row, d, r);
                    else write_part(a.ws + (int64_t)(2 * gridDim.x + 2 * eight + (e0 == c0)) * S::kSlot, row, d, r);
                }
                if (!only && arrive(kMaxCtas + kMaxCtas / 8 + c0, n))
                    for (int i = tid; i < n_rows * (S::kD / 4); i += kThreads) {
                        const int row = i / (S::kD / 4), d = i % (S::kD / 4) * 4;
                        write_out(row, d, join_parts<S>(n, row, d, [&](int k) {
                            return a.ws + (int64_t)(2 * gridDim.x + 2 * (c0 / 8 + k) + (k == 0)) * S::kSlot;
                        }));
                    }
            }
        }
        __syncthreads();
        // the copies that waited, and on to the next item
        copy(step);
        step ^= 1;
    }
    copies_wait<0>();
}

// ---------------------------------------------------------------------------------------------------------- host
// counters of the items' first CTAs and of each eight; of an item's eights, at its first CTA
constexpr size_t kCounterBytes = LORA_DECODE_COUNTER_BYTES;
static_assert((2 * kMaxCtas + kMaxCtas / 8) * sizeof(int32_t) <= kCounterBytes, "counters");

// CTAs on an SM: as many as registers and shared memory leave room for
template <class S>
constexpr int ctas_of() {
    return std::min(S::kRows > 8 ? 2 : 3, 227 * 1024 / (S::kSmem + 2048));
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return n;
}

template <class Go>
auto by_shape(bool e4m3, int D, int rows, Go go) {
    auto with_rows = [&](auto t, auto d) {
        constexpr bool kE4m3 = decltype(t)::value;
        constexpr int kD = decltype(d)::value;
        return rows <= 8 ? go(Shapes<kE4m3, kD, 8>()) : go(Shapes<kE4m3, kD, 16>());
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

struct Launch {
    int grid;
    size_t bytes;
};
Launch launch_of(bool e4m3, int D, int group) {
    return by_shape(e4m3, D, rows_of(group), [&](auto shapes) {
        using S = decltype(shapes);
        const int grid = std::min(sm_count() * ctas_of<S>(), kMaxCtas);
        return Launch{grid, kCounterBytes + (size_t)(2 * grid + 2 * (grid / 8 + 1)) * S::kSlot * sizeof(float)};
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
        const Launch s = launch_of(cache->dtype == LORA_CACHE_E4M3, cache->head_dim, n_heads / cache->n_heads);
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
        if (B > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 2^31 - 1025 sequences");
        if (!(fabsf(scale) < INFINITY) || !(softcap >= 0.f && softcap < INFINITY))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": scale must be finite, softcap finite and >= 0");
        // what scores are multiplied by: an infinite factor would make NaN of a score of zero
        if (softcap > 0.f ? !(fabsf(scale / softcap) < INFINITY && softcap * kLog2e < INFINITY)
                          : !(fabsf(scale * kLog2e) < INFINITY))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": scale / softcap and softcap log2(e), without a softcap "
                                                                  "scale log2(e), must be finite in float32");
        if (B == 0) return LORA_OK;
        const int64_t cols = (int64_t)n_heads * cache->head_dim;
        if ((rc = check_matrix(fn, "q", q, cols, ld_q, 2)) != LORA_OK) return rc;
        if ((rc = check_matrix(fn, "out", out, cols, ld_out, 2)) != LORA_OK) return rc;
        if (B > 1 && out == q && ld_out != ld_q)
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": in place, ld_out must be ld_q");
        if (!table || !lengths) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": table or lengths is NULL");
        if (table_width < 1 || ld_table < table_width)
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": rows of table are empty or overlap");
        if (!is_aligned(table, 4) || !is_aligned(lengths, 4) || (lse && !is_aligned(lse, 4)))
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": table, lengths and lse must be 4-byte aligned");
        const bool e4m3 = cache->dtype == LORA_CACHE_E4M3;
        a.group = n_heads / cache->n_heads;
        const Launch launch = launch_of(e4m3, cache->head_dim, a.group);
        if (launch.grid == 0) return refuse(LORA_ERR_CUDA, std::string(fn) + ": no CUDA device");
        if (!workspace || !is_aligned(workspace, 256) || ws_bytes < launch.bytes)
            return refuse(LORA_ERR_WORKSPACE, std::string(fn) + ": workspace missing, too small or not 256-byte aligned");
        a.q = static_cast<const __nv_bfloat16*>(q); a.ld_q = ld_q;
        a.out = static_cast<__nv_bfloat16*>(out); a.ld_out = ld_out; a.lse = lse;
        a.table = table; a.ld_table = ld_table; a.table_width = table_width; a.lengths = lengths;
        a.B = B; a.n_heads = n_heads; a.kv_heads = cache->n_heads; a.D = cache->head_dim;
        a.rows = rows_of(a.group);
        a.parts = (a.group + a.rows - 1) / a.rows;
        a.window = window; a.scale = scale; a.softcap = softcap;
        // rows are found by 32-bit numbers of the largest unit that divides both strides
        a.unit = 16;
        while (a.unit < (1u << 30) && (a.cache.page_stride | a.cache.row_stride) % (2ll * a.unit) == 0) a.unit *= 2;
        const int64_t pu = a.cache.page_stride / a.unit, ru = a.cache.row_stride / a.unit;
        if (cache->n_pages > 0 && (pu >= (1ll << 32) || ru >= (1ll << 32) ||
                                   (double)pu * (cache->n_pages - 1) + (double)ru * (cache->page_size - 1) >= 4294967295.0))
            return refuse(LORA_ERR_LIMIT, std::string(fn) + ": the cache's rows lie more than 2^32 units apart (the largest "
                                                            "power of two that divides the strides of pages and rows)");
        a.page_units = (uint32_t)pu;
        a.row_units = (uint32_t)ru;
        a.counters = static_cast<int32_t*>(workspace);
        a.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return enqueued(fn, by_shape(e4m3, a.D, a.rows, [&](auto shapes) -> cudaError_t {
            using S = decltype(shapes);
            const auto kernel = decode_kernel<S, ctas_of<S>()>;
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
            if (e != cudaSuccess) return e;
            return launch_pdl(kernel, dim3((unsigned)launch.grid), dim3(kThreads), S::kSmem, st, a);
        }));
    });
}
