// rotary.cu -- norm and rotary positions of query and key heads, forward and backward, and rows of the paged cache
// (include/lora_attention.h).
//
// Every kernel here moves each byte once and computes little per byte: the memory rate bounds them, if the instructions
// do not.  A head's row of D elements belongs to D / 16 neighbouring lanes (of the next power of two, at least four), 16
// elements each: two pieces of 8.  Where the row is turned in halves, a lane's two pieces are the two members of its 8
// pairs, so the rotation stays in the lane; a row's sum of squares, or its largest magnitude, is at most four shuffles
// away.  A warp takes a chunk of the heads of one row after another and shares nothing with other warps: it computes the
// row's angles, and copies the next row's pieces into shared memory, asynchronously, while it works on this one's.  (CTAs
// of a few rows each, whose loads, arithmetic and stores follow one another, took 56 us at best for 8192 rows of 72 heads,
// 54 now; a copy of these rows takes 46.)
#include <algorithm>
#include <type_traits>

#include "cache.h"
#include "tc_prims.h"

namespace lora {
namespace {

// Warps of a CTA: as many as two CTAs' registers leave room for (forward, 8192 rows of 72 heads: 8 warps 55.5 us, 10 53.6;
// backward, 2048 rows of 40 heads: 18.5 and 21.8)
constexpr int kForwardWarps = 10, kBackwardWarps = 8;
constexpr int kSms = 152;     // the grids and chunks are made for
constexpr int kCtas = 2;      // CTAs on an SM: with three, or four, registers spill and 8192 rows of 72 heads take 61 and 78 us

// The heads of a row, in chunks of one kind each; a warp takes a chunk
enum Kind { kQuery, kKey, kValue };
struct Chunks {
    int32_t heads[3];        // of each kind
    int32_t per;             // heads of a chunk, the last of a kind may have fewer
    __host__ __device__ int32_t of(int kind) const { return (heads[kind] + per - 1) / per; }
    __host__ __device__ int32_t all() const { return of(kQuery) + of(kKey) + of(kValue); }
};
struct Chunk {
    int kind, first, heads;
    __device__ __forceinline__ Chunk(const Chunks& c, int i) : kind(kQuery) {
        while (kind < kValue && i >= c.of(kind)) i -= c.of(kind++);
        first = i * c.per;
        heads = min(c.per, c.heads[kind] - first);
    }
};

struct Turns {
    const int64_t* positions;
    const int64_t* turns;
    int32_t rot;             // elements of a head that are turned (0: none)
    bool interleaved;
};

// cos and sin of a phase in units of 2^-64 turns.  The quarter turn nearest to it is taken off in whole numbers: what is
// left, an angle of at most pi / 4, is 5e-8 off in float32, and the two Taylor series break off at x^9 and x^10, 2e-9 and
// 1e-10 off there.  (Carrying what float32 leaves of the angle along halves the error and costs 5 % of the time.)
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int32_t rest = (int32_t)(uint32_t)((phase - ((uint64_t)quarter << 62)) >> 32);      // in 2^-32 turns
    const float x = (float)rest * (float)(6.283185307179586 * 0x1p-32), q = x * x;
    const float s = fmaf(x * q, fmaf(q, fmaf(q, fmaf(q, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float p = fmaf(q, fmaf(q, fmaf(q, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
    const float c = fmaf(q, fmaf(q, p, -0.5f), 1.f);
    const float c1 = quarter & 1 ? -s : c, s1 = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-c1, -s1) : make_float2(c1, s1);
}
// 1 / sqrt(v), the fast one improved by a step of Newton's method: its error is that of every element of a row, and in 8 bits
// a neighbouring code here and there.  Infinity for 0, 0 for infinity.
__device__ __forceinline__ float inverse_root(float v) {
    const float f = rsqrtf(v), better = fmaf(0.5f * f, fmaf(-v * f, f, 1.f), f);
    return v > 0.f && v < INFINITY ? better : f;
}

// Two products, or two fused sums, in one instruction
__device__ __forceinline__ void mul2(float (&d)[8], const float (&a)[8], const float (&b)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 "
            "{%0, %1}, d;\n\t}"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
}
__device__ __forceinline__ void mul2(float (&d)[8], const float (&a)[8], float b) {
    const float all[8] = {b, b, b, b, b, b, b, b};
    mul2(d, a, all);
}
// d = a b + c
__device__ __forceinline__ void fma2(float (&d)[8], const float (&a)[8], const float (&b)[8], const float (&c)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 "
            "d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]), "f"(c[i]), "f"(c[i + 1]));
}
__device__ __forceinline__ float sum8(const float (&v)[8]) {
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
// a . b + c . d
__device__ __forceinline__ float dot(const float (&a)[8], const float (&b)[8], const float (&c)[8], const float (&d)[8]) {
    float v[8];
    mul2(v, a, b);
    fma2(v, c, d, v);
    return sum8(v);
}

// The angles of a warp's row: cosines [rot / 2], then sines, by all its lanes
__device__ __forceinline__ void fill_angles(const Turns& a, uint64_t position, float* to) {
    const int half = a.rot / 2;
    for (int i = threadIdx.x % 32; i < half; i += 32) {
        const float2 v = cos_sin(position * (uint64_t)a.turns[i]);
        to[i] = v.x;
        to[half + i] = v.y;
    }
}
__device__ __forceinline__ void read8(const float* from, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(from), b = *reinterpret_cast<const float4*>(from + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// A warp's place in shared memory: two rows of a chunk's pieces, [piece][lane] of 16 bytes, so that each lane reads back what
// it copied; the rows' positions and slots; a row's angles.
constexpr int kRowBytes = 4096;       // a step of float32 heads, with their gradients, at the most
// Bytes that chunks of more steps take: half a row's place.  Forward in bf16, 8192 rows of 72 heads of 128: 1024 65 us, 2048
// 54, 4096 57; 4718 rows of 72 neighbour-paired heads of 80 48, 42, 41.  Where a step takes more, 2048 is one step: float32
// forward, 2301 rows of 51 heads of 96, 24 us and 27 with two; backward in bf16 with norms, 3027 rows of 40 neighbour-paired
// heads 27.0 and 27.6.  The rule loses in that backward with more rows (8192: 48 and 44) and with heads of 256 (forward,
// 2218 rows of 40: 21.3 and 19.9).
constexpr int kChunkBytes = 2048;
struct WarpPlace {
    uint4 piece[2][kRowBytes / 16];
    int64_t position[2], slot[2];
    float angles[kMaxHeadDim];
};
__device__ __forceinline__ void copy_async16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async8(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
// 8 elements of a row, as one or two pieces from number `at` on
template <class Row8>
__device__ __forceinline__ void copy8(uint4* pieces, int at, const void* from) {
    constexpr int kPieces = sizeof(Row8) / 16;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        copy_async16(pieces + (at * kPieces + i) * 32 + threadIdx.x % 32, static_cast<const char*>(from) + 16 * i);
}
template <class Row8>
__device__ __forceinline__ void read_pieces(const uint4* pieces, int at, float (&v)[8]) {
    constexpr int kPieces = sizeof(Row8) / 16;
    uint4 q[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) q[i] = pieces[(at * kPieces + i) * 32 + threadIdx.x % 32];
    reinterpret_cast<const Row8*>(q)->get(v);
}

// What is known of a head beforehand: nothing, or that it fills its lanes (D = 16 kLanes) and is turned whole, in halves.
enum Form { kAny, kTurned };

// The two pieces of a head's row that a lane holds: from elements at0 and at1
struct LanePieces {
    template <int kLanes, int kForm>
    static __device__ __forceinline__ LanePieces of(int lane, int D, const Turns& a) {
        LanePieces p(lane, D, a);
        if (kForm == kAny) return p;
        p.in = p.turned = true;
        p.at0 = 8 * lane;
        p.at1 = 8 * (kLanes + lane);
        return p;
    }
    int at0, at1;
    bool in, turned;
    __device__ __forceinline__ LanePieces(int lane, int D, const Turns& a) {
        in = 16 * lane < D;
        turned = 16 * lane < a.rot;
        const bool halves = turned && !a.interleaved;
        at0 = halves ? 8 * lane : 16 * lane;
        at1 = halves ? a.rot / 2 + 8 * lane : 16 * lane + 8;
    }
};

// turns 8 pairs, (u[i], w[i]) or neighbours within u and within w, by its angles (back: by their negatives), and multiplies by f
__device__ __forceinline__ void turn(float (&u)[8], float (&w)[8], const float* cosines, const float* sines, float f, bool back,
                                     bool interleaved) {
    float c[8], s[8], less[8];
    read8(sines, s);
    mul2(less, s, back ? f : -f);
    mul2(s, s, back ? -f : f);
    read8(cosines, c);
    mul2(c, c, f);
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = u[2 * i], b = u[2 * i + 1], d = w[2 * i], e = w[2 * i + 1];
            u[2 * i] = fmaf(b, less[i], a * c[i]);
            u[2 * i + 1] = fmaf(a, s[i], b * c[i]);
            w[2 * i] = fmaf(e, less[4 + i], d * c[4 + i]);
            w[2 * i + 1] = fmaf(d, s[4 + i], e * c[4 + i]);
        }
    } else {
        float p[8], q[8];
        mul2(p, u, c);
        mul2(q, w, c);
        fma2(q, u, s, q);
        fma2(u, w, less, p);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = q[i];
    }
}

template <int kLanes>
__device__ __forceinline__ float sum_over_lanes(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int kLanes>
__device__ __forceinline__ uint32_t max_over_lanes(uint32_t v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// ------------------------------------------------------------------------------------------------------- forward
struct Forward {
    const void* x;           // query heads, then key heads
    int64_t ld_x;
    const void* v;
    int64_t ld_v;
    void* out;
    int64_t ld_out;
    const void *wq, *wk;
    const int64_t* slots;
    Turns turns;
    CacheView cache;
    int64_t T;
    Chunks chunks;
    bool out_keys;           // keys go to out
    int32_t D;
    float eps, inv_d;
};

template <class Row8, int kLanes, int kForm, int kCache /* -1: none */>
__global__ void __launch_bounds__(32 * kForwardWarps, kCtas) rotary_kernel(const Forward a) {
    extern __shared__ __align__(16) char smem[];
    WarpPlace& mine = reinterpret_cast<WarpPlace*>(smem)[threadIdx.x / 32];
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kAcross = 32 / kLanes;
    const int64_t t0 = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, by = (int64_t)gridDim.x * (blockDim.x / 32);
    if (t0 >= a.T) return;
    const Chunk chunk(a.chunks, blockIdx.y);
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes;
    const bool value = chunk.kind == kValue, keeps = kCache >= 0 && chunk.kind != kQuery;
    const bool to_out = chunk.kind == kQuery || (chunk.kind == kKey && a.out_keys), turned = a.turns.rot > 0 && !value;
    const int D = kForm != kAny ? 16 * kLanes : a.D, steps = (chunk.heads + kAcross - 1) / kAcross;
    const LanePieces p = LanePieces::of<kLanes, kForm>(lane, D, a.turns);
    const int heads = p.in ? chunk.heads - sub : 0;      // this lane's are 0, kAcross, 2 kAcross, .. below that
    const int64_t head_at = (int64_t)(chunk.first + (chunk.kind == kKey ? a.chunks.heads[kQuery] : 0) + sub) * D;
    const void* weight = value ? nullptr : chunk.kind == kKey ? a.wk : a.wq;
    float g0[8] = {}, g1[8] = {};
    if (weight && p.in) {
        Row8 w[2];
        w[0].load(weight, p.at0);
        w[1].load(weight, p.at1);
        w[0].get(g0);
        w[1].get(g1);
    }
    // a lane's pieces that are not there are read as what the place held before: numbers that go nowhere
    auto copy = [&](int64_t t, int to) {
        if (t < a.T) {
            const char* from = static_cast<const char*>(Row8::at(value ? a.v : a.x, t * (value ? a.ld_v : a.ld_x) + head_at));
            for (int k = 0; k < steps; ++k) {
                if (k * kAcross >= heads) break;
                copy8<Row8>(mine.piece[to], 2 * k, Row8::at(static_cast<const void*>(from), k * kAcross * D + p.at0));
                copy8<Row8>(mine.piece[to], 2 * k + 1, Row8::at(static_cast<const void*>(from), k * kAcross * D + p.at1));
            }
            if (threadIdx.x % 32 == 0) {
                if (turned) copy_async8(&mine.position[to], a.turns.positions + t);
                if (keeps) copy_async8(&mine.slot[to], a.slots + t);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy(t0, 0);
    int now = 0;
    for (int64_t t = t0; t < a.T; t += by, now ^= 1) {
        copy(t + by, now ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        if (turned) {
            fill_angles(a.turns, (uint64_t)mine.position[now], mine.angles);
            __syncwarp();
        }
        void* const out = Row8::at(a.out, t * a.ld_out + head_at);
        const int64_t slot = keeps ? mine.slot[now] : -1;
        const bool cached = slot >= 0 && slot < a.cache.slots;
        const RowPlace place = cached ? RowPlace(a.cache, slot) : RowPlace();
#pragma unroll 2
        for (int k = 0; k < steps; ++k) {
            float y[8], z[8], f = 1.f;
            read_pieces<Row8>(mine.piece[now], 2 * k, y);
            read_pieces<Row8>(mine.piece[now], 2 * k + 1, z);
            const bool in = k * kAcross < heads;
            if (weight) {
                const float ss = p.in ? dot(y, y, z, z) : 0.f;
                f = inverse_root(sum_over_lanes<kLanes>(ss) * a.inv_d + a.eps);
                if (f == 0.f) {          // infinitely long: zeros before the weight, whose product may be infinite
                    mul2(y, y, f);
                    mul2(z, z, f);
                }
                mul2(y, y, g0);
                mul2(z, z, g1);
            }
            if (turned && p.turned) {
                const float* sines = mine.angles + (kForm == kTurned ? 8 * kLanes : a.turns.rot / 2);
                turn(y, z, mine.angles + 8 * lane, sines + 8 * lane, f, false, kForm == kAny && a.turns.interleaved);
            } else if (weight) {
                mul2(y, y, f);
                mul2(z, z, f);
            }
            if (in && to_out) {
                Row8::store(out, k * kAcross * D + p.at0, y);
                Row8::store(out, k * kAcross * D + p.at1, z);
            }
            if constexpr (kCache >= 0) {
                if (keeps) {
                    uint32_t amax = 0;
                    if (kCache == LORA_CACHE_E4M3)
                        amax = max_over_lanes<kLanes>(p.in ? max(abs_bits_max(y), abs_bits_max(z)) : 0);
                    if (in && cached) {
                        const int head = chunk.first + k * kAcross + sub;
                        char* to = (value ? a.cache.v : a.cache.k) + place.row + head * a.cache.head_stride;
                        if (kCache == LORA_CACHE_BF16) {
                            Row8Bf16::store(to, p.at0, y);
                            Row8Bf16::store(to, p.at1, z);
                        } else {
                            float inv;
                            const float sc = block_scale(amax, &inv);
                            *reinterpret_cast<uint2*>(to + p.at0) = encode8(y, inv);
                            *reinterpret_cast<uint2*>(to + p.at1) = encode8(z, inv);
                            if (lane == 0) (value ? a.cache.vs : a.cache.ks)[place.scale + head * a.cache.s_head] = sc;
                        }
                    }
                }
            }
        }
        __syncwarp();        // what this row's copies and angles were in is written anew
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------------------------------------------ backward
struct Backward {
    const void* x;
    int64_t ld_x;
    const void* dout;
    int64_t ld_dout;
    void* dx;
    int64_t ld_dx;
    const void *wq, *wk;
    float* parts;            // [chunks, CTAs across the rows, D]: each CTA's sums of the weights' gradients
    Turns turns;
    int64_t T;
    Chunks chunks;
    int32_t D;
    float eps, inv_d;
};

template <class Row8, int kLanes, int kForm, bool kNorm, bool kWeights>
__global__ void __launch_bounds__(32 * kBackwardWarps, kCtas) rotary_backward_kernel(const Backward a) {
    extern __shared__ __align__(16) char smem[];
    WarpPlace* const places = reinterpret_cast<WarpPlace*>(smem);
    WarpPlace& mine = places[threadIdx.x / 32];
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kAcross = 32 / kLanes;
    const int warps = (int)blockDim.x / 32, warp = threadIdx.x / 32;
    const Chunk chunk(a.chunks, blockIdx.y);
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 32 / kLanes;
    const int D = kForm != kAny ? 16 * kLanes : a.D, steps = (chunk.heads + kAcross - 1) / kAcross;
    const LanePieces p = LanePieces::of<kLanes, kForm>(lane, D, a.turns);
    const int heads = p.in ? chunk.heads - sub : 0;
    const int64_t head_at = (int64_t)(chunk.first + (chunk.kind == kKey ? a.chunks.heads[kQuery] : 0) + sub) * D;
    const void* weight = chunk.kind == kKey ? a.wk : a.wq;
    float g0[8] = {}, g1[8] = {};
    if (kNorm && weight && p.in) {
        Row8 w[2];
        w[0].load(weight, p.at0);
        w[1].load(weight, p.at1);
        w[0].get(g0);
        w[1].get(g1);
    }
    float sum[2][8] = {};
    const int64_t t0 = (int64_t)blockIdx.x * warps + warp, by = (int64_t)gridDim.x * warps;
    // pieces of dout, and with a norm of x, in turn
    constexpr int kEach = kNorm ? 4 : 2;
    auto copy = [&](int64_t t, int to) {
        if (t < a.T) {
            for (int k = 0; k < steps; ++k) {
                if (k * kAcross >= heads) break;
                const int64_t at = head_at + k * kAcross * D;
                copy8<Row8>(mine.piece[to], kEach * k, Row8::at(a.dout, t * a.ld_dout + at + p.at0));
                copy8<Row8>(mine.piece[to], kEach * k + 1, Row8::at(a.dout, t * a.ld_dout + at + p.at1));
                if (kNorm && weight) {
                    copy8<Row8>(mine.piece[to], kEach * k + 2, Row8::at(a.x, t * a.ld_x + at + p.at0));
                    copy8<Row8>(mine.piece[to], kEach * k + 3, Row8::at(a.x, t * a.ld_x + at + p.at1));
                }
            }
            if (threadIdx.x % 32 == 0 && a.turns.rot) copy_async8(&mine.position[to], a.turns.positions + t);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy(t0, 0);
    int now = 0;
    for (int64_t t = t0; t < a.T; t += by, now ^= 1) {
        copy(t + by, now ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncwarp();
        if (a.turns.rot) {
            fill_angles(a.turns, (uint64_t)mine.position[now], mine.angles);
            __syncwarp();
        }
        for (int k = 0; k < steps; ++k) {
            float y[8], z[8];
            read_pieces<Row8>(mine.piece[now], kEach * k, y);
            read_pieces<Row8>(mine.piece[now], kEach * k + 1, z);
            const bool in = k * kAcross < heads;
            if (p.turned) {
                const float* sines = mine.angles + (kForm == kTurned ? 8 * kLanes : a.turns.rot / 2);
                turn(y, z, mine.angles + 8 * lane, sines + 8 * lane, 1.f, true, kForm == kAny && a.turns.interleaved);
            }
            if (kNorm && weight) {
                float v[8], x[8];
                read_pieces<Row8>(mine.piece[now], kEach * k + 2, v);
                read_pieces<Row8>(mine.piece[now], kEach * k + 3, x);
                const float ss = p.in ? dot(v, v, x, x) : 0.f;
                const float f = inverse_root(sum_over_lanes<kLanes>(ss) * a.inv_d + a.eps);
                mul2(v, v, f);
                mul2(x, x, f);
                if (kWeights && in) {
                    fma2(sum[0], y, v, sum[0]);
                    fma2(sum[1], z, x, sum[1]);
                }
                mul2(y, y, g0);
                mul2(z, z, g1);
                const float yx = p.in ? dot(y, v, z, x) : 0.f;
                const float along = -a.inv_d * sum_over_lanes<kLanes>(yx);
                const float all[8] = {along, along, along, along, along, along, along, along};
                fma2(y, v, all, y);
                fma2(z, x, all, z);
                mul2(y, y, f);
                mul2(z, z, f);
            }
            if (in) {
                void* const to = Row8::at(a.dx, t * a.ld_dx + head_at);
                Row8::store(to, k * kAcross * D + p.at0, y);
                Row8::store(to, k * kAcross * D + p.at1, z);
            }
        }
        __syncwarp();        // what this row's copies and angles were in is written anew
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if constexpr (kWeights) {
        // each lane's 16 sums, then those of all lanes and warps that hold the same elements
        float* const to = reinterpret_cast<float*>(&mine);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) to[threadIdx.x % 32 * 16 + i] = sum[i / 8][i % 8];
        __syncthreads();
        for (int i = threadIdx.x; i < kLanes * 16; i += (int)blockDim.x) {
            const LanePieces q = LanePieces::of<kLanes, kForm>(i / 16, D, a.turns);
            if (!q.in) continue;
            float v = 0.f;
            for (int k = 0; k < warps; ++k)
#pragma unroll
                for (int j = 0; j < kAcross; ++j) v += reinterpret_cast<const float*>(places + k)[j * kLanes * 16 + i];
            const int d = i % 16 < 8 ? q.at0 + i % 16 : q.at1 + i % 16 - 8;
            a.parts[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * D + d] = v;
        }
    }
}

// Sums of the CTAs' parts, nq of the query weight's, then nk of the key weight's, [D] each, in a fixed order; 32 columns of
// [2 D] a CTA
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* parts, int nq, int nk, int D, float* dq, float* dk) {
    __shared__ float s[32][33];
    grid_dep_launch();
    grid_dep_wait();
    const int col = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
    float v = 0.f;
    if (col < 2 * D) {
        const bool key = col >= D;
        const float* from = key ? parts + (int64_t)nq * D + col - D : parts + col;
        const int n = key ? nk : nq;
#pragma unroll 4
        for (int i = y; i < n; i += 32) v += from[(int64_t)i * D];
    }
    s[y][threadIdx.x % 32] = v;
    __syncthreads();
    if (y > 0 || col >= 2 * D) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
    float* to = col < D ? dq : dk;
    if (to) to[col % D] = v;
}

// ------------------------------------------------------------------------------------------------------ cache rows
constexpr int kCacheWarps = 4;        // of a CTA (8: 37 us to read 32768 rows of 8 heads in 8 bits, 4: 34)
struct Rows {
    CacheView cache;
    const int64_t* slots;
    void *k, *v;
    int64_t ld_k, ld_v;
    int64_t T;
    int32_t across, down;
    int32_t n_heads, D;
};

// How a CTA's warps lie over heads (key heads, then value heads) and rows: `across` warps take neighbouring heads, `down` of
// such rows of warps take neighbouring rows.  A lane takes 8 elements of each half of a head of kRows rows, `down`
// apart.
template <class Row8, int kLanes, int kRows, int kCache>
__global__ void __launch_bounds__(32 * kCacheWarps) cache_read_kernel(const Rows a) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr bool kE4m3 = kCache == LORA_CACHE_E4M3;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % kLanes;
    const int both = ((int)blockIdx.y * a.across + warp % a.across) * (32 / kLanes) + threadIdx.x % 32 / kLanes;
    const int64_t t0 = (int64_t)blockIdx.x * (a.down * kRows) + warp / a.across;
    const bool value = both >= a.n_heads;
    const int head = value ? both - a.n_heads : both;
    if (head >= a.n_heads || 16 * lane >= a.D) return;
    const char* from = (value ? a.cache.v : a.cache.k) + head * a.cache.head_stride + (kE4m3 ? 8 : 16) * lane;
    const float* scales = kE4m3 ? (value ? a.cache.vs : a.cache.ks) + head * a.cache.s_head : nullptr;
    uint4 q[kRows][kE4m3 ? 1 : 2];
    float sc[kRows];
    int64_t slot[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t t = t0 + k * a.down;
        slot[k] = t < a.T ? a.slots[t] : -1;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        sc[k] = 0.f;
        for (auto& w : q[k]) w = make_uint4(0, 0, 0, 0);
        if (slot[k] < 0 || slot[k] >= a.cache.slots) continue;
        const RowPlace place(a.cache, slot[k]);
        if (kE4m3) sc[k] = scales[place.scale];
        if (kE4m3) {
            const uint2 lo = *reinterpret_cast<const uint2*>(from + place.row);
            const uint2 hi = *reinterpret_cast<const uint2*>(from + place.row + a.D / 2);
            q[k][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
            q[k][0] = *reinterpret_cast<const uint4*>(from + place.row);
            q[k][kE4m3 ? 0 : 1] = *reinterpret_cast<const uint4*>(from + place.row + a.D);
        }
    }
    void* to = value ? a.v : a.k;
    const int64_t ld = value ? a.ld_v : a.ld_k, col = (int64_t)head * a.D + 8 * lane;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t t = t0 + k * a.down;
        if (t >= a.T) continue;
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (kE4m3) {
                decode8(i ? make_uint2(q[k][0].z, q[k][0].w) : make_uint2(q[k][0].x, q[k][0].y), sc[k], x);
            } else {
                Row8Bf16 b;
                b.q = q[k][kE4m3 ? 0 : i];
                b.get(x);
            }
            Row8::store(to, t * ld + col + (i ? a.D / 2 : 0), x);
        }
    }
}

// The same the other way: rows are rounded, or quantized by the head's lanes together, and written to their slots.
template <class Row8, int kLanes, int kRows, int kCache>
__global__ void __launch_bounds__(32 * kCacheWarps) cache_write_kernel(const Rows a) {
    grid_dep_launch();
    grid_dep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % kLanes;
    const int both = ((int)blockIdx.y * a.across + warp % a.across) * (32 / kLanes) + threadIdx.x % 32 / kLanes;
    const int64_t t0 = (int64_t)blockIdx.x * (a.down * kRows) + warp / a.across;
    const bool value = both >= a.n_heads;
    const int head = value ? both - a.n_heads : both;
    const bool in = head < a.n_heads && 16 * lane < a.D;
    const void* from = value ? a.v : a.k;
    const int64_t ld = value ? a.ld_v : a.ld_k, col = (int64_t)head * a.D + 8 * lane;
    Row8 r[kRows][2];
    int64_t slot[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t t = t0 + k * a.down;
        r[k][0].zero();
        r[k][1].zero();
        slot[k] = -1;
        if (in && t < a.T) {
            r[k][0].load(from, t * ld + col);
            r[k][1].load(from, t * ld + col + a.D / 2);
            slot[k] = a.slots[t];
        }
    }
    constexpr int kElement = kCache == LORA_CACHE_E4M3 ? 1 : 2;
    char* const to = (value ? a.cache.v : a.cache.k) + head * a.cache.head_stride + 8 * lane * kElement;
    float* const scales = kCache == LORA_CACHE_E4M3 ? (value ? a.cache.vs : a.cache.ks) + head * a.cache.s_head : nullptr;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        uint32_t amax = 0;
        if (kCache == LORA_CACHE_E4M3) amax = max_over_lanes<kLanes>(max(r[k][0].abs_max(), r[k][1].abs_max()));
        if (slot[k] < 0 || slot[k] >= a.cache.slots) continue;
        const RowPlace place(a.cache, slot[k]);
        float y[8], z[8];
        r[k][0].get(y);
        r[k][1].get(z);
        if (kCache == LORA_CACHE_BF16) {
            Row8Bf16::store(to + place.row, 0, y);
            Row8Bf16::store(to + place.row, a.D / 2, z);
        } else {
            float inv;
            const float sc = block_scale(amax, &inv);
            *reinterpret_cast<uint2*>(to + place.row) = encode8(y, inv);
            *reinterpret_cast<uint2*>(to + place.row + a.D / 2) = encode8(z, inv);
            if (lane == 0) scales[place.scale] = sc;
        }
    }
}

// ---------------------------------------------------------------------------------------------------------- host
int lanes_of(int D) { return D <= 64 ? 4 : D <= 128 ? 8 : 16; }

template <class Go>
cudaError_t by_lanes(int D, Go go) {
    switch (lanes_of(D)) {
        case 4: return go(std::integral_constant<int, 4>());
        case 8: return go(std::integral_constant<int, 8>());
        default: return go(std::integral_constant<int, 16>());
    }
}
template <class Go>
cudaError_t by_type(lora_dtype_t dt, Go go) {
    return dt == LORA_BF16 ? go(Row8Bf16()) : go(Row8F32());
}

constexpr unsigned kMaxParts = kCtas * kSms + kMaxHeads;   // CTAs of a backward that sums the weights' gradients

// Chunks of one step of heads where all warps then fit the SMs at once.  Else as many steps, of those that fit a row's place,
// as waste the least: an empty head costs as much as a full one, and a chunk's angles as much as 0.6 steps.
Chunks chunks_of(int hq, int hk, int hv, int D, int64_t T, int bytes_per_head, int warps) {
    const int across = 32 / lanes_of(D);
    Chunks c{{hq, hk, hv}, across};
    if (T * c.all() <= (int64_t)kSms * kCtas * warps) return c;
    Chunks best = c;
    double least = c.all() * 1.6;
    for (int steps = 2; steps * across * bytes_per_head <= kChunkBytes; ++steps) {
        c.per = steps * across;
        const double cost = c.all() * (steps + 0.6);
        if (cost < least) {
            least = cost;
            best = c;
        }
    }
    return best;
}
// A launch's grid: across the rows as many CTAs as the SMs hold at once, or as there are rows for
struct Launch {
    dim3 grid;
    unsigned threads;
    size_t smem;
};
Launch launch_of(const Chunks& c, int64_t T, int warps) {
    const unsigned w = (unsigned)std::min<int64_t>(warps, T), y = (unsigned)c.all();
    const unsigned n = (unsigned)std::min<int64_t>((T + w - 1) / w, std::max(1u, unsigned(kSms * kCtas) / y));
    return Launch{dim3(n, y), 32 * w, w * sizeof(WarpPlace)};
}
// The limit of shared memory is the kernel's, not the call's: every thread that launches it sets the same, that of kWarps
// warps, so that none takes it from a call that another thread is about to launch.
template <int kWarps, class K, class A>
cudaError_t launch_rows(K kernel, const Launch& l, cudaStream_t st, const A& a) {
    if (l.smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)(kWarps * sizeof(WarpPlace)));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, l.grid, dim3(l.threads), l.smem, st, a);
}
bool turned_whole(int D, int lanes, const Turns& t) { return D == 16 * lanes && t.rot == D && !t.interleaved; }
// what a head's lanes take of a row's place, in bytes: 16 elements each; a step of 32 lanes is 4 KB with x in float32 beside
// the gradient
static_assert(2 * 32 * 16 * sizeof(float) <= kRowBytes, "a step fits a row's place");
int bytes_of(lora_dtype_t dt, int D) { return 16 * lanes_of(D) * elem_size(dt); }

// kernel(type, lanes, rows a lane, cache's type) over the rows of a cache
template <class Kernel>
cudaError_t launch_cache_rows(lora_dtype_t dt, int cache, Rows a, Kernel kernel, cudaStream_t st) {
    return by_type(dt, [&](auto row) {
        return by_lanes(a.D, [&](auto lanes) {
            // the heads in equal shares across, and as many rows of warps as are left room for
            const int per_warp = 32 / decltype(lanes)::value, all = (2 * a.n_heads + per_warp - 1) / per_warp;
            const int y = (all + kCacheWarps - 1) / kCacheWarps;
            a.across = (all + y - 1) / y;
            a.down = (int)std::min<int64_t>(kCacheWarps / a.across, a.T);
            auto go = [&](auto rows, auto c) {
                const int64_t per = (int64_t)a.down * decltype(rows)::value;
                return launch_pdl(kernel(row, lanes, rows, c), dim3((unsigned)((a.T + per - 1) / per), (unsigned)y),
                                  dim3((unsigned)(32 * a.across * a.down)), 0, st, a);
            };
            // a row a lane where all of them fit the SMs at once, else four
            auto sized = [&](auto c) {
                return a.T * y * a.across <= kSms * 32 ? go(std::integral_constant<int, 1>(), c)
                                                        : go(std::integral_constant<int, 4>(), c);
            };
            return cache == LORA_CACHE_BF16 ? sized(std::integral_constant<int, LORA_CACHE_BF16>())
                                            : sized(std::integral_constant<int, LORA_CACHE_E4M3>());
        });
    });
}

int check_rotary(const char* fn, int32_t T, lora_dtype_t dt, const lora_rotary_t* r) {
    const std::string f(fn);
    if (!r) return refuse(LORA_ERR_INVALID_ARG, f + ": rotary is NULL");
    if (dt != LORA_BF16 && dt != LORA_F32) return refuse(LORA_ERR_DTYPE, "unknown dtype");
    if (T < 0 || r->n_heads < 1 || r->n_kv_heads < 1)
        return refuse(LORA_ERR_INVALID_ARG, f + ": T must be >= 0, with at least one query and one key head");
    if (T > kMaxRowsOfX || r->n_heads > kMaxHeads || r->n_kv_heads > kMaxHeads || r->n_heads + 2 * r->n_kv_heads > kMaxHeads)
        return refuse(LORA_ERR_LIMIT, f + ": more than 2^31 - 1025 rows or 1024 heads");
    if (r->head_dim < 16 || r->head_dim > kMaxHeadDim || r->head_dim % 16 != 0)
        return refuse(LORA_ERR_LIMIT, f + ": a head's size must be a multiple of 16, at most 256");
    if (r->rot_dim < 0 || r->rot_dim > r->head_dim || r->rot_dim % 16 != 0)
        return refuse(LORA_ERR_LIMIT, f + ": the turned part of a head must be a multiple of 16, at most the head");
    if (r->rot_dim > 0 && !r->turns) return refuse(LORA_ERR_INVALID_ARG, f + ": turns is NULL");
    if (r->rot_dim > 0 && !is_aligned(r->turns, 8)) return refuse(LORA_ERR_ALIGNMENT, f + ": turns must be 8-byte aligned");
    if ((r->q_weight && !is_aligned(r->q_weight, 16)) || (r->k_weight && !is_aligned(r->k_weight, 16)))
        return refuse(LORA_ERR_ALIGNMENT, f + ": the weights must be 16-byte aligned");
    if ((r->q_weight || r->k_weight) && !(r->eps >= 0.f && r->eps < INFINITY))
        return refuse(LORA_ERR_INVALID_ARG, f + ": eps must be finite and not negative");
    return LORA_OK;
}
int check_slots(const char* fn, const int64_t* slots) {
    if (!slots) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": slots is NULL");
    if (!is_aligned(slots, 8)) return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": slots must be 8-byte aligned");
    return LORA_OK;
}

template <class Row8, int kCache>
cudaError_t launch_forward(const Forward& a, cudaStream_t st) {
    return by_lanes(a.D, [&](auto lanes) {
        constexpr int kLanes = decltype(lanes)::value;
        const Launch l = launch_of(a.chunks, a.T, kForwardWarps);
        if (turned_whole(a.D, kLanes, a.turns))
            return launch_rows<kForwardWarps>(rotary_kernel<Row8, kLanes, kTurned, kCache>, l, st, a);
        return launch_rows<kForwardWarps>(rotary_kernel<Row8, kLanes, kAny, kCache>, l, st, a);
    });
}
cudaError_t forward(lora_dtype_t dt, int cache, Forward a, cudaStream_t st) {
    const int32_t* h = a.chunks.heads;
    a.chunks = chunks_of(h[kQuery], h[kKey], h[kValue], a.D, a.T, bytes_of(dt, a.D), kForwardWarps);
    return by_type(dt, [&](auto row) {
        using Row8 = decltype(row);
        return cache < 0 ? launch_forward<Row8, -1>(a, st)
                         : cache == LORA_CACHE_BF16 ? launch_forward<Row8, LORA_CACHE_BF16>(a, st)
                                                    : launch_forward<Row8, LORA_CACHE_E4M3>(a, st);
    });
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_rotary_forward(int32_t T, lora_dtype_t dt, const lora_rotary_t* r, const void* x, int64_t ld_x,
                                   const int64_t* positions, void* out, int64_t ld_out, const void* v, int64_t ld_v,
                                   const lora_cache_t* cache, const int64_t* slots, int32_t keep_keys, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_rotary_forward";
        int rc = check_rotary(fn, T, dt, r);
        if (rc != LORA_OK) return rc;
        Forward a = {};
        if (cache) {
            rc = check_cache(fn, cache, &a.cache);
            if (rc != LORA_OK) return rc;
            if (cache->n_heads != r->n_kv_heads || cache->head_dim != r->head_dim)
                return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": the cache's heads are not the keys'");
        }
        if (T == 0) return LORA_OK;
        const int64_t D = r->head_dim, all = (int64_t)(r->n_heads + r->n_kv_heads) * D;
        a.out_keys = !cache || keep_keys;
        const int es = elem_size(dt);
        if ((rc = check_matrix(fn, "x", x, all, ld_x, es)) != LORA_OK) return rc;
        if ((rc = check_matrix(fn, "out", out, a.out_keys ? all : r->n_heads * D, ld_out, es)) != LORA_OK) return rc;
        if (T > 1 && out == x && ld_out != ld_x)
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": in place, ld_out must be ld_x");
        if (cache) {
            if ((rc = check_matrix(fn, "v", v, r->n_kv_heads * D, ld_v, es)) != LORA_OK) return rc;
            if ((rc = check_slots(fn, slots)) != LORA_OK) return rc;
        }
        if (r->rot_dim > 0 && !positions) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": positions is NULL");
        if (r->rot_dim > 0 && !is_aligned(positions, 8))
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": positions must be 8-byte aligned");
        a.x = x; a.ld_x = ld_x; a.v = v; a.ld_v = ld_v; a.out = out; a.ld_out = ld_out;
        a.wq = r->q_weight; a.wk = r->k_weight; a.slots = slots;
        a.turns = Turns{positions, r->turns, r->rot_dim, r->interleaved != 0};
        a.T = T;
        a.chunks = Chunks{{r->n_heads, r->n_kv_heads, cache ? r->n_kv_heads : 0}, 0};
        a.D = (int32_t)D; a.eps = r->eps; a.inv_d = 1.f / (float)D;
        return enqueued(fn, forward(dt, cache ? cache->dtype : -1, a, static_cast<cudaStream_t>(stream)));
    });
}

extern "C" size_t lora_rotary_workspace_size(int32_t T, const lora_rotary_t* r) {
    const int64_t n = guarded([&]() -> int64_t {
        if (check_rotary("lora_rotary_workspace_size", T, LORA_BF16, r) != LORA_OK) return 0;
        return (int64_t)kMaxParts * r->head_dim * sizeof(float);
    });
    return n > 0 ? (size_t)n : 0;
}

extern "C" int lora_rotary_backward(int32_t T, lora_dtype_t dt, const lora_rotary_t* r, const void* x, int64_t ld_x,
                                    const int64_t* positions, const void* dout, int64_t ld_dout, void* dx,
                                    int64_t ld_dx, float* dq_weight, float* dk_weight, void* workspace,
                                    size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_rotary_backward";
        int rc = check_rotary(fn, T, dt, r);
        if (rc != LORA_OK) return rc;
        const int64_t D = r->head_dim, all = (int64_t)(r->n_heads + r->n_kv_heads) * D;
        const bool norm = r->q_weight || r->k_weight, weights = dq_weight || dk_weight;
        if ((dq_weight && !r->q_weight) || (dk_weight && !r->k_weight))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": the gradient of a weight that is not given");
        if ((dq_weight && !is_aligned(dq_weight, 4)) || (dk_weight && !is_aligned(dk_weight, 4)))
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": the weights' gradients must be 4-byte aligned");
        if (weights && (!workspace || !is_aligned(workspace, 16) ||
                        ws_bytes < (size_t)kMaxParts * D * sizeof(float)))
            return refuse(LORA_ERR_WORKSPACE, std::string(fn) + ": workspace missing, too small or not 16-byte aligned");
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const int es = elem_size(dt);
        if (T > 0) {
            if ((rc = check_matrix(fn, "dout", dout, all, ld_dout, es)) != LORA_OK) return rc;
            if ((rc = check_matrix(fn, "dx", dx, all, ld_dx, es)) != LORA_OK) return rc;
            if (norm && (rc = check_matrix(fn, "x", x, all, ld_x, es)) != LORA_OK) return rc;
            if (T > 1 && dx == dout && ld_dx != ld_dout)
                return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": in place, ld_dx must be ld_dout");
            if (r->rot_dim > 0 && !positions)
                return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": positions is NULL");
            if (r->rot_dim > 0 && !is_aligned(positions, 8))
                return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": positions must be 8-byte aligned");
        } else if (!weights) {
            return LORA_OK;
        }
        Backward a = {};
        a.x = x; a.ld_x = ld_x; a.dout = dout; a.ld_dout = ld_dout; a.dx = dx; a.ld_dx = ld_dx;
        a.wq = r->q_weight; a.wk = r->k_weight; a.parts = static_cast<float*>(workspace);
        a.turns = Turns{positions, r->turns, r->rot_dim, r->interleaved != 0};
        a.T = T;
        a.D = (int32_t)D; a.eps = r->eps; a.inv_d = 1.f / (float)D;
        int nq = 0, nk = 0;
        cudaError_t e = cudaSuccess;
        if (T > 0)
            e = by_type(dt, [&](auto row) {
                using Row8 = decltype(row);
                return by_lanes(a.D, [&](auto lanes) {
                    constexpr int kLanes = decltype(lanes)::value;
                    a.chunks = chunks_of(r->n_heads, r->n_kv_heads, 0, a.D, T, (norm ? 2 : 1) * bytes_of(dt, a.D),
                                         kBackwardWarps);
                    const Launch l = launch_of(a.chunks, T, kBackwardWarps);
                    nq = (int)l.grid.x * a.chunks.of(kQuery);
                    nk = (int)l.grid.x * a.chunks.of(kKey);
                    auto go = [&](auto nrm, auto wts) {
                        constexpr bool kNorm = decltype(nrm)::value, kWeights = decltype(wts)::value;
                        const auto kernel = turned_whole(a.D, kLanes, a.turns)
                                                ? rotary_backward_kernel<Row8, kLanes, kTurned, kNorm, kWeights>
                                                : rotary_backward_kernel<Row8, kLanes, kAny, kNorm, kWeights>;
                        return launch_rows<kBackwardWarps>(kernel, l, st, a);
                    };
                    return !norm ? go(std::false_type(), std::false_type())
                                 : !weights ? go(std::true_type(), std::false_type()) : go(std::true_type(), std::true_type());
                });
            });
        if (e == cudaSuccess && weights)
            e = launch_pdl(weight_grad_kernel, dim3((unsigned)((2 * D + 31) / 32)), dim3(1024), 0, st,
                           static_cast<const float*>(workspace), nq, nk, (int)D, dq_weight, dk_weight);
        return enqueued(fn, e);
    });
}

extern "C" int lora_cache_write(int32_t T, lora_dtype_t dt, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                const lora_cache_t* cache, const int64_t* slots, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_cache_write";
        Rows a = {};
        if (dt != LORA_BF16 && dt != LORA_F32) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        int rc = check_cache(fn, cache, &a.cache);
        if (rc != LORA_OK) return rc;
        if (T < 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0");
        if (T > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 2^31 - 1025 rows");
        if (T == 0) return LORA_OK;
        const int64_t cols = (int64_t)cache->n_heads * cache->head_dim;
        if ((rc = check_matrix(fn, "k", k, cols, ld_k, elem_size(dt))) != LORA_OK) return rc;
        if ((rc = check_matrix(fn, "v", v, cols, ld_v, elem_size(dt))) != LORA_OK) return rc;
        if ((rc = check_slots(fn, slots)) != LORA_OK) return rc;
        a.slots = slots; a.k = const_cast<void*>(k); a.v = const_cast<void*>(v); a.ld_k = ld_k; a.ld_v = ld_v;
        a.T = T; a.n_heads = cache->n_heads; a.D = cache->head_dim;
        return enqueued(fn, launch_cache_rows(dt, cache->dtype, a, [](auto row, auto lanes, auto rows, auto c) {
            return cache_write_kernel<decltype(row), decltype(lanes)::value, decltype(rows)::value, decltype(c)::value>;
        }, static_cast<cudaStream_t>(stream)));
    });
}

extern "C" int lora_cache_read(int32_t T, lora_dtype_t dt, const lora_cache_t* cache, const int64_t* slots, void* k,
                               int64_t ld_k, void* v, int64_t ld_v, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_cache_read";
        Rows a = {};
        if (dt != LORA_BF16 && dt != LORA_F32) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        int rc = check_cache(fn, cache, &a.cache);
        if (rc != LORA_OK) return rc;
        if (T < 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0");
        if (T > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 2^31 - 1025 rows");
        if (T == 0) return LORA_OK;
        const int64_t cols = (int64_t)cache->n_heads * cache->head_dim;
        if ((rc = check_matrix(fn, "k", k, cols, ld_k, elem_size(dt))) != LORA_OK) return rc;
        if ((rc = check_matrix(fn, "v", v, cols, ld_v, elem_size(dt))) != LORA_OK) return rc;
        if ((rc = check_slots(fn, slots)) != LORA_OK) return rc;
        a.slots = slots; a.k = k; a.v = v; a.ld_k = ld_k; a.ld_v = ld_v;
        a.T = T; a.n_heads = cache->n_heads; a.D = cache->head_dim;
        return enqueued(fn, launch_cache_rows(dt, cache->dtype, a, [](auto row, auto lanes, auto rows, auto c) {
            return cache_read_kernel<decltype(row), decltype(lanes)::value, decltype(rows)::value, decltype(c)::value>;
        }, static_cast<cudaStream_t>(stream)));
    });
}
