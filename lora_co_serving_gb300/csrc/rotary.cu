// rotary.cu -- norm and rotary positions of query and key heads, forward and backward, and rows of the paged cache
// (include/lora_attention.h).
//
// Every kernel here moves each byte once and computes little per byte: the memory rate bounds them, if the instructions
// do not.  A head's row of D elements belongs to D / 16 neighbouring lanes (of the next power of two, at least four), 16
// elements each: two pieces of 8.  Where the row is turned in halves, a lane's two pieces are the two members of its 8
// pairs, so the rotation stays in the lane; a row's sum of squares, or its largest magnitude, is at most four shuffles
// away.  A lane keeps its head and takes several rows of it, so that what depends on the head (its weights, where it lies)
// is found once: numbering (row, head) units instead took twice the instructions and 61 us for 8192 rows of 72 heads, @ now.
// The angles of a CTA's rows are computed once, by all its threads, into shared memory, while the rows are on their way.
#include <algorithm>
#include <type_traits>

#include "cache.h"
#include "tc_prims.h"

namespace lora {
namespace {

constexpr int kMaxThreads = 256;

// How a CTA's warps lie over heads and rows: `across` warps take neighbouring heads, `down` of such rows of warps take
// neighbouring rows of the matrix.  A lane takes kRows rows, `down` apart.
struct Shape {
    int32_t across, down;
};
template <int kLanes, int kRows>
struct Spot {
    int lane, head, row;         // lane within the head; head; first of the lane's rows in the CTA
    int64_t t0;                  // the CTA's first row
    __device__ __forceinline__ Spot(const Shape& s, int64_t block) {
        const int warp = threadIdx.x / 32;
        lane = threadIdx.x % kLanes;
        head = ((int)blockIdx.y * s.across + warp % s.across) * (32 / kLanes) + threadIdx.x % 32 / kLanes;
        row = warp / s.across;
        t0 = block * (int64_t)(s.down * kRows);
    }
};

struct Turns {
    const int64_t* positions;
    const int64_t* turns;
    int32_t rot;             // elements of a head that are turned (0: none)
    bool interleaved;
};

// cos and sin of a phase in units of 2^-64 turns.  The quarter turn nearest to it is taken off in whole numbers: what is
// left is at most an eighth, so that its float32 value is 5e-8 off in angle at the most, and its sine and cosine a few
// units of 2^-24.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int32_t rest = (int32_t)(uint32_t)((phase - ((uint64_t)quarter << 62)) >> 32);      // in 2^-32 turns
    float s, c;
    sincospif((float)rest * 0x1p-31f, &s, &c);
    const float c1 = quarter & 1 ? -s : c, s1 = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-c1, -s1) : make_float2(c1, s1);
}

// Angles of rows [t0, t0 + n_rows) of this CTA: cosines [n_rows, rot / 2], then sines
struct Angles {
    float *cos_, *sin_;
    int half;
    __device__ __forceinline__ Angles(const Turns& a, float* smem, int n_rows)
        : cos_(smem), sin_(smem + n_rows * (a.rot / 2)), half(a.rot / 2) {}
    __device__ __forceinline__ void fill(const Turns& a, int64_t t0, int n_rows, int64_t T) {
        for (int i = threadIdx.x; i < n_rows * half; i += (int)blockDim.x) {
            const int64_t t = t0 + i / half;
            if (t >= T) break;
            const float2 v = cos_sin((uint64_t)a.positions[t] * (uint64_t)a.turns[i % half]);
            cos_[i] = v.x;
            sin_[i] = v.y;
        }
    }
    // of a lane's 8 pairs
    __device__ __forceinline__ void get(int row, int lane, float (&c)[8], float (&s)[8]) const {
        const float4* pc = reinterpret_cast<const float4*>(cos_ + row * half + 8 * lane);
        const float4* ps = reinterpret_cast<const float4*>(sin_ + row * half + 8 * lane);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 x = pc[i], y = ps[i];
            c[4 * i] = x.x; c[4 * i + 1] = x.y; c[4 * i + 2] = x.z; c[4 * i + 3] = x.w;
            s[4 * i] = y.x; s[4 * i + 1] = y.y; s[4 * i + 2] = y.z; s[4 * i + 3] = y.w;
        }
    }
};

// The two pieces of a head's row that a lane holds: from elements at0 and at1
struct LanePieces {
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

// turns 8 pairs: (u[i], w[i]), or neighbours within u and within w
__device__ __forceinline__ void turn(float (&u)[8], float (&w)[8], const float (&c)[8], const float (&s)[8],
                                     bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = u[2 * i], b = u[2 * i + 1], d = w[2 * i], e = w[2 * i + 1];
            u[2 * i] = a * c[i] - b * s[i];
            u[2 * i + 1] = b * c[i] + a * s[i];
            w[2 * i] = d * c[4 + i] - e * s[4 + i];
            w[2 * i + 1] = e * c[4 + i] + d * s[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = u[i], b = w[i];
            u[i] = a * c[i] - b * s[i];
            w[i] = b * c[i] + a * s[i];
        }
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
// Heads are query heads, key heads, and with a cache the value heads.
struct Forward {
    const void* x;
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
    Shape shape;
    int32_t hq, hk, heads;   // query heads, key heads, all
    int32_t out_heads;       // the first of them that go to out
    int32_t D;
    float eps, inv_d;
};

template <class Row8, int kLanes, int kRows, int kCache /* -1: none */>
__global__ void __launch_bounds__(kMaxThreads) rotary_kernel(const Forward a) {
    extern __shared__ __align__(16) float smem[];
    grid_dep_launch();
    grid_dep_wait();
    const Spot<kLanes, kRows> at(a.shape, blockIdx.x);
    const LanePieces p(at.lane, a.D, a.turns);
    const bool key = at.head >= a.hq, value = at.head >= a.hq + a.hk, in = p.in && at.head < a.heads;
    const void* from = value ? a.v : a.x;
    const int64_t ld = value ? a.ld_v : a.ld_x;
    const int64_t head_at = (int64_t)(value ? at.head - a.hq - a.hk : at.head) * a.D;
    Row8 r[kRows][2], w[2];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t t = at.t0 + at.row + k * a.shape.down;
        r[k][0].zero();
        r[k][1].zero();
        if (in && t < a.T) {
            r[k][0].load(from, t * ld + head_at + p.at0);
            r[k][1].load(from, t * ld + head_at + p.at1);
        }
    }
    const void* weight = value ? nullptr : key ? a.wk : a.wq;
    w[0].zero();
    w[1].zero();
    if (weight && in) {
        w[0].load(weight, p.at0);
        w[1].load(weight, p.at1);
    }
    Angles angles(a.turns, smem, a.shape.down * kRows);
    if (a.turns.rot) {
        angles.fill(a.turns, at.t0, a.shape.down * kRows, a.T);
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int row = at.row + k * a.shape.down;
        const int64_t t = at.t0 + row;
        float y[8], z[8], f = 1.f;
        r[k][0].get(y);
        r[k][1].get(z);
        if (a.wq || a.wk) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], fmaf(z[i], z[i], ss));
            ss = sum_over_lanes<kLanes>(ss);
            if (weight) {
                f = rsqrtf(ss * a.inv_d + a.eps);
                float g[8];
                w[0].get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= g[i];
                w[1].get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= g[i];
            }
        }
        if (p.turned && !value && t < a.T) {
            float c[8], s[8];
            angles.get(row, at.lane, c, s);
            if (weight) {            // the row's factor goes into its angles' cosines and sines
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] *= f;
                    s[i] *= f;
                }
            }
            turn(y, z, c, s, a.turns.interleaved);
        } else if (weight) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] *= f;
                z[i] *= f;
            }
        }
        const bool here = in && t < a.T;
        if (here && at.head < a.out_heads) {
            Row8::store(a.out, t * a.ld_out + head_at + p.at0, y);
            Row8::store(a.out, t * a.ld_out + head_at + p.at1, z);
        }
        if (kCache < 0) continue;
        uint32_t amax = 0;
        if (kCache == LORA_CACHE_E4M3) amax = max_over_lanes<kLanes>(max(abs_bits_max(y), abs_bits_max(z)));
        if (!here || !key) continue;
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= a.cache.slots) continue;
        const RowPlace place(a.cache, slot);
        const int head = at.head - a.hq - (value ? a.hk : 0);
        char* to = (value ? a.cache.v : a.cache.k) + place.row + head * a.cache.head_stride;
        if (kCache == LORA_CACHE_BF16) {
            Row8Bf16::store(to, p.at0, y);
            Row8Bf16::store(to, p.at1, z);
        } else {
            float inv;
            const float sc = block_scale(amax, &inv);
            *reinterpret_cast<uint2*>(to + p.at0) = encode8(y, inv);
            *reinterpret_cast<uint2*>(to + p.at1) = encode8(z, inv);
            if (at.lane == 0) (value ? a.cache.vs : a.cache.ks)[place.scale + head * a.cache.s_head] = sc;
        }
    }
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
    float* parts;            // [CTAs, 2, D]: each CTA's sums of the weights' gradients; null: not wanted
    Turns turns;
    int64_t T, n_blocks;     // rows are taken shape.down * kRows at a time
    Shape shape;
    int32_t hq, heads, D;
    float eps, inv_d;
};

template <class Row8, int kLanes, int kRows, bool kNorm, bool kWeights>
__global__ void __launch_bounds__(kMaxThreads) rotary_backward_kernel(const Backward a) {
    extern __shared__ __align__(16) float smem[];
    grid_dep_launch();
    grid_dep_wait();
    const int lane = threadIdx.x % kLanes;
    const LanePieces p(lane, a.D, a.turns);
    const Spot<kLanes, kRows> spot(a.shape, 0);
    const bool key = spot.head >= a.hq, in = p.in && spot.head < a.heads;
    const int64_t head_at = (int64_t)spot.head * a.D;
    const void* weight = key ? a.wk : a.wq;
    Row8 w[2];
    if (kNorm && weight && in) {
        w[0].load(weight, p.at0);
        w[1].load(weight, p.at1);
    }
    Angles angles(a.turns, smem, a.shape.down * kRows);
    float sum[kWeights ? 16 : 1] = {};
    for (int64_t block = blockIdx.x; block < a.n_blocks; block += gridDim.x) {
        const int64_t t0 = block * (int64_t)(a.shape.down * kRows);
        Row8 r[kRows][2], d[kRows][2];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t t = t0 + spot.row + k * a.shape.down;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                r[k][i].zero();
                d[k][i].zero();
            }
            if (in && t < a.T) {
                d[k][0].load(a.dout, t * a.ld_dout + head_at + p.at0);
                d[k][1].load(a.dout, t * a.ld_dout + head_at + p.at1);
                if (kNorm) {
                    r[k][0].load(a.x, t * a.ld_x + head_at + p.at0);
                    r[k][1].load(a.x, t * a.ld_x + head_at + p.at1);
                }
            }
        }
        if (a.turns.rot) {
            angles.fill(a.turns, t0, a.shape.down * kRows, a.T);
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int row = spot.row + k * a.shape.down;
            const int64_t t = t0 + row;
            float y[8], z[8];
            d[k][0].get(y);
            d[k][1].get(z);
            if (p.turned && t < a.T) {
                float c[8], s[8];
                angles.get(row, lane, c, s);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = -s[i];
                turn(y, z, c, s, a.turns.interleaved);
            }
            if (kNorm) {
                float v[8], x[8];
                r[k][0].get(v);
                r[k][1].get(x);
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], fmaf(x[i], x[i], ss));
                const float f = rsqrtf(sum_over_lanes<kLanes>(ss) * a.inv_d + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= f;
                    x[i] *= f;
                }
                if constexpr (kWeights)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        sum[i] = fmaf(y[i], v[i], sum[i]);
                        sum[8 + i] = fmaf(z[i], x[i], sum[8 + i]);
                    }
                float along = 0.f;
                if (weight && in) {
                    float g[8];
                    w[0].get(g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] *= g[i];
                        along = fmaf(y[i], v[i], along);
                    }
                    w[1].get(g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        z[i] *= g[i];
                        along = fmaf(z[i], x[i], along);
                    }
                }
                along = sum_over_lanes<kLanes>(along) * a.inv_d;
                if (weight) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        y[i] = f * fmaf(-v[i], along, y[i]);
                        z[i] = f * fmaf(-x[i], along, z[i]);
                    }
                }
            }
            if (in && t < a.T) {
                Row8::store(a.dx, t * a.ld_dx + head_at + p.at0, y);
                Row8::store(a.dx, t * a.ld_dx + head_at + p.at1, z);
            }
        }
        if (a.turns.rot) __syncthreads();      // the next rows' angles take these rows' place
    }
    if constexpr (kWeights) {
        // every head's sums, then the query heads' and the key heads' together
        constexpr int kHeads = kMaxThreads / kLanes;
        __shared__ float total[kHeads][kLanes * 16];
        const int group = threadIdx.x / kLanes;
#pragma unroll
        for (int i = 0; i < 16; ++i) total[group][lane * 16 + i] = sum[i];
        __syncthreads();
        const int groups = (int)blockDim.x / kLanes, across = a.shape.across * (32 / kLanes);
        for (int e = threadIdx.x; e < 2 * kLanes * 16; e += (int)blockDim.x) {
            const int j = e / (kLanes * 16), i = e % (kLanes * 16);
            const LanePieces q(i / 16, a.D, a.turns);
            if (!q.in) continue;
            float v = 0.f;
            for (int k = 0; k < groups; ++k) {
                const int head = (int)blockIdx.y * across + k % across;
                if (head < a.heads && (head >= a.hq) == (j == 1)) v += total[k][i];
            }
            const int d = i % 16 < 8 ? q.at0 + i % 16 : q.at1 + i % 16 - 8;
            a.parts[(((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 + j) * a.D + d] = v;
        }
    }
}

// Sums of the CTAs' parts [n, 2 D], in a fixed order; 32 columns a CTA
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* parts, int n, int D, float* dq, float* dk) {
    __shared__ float s[32][33];
    grid_dep_launch();
    grid_dep_wait();
    const int col = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
    float v = 0.f;
    if (col < 2 * D)
#pragma unroll 4
        for (int i = y; i < n; i += 32) v += parts[(int64_t)i * 2 * D + col];
    s[y][threadIdx.x % 32] = v;
    __syncthreads();
    if (y > 0 || col >= 2 * D) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
    float* to = col < D ? dq : dk;
    if (to) to[col % D] = v;
}

// ---------------------------------------------------------------------------------------------------- cache read
struct Read {
    CacheView cache;
    const int64_t* slots;
    void *k, *v;
    int64_t ld_k, ld_v;
    int64_t T;
    Shape shape;
    int32_t n_heads, D;
};

// Heads are key heads, then value heads; a lane takes 16 neighbouring elements.
template <class Row8, int kLanes, int kRows, int kCache>
__global__ void __launch_bounds__(kMaxThreads) cache_read_kernel(const Read a) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr bool kE4m3 = kCache == LORA_CACHE_E4M3;
    const Spot<kLanes, kRows> spot(a.shape, blockIdx.x);
    const bool value = spot.head >= a.n_heads;
    const int head = value ? spot.head - a.n_heads : spot.head;
    if (head >= a.n_heads || 16 * spot.lane >= a.D) return;
    const char* from = (value ? a.cache.v : a.cache.k) + head * a.cache.head_stride + (kE4m3 ? 16 : 32) * spot.lane;
    const float* scales = kE4m3 ? (value ? a.cache.vs : a.cache.ks) + head * a.cache.s_head : nullptr;
    uint4 q[kRows][kE4m3 ? 1 : 2];
    float sc[kRows];
    int64_t slot[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t t = spot.t0 + spot.row + k * a.shape.down;
        slot[k] = t < a.T ? a.slots[t] : -1;
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        sc[k] = 0.f;
        for (auto& w : q[k]) w = make_uint4(0, 0, 0, 0);
        if (slot[k] < 0 || slot[k] >= a.cache.slots) continue;
        const RowPlace place(a.cache, slot[k]);
        if (kE4m3) sc[k] = scales[place.scale];
        q[k][0] = *reinterpret_cast<const uint4*>(from + place.row);
        if (!kE4m3) q[k][kE4m3 ? 0 : 1] = *reinterpret_cast<const uint4*>(from + place.row + 16);
    }
    void* to = value ? a.v : a.k;
    const int64_t ld = value ? a.ld_v : a.ld_k, col = (int64_t)head * a.D + 16 * spot.lane;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t t = spot.t0 + spot.row + k * a.shape.down;
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
            Row8::store(to, t * ld + col + 8 * i, x);
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

// CTAs of up to eight warps: the heads in equal shares across, and as many rows of warps as are left room for.
struct Launch {
    Shape shape;
    unsigned y;
};
Launch launch_of(int heads, int D, int64_t T) {
    const int per_warp = 32 / lanes_of(D), all = (heads + per_warp - 1) / per_warp;
    Launch l;
    l.y = (unsigned)((all + 7) / 8);
    l.shape.across = (all + (int)l.y - 1) / (int)l.y;
    l.shape.down = (int)std::min<int64_t>(8 / l.shape.across, T);
    return l;
}
unsigned threads_of(const Launch& l) { return (unsigned)(32 * l.shape.across * l.shape.down); }
// Rows that a lane takes: one where all CTAs fit a round on the SMs, `most` else.
bool one_row(const Launch& l, int64_t T) { return T * l.y * threads_of(l) <= 152ll * 1024 * l.shape.down; }
int64_t blocks(const Launch& l, int64_t T, int rows) { return (T + l.shape.down * rows - 1) / (l.shape.down * rows); }
size_t angle_bytes(const Launch& l, int rows, int rot) { return (size_t)l.shape.down * rows * rot * sizeof(float); }

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
cudaError_t launch_forward(Forward a, cudaStream_t st) {
    return by_lanes(a.D, [&](auto lanes) {
        const Launch l = launch_of(a.heads, a.D, a.T);
        a.shape = l.shape;
        auto go = [&](auto rows) {
            constexpr int kRows = decltype(rows)::value;
            return launch_pdl(rotary_kernel<Row8, decltype(lanes)::value, kRows, kCache>,
                              dim3((unsigned)blocks(l, a.T, kRows), l.y), dim3(threads_of(l)),
                              angle_bytes(l, kRows, a.turns.rot), st, a);
        };
        return one_row(l, a.T) ? go(std::integral_constant<int, 1>()) : go(std::integral_constant<int, 4>());
    });
}
cudaError_t forward(lora_dtype_t dt, int cache, const Forward& a, cudaStream_t st) {
    return by_type(dt, [&](auto row) {
        using Row8 = decltype(row);
        return cache < 0 ? launch_forward<Row8, -1>(a, st)
                         : cache == LORA_CACHE_BF16 ? launch_forward<Row8, LORA_CACHE_BF16>(a, st)
                                                    : launch_forward<Row8, LORA_CACHE_E4M3>(a, st);
    });
}

constexpr unsigned kMaxParts = 608;  // CTAs of a backward that sums the weights' gradients: four on each SM

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
        a.out_heads = cache && !keep_keys ? r->n_heads : r->n_heads + r->n_kv_heads;
        const int es = elem_size(dt);
        if ((rc = check_matrix(fn, "x", x, all, ld_x, es)) != LORA_OK) return rc;
        if ((rc = check_matrix(fn, "out", out, a.out_heads * D, ld_out, es)) != LORA_OK) return rc;
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
        a.T = T; a.hq = r->n_heads; a.hk = r->n_kv_heads;
        a.heads = r->n_heads + r->n_kv_heads * (cache ? 2 : 1);
        a.D = (int32_t)D; a.eps = r->eps; a.inv_d = 1.f / (float)D;
        return enqueued(fn, forward(dt, cache ? cache->dtype : -1, a, static_cast<cudaStream_t>(stream)));
    });
}

extern "C" size_t lora_rotary_workspace_size(int32_t T, const lora_rotary_t* r) {
    const int64_t n = guarded([&]() -> int64_t {
        if (check_rotary("lora_rotary_workspace_size", T, LORA_BF16, r) != LORA_OK) return 0;
        return (int64_t)kMaxParts * 2 * r->head_dim * sizeof(float);
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
        if (weights && (!workspace || !is_aligned(workspace, 16) ||
                        ws_bytes < (size_t)kMaxParts * 2 * D * sizeof(float)))
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
        a.T = T; a.hq = r->n_heads; a.heads = r->n_heads + r->n_kv_heads;
        a.D = (int32_t)D; a.eps = r->eps; a.inv_d = 1.f / (float)D;
        int parts = 0;
        cudaError_t e = cudaSuccess;
        if (T > 0)
            e = by_type(dt, [&](auto row) {
                using Row8 = decltype(row);
                return by_lanes(a.D, [&](auto lanes) {
                    const Launch l = launch_of(a.heads, a.D, a.T);
                    a.shape = l.shape;
                    auto go = [&](auto rows, auto nrm, auto wts) {
                        constexpr int kRows = decltype(rows)::value;
                        constexpr bool kWeights = decltype(wts)::value;
                        a.n_blocks = blocks(l, a.T, kRows);
                        const int64_t n = kWeights ? std::min<int64_t>(a.n_blocks, std::max(1u, kMaxParts / l.y)) : a.n_blocks;
                        parts = (int)(n * l.y);
                        return launch_pdl(rotary_backward_kernel<Row8, decltype(lanes)::value, kRows, decltype(nrm)::value,
                                                                 kWeights>,
                                          dim3((unsigned)n, l.y), dim3(threads_of(l)), angle_bytes(l, kRows, a.turns.rot), st,
                                          a);
                    };
                    auto sized = [&](auto nrm, auto wts) {
                        return one_row(l, a.T) ? go(std::integral_constant<int, 1>(), nrm, wts)
                                               : go(std::integral_constant<int, 2>(), nrm, wts);
                    };
                    return !norm ? sized(std::false_type(), std::false_type())
                                 : !weights ? sized(std::true_type(), std::false_type())
                                            : sized(std::true_type(), std::true_type());
                });
            });
        if (e == cudaSuccess && weights)
            e = launch_pdl(weight_grad_kernel, dim3((unsigned)((2 * D + 31) / 32)), dim3(1024), 0, st,
                           static_cast<const float*>(workspace), parts, (int)D, dq_weight, dk_weight);
        return enqueued(fn, e);
    });
}

extern "C" int lora_cache_write(int32_t T, lora_dtype_t dt, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                const lora_cache_t* cache, const int64_t* slots, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_cache_write";
        Forward a = {};
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
        a.x = k; a.ld_x = ld_k; a.v = v; a.ld_v = ld_v; a.slots = slots;
        a.T = T; a.hk = cache->n_heads; a.heads = 2 * cache->n_heads; a.D = cache->head_dim;
        return enqueued(fn, forward(dt, cache->dtype, a, static_cast<cudaStream_t>(stream)));
    });
}

extern "C" int lora_cache_read(int32_t T, lora_dtype_t dt, const lora_cache_t* cache, const int64_t* slots, void* k,
                               int64_t ld_k, void* v, int64_t ld_v, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_cache_read";
        Read a = {};
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
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return enqueued(fn, by_type(dt, [&](auto row) {
            using Row8 = decltype(row);
            return by_lanes(a.D, [&](auto lanes) {
                const Launch l = launch_of(2 * a.n_heads, a.D, a.T);
                a.shape = l.shape;
                auto go = [&](auto rows, auto c) {
                    constexpr int kRows = decltype(rows)::value;
                    return launch_pdl(cache_read_kernel<Row8, decltype(lanes)::value, kRows, decltype(c)::value>,
                                      dim3((unsigned)blocks(l, a.T, kRows), l.y), dim3(threads_of(l)), 0, st, a);
                };
                auto sized = [&](auto c) {
                    return one_row(l, a.T) ? go(std::integral_constant<int, 1>(), c)
                                           : go(std::integral_constant<int, 4>(), c);
                };
                return cache->dtype == LORA_CACHE_BF16 ? sized(std::integral_constant<int, LORA_CACHE_BF16>())
                                                       : sized(std::integral_constant<int, LORA_CACHE_E4M3>());
            });
        }));
    });
}
