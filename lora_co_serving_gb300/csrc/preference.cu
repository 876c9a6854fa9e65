// preference.cu -- the preference loss of a fine-tuning step (include/lora_preference.h), forward and backward.
//
// Forward: one pass over each counted row of logits with a running maximum and sum (the row's log-sum-exp), then a
// small kernel that adds up each pair's sequences in about 48 bits, in a fixed order.  Backward: one pass that reads a
// row and writes its gradient.  Both passes move each logit once and are bounded by the memory rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "fp8.h"
#include "lora_preference.h"
#include "tc_prims.h"

namespace lora {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eHigh = 1.44268798828125f;        // log2(e) to 16 bits, and the rest of it
constexpr float kLog2eLow = (float)(1.4426950408889634 - (double)kLog2eHigh);
constexpr float kLn2High = 0.693145751953125f;         // log(2) to 16 bits, and the rest
constexpr float kLn2Low = (float)(0.6931471805599453 - (double)kLn2High);
// ex2.approx lies low by about this much on average: the mean error of 4096 rows' log-sum-exp was 2.4e-8 to 5.6e-8 over
// vocabularies of 500 to 128256 and standard deviations of the logits from 1 to 3.  It is nothing against a row's own
// rounding, 2e-7, but the same in every token of a sequence's sum.
constexpr float kExp2Low = 4e-8f;
constexpr int kPairThreads = 512;

// 2^x; 0 for x = -infinity, results below the smallest normal number are 0
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Elements of a row, and 16-byte pieces of it
struct Bf16 {
    typedef __nv_bfloat16 T;
    static constexpr int kN = 8;
    static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ uint4 lowest() {     // all -infinity
        return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
    }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&q)[N]) {
        const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(q);
        __nv_bfloat162 m = v[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = __hmax2(m, v[i]);
        return fmaxf(__low2float(m), __high2float(m));
    }
};
struct F32 {
    typedef float T;
    static constexpr int kN = 4;
    static __device__ __forceinline__ float get(T v) { return v; }
    static __device__ __forceinline__ T put(float v) { return v; }
    static __device__ __forceinline__ uint4 lowest() {
        return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
    }
    static __device__ __forceinline__ void unpack(const uint4& q, float (&x)[4]) {
        x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y);
        x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&q)[N]) {
        const float* v = reinterpret_cast<const float*>(q);
        float m = v[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = fmaxf(m, v[i]);
        return m;
    }
};

// Rows start anywhere (a row of odd length moves the next one off a 16-byte boundary): elements [0, head) come
// before the first boundary, then `vecs` pieces of 16 bytes, then the rest.
template <class E>
struct RowSpan {
    int head, vecs;
    __device__ __forceinline__ RowSpan(const typename E::T* row, int V) {
        head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(typename E::T)));
        vecs = (V - head) / E::kN;
    }
};

// Running sum of e^x over what was seen, as s 2^n.  n is a whole number, the smallest not below the largest
// x log2(e) so far: rescaling by 2^(n - n') is exact.  log2(e) is taken in two parts: its float32 value alone is
// 1.3e-8 off, which shifts every row's log-sum-exp the same way (by 7e-8 at a mean logit of 5), and a sequence's sum
// of log ratios, where random errors cancel, by that times its length.  The high part has 16 bits: what the low part
// adds is then far above a unit of the sum it is added to.
struct ExpSum {
    float n = -INFINITY, s = 0.f;
    static __device__ __forceinline__ float weight(float from, float to) {
        return from == to ? 1.f : exp2_fast(from - to);       // -infinity on both sides: an empty sum stays empty
    }
    __device__ __forceinline__ void join(float n2, float s2) {
        const float to = fmaxf(n, n2);
        s = s * weight(n, to) + s2 * weight(n2, to);
        n = to;
    }
    __device__ __forceinline__ void raise(float largest) {
        const float c = ceilf(largest * kLog2e);
        if (c > n) {
            s *= weight(n, c);
            n = c;
        }
    }
    // the terms of some elements not above `raise`d ones, added pairwise: small terms are not lost to a large sum
    template <int N>
    __device__ __forceinline__ float terms(const float (&x)[N]) const {
        const float off = n == -INFINITY ? 0.f : -n;
        float e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = exp2_fast(fmaf(x[i], kLog2eLow, fmaf(x[i], kLog2eHigh, off)));
#pragma unroll
        for (int w = 1; w < N; w *= 2)
#pragma unroll
            for (int i = 0; i + w < N; i += 2 * w) e[i] += e[i + w];
        return e[0];
    }
};

// The backward reads the logits once more.  The last kKept bytes of them are read so that L2 may hold them until then,
// the rest so that it is the first to go; dlogits_kernel takes the held rows and the others in turn.  The step of 4096
// rows of 32000 takes 98 us so, 104 us with plain reads and the backward from the last row to the first: 80 MB of its
// reads then hit L2 at its start, while all that memory does is write.  (Kept bytes of 60 and 100 MB: 98.3 and 98.2 us.)
constexpr int64_t kKept = 80ll << 20;
__device__ __forceinline__ uint64_t l2_policy(bool keep) {
    uint64_t normal, first;
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    return keep ? normal : first;
}
__device__ __forceinline__ uint4 load_hinted(const uint4* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}

// One CTA of kThreads per row; each thread takes kAhead pieces of 16 bytes at a time.
template <class E, int kThreads, int kAhead>
__global__ void __launch_bounds__(kThreads) logprob_kernel(int32_t V, const typename E::T* logits,
                                                           int64_t ld, const int64_t* labels,
                                                           float* logp, float* lse) {
    grid_dep_launch();
    grid_dep_wait();
    const int64_t t = blockIdx.x;
    const int64_t label = labels[t];
    if (label < 0) {
        if (threadIdx.x == 0) logp[t] = lse[t] = 0.f;
        return;
    }
    const typename E::T* row = logits + t * ld;
    const RowSpan<E> span(row, V);
    const uint4* q = reinterpret_cast<const uint4*>(row + span.head);
    const float at = (threadIdx.x == 0 && label < V) ? E::get(row[label]) : NAN;
    const uint64_t policy = l2_policy((gridDim.x - t) * V * (int64_t)sizeof(typename E::T) <= kKept);
    ExpSum a;
    for (int i0 = threadIdx.x; i0 < span.vecs; i0 += kThreads * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = i0 + j * kThreads < span.vecs ? load_hinted(q + i0 + j * kThreads, policy) : E::lowest();
        a.raise(E::largest(v));
        float e[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            float x[E::kN];
            E::unpack(v[j], x);
            e[j] = a.terms(x);
        }
#pragma unroll
        for (int w = 1; w < kAhead; w *= 2)
#pragma unroll
            for (int j = 0; j + w < kAhead; j += 2 * w) e[j] += e[j + w];
        a.s += e[0];
    }
    // head and tail: fewer than two pieces
    const int loose = V - span.vecs * E::kN;
    for (int i = threadIdx.x; i < loose; i += kThreads) {
        const float x[1] = {E::get(row[i < span.head ? i : span.vecs * E::kN + i])};
        a.raise(x[0]);
        a.s += a.terms(x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float n2 = __shfl_xor_sync(0xffffffffu, a.n, o), s2 = __shfl_xor_sync(0xffffffffu, a.s, o);
        a.join(n2, s2);
    }
    if constexpr (kThreads > 32) {
        constexpr int kWarps = kThreads / 32;
        __shared__ float sn[kWarps], ss[kWarps];
        if (threadIdx.x % 32 == 0) {
            sn[threadIdx.x / 32] = a.n;
            ss[threadIdx.x / 32] = a.s;
        }
        __syncthreads();
        if (threadIdx.x >= 32) return;
        a.n = threadIdx.x < kWarps ? sn[threadIdx.x] : -INFINITY;
        a.s = threadIdx.x < kWarps ? ss[threadIdx.x] : 0.f;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1) {
            const float n2 = __shfl_xor_sync(0xffffffffu, a.n, o), s2 = __shfl_xor_sync(0xffffffffu, a.s, o);
            a.join(n2, s2);
        }
    }
    // logits of 2^30 and beyond (a mask of the type's lowest value over the whole row) lose their differences in
    // x log2(e) - n: one warp takes such a row again, from its largest logit
    constexpr float kFar = 1073741824.f;
    if (!(fabsf(__shfl_sync(0xffffffffu, a.n, 0)) < kFar)) {
        float m = -INFINITY, s = 0.f;
        for (int i = threadIdx.x; i < V; i += 32) m = fmaxf(m, E::get(row[i]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int i = threadIdx.x; i < V; i += 32) s += __expf(E::get(row[i]) - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {                  // no finite logit: -infinity less itself, NaN
            lse[t] = m + logf(s);
            logp[t] = (at - m) - logf(s);
        }
        return;
    }
    if (threadIdx.x == 0) {
        // log of the sum is n log(2) + log(s), with s brought to [1, 2) first; x - lse is formed from its small parts,
        // not from the rounded lse.  (frexpf leaves a NaN as it is)
        int e;
        const float m = 2.f * frexpf(a.s, &e), n = a.n + (float)(e - 1);
        const float r = logf(m) + fmaf(n, kLn2Low, kExp2Low);
        lse[t] = fmaf(n, kLn2High, r);
        logp[t] = fmaf(-n, kLn2High, at) - r;
    }
}

// Sequences in increasing start order (zero-length ones left out): `id` = 2 pair + (0 chosen, 1 rejected).  Tables of up
// to kFewPairs pairs, a usual step's, travel in a smaller launch parameter than the 5 KB of the largest.
constexpr int kFewPairs = 16;
template <int kPairs>
struct Sequences {
    int32_t n;
    int32_t start[2 * kPairs], end[2 * kPairs];
    int16_t id[2 * kPairs];
};
template <int kPairs>
struct Pairs {
    lora_pair_t p[kPairs];
};

template <int kPairs>
__device__ __forceinline__ int sequence_of(const Sequences<kPairs>& s, int t) {
    int lo = 0, hi = s.n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s.start[mid] <= t) lo = mid + 1; else hi = mid;
    }
    return (lo > 0 && t < s.end[lo - 1]) ? s.id[lo - 1] : -1;
}

// A sum held in two float32 numbers (Knuth's two-sum: hi + lo is the exact sum of every addition's operands but for the
// rounding of lo), about 48 bits.  An infinity or NaN makes lo NaN and lives on in hi.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x, float x_lo = 0.f) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        hi = s;
        lo = __fadd_rn(lo, __fadd_rn(err, x_lo));
    }
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

// One CTA per pair, half of its threads for each sequence.  The differences lp - ref are small and their sums cancel:
// they are added up in about 48 bits (in float32 pairs: 64-bit arithmetic is slow on this GPU, 10 us against 4).
template <int kPairs>
__global__ void __launch_bounds__(kPairThreads) pair_loss_kernel(const __grid_constant__ Pairs<kPairs> pairs,
                                                                 const int64_t* labels,
                                                                 const float* logp,
                                                                 const float* ref, float beta, float eps,
                                                                 float* loss, float* rewards,
                                                                 float* coef) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr int kHalf = kPairThreads / 2, kWarps = kHalf / 32;
    __shared__ float sh[2][kWarps][2];
    const lora_pair_t p = pairs.p[blockIdx.x];
    const int side = threadIdx.x / kHalf;
    const int64_t t0 = side ? p.rejected_start : p.chosen_start;
    const int64_t t1 = t0 + (side ? p.rejected_len : p.chosen_len);
    Sum2 sum;
    for (int64_t t = t0 + threadIdx.x % kHalf; t < t1; t += kHalf) {
        const float a = logp[t], b = ref[t];
        if (labels[t] >= 0) sum.add(a - b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, sum.hi, o), lo = __shfl_xor_sync(0xffffffffu, sum.lo, o);
        sum.add(hi, lo);
    }
    if (threadIdx.x % 32 == 0) {
        sh[side][threadIdx.x % kHalf / 32][0] = sum.hi;
        sh[side][threadIdx.x % kHalf / 32][1] = sum.lo;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    Sum2 d2[2];
    for (int i = 0; i < 2; ++i)
        for (int w = 0; w < kWarps; ++w) d2[i].add(sh[i][w][0], sh[i][w][1]);
    const float d[2] = {beta * d2[0].value(), beta * d2[1].value()};
    Sum2 diff = d2[0];
    diff.add(-d2[1].hi, -d2[1].lo);
    const float m = beta * diff.value();
    const float e = expf(-fabsf(m)), soft = log1pf(e);     // -log sig(m) = max(-m, 0) + log(1 + e^-|m|)
    const float small = e / (1.f + e), large = 1.f / (1.f + e);
    const float sig = m >= 0.f ? large : small, sig_minus = m >= 0.f ? small : large;
    // without smoothing an infinite m of the certain side adds nothing (0 times infinity)
    const float smooth = eps > 0.f ? eps * (fmaxf(m, 0.f) + soft) : 0.f;
    loss[blockIdx.x] = isnan(m) ? NAN : (1.f - eps) * (fmaxf(-m, 0.f) + soft) + smooth;
    rewards[2 * blockIdx.x] = d[0];
    rewards[2 * blockIdx.x + 1] = d[1];
    const float k = isnan(m) ? NAN : beta * (eps * sig - (1.f - eps) * sig_minus);
    coef[2 * blockIdx.x] = k;
    coef[2 * blockIdx.x + 1] = -k;
}

// The backward's probabilities are e^(x - lse), and lse is one float32 number: half a unit of it, 2^-25 of its size, is
// every probability's relative error.  From kFarLse on that is 2^-17 and more (all of a probability where every logit is
// the type's lowest value), so the row is summed up once more, from its largest logit, and the probabilities are taken
// from there.  An lse that is not the row's own, by more than roundings, is the caller's and stays.
// 4096 rows of 32000 in 16 bits: 105 us where all of them are summed up again, 78 us where none is (without the one pass
// in 16-byte pieces: 169 us).
constexpr float kFarLse = 256.f;
struct RowBase {
    float from, less;                          // a probability is 2^((x - from) log2(e) - less)
};
template <class E, int kThreads>
__device__ __noinline__ RowBase far_row(const typename E::T* row, int V, float z) {
    constexpr int kWarps = kThreads / 32, kAhead = 4;
    __shared__ float sm[kWarps], ss[kWarps];
    const RowSpan<E> span(row, V);
    const uint4* q = reinterpret_cast<const uint4*>(row + span.head);
    float m = -INFINITY, s = 0.f;              // the largest logit so far, and the sum of e^(x - m)
    // (from == to: -infinity on both sides, an empty sum)
    auto weight = [](float from, float to) { return from == to ? 1.f : exp2_fast((from - to) * kLog2e); };
    auto take = [&](const auto& x, int n, float largest) {
        const float to = fmaxf(m, largest);
        s *= weight(m, to);
        m = to;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < n; ++i) sum += x[i] == -INFINITY ? 0.f : exp2_fast((x[i] - m) * kLog2e);
        s += sum;
    };
    for (int i0 = threadIdx.x; i0 < span.vecs; i0 += kThreads * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = i0 + j * kThreads < span.vecs ? q[i0 + j * kThreads] : E::lowest();
        const float largest = E::largest(v);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            float x[E::kN];
            E::unpack(v[j], x);
            take(x, E::kN, largest);
        }
    }
    for (int i = threadIdx.x; i < V - span.vecs * E::kN; i += kThreads) {
        const float x[1] = {E::get(row[i < span.head ? i : span.vecs * E::kN + i])};
        take(x, 1, x[0]);
    }
    auto join = [&](float m2, float s2) {
        const float to = fmaxf(m, m2);
        s = s * weight(m, to) + s2 * weight(m2, to);
        m = to;
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        join(m2, s2);
    }
    if (threadIdx.x % 32 == 0) {
        sm[threadIdx.x / 32] = m;
        ss[threadIdx.x / 32] = s;
    }
    __syncthreads();                           // in place: the row is written after this
    m = -INFINITY, s = 0.f;
    for (int w = 0; w < kWarps; ++w) join(sm[w], ss[w]);       // in one order for every thread
    // the forward's lse is a few units off at most
    const bool own = fabsf(m + logf(s) - z) <= 4.7683716e-7f * fabsf(z);         // 2^-21
    return own ? RowBase{m, log2f(s)} : RowBase{z, 0.f};
}

// One CTA per row; rows are taken from the end and from the start in turn, so that the rows that L2 still holds from
// the forward (see kKept) and those that come from memory are read side by side.  What is written is not read again
// here and does not push them out (st.cs).
template <class E, int kThreads, int kAhead, int kPairs>
__global__ void __launch_bounds__(kThreads) dlogits_kernel(int32_t V, const typename E::T* logits, int64_t ld,
                                                           const int64_t* labels,
                                                           const float* lse,
                                                           const float* coef,
                                                           const __grid_constant__ Sequences<kPairs> seqs,
                                                           const float* dloss, float dloss_all,
                                                           typename E::T* dlogits, int64_t ld_d) {
    grid_dep_wait();
    const int64_t t = blockIdx.x % 2 == 0 ? (int64_t)gridDim.x - 1 - blockIdx.x / 2 : blockIdx.x / 2;
    const int64_t label = labels[t];
    const typename E::T* row = logits + t * ld;
    typename E::T* out = dlogits + t * ld_d;
    const RowSpan<E> span(out, V);
    const int seq = label < 0 ? -1 : sequence_of(seqs, (int)t);
    if (seq < 0) {
        uint4* o = reinterpret_cast<uint4*>(out + span.head);
        for (int i = threadIdx.x; i < span.vecs; i += kThreads) __stcs(o + i, make_uint4(0, 0, 0, 0));
        for (int i = threadIdx.x; i < V - span.vecs * E::kN; i += kThreads)
            out[i < span.head ? i : span.vecs * E::kN + i] = E::put(0.f);
        return;
    }
    float k = coef[seq] * (dloss ? dloss[seq / 2] : dloss_all);
    if (label >= V) k = NAN;
    RowBase base{lse[t], 0.f};
    if (fabsf(base.from) >= kFarLse && fabsf(base.from) < INFINITY) base = far_row<E, kThreads>(row, V, base.from);
    const int hit = label < V ? (int)label : -1;
    auto grad = [&](float x, bool at) {
        const float p = exp2_fast(fmaf(x - base.from, kLog2e, -base.less));
        return at ? k * (1.f - p) : -k * p;
    };
    // both rows on the same 16-byte phase: whole pieces; else element by element
    const bool whole = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int vecs = whole ? span.vecs : 0;
    const uint4* q = reinterpret_cast<const uint4*>(row + span.head);
    uint4* o = reinterpret_cast<uint4*>(out + span.head);
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kThreads * kAhead) {
        uint4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j * kThreads < vecs) v[j] = __ldcs(q + i0 + j * kThreads);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            if (i >= vecs) break;
            float x[E::kN];
            E::unpack(v[j], x);
            const int in = hit - (span.head + i * E::kN);      // the label's place in this piece, if it is in it
            if ((unsigned)in < (unsigned)E::kN) {
#pragma unroll
                for (int c = 0; c < E::kN; ++c) x[c] = grad(x[c], c == in);
            } else {
#pragma unroll
                for (int c = 0; c < E::kN; ++c) x[c] = grad(x[c], false);
            }
            __stcs(o + i, E::pack(x));
        }
    }
    const int head = vecs > 0 ? span.head : 0;
    for (int i = threadIdx.x; i < V - vecs * E::kN; i += kThreads) {
        const int v = i < head ? i : vecs * E::kN + i;
        out[v] = E::put(grad(E::get(row[v]), v == hit));
    }
}

int check_logits(const char* fn, int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                 const void* labels) {
    if (dt != LORA_BF16 && dt != LORA_F32) return refuse(LORA_ERR_DTYPE, "unknown dtype");
    if (T < 0 || V <= 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0 and V > 0");
    if (T == 0) return LORA_OK;
    if (!logits || !labels) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": logits or labels is NULL");
    if (ld < V) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": rows of logits overlap (ld < V)");
    if (!is_aligned(logits, elem_size(dt)))
        return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": logits must be aligned to an element");
    return LORA_OK;
}

// The sequences inside [0, T), in increasing start order, none over another
int check_pairs(const char* fn, int32_t T, const lora_pair_t* pairs, int32_t n_pairs,
                Sequences<LORA_MAX_PAIRS>* out) {
    if (n_pairs < 0 || (n_pairs > 0 && !pairs))
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": pairs is NULL or their number negative");
    if (n_pairs > LORA_MAX_PAIRS)
        return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than " + std::to_string(LORA_MAX_PAIRS) + " pairs");
    struct Seq { int32_t start, end; int16_t id; };
    Seq s[2 * LORA_MAX_PAIRS];
    int n = 0;
    for (int32_t i = 0; i < n_pairs; ++i)
        for (int side = 0; side < 2; ++side) {
            const int32_t start = side ? pairs[i].rejected_start : pairs[i].chosen_start;
            const int32_t len = side ? pairs[i].rejected_len : pairs[i].chosen_len;
            if (start < 0 || len < 0 || (int64_t)start + len > T)
                return refuse(LORA_ERR_SEGMENTS, std::string(fn) + ": pair " + std::to_string(i) +
                                                     " leaves the batch's rows");
            if (len > 0) s[n++] = Seq{start, start + len, (int16_t)(2 * i + side)};
        }
    std::sort(s, s + n, [](const Seq& a, const Seq& b) { return a.start < b.start; });
    out->n = n;
    for (int i = 0; i < n; ++i) {
        if (i > 0 && s[i].start < s[i - 1].end)
            return refuse(LORA_ERR_SEGMENTS, std::string(fn) + ": sequences overlap at row " +
                                                 std::to_string(s[i].start));
        out->start[i] = s[i].start;
        out->end[i] = s[i].end;
        out->id[i] = s[i].id;
    }
    return LORA_OK;
}

// Threads per row: a warp for rows of up to four pieces a lane; for a launch of few long rows, which leaves SMs idle,
// 1024 (60 rows of 32000: 256 threads a row take 1.9 times as long); else kUsual.
template <class E, int kUsual, class Go>
cudaError_t by_row_size(int32_t T, int32_t V, Go go) {
    const int vecs = V / E::kN;
    if (vecs <= 128) return go(std::integral_constant<int, 32>());
    if (T <= 304 && vecs >= 1024) return go(std::integral_constant<int, 1024>());
    return go(std::integral_constant<int, kUsual>());
}

template <class E>
cudaError_t launch_logprob(int32_t T, int32_t V, const void* logits, int64_t ld, const int64_t* labels, float* logp,
                           float* lse, cudaStream_t st) {
    // 8 pieces ahead at 256 threads: 116 us for 4096 rows of 128256, 70 % of them counted (4 ahead: 123 us)
    return by_row_size<E, 256>(T, V, [&](auto threads) {
        constexpr int kThreads = decltype(threads)::value;
        return launch_pdl(logprob_kernel<E, kThreads, (kThreads == 256 ? 8 : 4)>, dim3(T), dim3(kThreads), 0, st, V,
                          static_cast<const typename E::T*>(logits), ld, labels, logp, lse);
    });
}

template <class E, int kPairs>
cudaError_t launch_dlogits(int32_t T, int32_t V, const void* logits, int64_t ld, const int64_t* labels,
                           const float* lse, const float* coef, const Sequences<kPairs>& seqs, const float* dloss,
                           float all, void* dlogits, int64_t ld_d, cudaStream_t st) {
    // 512 threads: 263 us for the same rows (256 threads: 270 us)
    return by_row_size<E, 512>(T, V, [&](auto threads) {
        constexpr int kThreads = decltype(threads)::value;
        return launch_pdl(dlogits_kernel<E, kThreads, 4, kPairs>, dim3(T), dim3(kThreads), 0, st, V,
                          static_cast<const typename E::T*>(logits), ld, labels, lse, coef, seqs, dloss, all,
                          static_cast<typename E::T*>(dlogits), ld_d);
    });
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_token_logprob(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                                  const int64_t* labels, float* logp, float* lse, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_token_logprob";
        const int rc = check_logits(fn, T, V, dt, logits, ld, labels);
        if (rc != LORA_OK || T == 0) return rc;
        if (!logp || !lse) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": logp or lse is NULL");
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        return enqueued(fn, dt == LORA_BF16 ? launch_logprob<Bf16>(T, V, logits, ld, labels, logp, lse, st)
                                            : launch_logprob<F32>(T, V, logits, ld, labels, logp, lse, st));
    });
}

extern "C" int lora_preference_forward(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                                       const int64_t* labels, const float* ref_logp, const lora_pair_t* pairs,
                                       int32_t n_pairs, float beta, float label_smoothing, float* loss,
                                       float* rewards, float* logp, float* lse, float* coef, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_preference_forward";
        int rc = check_logits(fn, T, V, dt, logits, ld, labels);
        if (rc != LORA_OK) return rc;
        if (!(beta > 0.f) || isinf(beta) || !(label_smoothing >= 0.f && label_smoothing < 0.5f))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": beta must be positive and finite, "
                                                                  "label_smoothing in [0, 0.5)");
        Sequences<LORA_MAX_PAIRS> seqs;
        rc = check_pairs(fn, T, pairs, n_pairs, &seqs);
        if (rc != LORA_OK) return rc;
        if (T > 0 && (!ref_logp || !logp || !lse))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": ref_logp, logp or lse is NULL");
        if (n_pairs > 0 && (!loss || !rewards || !coef))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": loss, rewards or coef is NULL");
        if (T == 0 && n_pairs == 0) return LORA_OK;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        cudaError_t e = cudaSuccess;
        if (T > 0)
            e = dt == LORA_BF16 ? launch_logprob<Bf16>(T, V, logits, ld, labels, logp, lse, st)
                                : launch_logprob<F32>(T, V, logits, ld, labels, logp, lse, st);
        if (e == cudaSuccess && n_pairs > 0) {
            auto go = [&](auto p) {
                constexpr int kPairs = sizeof(p.p) / sizeof(lora_pair_t);
                std::copy(pairs, pairs + n_pairs, p.p);      // the first n_pairs are read
                return launch_pdl(pair_loss_kernel<kPairs>, dim3(n_pairs), dim3(kPairThreads), 0, st, p, labels,
                                  static_cast<const float*>(logp), ref_logp, beta, label_smoothing, loss, rewards, coef);
            };
            e = n_pairs <= kFewPairs ? go(Pairs<kFewPairs>()) : go(Pairs<LORA_MAX_PAIRS>());
        }
        return enqueued(fn, e);
    });
}

extern "C" int lora_preference_backward(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                                        const int64_t* labels, const float* lse, const float* coef,
                                        const lora_pair_t* pairs, int32_t n_pairs, const float* dloss, void* dlogits,
                                        int64_t ld_d, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_preference_backward";
        int rc = check_logits(fn, T, V, dt, logits, ld, labels);
        if (rc != LORA_OK) return rc;
        Sequences<LORA_MAX_PAIRS> seqs;
        rc = check_pairs(fn, T, pairs, n_pairs, &seqs);
        if (rc != LORA_OK || T == 0) return rc;
        if (!lse || !dlogits || (n_pairs > 0 && !coef))
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": lse, coef or dlogits is NULL");
        if (ld_d < V) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": rows of dlogits overlap (ld_d < V)");
        if (!is_aligned(dlogits, elem_size(dt)))
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": dlogits must be aligned to an element");
        if (dlogits == logits && ld_d != ld)
            return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": in place, ld_d must be ld");
        const float all = n_pairs > 0 ? 1.f / (float)n_pairs : 0.f;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        auto go = [&](const auto& q) {
            return dt == LORA_BF16
                       ? launch_dlogits<Bf16>(T, V, logits, ld, labels, lse, coef, q, dloss, all, dlogits, ld_d, st)
                       : launch_dlogits<F32>(T, V, logits, ld, labels, lse, coef, q, dloss, all, dlogits, ld_d, st);
        };
        if (n_pairs > kFewPairs) return enqueued(fn, go(seqs));
        Sequences<kFewPairs> few;
        few.n = seqs.n;
        std::copy(seqs.start, seqs.start + seqs.n, few.start);
        std::copy(seqs.end, seqs.end + seqs.n, few.end);
        std::copy(seqs.id, seqs.id + seqs.n, few.id);
        return enqueued(fn, go(few));
    });
}
