// preference.cu -- the preference loss of a fine-tuning step (include/lora_preference.h), forward and backward.
//
// Forward: one pass over each counted row of logits with a running maximum and sum (the row's log-sum-exp), then a
// small kernel that adds up each pair's sequences in 64 bits, in a fixed order.  Backward: one pass that reads a
// row and writes its gradient.  Both passes move each logit once and are bounded by the memory rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <string>

#include "fp8.h"
#include "lora_preference.h"

namespace lora {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eHigh = 1.44268798828125f;        // log2(e) to 16 bits, and the rest of it
constexpr float kLog2eLow = (float)(1.4426950408889634 - (double)kLog2eHigh);
constexpr int kThreads = 256;

// 2^x; 0 for x = -infinity, results below the smallest normal number are 0
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <class T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class T>
struct Vec {                                   // 16 bytes of a row
    static constexpr int kN = 16 / sizeof(T);
    union {
        uint4 q;
        T e[kN];
    };
    __device__ __forceinline__ Vec() {}
};

// Rows start anywhere (a row of odd length moves the next one off a 16-byte boundary): elements [0, head) come
// before the first boundary, then `vecs` pieces of 16 bytes, then the rest.
template <class T>
struct RowSpan {
    int head, vecs;
    __device__ __forceinline__ RowSpan(const T* row, int V) {
        head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
        vecs = (V - head) / Vec<T>::kN;
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
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N]) {
        float c = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) c = fmaxf(c, x[i]);
        c = ceilf(c * kLog2e);
        if (c > n) {
            s *= weight(n, c);
            n = c;
        }
        const float off = n == -INFINITY ? 0.f : -n;
#pragma unroll
        for (int i = 0; i < N; ++i) s += exp2_fast(fmaf(x[i], kLog2eLow, fmaf(x[i], kLog2eHigh, off)));
    }
    // log of the sum, in 64 bits (once per row); NaN for a row without a finite logit
    __device__ __forceinline__ double log() const {
        return n == -INFINITY ? (double)NAN : (double)n * 0.6931471805599453 + ::log((double)s);
    }
};

template <class T>
__global__ void __launch_bounds__(kThreads) logprob_kernel(int32_t V, const T* __restrict__ logits, int64_t ld,
                                                           const int64_t* __restrict__ labels,
                                                           float* __restrict__ logp, float* __restrict__ lse) {
    const int64_t t = blockIdx.x;
    const int64_t label = labels[t];
    if (label < 0) {
        if (threadIdx.x == 0) logp[t] = lse[t] = 0.f;
        return;
    }
    const T* row = logits + t * ld;
    const RowSpan<T> span(row, V);
    const uint4* q = reinterpret_cast<const uint4*>(row + span.head);
    ExpSum a;
    for (int i = threadIdx.x; i < span.vecs; i += kThreads) {
        Vec<T> v;
        v.q = q[i];
        float x[Vec<T>::kN];
#pragma unroll
        for (int k = 0; k < Vec<T>::kN; ++k) x[k] = to_float(v.e[k]);
        a.add(x);
    }
    const int tail0 = span.head + span.vecs * Vec<T>::kN;
    if ((int)threadIdx.x < span.head) {
        const float x[1] = {to_float(row[threadIdx.x])};
        a.add(x);
    } else if (tail0 + (int)threadIdx.x - span.head < V) {
        const float x[1] = {to_float(row[tail0 + threadIdx.x - span.head])};
        a.add(x);
    }
    __shared__ float sn[kThreads / 32], ss[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float n2 = __shfl_xor_sync(0xffffffffu, a.n, o), s2 = __shfl_xor_sync(0xffffffffu, a.s, o);
        a.join(n2, s2);
    }
    if (threadIdx.x % 32 == 0) {
        sn[threadIdx.x / 32] = a.n;
        ss[threadIdx.x / 32] = a.s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) a.join(sn[w], ss[w]);
        const double z = a.log();
        lse[t] = (float)z;
        logp[t] = label < V ? (float)((double)to_float(row[label]) - z) : NAN;
    }
}

// Sequences in increasing start order (zero-length ones left out): `id` = 2 pair + (0 chosen, 1 rejected)
struct Sequences {
    int32_t n;
    int32_t start[2 * LORA_MAX_PAIRS], end[2 * LORA_MAX_PAIRS];
    int16_t id[2 * LORA_MAX_PAIRS];
};
struct Pairs {
    lora_pair_t p[LORA_MAX_PAIRS];
};

__device__ __forceinline__ int sequence_of(const Sequences& s, int t) {
    int lo = 0, hi = s.n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s.start[mid] <= t) lo = mid + 1; else hi = mid;
    }
    return (lo > 0 && t < s.end[lo - 1]) ? s.id[lo - 1] : -1;
}

__device__ double sum_block(double v, double* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
    __syncthreads();
    double r = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) r += sh[w];
    return r;
}

// One CTA per pair.  The differences lp - ref are small and their sums cancel: they are added up in 64 bits.
__global__ void __launch_bounds__(kThreads) pair_loss_kernel(const __grid_constant__ Pairs pairs,
                                                             const int64_t* __restrict__ labels,
                                                             const float* __restrict__ logp,
                                                             const float* __restrict__ ref, float beta, float eps,
                                                             float* __restrict__ loss, float* __restrict__ rewards,
                                                             float* __restrict__ coef) {
    __shared__ double sh[kThreads / 32];
    const lora_pair_t p = pairs.p[blockIdx.x];
    double d[2];
    for (int side = 0; side < 2; ++side) {
        const int64_t t0 = side ? p.rejected_start : p.chosen_start;
        const int64_t t1 = t0 + (side ? p.rejected_len : p.chosen_len);
        double v = 0.0;
        for (int64_t t = t0 + threadIdx.x; t < t1; t += kThreads)
            if (labels[t] >= 0) v += (double)logp[t] - (double)ref[t];
        d[side] = beta * sum_block(v, sh);
    }
    if (threadIdx.x != 0) return;
    const double m = d[0] - d[1];
    const double soft = log1p(exp(-fabs(m)));          // -log sig(m) = max(-m, 0) + log(1 + e^-|m|)
    const double sig = 1.0 / (1.0 + exp(-m));
    // a certain side (weight 0) does not meet the other's infinity
    const double miss = (1.0 - (double)eps) * (fmax(-m, 0.0) + soft);
    const double smooth = eps > 0.f ? (double)eps * (fmax(m, 0.0) + soft) : 0.0;
    loss[blockIdx.x] = isnan(m) ? NAN : (float)(miss + smooth);
    rewards[2 * blockIdx.x] = (float)d[0];
    rewards[2 * blockIdx.x + 1] = (float)d[1];
    // sig(-m) from its own exponential: 1 - sig(m) would lose it for large m
    const double k = (double)beta * ((double)eps * sig - (1.0 - (double)eps) / (1.0 + exp(m)));
    coef[2 * blockIdx.x] = (float)k;
    coef[2 * blockIdx.x + 1] = (float)-k;
}

template <class T>
__global__ void __launch_bounds__(kThreads) dlogits_kernel(int32_t V, const T* logits, int64_t ld,
                                                           const int64_t* __restrict__ labels,
                                                           const float* __restrict__ lse,
                                                           const float* __restrict__ coef,
                                                           const __grid_constant__ Sequences seqs,
                                                           const float* __restrict__ dloss, float dloss_all,
                                                           T* dlogits, int64_t ld_d) {
    const int64_t t = blockIdx.x;
    const int64_t label = labels[t];
    const int seq = label < 0 ? -1 : sequence_of(seqs, (int)t);
    const T* row = logits + t * ld;
    T* out = dlogits + t * ld_d;
    float k = 0.f, off = 0.f;
    if (seq >= 0) {
        k = coef[seq] * (dloss ? dloss[seq / 2] : dloss_all);
        if (label >= V) k = NAN;
        off = -lse[t] * kLog2e;
    }
    const int hit = label >= 0 && label < V ? (int)label : -1;
    auto grad = [&](float x, int v) {
        const float p = exp2_fast(fmaf(x, kLog2e, off));
        return k * ((v == hit ? 1.f : 0.f) - p);
    };
    const RowSpan<T> span(out, V);
    // both rows on the same 16-byte phase: whole pieces; else element by element
    const bool whole = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int head = span.head, vecs = (whole || seq < 0) ? span.vecs : 0;
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
        Vec<T> v;
        const int e0 = head + i * Vec<T>::kN;
        if (seq >= 0) {
            v.q = *reinterpret_cast<const uint4*>(row + e0);
#pragma unroll
            for (int j = 0; j < Vec<T>::kN; ++j) v.e[j] = from_float<T>(grad(to_float(v.e[j]), e0 + j));
        } else {
            v.q = make_uint4(0, 0, 0, 0);
        }
        *reinterpret_cast<uint4*>(out + e0) = v.q;
    }
    const int tail0 = vecs > 0 ? head + vecs * Vec<T>::kN : 0;
    if (vecs > 0 && (int)threadIdx.x < head)
        out[threadIdx.x] = from_float<T>(seq >= 0 ? grad(to_float(row[threadIdx.x]), threadIdx.x) : 0.f);
    for (int v = tail0 + threadIdx.x; v < V; v += kThreads)
        out[v] = from_float<T>(seq >= 0 ? grad(to_float(row[v]), v) : 0.f);
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
int check_pairs(const char* fn, int32_t T, const lora_pair_t* pairs, int32_t n_pairs, Sequences* out) {
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

void launch_logprob(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld, const int64_t* labels,
                    float* logp, float* lse, cudaStream_t st) {
    if (dt == LORA_BF16)
        logprob_kernel<<<T, kThreads, 0, st>>>(V, static_cast<const __nv_bfloat16*>(logits), ld, labels, logp, lse);
    else
        logprob_kernel<<<T, kThreads, 0, st>>>(V, static_cast<const float*>(logits), ld, labels, logp, lse);
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" int lora_token_logprob(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                                  const int64_t* labels, float* logp, float* lse, void* stream) {
    const char* fn = "lora_token_logprob";
    const int rc = check_logits(fn, T, V, dt, logits, ld, labels);
    if (rc != LORA_OK || T == 0) return rc;
    if (!logp || !lse) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": logp or lse is NULL");
    launch_logprob(T, V, dt, logits, ld, labels, logp, lse, static_cast<cudaStream_t>(stream));
    return launched(fn);
}

extern "C" int lora_preference_forward(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                                       const int64_t* labels, const float* ref_logp, const lora_pair_t* pairs,
                                       int32_t n_pairs, float beta, float label_smoothing, float* loss,
                                       float* rewards, float* logp, float* lse, float* coef, void* stream) {
    const char* fn = "lora_preference_forward";
    int rc = check_logits(fn, T, V, dt, logits, ld, labels);
    if (rc != LORA_OK) return rc;
    if (!(beta > 0.f) || isinf(beta) || !(label_smoothing >= 0.f && label_smoothing < 0.5f))
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": beta must be positive and finite, "
                                                              "label_smoothing in [0, 0.5)");
    Sequences seqs;
    rc = check_pairs(fn, T, pairs, n_pairs, &seqs);
    if (rc != LORA_OK) return rc;
    if (T > 0 && (!ref_logp || !logp || !lse))
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": ref_logp, logp or lse is NULL");
    if (n_pairs > 0 && (!loss || !rewards || !coef))
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": loss, rewards or coef is NULL");
    if (T == 0 && n_pairs == 0) return LORA_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T > 0) launch_logprob(T, V, dt, logits, ld, labels, logp, lse, st);
    if (n_pairs > 0) {
        Pairs p{};
        std::copy(pairs, pairs + n_pairs, p.p);
        pair_loss_kernel<<<n_pairs, kThreads, 0, st>>>(p, labels, logp, ref_logp, beta, label_smoothing, loss, rewards,
                                                       coef);
    }
    return launched(fn);
}

extern "C" int lora_preference_backward(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                                        const int64_t* labels, const float* lse, const float* coef,
                                        const lora_pair_t* pairs, int32_t n_pairs, const float* dloss, void* dlogits,
                                        int64_t ld_d, void* stream) {
    const char* fn = "lora_preference_backward";
    int rc = check_logits(fn, T, V, dt, logits, ld, labels);
    if (rc != LORA_OK) return rc;
    Sequences seqs;
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
    if (dt == LORA_BF16)
        dlogits_kernel<<<T, kThreads, 0, st>>>(V, static_cast<const __nv_bfloat16*>(logits), ld, labels, lse, coef,
                                               seqs, dloss, all, static_cast<__nv_bfloat16*>(dlogits), ld_d);
    else
        dlogits_kernel<<<T, kThreads, 0, st>>>(V, static_cast<const float*>(logits), ld, labels, lse, coef, seqs,
                                               dloss, all, static_cast<float*>(dlogits), ld_d);
    return launched(fn);
}
