// fp8.h -- the 8-bit block format (include/lora_fp8.h) on the device, and host checks shared by its entry points.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "lora_fp8.h"
#include "plan.h"

namespace lora {

constexpr int kQBlock = LORA_FP8_BLOCK;   // columns (and weight rows) that share a scale

// ------------------------------------------------------------------------------------------------------- device
// Scale of a block whose largest magnitude has the float bits `amax` (sign cleared), and its reciprocal: the smallest
// power of two s with amax <= 448 s.  448 = 1.75 * 2^8, so with amax = m 2^k the exponent is k - 8 for m <= 1.75 and
// k - 7 above; adding 0x1FFFFF to the bits carries into the exponent exactly when the mantissa exceeds 1.75.
// amax below 2^-100 counts as 2^-100 (no scale is zero).  Infinity or NaN: both NaN.
__device__ __forceinline__ float block_scale(uint32_t amax, float* inv) {
    const uint32_t b = max(amax, (127u - 100u) << 23);
    const uint32_t e = (b + 0x1FFFFFu) >> 23;
    const bool bad = amax >= 0x7F800000u;
    *inv = __uint_as_float(bad ? 0x7FC00000u : (262u - e) << 23);
    return __uint_as_float(bad ? 0x7FC00000u : (e - 8u) << 23);
}

// A block row is held by 16 neighbouring lanes, 8 elements each.
constexpr int kLanesPerBlock = kQBlock / 8;

__device__ __forceinline__ uint32_t abs_bits_max(const float (&v)[8]) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return a;
}
__device__ __forceinline__ uint32_t max_over_block(uint32_t a) {
#pragma unroll
    for (int o = kLanesPerBlock / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}
// codes of 8 values (inv: the reciprocal of their block's scale): one rounding each, since v * inv is exact
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * inv, v[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}
__device__ __forceinline__ void decode8(uint2 q, float s, float (&v)[8]) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * i] = f.x * s;
        v[2 * i + 1] = f.y * s;
    }
}

// 8 elements of a row in either element type
struct Row8Bf16 {
    uint4 q;
    static __device__ __forceinline__ const void* at(const void* p, int64_t i) { return static_cast<const __nv_bfloat16*>(p) + i; }
    static __device__ __forceinline__ void* at(void* p, int64_t i) { return static_cast<__nv_bfloat16*>(p) + i; }
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    }
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    // largest magnitude as float bits, NaN above all
    __device__ __forceinline__ uint32_t abs_max() const {
        const uint32_t w[4] = {q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu, q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu};
        const __nv_bfloat162* v = reinterpret_cast<const __nv_bfloat162*>(w);
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(v[0], v[1]), __hmax2_nan(v[2], v[3]));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
        return max(b << 16, b & 0xFFFF0000u);
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
struct Row8F32 {
    float4 a, b;
    static __device__ __forceinline__ const void* at(const void* p, int64_t i) { return static_cast<const float*>(p) + i; }
    static __device__ __forceinline__ void* at(void* p, int64_t i) { return static_cast<float*>(p) + i; }
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        a = s[0];
        b = s[1];
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ uint32_t abs_max() const {
        float v[8];
        get(v);
        return abs_bits_max(v);
    }
    static __device__ __forceinline__ void store(void* p, int64_t i, const float (&v)[8]) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// --------------------------------------------------------------------------------------------------------- host
inline int blocks_of(int64_t n) { return (int)((n + kQBlock - 1) / kQBlock); }
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int elem_size(lora_dtype_t dt) { return dt == LORA_BF16 ? 2 : 4; }

inline int refuse(int code, const std::string& msg) {
    set_last_error(msg.c_str());
    return code;
}
// A C entry's body: nothing it throws (host memory running out) leaves it
template <class Body>
auto guarded(Body body) -> decltype(body()) {
    try {
        return body();
    } catch (...) {
        set_last_error("out of host memory");
        return LORA_ERR_LIMIT;
    }
}

// Rows that a call takes: tiles are counted in 32 bits, past the last row by a tile's height at the most
constexpr int32_t kMaxRowsOfX = INT32_MAX - 1024;

// the return code of a call that launched, or failed to
inline int enqueued(const char* fn, cudaError_t e) {
    if (e == cudaSuccess) return LORA_OK;
    return refuse(LORA_ERR_CUDA, std::string(fn) + ": " + cudaGetErrorString(e));
}
// matrix argument: non-null, 16-byte aligned, rows at least `cols` long and a multiple of 16 bytes apart
inline int check_matrix(const char* fn, const char* name, const void* p, int64_t cols, int64_t ld, int esize) {
    if (!p) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " is NULL");
    if (ld < cols)
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": rows of " + name + " overlap (row distance " +
                                                std::to_string(ld) + " < " + std::to_string(cols) + ")");
    if (!is_aligned(p, 16) || (ld * esize) % 16 != 0)
        return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": " + name +
                                              " must be 16-byte aligned, its rows a multiple of 16 bytes apart");
    return LORA_OK;
}

// the quantizer behind lora_fp8_quantize (arguments checked); also lora_fp8_linear's first step
cudaError_t launch_quantize(int32_t T, int32_t K, lora_dtype_t dt, const void* x, int64_t ld_x, uint8_t* codes,
                            int64_t ld_codes, float* scales, cudaStream_t stream);

}  // namespace lora
