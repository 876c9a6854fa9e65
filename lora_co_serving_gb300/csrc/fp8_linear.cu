// fp8_linear.cu -- products with a frozen weight in 8 bits (include/lora_fp8.h):
//     y[t,n] = sum_b sx[t,b] sw[n/128,b] sum_{k in block b} qx[t,k] qw[n,k]
#include <string>

#include "fp8.h"

namespace lora {
namespace {

constexpr int kTile = 64;      // rows of x and of w per CTA
constexpr int kStep = 32;      // columns staged at a time (a quarter of a block)

// Each thread holds 4 x 4 outputs; a block's products are summed first and then scaled once.
__global__ void __launch_bounds__(256) linear_kernel(int32_t T, int32_t K, int32_t N, const uint8_t* __restrict__ x,
                                                     int64_t ld_x, const float* __restrict__ xs,
                                                     const uint8_t* __restrict__ w, const float* __restrict__ ws,
                                                     __nv_bfloat16* __restrict__ y, int64_t ld_y) {
    __shared__ float sx[kStep][kTile + 4], sw[kStep][kTile + 4];
    const int t0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, nb = (K + kQBlock - 1) / kQBlock;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int b = 0; b < nb; ++b) {
        float part[4][4] = {};
        for (int k0 = b * kQBlock; k0 < min(K, (b + 1) * kQBlock); k0 += kStep) {
            const int r = threadIdx.x / 4, c = (threadIdx.x % 4) * 8;
            float v[8], u[8];
            const bool in = k0 + c < K;
            decode8(in && t0 + r < T ? *reinterpret_cast<const uint2*>(x + (t0 + r) * ld_x + k0 + c) : make_uint2(0, 0),
                    1.f, v);
            decode8(in && n0 + r < N ? *reinterpret_cast<const uint2*>(w + (int64_t)(n0 + r) * K + k0 + c)
                                     : make_uint2(0, 0),
                    1.f, u);
            __syncthreads();
            for (int i = 0; i < 8; ++i) {
                sx[c + i][r] = v[i];
                sw[c + i][r] = u[i];
            }
            __syncthreads();
            for (int k = 0; k < kStep; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] += sx[k][ty * 4 + i] * sw[k][tx * 4 + j];
        }
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + ty * 4 + i;
            const float s = t < T ? xs[(int64_t)t * nb + b] * ws[(int64_t)(n0 / kQBlock) * nb + b] : 0.f;
            for (int j = 0; j < 4; ++j) acc[i][j] += s * part[i][j];
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (t < T && n < N) y[t * ld_y + n] = __float2bfloat16_rn(acc[i][j]);
        }
}

// Workspace: the status word, then x's codes and scales if x is quantized on the way
struct Scratch {
    size_t status = 0, codes = 0, scales = 0, end = 0;
};
Scratch layout_of(int32_t T, int32_t K, bool x_fp8) {
    auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
    Scratch L;
    L.codes = 256;
    L.scales = L.codes + (x_fp8 ? 0 : al((size_t)T * K));
    L.end = L.scales + (x_fp8 ? 0 : al((size_t)T * blocks_of(K) * sizeof(float)));
    return L;
}

int check_sizes(const char* fn, int32_t T, int32_t K, int32_t N) {
    if (T < 0 || K <= 0 || N <= 0)
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0, K and N > 0");
    if (K % 16 != 0 || N % 8 != 0)
        return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": K must be a multiple of 16 and N of 8");
    if (K > (1 << 22)) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": K above 2^22");
    return LORA_OK;
}

}  // namespace
}  // namespace lora

using namespace lora;

extern "C" size_t lora_fp8_workspace_size(int32_t T, int32_t K, int32_t N, int32_t x_fp8) {
    if (check_sizes("lora_fp8_workspace_size", T, K, N) != LORA_OK) return 0;
    return layout_of(T, K, x_fp8 != 0).end;
}

extern "C" int lora_fp8_linear(int32_t T, int32_t K, int32_t N, lora_dtype_t dt, const void* x, int64_t ld_x,
                               const float* x_scales, const void* w, const float* w_scales, void* y, int64_t ld_y,
                               void* workspace, size_t ws_bytes, void* stream) {
    const char* fn = "lora_fp8_linear";
    if (!x_scales && dt != LORA_BF16 && dt != LORA_F32) return refuse(LORA_ERR_DTYPE, "unknown dtype");
    int rc = check_sizes(fn, T, K, N);
    if (rc != LORA_OK || T == 0) return rc;
    rc = check_matrix(fn, "x", x, K, ld_x, x_scales ? 1 : elem_size(dt));
    if (rc == LORA_OK) rc = check_matrix(fn, "w", w, K, K, 1);
    if (rc == LORA_OK) rc = check_matrix(fn, "y", y, N, ld_y, 2);
    if (rc != LORA_OK) return rc;
    if (!w_scales) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": w_scales is NULL");
    const Scratch L = layout_of(T, K, x_scales != nullptr);
    if (!workspace) return refuse(LORA_ERR_WORKSPACE, "workspace is NULL");
    if (!is_aligned(workspace, 256)) return refuse(LORA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < L.end)
        return refuse(LORA_ERR_WORKSPACE, "workspace too small: need " + std::to_string(L.end) + " bytes, got " +
                                              std::to_string(ws_bytes));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaError_t e = cudaMemsetAsync(ws, 0, 256, st);
    if (e != cudaSuccess) return refuse(LORA_ERR_CUDA, std::string(fn) + ": " + cudaGetErrorString(e));
    if (!x_scales) {
        float* sc = reinterpret_cast<float*>(ws + L.scales);
        launch_quantize(T, K, dt, x, ld_x, ws + L.codes, K, sc, st);
        x = ws + L.codes;
        ld_x = K;
        x_scales = sc;
    }
    const dim3 grid((N + kTile - 1) / kTile, (T + kTile - 1) / kTile);
    linear_kernel<<<grid, 256, 0, st>>>(T, K, N, static_cast<const uint8_t*>(x), ld_x, x_scales,
                                        static_cast<const uint8_t*>(w), w_scales, static_cast<__nv_bfloat16*>(y), ld_y);
    return launched(fn);
}
