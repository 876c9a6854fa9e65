// fp8.cu -- the 8-bit block format: quantizers, and the MLP activation with its 8-bit checkpoint.
//
// Every kernel here moves each byte once and computes little per byte: the memory rate bounds them.  A block row (128
// columns of one row) belongs to 16 neighbouring lanes of 8 elements each, so a 16-bit row is read in 16-byte pieces,
// the block's largest magnitude is four shuffles away, and the codes leave in 8-byte pieces, 128 bytes per block.
#include <algorithm>
#include <type_traits>
#include <vector>

#include "fp8.h"
#include "tc_prims.h"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = kThreads / kLanesPerBlock;   // block rows that a CTA holds at a time

// A CTA takes `1 << log2_cols` neighbouring blocks of `kUnits >> log2_cols` rows at a time.
struct Shape {
    int32_t rows, cols;      // of the operand: rows, columns of one row (of one half, for gate|up)
    int32_t n_blocks;        // blocks of a row
    int32_t log2_cols;
};

// The width with the fewest idle lanes, the widest of equals: a row of 17 blocks taken 16 at a time would leave 15 of
// 32 slots empty.
Shape shape_of(int32_t rows, int32_t cols) {
    Shape s{rows, cols, blocks_of(cols), 0};
    int64_t best = 1ll << 62;
    for (int l = 4; l >= 0; --l) {
        const int64_t w = 1ll << l, slots = (s.n_blocks + w - 1) / w * w;
        if (slots < best) { best = slots; s.log2_cols = l; }
    }
    return s;
}
dim3 grid_of(const Shape& s, int rows_per_thread) {
    const int64_t rows_cta = (int64_t)(kUnits >> s.log2_cols) * rows_per_thread;
    const int w = 1 << s.log2_cols;
    return dim3((unsigned)((s.rows + rows_cta - 1) / rows_cta), (unsigned)((s.n_blocks + w - 1) / w));
}

// Row and column of this thread's i-th block row; rows of one thread lie kUnits >> log2_cols apart.
struct Place {
    int row0, row_step, col, block;
    bool in;
    __device__ __forceinline__ Place(const Shape& s, int rows_per_thread) {
        const int unit = threadIdx.x / kLanesPerBlock, lane = threadIdx.x % kLanesPerBlock;
        row_step = kUnits >> s.log2_cols;
        row0 = blockIdx.x * row_step * rows_per_thread + (unit >> s.log2_cols);
        block = (blockIdx.y << s.log2_cols) + (unit & ((1 << s.log2_cols) - 1));
        col = block * kQBlock + lane * 8;
        in = col < s.cols;
    }
};

// ---------------------------------------------------------------------------------------------------- quantizers
constexpr int kQuantRows = 2;      // rows a thread

template <class Row8>
__global__ void __launch_bounds__(kThreads) quantize_kernel(Shape s, const void* x, int64_t ld_x,
                                                            uint8_t* codes, int64_t ld_codes,
                                                            float* scales) {
    grid_dep_launch();     // a product may set itself up meanwhile
    grid_dep_wait();
    const Place p(s, kQuantRows);
    Row8 r[kQuantRows];
#pragma unroll
    for (int k = 0; k < kQuantRows; ++k) {
        const int row = p.row0 + k * p.row_step;
        r[k].zero();
        if (p.in && row < s.rows) r[k].load(x, row * ld_x + p.col);
    }
#pragma unroll
    for (int k = 0; k < kQuantRows; ++k) {
        const int row = p.row0 + k * p.row_step;
        float v[8], inv;
        const float sc = block_scale(max_over_block(r[k].abs_max()), &inv);
        if (!p.in || row >= s.rows) continue;
        r[k].get(v);
        *reinterpret_cast<uint2*>(codes + row * ld_codes + p.col) = encode8(v, inv);
        if (threadIdx.x % kLanesPerBlock == 0) scales[(int64_t)row * s.n_blocks + p.block] = sc;
    }
}

// One 128 x 128 block of a weight per CTA; its rows stay in registers (8 per thread) between the two uses.
template <class Row8>
__global__ void __launch_bounds__(kThreads) quantize_weight_kernel(int32_t N, int32_t K, const void* __restrict__ W,
                                                                   int64_t ld_w, uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
    constexpr int kRows = kQBlock / kUnits;
    __shared__ uint32_t warp_max[kThreads / 32];
    const int unit = threadIdx.x / kLanesPerBlock;
    const int col = blockIdx.x * kQBlock + (threadIdx.x % kLanesPerBlock) * 8;
    Row8 r[kRows];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = blockIdx.y * kQBlock + i * kUnits + unit;
        r[i].zero();
        if (row < N && col < K) r[i].load(W, row * ld_w + col);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) a = max(a, r[i].abs_max());
    a = __reduce_max_sync(0xffffffffu, a);
    if (threadIdx.x % 32 == 0) warp_max[threadIdx.x / 32] = a;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) a = max(a, warp_max[w]);
    float inv;
    const float sc = block_scale(a, &inv);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = blockIdx.y * kQBlock + i * kUnits + unit;
        float v[8];
        r[i].get(v);
        if (row < N && col < K) *reinterpret_cast<uint2*>(codes + (int64_t)row * K + col) = encode8(v, inv);
    }
    if (threadIdx.x == 0) scales[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = sc;
}

// -------------------------------------------------------------------------------------------------------- swiglu
// Fine-tuning segments in increasing start order: rows [start, start + len) go to checkpoint rows from `ck`.
struct TrainRanges {
    int32_t n;
    int32_t start[kMaxTrainSegs], len[kMaxTrainSegs], ck[kMaxTrainSegs];
};
// checkpoint row of a row, -1 if it is kept nowhere
__device__ __forceinline__ int checkpoint_row(const TrainRanges& t, int row) {
    int lo = 0, hi = t.n;                      // the last range that starts at or before the row is lo - 1
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (t.start[mid] <= row) lo = mid + 1; else hi = mid;
    }
    if (lo == 0 || row - t.start[lo - 1] >= t.len[lo - 1]) return -1;
    return t.ck[lo - 1] + row - t.start[lo - 1];
}

// sig(g) = 1 / (1 + e^-g) and sig(-g).
// kFull, where the result leaves as float32: from e^-|g|, which cannot overflow, by the full exponential and quotient; each
// is a few units of 2^-24 off.
// Else the result is rounded to 16 bits or 8: the fast forms, with numerator and denominator scaled by 2^-32, so that the
// denominator passes 2^126, where the fast reciprocal ends, only for gates below -109, whose sigmoid float32 cannot hold.
// e^-g is the square of e^(-g / 2), which stays finite there; it is off by |g| 2^-24 and a few units, 2^-17 where the
// sigmoid is next to nothing.  (Shifting the exponent by 32 instead rounds it at 2^-19 for every gate.)  sig(-g) is
// 1 - sig(g), 2^-24 off; it is added to 1 after a product with g.  (With the full forms the 16-bit forward of 8192 x 14336
// with 2048 rows kept takes 124 us for 113, float32 to 8 bits 188 for 163; float32 to float32 takes 211 with either.)
struct Sigmoid {
    float pos, neg;
};
template <bool kFull>
__device__ __forceinline__ Sigmoid sigmoid(float g) {
    if constexpr (kFull) {
        const float e = expf(-fabsf(g)), large = 1.f / (1.f + e), small = e * large;
        return g < 0.f ? Sigmoid{small, large} : Sigmoid{large, small};
    } else {
        constexpr float kHalfLog2e = 0.7213475204444817f, kUnit = 0x1p-32f;
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -kHalfLog2e));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e * kUnit, e, kUnit)));
        const float sig = kUnit * r;
        return Sigmoid{sig, 1.f - sig};
    }
}

// Two rows a thread: 64 bytes in flight in each.  16 bits, 8192 x 14336 with 2048 rows kept: 113 us, the memory rate (one
// row a thread: 133 us; two with 58 registers, four CTAs to an SM for five: 121 us).
constexpr int kForwardRows = 2;

template <class Row8, bool H8>
__global__ void __launch_bounds__(kThreads, std::is_same<Row8, Row8Bf16>::value && !H8 ? 5 : 4) swiglu_forward_kernel(
    Shape s, const void* gu, int64_t ld_gu, void* h, int64_t ld_h,
    float* h_scales, uint8_t* ck_codes, float* ck_scales,
    const __grid_constant__ TrainRanges train) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr bool kFull = std::is_same<Row8, Row8F32>::value && !H8;
    const Place p(s, kForwardRows);
    const bool lead = threadIdx.x % kLanesPerBlock == 0;
    Row8 rg[kForwardRows], ru[kForwardRows];
#pragma unroll
    for (int k = 0; k < kForwardRows; ++k) {
        const int row = p.row0 + k * p.row_step;
        rg[k].zero();
        ru[k].zero();
        if (p.in && row < s.rows) {
            rg[k].load(gu, row * ld_gu + p.col);
            ru[k].load(gu, row * ld_gu + s.cols + p.col);
        }
    }
#pragma unroll
    for (int k = 0; k < kForwardRows; ++k) {
        const int row = p.row0 + k * p.row_step;
        const bool in = p.in && row < s.rows;
        float g[8], u[8], v[8];
        rg[k].get(g);
        ru[k].get(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = g[i] * sigmoid<kFull>(g[i]).pos * u[i];
        if constexpr (H8) {
            float inv;
            const float sc = block_scale(max_over_block(abs_bits_max(v)), &inv);
            if (in) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(h) + row * ld_h + p.col) = encode8(v, inv);
                if (lead) h_scales[(int64_t)row * s.n_blocks + p.block] = sc;
            }
        } else {
            if (in) Row8::store(h, row * ld_h + p.col, v);
        }
        const int ck = (train.n > 0 && row < s.rows) ? checkpoint_row(train, row) : -1;
        if (!__any_sync(0xffffffffu, ck >= 0)) continue;
        float inv_g, inv_u;
        const float sg = block_scale(max_over_block(rg[k].abs_max()), &inv_g);
        const float su = block_scale(max_over_block(ru[k].abs_max()), &inv_u);
        if (!in || ck < 0) continue;
        uint8_t* c = ck_codes + (int64_t)ck * 2 * s.cols + p.col;
        *reinterpret_cast<uint2*>(c) = encode8(g, inv_g);
        *reinterpret_cast<uint2*>(c + s.cols) = encode8(u, inv_u);
        if (lead) {
            float* z = ck_scales + (int64_t)ck * 2 * s.n_blocks + p.block;
            z[0] = sg;
            z[s.n_blocks] = su;
        }
    }
}

// Eight CTAs to an SM keep enough reads in flight, which takes 32 registers a thread; the full forms of float32 need 40, and
// gain from them (2048 x 14336: 63 us, 64 with the fast forms and 32).
template <class Row8, bool D8>
__global__ void __launch_bounds__(kThreads, std::is_same<Row8, Row8F32>::value && !D8 ? 6 : 8) swiglu_backward_kernel(
    Shape s, const uint8_t* ck_codes, const float* ck_scales, const void* dh, int64_t ld_dh, void* dgu, int64_t ld_dgu,
    float* dgu_scales) {
    grid_dep_launch();
    grid_dep_wait();
    constexpr bool kFull = std::is_same<Row8, Row8F32>::value && !D8;
    const Place p(s, 1);
    const int row = p.row0;
    const bool in = p.in && row < s.rows;
    Row8 rd;
    rd.zero();
    uint2 qg = make_uint2(0, 0), qu = qg;
    float sg = 0.f, su = 0.f;
    if (in) {
        const uint8_t* c = ck_codes + (int64_t)row * 2 * s.cols + p.col;
        const float* z = ck_scales + (int64_t)row * 2 * s.n_blocks + p.block;
        qg = *reinterpret_cast<const uint2*>(c);
        qu = *reinterpret_cast<const uint2*>(c + s.cols);
        sg = z[0];
        su = z[s.n_blocks];
        rd.load(dh, row * ld_dh + p.col);
    }
    float g[8], u[8], d[8];
    decode8(qg, sg, g);
    decode8(qu, su, u);
    rd.get(d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const Sigmoid sig = sigmoid<kFull>(g[i]);
        const float dsig = d[i] * sig.pos;
        d[i] = dsig * u[i] * (1.f + g[i] * sig.neg);       // gate's gradient
        u[i] = dsig * g[i];                                // up's
    }
    if constexpr (D8) {
        float inv_g, inv_u;
        const float zg = block_scale(max_over_block(abs_bits_max(d)), &inv_g);
        const float zu = block_scale(max_over_block(abs_bits_max(u)), &inv_u);
        if (!in) return;
        uint8_t* c = static_cast<uint8_t*>(dgu) + row * ld_dgu + p.col;
        *reinterpret_cast<uint2*>(c) = encode8(d, inv_g);
        *reinterpret_cast<uint2*>(c + s.cols) = encode8(u, inv_u);
        if (threadIdx.x % kLanesPerBlock == 0) {
            float* z = dgu_scales + (int64_t)row * 2 * s.n_blocks + p.block;
            z[0] = zg;
            z[s.n_blocks] = zu;
        }
    } else if (in) {
        Row8::store(dgu, row * ld_dgu + p.col, d);
        Row8::store(dgu, row * ld_dgu + s.cols + p.col, u);
    }
}

// Rows of at most this many columns: blocks of a row are spread over the grid's second dimension (< 65536)
constexpr int32_t kMaxCols = 1 << 22;

bool known_dtype(lora_dtype_t dt) { return dt == LORA_BF16 || dt == LORA_F32; }

// The fine-tuning segments of a table that covers [0, T) once, in increasing start order; their rows, or an error
int64_t train_ranges(const char* fn, int32_t T, const lora_segment_t* segs, int32_t n_segs, TrainRanges* out) {
    if (n_segs < 0 || (n_segs > 0 && !segs))
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": segment table is NULL or its size negative");
    std::vector<lora_segment_t> copy;          // in increasing start order, made only if the table is not
    const auto before = [](const lora_segment_t& a, const lora_segment_t& b) {
        return a.start != b.start ? a.start < b.start : a.len < b.len;      // empty ones first
    };
    if (!std::is_sorted(segs, segs + n_segs, before)) {
        copy.assign(segs, segs + n_segs);
        std::sort(copy.begin(), copy.end(), before);
        segs = copy.data();
    }
    int64_t at = 0;
    int32_t rows = 0;
    out->n = 0;
    for (int32_t i = 0; i < n_segs; ++i) {
        const lora_segment_t& q = segs[i];
        if (q.len < 0 || q.start < 0)
            return refuse(LORA_ERR_SEGMENTS, std::string(fn) + ": negative segment start or length");
        if (q.len == 0) continue;
        if (q.start != at)
            return refuse(LORA_ERR_SEGMENTS, std::string(fn) + ": segments overlap or leave a gap at token " +
                                                 std::to_string(std::min<int64_t>(at, q.start)));
        at += q.len;
        if (at > T) break;
        if (!q.is_train) continue;
        if (out->n == kMaxTrainSegs)
            return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 48 fine-tuning segments");
        out->start[out->n] = q.start;
        out->len[out->n] = q.len;
        out->ck[out->n++] = rows;
        rows += q.len;
    }
    if (at != T) return refuse(LORA_ERR_SEGMENTS, std::string(fn) + ": segments do not cover [0, T)");
    return rows;
}

}  // namespace

cudaError_t launch_quantize(int32_t T, int32_t K, lora_dtype_t dt, const void* x, int64_t ld_x, uint8_t* codes,
                            int64_t ld_codes, float* scales, cudaStream_t stream) {
    const Shape s = shape_of(T, K);
    return launch_pdl(dt == LORA_BF16 ? quantize_kernel<Row8Bf16> : quantize_kernel<Row8F32>, grid_of(s, kQuantRows),
                      dim3(kThreads), 0, stream, s, x, ld_x, codes, ld_codes, scales);
}

}  // namespace lora

using namespace lora;

extern "C" int lora_fp8_quantize(int32_t T, int32_t K, lora_dtype_t dt, const void* x, int64_t ld_x, void* codes,
                                 int64_t ld_codes, float* scales, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_fp8_quantize";
        if (!known_dtype(dt)) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        if (T < 0 || K <= 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0 and K > 0");
        if (K > kMaxCols) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 2^22 columns");
        if (T > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": T above 2^31 - 1025");
        if (K % 16 != 0) return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": K must be a multiple of 16");
        if (T == 0) return LORA_OK;
        int rc = check_matrix(fn, "x", x, K, ld_x, elem_size(dt));
        if (rc == LORA_OK) rc = check_matrix(fn, "codes", codes, K, ld_codes, 1);
        if (rc != LORA_OK) return rc;
        if (!scales) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": scales is NULL");
        return enqueued(fn, launch_quantize(T, K, dt, x, ld_x, static_cast<uint8_t*>(codes), ld_codes, scales,
                                            static_cast<cudaStream_t>(stream)));
    });
}

extern "C" int lora_fp8_quantize_weight(int32_t N, int32_t K, lora_dtype_t dt, const void* W, int64_t ld_w,
                                        void* codes, float* scales, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_fp8_quantize_weight";
        if (!known_dtype(dt)) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        if (N <= 0 || K <= 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": N and K must be > 0");
        if (K % 16 != 0) return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": K must be a multiple of 16");
        int rc = check_matrix(fn, "W", W, K, ld_w, elem_size(dt));
        if (rc == LORA_OK) rc = check_matrix(fn, "codes", codes, K, K, 1);
        if (rc != LORA_OK) return rc;
        if (!scales) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": scales is NULL");
        if (blocks_of(N) > 65535) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 65535 * 128 weight rows");
        const dim3 grid(blocks_of(K), blocks_of(N));
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        if (dt == LORA_BF16)
            quantize_weight_kernel<Row8Bf16>
                <<<grid, kThreads, 0, st>>>(N, K, W, ld_w, static_cast<uint8_t*>(codes), scales);
        else
            quantize_weight_kernel<Row8F32>
                <<<grid, kThreads, 0, st>>>(N, K, W, ld_w, static_cast<uint8_t*>(codes), scales);
        return enqueued(fn, cudaGetLastError());
    });
}

extern "C" int64_t lora_checkpoint_rows(int32_t T, const lora_segment_t* segs, int32_t n_segs) {
    return guarded([&]() -> int64_t {
        TrainRanges t;
        if (T < 0) return refuse(LORA_ERR_INVALID_ARG, "lora_checkpoint_rows: T must be >= 0");
        return train_ranges("lora_checkpoint_rows", T, segs, n_segs, &t);
    });
}

extern "C" int lora_swiglu_forward(int32_t T, int32_t I, lora_dtype_t dt, const void* gu, int64_t ld_gu,
                                   const lora_segment_t* segs, int32_t n_segs, void* h, int64_t ld_h, float* h_scales,
                                   void* ck_codes, float* ck_scales, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_swiglu_forward";
        if (!known_dtype(dt)) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        if (T < 0 || I <= 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0 and I > 0");
        if (I > kMaxCols) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 2^22 columns");
        if (T > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": T above 2^31 - 1025");
        if (I % 8 != 0) return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": I must be a multiple of 8");
        TrainRanges train;
        train.n = 0;
        if (ck_codes || n_segs != 0) {
            const int64_t rows = train_ranges(fn, T, segs, n_segs, &train);
            if (rows < 0) return (int)rows;
        }
        if (!ck_codes) train.n = 0;
        if (T == 0) return LORA_OK;
        int rc = check_matrix(fn, "gu", gu, 2 * (int64_t)I, ld_gu, elem_size(dt));
        if (rc == LORA_OK) rc = check_matrix(fn, "h", h, I, ld_h, h_scales ? 1 : elem_size(dt));
        if (rc == LORA_OK && train.n > 0) rc = check_matrix(fn, "ck_codes", ck_codes, 2 * (int64_t)I, 2 * (int64_t)I, 1);
        if (rc != LORA_OK) return rc;
        if (train.n > 0 && !ck_scales) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": ck_scales is NULL");
        const Shape s = shape_of(T, I);
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, grid_of(s, kForwardRows), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), s, gu, ld_gu, h,
                              ld_h, h_scales, static_cast<uint8_t*>(ck_codes), ck_scales, train);
        };
        if (dt == LORA_BF16)
            return enqueued(fn, h_scales ? go(swiglu_forward_kernel<Row8Bf16, true>)
                                         : go(swiglu_forward_kernel<Row8Bf16, false>));
        return enqueued(fn, h_scales ? go(swiglu_forward_kernel<Row8F32, true>)
                                     : go(swiglu_forward_kernel<Row8F32, false>));
    });
}

extern "C" int lora_swiglu_backward(int32_t R, int32_t I, lora_dtype_t dt, const void* ck_codes,
                                    const float* ck_scales, const void* dh, int64_t ld_dh, void* dgu, int64_t ld_dgu,
                                    float* dgu_scales, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_swiglu_backward";
        if (!known_dtype(dt)) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        if (R < 0 || I <= 0) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": R must be >= 0 and I > 0");
        if (I > kMaxCols) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": more than 2^22 columns");
        if (R > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": R above 2^31 - 1025");
        if (I % 8 != 0) return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": I must be a multiple of 8");
        if (dgu_scales && I % kQBlock != 0)
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": I must be a multiple of 128 for a gradient in 8 bits");
        if (R == 0) return LORA_OK;
        int rc = check_matrix(fn, "ck_codes", ck_codes, 2 * (int64_t)I, 2 * (int64_t)I, 1);
        if (rc == LORA_OK) rc = check_matrix(fn, "dh", dh, I, ld_dh, elem_size(dt));
        if (rc == LORA_OK) rc = check_matrix(fn, "dgu", dgu, 2 * (int64_t)I, ld_dgu, dgu_scales ? 1 : elem_size(dt));
        if (rc != LORA_OK) return rc;
        if (!ck_scales) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": ck_scales is NULL");
        const Shape s = shape_of(R, I);
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, grid_of(s, 1), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), s,
                              static_cast<const uint8_t*>(ck_codes), ck_scales, dh, ld_dh, dgu, ld_dgu, dgu_scales);
        };
        if (dt == LORA_BF16)
            return enqueued(fn, dgu_scales ? go(swiglu_backward_kernel<Row8Bf16, true>)
                                           : go(swiglu_backward_kernel<Row8Bf16, false>));
        return enqueued(fn, dgu_scales ? go(swiglu_backward_kernel<Row8F32, true>)
                                       : go(swiglu_backward_kernel<Row8F32, false>));
    });
}
