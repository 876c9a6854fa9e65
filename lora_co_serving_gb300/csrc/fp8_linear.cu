// fp8_linear.cu -- products with a frozen weight in 8 bits (include/lora_fp8.h):
//     y[t,n] = sum_b sx[t,b] sw[n/128,b] sum_{k in block b} qx[t,k] qw[n,k]
//
// tcgen05.mma.kind::f8f6f4 multiplies the codes; a block's sum starts afresh in a TMEM accumulator and is then read
// back, scaled and added to sums that stay in registers (a scale changes every 128 columns, and the accumulators of
// the tensor cores cannot be rescaled in place).  Two accumulators alternate, so the MMAs of one block run while the
// last block's sums are scaled.
#include <cuda.h>

#include <algorithm>
#include <mutex>
#include <string>
#include <type_traits>
#include <vector>

#include "fp8.h"
#include "tc_kernel.h"
#include "tc_prims.h"

namespace lora {
namespace {

// The wait without a call: a kernel that calls a function cannot move registers between its warps (setmaxnreg)
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    return mbar_try_wait(bar, parity) || wait_phase_loop(bar, parity, abort_flag, status, 0);
}

// Two waits whose first tests are under way together: a test takes about 80 cycles, on the chain of every block that is
// issued (500 x 4096 x 4096 10.8 us so, 11.0 us one after the other; 256 x 4096 x 28672 33.7 and 33.9)
__device__ __forceinline__ void wait_both(uint32_t bar, uint32_t parity, uint32_t bar2, uint32_t parity2,
                                          volatile int* abort_flag, int32_t* status) {
    const bool ok = mbar_try_wait(bar, parity), ok2 = mbar_try_wait(bar2, parity2);
    if (!ok) wait_phase_loop(bar, parity, abort_flag, status, 0);
    if (!ok2) wait_phase_loop(bar2, parity2, abort_flag, status, 0);
}

// After a time-out: waits, with a limit of its own, for the loads of the last `stages` of `used` stages, so that none
// lands in the shared memory of the SM's next CTA.
__device__ __forceinline__ void drain_loads(uint32_t full, uint32_t used, int stages) {
    const uint64_t t0 = global_timer(), limit = g_wait_limit_ns;
    for (uint32_t u = used > (uint32_t)stages ? used - stages : 0; u < used; ++u)
        while (!mbar_try_wait(full + u % stages * 8, (u / stages) & 1u))
            if (global_timer() - t0 > limit) return;
}

template <int kStages>
struct StageRing {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
    }
};
// The last commits arrive on the stages' barriers (`empty`): none may be under way when the CTA ends and its shared memory
// goes to another.  `ring`: after the last load.
template <int kStages>
__device__ __forceinline__ void await_commits(StageRing<kStages> ring, uint32_t empty, volatile int* abort_flag,
                                              int32_t* status) {
    for (int s = 0; s < kStages; ++s, ring.next())
        if (!wait_here(empty + ring.stage * 8, ring.phase ^ 1u, abort_flag, status)) return;
}

// kind::f8f6f4: e4m3 A and B, fp32 accumulator, both operands K-major
__host__ __device__ constexpr uint32_t instr_desc_e4m3(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// (a.lo, a.hi) += (d0, d1) * (s.lo, s.hi).  volatile: d comes from a TMEM read and must stay behind its wait
__device__ __forceinline__ void fma2(uint64_t& a, uint32_t d0, uint32_t d1, uint64_t s) {
    asm volatile("{\n\t.reg .b64 d;\n\t"
        "mov.b64 d, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, d, %3, %0;\n\t}"
        : "+l"(a)
        : "r"(d0), "r"(d1), "l"(s));
}
__device__ __forceinline__ uint64_t both(float s) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(__float_as_uint(s)));
    return r;
}
__device__ __forceinline__ uint64_t two(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(__float_as_uint(lo)), "r"(__float_as_uint(hi)));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t a) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(a));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}

// =============================================================================================================
// Many rows: one CTA's tile is 128 rows of x by 256 outputs (rows of w), or by 128.
//
// The CTA loads its rows of x and of w, 48 KB a block for 128 * 256 * 128 products; an accumulator goes to and fro
// between the issuing warp and the adding warps once per block.
//
// What bounds it: a block's MMAs are 512 cycles of tensor work; its 48 KB are written to shared memory once and read
// once, 750 cycles at 128 bytes a cycle; scaling and adding takes an accumulator about 550 cycles, of which 256 are its
// 128 x 256 multiply-adds, and handing it over and back comes on top.  Two accumulators hide part of that.
// 8192 x 8192 x 28672 takes 1.455 ms (2640 TFLOP/s) in runs of a few milliseconds, at 2.07 GHz; longer ones meet the power
// limit, which lowers the clock: 2048 x 28672 x 8192 takes 336 us at first and 373 us, at 1.63 GHz, when it runs for half a
// second.
//
// Neighbouring CTAs load the same rows of w, each for itself, from L2.
//
// 384 threads: warp 0 loads (TMA), warp 1 issues, warps 4..11 scale and add: each thread has one row of x and 128
// outputs, which are one block of w's rows, so a block's 128 sums share one scale, sx[row] * sw[block].  The CTA
// starts with 168 registers a thread (64512 in all); the first warpgroup gives up 96 of them and the adding warps,
// whose 128 sums must not spill, take 48 more: 128 * 72 + 256 * 216 = 64512.
// =============================================================================================================
constexpr int kOperandBytes = 128 * kQBlock;             // 128 rows of x or w, one block of columns
constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr int kAddWarps = 8;
constexpr int kPieceBytes = 32 * 32 * 2;                 // an adding warp's 32 rows by 32 outputs on their way out
constexpr int kScaleSlots = 16;                          // blocks whose scales are at hand (see TileCfg)
constexpr int kScaleFloats = 132;                        // 128 rows of x, up to two blocks of w's rows
constexpr int kGroupRows = 4096;                         // rows of x that share a sweep over w (see tile_at)

// The shapes: a tile is 128 rows of x by kPN outputs.  256 moves and reads the least per product; 128 has twice the tiles,
// for products whose tiles of 256 leave SMs idle.  spread_of() weighs them.
template <int kPN_>
struct TileCfg {
    static constexpr int kPN = kPN_;
    static constexpr int kWBytes = kPN * kQBlock;        // the tile's rows of w
    // What passes the barriers at a time: one block, or two of 128 outputs, whose MMAs take 256 cycles each: issuing a
    // block (two barrier tests, four MMAs, two commits: about 400 cycles) would take longer.  500 x 4096 x 4096 takes
    // 10.8 us so, 12.1 us a block at a time (300 x 5120 x 5120: 13.6 and 14.4; 256 x 4096 x 28672: 33.7 and 32.9).
    static constexpr int kStep = 256 / kPN;
    static constexpr int kBlockBytes = kOperandBytes + kWBytes, kStageBytes = kStep * kBlockBytes;
    static constexpr int kStages = kPN == 256 ? 4 : 3;
    static constexpr int kAccCols = kStep * kPN;
    static constexpr int kCols = kPN / 2;                // outputs of an adding thread
    static constexpr int kIssueRegs = kPN == 256 ? 72 : 104, kAddRegs = kPN == 256 ? 216 : 200;
    static_assert(128 * kIssueRegs + 256 * kAddRegs <= kThreads * kLaunchRegs, "register split above the launch's");
    static constexpr int kBars = 2 * kStages + 4;
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kAddWarps * kPieceBytes +
                                    kScaleSlots * kScaleFloats * 4 + (kBars + 1) * 8 + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
    static_assert(kScaleSlots >= kStep * (kStages + 2), "a slot would be overwritten while it is read");
};

struct TileParams {
    CUtensorMap tm_x, tm_w, tm_y;
    const float* xs;
    const float* ws;
    int32_t T, N, nb;          // nb: blocks of a row
    int32_t wide_scales;       // both scales' rows are 16-byte aligned
    int32_t tiles_m, tiles_n;
    int32_t n_whole, n_split;  // tiles [0, n_whole) are whole; each of the others is cut into n_split pieces of its
    int32_t n_items;           //   blocks, whose sums go to `part` and are added up by linear_join_kernel
    float* part;
    int32_t* status;           // cleared by the first CTA as it begins: a wait that runs out records that a millisecond
};                             //   later at the soonest

// Item i of the grid's list: a tile, and the blocks [kb0, kb1) of it
struct Item {
    int tm, tn, kb0, kb1, piece;               // piece: its place in `part`, -1 for a whole tile
};

// Tiles in bands of kGroupRows rows of x: a band's columns are swept one after another, so that the tiles at work at any
// time share few rows of x and of w.
__host__ __device__ __forceinline__ void tile_at(int tiles_m, int tiles_n, int i, int* tm, int* tn) {
    constexpr int kGroup = kGroupRows / 128;
    const int band = kGroup * tiles_n;
    const int m0 = i / band * kGroup;
    const int left = tiles_m - m0, rows = left < kGroup ? left : kGroup;
    const int r = i % band;
    *tm = m0 + r % rows;
    *tn = r / rows;
}
template <class C>
__device__ __forceinline__ Item item_at(const TileParams& P, int i) {
    Item it;
    it.kb0 = 0;
    it.kb1 = P.nb;
    it.piece = i - P.n_whole;
    int tile = i;
    if (it.piece < 0) {
        it.piece = -1;
    } else {
        const int q = it.piece % P.n_split;
        tile = P.n_whole + it.piece / P.n_split;
        it.kb0 = (int)((int64_t)P.nb * q / P.n_split) / C::kStep * C::kStep;
        if (q + 1 < P.n_split) it.kb1 = (int)((int64_t)P.nb * (q + 1) / P.n_split) / C::kStep * C::kStep;
    }
    tile_at(P.tiles_m, P.tiles_n, tile, &it.tm, &it.tn);
    return it;
}

struct Bars {
    uint32_t full, empty, tfull, tempty;       // per stage: loaded, free; per accumulator: summed, read
    volatile int* abort_flag;
};

// The whole warp runs this loop too (see tile_issue); in a loop of one lane 600 x 2704 x 2704 took 3 % longer
template <class C>
__device__ __forceinline__ void tile_load(const TileParams& P, const Bars& B, uint8_t* smem) {
    const bool one = elect_one();
    StageRing<C::kStages> ring;
    uint32_t used = 0;
    for (int i = blockIdx.x; i < P.n_items; i += gridDim.x) {
        const Item it = item_at<C>(P, i);
        const int row_x = it.tm * 128, row_w = it.tn * C::kPN;
        for (int kb = it.kb0; kb < it.kb1; kb += C::kStep) {
            const bool ok = wait_here(B.empty + ring.stage * 8, ring.phase ^ 1u, B.abort_flag, P.status);
            if (!__all_sync(0xffffffffu, ok)) {
                drain_loads(B.full, used, C::kStages);
                return;
            }
            const int n = min(C::kStep, it.kb1 - kb);
            const uint32_t full = B.full + ring.stage * 8, sa = smem_u32(smem + ring.stage * C::kStageBytes);
            if (one) {
                mbar_expect_tx(full, n * C::kBlockBytes);
#pragma unroll
                for (int g = 0; g < C::kStep; ++g) {
                    if (g >= n) break;
                    const uint32_t sx = sa + g * C::kBlockBytes, sw = sx + kOperandBytes;
                    tma_load_2d(sx, &P.tm_x, (kb + g) * kQBlock, row_x, full);
                    tma_load_2d(sw, &P.tm_w, (kb + g) * kQBlock, row_w, full);
                }
            }
            __syncwarp();
            ring.next();
            ++used;
        }
    }
    await_commits(ring, B.empty, B.abort_flag, P.status);
}

// The whole warp runs this loop, and one lane issues: what the MMAs take (descriptors, addresses) is then uniform over
// the warp.  In a loop of one lane alone, issuing a block took 480 cycles, more than its MMAs.
template <class C>
__device__ __forceinline__ void tile_issue(const TileParams& P, const Bars& B, uint8_t* smem, uint32_t tmem) {
    const bool one = elect_one();
    const uint64_t desc_x = smem_desc(smem_u32(smem), 16, 1024);
    const uint64_t desc_w = smem_desc(smem_u32(smem) + kOperandBytes, 16, 1024);
    StageRing<C::kStages> ring;
    uint32_t use = 0;                          // steps so far: accumulator use & 1
    for (int i = blockIdx.x; i < P.n_items; i += gridDim.x) {
        const Item it = item_at<C>(P, i);
        for (int kb = it.kb0; kb < it.kb1; kb += C::kStep, ++use) {
            const uint32_t acc = use & 1u;
            // after a time-out no wait holds any longer, here and in tile_add: the blocks are gone through to the end,
            // their values lost
            wait_both(B.full + ring.stage * 8, ring.phase, B.tempty + acc * 8, ((use >> 1) & 1u) ^ 1u, B.abort_flag,
                      P.status);
            __syncwarp();
            tc_fence_after();
            const uint64_t at = (uint64_t)(ring.stage * (C::kStageBytes >> 4));
            if (one) {
#pragma unroll
                for (int g = 0; g < C::kStep; ++g) {
                    if (kb + g >= it.kb1) break;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_e4m3(tmem + acc * C::kAccCols + g * C::kPN, desc_x + at + g * (C::kBlockBytes >> 4) + 2 * k,
                                 desc_w + at + g * (C::kBlockBytes >> 4) + 2 * k, instr_desc_e4m3(128, C::kPN), k > 0);
                }
                mma_commit(B.tfull + acc * 8);
                mma_commit(B.empty + ring.stage * 8);
            }
            __syncwarp();
            ring.next();
        }
    }
}

// Warps 2 and 3 bring the scales of each block to shared memory: sx of this warp's 64 rows of x and sw of one of the
// tile's two blocks of w's rows.  Read by the adding warps themselves, from global memory, they cost 8 % of an
// 8192 x 8192 x 28672 product: a read under way has to end before a wait's loop is entered.
// They arrive on the stage's barrier, so a block's MMAs, and with them its sums, come after its scales.
// Slot kb % kScaleSlots is free once the MMAs of block kb - kStages are done, as they began after the adding warps had
// finished with block kb - kStages - 2.
template <class C>
__device__ __forceinline__ void tile_scales(const TileParams& P, const Bars& B, float* slots, int which, int lane) {
    StageRing<C::kStages> ring;
    uint32_t use = 0;
    for (int i = blockIdx.x; i < P.n_items; i += gridDim.x) {
        const Item it = item_at<C>(P, i);
        const int t = it.tm * 128 + 64 * which + lane;
        const int n0 = it.tn * C::kPN + (C::kPN == 256 ? 128 * which : 0);
        const float* x0 = P.xs + (int64_t)min(t, P.T - 1) * P.nb;          // rows past the end: any scale will do
        const float* x1 = P.xs + (int64_t)min(t + 32, P.T - 1) * P.nb;
        const float* w = P.ws + (int64_t)min(n0 / kQBlock, (P.N - 1) / kQBlock) * P.nb;
        for (int kb0 = it.kb0; kb0 < it.kb1; kb0 = (kb0 & ~3) + 4) {       // groups of four by block number
            float a[4], b[4], c[4];
            const int g0 = kb0 & ~3;
            if (P.wide_scales) {               // rows of scales 16-byte aligned: four blocks at a time
                const float4 va = *reinterpret_cast<const float4*>(x0 + g0);
                const float4 vb = *reinterpret_cast<const float4*>(x1 + g0);
                const float4 vc = *reinterpret_cast<const float4*>(w + g0);
                a[0] = va.x; a[1] = va.y; a[2] = va.z; a[3] = va.w;
                b[0] = vb.x; b[1] = vb.y; b[2] = vb.z; b[3] = vb.w;
                c[0] = vc.x; c[1] = vc.y; c[2] = vc.z; c[3] = vc.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kb = min(g0 + j, P.nb - 1);
                    a[j] = x0[kb];
                    b[j] = x1[kb];
                    c[j] = w[kb];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (g0 + j < kb0 || g0 + j >= it.kb1) continue;
                if (j % C::kStep == 0) {       // items start with a step
                    const bool ok = wait_here(B.empty + ring.stage * 8, ring.phase ^ 1u, B.abort_flag, P.status);
                    if (!__all_sync(0xffffffffu, ok)) return;
                }
                float* s = slots + (use * C::kStep + j % C::kStep) % kScaleSlots * kScaleFloats;
                s[64 * which + lane] = a[j];
                s[64 * which + 32 + lane] = b[j];
                if (lane == 0) s[128 + which] = c[j];
                if (j % C::kStep == C::kStep - 1 || g0 + j == it.kb1 - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.full + ring.stage * 8);
                    ++use;
                    ring.next();
                }
            }
        }
    }
}

template <class C>
__device__ __forceinline__ void tile_add(const TileParams& P, const Bars& B, uint32_t tmem, int warp, int lane,
                                         const float* slots, uint32_t stage_out) {
    const int quarter = warp & 3, half = (warp - 4) / 4;
    const uint32_t taddr0 = tmem + ((uint32_t)(quarter * 32) << 16) + half * C::kCols;
    uint32_t use = 0;
    for (int i = blockIdx.x; i < P.n_items; i += gridDim.x) {
        const Item it = item_at<C>(P, i);
        const int t0 = it.tm * 128 + quarter * 32;
        const int n0 = it.tn * C::kPN + half * C::kCols;
        uint64_t acc[C::kCols / 2];
#pragma unroll
        for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
        for (int kb = it.kb0; kb < it.kb1; kb += C::kStep, ++use) {
            const uint32_t buf = use & 1u;
            wait_here(B.tfull + buf * 8, (use >> 1) & 1u, B.abort_flag, P.status);
            __syncwarp();
            tc_fence_after();
            const uint32_t ta = taddr0 + buf * C::kAccCols;
            uint32_t d[2][16];
            tmem_ld16(ta, d[0]);
            // written before the step's MMAs were issued (see tile_scales); of a block past the end: any value
            uint64_t sc[C::kStep];
#pragma unroll
            for (int g = 0; g < C::kStep; ++g) {
                const float* s = slots + (use * C::kStep + g) % kScaleSlots * kScaleFloats;
                sc[g] = both(s[quarter * 32 + lane] * s[128 + half * C::kCols / 128]);
            }
            constexpr int kChunks = C::kCols / 16;
#pragma unroll
            for (int i = 0; i < C::kStep * kChunks; ++i) {
                const int g = i / kChunks, c = i % kChunks;
                if (kb + g >= it.kb1) break;
                tmem_ld_wait();
                if (c < kChunks - 1 || (g < C::kStep - 1 && kb + g + 1 < it.kb1)) {
                    tmem_ld16(ta + (i + 1) / kChunks * C::kPN + (i + 1) % kChunks * 16, d[(i + 1) & 1]);
                } else {                       // read to the end: the accumulator goes back before the last sums
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.tempty + buf * 8);
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) fma2(acc[8 * c + q], d[i & 1][2 * q], d[i & 1][2 * q + 1], sc[g]);
            }
        }
        if (it.piece >= 0) {
            // [128 rows][kPN outputs] as groups of 4 outputs: a warp writes 512 contiguous bytes per group
            float* part = P.part + (int64_t)it.piece * (128 * C::kPN) +
                          ((int64_t)half * (C::kCols / 4) * 128 + quarter * 32 + lane) * 4;
            if (t0 < P.T && n0 < P.N) {
#pragma unroll
                for (int c = 0; c < C::kCols / 4; ++c) {
                    const float2 f = halves(acc[2 * c]), g = halves(acc[2 * c + 1]);
                    __stcg(reinterpret_cast<float4*>(part + c * 512), make_float4(f.x, f.y, g.x, g.y));
                }
            }
            continue;
        }
        // a warp's 32 rows leave in pieces of 32 columns, through shared memory, as one TMA store each (rows and
        // columns past the end are cut off there)
#pragma unroll
        for (int piece = 0; piece < C::kCols / 32; ++piece) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");      // the last piece is out
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = halves(acc[16 * piece + 4 * c + k]);
                    q[k] = pack_bf16(f.x, f.y);
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage_out + lane * 64 +
                                                                             ((c ^ ((lane >> 1) & 3)) * 16)),
                             "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3])
                             : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0 && t0 < P.T && n0 + 32 * piece < P.N) tma_store_2d(&P.tm_y, stage_out, n0 + 32 * piece, t0);
        }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1) linear_tile_kernel(const __grid_constant__ TileParams P) {
    extern __shared__ uint8_t dsmem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t* out = smem + C::kStages * C::kStageBytes;
    float* slots = reinterpret_cast<float*>(out + kAddWarps * kPieceBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(slots + kScaleSlots * kScaleFloats);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kBars);
    Bars B;
    B.abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    B.full = smem_u32(bars);
    B.empty = B.full + C::kStages * 8;
    B.tfull = B.empty + C::kStages * 8;
    B.tempty = B.tfull + 16;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(B.full + s * 8, 3);            // the arm and its bytes; warps 2 and 3
            mbar_init(B.empty + s * 8, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(B.tfull + b * 8, 1);
            mbar_init(B.tempty + b * 8, kAddWarps);
        }
        *B.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(2 * C::kAccCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kIssueRegs));
        if (warp == 0) tile_load<C>(P, B, smem);
        if (warp == 1) tile_issue<C>(P, B, smem, tmem);
        if (warp >= 2) tile_scales<C>(P, B, slots, warp - 2, lane);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kAddRegs));
        tile_add<C>(P, B, tmem, warp, lane, slots, smem_u32(out) + (uint32_t)((warp - 4) * kPieceBytes));
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * C::kAccCols) : "memory");
}

// Adds up the pieces of each cut tile, in their order, and writes its outputs.  One CTA per 32 rows by 64 outputs of
// a tile; each warp adds 8 columns, a lane one row, so that every read is 512 contiguous bytes.
template <class C>
__global__ void __launch_bounds__(256) linear_join_kernel(const float* part, __nv_bfloat16* y,
                                                          int64_t ld_y, int32_t T, int32_t N, int32_t tiles_m,
                                                          int32_t tiles_n, int32_t n_whole, int32_t n_split) {
    grid_dep_wait();
    constexpr int kPerRow = C::kPN / 64, kPerTile = 4 * kPerRow;
    const int cut = blockIdx.x / kPerTile, sub = blockIdx.x % kPerTile;
    int tm, tn;
    tile_at(tiles_m, tiles_n, n_whole + cut, &tm, &tn);
    const int row = sub / kPerRow * 32 + threadIdx.x % 32, col = sub % kPerRow * 64 + threadIdx.x / 32 * 8;
    const int t = tm * 128 + row, n = tn * C::kPN + col;
    if (t >= T || n >= N) return;
    const float* p = part + (int64_t)cut * n_split * (128 * C::kPN) + (int64_t)col * 128 + row * 4;
    float v[8] = {};
    for (int q = 0; q < n_split; ++q, p += 128 * C::kPN) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
        const float4 b = __ldcg(reinterpret_cast<const float4*>(p + 512));
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    *reinterpret_cast<uint4*>(y + t * ld_y + n) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// =============================================================================================================
// Few rows (decode): 128 rows of w by all rows of x, K cut over a cluster.
//
// Here the weight's bytes are the work, so w's rows are the MMA's M (128 outputs a CTA) and x's rows its N, padded to
// NT: a product costs few tensor cycles and the sums of all NT rows of x stay in one thread per output.  K is cut over
// the CTAs of a cluster, each with its own stages in flight, and their sums meet through distributed shared memory,
// added in rank order.  An x of few rows may be quantized on the way, by each CTA for its own K range (see
// quantized_on_the_way); else it comes quantized.
//
// 256 threads: warp 0 loads (TMA), warp 1 issues, warps 2 and 3 bring the scales (and quantize), warps 4..7 scale and
// add: each thread has one output.
// =============================================================================================================
constexpr int kRThreads = 256;
constexpr int kMaxCluster = 8;
template <int NT>
struct RowsCfg {
    static constexpr int kStageB = kOperandBytes + NT * kQBlock;
    static constexpr int kStages = 4;                      // 3 CTAs of 16 rows to an SM, 2 of 32 and of 64
    static constexpr int kSlots = 8;                       // blocks whose scales are at hand
    static constexpr int kSlotFloats = NT + 4;             // rows of x, one block of w's rows
    static constexpr uint32_t kCols = 2 * NT;              // two accumulators
    static constexpr size_t kSmem = (size_t)kStages * kStageB + kSlots * kSlotFloats * 4 + (2 * kStages + 5) * 8 + 1024;
    static_assert(kSlots >= kStages + 2, "a slot would be overwritten while it is read");
    static_assert(NT * 128 * 4 <= kStages * kStageB, "the sums must fit the stages");
    // CTAs that share an SM must find their accumulators free (allocation waits, and a cluster's CTAs wait for one
    // another): as many as fit the shared memory fit the 512 columns
    static_assert((227 * 1024 / kSmem) * kCols <= 512, "accumulators of the CTAs on one SM");
};

struct RowsParams {
    CUtensorMap tm_w, tm_x;        // tm_x: quantized x
    const void* x;                 // else x itself, ld_x elements apart
    int64_t ld_x;
    const float* xs;
    const float* ws;
    __nv_bfloat16* y;
    int64_t ld_y;
    int32_t T, K, N, nb;
    int32_t* status;
};

// Quantizes block kb of x's NT rows into a stage (rows of 128 bytes, 16-byte pieces swizzled as the MMA reads them) and
// its scales into a slot; two warps share the rows, two rows of a warp at a time.  Rows past the last one keep whatever
// the stage and the slot hold: their sums are stored nowhere.
template <int NT, class Row8>
struct RowsQuant {
    static constexpr int kSteps = NT / 4;
    Row8 r[kSteps];
    __device__ __forceinline__ void load(const RowsParams& P, int kb, int which, int lane) {
        const int col = kb * kQBlock + lane % kLanesPerBlock * 8;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int t = 2 * (2 * i + which) + lane / kLanesPerBlock;
            r[i].zero();
            if (t < P.T && col < P.K) r[i].load(P.x, t * P.ld_x + col);
        }
    }
    __device__ __forceinline__ void store(int T, uint8_t* stage, float* slot, int which, int lane) const {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int t = 2 * (2 * i + which) + lane / kLanesPerBlock, c = lane % kLanesPerBlock;
            if (t - lane / kLanesPerBlock >= T) break;
            float v[8], inv;
            r[i].get(v);
            const float sc = block_scale(max_over_block(r[i].abs_max()), &inv);
            *reinterpret_cast<uint2*>(stage + t * 128 + (((c >> 1) ^ (t & 7)) * 16) + (c & 1) * 8) = encode8(v, inv);
            if (c == 0) slot[t] = sc;
        }
    }
};

// Row8: the type of an x that is quantized here, void for one that comes in 8 bits
template <int NT, class Row8>
__global__ void __launch_bounds__(kRThreads) linear_rows_kernel(const __grid_constant__ RowsParams P) {
    using C = RowsCfg<NT>;
    constexpr bool kQuant = !std::is_same<Row8, void>::value;
    extern __shared__ uint8_t dsmem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    float* slots = reinterpret_cast<float*>(smem + C::kStages * C::kStageB);
    uint64_t* bars = reinterpret_cast<uint64_t*>(slots + C::kSlots * C::kSlotFloats);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::kStages + 4);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t full = smem_u32(bars), empty = full + C::kStages * 8, tfull = empty + C::kStages * 8,
                   tempty = tfull + 16;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint32_t n_ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n_ranks));
    const uint32_t rank = cluster_ctarank();
    const int n0 = (int)(blockIdx.x / n_ranks) * 128;
    const int kb0 = (int)((int64_t)P.nb * rank / n_ranks), kb1 = (int)((int64_t)P.nb * (rank + 1) / n_ranks);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full + s * 8, 3);          // the arm and its bytes; warps 2 and 3
            mbar_init(empty + s * 8, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull + b * 8, 1);
            mbar_init(tempty + b * 8, 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dep_launch();
    grid_dep_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *P.status = 0;      // see TileParams::status

    if (warp == 0) {
        // the whole warp (see tile_load): 16 x 8192 x 28672 40.7 us so, 41.3 us in a loop of one lane
        const bool one = elect_one();
        StageRing<C::kStages> ring;
        for (int kb = kb0; kb < kb1; ++kb) {
            const bool ok = wait_here(empty + ring.stage * 8, ring.phase ^ 1u, abort_flag, P.status);
            if (!__all_sync(0xffffffffu, ok)) {
                drain_loads(full, kb - kb0, C::kStages);
                break;
            }
            const uint32_t bar = full + ring.stage * 8, sa = smem_u32(smem + ring.stage * C::kStageB);
            if (one) {
                mbar_expect_tx(bar, kQuant ? kOperandBytes : C::kStageB);
                tma_load_2d(sa, &P.tm_w, kb * kQBlock, n0, bar);
                if constexpr (!kQuant) tma_load_2d(sa + kOperandBytes, &P.tm_x, kb * kQBlock, 0, bar);
            }
            __syncwarp();
            ring.next();
        }
        await_commits(ring, empty, abort_flag, P.status);
    } else if (warp == 1) {
        // the whole warp, so that descriptors are uniform (see tile_issue)
        const bool one = elect_one();
        const uint64_t desc_w = smem_desc(smem_u32(smem), 16, 1024);
        const uint64_t desc_x = smem_desc(smem_u32(smem) + kOperandBytes, 16, 1024);
        StageRing<C::kStages> ring;
        for (int kb = kb0, use = 0; kb < kb1; ++kb, ++use) {
            const uint32_t acc = use & 1u;
            wait_both(full + ring.stage * 8, ring.phase, tempty + acc * 8, ((use >> 1) & 1u) ^ 1u, abort_flag, P.status);
            __syncwarp();
            tc_fence_after();
            const uint64_t at = (uint64_t)(ring.stage * (C::kStageB >> 4));
            if (one) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3(tmem + acc * NT, desc_w + at + 2 * k, desc_x + at + 2 * k, instr_desc_e4m3(128, NT), k > 0);
                mma_commit(tfull + acc * 8);
                mma_commit(empty + ring.stage * 8);
            }
            __syncwarp();
            ring.next();
        }
    } else if (warp < 4) {
        const int which = warp - 2;
        StageRing<C::kStages> ring;
        const float* ws = P.ws + (int64_t)(n0 / kQBlock) * P.nb;
        if constexpr (kQuant) {
            RowsQuant<NT, Row8> q;
            q.load(P, kb0, which, lane);
            float w = ws[min(kb0, P.nb - 1)];
            for (int kb = kb0, use = 0; kb < kb1; ++kb, ++use) {
                const RowsQuant<NT, Row8> now = q;
                const float w_now = w;
                if (kb + 1 < kb1) {
                    q.load(P, kb + 1, which, lane);
                    w = ws[kb + 1];
                }
                const bool ok = wait_phase(empty + ring.stage * 8, ring.phase ^ 1u, abort_flag, P.status);
                if (!__all_sync(0xffffffffu, ok)) break;
                float* slot = slots + use % C::kSlots * C::kSlotFloats;
                now.store(P.T, smem + ring.stage * C::kStageB + kOperandBytes, slot, which, lane);
                if (which == 0 && lane == 0) slot[NT] = w_now;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");     // the MMA reads what was stored
                __syncwarp();
                if (lane == 0) mbar_arrive(full + ring.stage * 8);
                ring.next();
            }
        } else {
            // rows of x that do not exist have codes of zero (TMA) and the last row's scale
            const int t = (NT == 64 ? 32 * which : 0) + lane;
            const float* xs = P.xs + (int64_t)min(t, P.T - 1) * P.nb;
            for (int kb = kb0, use = 0; kb < kb1; ++kb, ++use) {
                const float a = xs[kb], w = ws[kb];
                const bool ok = wait_phase(empty + ring.stage * 8, ring.phase ^ 1u, abort_flag, P.status);
                if (!__all_sync(0xffffffffu, ok)) break;
                float* slot = slots + use % C::kSlots * C::kSlotFloats;
                if (NT == 64 || (which == 0 && lane < NT)) slot[t] = a;
                if (which == 0 && lane == 0) slot[NT] = w;
                __syncwarp();
                if (lane == 0) mbar_arrive(full + ring.stage * 8);
                ring.next();
            }
        }
    } else {
        const int quarter = warp & 3;
        const uint32_t taddr0 = tmem + ((uint32_t)(quarter * 32) << 16);
        uint64_t acc[NT / 2];
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) acc[j] = 0;
        for (int kb = kb0, use = 0; kb < kb1; ++kb, ++use) {
            const uint32_t buf = use & 1u;
            wait_phase(tfull + buf * 8, (use >> 1) & 1u, abort_flag, P.status);    // after a time-out: on to the end
            __syncwarp();
            tc_fence_after();
            const float* s = slots + use % C::kSlots * C::kSlotFloats;
            const float w = s[NT];
#pragma unroll
            for (int c = 0; c < NT / 16; ++c) {
                uint32_t d[16];
                tmem_ld16(taddr0 + buf * NT + 16 * c, d);
                float4 f[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) f[q] = *reinterpret_cast<const float4*>(s + 16 * c + 4 * q);
                tmem_ld_wait();
                if (c == NT / 16 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty + buf * 8);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    fma2(acc[8 * c + 2 * q], d[4 * q], d[4 * q + 1], two(f[q].x * w, f[q].y * w));
                    fma2(acc[8 * c + 2 * q + 1], d[4 * q + 2], d[4 * q + 3], two(f[q].z * w, f[q].w * w));
                }
            }
        }
        // every stage has been read: its memory takes the sums, [NT rows of x][128 outputs]
        float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
            const float2 f = halves(acc[j]);
            sums[(2 * j) * 128 + quarter * 32 + lane] = f.x;
            sums[(2 * j + 1) * 128 + quarter * 32 + lane] = f.y;
        }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
    // the cluster's CTAs share the rows of y out: each adds its rows' sums of all ranks, two outputs a thread
    const int n = n0 + (threadIdx.x & 63) * 2;
    for (int t = (int)rank + (int)n_ranks * (threadIdx.x / 64); t < P.T; t += (int)n_ranks * (kRThreads / 64)) {
        const uint32_t at = smem_u32(smem) + (uint32_t)(t * 128 + (threadIdx.x & 63) * 2) * 4;
        float2 v = make_float2(0.f, 0.f);
        for (uint32_t r = 0; r < n_ranks; ++r) {
            float a, b;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"(mapa_shared(at, r)));
            v.x += a;
            v.y += b;
        }
        if (n < P.N) *reinterpret_cast<uint32_t*>(P.y + t * P.ld_y + n) = pack_bf16(v.x, v.y);
    }
    cluster_sync_all();                          // no CTA ends while another reads its sums
}

// --------------------------------------------------------------------------------------------------------- host
// [rows, K] codes, rows ld bytes apart, as 128-byte swizzled boxes of {128 columns, box_rows}; past the end reads 0
bool encode_codes(CUtensorMap* m, const void* base, uint64_t K, uint64_t rows, uint64_t ld, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {K, rows};
    cuuint64_t strides[1] = {ld};
    cuuint32_t box[2] = {kQBlock, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y [T, N] as 64-byte swizzled boxes of {32 columns, 32 rows}: what an adding warp stores at a time
bool encode_y(CUtensorMap* m, const void* base, uint64_t N, uint64_t T, uint64_t ld) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {N, T};
    cuuint64_t strides[1] = {ld * 2};
    cuuint32_t box[2] = {32, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SM count of the current device; on a device's first use its kernels' shared memory limits are raised
cudaError_t device_sms(int* sms) {
    static std::mutex mu;
    static std::vector<int> known;             // by device, 0: not used yet
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    if ((int)known.size() <= d) known.resize(d + 1, 0);
    if (known[d] == 0) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d);
        auto allow = [&](auto kernel, size_t smem) {
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        };
        allow(linear_tile_kernel<TileCfg<256>>, TileCfg<256>::kSmem);
        allow(linear_tile_kernel<TileCfg<128>>, TileCfg<128>::kSmem);
        allow(linear_rows_kernel<16, Row8Bf16>, RowsCfg<16>::kSmem);
        allow(linear_rows_kernel<16, Row8F32>, RowsCfg<16>::kSmem);
        allow(linear_rows_kernel<16, void>, RowsCfg<16>::kSmem);
        allow(linear_rows_kernel<32, void>, RowsCfg<32>::kSmem);
        allow(linear_rows_kernel<64, void>, RowsCfg<64>::kSmem);
        if (e != cudaSuccess) return e;
        known[d] = n;
    }
    *sms = known[d];
    return cudaSuccess;
}

// Whether a product runs on linear_rows_kernel: up to 32 rows, and up to 64 where K is long enough to be cut and N does not
// fill the SMs by itself.  64 x 8192 x 8192 takes 17.0 us there (17.9 us on tiles), 64 x 2704 x 2704 7.8 us (7.8 us);
// 64 x 512 x 2704 7.1 us (4.3 us), 64 x 4096 x 28672 28.7 us (24.6 us); 32 x 4096 x 4096 6.5 us (7.2 us), 32 x 4096 x
// 28672 23.9 us (23.8 us).  The rule loses where K is of middling length: 48 x 4096 x 4096 8.4 us (7.4 us).
bool few_rows(int32_t T, int32_t K, int32_t N) { return T <= 32 || (T <= 64 && K > 1024 && N <= 8192); }
// Whether that kernel quantizes x itself: a launch less, but a part of every 128 outputs' work, so for few products.  From
// a program's loop, which two launches and a workspace hold up, and replayed from a graph: 16 x 4096 x 4096 takes 13 and
// 7.7 us so (quantized first: 18 and 6.9 us), 1 x 4096 x 28672 24.5 and 24.0 us (24.6 and 23.2 us), 16 x 5120 x 5120 13.3
// and 12.7 us (18 and 8.2 us).
bool quantized_on_the_way(int32_t T, int32_t K, int32_t N) { return T <= 16 && (int64_t)T * K * N <= (1 << 28); }

// A product's shape, and how its tiles are spread over the SMs.  Tiles beyond the last full round may be cut along K, into
// as many pieces as SMs are left for each, at most kMaxSplit, of at least kMinBlocks blocks: a last round of 8 tiles would
// leave 144 of 152 SMs idle for a tile's whole time.  The choice is by an estimate whose numbers were fitted.  For 169
// products of 68 to 8192 rows (K and N from 512 to 28672) it is 11 % off (rms; the 3 us that every launch takes are left
// out of it), the shape it takes 0.2 % slower than the better of the two, 10 % at the worst (384 x 2704 x 2704).
// Measured in us, x in 8 bits, weights of fp8_quantize_weight, three in turn, in replayed graphs of a few milliseconds:
//                               256     128
//    300 x   512 x  2704        5.4     4.5
//    500 x  4096 x  4096       15.6    10.8
//    256 x  4096 x 28672       37.4    33.6
//    600 x  2704 x  2704       14.4    12.7
//   1500 x  2704 x  2704       16.6    20.6
//    300 x  5120 x  5120       17.2    13.5   120 narrow tiles in one round
//    777 x  5120 x  5120       20.3    23.3   140 wide tiles in one round
//   1111 x 14336 x  4096       48.5    60.7   144 wide tiles in one round (54 us in a long run, at 1.78 GHz)
//   2048 x 28672 x  8192        334     428
//   8192 x  8192 x 28672       1455    1630
constexpr int kMaxSplit = 8, kMinBlocks = 4;
constexpr int kSms = 152;                                // planned for; right on any device
struct Spread {
    int pn;                                              // TileCfg
    int tiles_m, tiles_n, n_whole, n_split, n_items;
    double us;                                           // estimate
    int n_cut() const { return tiles_m * tiles_n - n_whole; }
};
Spread spread_as(int32_t T, int32_t K, int32_t N, int pn) {
    // a block; a tile's outputs on their way out, while no sums are added up; a join, and each 256 KB that it reads
    const double block = pn == 256 ? 0.436 : 0.255, out = pn == 256 ? 1.3 : 0.8, join = 2.7, join_sums = 0.05;
    Spread s{};
    s.pn = pn;
    s.tiles_m = (int)(((int64_t)T + 127) / 128);
    s.tiles_n = (N + pn - 1) / pn;
    const int tiles = s.tiles_m * s.tiles_n, rest = tiles % kSms, nb = blocks_of(K), rounds = tiles / kSms;
    s.n_whole = tiles;
    s.us = (double)(rounds + (rest > 0)) * (nb * block + out);
    const int pieces = rest ? std::min({kSms / rest, kMaxSplit, nb / kMinBlocks}) : 0;
    if (pieces >= 2) {
        const double sums = (double)rest * pieces * pn / 512.0;
        const double cut = (double)rounds * (nb * block + out) + (double)((nb + pieces - 1) / pieces) * block + join +
                           join_sums * sums;
        if (cut < s.us) {
            s.us = cut;
            s.n_split = pieces;
            s.n_whole = tiles - rest;
        }
    }
    s.n_items = s.n_whole + s.n_cut() * s.n_split;
    return s;
}
Spread spread_of(int32_t T, int32_t K, int32_t N) {
    if (few_rows(T, K, N)) return Spread{};
    const Spread wide = spread_as(T, K, N, 256), narrow = spread_as(T, K, N, 128);
    return narrow.us < wide.us ? narrow : wide;
}

// Workspace: the status word, then x's codes and scales if x is quantized on the way, then the cut tiles' sums
struct Scratch {
    size_t codes = 0, scales = 0, part = 0, end = 0;
};
Scratch layout_of(int32_t T, int32_t K, bool x_fp8, const Spread& s) {
    auto al = [](size_t v) { return (v + 255) & ~size_t(255); };
    Scratch L;
    L.codes = 256;
    L.scales = L.codes + (x_fp8 ? 0 : al((size_t)T * K));
    L.part = L.scales + (x_fp8 ? 0 : al((size_t)T * blocks_of(K) * sizeof(float)));
    L.end = L.part + (size_t)s.n_cut() * s.n_split * 128 * s.pn * sizeof(float);
    return L;
}
// CTAs of a cluster that share 128 outputs' K: more while the launch has fewer than one per SM and each keeps
// kMinBlocks blocks.  Up to two per SM cost 64 x 4096 x 14336 22 us instead of 18 (another round of CTAs, each with its
// set-up), and gained 16 x 8192 x 28672 1 us of 43.
int ranks_of(int32_t N, int32_t nb) {
    const int tiles = (N + 127) / 128;
    int r = 1;
    while (r < kMaxCluster && tiles * r < kSms && nb / (2 * r) >= kMinBlocks) r *= 2;
    return r;
}

template <int NT, class Row8>
cudaError_t launch_rows(const RowsParams& P, int ranks, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((P.N + 127) / 128 * ranks));
    cfg.blockDim = dim3(kRThreads);
    cfg.dynamicSmemBytes = RowsCfg<NT>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, linear_rows_kernel<NT, Row8>, P);
}

template <class C>
cudaError_t launch_tiles(const TileParams& P, const Spread& sp, int sms, __nv_bfloat16* y, int64_t ld_y,
                         cudaStream_t st) {
    const cudaError_t e = launch_pdl(linear_tile_kernel<C>, dim3((unsigned)std::min(sms, sp.n_items)), dim3(kThreads),
                                     C::kSmem, st, P);
    if (e != cudaSuccess || sp.n_cut() == 0) return e;
    return launch_pdl(linear_join_kernel<C>, dim3((unsigned)(4 * (C::kPN / 64) * sp.n_cut())), dim3(256), 0, st,
                      static_cast<const float*>(P.part), y, ld_y, P.T, P.N, sp.tiles_m, sp.tiles_n, sp.n_whole,
                      sp.n_split);
}

int check_sizes(const char* fn, int32_t T, int32_t K, int32_t N) {
    if (T < 0 || K <= 0 || N <= 0)
        return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": T must be >= 0, K and N > 0");
    if (K % 16 != 0 || N % 8 != 0)
        return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": K must be a multiple of 16 and N of 8");
    if (K > (1 << 22)) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": K above 2^22");
    if (T > kMaxRowsOfX) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": T above 2^31 - 1025");
    const int64_t tiles = (((int64_t)T + 127) / 128) * (((int64_t)N + 127) / 128);
    if (tiles > INT32_MAX / 2) return refuse(LORA_ERR_LIMIT, std::string(fn) + ": T x N above 2^44");
    return LORA_OK;
}

}  // namespace

cudaError_t fp8_set_wait_limit_ns(uint64_t ns) { return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns)); }

}  // namespace lora

using namespace lora;

extern "C" size_t lora_fp8_workspace_size(int32_t T, int32_t K, int32_t N, int32_t x_fp8) {
    if (check_sizes("lora_fp8_workspace_size", T, K, N) != LORA_OK) return 0;
    return layout_of(T, K, x_fp8 != 0 || quantized_on_the_way(T, K, N), spread_of(T, K, N)).end;
}

extern "C" int lora_fp8_linear(int32_t T, int32_t K, int32_t N, lora_dtype_t dt, const void* x, int64_t ld_x,
                               const float* x_scales, const void* w, const float* w_scales, void* y, int64_t ld_y,
                               void* workspace, size_t ws_bytes, void* stream) {
    return guarded([&]() -> int {
        const char* fn = "lora_fp8_linear";
        if (!x_scales && dt != LORA_BF16 && dt != LORA_F32) return refuse(LORA_ERR_DTYPE, "unknown dtype");
        int rc = check_sizes(fn, T, K, N);
        if (rc != LORA_OK || T == 0) return rc;
        rc = check_matrix(fn, "x", x, K, ld_x, x_scales ? 1 : elem_size(dt));
        if (rc == LORA_OK) rc = check_matrix(fn, "w", w, K, K, 1);
        if (rc == LORA_OK) rc = check_matrix(fn, "y", y, N, ld_y, 2);
        if (rc != LORA_OK) return rc;
        if (!w_scales) return refuse(LORA_ERR_INVALID_ARG, std::string(fn) + ": w_scales is NULL");
        if (!is_aligned(w_scales, 4) || !is_aligned(x_scales, 4))
            return refuse(LORA_ERR_ALIGNMENT, std::string(fn) + ": scales must be aligned to a float");
        const Spread sp = spread_of(T, K, N);
        const Scratch L = layout_of(T, K, x_scales != nullptr || quantized_on_the_way(T, K, N), sp);
        if (!workspace) return refuse(LORA_ERR_WORKSPACE, "workspace is NULL");
        if (!is_aligned(workspace, 256)) return refuse(LORA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
        if (ws_bytes < L.end)
            return refuse(LORA_ERR_WORKSPACE, "workspace too small: need " + std::to_string(L.end) + " bytes, got " +
                                                  std::to_string(ws_bytes));
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        int sms = 0;
        cudaError_t e = device_sms(&sms);
        if (e != cudaSuccess) return enqueued(fn, e);
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const bool quant_here = !x_scales && quantized_on_the_way(T, K, N);
        const bool quant_first = !x_scales && !quant_here;
        const void* xc = quant_first ? ws + L.codes : x;
        const float* xs = quant_first ? reinterpret_cast<const float*>(ws + L.scales) : x_scales;
        const int64_t ld_c = quant_first ? K : ld_x;
        // every tensor map before the first launch
        auto bad_map = [&] { return refuse(LORA_ERR_CUDA, std::string(fn) + ": cuTensorMapEncodeTiled failed"); };
        auto quantize = [&] {
            return quant_first ? launch_quantize(T, K, dt, x, ld_x, ws + L.codes, K, reinterpret_cast<float*>(ws + L.scales),
                                                 st)
                               : cudaSuccess;
        };
        if (few_rows(T, K, N)) {
            RowsParams R{};
            const int nt = T <= 16 ? 16 : T <= 32 ? 32 : 64;
            if (!encode_codes(&R.tm_w, w, K, N, K, 128) || (!quant_here && !encode_codes(&R.tm_x, xc, K, T, ld_c, nt)))
                return bad_map();
            R.x = x;
            R.ld_x = ld_x;
            R.xs = xs;
            R.ws = w_scales;
            R.y = static_cast<__nv_bfloat16*>(y);
            R.ld_y = ld_y;
            R.T = T;
            R.K = K;
            R.N = N;
            R.nb = blocks_of(K);
            R.status = reinterpret_cast<int32_t*>(ws);
            const int ranks = ranks_of(N, R.nb);
            e = quantize();
            if (e != cudaSuccess) return enqueued(fn, e);
            if (quant_here)
                e = dt == LORA_BF16 ? launch_rows<16, Row8Bf16>(R, ranks, st) : launch_rows<16, Row8F32>(R, ranks, st);
            else
                e = nt == 16   ? launch_rows<16, void>(R, ranks, st)
                    : nt == 32 ? launch_rows<32, void>(R, ranks, st)
                               : launch_rows<64, void>(R, ranks, st);
            return enqueued(fn, e);
        }
        TileParams P{};
        if (!encode_codes(&P.tm_x, xc, K, T, ld_c, 128) || !encode_codes(&P.tm_w, w, K, N, K, sp.pn) ||
            !encode_y(&P.tm_y, y, N, T, ld_y))
            return bad_map();
        P.xs = xs;
        P.ws = w_scales;
        P.T = T;
        P.N = N;
        P.nb = blocks_of(K);
        P.wide_scales = P.nb % 4 == 0 && is_aligned(P.xs, 16) && is_aligned(P.ws, 16);
        P.tiles_m = sp.tiles_m;
        P.tiles_n = sp.tiles_n;
        P.n_whole = sp.n_whole;
        P.n_split = sp.n_split;
        P.n_items = sp.n_items;
        P.part = reinterpret_cast<float*>(ws + L.part);
        P.status = reinterpret_cast<int32_t*>(ws);
        e = quantize();
        if (e != cudaSuccess) return enqueued(fn, e);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(y);
        e = sp.pn == 256 ? launch_tiles<TileCfg<256>>(P, sp, sms, out, ld_y, st)
                         : launch_tiles<TileCfg<128>>(P, sp, sms, out, ld_y, st);
        return enqueued(fn, e);
    });
}
