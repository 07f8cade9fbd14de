// Newton-Schulz orthogonalisation of a matrix (the step the Muon optimiser
// takes on a weight's gradient; the Puro-2B-Base model card's training-setup
// paragraph names MuonH):
//
//   X <- G / (|G|_F + eps)
//   per step, coefficients (a, b, c):   S = X X^T   (X^T X for a tall X)
//                                       Q = a I + b S + c S S
//                                       X <- Q X    (X Q)
//
// S, and with it Q, has the shorter side s of G; products are taken on the
// shorter side, so a tall G needs no transposition: its S contracts over rows
// (operands whose contraction is not contiguous, which the tensor cores read
// as they are) and Q is symmetric.
//
// Precision.  The products' operands are FP16 with FP32 accumulation: every
// value here is below about 4 by construction, so FP16's range suffices and
// its 11 bits round 8 times finer than bfloat16's at the same speed.  X, whose
// entries are near 1 / sqrt(m n) at first and would reach FP16's subnormals, is
// kept multiplied by a power of two near sqrt(m n) all along; the products'
// epilogues take it out of S and of the result.  S, Q and X are each rounded
// once per step.  The directions in which X is small are the ones the
// iteration lifts, by up to a^5 = 485, and early roundings of X with them;
// so the first kCarry + 1 steps carry X as a sum of two FP16 numbers (22 bits) for
// the linear term, Q = b S + c S S, X <- a (X_hi + X_lo) + Q X_hi: what the
// products leave out, Q X_lo, is small just there.  Later steps fold a I into
// Q, and X needs no second read.  (Measured against 64 bits on a gradient with
// a decaying spectrum, [520, 1100]: the result's own bfloat16 rounding is
// 1.66e-3 in the 2-norm; all steps folded 2.5e-3, kCarry = 0 2.2e-3, 1 2.0e-3,
// 2 1.8e-3.)
//
// One GEMM kernel, C = A B^T in 256 x 256 tiles of CTA pairs, persistent:
//   warp 0     operands by TMA into a ring of 64-deep stages
//   warp 1     tcgen05.mma.cta_group::2.kind::f16 into one of two 256-column
//              TMEM accumulators (leader CTA)
//   warps 4-11 epilogue: thread = one row, 128 columns; the other accumulator
//              fills meanwhile
// S and Q are symmetric: only tiles on or above the diagonal are computed, and
// the epilogue stores each also transposed.  The tiles of a last, partly filled
// wave are cut into two halves of 128 columns where the pairs suffice.
#pragma once

#include <cuda_fp16.h>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace fp8blk {
namespace ns {

constexpr int BM = 128;                    // output rows per CTA (256 per pair)
constexpr int BN = 256;                    // output columns per pair tile
constexpr int BK = 64;                     // contraction per stage: 128 bytes of FP16
constexpr int STAGES = 5;
constexpr int A_BYTES = BM * BK * 2;
constexpr int B_BYTES = (BN / 2) * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * 64 * 2;     // a 64 x 64 box of an operand whose contraction runs along rows
constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int THREADS = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int TMEM_COLS = 512;
constexpr int OUT_BYTES = 4096;            // 32 rows x 64 columns of 16 bits
constexpr int OFF_OUT = STAGES * STAGE_BYTES;
constexpr int OFF_BARS = OFF_OUT + EPI_WARPS * 2 * OUT_BYTES;
constexpr int NUM_BARS = 2 * STAGES + 2 + 2 + 1;
constexpr int OFF_TMEM_SLOT = OFF_BARS + NUM_BARS * 8;
constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");
static_assert(OFF_OUT % 1024 == 0, "swizzled staging must be 1024-byte aligned");

constexpr int kMaxSide = 32768;
constexpr int kCarry = 1;                  // steps whose X leaves as two FP16 numbers
constexpr uint32_t kProducerSleepNs = 64;

enum Mode : int { kGram = 0, kPoly = 1, kApply = 2 };

struct Params {
    int M, N, K;                // output rows, output columns, contraction
    int tiles_m, tiles_n;       // 256 x 256 tiles
    int tiles;                  // per matrix (upper triangle for kGram, kPoly)
    int full;                   // tiles (of all matrices) taken whole; the others as two halves
    int units;                  // full + 2 * others
    int row_fast;               // kApply: tiles of one column panel in a row (else of one row panel)
    float alpha;                // kGram: the accumulator's factor; kApply: the final output's
    float a, b, c;              // kPoly: Q = a I + b S + c S S; kApply: a of the linear term
    const __half* e0;           // kPoly: S; kApply: X_hi of the linear term, or null
    const __half* e1;           // kApply: X_lo of the linear term
    int64_t e_ld;               // their row stride ([batch][M][e_ld])
    int carry;                  // kApply: also store what the FP16 rounding leaves of X (tmT)
    int final_out;              // kApply: bfloat16 output
    __nv_bfloat16* out;         // final output by plain stores (its rows not 16-byte multiples), else null
    uint64_t wait_ns;
};

// 3-D tiled load into this CTA's shared memory, completing on a barrier of
// either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an operand whose contraction runs along the rows of its
// boxes (64 contraction rows of 64 contiguous output rows or columns, 128-byte
// swizzle): 8 contraction rows 1024 bytes apart, the next 64 outputs one box on.
__device__ __forceinline__ uint64_t smem_desc_mn64_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(BOX_BYTES >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

// FP16 x FP16 -> F32, M x N, the operands' orientation.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// One unit of work: matrix z, output rows row0 .. + 255, columns col0 .. +
// cols - 1 (256, or 128 for a half tile or where the matrix ends there).
// diag: a tile on the diagonal, which is not mirrored.
struct Unit {
    int z, row0, col0, cols;
    bool diag;
};

// Unit u, or false where a half tile lies behind the matrix.
template <int MODE>
__device__ __forceinline__ bool unit_at(const Params& p, int u, Unit& w) {
    int tile = u, sub = 0;
    w.cols = BN;
    if (u >= p.full) {
        tile = p.full + ((u - p.full) >> 1);
        sub = (u - p.full) & 1;
        w.cols = BN / 2;
    }
    w.z = tile / p.tiles;
    int i = tile - w.z * p.tiles;
    int tm = 0, tn;
    if (MODE == kApply) {
        if (p.row_fast) {
            tn = i / p.tiles_m;
            tm = i - tn * p.tiles_m;
        } else {
            tm = i / p.tiles_n;
            tn = i - tm * p.tiles_n;
        }
    } else {                               // upper triangle, row by row
        while (i >= p.tiles_n - tm) {
            i -= p.tiles_n - tm;
            ++tm;
        }
        tn = tm + i;
    }
    w.row0 = tm * 2 * BM;
    w.col0 = tn * BN + sub * (BN / 2);
    w.diag = tm == tn;
    if (p.N - w.col0 <= BN / 2) w.cols = BN / 2;
    return w.col0 < p.N;
}

// tmA, tmB: operands, [batch][rows][cols] FP16; box 64 x 128 for A, 64 x 64 for
// B and for operands whose contraction runs along rows (A_MN, B_MN), 128-byte
// swizzle.  tmC: output, box 64 x 32, 128-byte swizzle.  tmT: kGram, kPoly: the
// same output, box 32 x 64, not swizzled (the mirrored tile); kApply: X_lo, box
// as tmC.
template <int MODE, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmT, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();            // 0 = leader of the pair
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;
    const int num_kb = (p.K + BK - 1) / BK;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const uint32_t full = sbase + OFF_BARS, empty = full + 8 * STAGES, tfull = empty + 8 * STAGES,
                   tempty = tfull + 16, drain = tempty + 16;

    // The next kernel may set itself up on idle SMs, or as CTAs of this one
    // leave; it waits for this one's end before it touches memory.
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + 8 * s, 1);        // leader: its producer's arrive + both CTAs' bytes
            mbar_init(empty + 8 * s, 1);       // one commit to both CTAs
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull + 8 * b, 1);
            mbar_init(tempty + 8 * b, 2 * EPI_WARPS);    // leader: both CTAs' epilogue warps
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(sbase + OFF_TMEM_SLOT, TMEM_COLS);
        tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmC);
        prefetch_tensormap(&tmT);
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();                                      // barriers and TMEM ready in both CTAs
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM_SLOT);
    griddep_wait();                                      // inputs of the preceding kernel are complete

    if (warp == 0) {
        // -------------------------------------------------------- operands
        if (lane == 0) {
            const uint32_t full_leader = map_to_cta(full, 0);
            int it = 0;
            bool ok = true;
            Unit w;
            for (int u = pair; ok && u < p.units; u += npairs) {
                if (!unit_at<MODE>(p, u, w)) continue;
                const int m0 = w.row0 + static_cast<int>(rank) * BM;
                const int n0 = w.col0 + static_cast<int>(rank) * (w.cols / 2);
                const uint32_t bytes = 2 * (A_BYTES + (w.cols / 2) * BK * 2);
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(empty + 8 * s, ((it / STAGES) & 1) ^ 1, abort_flag, p.wait_ns, kErrTimeout,
                                   kProducerSleepNs)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + s * STAGE_BYTES, bar = full_leader + 8 * s;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
                    if (A_MN) {
                        tma_load_3d_pair(dst, &tmA, m0, kb * BK, w.z, bar);
                        tma_load_3d_pair(dst + BOX_BYTES, &tmA, m0 + 64, kb * BK, w.z, bar);
                    } else {
                        tma_load_3d_pair(dst, &tmA, kb * BK, m0, w.z, bar);
                    }
                    for (int h = 0; h < w.cols / 128; ++h) {
                        if (B_MN)
                            tma_load_3d_pair(dst + A_BYTES + h * BOX_BYTES, &tmB, n0 + 64 * h, kb * BK, w.z, bar);
                        else
                            tma_load_3d_pair(dst + A_BYTES + h * BOX_BYTES, &tmB, kb * BK, n0 + 64 * h, w.z, bar);
                    }
                }
            }
            if (!ok && rank == 0) {
                // let every copy already requested land (both CTAs' copies
                // complete on the leader's barriers) before the pair exits
                for (int j = max(0, it - STAGES); j < it; ++j) drain_wait(full + 8 * (j % STAGES), (j / STAGES) & 1, p.wait_ns);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader)
        if (lane == 0 && rank == 0) {
            int it = 0, n = 0;
            bool ok = true;
            Unit w;
            for (int u = pair; ok && u < p.units; u += npairs) {
                if (!unit_at<MODE>(p, u, w)) continue;
                const int buf = n & 1;
                if (!mbar_wait(tempty + 8 * buf, ((n >> 1) & 1) ^ 1, abort_flag, p.wait_ns, kErrTimeout)) break;
                ++n;
                const uint32_t d_tmem = tmem_base + buf * BN;
                const uint32_t idesc = w.cols == BN ? idesc_f16_f32(2 * BM, BN, A_MN, B_MN)
                                                    : idesc_f16_f32(2 * BM, BN / 2, A_MN, B_MN);
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(full + 8 * s, (it / STAGES) & 1, abort_flag, p.wait_ns, kErrTimeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = sbase + s * STAGE_BYTES;
                    const uint64_t a_desc = A_MN ? smem_desc_mn64_sw128(a_addr) : smem_desc_k128_sw128(a_addr);
                    const uint64_t b_desc =
                        B_MN ? smem_desc_mn64_sw128(a_addr + A_BYTES) : smem_desc_k128_sw128(a_addr + A_BYTES);
                    // 16 of the contraction: 32 bytes along a swizzled row, or 16 rows of 128 bytes
                    constexpr uint64_t adv_a = (A_MN ? 16 * 128 : 32) >> 4, adv_b = (B_MN ? 16 * 128 : 32) >> 4;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_f16_pair(d_tmem, a_desc + k * adv_a, b_desc + k * adv_b, idesc, (kb | k) != 0 ? 1u : 0u);
                    mma_commit_pair(empty + 8 * s, 0x3);
                }
                if (ok) mma_commit_pair(tfull + 8 * buf, 0x3);
            }
            // all MMAs done before the pair may free TMEM
            mma_commit_pair(drain, 0x1);
            drain_wait(drain, 0, p.wait_ns);
        }
        __syncwarp();
    } else if (warp >= EPI_WARP0) {
        // ---------------------------------------------------------- epilogue
        const int ew = warp - EPI_WARP0;
        const int quarter = warp & 3;          // TMEM lanes this warp may read
        const int half = ew >> 2;              // which half of the unit's columns
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t tempty_leader = map_to_cta(tempty, 0);
        uint8_t* stage = smem + OFF_OUT + ew * 2 * OUT_BYTES;
        const uint32_t stage_addr = smem_u32(stage);
        const bool lin = MODE == kApply && p.e0 != nullptr;
        constexpr int NE = MODE == kGram ? 1 : MODE == kPoly ? 4 : 8;    // 16-byte pieces of S or X per 32 columns
        int n = 0;
        Unit w;
        for (int u = pair; u < p.units; u += npairs) {
            if (!unit_at<MODE>(p, u, w)) continue;
            const int buf = n & 1;
            const int row0 = w.row0 + static_cast<int>(rank) * BM + quarter * 32;
            const int row = row0 + lane;
            const int chunks = w.cols / 64;        // of 32 columns, per half
            const int cbase = w.col0 + half * (w.cols / 2);
            // S, or X's two parts, of the row's 32 columns from c on
            uint4 e[NE];
            auto fetch = [&](int c) {
                if (MODE == kGram || (MODE == kApply && !lin)) return;
                const bool in = row < p.M && c < p.e_ld;
                const int64_t at = (static_cast<int64_t>(w.z) * p.M + row) * p.e_ld + c;
#pragma unroll
                for (int j = 0; j < NE; ++j) {
                    const __half* src = j < 4 ? p.e0 : p.e1;
                    e[j] = in ? __ldg(reinterpret_cast<const uint4*>(src + at) + (j & 3)) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            fetch(cbase);
            const bool got = mbar_wait(tfull + 8 * buf, (n >> 1) & 1, abort_flag, p.wait_ns, kErrTimeout);
            if (!__all_sync(0xffffffffu, got)) break;
            ++n;
            tc_fence_after();
#pragma unroll 1
            for (int ch = 0; ch < chunks; ++ch) {
                const int col = cbase + 32 * ch;
                uint32_t r[32];
                tmem_ld_32x32b_x32(lane_base + buf * BN + half * (w.cols / 2) + 32 * ch, r);
                tmem_ld_wait();
                if (ch == chunks - 1) {            // the accumulator may be refilled
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(tempty + 8 * buf);
                        else
                            mbar_arrive_remote(tempty_leader + 8 * buf);
                    }
                }
                uint32_t o[16], lo[16];            // the row's 32 results, two per word
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float v0 = __uint_as_float(r[2 * j]), v1 = __uint_as_float(r[2 * j + 1]);
                    if (MODE == kGram) {
                        v0 *= p.alpha;
                        v1 *= p.alpha;
                    }
                    if (MODE == kPoly) {
                        const uint32_t sw = reinterpret_cast<const uint32_t*>(&e[j >> 2])[j & 3];
                        const float2 s2 = __half22float2(*reinterpret_cast<const __half2*>(&sw));
                        v0 = fmaf(p.c, v0, p.b * s2.x) + (row == col + 2 * j && row < p.M ? p.a : 0.0f);
                        v1 = fmaf(p.c, v1, p.b * s2.y) + (row == col + 2 * j + 1 && row < p.M ? p.a : 0.0f);
                    }
                    if (MODE == kApply) {
                        if (lin) {
                            const uint32_t hw = reinterpret_cast<const uint32_t*>(&e[(j >> 2) % NE])[j & 3];
                            const uint32_t lw = reinterpret_cast<const uint32_t*>(&e[(4 + (j >> 2)) % NE])[j & 3];
                            const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(&hw));
                            const float2 l2 = __half22float2(*reinterpret_cast<const __half2*>(&lw));
                            v0 = fmaf(p.a, h2.x + l2.x, v0);
                            v1 = fmaf(p.a, h2.y + l2.y, v1);
                        }
                        if (p.final_out) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(v0 * p.alpha, v1 * p.alpha);
                            o[j] = *reinterpret_cast<const uint32_t*>(&b2);
                            continue;
                        }
                    }
                    const __half2 h2 = __floats2half2_rn(v0, v1);
                    o[j] = *reinterpret_cast<const uint32_t*>(&h2);
                    if (MODE == kApply && p.carry) {
                        const float2 back = __half22float2(h2);
                        const __half2 l2 = __floats2half2_rn(v0 - back.x, v1 - back.y);
                        lo[j] = *reinterpret_cast<const uint32_t*>(&l2);
                    }
                }
                if (ch + 1 < chunks) fetch(col + 32);
                const bool mirror = MODE != kApply && !w.diag;
                if ((ch & 1) == 0) {               // a fresh box of 64 columns: the previous stores have read it
                    if (lane == 0) bulk_wait_group_read0();
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st_shared_v4(stage_addr + lane * 128 + ((((ch & 1) * 4 + c) ^ (lane & 7)) << 4),
                                 make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
                if (MODE == kApply && p.carry) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4(stage_addr + OUT_BYTES + lane * 128 + ((((ch & 1) * 4 + c) ^ (lane & 7)) << 4),
                                     make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]));
                }
                if (mirror) {
                    // two rows' values of a column in one word: even lanes
                    // store column 2 j, odd lanes column 2 j + 1
                    uint32_t* tr = reinterpret_cast<uint32_t*>(stage + OUT_BYTES) + ((ch & 1) * 32 + (lane & 1)) * 16 + (lane >> 1);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const uint32_t other = __shfl_xor_sync(0xffffffffu, o[j], 1);
                        tr[j * 32] = (lane & 1) ? __byte_perm(other, o[j], 0x7632) : __byte_perm(o[j], other, 0x5410);
                    }
                }
                if (!(ch & 1)) continue;
                const int box = col - 32;          // the finished box's first column
                const bool any = row0 < p.M && box < p.N;
                if (MODE == kApply && p.out) {
                    // rows that TMA cannot store: 32 lanes along each row
                    __syncwarp();
                    for (int i = 0; i < 32; ++i) {
                        if (row0 + i >= p.M) break;
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const int c = lane + 32 * v;
                            if (box + c < p.N) {
                                const uint8_t* src = stage + i * 128 + (((c >> 3) ^ (i & 7)) << 4) + (c & 7) * 2;
                                p.out[(static_cast<int64_t>(w.z) * p.M + row0 + i) * p.N + box + c] =
                                    *reinterpret_cast<const __nv_bfloat16*>(src);
                            }
                        }
                    }
                    __syncwarp();
                } else {
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0 && any) {
                        tma_store_3d(&tmC, stage_addr, box, row0, w.z);
                        if (MODE == kApply && p.carry) tma_store_3d(&tmT, stage_addr + OUT_BYTES, box, row0, w.z);
                        if (MODE != kApply && !w.diag) tma_store_3d(&tmT, stage_addr + OUT_BYTES, row0, box, w.z);
                        bulk_commit_group();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_group0();                 // output stores complete
        __syncwarp();
    }

    tc_fence_before();
    __syncwarp();
    cluster_sync();                                      // partner done with our smem and barriers
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// --------------------------------------------------- Frobenius norm and cast

constexpr int kNormBlocks = 256;            // at most, per matrix
constexpr int kNormThreads = 256;

__device__ __forceinline__ double block_sum(double v, double* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kNormThreads / 32; ++w) v += red[w];
    return v;
}

template <typename T> __device__ __forceinline__ float to_float(T v);
template <> __device__ __forceinline__ float to_float(float v) { return v; }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// partial[z][block] = sum of squares of the block's share of matrix z (n
// elements), in FP64: no input overflows it.  VEC: 16-byte aligned loads.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const T* __restrict__ g, int64_t n, double* __restrict__ partial) {
    __shared__ double red[kNormThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const T* x = g + blockIdx.y * n;
    double sum = 0.0;
    if (VEC) {
        constexpr int E = 16 / sizeof(T);
        const int64_t nv = n / E, step = static_cast<int64_t>(gridDim.x) * kNormThreads;
#pragma unroll 4
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x; i < nv; i += step) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + i);
            const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const double d = to_float(e[j]);
                sum = fma(d, d, sum);
            }
        }
    } else {
        const int64_t step = static_cast<int64_t>(gridDim.x) * kNormThreads;
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x; i < n; i += step) {
            const double d = to_float(x[i]);
            sum = fma(d, d, sum);
        }
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) partial[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = sum;
}

// hi[z][row][0 .. ld) = FP16(v) and lo = FP16(v - hi) of v = g * scale / (norm
// + eps), columns behind n zero.
// The factor is applied as two powers of two and a value in [1, 2), so that
// neither a tiny nor a huge norm overflows or loses digits.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kNormThreads)
    cast_kernel(const T* __restrict__ g, int rows, int n, int ld, const double* __restrict__ partial, int parts,
                float eps, float scale, __half* __restrict__ hi, __half* __restrict__ lo) {
    __shared__ double red[kNormThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t z = blockIdx.y;
    const double norm = sqrt(block_sum(static_cast<int>(threadIdx.x) < parts ? partial[z * parts + threadIdx.x] : 0.0, red)) +
                        static_cast<double>(eps);
    double f = norm > 0.0 ? static_cast<double>(scale) / norm : norm == norm ? 0.0 : norm;
    float p1 = 1.0f, p2 = 1.0f, fr;
    if (f > 0.0 && f < 1e300) {
        int e;
        fr = static_cast<float>(frexp(f, &e));
        p1 = scalbnf(1.0f, e / 2);
        p2 = scalbnf(1.0f, e - e / 2);
    } else {
        fr = static_cast<float>(f);
    }
    const int64_t per_row = ld / 8, total = static_cast<int64_t>(rows) * per_row;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kNormThreads) {
        const int64_t r = i / per_row;
        const int c = static_cast<int>(i - r * per_row) * 8;
        const T* src = g + (z * rows + r) * n + c;
        float v[8];
        if (VEC) {
            constexpr int E = 16 / sizeof(T);
#pragma unroll
            for (int k = 0; k < 8 / E; ++k) {
                const uint4 q = c < n ? __ldg(reinterpret_cast<const uint4*>(src) + k) : make_uint4(0u, 0u, 0u, 0u);
                const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
                for (int j = 0; j < E; ++j) v[k * E + j] = to_float(e[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c + j < n ? to_float(src[j]) : 0.0f;
        }
        uint32_t w[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v0 = c + 2 * j < n ? v[2 * j] * p1 * p2 * fr : 0.0f;
            const float v1 = c + 2 * j + 1 < n ? v[2 * j + 1] * p1 * p2 * fr : 0.0f;
            const __half2 h = __floats2half2_rn(v0, v1);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
            const float2 back = __half22float2(h);
            const __half2 rest = __floats2half2_rn(v0 - back.x, v1 - back.y);
            l[j] = *reinterpret_cast<const uint32_t*>(&rest);
        }
        *reinterpret_cast<uint4*>(hi + (z * rows + r) * ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(lo + (z * rows + r) * ld + c) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

}  // namespace ns
}  // namespace fp8blk
