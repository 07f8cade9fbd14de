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
// its 11 bits round 8 times finer than bfloat16's at the same speed.  The first
// X, whose entries are near 1 / sqrt(m n) and would reach FP16's subnormals, is
// kept multiplied by the power of two below sqrt(m n); the first step's
// epilogues take it out again.  S, Q and X are each rounded once per step; a I
// is added to Q before its rounding, so X needs no second read.  The result is
// rounded to bfloat16.
//
// One GEMM kernel, C = A B^T in 256 x 256 tiles of CTA pairs, persistent:
//   warp 0     operands by TMA into a ring of 64-deep stages
//   warp 1     tcgen05.mma.cta_group::2.kind::f16 into one of two 256-column
//              TMEM accumulators (leader CTA)
//   warps 4-11 epilogue: thread = one row, 128 columns; the other accumulator
//              fills meanwhile
// S and Q are symmetric: only tiles on or above the diagonal are computed, and
// the epilogue stores each also transposed.
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
constexpr uint32_t kProducerSleepNs = 64;

enum Mode : int { kGram = 0, kPoly = 1, kApply = 2 };

struct Params {
    int M, N, K;                // output rows, output columns, contraction
    int tiles_m, tiles_n;       // 256 x 256 tiles
    int tiles;                  // per matrix (upper triangle for kGram, kPoly)
    int batch;
    int row_fast;               // kApply: tiles of one column panel in a row (else of one row panel)
    float alpha;                // kGram, kApply: the accumulator's factor
    float a, b, c;              // kPoly
    const __half* s;            // kPoly: S [batch][N][s_ld]
    int64_t s_ld;
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

// Matrix, tile row and tile column of a tile index.
template <int MODE>
__device__ __forceinline__ void tile_at(const Params& p, int tile, int& z, int& tm, int& tn) {
    z = tile / p.tiles;
    int i = tile - z * p.tiles;
    if (MODE == kApply) {
        if (p.row_fast) {
            tn = i / p.tiles_m;
            tm = i - tn * p.tiles_m;
        } else {
            tm = i / p.tiles_n;
            tn = i - tm * p.tiles_n;
        }
    } else {                               // upper triangle, row by row
        tm = 0;
        while (i >= p.tiles_n - tm) {
            i -= p.tiles_n - tm;
            ++tm;
        }
        tn = tm + i;
    }
}

// tmA, tmB: operands, [batch][rows][cols] FP16; box 64 x 128 (contraction
// contiguous) or 64 x 64 (A_MN, B_MN: contraction along rows), 128-byte
// swizzle.  tmC: output, box 64 x 32, 128-byte swizzle.  tmT: the same output,
// box 32 x 64, not swizzled (the transposed tile; kGram and kPoly).
template <int MODE, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmT, const Params p) {
    constexpr uint32_t IDESC = idesc_f16_f32(2 * BM, BN, A_MN, B_MN);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();            // 0 = leader of the pair
    const int pair = blockIdx.x >> 1;
    const int npairs = gridDim.x >> 1;
    const int total = p.tiles * p.batch;
    const int num_kb = (p.K + BK - 1) / BK;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const uint32_t full = sbase + OFF_BARS, empty = full + 8 * STAGES, tfull = empty + 8 * STAGES,
                   tempty = tfull + 16, drain = tempty + 16;

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
            for (int tile = pair; ok && tile < total; tile += npairs) {
                int z, tm, tn;
                tile_at<MODE>(p, tile, z, tm, tn);
                const int m0 = tm * 2 * BM + static_cast<int>(rank) * BM;
                const int n0 = tn * BN + static_cast<int>(rank) * (BN / 2);
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait(empty + 8 * s, ((it / STAGES) & 1) ^ 1, abort_flag, p.wait_ns, kErrTimeout,
                                   kProducerSleepNs)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + s * STAGE_BYTES, bar = full_leader + 8 * s;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * STAGE_BYTES);
                    if (A_MN) {
                        tma_load_3d_pair(dst, &tmA, m0, kb * BK, z, bar);
                        tma_load_3d_pair(dst + BOX_BYTES, &tmA, m0 + 64, kb * BK, z, bar);
                    } else {
                        tma_load_3d_pair(dst, &tmA, kb * BK, m0, z, bar);
                    }
                    if (B_MN) {
                        tma_load_3d_pair(dst + A_BYTES, &tmB, n0, kb * BK, z, bar);
                        tma_load_3d_pair(dst + A_BYTES + BOX_BYTES, &tmB, n0 + 64, kb * BK, z, bar);
                    } else {
                        tma_load_3d_pair(dst + A_BYTES, &tmB, kb * BK, n0, z, bar);
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
            for (int tile = pair; ok && tile < total; tile += npairs, ++n) {
                const int buf = n & 1;
                if (!mbar_wait(tempty + 8 * buf, ((n >> 1) & 1) ^ 1, abort_flag, p.wait_ns, kErrTimeout)) break;
                const uint32_t d_tmem = tmem_base + buf * BN;
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
                        mma_f16_pair(d_tmem, a_desc + k * adv_a, b_desc + k * adv_b, IDESC, (kb | k) != 0 ? 1u : 0u);
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
        const int half = ew >> 2;              // which 128 of the 256 columns
        const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t tempty_leader = map_to_cta(tempty, 0);
        uint8_t* stage = smem + OFF_OUT + ew * 2 * OUT_BYTES;
        const uint32_t stage_addr = smem_u32(stage);
        int n = 0;
        for (int tile = pair; tile < total; tile += npairs, ++n) {
            int z, tm, tn;
            tile_at<MODE>(p, tile, z, tm, tn);
            const int buf = n & 1;
            const int row0 = tm * 2 * BM + static_cast<int>(rank) * BM + quarter * 32;
            const int row = row0 + lane;
            const bool got = mbar_wait(tfull + 8 * buf, (n >> 1) & 1, abort_flag, p.wait_ns, kErrTimeout);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col0 = tn * BN + half * 128 + h * 64;
                uint32_t r0[32], r1[32];
                const uint32_t taddr = lane_base + buf * BN + half * 128 + h * 64;
                tmem_ld_32x32b_x32(taddr, r0);
                tmem_ld_32x32b_x32(taddr + 32, r1);
                uint4 sv[8];
                if (MODE == kPoly) {
                    const bool in = row < p.M && col0 < p.s_ld;
                    const uint4* sp = reinterpret_cast<const uint4*>(p.s + (static_cast<int64_t>(z) * p.M + row) * p.s_ld + col0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sv[j] = in ? __ldg(sp + j) : make_uint4(0u, 0u, 0u, 0u);
                }
                tmem_ld_wait();
                if (h == 1) {                  // the accumulator may be refilled
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0)
                            mbar_arrive(tempty + 8 * buf);
                        else
                            mbar_arrive_remote(tempty_leader + 8 * buf);
                    }
                }
                uint32_t w[32];                // the row's 64 results, two per word
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float v0 = __uint_as_float(j < 16 ? r0[2 * j] : r1[2 * j - 32]);
                    float v1 = __uint_as_float(j < 16 ? r0[2 * j + 1] : r1[2 * j - 31]);
                    if (MODE == kPoly) {
                        const uint32_t sw = reinterpret_cast<const uint32_t*>(&sv[j >> 2])[j & 3];
                        const float2 s2 = __half22float2(*reinterpret_cast<const __half2*>(&sw));
                        v0 = fmaf(p.c, v0, p.b * s2.x) + (row == col0 + 2 * j && row < p.M ? p.a : 0.0f);
                        v1 = fmaf(p.c, v1, p.b * s2.y) + (row == col0 + 2 * j + 1 && row < p.M ? p.a : 0.0f);
                    } else {
                        v0 *= p.alpha;
                        v1 *= p.alpha;
                    }
                    if (MODE == kApply && p.final_out) {
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v0, v1);
                        w[j] = *reinterpret_cast<const uint32_t*>(&b2);
                    } else {
                        const __half2 h2 = __floats2half2_rn(v0, v1);
                        w[j] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                }
                if (lane == 0) bulk_wait_group_read0();          // the previous stores have read the staging
                __syncwarp();
                const bool normal = row0 < p.M && col0 < p.N;
                const bool mirror = MODE != kApply && tm != tn && normal;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_shared_v4(stage_addr + lane * 128 + ((c ^ (lane & 7)) << 4),
                                 make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
                if (mirror) {
                    uint16_t* tr = reinterpret_cast<uint16_t*>(stage + OUT_BYTES) + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        tr[(2 * j) * 32] = static_cast<uint16_t>(w[j]);
                        tr[(2 * j + 1) * 32] = static_cast<uint16_t>(w[j] >> 16);
                    }
                }
                if (MODE == kApply && p.out) {
                    // rows that TMA cannot store: 32 lanes along each row
                    __syncwarp();
                    for (int i = 0; i < 32; ++i) {
                        if (row0 + i >= p.M) break;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int c = lane + 32 * u;
                            if (col0 + c < p.N) {
                                const uint8_t* src = stage + i * 128 + (((c >> 3) ^ (i & 7)) << 4) + (c & 7) * 2;
                                p.out[(static_cast<int64_t>(z) * p.M + row0 + i) * p.N + col0 + c] =
                                    *reinterpret_cast<const __nv_bfloat16*>(src);
                            }
                        }
                    }
                    __syncwarp();
                } else {
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (normal) tma_store_3d(&tmC, stage_addr, col0, row0, z);
                        if (mirror) tma_store_3d(&tmT, stage_addr + OUT_BYTES, row0, col0, z);
                        bulk_commit_group();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_group0();                 // output stores complete
        __syncwarp();
    }

    griddep_launch_dependents();
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
    griddep_launch_dependents();
}

// x[z][row][0 .. ld) = FP16(g * scale / (norm + eps)), columns behind n zero.
// The factor is applied as two powers of two and a value in [1, 2), so that
// neither a tiny nor a huge norm overflows or loses digits.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kNormThreads)
    cast_kernel(const T* __restrict__ g, int rows, int n, int ld, const double* __restrict__ partial, int parts,
                float eps, float scale, __half* __restrict__ x) {
    __shared__ double red[kNormThreads / 32];
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
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v0 = c + 2 * j < n ? v[2 * j] * p1 * p2 * fr : 0.0f;
            const float v1 = c + 2 * j + 1 < n ? v[2 * j + 1] * p1 * p2 * fr : 0.0f;
            const __half2 h = __floats2half2_rn(v0, v1);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(x + (z * rows + r) * ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    griddep_launch_dependents();
}

}  // namespace ns
}  // namespace fp8blk
