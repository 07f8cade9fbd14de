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
//   warps 0, 2 operands by TMA into a ring of 64-deep stages, every other stage
//              each (one thread needs about 260 clocks for a stage's barriers
//              and 46 for each copy; a stage's products take 512)
//   warp 1     tcgen05.mma.cta_group::2.kind::f16 into one of two 256-column
//              TMEM accumulators (leader CTA)
//   warps 4-11 epilogue: thread = one row, 128 columns; the other accumulator
//              fills meanwhile
// S and Q are symmetric: only tiles on or above the diagonal are computed, and
// the epilogue stores each also transposed.
//
// The tiles of a last, partly filled wave are cut where there are pairs for the
// pieces: into two halves of 128 columns, whose epilogues are half as long (their
// stages hardly are: with both operands in shared memory its bandwidth, 32 KB
// written and 32 to 48 KB read a stage, bounds a stage of 256 columns at 576
// clocks, where the tensor cores need 512, and one of 128 columns still at 505, by
// two issuing threads; by one its commits hold it at 576), and along the
// contraction, where the parts before the last leave their FP32 sums in the
// workspace and the pair with the last one adds them in order.
//
// On a B200, five steps: [12288, 2048] FP32 782 us (1.04 PFLOP/s, the symmetric
// products' halves counted once; a library product of that size runs at 1.33
// PFLOP/s on the same data, held by the power limit), [2048, 6144] 470 us, [4096,
// 2048] 378 us, [2048, 2048] 272 us; over a second of runs, the clock then at 1.57
// GHz, 920, 540, 406 and 272.  A product's stages take 0.30 us each at full clock (the tensor
// cores' 512 clocks are 0.27); around them stand about 1.5 us until the first
// operands arrive, 2 to 4 us of epilogue and 1.5 us between kernels, which is
// what bounds matrices of a few hundred rows ([6, 520, 1100] 195 us, 13 us a
// product).  Smaller ones take one launch for all steps (newton_schulz_small.cuh).
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
constexpr uint32_t kProducerSleepNs = 64, kEpilogueSleepNs = 128;

enum Mode : int { kGram = 0, kPoly = 1, kApply = 2 };

struct Params {
    int M, N, K;                // output rows, output columns, contraction
    int tiles_m, tiles_n;       // 256 x 256 tiles
    int tiles;                  // per matrix (upper triangle for kGram, kPoly)
    int full;                   // tiles (of all matrices) taken whole
    int halves, parts;          // into which each tile behind those is cut: columns, contraction
    int units;                  // full + halves * parts * others
    int row_fast;               // kApply: tiles of one column panel in a row (else of one row panel)
    float alpha;                // kGram: the accumulator's factor; kApply: the final output's
    float a, b, c;              // kPoly: Q = a I + b S + c S S; kApply: a of the linear term
    const __half* e0;           // kPoly: S; kApply: X_hi of the linear term, or null
    const __half* e1;           // kApply: X_lo of the linear term
    int64_t e_ld;               // their row stride ([batch][M][e_ld])
    int carry;                  // kApply: also store what the FP16 rounding leaves of X (tmT)
    int final_out;              // kApply: bfloat16 output
    __nv_bfloat16* out;         // final output by plain stores (its rows not 16-byte multiples), else null
    float4* sums;               // [slot][CTA][epilogue warp][4 chunks][8][lane]: partial sums
    int* flags;                 // [slot][CTA][epilogue warp]: the product whose partial sums are there
    int product;                // 1, 2, .. within a call
    uint64_t wait_ns;
};

constexpr int kMaxParts = 8;               // of one tile
// What a tile costs besides its stages, in stages (0.3 us): the epilogue 6 us,
// leaving partial sums 3 us, adding each 1 us.
constexpr int kEpilogue = 20, kHandOver = 12, kAddPart = 4;
constexpr int kSlots = 74;                 // partial sums at once, at most
constexpr int kSlotFloat4 = 2 * EPI_WARPS * 4 * 8 * 32;

// How `rest` tiles of num_kb stages are best cut for `pairs` pairs, with room
// for `slots` partial sums.
struct Cut {
    int halves, parts;
};
inline Cut best_cut(int64_t rest, int pairs, int num_kb, int slots) {
    Cut best = {1, 1};
    int least = num_kb + kEpilogue;
    for (int h = 1; h <= 2; ++h)
        for (int c = 1; c <= kMaxParts && c <= num_kb && h * c * rest <= pairs && h * (c - 1) * rest <= slots; ++c) {
            const int cost = (num_kb + c - 1) / c + (kEpilogue + (c > 1 ? kHandOver + kAddPart * (c - 1) : 0)) / h;
            if (cost < least) {
                best = {h, c};
                least = cost;
            }
        }
    return best;
}
// Partial sums a product of `tiles` tiles may leave, whatever the number of pairs.
inline int slots_for(int64_t tiles, int64_t num_kb) {
    if (num_kb <= kHandOver + kAddPart) return 0;       // (half of what is saved goes into handing over)
    const int64_t most = 2 * tiles * (kMaxParts - 1);
    return static_cast<int>(most < kSlots ? most : kSlots);
}

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

// One unit of work: output rows row0 .. + 255, columns col0 .. + cols - 1 (256,
// or 128 for half a tile or where the matrix ends there) of matrix z, over
// stages kb0 .. kb1 - 1 of the contraction.  diag: a tile on the diagonal, which
// is not mirrored.  slot: the first partial sum of these columns.
struct Unit {
    int z, row0, col0, cols, kb0, kb1, part, slot;
    bool diag;
};

// Unit u, or false where half a tile lies behind the matrix.
template <int MODE>
__device__ __forceinline__ bool unit_at(const Params& p, int num_kb, int u, Unit& w) {
    int tile = u, sub = 0;
    w.cols = BN;
    w.part = w.slot = w.kb0 = 0;
    w.kb1 = num_kb;
    if (u >= p.full) {
        const int v = u - p.full, piece = v / p.parts;     // piece: columns of a tile
        w.part = v - piece * p.parts;
        w.slot = piece * (p.parts - 1);
        w.kb0 = w.part * num_kb / p.parts;
        w.kb1 = (w.part + 1) * num_kb / p.parts;
        tile = p.full + piece / p.halves;
        sub = piece % p.halves;
        if (p.halves == 2) w.cols = BN / 2;
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

__device__ __forceinline__ void st_release_flag(int* addr, int v) {
    asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_acquire_flag(const int* addr) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float2 half2_at(const uint4& v, int i) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Wait, no longer than limit_ns, until *flag is `want`.
__device__ __forceinline__ bool flag_wait(const int* flag, int want, volatile int* abort, uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; ld_acquire_flag(flag) != want; ++it) {
        if ((it & 15u) != 0) continue;
        if (*abort) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) {
            t0 = now;
        } else if (now - t0 > limit_ns) {
            record_error(kErrTimeout);
            *abort = 1;
            return false;
        }
    }
    return true;
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

    if (warp == 0 || warp == 2) {
        // -------------------------------------------------------- operands
        if (lane == 0) {
            const uint32_t full_leader = map_to_cta(full, 0);
            const int odd = warp >> 1;         // this warp's stages: the odd or the even ones of the block's sequence
            int it = 0;                        // stages of the block so far
            int st = odd, ph = 1;              // this warp's next stage in the ring, and its parity
            int mine = 0;                      // stages this warp has requested
            bool ok = true;
            Unit w;
            for (int u = pair; ok && u < p.units; u += npairs) {
                if (!unit_at<MODE>(p, num_kb, u, w)) continue;
                const int m0 = w.row0 + static_cast<int>(rank) * BM;
                const int n0 = w.col0 + static_cast<int>(rank) * (w.cols / 2);
                const bool whole = w.cols == BN;
                const uint32_t bytes = 2 * (A_BYTES + (w.cols / 2) * BK * 2);
                for (int kb = w.kb0 + ((it ^ odd) & 1); kb < w.kb1; kb += 2) {
                    if (!mbar_wait(empty + 8 * st, ph, abort_flag, p.wait_ns, kErrTimeout, kProducerSleepNs)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + st * STAGE_BYTES, bar = full_leader + 8 * st;
                    const int k = kb * BK;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * st, bytes);
                    if (A_MN) {
                        tma_load_3d_pair(dst, &tmA, m0, k, w.z, bar);
                        tma_load_3d_pair(dst + BOX_BYTES, &tmA, m0 + 64, k, w.z, bar);
                    } else {
                        tma_load_3d_pair(dst, &tmA, k, m0, w.z, bar);
                    }
                    if (B_MN) {
                        tma_load_3d_pair(dst + A_BYTES, &tmB, n0, k, w.z, bar);
                        if (whole) tma_load_3d_pair(dst + A_BYTES + BOX_BYTES, &tmB, n0 + 64, k, w.z, bar);
                    } else {
                        tma_load_3d_pair(dst + A_BYTES, &tmB, k, n0, w.z, bar);
                        if (whole) tma_load_3d_pair(dst + A_BYTES + BOX_BYTES, &tmB, k, n0 + 64, w.z, bar);
                    }
                    ++mine;
                    if ((st += 2) >= STAGES) {
                        st -= STAGES;
                        ph ^= 1;
                    }
                }
                it += w.kb1 - w.kb0;
            }
            if (!ok && rank == 0) {
                // let every copy this warp has requested land (both CTAs'
                // copies complete on the leader's barriers) before the pair exits
                for (int j = max(0, mine - STAGES); j < mine; ++j) {
                    const int i = 2 * j + odd;
                    drain_wait(full + 8 * (i % STAGES), (i / STAGES) & 1, p.wait_ns);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer (leader)
        if (lane == 0 && rank == 0) {
            int n = 0, st = 0, ph = 0;
            bool ok = true;
            Unit w;
            for (int u = pair; ok && u < p.units; u += npairs) {
                if (!unit_at<MODE>(p, num_kb, u, w)) continue;
                const int buf = n & 1;
                if (!mbar_wait(tempty + 8 * buf, ((n >> 1) & 1) ^ 1, abort_flag, p.wait_ns, kErrTimeout)) break;
                ++n;
                const uint32_t d_tmem = tmem_base + buf * BN;
                const uint32_t idesc = w.cols == BN ? idesc_f16_f32(2 * BM, BN, A_MN, B_MN)
                                                    : idesc_f16_f32(2 * BM, BN / 2, A_MN, B_MN);
                bool ready = mbar_try_wait(full + 8 * st, ph);
                for (int kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!ready && !mbar_wait(full + 8 * st, ph, abort_flag, p.wait_ns, kErrTimeout)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = sbase + st * STAGE_BYTES, done = empty + 8 * st;
                    const uint64_t a_desc = A_MN ? smem_desc_mn64_sw128(a_addr) : smem_desc_k128_sw128(a_addr);
                    const uint64_t b_desc =
                        B_MN ? smem_desc_mn64_sw128(a_addr + A_BYTES) : smem_desc_k128_sw128(a_addr + A_BYTES);
                    if (++st == STAGES) {
                        st = 0;
                        ph ^= 1;
                    }
                    // 16 of the contraction: 32 bytes along a swizzled row, or 16 rows of 128 bytes
                    constexpr uint64_t adv_a = (A_MN ? 16 * 128 : 32) >> 4, adv_b = (B_MN ? 16 * 128 : 32) >> 4;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_f16_pair(d_tmem, a_desc + k * adv_a, b_desc + k * adv_b, idesc, (kb > w.kb0 || k > 0) ? 1u : 0u);
                    mma_commit_pair(done, 0x3);
                    ready = kb + 1 < w.kb1 && mbar_try_wait(full + 8 * st, ph);    // (asked while these products run)
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
            if (!unit_at<MODE>(p, num_kb, u, w)) continue;
            const int buf = n & 1;
            const int row0 = w.row0 + static_cast<int>(rank) * BM + quarter * 32;
            const int row = row0 + lane;
            const int cbase = w.col0 + half * (w.cols / 2);
            const int chunks = min(w.cols / 64, 2 * ((max(p.N - cbase, 0) + 63) / 64));      // of 32 columns: whole boxes
            const bool last_part = u < p.full || w.part == p.parts - 1;
            const int others = w.part;             // partial sums to add
            // this warp's piece of partial sum `part`
            auto sums = [&](int part) {
                return p.sums + (static_cast<int64_t>(w.slot + part) * 2 * EPI_WARPS + rank * EPI_WARPS + ew) * (4 * 8 * 32) + lane;
            };
            auto flag = [&](int part) { return p.flags + (w.slot + part) * 2 * EPI_WARPS + rank * EPI_WARPS + ew; };
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
            if (last_part) fetch(cbase);
            bool got = mbar_wait(tfull + 8 * buf, (n >> 1) & 1, abort_flag, p.wait_ns, kErrTimeout, kEpilogueSleepNs);
            if (!__all_sync(0xffffffffu, got)) break;
            ++n;
            tc_fence_after();
            if (last_part && others > 0) {
                if (lane < others) got = flag_wait(flag(lane), p.product, abort_flag, p.wait_ns);
                if (!__all_sync(0xffffffffu, got)) break;
                __syncwarp();                      // what its lanes acquired holds for the warp (a vote orders no memory)
            }
            auto release = [&] {                   // the accumulator may be refilled
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0)
                        mbar_arrive(tempty + 8 * buf);
                    else
                        mbar_arrive_remote(tempty_leader + 8 * buf);
                }
            };
            if (chunks == 0) release();
#pragma unroll 1
            for (int ch = 0; ch < chunks; ++ch) {
                const int col = cbase + 32 * ch;
                uint32_t r[32];
                tmem_ld_32x32b_x32(lane_base + buf * BN + half * (w.cols / 2) + 32 * ch, r);
                tmem_ld_wait();
                if (ch == chunks - 1) release();
                if (!last_part) {
                    float4* dst = sums(w.part) + ch * (8 * 32);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        __stcg(dst + j * 32, make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                                         __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
                    continue;
                }
                for (int q = 0; q < others; ++q) {
                    const float4* src = sums(q) + ch * (8 * 32);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 v = __ldcg(src + j * 32);
                        r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + v.x);
                        r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + v.y);
                        r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + v.z);
                        r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + v.w);
                    }
                }
                // (branches outside the loops: inside them each costs the epilogue more than the arithmetic)
                float2 v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    v[j] = make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    if (MODE == kGram) v[j] = __fmul2_rn(v[j], make_float2(p.alpha, p.alpha));
                    if (MODE == kPoly)
                        v[j] = __ffma2_rn(make_float2(p.c, p.c), v[j],
                                          __fmul2_rn(make_float2(p.b, p.b), half2_at(e[(j >> 2) % NE], j & 3)));
                }
                if (MODE == kPoly && row0 == col) {                        // a I: each lane's own column
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[j].x += lane == 2 * j ? p.a : 0.0f;
                        v[j].y += lane == 2 * j + 1 ? p.a : 0.0f;
                    }
                }
                if (lin) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = __ffma2_rn(make_float2(p.a, p.a),
                                          __fadd2_rn(half2_at(e[(j >> 2) % NE], j & 3), half2_at(e[(4 + (j >> 2)) % NE], j & 3)),
                                          v[j]);
                }
                uint32_t o[16], lo[16];            // the row's 32 results, two per word
                if (MODE == kApply && p.final_out) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[j].x * p.alpha, v[j].y * p.alpha);
                        o[j] = *reinterpret_cast<const uint32_t*>(&b2);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __half2 h2 = __floats2half2_rn(v[j].x, v[j].y);
                        o[j] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                }
                if (MODE == kApply && p.carry) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&o[j]));
                        const __half2 l2 = __floats2half2_rn(v[j].x - back.x, v[j].y - back.y);
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
            if (!last_part) {
                __syncwarp();
                if (lane == 0) st_release_flag(flag(w.part), p.product);
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

constexpr int kNormBlocks = 1024;           // at most, per matrix
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

// Multiplication by scale / norm, as two powers of two and a value in [0.5, 1), so
// that neither a tiny nor a huge norm overflows or loses digits.  A zero norm
// gives zeros, a non-finite one NaN.
struct Factor {
    float p1 = 1.0f, p2 = 1.0f, fr;
    __device__ __forceinline__ Factor(double norm, float scale) {
        const double f = norm > 0.0 ? static_cast<double>(scale) / norm : norm == norm ? 0.0 : norm;
        if (f > 0.0 && f < 1e300) {
            int e;
            fr = static_cast<float>(frexp(f, &e));
            p1 = scalbnf(1.0f, e / 2);
            p2 = scalbnf(1.0f, e - e / 2);
        } else {
            fr = static_cast<float>(f);
        }
    }
    __device__ __forceinline__ float operator()(float v) const { return v * p1 * p2 * fr; }
};

// hi[z][row][0 .. ld) = FP16(v) and lo = FP16(v - hi) of v = g * scale / (norm
// + eps), columns behind n zero.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kNormThreads)
    cast_kernel(const T* __restrict__ g, int rows, int n, int ld, const double* __restrict__ partial, int parts,
                float eps, float scale, __half* __restrict__ hi, __half* __restrict__ lo, int* __restrict__ flags,
                int num_flags) {
    __shared__ double red[kNormThreads / 32];
    griddep_launch_dependents();
    griddep_wait();
    const int64_t z = blockIdx.y;
    if (blockIdx.x == 0 && z == 0)         // no product's partial sums are there yet
        for (int i = threadIdx.x; i < num_flags; i += kNormThreads) flags[i] = 0;
    double mine = 0.0;
    for (int i = threadIdx.x; i < parts; i += kNormThreads) mine += partial[z * parts + i];
    const Factor factor(sqrt(block_sum(mine, red)) + static_cast<double>(eps), scale);
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
            const float v0 = c + 2 * j < n ? factor(v[2 * j]) : 0.0f;
            const float v1 = c + 2 * j + 1 < n ? factor(v[2 * j + 1]) : 0.0f;
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
