// Newton-Schulz orthogonalisation of small matrices in one launch: a shorter
// side s of up to 128 and a longer side l of up to 8192 as far as a CTA's shared
// memory holds an eighth of it, which is 2432 at s = 128, 6528 at 64 and all at 48
// (the iteration and its roundings are newton_schulz.cuh's).
//
// There every product is a launch, and on matrices this small a launch is all
// there is: some 5.5 us of set-up, first load, epilogue and exit for well under a
// microsecond of products, 85 to 105 us for five steps.  Here a cluster of 1 to 8
// CTAs keeps one matrix in shared memory for all steps, X as s x l (a tall matrix
// transposed), each CTA a share of the longer side.  Per step
//   S       each CTA's share of X X^T; the CTAs add up each other's FP32 shares
//           (a slice of S each, in rank order) through distributed shared memory
//           and hand the FP16 result back to all
//   Q       computed by every CTA for itself
//   X       each CTA its own columns
// The products go through mma.sync: their operands change hands between products
// in the registers' layout, and at a few hundred thousand multiply-adds per SM and
// product the tensor memory's round trip would cost more than its rate gains.
// Bound by latency: barriers, fragment loads and, for s near 128, mma.sync's rate.
// One matrix, five steps, against the launch per product (us, graph replay):
//   17 x 17    13 against 63      64 x 500   31 against 87      128 x 1000   68 against 105
//   64 x 64    17 against 68     128 x 128   43 against 82      128 x 2048   95 against 120
//   32 x 1000  25 against 90     128 x 500   63 against 98     2000 x 100    82 against 124
//   32 x 4096  41 against 105     64 x 4096  61 against 107     128 x 2112  102 against 120
//   32 x 8192  66 against 120     64 x 6144  82 against 117      96 x 3500   94 against 128
// (The entry point says how many matrices at a time are worth it.)  Of a step's 21,000
// clocks at 128 x 1000, S takes 3,000, its exchange 9,000, Q 4,300 and X 5,300.
#pragma once

#include "newton_schulz.cuh"

namespace fp8blk {
namespace ns {
namespace small {

constexpr int kMaxShort = 128, kMaxLong = 8192, kMaxRanks = 8;
constexpr int kTiles = 4;                         // of 16 x 16, a warp's piece of a product at a time
constexpr int kThreads = 512;
constexpr int kMaxSteps = 32;
constexpr int kMaxShortOfAnyBatch = 80;           // up to here one launch takes any batch
constexpr int kLeastShare = 128;                  // columns of X per CTA, at least (where there are as many)

struct Params {
    int m, n;                   // the matrix as it lies in memory
    int s, l;                   // shorter and longer side
    int tall;                   // more rows than columns
    int ranks, share;           // CTAs per matrix; columns of X per CTA (a multiple of 16)
    int apart;                  // the FP32 share of S lies over Q alone
    int steps;
    float eps, scale;           // X is kept times scale
    float coeff[3 * kMaxSteps];
};

__host__ __device__ constexpr int up16(int v) { return (v + 15) / 16 * 16; }
// Shared memory: X_hi and X_lo [sp][share + 8], then S and Q [sp][sp + 8] or, over
// both, the FP32 share of S [sp][sp + 4].  (Rows of 16 bytes more than a multiple
// of 32 spread a fragment's rows over all banks.)
__host__ __device__ constexpr int x_bytes(int sp, int share) { return sp * (share + 8) * 2; }
__host__ __device__ constexpr int s_bytes(int sp) { return sp * (sp + 8) * 2; }
constexpr int smem_bytes(int s, int share) { return 2 * x_bytes(up16(s), share) + 2 * s_bytes(up16(s)); }
// The same with the FP32 share over Q and what follows: S may then be handed round
// while others still read their shares, which saves one barrier of the cluster (64 x 500: 33 to
// 31 us, 128 x 1000: 70 to 68).
constexpr int smem_bytes_apart(int s, int share) {
    return 2 * x_bytes(up16(s), share) + s_bytes(up16(s)) + 4 * up16(s) * (up16(s) + 4);
}
constexpr int kMaxSmem = 227 * 1024 - 1024;       // what a CTA may have, without the static part

inline bool takes(int64_t m, int64_t n) {
    const int64_t s = m < n ? m : n, l = m < n ? n : m;
    return s <= kMaxShort && l <= kMaxLong &&
           smem_bytes(static_cast<int>(s), up16(static_cast<int>(l + kMaxRanks - 1) / kMaxRanks)) <= kMaxSmem;
}

// Whether a batch takes one launch whatever the number of clusters that run at
// once (the exceptions concern matrices of several CTAs, of more than 80 rows, in
// more than one round).
inline bool always_takes(int64_t batch, int64_t m, int64_t n) {
    const int64_t s = m < n ? m : n, l = m < n ? n : m;
    return takes(m, n) && (batch == 1 || s <= kMaxShortOfAnyBatch || l <= kLeastShare);
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// acc = 16 rows of A times NT tiles of 16 columns of B, over `steps` times 16 of k;
// pa, pb: this lane's row of the first fragments, `tile` and `step` bytes on for the
// next tile and the next 16 of k.
template <int NT, bool B_K>
__device__ __forceinline__ void product_of(float (&acc)[2 * kTiles][4], uint32_t pa, uint32_t pb, uint32_t tile, uint32_t step,
                                           int steps) {
#pragma unroll 2
    for (int k = 0; k < steps; ++k) {
        uint32_t fa[4], fb[NT][4];
        ldmatrix4<false>(fa, pa + 32 * k);
#pragma unroll
        for (int t = 0; t < NT; ++t) ldmatrix4<!B_K>(fb[t], pb + k * step + t * tile);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mma16816(acc[2 * t], fa, fb[t][0], fb[t][1]);
            mma16816(acc[2 * t + 1], fa, fb[t][2], fb[t][3]);
        }
    }
}

// acc = rows r0 .. + 15 of A times `tiles` (1 to kTiles) tiles of 16 columns of B
// from c0 on, over k < K.  A: [row][k], rows of lda.  B: [column][k] (B_K) or
// [k][column], rows of ldb.
template <bool B_K>
__device__ __forceinline__ void product(float (&acc)[2 * kTiles][4], const __half* a, int lda, int r0, const __half* b, int ldb,
                                        int c0, int tiles, int K, int lane) {
#pragma unroll
    for (int t = 0; t < 2 * kTiles; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][j] = 0.0f;
    const uint32_t pa = smem_u32(a + (r0 + (lane & 15)) * lda + (lane >> 4) * 8);
    const uint32_t pb = smem_u32(B_K ? b + (c0 + (lane & 7) + ((lane >> 4) << 3)) * ldb + ((lane >> 3) & 1) * 8
                                     : b + ((lane & 7) + ((lane >> 3) & 1) * 8) * ldb + c0 + (lane >> 4) * 8);
    const uint32_t tile = (B_K ? 16 * ldb : 16) * 2, step = (B_K ? 16 : 16 * ldb) * 2;      // bytes
    static_assert(kTiles == 4, "one case each");
    switch (tiles) {                       // the same for the warp
        case 1: product_of<1, B_K>(acc, pa, pb, tile, step, K / 16); break;
        case 2: product_of<2, B_K>(acc, pa, pb, tile, step, K / 16); break;
        case 3: product_of<3, B_K>(acc, pa, pb, tile, step, K / 16); break;
        default: product_of<4, B_K>(acc, pa, pb, tile, step, K / 16); break;
    }
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint2 v) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    iterate_kernel(const T* __restrict__ g, __nv_bfloat16* __restrict__ out, const __grid_constant__ Params p) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ double red[kThreads / 32], share_sum;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = p.ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t at = static_cast<int64_t>(blockIdx.x / p.ranks) * p.m * p.n;
    const int sp = up16(p.s), ldx = p.share + 8, lds = sp + 8, ldp = sp + 4;
    const int c0 = rank * p.share, cl = min(p.share, p.l - c0), lp = up16(cl);      // this CTA's columns
    __half* xh = reinterpret_cast<__half*>(smem_raw);
    __half* xl = xh + sp * ldx;
    __half* S = xl + sp * ldx;
    __half* Q = S + sp * lds;
    float* part = reinterpret_cast<float*>(p.apart ? Q : S);
    static_assert(4 * (kMaxShort + 4) <= 2 * 2 * (kMaxShort + 8), "the FP32 share lies over S and Q");

    griddep_launch_dependents();
    griddep_wait();
    // column j of this CTA's part of X begins at j, or j n of a tall matrix
    const int64_t dj = p.tall ? p.n : 1;
    const T* src = g + at + c0 * dj;
    const int inner = p.tall ? p.s : cl, outer = p.tall ? cl : p.s;        // along and across memory's rows
    for (int e = t; e < 2 * sp * ldx / 8; e += kThreads) reinterpret_cast<uint4*>(xh)[e] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    // One pass over memory, eight rows' loads at a time: the norm, and the elements'
    // upper and lower halves into X_hi's and X_lo's places.
    constexpr int kAtOnce = 8;
    double sum = 0.0;
    for (int o = warp; o < outer; o += kAtOnce * (kThreads / 32))
        for (int i = lane; i < inner; i += 32) {
            float v[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int r = o + q * (kThreads / 32);
                v[q] = r < outer ? to_float(src[static_cast<int64_t>(r) * p.n + i]) : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int r = o + q * (kThreads / 32);
                sum = fma(static_cast<double>(v[q]), static_cast<double>(v[q]), sum);
                if (r < outer) {
                    const uint32_t u = __float_as_uint(v[q]);
                    const int at_x = p.tall ? i * ldx + r : r * ldx + i;
                    reinterpret_cast<uint16_t*>(xh)[at_x] = static_cast<uint16_t>(u >> 16);
                    reinterpret_cast<uint16_t*>(xl)[at_x] = static_cast<uint16_t>(u);
                }
            }
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) sum += red[w];
    if (p.ranks > 1) {
        if (t == 0) share_sum = sum;
        cluster_sync();
        sum = 0.0;
        for (int r = 0; r < p.ranks; ++r) sum += ld_cluster_f64(map_to_cta(smem_u32(&share_sum), static_cast<uint32_t>(r)));
    }
    const Factor f(sqrt(sum) + static_cast<double>(p.eps), p.scale);
    for (int e = t; e < sp * ldx / 2; e += kThreads) {       // two elements where they are; what is padding stays 0
        uint32_t& h = reinterpret_cast<uint32_t*>(xh)[e];
        uint32_t& l = reinterpret_cast<uint32_t*>(xl)[e];
        const float v0 = f(__uint_as_float((h << 16) | (l & 0xFFFFu))), v1 = f(__uint_as_float((h & 0xFFFF0000u) | (l >> 16)));
        const __half2 hi = __floats2half2_rn(v0, v1);
        const float2 back2 = __half22float2(hi);
        const __half2 lo = __floats2half2_rn(v0 - back2.x, v1 - back2.y);
        h = *reinterpret_cast<const uint32_t*>(&hi);
        l = *reinterpret_cast<const uint32_t*>(&lo);
    }
    __syncthreads();

    // a warp's piece of a product: 16 rows, and its group's share of the columns
    // (as many groups as there are warps for)
    const int row_tiles = sp / 16, groups = kThreads / 32 / row_tiles, group = warp % groups;
    const int r0 = warp / groups * 16;
    const int fr = lane >> 2, fc = 2 * (lane & 3);                        // its fragment's row and column
    const int s_first = group * row_tiles / groups, s_c0 = 16 * s_first;
    const int s_tiles = r0 < sp ? (group + 1) * row_tiles / groups - s_first : 0;
    // X in as many passes over its columns as leave a warp kTiles at most
    const int passes = (lp / 16 + groups * kTiles - 1) / (groups * kTiles), x_pass = (lp / 16 + passes - 1) / passes;
    const float alpha = 1.0f / (p.scale * p.scale), back = 1.0f / p.scale;

    for (int k = 0; k < p.steps; ++k) {
        const float a = p.coeff[3 * k], b = p.coeff[3 * k + 1], c = p.coeff[3 * k + 2];
        const bool lin = k <= kCarry, last = k == p.steps - 1;
        // ------------------------------------------------------------------ S
        if (s_tiles > 0) {
            float acc[2 * kTiles][4];
            product<true>(acc, xh, ldx, r0, xh, ldx, s_c0, s_tiles, lp, lane);
#pragma unroll
            for (int u = 0; u < 2 * kTiles; ++u) {
                if (u < 2 * s_tiles)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = r0 + fr + 8 * h, col = s_c0 + 8 * u + fc;
                    if (p.ranks > 1)
                        *reinterpret_cast<float2*>(part + row * ldp + col) = make_float2(acc[u][2 * h], acc[u][2 * h + 1]);
                    else
                        *reinterpret_cast<__half2*>(S + row * lds + col) =
                            __floats2half2_rn(acc[u][2 * h] * alpha, acc[u][2 * h + 1] * alpha);
                }
            }
        }
        if (p.ranks > 1) {
            cluster_sync();                // every share is in
            // this rank's rows of S: a warp has a row, a lane 4 columns of it
            const int rows = (sp + p.ranks - 1) / p.ranks, first = rank * rows, end = min(first + rows, sp);
            constexpr int kPasses = kMaxShort / 2 / (kThreads / 32);       // (two ranks: 64 rows each)
            uint2 v[kPasses];
#pragma unroll
            for (int q = 0; q < kPasses; ++q) {
                const int row = first + warp + q * (kThreads / 32);
                if (row < end && 4 * lane < sp) {
                    const uint32_t from = smem_u32(part + row * ldp + 4 * lane);
                    float4 o[kMaxRanks];       // loaded together, added in rank order
#pragma unroll
                    for (int r = 0; r < kMaxRanks; ++r)
                        o[r] = r < p.ranks ? ld_cluster_v4(map_to_cta(from, static_cast<uint32_t>(r))) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float4 w = o[0];
#pragma unroll
                    for (int r = 1; r < kMaxRanks; ++r) w = make_float4(w.x + o[r].x, w.y + o[r].y, w.z + o[r].z, w.w + o[r].w);
                    const __half2 lo = __floats2half2_rn(w.x * alpha, w.y * alpha), hi = __floats2half2_rn(w.z * alpha, w.w * alpha);
                    v[q] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
                }
            }
            if (!p.apart) cluster_sync();  // every share has been read: S may take its place
#pragma unroll
            for (int q = 0; q < kPasses; ++q) {
                const int row = first + warp + q * (kThreads / 32);
                if (row < end && 4 * lane < sp) {
                    const uint32_t to = smem_u32(S + row * lds + 4 * lane);
                    for (int r = 0; r < p.ranks; ++r) st_cluster_v2(map_to_cta(to, static_cast<uint32_t>(r)), v[q]);
                }
            }
            cluster_sync();                // S is whole everywhere
        } else {
            __syncthreads();
        }
        // ------------------------------------------------------------------ Q
        if (s_tiles > 0) {
            float acc[2 * kTiles][4];
            product<false>(acc, S, lds, r0, S, lds, s_c0, s_tiles, sp, lane);
#pragma unroll
            for (int u = 0; u < 2 * kTiles; ++u) {
                if (u < 2 * s_tiles)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = r0 + fr + 8 * h, col = s_c0 + 8 * u + fc;
                    const float2 s2 = __half22float2(*reinterpret_cast<const __half2*>(S + row * lds + col));
                    const float diag = lin ? 0.0f : a;
                    const float q0 = fmaf(c, acc[u][2 * h], b * s2.x) + (row == col ? diag : 0.0f);
                    const float q1 = fmaf(c, acc[u][2 * h + 1], b * s2.y) + (row == col + 1 ? diag : 0.0f);
                    *reinterpret_cast<__half2*>(Q + row * lds + col) = __floats2half2_rn(q0, q1);
                }
            }
        }
        __syncthreads();
        // ------------------------------------------------------------------ X
        for (int from = 0; from < lp / 16; from += x_pass) {
            const int tiles = min(x_pass, lp / 16 - from), first = group * tiles / groups;
            const int x_tiles = r0 < sp ? (group + 1) * tiles / groups - first : 0, x_c0 = 16 * (from + first);
            float acc[2 * kTiles][4];
            if (x_tiles > 0) product<false>(acc, Q, lds, r0, xh, ldx, x_c0, x_tiles, sp, lane);
            __syncthreads();               // every warp has read these columns of X
            if (x_tiles > 0) {
#pragma unroll
                for (int u = 0; u < 2 * kTiles; ++u) {
                    if (u < 2 * x_tiles)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = r0 + fr + 8 * h, col = x_c0 + 8 * u + fc, o = row * ldx + col;
                        float2 v = make_float2(acc[u][2 * h], acc[u][2 * h + 1]);
                        if (lin) {
                            const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(xh + o));
                            const float2 l2 = __half22float2(*reinterpret_cast<const __half2*>(xl + o));
                            v = make_float2(fmaf(a, h2.x + l2.x, v.x), fmaf(a, h2.y + l2.y, v.y));
                        }
                        if (!last) {
                            const __half2 hi = __floats2half2_rn(v.x, v.y);
                            *reinterpret_cast<__half2*>(xh + o) = hi;
                            if (k < kCarry) {
                                const float2 f2 = __half22float2(hi);
                                *reinterpret_cast<__half2*>(xl + o) = __floats2half2_rn(v.x - f2.x, v.y - f2.y);
                            }
                        } else {           // the result, in X's place
                            *reinterpret_cast<__nv_bfloat162*>(xh + o) = __floats2bfloat162_rn(v.x * back, v.y * back);
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
    __nv_bfloat16* dst = out + at + c0 * dj;
    for (int r = warp; r < outer; r += kThreads / 32)
        for (int i = lane; i < inner; i += 32)
            dst[static_cast<int64_t>(r) * p.n + i] = *reinterpret_cast<const __nv_bfloat16*>(xh + (p.tall ? i * ldx + r : r * ldx + i));
    if (p.ranks > 1) cluster_sync();       // nobody leaves while its shared memory is read
}

}  // namespace small
}  // namespace ns
}  // namespace fp8blk
