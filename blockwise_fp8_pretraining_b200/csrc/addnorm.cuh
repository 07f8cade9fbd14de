// Residual addition, RMSNorm and the E4M3 quantization of its output in one
// pass over the data, and the gradient through the norm.
//
//   s    = bf16(x + residual)                  (s = x without a residual)
//   r    = fp32(1 / sqrt(mean_k s[k]^2 + eps))   per row, FP64 sum of squares
//   y[k] = bf16(gamma[k] * bf16(fp32(s[k] * r)))
//   codes and scales of y in 1x128 groups (and 128x1 groups along tokens)
//
// (rmsnorm.cuh has the same r and y for a given x; here the row's values stay
// on the chip between the statistic and the quantization, so s is read zero
// times instead of twice.)  bf16(x + residual) and bf16(gamma * t) are one
// packed bfloat16 instruction each: a single rounding to nearest even of the
// exact sum or product, subnormals kept.
//
// Gradient, with n = s r and g = gamma dy for the gradient dy of y, the
// roundings of the forward pass passed straight through:
//   ds     = r (g - n mean_k(g n)) + dresidual
//   dgamma = sum over rows of dy n
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"
#include "quantize.cuh"

namespace fp8blk {
namespace addnorm {

constexpr int kMaxCols = 16384;      // longest row the kernels hold on the chip

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) { return as_u32(__hadd2_rn(as_bf162(a), as_bf162(b))); }
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return as_u32(__hmax2(as_bf162(a), as_bf162(b))); }
__device__ __forceinline__ uint32_t abs2(uint32_t a) { return a & 0x7FFF7FFFu; }

// Sum of the squares of two bf16, added to acc in FP64 (each square exact).
__device__ __forceinline__ double sumsq2(uint32_t w, double acc) {
    const float2 f = unpack_bf16x2(w);
    const double a = f.x, b = f.y;
    return fma(b, b, fma(a, a, acc));
}

// y of two elements: gamma * bf16(s * r), each rounding to nearest even.
__device__ __forceinline__ uint32_t norm2(uint32_t s, float r, uint32_t gamma) {
    const float2 f = unpack_bf16x2(s);
    const __nv_bfloat162 t = __floats2bfloat162_rn(__fmul_rn(f.x, r), __fmul_rn(f.y, r));
    return as_u32(__hmul2_rn(as_bf162(gamma), t));
}

__device__ __forceinline__ float rstd_of(double sum, int64_t cols, float eps) {
    return static_cast<float>(1.0 / sqrt(sum / static_cast<double>(cols) + static_cast<double>(eps)));
}

// Codes of the 8 values of a chunk, one scale.
__device__ __forceinline__ uint2 encode8_group(const uint4& y, float s) {
    const Quotient q(s);
    if (q.fast) {
        const QuotientPair p(q, q);
        return make_uint2(p.codes(y.x) | (p.codes(y.y) << 16), p.codes(y.z) | (p.codes(y.w) << 16));
    }
    return make_uint2(codes_pair_general(y.x, q, q) | (codes_pair_general(y.y, q, q) << 16),
                      codes_pair_general(y.z, q, q) | (codes_pair_general(y.w, q, q) << 16));
}

// ------------------------------------------------------- groups along rows

// A row is held by `wpr` warps, CPL chunks of 8 elements per lane; a block
// holds blockDim / 32 / wpr rows (a whole number).  A 1x128 group is 16
// consecutive chunks, a half-warp, so only the row's sum of squares crosses
// warps.  Any number of rows.  q == nullptr leaves the quantization out (s and
// r only).  sum_out may be x or residual: every element is read and then
// written by one thread.
template <int CPL, int MAX_THREADS>
__global__ void __launch_bounds__(MAX_THREADS)
    row_kernel(const uint4* x, const uint4* residual, const uint4* __restrict__ gamma, int64_t rows, int chunks,
               float eps, int wpr, uint4* sum_out, float* __restrict__ rstd,
               uint2* __restrict__ q, float* __restrict__ s_row) {
    __shared__ double red[32];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int teams = (blockDim.x >> 5) / wpr;
    const int team = warp / wpr, tw = warp - team * wpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * teams + team;
    griddep_wait();                    // inputs of the preceding kernel are complete
    if (row < rows) {                  // the same for a whole team
        const int64_t base = row * chunks;
        const int c0 = tw * CPL * 32 + lane;
        uint4 s[CPL];
#pragma unroll
        for (int i = 0; i < CPL; ++i)
            s[i] = (c0 + 32 * i < chunks) ? x[base + c0 + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
        if (residual) {
            uint4 e[CPL];
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                e[i] = (c0 + 32 * i < chunks) ? residual[base + c0 + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                s[i] = make_uint4(add2(s[i].x, e[i].x), add2(s[i].y, e[i].y), add2(s[i].z, e[i].z), add2(s[i].w, e[i].w));
                if (c0 + 32 * i < chunks) sum_out[base + c0 + 32 * i] = s[i];
            }
        }
        double sq = 0.0;
#pragma unroll
        for (int i = 0; i < CPL; ++i) sq = sumsq2(s[i].w, sumsq2(s[i].z, sumsq2(s[i].y, sumsq2(s[i].x, sq))));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (wpr > 1) {
            if (lane == 0) red[warp] = sq;
            named_bar_sync(1 + team, 32 * wpr);
            sq = 0.0;
            for (int w = 0; w < wpr; ++w) sq += red[team * wpr + w];
        }
        const float r = rstd_of(sq, static_cast<int64_t>(chunks) * 8, eps);
        if (tw == 0 && lane == 0) rstd[row] = r;
        if (q) {
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                const int c = c0 + 32 * i;
                const uint4 g = (c < chunks) ? __ldg(gamma + c) : make_uint4(0u, 0u, 0u, 0u);
                const uint4 y = make_uint4(norm2(s[i].x, r, g.x), norm2(s[i].y, r, g.y), norm2(s[i].z, r, g.z),
                                           norm2(s[i].w, r, g.w));
                const float sc = group_scale(halfwarp_max(amax8_packed(y)));
                if (c < chunks) {
                    q[base + c] = encode8_group(y, sc);
                    if ((lane & 15) == 0) s_row[static_cast<int64_t>(c >> 4) * rows + row] = sc;
                }
            }
        }
    }
    griddep_launch_dependents();
}

// ------------------------------------------- groups along tokens (and rows)

constexpr int kTileThreads = 512;

// Rows of a value held by the lanes of a warp, 8 per lane, folded over the
// warp: afterwards lane l holds (in v[0]) the fold of row fold_row(l) over
// all 32 lanes.  Three halving steps exchange half of the rows each, two more
// combine what is left.
__device__ __forceinline__ int fold_row(int lane) { return ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1); }
__device__ __forceinline__ int fold_lane(int row) { return ((row >> 2) & 1) * 16 + ((row >> 1) & 1) * 8 + (row & 1) * 4; }

template <typename T, typename Op>
__device__ __forceinline__ T fold8(T (&v)[8], int lane, Op op) {
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        const int half = 4 >> step, mask = 16 >> step;
        const bool up = (lane & mask) != 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < half) {
                const T send = up ? v[j] : v[j + half];
                const T keep = up ? v[j + half] : v[j];
                v[j] = op(keep, __shfl_xor_sync(0xffffffffu, send, mask));
            }
        }
    }
    T a = v[0];
    a = op(a, __shfl_xor_sync(0xffffffffu, a, 2));
    return op(a, __shfl_xor_sync(0xffffffffu, a, 1));
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

// A cluster of CTAs holds 128 rows; each CTA holds TPC tiles of 128 columns in
// registers (tile `rank + k * ranks`, the last ones of some CTAs empty).  Warp
// w holds rows 8 w .. 8 w + 7 of a tile, lane l columns 4 l .. 4 l + 3, so
// loads, s and the row codes are whole 128- or 256-byte runs of a row.  The
// CTAs exchange their rows' partial sums of squares through distributed shared
// memory (added in rank order), and then each quantizes its own tiles: row
// groups by shuffles, column groups through shared memory, the transposed
// codes staged there to leave in 128-byte runs.
template <int TPC>
__global__ void __launch_bounds__(kTileThreads, TPC <= 2 ? 2 : 1)
    tile_kernel(const __nv_bfloat16* x, const __nv_bfloat16* residual, const __nv_bfloat16* __restrict__ gamma,
                int64_t rows, int64_t cols, float eps, int ranks, __nv_bfloat16* sum_out,
                float* __restrict__ rstd, uint8_t* __restrict__ q_row,
                float* __restrict__ s_row, uint8_t* __restrict__ q_colT, float* __restrict__ s_col) {
    __shared__ double part[kGroup];
    __shared__ float rrow[kGroup];
    __shared__ __align__(16) uint2 colmax[16][32];       // [warp][lane]: maxima of 4 columns over 8 rows
    __shared__ float2 colq[kGroup];                      // a column's scale and its reciprocal
    __shared__ __align__(16) uint8_t stage[kGroup * kGroup];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / ranks) * kGroup;
    const int tiles = static_cast<int>(cols / kGroup);
    griddep_wait();                    // inputs of the preceding kernel are complete

    uint2 v[TPC][8];
    double sq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sq[i] = 0.0;
#pragma unroll
    for (int k = 0; k < TPC; ++k) {
        const int tile = rank + k * ranks;
        if (tile < tiles) {
            const int64_t at = (row0 + 8 * warp) * cols + tile * kGroup + 4 * lane;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = *reinterpret_cast<const uint2*>(x + at + i * cols);
            if (residual) {
                uint2 e[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = *reinterpret_cast<const uint2*>(residual + at + i * cols);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[k][i] = make_uint2(add2(v[k][i].x, e[i].x), add2(v[k][i].y, e[i].y));
                    *reinterpret_cast<uint2*>(sum_out + at + i * cols) = v[k][i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) sq[i] = sumsq2(v[k][i].y, sumsq2(v[k][i].x, sq[i]));
        }
    }
    {
        const double a = fold8(sq, lane, [](double p, double q) { return p + q; });
        if ((lane & 3) == 0) part[8 * warp + fold_row(lane)] = a;
    }
    cluster_sync();                    // every rank's partial sums are in
    if (t < kGroup) {
        double a = 0.0;
        const uint32_t mine = smem_u32(&part[t]);
        for (int k = 0; k < ranks; ++k) a += ld_cluster_f64(map_to_cta(mine, static_cast<uint32_t>(k)));
        const float r = rstd_of(a, cols, eps);
        rrow[t] = r;
        if (rank == 0) rstd[row0 + t] = r;
    }
    __syncthreads();
    // this CTA has read the others' sums; it leaves only when all have
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

#pragma unroll
    for (int k = 0; k < TPC; ++k) {
        const int tile = rank + k * ranks;
        if (tile >= tiles) break;      // the same for the whole CTA
        const uint2 g = __ldg(reinterpret_cast<const uint2*>(gamma + tile * kGroup + 4 * lane));
        uint2 cm = make_uint2(0u, 0u);
        uint32_t rm[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float r = rrow[8 * warp + i];
            v[k][i] = make_uint2(norm2(v[k][i].x, r, g.x), norm2(v[k][i].y, r, g.y));
            const uint32_t a = abs2(v[k][i].x), b = abs2(v[k][i].y);
            rm[i] = max2(a, b);
            cm = make_uint2(max2(cm.x, a), max2(cm.y, b));
        }
        if (q_colT) colmax[warp][lane] = cm;
        if (q_row) {
            const uint32_t m = fold8(rm, lane, [](uint32_t p, uint32_t q) { return max2(p, q); });
            const float sc = group_scale(fmaxf(bf16_lo(m), bf16_hi(m)));
            if ((lane & 3) == 0) s_row[static_cast<int64_t>(tile) * rows + row0 + 8 * warp + fold_row(lane)] = sc;
            const float rc = __frcp_rn(sc);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float si = __shfl_sync(0xffffffffu, sc, fold_lane(i));
                const Quotient q(si, __shfl_sync(0xffffffffu, rc, fold_lane(i)));
                uint32_t code;
                if (q.fast) {
                    const QuotientPair p(q, q);
                    code = p.codes(v[k][i].x) | (p.codes(v[k][i].y) << 16);
                } else {
                    code = codes_pair_general(v[k][i].x, q, q) | (codes_pair_general(v[k][i].y, q, q) << 16);
                }
                *reinterpret_cast<uint32_t*>(q_row + (row0 + 8 * warp + i) * cols + tile * kGroup + 4 * lane) = code;
            }
        }
        if (!q_colT) continue;
        __syncthreads();
        if (t < kGroup) {              // column t of the tile
            const uint16_t* cmp = reinterpret_cast<const uint16_t*>(&colmax[0][0]) + t;
            uint32_t m = 0;            // maxima of absolute values: their bits order like integers
#pragma unroll
            for (int w = 0; w < 16; ++w) m = max(m, static_cast<uint32_t>(cmp[w * kGroup]));
            const float sc = group_scale(__uint_as_float(m << 16));
            colq[t] = make_float2(sc, __frcp_rn(sc));
            s_col[(row0 / kGroup) * cols + tile * kGroup + t] = sc;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 c = colq[4 * lane + j];
            const Quotient q(c.x, c.y);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = j < 2 ? v[k][2 * i].x : v[k][2 * i].y;
                const uint32_t b = j < 2 ? v[k][2 * i + 1].x : v[k][2 * i + 1].y;
                w[i] = __byte_perm(a, b, (j & 1) ? 0x7632 : 0x5410);    // two tokens of the column
            }
            uint2 o;
            if (q.fast) {
                const QuotientPair p(q, q);
                o = make_uint2(p.codes(w[0]) | (p.codes(w[1]) << 16), p.codes(w[2]) | (p.codes(w[3]) << 16));
            } else {
                o = make_uint2(codes_pair_general(w[0], q, q) | (codes_pair_general(w[1], q, q) << 16),
                               codes_pair_general(w[2], q, q) | (codes_pair_general(w[3], q, q) << 16));
            }
            // the column's 16 runs of 8 tokens, run w at w ^ (column / 4 % 16):
            // the half-warp's 16 columns then fill all banks
            *reinterpret_cast<uint2*>(stage + (4 * lane + j) * kGroup + ((warp ^ (lane & 15)) << 3)) = o;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = t + i * kTileThreads;          // 16 bytes: column u / 8, tokens 16 (u % 8) ..
            const int c = u >> 3, key = (c >> 2) & 15;
            const uint4 o = *reinterpret_cast<const uint4*>(stage + c * kGroup + ((((u & 7) * 2) ^ (key & 14)) << 3));
            const uint4 out = (key & 1) ? make_uint4(o.z, o.w, o.x, o.y) : o;
            *reinterpret_cast<uint4*>(q_colT + (static_cast<int64_t>(tile) * kGroup + c) * rows + row0 + 16 * (u & 7)) = out;
        }
    }
    griddep_launch_dependents();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ gradient

constexpr int kBwdThreads = 256;     // most threads of a block

// A row is held by `wpr` warps, CPT chunks of 8 elements per lane; a block
// has blockDim / 32 / wpr such teams (a whole number; several only with CPT ==
// 1).  Each team walks over rows, R at once, keeping its columns' part of
// dgamma in FP32 registers; the block's teams are added in order at the end
// and leave as one row of `partial` (or as dgamma itself when the grid is one
// block).  ds may be dy or dres: every element is read and then written by
// one thread.
template <int CPT, int R>
__global__ void __launch_bounds__(kBwdThreads)
    bwd_kernel(const uint4* dy, const uint4* __restrict__ s, const float* __restrict__ rstd,
               const uint4* __restrict__ gamma, const uint4* dres, int64_t rows, int chunks, int wpr, uint4* ds,
               float* __restrict__ partial, float* __restrict__ dgamma, int accumulate) {
    __shared__ float red[2][kBwdThreads / 32][R];
    __shared__ float gsum[CPT == 1 ? kBwdThreads * 8 : 1];   // [team][column]
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int teams = (blockDim.x >> 5) / wpr;
    const int team = warp / wpr, tw = warp - team * wpr;
    const int c0 = tw * CPT * 32 + lane;
    const float inv = 1.0f / (8.0f * static_cast<float>(chunks));
    griddep_wait();                    // inputs of the preceding kernel are complete

    uint4 gm[CPT];
    float acc[CPT][8];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        gm[i] = (c0 + 32 * i < chunks) ? __ldg(gamma + c0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R;
    int buf = 0;
    for (int64_t row = (static_cast<int64_t>(blockIdx.x) * teams + team) * R; row < rows; row += step, buf ^= 1) {
        uint4 vd[R][CPT], vs[R][CPT], ve[R][CPT];
        float r[R], dot[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const bool live = row + a < rows;
            const int64_t base = (row + a) * chunks + c0;
            r[a] = live ? __ldg(rstd + row + a) : 0.0f;
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const bool in = live && c0 + 32 * i < chunks;
                vd[a][i] = in ? dy[base + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
                vs[a][i] = in ? __ldg(s + base + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
                ve[a][i] = in && dres ? dres[base + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
            }
        }
#pragma unroll
        for (int a = 0; a < R; ++a) {
            dot[a] = 0.0f;
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const uint32_t* dw = reinterpret_cast<const uint32_t*>(&vd[a][i]);
                const uint32_t* sw = reinterpret_cast<const uint32_t*>(&vs[a][i]);
                const uint32_t* gw = reinterpret_cast<const uint32_t*>(&gm[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = unpack_bf16x2(dw[j]), f = unpack_bf16x2(sw[j]), g = unpack_bf16x2(gw[j]);
                    const float p0 = d.x * (f.x * r[a]), p1 = d.y * (f.y * r[a]);    // dy n
                    acc[i][2 * j] += p0;
                    acc[i][2 * j + 1] += p1;
                    dot[a] = fmaf(g.y, p1, fmaf(g.x, p0, dot[a]));
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int a = 0; a < R; ++a) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
        if (wpr > 1) {
            if (lane == 0)
#pragma unroll
                for (int a = 0; a < R; ++a) red[buf][warp][a] = dot[a];
            named_bar_sync(1 + team, 32 * wpr);
#pragma unroll
            for (int a = 0; a < R; ++a) {
                dot[a] = 0.0f;
                for (int w = 0; w < wpr; ++w) dot[a] += red[buf][team * wpr + w][a];
            }
        }
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const float m = dot[a] * inv;
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const uint32_t* dw = reinterpret_cast<const uint32_t*>(&vd[a][i]);
                const uint32_t* sw = reinterpret_cast<const uint32_t*>(&vs[a][i]);
                const uint32_t* ew = reinterpret_cast<const uint32_t*>(&ve[a][i]);
                const uint32_t* gw = reinterpret_cast<const uint32_t*>(&gm[i]);
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = unpack_bf16x2(dw[j]), f = unpack_bf16x2(sw[j]), g = unpack_bf16x2(gw[j]),
                                 e = unpack_bf16x2(ew[j]);
                    const float a0 = fmaf(-(f.x * r[a]), m, g.x * d.x), a1 = fmaf(-(f.y * r[a]), m, g.y * d.y);
                    o[j] = as_u32(__floats2bfloat162_rn(fmaf(r[a], a0, e.x), fmaf(r[a], a1, e.y)));
                }
                if (row + a < rows && c0 + 32 * i < chunks)
                    ds[(row + a) * chunks + c0 + 32 * i] = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    if (dgamma) {
        const int cols = 8 * chunks;
        float* out = gridDim.x == 1 ? dgamma : partial + static_cast<int64_t>(blockIdx.x) * cols;
        const bool add = gridDim.x == 1 && accumulate;
        if (CPT == 1 && teams > 1) {
            if (c0 < chunks)
#pragma unroll
                for (int j = 0; j < 8; ++j) gsum[team * cols + 8 * c0 + j] = acc[0][j];
            __syncthreads();
            for (int c = threadIdx.x; c < cols; c += blockDim.x) {
                float a = 0.0f;
                for (int k = 0; k < teams; ++k) a += gsum[k * cols + c];
                out[c] = add ? out[c] + a : a;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CPT; ++i)
                if (c0 + 32 * i < chunks)
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        float4* o = reinterpret_cast<float4*>(out + 8 * (c0 + 32 * i) + j);
                        float4 a = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
                        if (add) {
                            const float4 b = *o;
                            a = make_float4(b.x + a.x, b.y + a.y, b.z + a.z, b.w + a.w);
                        }
                        *o = a;
                    }
        }
    }
    griddep_launch_dependents();
}

// dgamma (+)= the sum of the blocks' partial rows, in a fixed order: 32
// columns per block, the rows dealt out to its 8 warps.
__global__ void __launch_bounds__(256) dgamma_kernel(const float* __restrict__ partial, int parts, int cols,
                                                     float* __restrict__ dgamma, int accumulate) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    griddep_wait();
    float a = 0.0f;
#pragma unroll 8
    for (int p = warp; p < parts; p += 8) a += __ldcg(partial + static_cast<int64_t>(p) * cols + c);
    sums[warp][lane] = a;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int w = 1; w < 8; ++w) a += sums[w][lane];
        dgamma[c] = accumulate ? dgamma[c] + a : a;
    }
    griddep_launch_dependents();
}

}  // namespace addnorm
}  // namespace fp8blk
