// Residual addition, RMSNorm and the E4M3 quantization of its output, and the
// gradient through the norm.
//
//   s    = bf16(x + residual)                  (s = x without a residual)
//   r    = fp32(1 / sqrt(mean_k s[k]^2 + eps))   per row, FP64 sum of squares
//   y[k] = bf16(gamma[k] * bf16(fp32(s[k] * r)))
//   codes and scales of y in 1x128 groups (and 128x1 groups along tokens)
//
// (rmsnorm.cuh has the same r and y for a given x; here a row's values stay on
// the chip between the statistic and the row-wise codes, so s is read zero
// times instead of twice.  Groups along tokens take a second launch, which reads
// s from the L2 cache.)  bf16(x + residual) and bf16(gamma * t) are one packed
// bfloat16 instruction each: a single rounding to nearest even of the exact sum
// or product, subnormals kept.
//
// All of it is bound by HBM: x, the residual, s and the codes, 6 to 8 bytes an
// element.  On a B200, [8192, 2048]: row-wise 22.3 us (5.3 TB/s, 0.82 of a plain
// copy's rate), both groupings 31.8 us; [1037, 6144] row-wise 11.5 us; one token
// 2.1 us.
//
// Gradient, with n = s r and g = gamma dy for the gradient dy of y, the
// roundings of the forward pass passed straight through:
//   ds     = r (g - n mean_k(g n)) + dresidual
//   dgamma = sum over rows of dy n
// 8 bytes an element; [8192, 2048] 27.4 us (4.9 TB/s) with the launch that adds up
// the blocks' shares of dgamma (about 3 us).
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

// fp32(1 / sqrt(sum / cols + eps)).  Inside FP32's range one Newton step in FP64
// from rsqrtf's answer (off by 2^-22 at most) leaves a relative error of 3/2
// 2^-44: the rounding to FP32 then differs from the exact value's in one of a
// million rows, by one unit.  (Every lane computes it; the division and square
// root in FP64 were a fifth of the kernel's instructions.)
__device__ __forceinline__ float rstd_of(double sum, int64_t cols, float eps) {
    const double v = fma(sum, 1.0 / static_cast<double>(cols), static_cast<double>(eps));
    if (v > 1e-30 && v < 1e30) {
        const double y = rsqrtf(static_cast<float>(v));
        return static_cast<float>(fma(0.5 * y, fma(-v * y, y, 1.0), y));
    }
    return static_cast<float>(1.0 / sqrt(v));
}

// amax / 448 rounded to nearest, as group_scale: the residual of the product
// with RN(1 / 448) corrects it (exact as long as nothing underflows).
__device__ __forceinline__ float scale_of(float amax) {
    if (amax < 0x1p-100f) return group_scale(amax);
    constexpr float r = 1.0f / 448.0f;
    const float q = amax * r;
    return fmaf(fmaf(-448.0f, q, amax), r, q);
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

// Few rows: a block per row, CPL chunks of 8 elements per lane.  A 1x128
// group is 16 consecutive chunks, a half-warp, so only the row's sum of squares
// crosses warps.  q == nullptr leaves the quantization out (s and r only).
// sum_out may be x or residual: every element is read and then written by one
// thread.
template <int CPL>
__global__ void __launch_bounds__(1024)
    row_kernel(const uint4* x, const uint4* residual, const uint4* __restrict__ gamma, int64_t rows, int chunks,
               float eps, uint4* sum_out, float* __restrict__ rstd, uint2* __restrict__ q, float* __restrict__ s_row) {
    __shared__ double red[32];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int warps = blockDim.x >> 5;
    const int64_t row = blockIdx.x;
    const int64_t base = row * chunks;
    const int c0 = warp * CPL * 32 + lane;
    griddep_launch_dependents();
    griddep_wait();                    // inputs of the preceding kernel are complete
    uint4 s[CPL], e[CPL], g[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        const bool in = c0 + 32 * i < chunks;
        s[i] = in ? x[base + c0 + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
        e[i] = in && residual ? residual[base + c0 + 32 * i] : make_uint4(0u, 0u, 0u, 0u);
        g[i] = in && q ? __ldg(gamma + c0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
    double sq = 0.0;
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
        if (residual) {
            s[i] = make_uint4(add2(s[i].x, e[i].x), add2(s[i].y, e[i].y), add2(s[i].z, e[i].z), add2(s[i].w, e[i].w));
            if (c0 + 32 * i < chunks) sum_out[base + c0 + 32 * i] = s[i];
        }
        sq = sumsq2(s[i].w, sumsq2(s[i].z, sumsq2(s[i].y, sumsq2(s[i].x, sq))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (warps > 1) {
        if (lane == 0) red[warp] = sq;
        __syncthreads();
        sq = 0.0;
        for (int w = 0; w < warps; ++w) sq += red[w];
    }
    const float r = rstd_of(sq, static_cast<int64_t>(chunks) * 8, eps);
    if (threadIdx.x == 0) rstd[row] = r;
    if (q) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) {
            const int c = c0 + 32 * i;
            const uint4 y = make_uint4(norm2(s[i].x, r, g[i].x), norm2(s[i].y, r, g[i].y), norm2(s[i].z, r, g[i].z),
                                       norm2(s[i].w, r, g[i].w));
            const float sc = scale_of(halfwarp_max(amax8_packed(y)));
            if (c < chunks) {
                q[base + c] = encode8_group(y, sc);
                if ((lane & 15) == 0) s_row[static_cast<int64_t>(c >> 4) * rows + row] = sc;
            }
        }
    }
}

// Many rows: a block stays and walks over rows, R per team at once, with the
// loads of its next rows in flight while it works on these (R * CPL = 2 or 4
// chunks of x and of the residual per lane: 2 leave room for 24 warps per SM, 4
// hold longer rows with 16).  A row is held by `wpr` warps; a block has
// blockDim / 32 / wpr such teams (a whole number).  Groups and aliasing as above;
// red is double buffered, so one barrier per step keeps its readers and writers
// apart.
template <int CPL, int R> constexpr int kStreamThreads = CPL * R == 2 ? 384 : 512;   // most threads of a block
template <int CPL, int R> constexpr int kStreamBlocks = CPL * R == 2 ? 2 : 1;         // of which an SM holds these

template <int CPL, int R>
__global__ void __launch_bounds__(kStreamThreads<CPL, R>, kStreamBlocks<CPL, R>)
    stream_kernel(const uint4* x, const uint4* residual, const uint4* __restrict__ gamma, int64_t rows, int chunks,
                  float eps, int wpr, uint4* sum_out, float* __restrict__ rstd, uint2* __restrict__ q,
                  float* __restrict__ s_row) {
    __shared__ double red[2][kStreamThreads<CPL, R> / 32][R];
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int teams = (blockDim.x >> 5) / wpr;
    const int team = warp / wpr, tw = warp - team * wpr;
    const int c0 = tw * CPL * 32 + lane;
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R;
    int64_t row = (static_cast<int64_t>(blockIdx.x) * teams + team) * R;
    griddep_launch_dependents();
    griddep_wait();                    // inputs of the preceding kernel are complete

    // The next rows.  Lanes behind a row's end hold zeros throughout; rows behind
    // the last hold what was there (they are worked on and left unstored).
    uint4 nx[R][CPL], ne[R][CPL];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int i = 0; i < CPL; ++i) nx[a][i] = ne[a][i] = make_uint4(0u, 0u, 0u, 0u);
    auto fetch = [&](int64_t at) {
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                if (at + a < rows && c0 + 32 * i < chunks) {
                    const int64_t k = (at + a) * chunks + c0 + 32 * i;
                    // (read once: s, which may be read again, is to stay in the cache)
                    nx[a][i] = __ldcs(x + k);
                    if (residual) ne[a][i] = __ldcs(residual + k);
                }
            }
    };
    fetch(row);
    uint4 g[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) g[i] = q && c0 + 32 * i < chunks ? __ldg(gamma + c0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);

    for (int buf = 0; row < rows; row += step, buf ^= 1) {      // the same for a whole team
        uint4 s[R][CPL];
#pragma unroll
        for (int a = 0; a < R; ++a)
#pragma unroll
            for (int i = 0; i < CPL; ++i)
                s[a][i] = residual ? make_uint4(add2(nx[a][i].x, ne[a][i].x), add2(nx[a][i].y, ne[a][i].y),
                                                add2(nx[a][i].z, ne[a][i].z), add2(nx[a][i].w, ne[a][i].w))
                                   : nx[a][i];
        fetch(row + step);
        double sq[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            sq[a] = 0.0;
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                if (residual && row + a < rows && c0 + 32 * i < chunks) sum_out[(row + a) * chunks + c0 + 32 * i] = s[a][i];
                sq[a] = sumsq2(s[a][i].w, sumsq2(s[a][i].z, sumsq2(s[a][i].y, sumsq2(s[a][i].x, sq[a]))));
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int a = 0; a < R; ++a) sq[a] += __shfl_xor_sync(0xffffffffu, sq[a], o);
        if (wpr > 1) {
            if (lane == 0)
#pragma unroll
                for (int a = 0; a < R; ++a) red[buf][warp][a] = sq[a];
            named_bar_sync(1 + team, 32 * wpr);
#pragma unroll
            for (int a = 0; a < R; ++a) {
                sq[a] = 0.0;
                for (int w = 0; w < wpr; ++w) sq[a] += red[buf][team * wpr + w][a];
            }
        }
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const float r = rstd_of(sq[a], static_cast<int64_t>(chunks) * 8, eps);
            const bool live = row + a < rows;
            if (tw == 0 && lane == 0 && live) rstd[row + a] = r;
            if (!q) continue;
#pragma unroll
            for (int i = 0; i < CPL; ++i) {
                const int c = c0 + 32 * i;
                const uint4 v = s[a][i];
                const uint4 y = make_uint4(norm2(v.x, r, g[i].x), norm2(v.y, r, g[i].y), norm2(v.z, r, g[i].z),
                                           norm2(v.w, r, g[i].w));
                const float sc = scale_of(halfwarp_max(amax8_packed(y)));
                if (live && c < chunks) {
                    q[(row + a) * chunks + c] = encode8_group(y, sc);
                    if ((lane & 15) == 0) s_row[static_cast<int64_t>(c >> 4) * rows + row + a] = sc;
                }
            }
        }
    }
}

// ------------------------------------------------------- groups along tokens

// Codes and scales of y in 128x1 groups, from s and r: the second launch, which
// finds s in the L2 cache where it was just written.  (One launch for
// everything, a cluster of CTAs holding 128 rows in registers, took 43.6 us on
// [8192, 2048]: its cluster-wide wait for the rows' statistics left loads,
// arithmetic and stores one after the other.)
//
// A block has a 128 x 128 tile.  Warp w holds rows 16 w .. 16 w + 15, lane l
// columns 4 l .. 4 l + 3, so loads are whole 256-byte runs of a row; the
// columns' maxima meet in shared memory, and the codes are transposed there to
// leave in 128-byte runs.
constexpr int kColThreads = 256;

__global__ void __launch_bounds__(kColThreads, 4)
    col_kernel(const __nv_bfloat16* __restrict__ s, const float* __restrict__ rstd,
               const __nv_bfloat16* __restrict__ gamma, int64_t rows, int64_t cols, uint8_t* __restrict__ q_colT,
               float* __restrict__ s_col) {
    __shared__ __align__(16) uint2 colmax[8][32];        // [warp][lane]: maxima of 4 columns over 16 rows
    __shared__ float2 colq[kGroup];                      // a column's scale and its reciprocal
    __shared__ __align__(16) uint8_t stage[kGroup * kGroup];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t tiles = cols / kGroup;
    const int64_t block = blockIdx.x / tiles, tile = blockIdx.x - block * tiles;
    const int64_t row0 = block * kGroup + 16 * warp, col0 = tile * kGroup;
    griddep_launch_dependents();
    griddep_wait();                    // s and r are complete

    uint2 v[16];
    const __nv_bfloat16* src = s + row0 * cols + col0 + 4 * lane;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __ldg(reinterpret_cast<const uint2*>(src + i * cols));
    const uint2 g = __ldg(reinterpret_cast<const uint2*>(gamma + col0 + 4 * lane));
    const float rl = __ldg(rstd + row0 + (lane & 15));
    uint2 m = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float r = __shfl_sync(0xffffffffu, rl, i);
        v[i] = make_uint2(norm2(v[i].x, r, g.x), norm2(v[i].y, r, g.y));
        m = make_uint2(max2(m.x, abs2(v[i].x)), max2(m.y, abs2(v[i].y)));
    }
    colmax[warp][lane] = m;
    __syncthreads();
    if (t < kGroup) {                  // column t of the tile
        const uint16_t* cm = reinterpret_cast<const uint16_t*>(&colmax[0][0]) + t;
        uint32_t a = 0;                // maxima of absolute values: their bits order like integers
#pragma unroll
        for (int w = 0; w < 8; ++w) a = max(a, static_cast<uint32_t>(cm[w * kGroup]));
        const float sc = scale_of(__uint_as_float(a << 16));
        colq[t] = make_float2(sc, __frcp_rn(sc));
        s_col[block * cols + col0 + t] = sc;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 c = colq[4 * lane + j];
        const Quotient q(c.x, c.y);
        uint32_t w[8];                 // two tokens of the column each
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = j < 2 ? v[2 * i].x : v[2 * i].y;
            const uint32_t b = j < 2 ? v[2 * i + 1].x : v[2 * i + 1].y;
            w[i] = __byte_perm(a, b, (j & 1) ? 0x7632 : 0x5410);
        }
        uint4 o;
        if (q.fast) {
            const QuotientPair p(q, q);
            o = make_uint4(p.codes(w[0]) | (p.codes(w[1]) << 16), p.codes(w[2]) | (p.codes(w[3]) << 16),
                           p.codes(w[4]) | (p.codes(w[5]) << 16), p.codes(w[6]) | (p.codes(w[7]) << 16));
        } else {
            uint32_t* ow = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
            for (int i = 0; i < 4; ++i) ow[i] = codes_pair_general(w[2 * i], q, q) | (codes_pair_general(w[2 * i + 1], q, q) << 16);
        }
        // run w of 16 tokens at w ^ (column / 4 % 8): 8 lanes then fill all banks
        *reinterpret_cast<uint4*>(stage + (4 * lane + j) * kGroup + ((warp ^ (lane & 7)) << 4)) = o;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = t + i * kColThreads;               // 16 bytes: column u / 8, tokens 16 (u % 8) ..
        const int c = u >> 3;
        const uint4 o = *reinterpret_cast<const uint4*>(stage + c * kGroup + (((u & 7) ^ ((c >> 2) & 7)) << 4));
        *reinterpret_cast<uint4*>(q_colT + (col0 + c) * rows + block * kGroup + 16 * (u & 7)) = o;
    }
}

// ------------------------------------------------------------------ gradient

constexpr int kBwdThreads = 512;     // most threads of a block

// A row is held by `wpr` warps, CPT chunks of 8 elements per lane; a block
// has blockDim / 32 / wpr such teams (a whole number; several only in blocks of
// at most 256 threads and with CPT == 1).  Each team walks over rows, R at once,
// the loads of its next rows in flight (AHEAD) while it works on these, keeping
// its columns' part of dgamma in FP32 registers; the block's teams are added in
// order at the end and leave as one row of `partial` (or as dgamma itself when
// the grid is one block).  ds may be dy or dres: every element is read and then
// written by one thread.
template <int CPT, int R, bool AHEAD>
__global__ void __launch_bounds__(kBwdThreads, 1)
    bwd_kernel(const uint4* dy, const uint4* __restrict__ s, const float* __restrict__ rstd,
               const uint4* __restrict__ gamma, const uint4* dres, int64_t rows, int chunks, int wpr, uint4* ds,
               float* __restrict__ partial, float* __restrict__ dgamma, int accumulate) {
    __shared__ float red[2][kBwdThreads / 32][R];
    __shared__ __align__(16) float gsum[CPT == 1 ? 256 * 8 : 2];          // [team][column]
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int teams = (blockDim.x >> 5) / wpr;
    const int team = warp / wpr, tw = warp - team * wpr;
    const int c0 = tw * CPT * 32 + lane;
    const float inv = 1.0f / (8.0f * static_cast<float>(chunks));
    griddep_launch_dependents();
    griddep_wait();                    // inputs of the preceding kernel are complete

    // AHEAD: n = s r, gamma dy and gamma stay unpacked, as the next rows take the
    // loads' registers; else everything is unpacked where it is used.
    uint4 gp[CPT];
    float2 gm[CPT][4], acc[CPT][4];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        gp[i] = (c0 + 32 * i < chunks) ? __ldg(gamma + c0 + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {gp[i].x, gp[i].y, gp[i].z, gp[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            gm[i][j] = unpack_bf16x2(w[j]);
            acc[i][j] = make_float2(0.0f, 0.0f);
        }
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams * R;
    int64_t row = (static_cast<int64_t>(blockIdx.x) * teams + team) * R;
    // The next rows.  Lanes behind a row's end hold zeros throughout; a row behind
    // the last has rstd = 0, which takes it out of dgamma.
    uint4 nd[R][CPT], ns[R][CPT], ne[R][CPT];
    float nr[R];
#pragma unroll
    for (int a = 0; a < R; ++a)
#pragma unroll
        for (int i = 0; i < CPT; ++i) nd[a][i] = ns[a][i] = ne[a][i] = make_uint4(0u, 0u, 0u, 0u);
    auto fetch = [&](int64_t at) {
#pragma unroll
        for (int a = 0; a < R; ++a) {
            const bool live = at + a < rows;
            const int64_t base = (at + a) * chunks + c0;
            nr[a] = live ? __ldg(rstd + at + a) : 0.0f;
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                if (live && c0 + 32 * i < chunks) {
                    nd[a][i] = dy[base + 32 * i];
                    ns[a][i] = __ldg(s + base + 32 * i);
                    if (dres) ne[a][i] = dres[base + 32 * i];
                } else if (R > 1) {        // (its values, NaN among them, must not meet rstd = 0)
                    nd[a][i] = ns[a][i] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    };
    if (AHEAD) fetch(row);
    int buf = 0;
    for (; row < rows; row += step, buf ^= 1) {
        if (!AHEAD) fetch(row);
        float2 n[R][CPT][4], gd[R][CPT][4];      // s r and gamma dy
        uint4 ve[R][CPT];
        float r[R], dot[R];
#pragma unroll
        for (int a = 0; a < R; ++a) {
            r[a] = nr[a];
            float2 dots = make_float2(0.0f, 0.0f);
            const float2 r2 = make_float2(r[a], r[a]);
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const uint32_t dw[4] = {nd[a][i].x, nd[a][i].y, nd[a][i].z, nd[a][i].w};
                const uint32_t sw[4] = {ns[a][i].x, ns[a][i].y, ns[a][i].z, ns[a][i].w};
                const uint32_t gw[4] = {gp[i].x, gp[i].y, gp[i].z, gp[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 dv = unpack_bf16x2(dw[j]), nv = __fmul2_rn(unpack_bf16x2(sw[j]), r2);
                    const float2 gv = __fmul2_rn(AHEAD ? gm[i][j] : unpack_bf16x2(gw[j]), dv);
                    acc[i][j] = __ffma2_rn(dv, nv, acc[i][j]);
                    dots = __ffma2_rn(gv, nv, dots);
                    if (AHEAD) {
                        n[a][i][j] = nv;
                        gd[a][i][j] = gv;
                    }
                }
                if (AHEAD) ve[a][i] = ne[a][i];
            }
            dot[a] = dots.x + dots.y;
        }
        if (AHEAD) fetch(row + step);
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
            const float m = -dot[a] * inv;
            const float2 m2 = make_float2(m, m), r2 = make_float2(r[a], r[a]);
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const uint4 e = AHEAD ? ve[a][i] : ne[a][i];
                const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
                const uint32_t dw[4] = {nd[a][i].x, nd[a][i].y, nd[a][i].z, nd[a][i].w};
                const uint32_t sw[4] = {ns[a][i].x, ns[a][i].y, ns[a][i].z, ns[a][i].w};
                const uint32_t gw[4] = {gp[i].x, gp[i].y, gp[i].z, gp[i].w};
                uint32_t o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 nv = AHEAD ? n[a][i][j] : __fmul2_rn(unpack_bf16x2(sw[j]), r2);
                    const float2 gv = AHEAD ? gd[a][i][j] : __fmul2_rn(unpack_bf16x2(gw[j]), unpack_bf16x2(dw[j]));
                    const float2 v = __ffma2_rn(r2, __ffma2_rn(nv, m2, gv), unpack_bf16x2(ew[j]));
                    o[j] = as_u32(__floats2bfloat162_rn(v.x, v.y));
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
                for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(&gsum[team * cols + 8 * c0 + 2 * j]) = acc[0][j];
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
                    for (int j = 0; j < 4; j += 2) {
                        float4* o = reinterpret_cast<float4*>(out + 8 * (c0 + 32 * i) + 2 * j);
                        float4 a = make_float4(acc[i][j].x, acc[i][j].y, acc[i][j + 1].x, acc[i][j + 1].y);
                        if (add) {
                            const float4 b = *o;
                            a = make_float4(b.x + a.x, b.y + a.y, b.z + a.z, b.w + a.w);
                        }
                        *o = a;
                    }
        }
    }
}

// dgamma (+)= the sum of the blocks' partial rows, in a fixed order: 32
// columns per block, the rows dealt out to its 32 warps, whose loads are all in
// flight together.
constexpr int kDgammaWarps = 32;

__global__ void __launch_bounds__(32 * kDgammaWarps) dgamma_kernel(const float* __restrict__ partial, int parts, int cols,
                                                                   float* __restrict__ dgamma, int accumulate) {
    __shared__ float sums[kDgammaWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    griddep_launch_dependents();
    griddep_wait();
    float a = 0.0f;
#pragma unroll 16
    for (int p = warp; p < parts; p += kDgammaWarps) a += __ldcg(partial + static_cast<int64_t>(p) * cols + c);
    sums[warp][lane] = a;
    __syncthreads();
    // warp w takes column w: its 32 sums by shuffles
    a = sums[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane == 0) {
        float* out = dgamma + blockIdx.x * 32 + warp;
        *out = accumulate ? *out + a : a;
    }
}

}  // namespace addnorm
}  // namespace fp8blk
