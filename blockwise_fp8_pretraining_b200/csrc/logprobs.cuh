// Log probabilities of given tokens with the distribution's entropy and its
// most likely tokens, from one read of the logits, and the gradient of the
// logits.  For a row of logits x, with m = max x and d = x - m:
//
//   L       = log(sum_v exp(d_v))
//   logp_v  = d_v - L
//   H       = -sum_v p_v logp_v = L - (sum_v exp(d_v) d_v) / sum_v exp(d_v)
//   dx_v    = g (1[v = target] - p_v) - h p_v (logp_v + H)
//
// for the gradients g of the target's log probability and h of the entropy.  (1 -
// p of the target itself is -expm1(logp), which keeps its digits when p is near 1.)
//
// Everything is referred to the row's maximum: rows of the type's lowest value,
// or of huge values, come out right, and neither L nor H subtracts large
// numbers from each other.  The sums hold e_v = 2^(x_v k - R) with k =
// fp32(log2 e) and R = fp32(m k), one fused multiply-add per element; R is off
// m k by o = m k - R, which is known exactly and taken out at the end, so the
// reference's rounding costs nothing.  (From |m| = 2^15 on, where o would grow,
// the difference x - m is taken first and o = 0.)  The maximum's own term is
// taken out of the element stream and counted in an integer n beside the sum l
// of the others, so that L = log1p(l) keeps its digits when one token has
// almost all the probability.
//
// A row is read by a cluster of 1 to 8 CTAs (few rows are split, so that one
// row's 300 KB do not wait for one SM); a thread loads its next batch while it
// works on the last.  Each warp keeps a common maximum, each thread (n, l, sum
// e a) over its elements; the partial results meet by shuffles, shared memory
// and distributed shared memory in a fixed order, so results repeat run to run.
//
// The alternatives: every warp keeps the 32 best of its elements, one per
// lane, sorted, as 64-bit keys (order-preserving bits of the value, then the
// complement of the index, so that equal logits rank by index).  Elements
// reach the list only when they are not below a bound that k elements of the
// block are known to reach: the k-th largest of the maxima of some lanes' first
// batches, later raised to the smallest, over the block's nw warps, of the
// ceil(k / nw)-th best each warp has seen.  What is left at the end is bounded
// once more in the same way and ranked by counting, for each key, the larger ones.
// (Candidates listed in shared memory and cut by ranking instead of inserted one
// by one took up to twice as long.)
//
// Without alternatives the kernel is bound by HBM ([4096, 151936] bf16 197 us, 6.3
// TB/s; [1024, 151936] FP32 92 us, 6.7 TB/s), a few rows by the latency of one
// load and the joins (one row 5.3 us).  Alternatives add the insertions: 20 of them
// 294 us on [4096, 151936], 10.7 us on one row.  The gradient reads and writes at
// 6.7 TB/s ([4096, 151936] bf16 371 us).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "ptx.cuh"

namespace fp8blk {
namespace logp {

constexpr int kMaxThreads = 512;
constexpr int kMaxRanks = 8;
constexpr int kBatch = 4;                 // 16-byte vectors a thread works on at once
constexpr int kMaxTopK = 32;
constexpr int kTeams = 8;                 // rows per block where a row has one warp
constexpr int kPosts = 96;                // lane maxima the first bound is taken from, at most (2 kMaxTopK + 16, rounded up)
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNear = 32768.0f;         // below it in magnitude: the maxima whose product with k serves as reference
constexpr float kFloor = -61440.0f;       // (exact in bfloat16) logits below it have probability 0 beside such a maximum
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -1.0e4f;           // exp of anything below is 0
constexpr float kLowest = -3.402823466e+38f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max(a, b), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The warp's maximum; NaN is passed over.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// How a 16-byte vector of logits is unpacked.
template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    __device__ __forceinline__ static float vmax(const uint4& v) {        // NaN is passed over
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
        return fmaxf(bf16_lo(u), bf16_hi(u));
    }
    __device__ __forceinline__ static uint4 floored(uint4 v) {            // max(kFloor, x); NaN stays
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        const __nv_bfloat162 lo = __floats2bfloat162_rn(kFloor, kFloor);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), lo);
            w[i] = *reinterpret_cast<const uint32_t*>(&m);
        }
        return v;
    }
    // x with its elements equal to m (of which there are some) as -inf, their number in n
    __device__ __forceinline__ static void take_out(uint4& v, float m, float& n) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
        const uint32_t b = __float_as_uint(m) >> 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if ((w[i] & 0xFFFFu) == b) { w[i] = (w[i] & 0xFFFF0000u) | 0xFF80u; n += 1.0f; }
            if ((w[i] >> 16) == b) { w[i] = (w[i] & 0xFFFFu) | 0xFF800000u; n += 1.0f; }
        }
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[8]) {
        uint4 o;
        uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return o;
    }
    __device__ __forceinline__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ __forceinline__ static void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
    __device__ __forceinline__ static uint4 masked() { return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
};
template <> struct Elem<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static float vmax(const uint4& v) {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    __device__ __forceinline__ static uint4 floored(uint4 v) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(max_nan(__uint_as_float(w[i]), kFloor));
        return v;
    }
    __device__ __forceinline__ static void take_out(uint4& v, float m, float& n) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (w[i] == __float_as_uint(m)) { w[i] = 0xFF800000u; n += 1.0f; }
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ __forceinline__ static float load(const float* p) { return *p; }
    __device__ __forceinline__ static void store(float* p, float v) { *p = v; }
    __device__ __forceinline__ static uint4 masked() { return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u); }
};

// Elements before the first 16-byte boundary of a row.
template <typename T> __device__ __forceinline__ int64_t head_of(const T* row, int64_t n) {
    const int64_t mis = static_cast<int64_t>(reinterpret_cast<uintptr_t>(row) & 15u) / static_cast<int64_t>(sizeof(T));
    const int64_t h = mis ? Elem<T>::N - mis : 0;
    return h < n ? h : n;
}

// o of a maximum: what fp32(m k) leaves of m k (0 where x - m is taken first).
__device__ __forceinline__ float offset_of(float m) {
    return fabsf(m) < kNear ? fmaf(m, kLog2e, -__fmul_rn(m, kLog2e)) : 0.0f;
}

// Partial result over some elements: their maximum m (kLowest before the
// first finite one), how many elements equal to it the counted n are, and over
// the other elements l = sum e and sa = sum e a with a = (x - m) k + o(m), e =
// 2^a.
struct Part {
    float m, n, l, sa;
    // refer the sums to the maximum M >= m
    __device__ __forceinline__ void refer(float M) {
        if (M > m) {
            const float o = offset_of(m), top = n * ex2(o), e = l + top;
            const float shift = fmaxf(fmaf(m - M, kLog2e, offset_of(M) - o), kFar), c = ex2(shift);
            sa = c * fmaf(shift, e, fmaf(top, o, sa));
            l = c * e;
            n = 0.0f;
            m = M;
        }
    }
    __device__ __forceinline__ void add(float x) {             // one element
        refer(x);
        const float d = x - m;
        if (d == 0.0f && n == 0.0f) {
            n = 1.0f;
        } else {
            const float a = max_nan(fmaf(d, kLog2e, offset_of(m)), kFar), e = ex2(a);
            l += e;
            sa = fmaf(e, a, sa);
        }
    }
    __device__ __forceinline__ void warp_join() {
        refer(warp_max(m));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            l += __shfl_xor_sync(0xffffffffu, l, o);
            sa += __shfl_xor_sync(0xffffffffu, sa, o);
        }
    }
};

// The terms of N elements.  NEAR: |m| < kNear and the elements are floored.
template <int N, bool NEAR>
__device__ __forceinline__ void add_terms(Part& p, const float (&f)[N]) {
    const float ref = NEAR ? -__fmul_rn(p.m, kLog2e) : -p.m;
    const float2 r2 = make_float2(ref, ref), k2 = make_float2(kLog2e, kLog2e);
    float2 l2 = make_float2(0.0f, 0.0f), s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float2 a = make_float2(f[i], f[i + 1]);
        if (NEAR) {
            a = __ffma2_rn(a, k2, r2);
        } else {
            a = __fmul2_rn(__fadd2_rn(a, r2), k2);
            a.x = max_nan(a.x, kFar);
            a.y = max_nan(a.y, kFar);
        }
        const float2 e = make_float2(ex2(a.x), ex2(a.y));
        l2 = __fadd2_rn(l2, e);
        s2 = __ffma2_rn(e, a, s2);
    }
    p.l += l2.x + l2.y;
    p.sa += s2.x + s2.y;
}

// ------------------------------------------------------------ best tokens

// Order-preserving bits of a logit (-0 as +0).
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int64_t index) {
    return (static_cast<uint64_t>(order_of(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

// The warp's list: lane i holds the i-th largest key (0: none).
struct TopList {
    uint64_t key;
    // every lane offers one key (0: none); `at`: the last entry that matters
    __device__ __forceinline__ void offer(uint64_t k, int at, int lane) {
        uint32_t left = __ballot_sync(0xffffffffu, k > __shfl_sync(0xffffffffu, key, at));
        while (left) {                     // (a key that no longer belongs finds no place)
            const int src = __ffs(left) - 1;
            left &= left - 1;
            const uint64_t c = __shfl_sync(0xffffffffu, k, src);
            const uint64_t up = __shfl_up_sync(0xffffffffu, key, 1);
            const int pos = __popc(__ballot_sync(0xffffffffu, key > c));
            key = lane < pos ? key : lane == pos ? c : up;
        }
    }
    __device__ __forceinline__ uint32_t order() const { return static_cast<uint32_t>(key >> 32); }
};

// A bound that topk elements of the block reach: the topk-th largest of what
// its warps post, r values each in descending order (lane i < r: the i-th).  Each
// warp counts for its own values how many of all reach them.  *cut starts at 0.
__device__ __forceinline__ uint32_t block_bound(uint32_t* posts, uint32_t* cut, uint32_t value, int r, int nw, int topk,
                                                int warp, int lane) {
    if (lane < r) posts[warp * r + lane] = value;
    __syncthreads();
    const int posted = nw * r;             // at most 79
    const uint32_t p0 = lane < posted ? posts[lane] : 0u, p1 = lane + 32 < posted ? posts[lane + 32] : 0u,
                   p2 = lane + 64 < posted ? posts[lane + 64] : 0u;
    for (int i = 0; i < r; ++i) {
        const uint32_t v = __shfl_sync(0xffffffffu, value, i);
        if (v == 0) break;
        int reached = __popc(__ballot_sync(0xffffffffu, p0 >= v));
        if (posted > 32) reached += __popc(__ballot_sync(0xffffffffu, p1 >= v));
        if (posted > 64) reached += __popc(__ballot_sync(0xffffffffu, p2 >= v));
        if (reached >= topk) {             // the warp's largest such value
            if (lane == 0) atomicMax(cut, v);
            break;
        }
    }
    __syncthreads();
    return *cut;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// The keys of cand[0 .. count) that have fewer than topk larger ones, each at
// its rank in out; by `threads` threads, of which this is number t.  cand is
// 16-byte aligned.
__device__ __forceinline__ void rank_keys(const uint64_t* cand, int count, int topk, uint64_t* out, int t, int threads) {
    const ulonglong2* two = reinterpret_cast<const ulonglong2*>(cand);
    for (int i = t; i < count; i += threads) {
        const uint64_t k = cand[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < count / 2; ++j) {
            const ulonglong2 c = two[j];
            rank += (c.x > k) + (c.y > k);
        }
        if (count & 1) rank += cand[count - 1] > k;
        if (rank < topk && k != 0) out[rank] = k;
    }
}

// A row is one cluster of `ranks` CTAs of blockDim.x (a power of two)
// threads, or one warp of a block of kTeams (ranks == 1).
template <typename T, bool TOPK>
__global__ void __launch_bounds__(kMaxThreads, 2)
    forward_kernel(const T* __restrict__ logits, int64_t rows, int64_t vocab, int64_t ld,
                   const int64_t* __restrict__ targets, int topk, int ranks, int row_warps, float* __restrict__ logprob,
                   float* __restrict__ entropy, float2* __restrict__ stats, float* __restrict__ top_logprob,
                   int64_t* __restrict__ top_index) {
    using E = Elem<T>;
    constexpr int kWarps = kMaxThreads / 32;
    __shared__ float4 parts[kWarps];
    __shared__ float4 block_part;
    __shared__ uint32_t bound[kWarps];
    __shared__ uint32_t posts[TOPK ? kPosts : 1], cut[2];
    __shared__ unsigned long long cut_key;
    __shared__ int kept;
    __shared__ __align__(16) uint64_t cand[TOPK ? kWarps * 32 : 1];     // kTeams * 32 at least
    __shared__ uint64_t best[TOPK ? kTeams : 1][32];
    __shared__ int count[kTeams];
    const int nw = row_warps, lane = threadIdx.x & 31;
    // one warp per row: warp `team` of the block on its own; else team 0 is the block
    const int team = nw == 1 ? static_cast<int>(threadIdx.x >> 5) : 0;
    const int warp = nw == 1 ? 0 : static_cast<int>(threadIdx.x >> 5);
    const int t = warp * 32 + lane, row_threads = nw * 32;
    const int rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int64_t row = nw == 1 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + team : blockIdx.x / ranks;
    auto sync = [&] {
        if (nw == 1)
            __syncwarp();
        else
            __syncthreads();
    };
    griddep_launch_dependents();
    griddep_wait();                    // inputs of the preceding kernel are complete
    if (row >= rows) return;           // (a whole warp of its own)

    const T* x = logits + row * ld;
    const int64_t head = head_of(x, vocab);
    const int nvec = static_cast<int>((vocab - head) / E::N);
    const int64_t tail0 = head + static_cast<int64_t>(nvec) * E::N;
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    // vector i0 + 32 u of a warp's batch; its next batch lies `step` vectors on
    const int step = ranks * nw * kBatch * 32;

    // what the target's log probability needs, loaded ahead (by the thread that stores it)
    int64_t target = -1;
    float at_target = 0.0f;
    if (logprob && rank == 0 && t == 0) {
        target = targets[row];
        if (target >= 0 && target < vocab) at_target = E::load(x + target);
    }
    Part p = {kLowest, 0.0f, 0.0f, 0.0f};
    TopList top = {0ull};
    uint32_t own = 0;                  // order of the list's topk-th entry
    uint32_t reach0 = 0;               // topk elements of the block reach it
    const int jth = TOPK ? (topk + nw - 1) / nw : 0;
    volatile uint32_t* bounds = bound + team;          // [warp]

    if (rank == 0 && warp == 0 && head > 0) {
        const bool in = lane < head;
        const float f = in ? E::load(x + lane) : -INFINITY;
        if (in) p.add(f);
        if (TOPK) top.offer(in && f == f ? key_of(f, lane) : 0ull, topk - 1, lane);
    }
    if (TOPK) {
        if (lane == 0) bounds[warp] = 0;
        if (t == 0) count[team] = 0;
        if (threadIdx.x == 0) {
            cut[0] = cut[1] = 0;
            cut_key = 0;
            kept = 0;
        }
        if (t < 32) best[team][t] = 0ull;
    }

    bool first = TOPK;
    // every warp makes the same number of rounds (the first has a barrier)
    const int rounds = (nvec + step - 1) / step;
    uint4 next[kBatch];
    auto fetch = [&](int i) {
        if (i - lane + kBatch * 32 <= nvec) {            // the warp's whole batch
#pragma unroll
            for (int u = 0; u < kBatch; ++u) next[u] = __ldg(xv + i + 32 * u);
        } else {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) next[u] = i + 32 * u < nvec ? __ldg(xv + i + 32 * u) : E::masked();
        }
    };
    int i0 = (rank * nw + warp) * kBatch * 32 + lane;
    fetch(i0);
#pragma unroll(TOPK ? 1 : 2)
    for (int rd = 0; rd < rounds; ++rd, i0 += step) {
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = next[u];
        if (rd + 1 < rounds) fetch(i0 + step);           // in flight while this batch is worked on
        float bm = E::vmax(v[0]);
#pragma unroll
        for (int u = 1; u < kBatch; ++u) bm = fmaxf(bm, E::vmax(v[u]));
        // One maximum for the warp: a lane's own would change in so many
        // rounds that some lane of 32 takes the longer way almost every time.
        if (__any_sync(0xffffffffu, bm > p.m)) {
            p.refer(warp_max(fmaxf(bm, p.m)));
            if (bm == p.m) {                   // (few lanes)
#pragma unroll
                for (int u = 0; u < kBatch; ++u) E::take_out(v[u], p.m, p.n);
            }
        }
        if (i0 - lane < nvec) {                // (the warp has a batch)
            if (fabsf(p.m) < kNear) {          // the same for the warp
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    float f[E::N];
                    E::unpack(E::floored(v[u]), f);
                    add_terms<E::N, true>(p, f);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    float f[E::N];
                    E::unpack(v[u], f);
                    add_terms<E::N, false>(p, f);
                }
            }
        }
        if (TOPK) {
            const uint32_t bo = i0 < nvec && bm == bm ? order_of(bm) : 0u;
            if (first) {
                // The lanes' maxima are distinct elements: the topk-th largest of some of
                // them is a bound.  One warp takes it from its own; several post their `r`
                // largest each, 2 topk of the block or more.
                const int r = nw == 1 ? topk : (2 * topk + nw - 1) / nw;
                uint32_t value = 0;                    // lane i: the i-th largest lane maximum
                if (r <= 8) {
                    uint32_t left = bo;
                    for (int i = 0; i < r; ++i) {
                        const uint32_t m = __reduce_max_sync(0xffffffffu, left);
                        if (lane == __ffs(__ballot_sync(0xffffffffu, left == m)) - 1) left = 0;
                        if (lane == i) value = m;
                    }
                } else {
                    int above = 0;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const uint32_t o = __shfl_sync(0xffffffffu, bo, j);
                        above += (o > bo || (o == bo && j < lane)) ? 1 : 0;
                    }
                    for (int i = nw == 1 ? r - 1 : 0; i < r; ++i) {
                        const uint32_t who = __ballot_sync(0xffffffffu, above == i);
                        const uint32_t m = __shfl_sync(0xffffffffu, bo, __ffs(who) - 1);
                        if (lane == i) value = m;
                    }
                }
                reach0 = nw == 1 ? __shfl_sync(0xffffffffu, value, topk - 1)
                                 : block_bound(posts, &cut[0], value, r, nw, topk, warp, lane);
            }
            uint32_t reach = max(reach0, __reduce_min_sync(0xffffffffu, bounds[lane & (nw - 1)]));
            // own entries of earlier rounds have lower indices: an equal logit loses to them
            uint32_t owners = __ballot_sync(0xffffffffu, bo != 0 && bo >= reach && (first || bo > own));
            first = false;
            if (owners) {
                while (owners) {
                    const int src = __ffs(owners) - 1;
                    owners &= owners - 1;
                    // the owner's elements, one per lane, read again (they are in the cache)
                    const int base = __shfl_sync(0xffffffffu, i0, src);
                    const int vec = base + (lane / E::N) * 32;
                    const int64_t at = head + static_cast<int64_t>(vec) * E::N + lane % E::N;
                    uint64_t k = 0;
                    if (lane < kBatch * E::N && vec < nvec) {
                        const float f = E::load(x + at);
                        if (f == f && order_of(f) >= reach) k = key_of(f, at);
                    }
                    top.offer(k, topk - 1, lane);
                }
                own = static_cast<uint32_t>(__shfl_sync(0xffffffffu, top.key, topk - 1) >> 32);
                const uint32_t mine = static_cast<uint32_t>(__shfl_sync(0xffffffffu, top.key, jth - 1) >> 32);
                if (lane == 0 && mine > bounds[warp]) bounds[warp] = mine;
            }
        }
    }
    if (rank == 0 && warp == 0 && tail0 < vocab) {
        const bool in = lane < vocab - tail0;
        const float f = in ? E::load(x + tail0 + lane) : -INFINITY;
        if (in) p.add(f);
        if (TOPK) top.offer(in && f == f ? key_of(f, tail0 + lane) : 0ull, topk - 1, lane);
    }

    p.warp_join();
    if (nw > 1 && lane == 0) parts[warp] = make_float4(p.m, p.n, p.l, p.sa);
    if (TOPK) {
        if (nw > 1) {                  // the same bound from the lists, so that few more than topk keys are ranked
            const uint32_t mine = top.order();
            reach0 = max(reach0, block_bound(posts, &cut[1], mine, (2 * topk + nw - 1) / nw, nw, topk, warp, lane));
        } else {
            __syncwarp();              // (the counter's start)
        }
        // a list's entries that reach the bound, in front of it: topk at most, as no more can be asked for
        const uint32_t mine = __ballot_sync(0xffffffffu, lane < topk && top.key != 0 && top.order() >= reach0);
        int at = 0;
        if (lane == 0 && mine) at = atomicAdd(&count[team], __popc(mine));
        at = __shfl_sync(0xffffffffu, at, 0);
        if (lane < __popc(mine)) cand[team * 32 + at + lane] = top.key;
    }
    if (nw > 1 || TOPK) sync();
    if (nw > 1 && warp == 0) {
        const float4 q = lane < nw ? parts[lane] : make_float4(kLowest, 0.0f, 0.0f, 0.0f);
        p = {q.x, q.y, q.z, q.w};
        p.warp_join();
        if (ranks > 1 && lane == 0) block_part = make_float4(p.m, p.n, p.l, p.sa);
    }
    if (TOPK) {
        rank_keys(cand + team * 32, count[team], topk, best[team], t, row_threads);
        sync();
    }
    if (ranks > 1) {
        cluster_sync();                // every rank's partial result and list are in
        if (rank == 0) {
            if (warp == 0) {
                float4 q = make_float4(kLowest, 0.0f, 0.0f, 0.0f);
                if (lane < ranks) q = ld_cluster_f4(map_to_cta(smem_u32(&block_part), static_cast<uint32_t>(lane)));
                p = {q.x, q.y, q.z, q.w};
                p.warp_join();
            }
            if (TOPK) {
                // (a block of a split row has 8 warps or more: one warp per rank)
                uint64_t k = 0;
                if (warp < ranks) k = ld_cluster_u64(map_to_cta(smem_u32(&best[0][lane]), static_cast<uint32_t>(warp)));
                if (lane >= topk) k = 0;
                // each rank's topk-th is a bound
                if (lane == topk - 1 && k != 0) atomicMax(&cut_key, static_cast<unsigned long long>(k));
                __syncthreads();
                if (k != 0 && k >= cut_key) cand[atomicAdd(&kept, 1)] = k;
                __syncthreads();
                rank_keys(cand, kept, topk, best[0], t, row_threads);
                __syncthreads();
            }
        }
        cluster_arrive();              // rank 0 has read the others' shared memory
    }
    if (rank == 0 && warp == 0) {
        // the sums at o = 0
        const float o = offset_of(p.m), scale = ex2(-o);
        const float rest = p.m == INFINITY ? __int_as_float(0x7FC00000) : p.l * scale;
        const float rest_d = kLn2 * scale * fmaf(-o, p.l, p.sa);
        const float total = p.n + rest;
        const bool empty = total == 0.0f;              // every logit is -inf
        const float log_sum = empty ? 0.0f : p.n == 1.0f ? log1pf(rest) : logf(total);
        if (lane == 0) {
            stats[row] = make_float2(empty ? -INFINITY : p.m, log_sum);
            if (entropy) entropy[row] = empty ? 0.0f : log_sum - rest_d / total;
            if (logprob) {
                float r = 0.0f;
                if (target >= vocab)
                    r = __int_as_float(0x7FC00000);     // no such token
                else if (target >= 0)
                    r = empty ? -INFINITY : (at_target - p.m) - log_sum;
                logprob[row] = r;
            }
        }
        if (TOPK && lane < topk) {
            const uint64_t k = best[team][lane];
            const float f = value_of(static_cast<uint32_t>(k >> 32));
            top_logprob[row * topk + lane] = k == 0 ? __int_as_float(0x7FC00000) : empty ? -INFINITY : (f - p.m) - log_sum;
            top_index[row * topk + lane] = k == 0 ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        }
    }
    __syncwarp();
    if (ranks > 1) cluster_wait();
}

// ------------------------------------------------------------------ gradient

// blockIdx.x = row * chunks + chunk; a chunk is blockDim.x * kBatch vectors of
// the row (the first also takes the elements before the first 16-byte
// boundary, the last those after the last).  dlogits may be logits itself:
// every element is read and then written by one thread.
// ENT: with the entropy's gradient.
template <typename T, bool ENT>
__global__ void __launch_bounds__(kMaxThreads, 3)
    backward_kernel(const T* logits, int64_t vocab, int64_t ld, const int64_t* __restrict__ targets,
                    const float2* __restrict__ stats, const float* __restrict__ dlogprob,
                    const float* __restrict__ entropy, const float* __restrict__ dentropy, int64_t chunks, T* dlogits,
                    int64_t ld_out) {
    using E = Elem<T>;
    griddep_launch_dependents();
    griddep_wait();                    // inputs of the preceding kernel are complete
    const int64_t row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
    const T* x = logits + row * ld;
    T* out = dlogits + row * ld_out;
    const int64_t head = head_of(x, vocab);
    const int64_t nvec = (vocab - head) / E::N;
    const int64_t tail0 = head + nvec * E::N;
    const int64_t i0 = chunk * blockDim.x * kBatch + threadIdx.x;
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    uint4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
        v[u] = i0 + u * static_cast<int64_t>(blockDim.x) < nvec ? xv[i0 + u * static_cast<int64_t>(blockDim.x)] : E::masked();

    const float2 st = __ldg(stats + row);
    const float nm = st.x == -INFINITY ? 0.0f : -st.x;
    const int64_t target = dlogprob ? __ldg(targets + row) : -1;
    float g = target >= 0 ? __ldg(dlogprob + row) : 0.0f;
    if (target >= vocab) g = __int_as_float(0x7FC00000);             // no such token
    const float h = ENT ? __ldg(dentropy + row) : 0.0f;
    const float H = ENT ? __ldg(entropy + row) : 0.0f;

    // an element that is not the target
    auto grad2 = [&](float& a, float& b) {
        float2 lp = __fadd2_rn(__fadd2_rn(make_float2(a, b), make_float2(nm, nm)), make_float2(-st.y, -st.y));
        if (ENT) {                     // (0 * -inf would be NaN)
            lp.x = max_nan(lp.x, kFar);
            lp.y = max_nan(lp.y, kFar);
        }
        const float2 t = __fmul2_rn(lp, make_float2(kLog2e, kLog2e));
        float2 w = make_float2(-g, -g);
        if (ENT) w = __ffma2_rn(make_float2(-h, -h), __fadd2_rn(lp, make_float2(H, H)), w);
        const float2 r = __fmul2_rn(make_float2(ex2(t.x), ex2(t.y)), w);
        a = r.x;
        b = r.y;
    };
    auto single = [&](int64_t at) {
        float f = E::load(x + at), unused = 0.0f;
        grad2(f, unused);
        E::store(out + at, f);
    };
    // The target's element is stored a second time, by the thread that has it (and
    // read ahead, as out may be x).
    bool mine;
    if (target < head) {
        mine = chunk == 0 && target == threadIdx.x;
    } else if (target < tail0) {
        const int64_t d = (target - head) / E::N - i0;
        mine = d >= 0 && d < static_cast<int64_t>(blockDim.x) * kBatch && (d & (blockDim.x - 1)) == 0;
    } else {
        mine = chunk == chunks - 1 && target == tail0 + threadIdx.x && target < vocab;
    }
    float hit = 0.0f;
    if (mine) {
        // g (1 - p) of a likely target from log p: g - g p would lose its digits
        float unused = 0.0f;
        hit = E::load(x + target);
        const float lp = (hit + nm) - st.y;
        grad2(hit, unused);
        if (lp > -kLn2) {
            hit = -g * expm1f(lp);
            if (ENT) hit = fmaf(-h * ex2(lp * kLog2e), lp + H, hit);
        } else {                       // (NaN among them)
            hit += g;
        }
    }
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int64_t i = i0 + u * static_cast<int64_t>(blockDim.x);
        if (i < nvec) {
            float f[E::N];
            E::unpack(v[u], f);
            const int64_t at = head + i * E::N;
#pragma unroll
            for (int j = 0; j < E::N; j += 2) grad2(f[j], f[j + 1]);
            if (same) {
                *reinterpret_cast<uint4*>(out + at) = E::pack(f);
            } else {
#pragma unroll
                for (int j = 0; j < E::N; ++j) E::store(out + at + j, f[j]);
            }
        }
    }
    if (chunk == 0 && threadIdx.x < head) single(threadIdx.x);
    if (chunk == chunks - 1 && threadIdx.x < vocab - tail0) single(tail0 + threadIdx.x);
    if (mine) E::store(out + target, hit);
}

}  // namespace logp
}  // namespace fp8blk
