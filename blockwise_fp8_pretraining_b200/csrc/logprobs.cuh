// Log probabilities of given tokens with the distribution's entropy and its
// most likely tokens, from one read of the logits, and the gradient of the
// logits.  For a row of logits x, with m = max x and d = x - m:
//
//   L       = log(sum_v exp(d_v))
//   logp_v  = d_v - L
//   H       = -sum_v p_v logp_v = L - (sum_v exp(d_v) d_v) / sum_v exp(d_v)
//   dx_v    = g (1[v = target] - p_v) - h p_v (logp_v + H)
//
// for the gradients g of the target's log probability and h of the entropy.
//
// Everything is referred to the row's maximum, which is subtracted before the
// product with log2(e): rows of the type's lowest value, or of huge values,
// come out right, and neither L nor H subtracts large numbers from each other.
// The maximum's own term, exp(0) = 1, is counted in an integer n beside the
// sum l of the others, so that L = log1p(l) keeps its digits when one token
// has almost all the probability.
//
// A row is read by a cluster of 1 to 8 CTAs (few rows are split, so that one
// row's 300 KB do not wait for one SM).  Each thread keeps (m, n, l, sum e d)
// over its elements; the partial results meet by shuffles, shared memory and
// distributed shared memory in a fixed order, so results repeat run to run.
//
// The alternatives: every warp keeps the 32 best of its elements, one per
// lane, sorted, as 64-bit keys (order-preserving bits of the value, then the
// complement of the index, so that equal logits rank by index).  Elements
// reach the list only when they are not below a bound that k elements of the
// block are known to reach: the smallest, over the block's nw warps, of the
// ceil(k / nw)-th best each warp has seen.
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

// Partial result over some elements: their maximum m (kLowest before the
// first finite one), how many of them the counted n are (each exp(0)), the
// sum l of the others' exp(x - m), and sx = sum exp(x - m) (x - m).
struct Part {
    float m, n, l, sx;
    // refer the sums to the maximum M >= m
    __device__ __forceinline__ void refer(float M) {
        if (M > m) {
            const float delta = fmaxf(m - M, kFar), c = ex2(delta * kLog2e), e = l + n;
            sx = c * fmaf(delta, e, sx);
            l = c * e;
            n = 0.0f;
            m = M;
        }
    }
    __device__ __forceinline__ void add(float x) {             // one element
        refer(x);
        const float d = max_nan(x - m, kFar);
        if (d == 0.0f && n == 0.0f) {
            n = 1.0f;
        } else {
            const float e = ex2(d * kLog2e);
            l += e;
            sx = fmaf(e, d, sx);
        }
    }
    __device__ __forceinline__ void warp_join() {
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        refer(M);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            l += __shfl_xor_sync(0xffffffffu, l, o);
            sx += __shfl_xor_sync(0xffffffffu, sx, o);
        }
    }
};

// The terms of N elements; EXCL counts those at the maximum in n.
template <int N, bool EXCL>
__device__ __forceinline__ void add_terms(Part& p, const float (&f)[N]) {
    const float2 nm = make_float2(-p.m, -p.m), k2 = make_float2(kLog2e, kLog2e);
    float2 l2 = make_float2(0.0f, 0.0f), s2 = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float2 d = __fadd2_rn(make_float2(f[i], f[i + 1]), nm);
        d.x = max_nan(d.x, kFar);
        d.y = max_nan(d.y, kFar);
        const float2 a = __fmul2_rn(d, k2);
        float2 e = make_float2(ex2(a.x), ex2(a.y));
        if (EXCL) {
            if (d.x == 0.0f) { p.n += 1.0f; e.x = 0.0f; }
            if (d.y == 0.0f) { p.n += 1.0f; e.y = 0.0f; }
        }
        l2 = __fadd2_rn(l2, e);
        s2 = __ffma2_rn(e, d, s2);
    }
    p.l += l2.x + l2.y;
    p.sx += s2.x + s2.y;
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
    __device__ __forceinline__ void insert(uint64_t k, int lane) {
        const int pos = __popc(__ballot_sync(0xffffffffu, key > k));
        const uint64_t up = __shfl_up_sync(0xffffffffu, key, 1);
        key = lane < pos ? key : lane == pos ? k : up;
    }
    // every lane offers one key (0: none) that beats the list's entry `at`
    __device__ __forceinline__ void offer(uint64_t k, int at, int lane) {
        uint64_t worst = __shfl_sync(0xffffffffu, key, at);
        uint32_t left = __ballot_sync(0xffffffffu, k > worst);
        while (left) {
            const int src = __ffs(left) - 1;
            left &= left - 1;
            const uint64_t c = __shfl_sync(0xffffffffu, k, src);
            if (c > worst) {
                insert(c, lane);
                worst = __shfl_sync(0xffffffffu, key, at);
            }
        }
    }
    // the 32 largest of this list and another (sorted the same way)
    __device__ __forceinline__ void merge(const uint64_t* other, int lane) {
        const uint64_t o = other[31 - lane];
        key = key > o ? key : o;               // bitonic: the 32 largest of the 64
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
            const uint64_t q = __shfl_xor_sync(0xffffffffu, key, s);
            const bool keep_max = (lane & s) == 0;
            key = (keep_max == (key > q)) ? key : q;
        }
    }
};

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

// One cluster of `ranks` CTAs per row; blockDim.x = 32 * a power of two.
template <typename T, bool TOPK>
__global__ void __launch_bounds__(kMaxThreads, 2)
    forward_kernel(const T* __restrict__ logits, int64_t vocab, int64_t ld, const int64_t* __restrict__ targets,
                   int topk, int ranks, float* __restrict__ logprob, float* __restrict__ entropy,
                   float2* __restrict__ stats, float* __restrict__ top_logprob, int64_t* __restrict__ top_index) {
    using E = Elem<T>;
    __shared__ float4 parts[kMaxThreads / 32];
    __shared__ float4 block_part;
    __shared__ uint64_t lists[TOPK ? kMaxThreads / 32 : 1][32];     // (at least kMaxRanks)
    __shared__ uint32_t bound[kMaxThreads / 32];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, nw = blockDim.x >> 5;
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t row = blockIdx.x / ranks;
    griddep_wait();                    // inputs of the preceding kernel are complete

    const T* x = logits + row * ld;
    const int64_t head = head_of(x, vocab);
    const int64_t nvec = (vocab - head) / E::N;
    const int64_t tail0 = head + nvec * E::N;
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    const int64_t stride = static_cast<int64_t>(ranks) * blockDim.x;

    Part p = {kLowest, 0.0f, 0.0f, 0.0f};
    TopList top = {0ull};
    const int jth = TOPK ? (topk + nw - 1) / nw : 0;
    uint32_t own = 0;                  // order of the list's topk-th entry
    volatile uint32_t* bounds = bound;

    if (rank == 0 && warp == 0 && head > 0) {
        const bool in = lane < head;
        const float f = in ? E::load(x + lane) : -INFINITY;
        if (in) p.add(f);
        if (TOPK) top.offer(in && f == f ? key_of(f, lane) : 0ull, topk - 1, lane);
    }

    bool first = TOPK;
    // every warp makes the same number of rounds (the first has a barrier)
    const int64_t rounds = nvec > 0 ? (nvec + stride * kBatch - 1) / (stride * kBatch) : 0;
    for (int64_t rd = 0; rd < rounds; ++rd) {
        const int64_t i0 = rd * stride * kBatch + rank * static_cast<int64_t>(blockDim.x) + t;
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = i0 + u * stride < nvec ? __ldg(xv + i0 + u * stride) : E::masked();
        float bm = E::vmax(v[0]);
#pragma unroll
        for (int u = 1; u < kBatch; ++u) bm = fmaxf(bm, E::vmax(v[u]));
        if (bm > p.m) {
            p.refer(bm);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                float f[E::N];
                E::unpack(v[u], f);
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
        if (TOPK) {
            const uint32_t bo = order_of(bm);
            if (first) {
                // lane maxima are distinct elements: the jth of them is reached by j
                uint32_t left = i0 < nvec && bm == bm ? bo : 0u, got = 0;
                for (int j = 0; j < jth; ++j) {
                    got = __reduce_max_sync(0xffffffffu, left);
                    const uint32_t who = __ballot_sync(0xffffffffu, left == got);
                    if (lane == __ffs(who) - 1) left = 0;
                }
                if (lane == 0) bounds[warp] = got;
                __syncthreads();
            }
            uint32_t reach = bounds[lane & (nw - 1)];
            reach = __reduce_min_sync(0xffffffffu, reach);
            // own entries of earlier rounds have lower indices: an equal logit loses to them
            uint32_t owners = __ballot_sync(0xffffffffu, i0 < nvec && bo >= reach && (first || bo > own));
            first = false;
            if (owners) {
                while (owners) {
                    const int src = __ffs(owners) - 1;
                    owners &= owners - 1;
                    // the owner's elements, one per lane, read again (they are in the cache)
                    const int64_t base = __shfl_sync(0xffffffffu, i0, src);
                    const int64_t vec = base + (lane / E::N) * stride;
                    const int64_t at = head + vec * E::N + lane % E::N;
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
    if (lane == 0) parts[warp] = make_float4(p.m, p.n, p.l, p.sx);
    if (TOPK) lists[warp][lane] = top.key;
    __syncthreads();
    if (warp == 0) {
        const float4 q = lane < nw ? parts[lane] : make_float4(kLowest, 0.0f, 0.0f, 0.0f);
        p = {q.x, q.y, q.z, q.w};
        p.warp_join();
        if (ranks > 1 && lane == 0) block_part = make_float4(p.m, p.n, p.l, p.sx);
    }
    if (TOPK) {
        for (int s = nw >> 1; s > 0; s >>= 1) {
            if (warp < s) {
                top.merge(lists[warp + s], lane);
                lists[warp][lane] = top.key;
            }
            __syncthreads();
        }
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
                // lists[0] is read by this CTA only; the other ranks' come over beside it
                for (int r = 1 + warp; r < ranks; r += nw) {
                    const uint64_t k = ld_cluster_u64(map_to_cta(smem_u32(&lists[0][lane]), static_cast<uint32_t>(r)));
                    lists[r][lane] = k;
                }
                __syncthreads();
                for (int s = ranks >> 1; s > 0; s >>= 1) {
                    if (warp < s) {
                        top.key = lists[warp][lane];
                        top.merge(lists[warp + s], lane);
                        lists[warp][lane] = top.key;
                    }
                    __syncthreads();
                }
            }
        }
        cluster_sync();                // rank 0 has read the others' shared memory
    }
    if (rank == 0 && warp == 0) {
        const float total = p.n + p.l;
        const bool empty = total == 0.0f;              // every logit is -inf
        const float log_sum = empty ? 0.0f : p.n == 1.0f ? log1pf(p.l) : logf(total);
        if (lane == 0) {
            stats[row] = make_float2(empty ? -INFINITY : p.m, log_sum);
            if (entropy) entropy[row] = empty ? 0.0f : log_sum - p.sx / total;
            if (logprob) {
                const int64_t y = targets[row];
                float r = 0.0f;
                if (y >= vocab)
                    r = __int_as_float(0x7FC00000);     // no such token
                else if (y >= 0)
                    r = empty ? -INFINITY : (E::load(x + y) - p.m) - log_sum;
                logprob[row] = r;
            }
        }
        if (TOPK && lane < topk) {
            const uint64_t k = top.key;
            const float f = value_of(static_cast<uint32_t>(k >> 32));
            top_logprob[row * topk + lane] = k == 0 ? __int_as_float(0x7FC00000) : empty ? -INFINITY : (f - p.m) - log_sum;
            top_index[row * topk + lane] = k == 0 ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(k));
        }
    }
    griddep_launch_dependents();
}

// ------------------------------------------------------------------ gradient

// blockIdx.x = row * chunks + chunk; a chunk is blockDim.x * kBatch vectors of
// the row (the first also takes the elements before the first 16-byte
// boundary, the last those after the last).  dlogits may be logits itself:
// every element is read and then written by one thread (the target's own
// logit is an element like any other).
template <typename T>
__global__ void __launch_bounds__(kMaxThreads)
    backward_kernel(const T* logits, int64_t vocab, int64_t ld, const int64_t* __restrict__ targets,
                    const float2* __restrict__ stats, const float* __restrict__ dlogprob,
                    const float* __restrict__ entropy, const float* __restrict__ dentropy, int64_t chunks, T* dlogits,
                    int64_t ld_out) {
    using E = Elem<T>;
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
    const bool empty = st.x == -INFINITY;
    const float m = empty ? 0.0f : st.x;
    const int64_t target = dlogprob ? __ldg(targets + row) : -1;
    float g = target >= 0 ? __ldg(dlogprob + row) : 0.0f;
    if (target >= vocab) g = __int_as_float(0x7FC00000);             // no such token
    const float h = dentropy ? __ldg(dentropy + row) : 0.0f;
    const float H = dentropy ? __ldg(entropy + row) : 0.0f;

    auto grad = [&](float f, int64_t at) {
        const float lp = max_nan((f - m) - st.y, kFar);
        const float pr = ex2(lp * kLog2e);
        float r = -pr * fmaf(h, lp + H, g);
        if (at == target) r += g;
        return r;
    };
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int64_t i = i0 + u * static_cast<int64_t>(blockDim.x);
        if (i < nvec) {
            float f[E::N];
            E::unpack(v[u], f);
            const int64_t at = head + i * E::N;
#pragma unroll
            for (int j = 0; j < E::N; ++j) f[j] = grad(f[j], at + j);
            if (same) {
                *reinterpret_cast<uint4*>(out + at) = E::pack(f);
            } else {
#pragma unroll
                for (int j = 0; j < E::N; ++j) E::store(out + at + j, f[j]);
            }
        }
    }
    if (chunk == 0 && threadIdx.x < head) {
        const int64_t at = threadIdx.x;
        E::store(out + at, grad(E::load(x + at), at));
    }
    if (chunk == chunks - 1 && threadIdx.x < vocab - tail0) {
        const int64_t at = tail0 + threadIdx.x;
        E::store(out + at, grad(E::load(x + at), at));
    }
    griddep_launch_dependents();
}

}  // namespace logp
}  // namespace fp8blk
