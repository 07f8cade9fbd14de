// C ABI of the blockwise-E4M3 FP8 linear-layer library (see include/fp8blk.h
// for the contract of every entry point).  Host code here only checks
// arguments, builds TMA tensor maps and launches kernels on the caller's
// stream; it never allocates or synchronizes (except fp8_get_error /
// fp8_clear_error, which read or reset the device error word).
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/fp8blk.h"
#include "addnorm.cuh"
#include "gemm.cuh"
#include "logprobs.cuh"
#include "newton_schulz.cuh"
#include "newton_schulz_small.cuh"
#include "quantize.cuh"

static_assert(fp8blk::kErrTimeout == static_cast<unsigned int>(FP8_ERR_TIMEOUT),
              "device time-out code must match the C ABI");
static_assert(fp8blk::logp::kMaxTopK == FP8_MAX_TOPK, "alternatives limit must match the C ABI");
static_assert(fp8blk::ns::small::kMaxSteps == FP8_NS_MAX_STEPS, "steps limit must match the C ABI");
static_assert(fp8blk::addnorm::kMaxCols == FP8_MAX_NORM_COLS, "row length limit must match the C ABI");

namespace {

// Launch with programmatic stream serialization: the kernel may begin
// launching while the preceding kernel of the stream finishes; it waits for
// that kernel's results in griddep_wait before touching global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}


using namespace fp8blk;

constexpr uint64_t kDefaultWaitNs = 2000000000ull;
std::atomic<uint64_t> g_wait_ns{kDefaultWaitNs};

// Test only (fp8_selftest_stall_next): bit 0 arms the next GEMM launch,
// bit 1 the next tile-quantizer launch, to over-state one barrier's bytes.
std::atomic<int> g_stall_next{0};
constexpr uint32_t kStallBytes = 16;

inline uint32_t take_stall(int bit) {
    return (g_stall_next.fetch_and(~bit) & bit) ? kStallBytes : 0u;
}

constexpr int kMaxDevices = 64;
std::atomic<int> g_sm_count[kMaxDevices];
std::atomic<int> g_gemm_attr_done[kMaxDevices];
std::atomic<int> g_gemm_pairs[kMaxDevices][12];  // co-resident CTA pairs per kernel variant

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 40;     // row strides; rows * stride stays far inside 64 bits

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Text of the last CUDA failure this thread saw (for fp8_last_cuda_error).
thread_local char g_detail[256] = "";

fp8_status cuda_fail(const char* where, cudaError_t e) {
    snprintf(g_detail, sizeof g_detail, "%s: %s (%d)", where, cudaGetErrorString(e), static_cast<int>(e));
    return FP8_ERR_CUDA;
}

inline fp8_status last_launch_status(const char* where) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? FP8_OK : cuda_fail(where, e);
}

fp8_status current_device(int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
    if (*dev < 0 || *dev >= kMaxDevices) return cuda_fail("device ordinal out of range", cudaErrorInvalidDevice);
    return FP8_OK;
}

fp8_status sm_count(int dev, int* out) {
    int n = g_sm_count[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
        const cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail("cudaDeviceGetAttribute", e);
        g_sm_count[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return FP8_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
        if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) {
            snprintf(g_detail, sizeof g_detail, "cudaGetDriverEntryPoint(cuTensorMapEncodeTiled): %s, query %d",
                     cudaGetErrorString(e), static_cast<int>(q));
            return nullptr;
        }
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// Row-major [rows, cols] byte matrix, boxes of box_rows x 128 bytes in the
// 128-byte swizzle the MMA descriptors expect; out-of-range rows read as 0.
fp8_status make_operand_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int64_t cols,
                            int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return FP8_ERR_CUDA;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estride[2] = {1u, 1u};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides,
                     box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(g_detail, sizeof g_detail, "cuTensorMapEncodeTiled: CUresult %d", static_cast<int>(r));
        return FP8_ERR_CUDA;
    }
    return FP8_OK;
}

// Row-major [rows, cols] GEMM output, boxes of 32 rows x 128 bytes (64 BF16
// or 32 FP32 columns) in the 128-byte swizzle of the epilogue's staging
// buffers.
fp8_status make_output_map(CUtensorMap* map, void* base, int64_t rows, int64_t cols, bool f32) {
    auto enc = tensor_map_encoder();
    if (!enc) return FP8_ERR_CUDA;
    const int esize = f32 ? 4 : 2;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * esize};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esize), 32u};
    cuuint32_t estride[2] = {1u, 1u};
    CUresult r = enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims,
                     strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(g_detail, sizeof g_detail, "cuTensorMapEncodeTiled(output): CUresult %d", static_cast<int>(r));
        return FP8_ERR_CUDA;
    }
    return FP8_OK;
}

// 2-D row-major map with a box of box_x (inner) by box_y elements.
fp8_status make_map_2d(CUtensorMap* map, CUtensorMapDataType type, int elem_bytes, const void* base,
                       int64_t rows, int64_t cols, uint32_t box_x, uint32_t box_y,
                       CUtensorMapSwizzle swizzle, const char* what) {
    auto enc = tensor_map_encoder();
    if (!enc) return FP8_ERR_CUDA;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * elem_bytes};
    cuuint32_t box[2] = {box_x, box_y};
    cuuint32_t estride[2] = {1u, 1u};
    CUresult r = enc(map, type, 2, const_cast<void*>(base), dims, strides, box, estride,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(g_detail, sizeof g_detail, "cuTensorMapEncodeTiled(%s): CUresult %d", what, static_cast<int>(r));
        return FP8_ERR_CUDA;
    }
    return FP8_OK;
}

std::atomic<int> g_tile_attr_done[kMaxDevices];

// Persistent 128 x 128 tile quantizer (column-wise, both, weight blocks;
// with kProdSwiglu the SwiGLU product of a gate_up activation [rows, 2 *
// cols], with kProdNorm the RMSNorm output of x given r and gamma).
template <int MODE, int PROD>
fp8_status launch_tile_quant(const void* x, int64_t rows, int64_t cols, uint8_t* q, float* s_row,
                             uint8_t* qT, float* s_col, cudaStream_t stream, const float* norm_r = nullptr,
                             const void* norm_gamma = nullptr) {
    constexpr bool SWIGLU = PROD == kProdSwiglu;
    using L = tile::Layout<SWIGLU>;
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    const int flag = 1 << (MODE + 4 * PROD);
    if ((g_tile_attr_done[dev].load(std::memory_order_relaxed) & flag) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(quant_tile_kernel<MODE, PROD>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   L::SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(quantize)", e);
        g_tile_attr_done[dev].fetch_or(flag, std::memory_order_relaxed);
    }
    CUtensorMap mx, mq, mqt;
    if ((st = make_map_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, rows, SWIGLU ? 2 * cols : cols, 64, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B, "quantize input")) != FP8_OK)
        return st;
    // Unused maps still need a valid encoding: point them at an output.
    const void* qbase = q ? static_cast<const void*>(q) : static_cast<const void*>(qT);
    const void* qtbase = qT ? static_cast<const void*>(qT) : static_cast<const void*>(q);
    if ((st = make_map_2d(&mq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, qbase, q ? rows : cols, q ? cols : rows,
                          128, 128, CU_TENSOR_MAP_SWIZZLE_128B, "row codes")) != FP8_OK)
        return st;
    if ((st = make_map_2d(&mqt, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, qtbase, qT ? cols : rows, qT ? rows : cols,
                          128, 128, CU_TENSOR_MAP_SWIZZLE_128B, "transposed codes")) != FP8_OK)
        return st;
    const int64_t tiles = (rows / 128) * (cols / 128);
    const int64_t cap = static_cast<int64_t>(L::BLOCKS_PER_SM) * sms;
    const unsigned grid = static_cast<unsigned>(tiles < cap ? tiles : cap);
    const cudaError_t e = launch_pdl(quant_tile_kernel<MODE, PROD>, dim3(grid), dim3(tile::THREADS),
                                     L::SMEM_BYTES, stream, mx, mq, mqt, rows, cols, s_row, s_col,
                                     qT != nullptr ? 1 : 0, g_wait_ns.load(std::memory_order_relaxed),
                                     take_stall(2), norm_r, static_cast<const __nv_bfloat16*>(norm_gamma));
    if (e != cudaSuccess) return cuda_fail("tile quantize launch", e);
    return last_launch_status("tile quantize launch");
}

// Workspace of the split schedule for `pairs` CTA pairs: FP32 partial sums
// [pairs][2][EPI_WARPS][32][32][4], then one flag per pair, CTA, warp and lane.
constexpr size_t kPartialFloatsPerPair = size_t(2) * gemm::EPI_WARPS * 128 * 32;
inline size_t gemm_workspace_bytes(int pairs) {
    const size_t partial = size_t(pairs) * kPartialFloatsPerPair * sizeof(float);
    const size_t flags = size_t(pairs) * 2 * gemm::EPI_WARPS * 32 * sizeof(int);
    return (partial + flags + 255) / 256 * 256;
}

// Whole tiles round-robin for all waves but the last two when the last wave
// would leave more than 5% of the pairs idle, a tile has at least 32 slabs
// and each pair has at least g_split_min_units (tile, slab) units of work;
// those tiles are then cut into ranges of slabs of equal length, one per
// pair.  (Measured on B200: handing partial sums over costs a few
// microseconds per launch, more than the idle pairs cost with 16 slabs per
// tile or with under about 150 units per pair.)
constexpr int kMinSplitSlabs = 32;
constexpr int64_t kDefaultSplitMinUnits = FP8_GEMM_SPLIT_MIN_WORK_DEFAULT;
std::atomic<int64_t> g_split_min_units{kDefaultSplitMinUnits};
inline int dp_tiles_for(int64_t tiles, int pairs, int num_kb) {
    const int64_t waves = (tiles + pairs - 1) / pairs;
    if (num_kb < kMinSplitSlabs || tiles >= waves * pairs * 95 / 100 ||
        tiles * num_kb < g_split_min_units.load(std::memory_order_relaxed) * pairs)
        return static_cast<int>(tiles);
    const int64_t full = tiles / pairs;
    return static_cast<int>(full >= 1 ? (full - 1) * pairs : 0);
}

// One-time set-up of a GEMM kernel variant on a device: its shared-memory
// limit, and how many CTA pairs can be resident at once (the persistent grid
// must not exceed it, or the last pairs would wait for a second wave).
template <int SCALE, int OUT, bool SPLIT>
fp8_status gemm_pairs(int dev, int sms, int* pairs_out) {
    constexpr int variant = SCALE + 2 * OUT + 6 * (SPLIT ? 1 : 0);
    const int flag = 1 << variant;
    if ((g_gemm_attr_done[dev].load(std::memory_order_relaxed) & flag) == 0) {
        cudaError_t e = cudaFuncSetAttribute(gemm::gemm_kernel<SCALE, OUT, SPLIT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             gemm::SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(gemm)", e);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1), 1, 1);
        cfg.blockDim = dim3(gemm::THREADS, 1, 1);
        cfg.dynamicSmemBytes = gemm::SMEM_BYTES;
        int pairs = 0;
        e = cudaOccupancyMaxActiveClusters(&pairs, gemm::gemm_kernel<SCALE, OUT, SPLIT>, &cfg);
        if (e != cudaSuccess) return cuda_fail("cudaOccupancyMaxActiveClusters(gemm)", e);
        if (pairs <= 0) return cuda_fail("gemm kernel cannot be resident", cudaErrorInvalidConfiguration);
        g_gemm_pairs[dev][variant].store(pairs, std::memory_order_relaxed);
        g_gemm_attr_done[dev].fetch_or(flag, std::memory_order_relaxed);
    }
    *pairs_out = g_gemm_pairs[dev][variant].load(std::memory_order_relaxed);
    return FP8_OK;
}

// Shared launcher of the GEMMs.  A: [M_out, Kc] codes, B: [N_out, Kc]
// codes, both K-major; scales described by `p`; out: [M_out, N_out] BF16, or
// FP32 added to in place (OUT == kOutAccF32).  Launches the split-schedule
// variant of the kernel only when the schedule splits tiles: the plain
// variant's promotion loop carries nothing for it.
template <int SCALE, int OUT>
fp8_status launch_gemm(const uint8_t* a, const uint8_t* b, void* out, gemm::Params p, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    int max_pairs = 0, split_pairs = 0;
    if ((st = gemm_pairs<SCALE, OUT, false>(dev, sms, &max_pairs)) != FP8_OK) return st;

    CUtensorMap ma, mb, mc;
    if ((st = make_operand_map(&ma, a, p.M, p.K, gemm::BM)) != FP8_OK) return st;
    if ((st = make_operand_map(&mb, b, p.N, p.K, gemm::BN / 2)) != FP8_OK) return st;
    // (main-gradient mode writes through p.out_f32; the map still needs a
    // valid encoding)
    if ((st = make_output_map(&mc, out, OUT == gemm::kOutAccF32Shards ? (p.shard_rows > 32 ? p.shard_rows : 32) : p.M, p.N,
                              OUT != gemm::kOutBf16)) != FP8_OK)
        return st;
    if (OUT == gemm::kOutAccF32) p.out_f32 = static_cast<float*>(out);

    p.tiles_m = static_cast<int>((p.M + 2 * gemm::BM - 1) / (2 * gemm::BM));
    p.tiles_n = static_cast<int>((p.N + gemm::BN - 1) / gemm::BN);
    p.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    p.stall_tx = take_stall(1);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    p.dp_tiles = static_cast<int>(tiles);
    p.ws_partial = nullptr;
    p.ws_flags = nullptr;
    if (workspace && workspace_bytes >= gemm_workspace_bytes(max_pairs))
        p.dp_tiles = dp_tiles_for(tiles, max_pairs, p.K / gemm::BK);
    if (p.dp_tiles < tiles) {
        // Same resources as the plain variant, so the same residency; a
        // smaller answer would leave pairs whose partial sums never arrive.
        if ((st = gemm_pairs<SCALE, OUT, true>(dev, sms, &split_pairs)) != FP8_OK) return st;
        if (split_pairs < max_pairs) p.dp_tiles = static_cast<int>(tiles);
    }
    cudaError_t e;
    if (p.dp_tiles < tiles) {
        p.ws_partial = static_cast<float*>(workspace);
        p.ws_flags = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) +
                                            size_t(max_pairs) * kPartialFloatsPerPair * sizeof(float));
        e = launch_pdl(gemm::gemm_kernel<SCALE, OUT, true>, dim3(2 * max_pairs), dim3(gemm::THREADS),
                       gemm::SMEM_BYTES, stream, ma, mb, mc, p);
    } else {
        const int grid_pairs = static_cast<int>(tiles < max_pairs ? tiles : max_pairs);
        e = launch_pdl(gemm::gemm_kernel<SCALE, OUT, false>, dim3(2 * grid_pairs), dim3(gemm::THREADS),
                       gemm::SMEM_BYTES, stream, ma, mb, mc, p);
    }
    if (e != cudaSuccess) return cuda_fail("gemm launch", e);
    return last_launch_status("gemm launch");
}

// wgrad: dW [N, K] over M tokens; A = dY^T codes [N, M], B = X^T codes [K, M].
gemm::Params wgrad_params(const float* sdyT, const float* sxT, int64_t N, int64_t K, int64_t M) {
    gemm::Params p{};
    p.sa = sdyT;
    p.sa_ld = N;                 // sdyT [M/128, N]
    p.sb = sxT;
    p.sb_ld = K;                 // sxT [M/128, K]
    p.M = static_cast<int>(N);
    p.N = static_cast<int>(K);
    p.K = static_cast<int>(M);
    return p;
}

bool dims_ok_gemm(int64_t M, int64_t N, int64_t K, bool m_positive) {
    if (M < 0 || N <= 0 || K <= 0) return false;
    if (m_positive && M == 0) return false;
    if (M % 128 || N % 128 || K % 128) return false;
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return false;
    if (static_cast<int64_t>((M + 255) / 256) * ((N + gemm::BN - 1) / gemm::BN) > kMaxDim) return false;
    return true;
}

// As launch_pdl, in clusters of `ranks` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, unsigned ranks,
                               cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// add + RMSNorm (+ row-wise quantization when q is given): one launch.
template <int CPL, int R>
cudaError_t launch_norm_stream(const void* x, const void* residual, const void* gamma, int64_t rows, int chunks,
                               float eps, void* sum_out, float* rstd, uint8_t* q, float* s_row, int sms,
                               cudaStream_t stream) {
    const int wpr = (chunks + 32 * CPL - 1) / (32 * CPL);
    const int teams = wpr < 8 ? 8 / wpr : 1;
    const int threads = 32 * wpr * teams;
    const int64_t need = (rows + teams * R - 1) / (teams * R);
    const int64_t cap = static_cast<int64_t>(sms) * (addnorm::kStreamThreads<CPL, R> * addnorm::kStreamBlocks<CPL, R> / threads);
    return launch_pdl(addnorm::stream_kernel<CPL, R>, dim3(static_cast<unsigned>(need < cap ? need : cap)),
                      dim3(static_cast<unsigned>(threads)), 0, stream, static_cast<const uint4*>(x),
                      static_cast<const uint4*>(residual), static_cast<const uint4*>(gamma), rows, chunks, eps, wpr,
                      static_cast<uint4*>(sum_out), rstd, reinterpret_cast<uint2*>(q), s_row);
}

// Few rows: one step per block.
template <int CPL>
cudaError_t launch_norm_rows(const void* x, const void* residual, const void* gamma, int64_t rows, int chunks,
                             float eps, void* sum_out, float* rstd, uint8_t* q, float* s_row, cudaStream_t stream) {
    const int wpr = (chunks + 32 * CPL - 1) / (32 * CPL);
    return launch_pdl(addnorm::row_kernel<CPL>, dim3(static_cast<unsigned>(rows)), dim3(32 * wpr), 0, stream,
                      static_cast<const uint4*>(x), static_cast<const uint4*>(residual),
                      static_cast<const uint4*>(gamma), rows, chunks, eps, static_cast<uint4*>(sum_out), rstd,
                      reinterpret_cast<uint2*>(q), s_row);
}

fp8_status norm_rows(const void* x, const void* residual, const void* gamma, int64_t rows, int64_t cols, float eps,
                     void* sum_out, float* rstd, uint8_t* q, float* s_row, cudaStream_t s) {
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    const int chunks = static_cast<int>(cols / 8);
    cudaError_t e;
    // Few rows: a row over as many warps as it has 512-byte runs, so that a
    // token's latency is one load and one short pass.  Many rows: 2 chunks per
    // lane and step, of two rows where one is enough for a row, and 4 where a row
    // would not fit 12 warps otherwise.
    if (rows <= 2 * sms && chunks <= 1024)
        e = launch_norm_rows<1>(x, residual, gamma, rows, chunks, eps, sum_out, rstd, q, s_row, s);
    else if (rows <= 2 * sms)
        e = launch_norm_rows<2>(x, residual, gamma, rows, chunks, eps, sum_out, rstd, q, s_row, s);
    else if (chunks <= 32)
        e = launch_norm_stream<1, 2>(x, residual, gamma, rows, chunks, eps, sum_out, rstd, q, s_row, sms, s);
    else if (chunks <= 768)
        e = launch_norm_stream<2, 1>(x, residual, gamma, rows, chunks, eps, sum_out, rstd, q, s_row, sms, s);
    else
        e = launch_norm_stream<4, 1>(x, residual, gamma, rows, chunks, eps, sum_out, rstd, q, s_row, sms, s);
    if (e != cudaSuccess) return cuda_fail("add + rmsnorm launch", e);
    return last_launch_status("add + rmsnorm launch");
}

fp8_status norm_cols(const void* sum, const float* rstd, const void* gamma, int64_t rows, int64_t cols,
                     uint8_t* q_colT, float* s_col, cudaStream_t s) {
    const cudaError_t e = launch_pdl(addnorm::col_kernel, dim3(static_cast<unsigned>((rows / 128) * (cols / 128))),
                                     dim3(addnorm::kColThreads), 0, s, static_cast<const __nv_bfloat16*>(sum), rstd,
                                     static_cast<const __nv_bfloat16*>(gamma), rows, cols, q_colT, s_col);
    if (e != cudaSuccess) return cuda_fail("rmsnorm column groups launch", e);
    return last_launch_status("rmsnorm column groups launch");
}

// Blocks of the norm's gradient: at most as many as can be resident, with
// equal shares of the rows; each leaves one row of dgamma's partial sums.
struct BwdShape {
    int chunks, cpt, wpr, teams, rows_at_once;
    unsigned grid;
};
BwdShape norm_bwd_shape(int64_t rows, int64_t cols, int sms) {
    BwdShape b;
    b.chunks = static_cast<int>(cols / 8);
    b.cpt = b.chunks <= 512 ? 1 : b.chunks <= 1024 ? 2 : 4;
    b.rows_at_once = b.cpt == 1 ? 2 : 1;
    b.wpr = (b.chunks + 32 * b.cpt - 1) / (32 * b.cpt);
    b.teams = b.cpt == 1 && b.wpr < 8 ? 8 / b.wpr : 1;
    const int64_t per = static_cast<int64_t>(b.teams) * b.rows_at_once;
    const int64_t need = (rows + per - 1) / per;
    const int64_t cap = static_cast<int64_t>(sms) * (addnorm::kBwdThreads / (32 * b.wpr * b.teams));
    const int64_t each = (need + cap - 1) / cap;
    b.grid = static_cast<unsigned>((need + each - 1) / each);
    return b;
}

template <int CPT, int R, bool AHEAD>
cudaError_t launch_norm_bwd(const BwdShape& b, const void* dy, const void* x, const float* rstd, const void* gamma,
                            const void* dres, int64_t rows, void* ds, float* partial, float* dgamma, int accumulate,
                            cudaStream_t s) {
    return launch_pdl(addnorm::bwd_kernel<CPT, R, AHEAD>, dim3(b.grid), dim3(32 * b.wpr * b.teams), 0, s,
                      static_cast<const uint4*>(dy), static_cast<const uint4*>(x), rstd,
                      static_cast<const uint4*>(gamma), static_cast<const uint4*>(dres), rows, b.chunks, b.wpr,
                      static_cast<uint4*>(ds), partial, dgamma, accumulate);
}

// Power of two >= v, within [lo, hi] (both powers of two).
inline int pow2_between(int64_t v, int lo, int hi) {
    int p = lo;
    while (p < hi && p < v) p *= 2;
    return p;
}

bool dtype_ok(int dtype) { return dtype == FP8_BF16 || dtype == FP8_F32; }
bool element_aligned(const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == FP8_BF16 ? 1u : 3u)) == 0;
}

// A row of logits over `ranks` CTAs.  Few rows are split as long as every CTA
// can be resident at once and has 16 KB of the row.  The more rows there are, the
// smaller their blocks: more rows are then under way at once, whose beginnings and
// ends hide behind one another ([4096, 151936] bf16 took 225 us in blocks of 512
// threads, 198 of 256, 195 of 128, 197 of 64, and with 20 alternatives 417, 343,
// 304 and 302; [600, 151936] 43, 42 and, of 128, 60).  A thread has at least one
// batch of 16-byte vectors, and four where rows abound; rows of one warp share a
// block.
template <typename T>
fp8_status launch_logp(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int64_t* targets, int topk,
                       float* logprob, float* entropy, float* stats, float* top_logprob, int64_t* top_index,
                       cudaStream_t s) {
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    const int64_t bytes = vocab * static_cast<int64_t>(sizeof(T));
    int ranks = 1;
    while (ranks < logp::kMaxRanks && rows * ranks <= sms && bytes / (2 * ranks) >= 16384) ranks *= 2;
    const int64_t ctas = rows * ranks;
    const int most = ctas <= 3 * sms ? logp::kMaxThreads : ctas <= 7 * sms ? 256 : ctas <= 16 * sms ? 128 : 64;
    const int batches = ctas > 32 * static_cast<int64_t>(sms) ? 4 : 1;
    const int threads = pow2_between(bytes / ranks / (16 * logp::kBatch * batches), 32, most);
    const int warps = threads / 32, teams = warps == 1 ? logp::kTeams : 1;
    const int64_t grid = (ctas + teams - 1) / teams;
    if (grid > kMaxDim) return FP8_ERR_SHAPE;
    auto kernel = topk ? logp::forward_kernel<T, true> : logp::forward_kernel<T, false>;
    const T* x = static_cast<const T*>(logits);
    float2* st2 = reinterpret_cast<float2*>(stats);
    const dim3 blocks(static_cast<unsigned>(grid)), block(static_cast<unsigned>(threads * teams));
    const cudaError_t e =
        ranks > 1 ? launch_pdl_cluster(kernel, blocks, block, 0, static_cast<unsigned>(ranks), s, x, rows, vocab, ld,
                                       targets, topk, ranks, warps, logprob, entropy, st2, top_logprob, top_index)
                  : launch_pdl(kernel, blocks, block, 0, s, x, rows, vocab, ld, targets, topk, ranks, warps, logprob,
                               entropy, st2, top_logprob, top_index);
    if (e != cudaSuccess) return cuda_fail("token log probabilities launch", e);
    return last_launch_status("token log probabilities launch");
}

template <typename T>
fp8_status launch_logp_bwd(const void* logits, int64_t rows, int64_t vocab, int64_t ld, const int64_t* targets,
                           const float* stats, const float* dlogprob, const float* entropy, const float* dentropy,
                           void* dlogits, int64_t ld_out, cudaStream_t s) {
    const int64_t nvec = vocab / logp::Elem<T>::N;
    const int threads = pow2_between((nvec + logp::kBatch - 1) / logp::kBatch, 32, logp::kMaxThreads);
    const int64_t per = static_cast<int64_t>(threads) * logp::kBatch;
    const int64_t chunks = nvec > per ? (nvec + per - 1) / per : 1;
    if (rows > kMaxDim / chunks) return FP8_ERR_SHAPE;
    auto kernel = dentropy ? logp::backward_kernel<T, true> : logp::backward_kernel<T, false>;
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(rows * chunks)),
                                     dim3(static_cast<unsigned>(threads)), 0, s, static_cast<const T*>(logits), vocab, ld,
                                     targets, reinterpret_cast<const float2*>(stats), dlogprob, entropy, dentropy,
                                     chunks, static_cast<T*>(dlogits), ld_out);
    if (e != cudaSuccess) return cuda_fail("token log probabilities gradient launch", e);
    return last_launch_status("token log probabilities gradient launch");
}

// Newton-Schulz: the workspace's parts, each at a multiple of 256 bytes.
struct NsLayout {
    int64_t s, l;               // shorter and longer side
    int64_t x_ld, s_ld;         // row strides of X and of S, Q (multiples of 64)
    bool tall;                  // more rows than columns
    size_t partial, x[2], lo[2], gram, poly, sums, flags, bytes;   // X and what FP16 leaves of it, twice
    int slots;                  // partial sums of cut tiles
};
NsLayout ns_layout(int64_t batch, int64_t m, int64_t n) {
    NsLayout w;
    w.tall = m > n;
    w.s = w.tall ? n : m;
    w.l = w.tall ? m : n;
    w.x_ld = (n + 63) / 64 * 64;
    w.s_ld = (w.s + 63) / 64 * 64;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t x = up(static_cast<size_t>(batch * m * w.x_ld) * 2), q = up(static_cast<size_t>(batch * w.s * w.s_ld) * 2);
    w.partial = 0;
    w.x[0] = up(static_cast<size_t>(batch) * ns::kNormBlocks * sizeof(double));
    w.x[1] = w.x[0] + x;
    w.lo[0] = w.x[1] + x;
    w.lo[1] = w.lo[0] + x;
    w.gram = w.lo[1] + x;
    w.poly = w.gram + q;
    const int64_t side = (w.s + 255) / 256, symmetric = side * (side + 1) / 2 * batch;
    const int64_t apply = side * ((w.l + 255) / 256) * batch, kb_s = (w.s + 63) / 64, kb_l = (w.l + 63) / 64;
    w.slots = ns::slots_for(symmetric, kb_l);
    if (ns::slots_for(apply, kb_s) > w.slots) w.slots = ns::slots_for(apply, kb_s);
    w.sums = w.poly + q;
    w.flags = w.sums + static_cast<size_t>(w.slots) * ns::kSlotFloat4 * sizeof(float4);
    w.bytes = w.flags + up(static_cast<size_t>(w.slots) * 2 * ns::EPI_WARPS * sizeof(int));
    return w;
}

// What a call has to bring.  Where one launch takes the batch it uses none of it;
// a page all the same, so that a workspace is never NULL.
constexpr size_t kNsLeastWorkspace = 4096;
size_t ns_workspace(int64_t batch, int64_t m, int64_t n) {
    return ns::small::always_takes(batch, m, n) ? kNsLeastWorkspace : ns_layout(batch, m, n).bytes;
}

// [batch][rows][cols] 16-bit row-major matrices with rows of ld elements.
fp8_status make_map_3d(CUtensorMap* map, const void* base, int64_t cols, int64_t rows, int64_t batch, int64_t ld,
                       uint32_t box_x, uint32_t box_y, CUtensorMapSwizzle swizzle) {
    auto enc = tensor_map_encoder();
    if (!enc) return FP8_ERR_CUDA;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(ld) * rows * 2};
    cuuint32_t box[3] = {box_x, box_y, 1u};
    cuuint32_t estride[3] = {1u, 1u, 1u};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, estride,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        snprintf(g_detail, sizeof g_detail, "cuTensorMapEncodeTiled(3-D): CUresult %d", static_cast<int>(r));
        return FP8_ERR_CUDA;
    }
    return FP8_OK;
}

std::atomic<int> g_ns_attr_done[kMaxDevices];
std::atomic<int> g_ns_pairs[kMaxDevices][8];     // co-resident CTA pairs per kernel variant

template <int MODE, bool A_MN, bool B_MN>
fp8_status launch_ns_gemm(int dev, int sms, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c,
                          const CUtensorMap& t, ns::Params p, int64_t batch, int slots, cudaStream_t s) {
    constexpr int variant = MODE * 2 + (MODE == ns::kGram ? A_MN : B_MN);
    auto kernel = ns::gemm_kernel<MODE, A_MN, B_MN>;
    if ((g_ns_attr_done[dev].load(std::memory_order_acquire) & (1 << variant)) == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ns::SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(newton-schulz)", e);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1), 1, 1);
        cfg.blockDim = dim3(ns::THREADS, 1, 1);
        cfg.dynamicSmemBytes = ns::SMEM_BYTES;
        int pairs = 0;
        e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
        if (e != cudaSuccess) return cuda_fail("cudaOccupancyMaxActiveClusters(newton-schulz)", e);
        if (pairs <= 0) return cuda_fail("newton-schulz kernel cannot be resident", cudaErrorInvalidConfiguration);
        g_ns_pairs[dev][variant].store(pairs, std::memory_order_relaxed);
        g_ns_attr_done[dev].fetch_or(1 << variant, std::memory_order_release);
    }
    const int64_t total = static_cast<int64_t>(p.tiles) * batch;
    const int pairs = g_ns_pairs[dev][variant].load(std::memory_order_relaxed);
    // Whole tiles for the full waves; the rest cut.
    const int64_t rest = total % pairs;
    p.full = static_cast<int>(total - rest);
    const ns::Cut cut = ns::best_cut(rest, pairs, (p.K + ns::BK - 1) / ns::BK, slots);
    p.halves = cut.halves;
    p.parts = cut.parts;
    p.units = static_cast<int>(p.full + rest * cut.halves * cut.parts);
    const unsigned grid = 2u * static_cast<unsigned>(p.units < pairs ? p.units : pairs);
    const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(ns::THREADS), ns::SMEM_BYTES, s, a, b, c, t, p);
    if (e != cudaSuccess) return cuda_fail("newton-schulz product launch", e);
    return last_launch_status("newton-schulz product launch");
}

template <typename T>
fp8_status launch_ns_cast(const T* g, int64_t batch, int64_t m, int64_t n, int64_t ld, double* partial, float eps,
                          float scale, __half* hi, __half* lo, int* flags, int num_flags, int sms, cudaStream_t s) {
    const bool vec = n % 8 == 0;             // every row begins at a multiple of 16 bytes, as g does
    const int64_t per_block = static_cast<int64_t>(ns::kNormThreads) * 16;
    int64_t parts = (m * n + per_block - 1) / per_block;
    const int64_t want = (8 * static_cast<int64_t>(sms) + batch - 1) / batch;
    if (parts > want) parts = want;
    if (parts > ns::kNormBlocks) parts = ns::kNormBlocks;
    const dim3 block(ns::kNormThreads);
    cudaError_t e;
    auto norm = vec ? ns::norm_kernel<T, true> : ns::norm_kernel<T, false>;
    e = launch_pdl(norm, dim3(static_cast<unsigned>(parts), static_cast<unsigned>(batch)), block, 0, s, g, m * n, partial);
    if (e != cudaSuccess) return cuda_fail("newton-schulz norm launch", e);
    int64_t blocks = (m * (ld / 8) + ns::kNormThreads - 1) / ns::kNormThreads;
    const int64_t cap = (16 * static_cast<int64_t>(sms) + batch - 1) / batch;
    if (blocks > cap) blocks = cap;
    auto cast = vec ? ns::cast_kernel<T, true> : ns::cast_kernel<T, false>;
    e = launch_pdl(cast, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(batch)), block, 0, s, g,
                   static_cast<int>(m), static_cast<int>(n), static_cast<int>(ld), static_cast<const double*>(partial),
                   static_cast<int>(parts), eps, scale, hi, lo, flags, num_flags);
    if (e != cudaSuccess) return cuda_fail("newton-schulz cast launch", e);
    return last_launch_status("newton-schulz cast launch");
}

std::atomic<int> g_ns_small_attr_done[kMaxDevices];
std::atomic<int> g_ns_small_clusters[kMaxDevices][ns::small::kMaxRanks + 1];

template <typename T>
fp8_status ns_small_ready(int dev) {
    constexpr int bit = sizeof(T) == 4 ? 1 : 2;
    if ((g_ns_small_attr_done[dev].load(std::memory_order_acquire) & bit) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(ns::small::iterate_kernel<T>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, ns::small::kMaxSmem);
        if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(newton-schulz, small)", e);
        g_ns_small_attr_done[dev].fetch_or(bit, std::memory_order_release);
    }
    return FP8_OK;
}

// How many clusters of `ranks` CTAs run at once (a CTA fills its SM: its registers do).
template <typename T>
fp8_status ns_small_clusters(int dev, int sms, int ranks, int* clusters) {
    *clusters = ranks == 1 ? sms : g_ns_small_clusters[dev][ranks].load(std::memory_order_acquire);
    if (*clusters > 0) return FP8_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ranks));
    cfg.blockDim = dim3(ns::small::kThreads);
    cfg.dynamicSmemBytes = ns::small::kMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(clusters, ns::small::iterate_kernel<T>, &cfg);
    if (e != cudaSuccess) return cuda_fail("cudaOccupancyMaxActiveClusters(newton-schulz, small)", e);
    if (*clusters < 1) *clusters = 1;
    g_ns_small_clusters[dev][ranks].store(*clusters, std::memory_order_release);
    return FP8_OK;
}

// Whether one launch of clusters takes a batch (share > 0), and how it divides a
// matrix.  128 columns of X per CTA finish one matrix sooner than 256 (s x l = 64 x
// 1024: 34 against 42 us, 96 x 512: 45 against 62), but half as many matrices run at
// once, so 256 where that saves a round of clusters (32 x 64 x 1024: 43 against 102
// us).  Rounds follow one another, while the launch per product spreads a batch over
// tensor cores that a single matrix leaves idle.  Its tiles are 128 rows high: up to
// s = 80 it does not win (300 x 64 x 1024: 556 against 446; 148 x 80 x 640: 220 against
// 205), nor where a matrix has one CTA (1200 x 128 x 128: 573 against 453).  Else it
// does where the last of several rounds would be short (36 x 128 x 1024, 34 at once:
// 152 against 178; 100 x 100 x 640, 49 at once: 200 against 222; but 60 x 96 x 2500,
// 15 at once: 394 against 324), and for many matrices that nearly fill its tiles (100 x
// 128 x 1024: 281 against 366; 75 x 104 x 2048: 359 against 431; but 40 x 120 x 1500: 224
// against 188, 60 x 128 x 1024: 190 against 183).
template <typename T>
fp8_status ns_small_plan(int dev, int sms, int64_t batch, int s, int l, int* ranks, int* share) {
    const fp8_status ready = ns_small_ready<T>(dev);
    if (ready != FP8_OK) return ready;
    int64_t best = 0, room = 0;
    for (int columns = ns::small::kLeastShare; columns <= 2 * ns::small::kLeastShare; columns *= 2) {
        int r = (l + columns - 1) / columns;
        if (r > ns::small::kMaxRanks) r = ns::small::kMaxRanks;
        const int each = ns::small::up16((l + r - 1) / r);
        r = (l + each - 1) / each;                           // none without columns
        int clusters = 0;
        const fp8_status st = ns_small_clusters<T>(dev, sms, r, &clusters);
        if (st != FP8_OK) return st;
        const int64_t rounds = (batch + clusters - 1) / clusters;
        if (best != 0 && rounds >= best) continue;
        best = rounds;
        room = rounds * clusters;
        *ranks = r;
        *share = each;
    }
    const bool short_last = s > ns::small::kMaxShortOfAnyBatch && *ranks > 1 && best > 1 && 4 * batch < 3 * room;
    const bool many = s > 96 && *ranks > 2 && best > 1 && batch > 48;
    if (short_last || many) *share = 0;
    return FP8_OK;
}

// Small matrices, one launch.
template <typename T>
fp8_status launch_ns_small(const void* g, int64_t batch, int64_t m, int64_t n, const float* coefficients, int steps,
                           float eps, float scale, void* out, int ranks, int share, cudaStream_t s) {
    ns::small::Params p{};
    p.m = static_cast<int>(m);
    p.n = static_cast<int>(n);
    p.tall = m > n;
    p.s = p.tall ? p.n : p.m;
    p.l = p.tall ? p.m : p.n;
    p.ranks = ranks;
    p.share = share;
    p.steps = steps;
    p.eps = eps;
    p.scale = scale;
    for (int i = 0; i < 3 * steps; ++i) p.coeff[i] = coefficients[i];
    auto kernel = ns::small::iterate_kernel<T>;
    const dim3 grid(static_cast<unsigned>(batch * p.ranks)), block(ns::small::kThreads);
    p.apart = ranks > 1 && ns::small::smem_bytes_apart(p.s, share) <= ns::small::kMaxSmem;
    const size_t smem = static_cast<size_t>(p.apart ? ns::small::smem_bytes_apart(p.s, share) : ns::small::smem_bytes(p.s, share));
    const T* x = static_cast<const T*>(g);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(out);
    const cudaError_t e = p.ranks > 1 ? launch_pdl_cluster(kernel, grid, block, smem, static_cast<unsigned>(p.ranks), s, x, y, p)
                                      : launch_pdl(kernel, grid, block, smem, s, x, y, p);
    if (e != cudaSuccess) return cuda_fail("newton-schulz launch (small)", e);
    return last_launch_status("newton-schulz launch (small)");
}

// Scratch of fp8_block_gemm_wgrad_static_ws: the split schedule's workspace
// as a file-scope device array, for callers that cannot allocate device
// memory.  Every GPU that loads the library holds it until the process
// exits; it starts zeroed (module load) and every call clears the flags it
// needs zeroed.
constexpr size_t kStaticWsBytes = size_t(24) << 20;     // 24 MiB: up to 94 CTA pairs
static __device__ __align__(256) uint8_t g_static_ws[kStaticWsBytes];
std::atomic<void*> g_static_ws_ptr[kMaxDevices];         // its device address, per device
std::atomic<int> g_static_ws_pairs[kMaxDevices];         // resident GEMM CTA pairs, per device

}  // namespace

extern "C" {

fp8_status fp8_quantize_act_1x128(const void* x_bf16, int64_t rows, int64_t cols, int mode,
                                  uint8_t* q_row, float* s_row, uint8_t* q_colT, float* s_col,
                                  void* stream) {
    if (mode != FP8_ROWWISE && mode != FP8_COLWISE && mode != FP8_BOTH) return FP8_ERR_MODE;
    if (rows < 0 || cols < 0 || cols % 128 != 0 || rows > kMaxDim || cols > kMaxDim)
        return FP8_ERR_SHAPE;
    if ((mode & FP8_COLWISE) && rows % 128 != 0) return FP8_ERR_SHAPE;
    if (rows == 0 || cols == 0) return FP8_OK;
    if (!x_bf16) return FP8_ERR_NULL;
    if ((mode & FP8_ROWWISE) && (!q_row || !s_row)) return FP8_ERR_NULL;
    if ((mode & FP8_COLWISE) && (!q_colT || !s_col)) return FP8_ERR_NULL;
    if (!aligned16(x_bf16)) return FP8_ERR_ALIGN;
    if ((mode & FP8_ROWWISE) && (!aligned16(q_row) || !aligned16(s_row))) return FP8_ERR_ALIGN;
    if ((mode & FP8_COLWISE) && (!aligned16(q_colT) || !aligned16(s_col))) return FP8_ERR_ALIGN;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint4* x = static_cast<const uint4*>(x_bf16);
    if (mode == FP8_ROWWISE) {
        int dev = 0, sms = 0;
        fp8_status st = current_device(&dev);
        if (st != FP8_OK) return st;
        if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
        constexpr int kUnroll = 4;
        const int64_t groups = cols / 128;
        const int64_t units = rows * groups;
        const int64_t warps_needed = (units + 2 * kUnroll - 1) / (2 * kUnroll);
        int64_t blocks = (warps_needed + 7) / 8;
        const int64_t cap = static_cast<int64_t>(sms) * 8;
        if (blocks > cap) blocks = cap;
        const cudaError_t e = launch_pdl(quant_rowwise_kernel<kUnroll>, dim3(static_cast<unsigned>(blocks)),
                                         dim3(256), 0, s, x, units, rows, groups,
                                         reinterpret_cast<uint2*>(q_row), s_row);
        if (e != cudaSuccess) return cuda_fail("row-wise quantize launch", e);
        return last_launch_status("row-wise quantize launch");
    }
    if (mode == FP8_COLWISE)
        return launch_tile_quant<kTileColwise, kProdPlain>(x_bf16, rows, cols, nullptr, nullptr, q_colT, s_col, s);
    return launch_tile_quant<kTileBoth, kProdPlain>(x_bf16, rows, cols, q_row, s_row, q_colT, s_col, s);
}

fp8_status fp8_swiglu_quantize_1x128(const void* gate_up_bf16, int64_t rows, int64_t ffn, int mode,
                                     uint8_t* q_row, float* s_row, uint8_t* q_colT, float* s_col,
                                     void* stream) {
    if (mode != FP8_ROWWISE && mode != FP8_COLWISE && mode != FP8_BOTH) return FP8_ERR_MODE;
    if (rows < 0 || ffn < 0 || rows % 128 || ffn % 128 || rows > kMaxDim || ffn > kMaxDim / 2)
        return FP8_ERR_SHAPE;
    if (rows == 0 || ffn == 0) return FP8_OK;
    if (!gate_up_bf16) return FP8_ERR_NULL;
    if ((mode & FP8_ROWWISE) && (!q_row || !s_row)) return FP8_ERR_NULL;
    if ((mode & FP8_COLWISE) && (!q_colT || !s_col)) return FP8_ERR_NULL;
    if (!aligned16(gate_up_bf16)) return FP8_ERR_ALIGN;
    if ((mode & FP8_ROWWISE) && (!aligned16(q_row) || !aligned16(s_row))) return FP8_ERR_ALIGN;
    if ((mode & FP8_COLWISE) && (!aligned16(q_colT) || !aligned16(s_col))) return FP8_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (mode == FP8_ROWWISE)
        return launch_tile_quant<kTileRowwise, kProdSwiglu>(gate_up_bf16, rows, ffn, q_row, s_row, nullptr, nullptr, s);
    if (mode == FP8_COLWISE)
        return launch_tile_quant<kTileColwise, kProdSwiglu>(gate_up_bf16, rows, ffn, nullptr, nullptr, q_colT, s_col, s);
    return launch_tile_quant<kTileBoth, kProdSwiglu>(gate_up_bf16, rows, ffn, q_row, s_row, q_colT, s_col, s);
}

fp8_status fp8_rmsnorm_rstd(const void* x_bf16, int64_t rows, int64_t cols, float eps, float* rstd,
                            void* stream) {
    if (rows < 0 || cols < 0 || cols % 8 || rows > kMaxDim || cols > kMaxDim) return FP8_ERR_SHAPE;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8_ERR_SHAPE;
    if (rows == 0 || cols == 0) return FP8_OK;
    if (!x_bf16 || !rstd) return FP8_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned16(rstd)) return FP8_ERR_ALIGN;
    const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
    const cudaError_t e = launch_pdl(rmsnorm_rstd_kernel, dim3(grid), dim3(256), 0, static_cast<cudaStream_t>(stream),
                                     static_cast<const uint4*>(x_bf16), rows, cols, eps, rstd);
    if (e != cudaSuccess) return cuda_fail("rmsnorm rstd launch", e);
    return last_launch_status("rmsnorm rstd launch");
}

fp8_status fp8_rmsnorm_quantize_1x128(const void* x_bf16, int64_t rows, int64_t cols, const float* rstd,
                                      const void* gamma_bf16, int mode, uint8_t* q_row, float* s_row,
                                      uint8_t* q_colT, float* s_col, void* stream) {
    if (mode != FP8_ROWWISE && mode != FP8_COLWISE && mode != FP8_BOTH) return FP8_ERR_MODE;
    if (rows < 0 || cols < 0 || rows % 128 || cols % 128 || rows > kMaxDim || cols > kMaxDim)
        return FP8_ERR_SHAPE;
    if (rows == 0 || cols == 0) return FP8_OK;
    if (!x_bf16 || !rstd || !gamma_bf16) return FP8_ERR_NULL;
    if ((mode & FP8_ROWWISE) && (!q_row || !s_row)) return FP8_ERR_NULL;
    if ((mode & FP8_COLWISE) && (!q_colT || !s_col)) return FP8_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned16(rstd) || !aligned16(gamma_bf16)) return FP8_ERR_ALIGN;
    if ((mode & FP8_ROWWISE) && (!aligned16(q_row) || !aligned16(s_row))) return FP8_ERR_ALIGN;
    if ((mode & FP8_COLWISE) && (!aligned16(q_colT) || !aligned16(s_col))) return FP8_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (mode == FP8_ROWWISE)
        return launch_tile_quant<kTileRowwise, kProdNorm>(x_bf16, rows, cols, q_row, s_row, nullptr, nullptr, s,
                                                          rstd, gamma_bf16);
    if (mode == FP8_COLWISE)
        return launch_tile_quant<kTileColwise, kProdNorm>(x_bf16, rows, cols, nullptr, nullptr, q_colT, s_col, s,
                                                          rstd, gamma_bf16);
    return launch_tile_quant<kTileBoth, kProdNorm>(x_bf16, rows, cols, q_row, s_row, q_colT, s_col, s, rstd,
                                                   gamma_bf16);
}

fp8_status fp8_add_rmsnorm_quantize_1x128(const void* x_bf16, const void* residual_bf16, int64_t rows, int64_t cols,
                                          float eps, const void* gamma_bf16, int mode, void* sum_bf16, float* rstd,
                                          uint8_t* q_row, float* s_row, uint8_t* q_colT, float* s_col, void* stream) {
    if (mode != FP8_ROWWISE && mode != FP8_COLWISE && mode != FP8_BOTH) return FP8_ERR_MODE;
    if (rows < 0 || cols < 0 || cols % 128 || rows > kMaxDim || cols > FP8_MAX_NORM_COLS) return FP8_ERR_SHAPE;
    if ((mode & FP8_COLWISE) && rows % 128) return FP8_ERR_SHAPE;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return FP8_ERR_SHAPE;
    if (rows == 0 || cols == 0) return FP8_OK;
    if (!x_bf16 || !rstd || !gamma_bf16 || (residual_bf16 && !sum_bf16)) return FP8_ERR_NULL;
    if ((mode & FP8_ROWWISE) && (!q_row || !s_row)) return FP8_ERR_NULL;
    if ((mode & FP8_COLWISE) && (!q_colT || !s_col)) return FP8_ERR_NULL;
    if (!aligned16(x_bf16) || !aligned16(rstd) || !aligned16(gamma_bf16) || !aligned16(residual_bf16) ||
        !aligned16(sum_bf16))
        return FP8_ERR_ALIGN;
    if ((mode & FP8_ROWWISE) && (!aligned16(q_row) || !aligned16(s_row))) return FP8_ERR_ALIGN;
    if ((mode & FP8_COLWISE) && (!aligned16(q_colT) || !aligned16(s_col))) return FP8_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!(mode & FP8_ROWWISE)) q_row = nullptr;
    const fp8_status st = norm_rows(x_bf16, residual_bf16, gamma_bf16, rows, cols, eps, sum_bf16, rstd, q_row, s_row, s);
    if (st != FP8_OK || mode == FP8_ROWWISE) return st;
    return norm_cols(residual_bf16 ? sum_bf16 : x_bf16, rstd, gamma_bf16, rows, cols, q_colT, s_col, s);
}

fp8_status fp8_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes) return FP8_ERR_NULL;
    if (rows < 0 || cols < 0 || cols % 128 || rows > kMaxDim || cols > FP8_MAX_NORM_COLS) return FP8_ERR_SHAPE;
    *bytes = 0;
    if (rows == 0 || cols == 0) return FP8_OK;
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    const BwdShape b = norm_bwd_shape(rows, cols, sms);
    if (b.grid > 1) *bytes = static_cast<size_t>(b.grid) * static_cast<size_t>(cols) * sizeof(float);
    return FP8_OK;
}

fp8_status fp8_rmsnorm_backward(const void* dy_bf16, const void* s_bf16, const float* rstd, const void* gamma_bf16,
                                const void* dresidual_bf16, int64_t rows, int64_t cols, void* ds_bf16,
                                float* dgamma_f32, int accumulate, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (accumulate != 0 && accumulate != 1) return FP8_ERR_MODE;
    if (rows < 0 || cols < 0 || cols % 128 || rows > kMaxDim || cols > FP8_MAX_NORM_COLS) return FP8_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cols == 0) return FP8_OK;
    if (!aligned16(dgamma_f32) || !aligned16(workspace)) return FP8_ERR_ALIGN;
    if (rows == 0) {                   // the sum over no rows
        if (dgamma_f32 && !accumulate) {
            const cudaError_t e = cudaMemsetAsync(dgamma_f32, 0, static_cast<size_t>(cols) * sizeof(float), s);
            if (e != cudaSuccess) return cuda_fail("cudaMemsetAsync(dgamma)", e);
        }
        return FP8_OK;
    }
    if (!dy_bf16 || !s_bf16 || !rstd || !gamma_bf16 || !ds_bf16) return FP8_ERR_NULL;
    if (!aligned16(dy_bf16) || !aligned16(s_bf16) || !aligned16(rstd) || !aligned16(gamma_bf16) ||
        !aligned16(dresidual_bf16) || !aligned16(ds_bf16))
        return FP8_ERR_ALIGN;
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    const BwdShape b = norm_bwd_shape(rows, cols, sms);
    if (dgamma_f32 && b.grid > 1) {
        if (!workspace) return FP8_ERR_NULL;
        if (workspace_bytes < static_cast<size_t>(b.grid) * static_cast<size_t>(cols) * sizeof(float))
            return FP8_ERR_SHAPE;
    }
    float* partial = static_cast<float*>(workspace);
    cudaError_t e;
    if (b.cpt == 1)
        e = launch_norm_bwd<1, 2, true>(b, dy_bf16, s_bf16, rstd, gamma_bf16, dresidual_bf16, rows, ds_bf16, partial,
                                        dgamma_f32, accumulate, s);
    else if (b.cpt == 2)
        e = launch_norm_bwd<2, 1, true>(b, dy_bf16, s_bf16, rstd, gamma_bf16, dresidual_bf16, rows, ds_bf16, partial,
                                        dgamma_f32, accumulate, s);
    else                               // (its registers do not hold two rows' chunks)
        e = launch_norm_bwd<4, 1, false>(b, dy_bf16, s_bf16, rstd, gamma_bf16, dresidual_bf16, rows, ds_bf16, partial,
                                         dgamma_f32, accumulate, s);
    if (e != cudaSuccess) return cuda_fail("rmsnorm backward launch", e);
    if ((st = last_launch_status("rmsnorm backward launch")) != FP8_OK) return st;
    if (dgamma_f32 && b.grid > 1) {
        e = launch_pdl(addnorm::dgamma_kernel, dim3(static_cast<unsigned>(cols / 32)), dim3(32 * addnorm::kDgammaWarps), 0, s,
                       static_cast<const float*>(partial), static_cast<int>(b.grid), static_cast<int>(cols),
                       dgamma_f32, accumulate);
        if (e != cudaSuccess) return cuda_fail("dgamma launch", e);
        return last_launch_status("dgamma launch");
    }
    return FP8_OK;
}

fp8_status fp8_token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                              const int64_t* targets, int topk, float* logprob, float* entropy, float* stats,
                              float* top_logprob, int64_t* top_index, void* stream) {
    if (!dtype_ok(dtype)) return FP8_ERR_MODE;
    if (rows < 0 || vocab < 1 || ld < vocab || rows > kMaxDim || vocab > kMaxDim || ld > kMaxLd) return FP8_ERR_SHAPE;
    if (topk < 0 || topk > FP8_MAX_TOPK || topk > vocab) return FP8_ERR_SHAPE;
    if (rows == 0) return FP8_OK;
    if (!logits || !stats || (logprob && !targets) || (topk && (!top_logprob || !top_index))) return FP8_ERR_NULL;
    if (!element_aligned(logits, dtype) || !aligned16(targets) || !aligned16(logprob) || !aligned16(entropy) ||
        !aligned16(stats) || !aligned16(top_logprob) || !aligned16(top_index))
        return FP8_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FP8_BF16)
        return launch_logp<__nv_bfloat16>(logits, rows, vocab, ld, targets, topk, logprob, entropy, stats, top_logprob,
                                          top_index, s);
    return launch_logp<float>(logits, rows, vocab, ld, targets, topk, logprob, entropy, stats, top_logprob, top_index,
                              s);
}

fp8_status fp8_token_logprobs_backward(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld,
                                       const int64_t* targets, const float* stats, const float* dlogprob,
                                       const float* entropy, const float* dentropy, void* dlogits, int64_t ld_out,
                                       void* stream) {
    if (!dtype_ok(dtype)) return FP8_ERR_MODE;
    if (rows < 0 || vocab < 1 || ld < vocab || ld_out < vocab || rows > kMaxDim || vocab > kMaxDim || ld > kMaxLd ||
        ld_out > kMaxLd)
        return FP8_ERR_SHAPE;
    if (rows == 0) return FP8_OK;
    if (!logits || !stats || !dlogits || (dlogprob && !targets) || (dentropy && !entropy)) return FP8_ERR_NULL;
    if (!element_aligned(logits, dtype) || !element_aligned(dlogits, dtype) || !aligned16(targets) ||
        !aligned16(stats) || !aligned16(dlogprob) || !aligned16(entropy) || !aligned16(dentropy))
        return FP8_ERR_ALIGN;
    if (logits == dlogits && ld != ld_out) return FP8_ERR_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FP8_BF16)
        return launch_logp_bwd<__nv_bfloat16>(logits, rows, vocab, ld, targets, stats, dlogprob, entropy, dentropy,
                                              dlogits, ld_out, s);
    return launch_logp_bwd<float>(logits, rows, vocab, ld, targets, stats, dlogprob, entropy, dentropy, dlogits,
                                  ld_out, s);
}

fp8_status fp8_newton_schulz_workspace_bytes(int64_t batch, int64_t m, int64_t n, size_t* bytes) {
    if (!bytes) return FP8_ERR_NULL;
    if (batch < 0 || m < 1 || n < 1 || batch > FP8_NS_MAX_BATCH || m > ns::kMaxSide || n > ns::kMaxSide)
        return FP8_ERR_SHAPE;
    *bytes = batch ? ns_workspace(batch, m, n) : 0;
    return FP8_OK;
}

fp8_status fp8_newton_schulz(const void* g, int dtype, int64_t batch, int64_t m, int64_t n, const float* coefficients,
                             int steps, float eps, void* out_bf16, void* workspace, size_t workspace_bytes,
                             void* stream) {
    if (!dtype_ok(dtype)) return FP8_ERR_MODE;
    if (batch < 0 || m < 1 || n < 1 || batch > FP8_NS_MAX_BATCH || m > ns::kMaxSide || n > ns::kMaxSide)
        return FP8_ERR_SHAPE;
    if (steps < 1 || steps > FP8_NS_MAX_STEPS || !(eps >= 0.0f) || eps > 3.0e38f) return FP8_ERR_SHAPE;
    if (!coefficients) return FP8_ERR_NULL;
    for (int i = 0; i < 3 * steps; ++i)
        if (!(coefficients[i] >= -FP8_NS_MAX_COEFFICIENT && coefficients[i] <= FP8_NS_MAX_COEFFICIENT)) return FP8_ERR_SHAPE;
    if (batch == 0) return FP8_OK;
    if (!g || !out_bf16 || !workspace) return FP8_ERR_NULL;
    if (!aligned16(g) || !aligned16(out_bf16) || !aligned16(workspace)) return FP8_ERR_ALIGN;
    if (workspace_bytes < ns_workspace(batch, m, n)) return FP8_ERR_SHAPE;
    int dev = 0, sms = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    // X is kept times the power of two at or below sqrt(m n), at most 2^13
    // (entries of X up to 8 then stay inside FP16's range).
    float scale = 1.0f;
    while (scale < 8192.0f && 4.0 * scale * scale <= static_cast<double>(m) * static_cast<double>(n)) scale *= 2.0f;
    if (ns::small::takes(m, n)) {
        const int shorter = static_cast<int>(m < n ? m : n), longer = static_cast<int>(m < n ? n : m);
        const bool f32 = dtype == FP8_F32;
        int ranks = 0, share = 0;
        st = f32 ? ns_small_plan<float>(dev, sms, batch, shorter, longer, &ranks, &share)
                 : ns_small_plan<__nv_bfloat16>(dev, sms, batch, shorter, longer, &ranks, &share);
        if (st != FP8_OK) return st;
        if (share > 0)
            return f32 ? launch_ns_small<float>(g, batch, m, n, coefficients, steps, eps, scale, out_bf16, ranks, share, s)
                       : launch_ns_small<__nv_bfloat16>(g, batch, m, n, coefficients, steps, eps, scale, out_bf16, ranks,
                                                        share, s);
    }
    const NsLayout w = ns_layout(batch, m, n);
    if (workspace_bytes < w.bytes) return FP8_ERR_SHAPE;         // (a page was enough only for one launch)
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    __half *x[2], *lo[2];
    for (int i = 0; i < 2; ++i) {
        x[i] = reinterpret_cast<__half*>(ws + w.x[i]);
        lo[i] = reinterpret_cast<__half*>(ws + w.lo[i]);
    }
    __half* gram = reinterpret_cast<__half*>(ws + w.gram);
    __half* poly = reinterpret_cast<__half*>(ws + w.poly);
    double* partial = reinterpret_cast<double*>(ws + w.partial);
    int* flags = reinterpret_cast<int*>(ws + w.flags);
    const int num_flags = w.slots * 2 * ns::EPI_WARPS;
    st = dtype == FP8_F32 ? launch_ns_cast(static_cast<const float*>(g), batch, m, n, w.x_ld, partial, eps, scale, x[0],
                                           lo[0], flags, num_flags, sms, s)
                          : launch_ns_cast(static_cast<const __nv_bfloat16*>(g), batch, m, n, w.x_ld, partial, eps, scale,
                                           x[0], lo[0], flags, num_flags, sms, s);
    if (st != FP8_OK) return st;

    constexpr CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B, flat = CU_TENSOR_MAP_SWIZZLE_NONE;
    CUtensorMap x_rows[2], x_half[2], x_out[2], lo_out[2], s_in, s_half, s_out, s_outT, q_in, q_half, q_out, q_outT,
        final_map;
    for (int i = 0; i < 2; ++i) {
        if ((st = make_map_3d(&x_rows[i], x[i], w.x_ld, m, batch, w.x_ld, 64, 128, sw)) != FP8_OK) return st;
        if ((st = make_map_3d(&x_half[i], x[i], w.x_ld, m, batch, w.x_ld, 64, 64, sw)) != FP8_OK) return st;
        if ((st = make_map_3d(&lo_out[i], lo[i], w.x_ld, m, batch, w.x_ld, 64, 32, sw)) != FP8_OK) return st;
        if ((st = make_map_3d(&x_out[i], x[i], w.x_ld, m, batch, w.x_ld, 64, 32, sw)) != FP8_OK) return st;
    }
    if ((st = make_map_3d(&s_in, gram, w.s_ld, w.s, batch, w.s_ld, 64, 128, sw)) != FP8_OK) return st;
    if ((st = make_map_3d(&s_half, gram, w.s_ld, w.s, batch, w.s_ld, 64, 64, sw)) != FP8_OK) return st;
    if ((st = make_map_3d(&s_out, gram, w.s_ld, w.s, batch, w.s_ld, 64, 32, sw)) != FP8_OK) return st;
    if ((st = make_map_3d(&s_outT, gram, w.s_ld, w.s, batch, w.s_ld, 32, 64, flat)) != FP8_OK) return st;
    if ((st = make_map_3d(&q_in, poly, w.s_ld, w.s, batch, w.s_ld, 64, 128, sw)) != FP8_OK) return st;
    if ((st = make_map_3d(&q_half, poly, w.s_ld, w.s, batch, w.s_ld, 64, 64, sw)) != FP8_OK) return st;
    if ((st = make_map_3d(&q_out, poly, w.s_ld, w.s, batch, w.s_ld, 64, 32, sw)) != FP8_OK) return st;
    if ((st = make_map_3d(&q_outT, poly, w.s_ld, w.s, batch, w.s_ld, 32, 64, flat)) != FP8_OK) return st;
    const bool tma_out = n % 8 == 0;             // the output's rows are multiples of 16 bytes
    if (tma_out) {
        if ((st = make_map_3d(&final_map, out_bf16, n, m, batch, n, 64, 32, sw)) != FP8_OK) return st;
    } else {
        final_map = x_out[0];                    // not used
    }

    ns::Params base{};
    base.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    base.sums = reinterpret_cast<float4*>(ws + w.sums);
    base.flags = flags;
    const int side = static_cast<int>((w.s + 255) / 256);
    for (int i = 0; i < steps; ++i) {
        const int cur = i & 1;
        const bool lin = i <= ns::kCarry;                    // X's linear term from both its parts
        ns::Params p = base;                                 // S
        p.M = p.N = static_cast<int>(w.s);
        p.K = static_cast<int>(w.l);
        p.tiles_m = p.tiles_n = side;
        p.tiles = side * (side + 1) / 2;
        p.alpha = 1.0f / (scale * scale);
        p.product = 3 * i + 1;
        st = w.tall ? launch_ns_gemm<ns::kGram, true, true>(dev, sms, x_half[cur], x_half[cur], s_out, s_outT, p, batch,
                                                            w.slots, s)
                    : launch_ns_gemm<ns::kGram, false, false>(dev, sms, x_rows[cur], x_half[cur], s_out, s_outT, p, batch,
                                                              w.slots, s);
        if (st != FP8_OK) return st;
        p.K = static_cast<int>(w.s);                         // Q
        p.a = lin ? 0.0f : coefficients[3 * i];
        p.b = coefficients[3 * i + 1];
        p.c = coefficients[3 * i + 2];
        p.e0 = gram;
        p.e_ld = w.s_ld;
        p.product = 3 * i + 2;
        st = launch_ns_gemm<ns::kPoly, false, false>(dev, sms, s_in, s_half, q_out, q_outT, p, batch, w.slots, s);
        if (st != FP8_OK) return st;
        p = base;                                            // X
        p.M = static_cast<int>(m);
        p.N = static_cast<int>(n);
        p.K = static_cast<int>(w.s);
        p.tiles_m = static_cast<int>((m + 255) / 256);
        p.tiles_n = static_cast<int>((n + 255) / 256);
        p.tiles = p.tiles_m * p.tiles_n;
        p.row_fast = w.tall ? 0 : 1;
        p.alpha = 1.0f / scale;
        p.final_out = i == steps - 1;
        if (lin) {
            p.a = coefficients[3 * i];
            p.e0 = x[cur];
            p.e1 = lo[cur];
            p.e_ld = w.x_ld;
        }
        p.carry = i < ns::kCarry && !p.final_out;
        p.out = p.final_out && !tma_out ? static_cast<__nv_bfloat16*>(out_bf16) : nullptr;
        const CUtensorMap& c = p.final_out ? final_map : x_out[cur ^ 1];
        p.product = 3 * i + 3;
        st = w.tall ? launch_ns_gemm<ns::kApply, false, false>(dev, sms, x_rows[cur], q_half, c, lo_out[cur ^ 1], p, batch,
                                                               w.slots, s)
                    : launch_ns_gemm<ns::kApply, false, true>(dev, sms, q_in, x_half[cur], c, lo_out[cur ^ 1], p, batch,
                                                              w.slots, s);
        if (st != FP8_OK) return st;
    }
    return FP8_OK;
}

fp8_status fp8_quantize_weight_128x128(const void* w_bf16, int64_t n, int64_t k, uint8_t* wq,
                                       float* sw, uint8_t* wqT, void* stream) {
    if (n < 0 || k < 0 || n % 128 || k % 128 || n > kMaxDim || k > kMaxDim) return FP8_ERR_SHAPE;
    if (n == 0 || k == 0) return FP8_OK;
    if (!w_bf16 || !wq || !sw) return FP8_ERR_NULL;
    if (!aligned16(w_bf16) || !aligned16(wq) || !aligned16(sw) || (wqT && !aligned16(wqT)))
        return FP8_ERR_ALIGN;
    return launch_tile_quant<kTileWeight, kProdPlain>(w_bf16, n, k, wq, nullptr, wqT, sw,
                                          static_cast<cudaStream_t>(stream));
}

fp8_status fp8_block_gemm_fprop(const uint8_t* xq, const float* sx, const uint8_t* wq,
                                const float* sw, void* y_bf16, int64_t M, int64_t N, int64_t K,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (!dims_ok_gemm(M, N, K, false) || K > FP8_MAX_CONTRACTION_FPROP) return FP8_ERR_SHAPE;
    if (M == 0) return FP8_OK;
    if (!xq || !sx || !wq || !sw || !y_bf16) return FP8_ERR_NULL;
    if (!aligned16(xq) || !aligned16(sx) || !aligned16(wq) || !aligned16(sw) || !aligned16(y_bf16) ||
        !aligned16(workspace))
        return FP8_ERR_ALIGN;
    gemm::Params p{};
    p.sa = sx;
    p.sa_ld = M;                 // sx [K/128, M]
    p.sb = sw;
    p.sb_sn = K / 128;           // sw [N/128, K/128]
    p.sb_sk = 1;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    return launch_gemm<gemm::kScaleRowBlock, gemm::kOutBf16>(xq, wq, y_bf16, p, workspace, workspace_bytes,
                                                             static_cast<cudaStream_t>(stream));
}

fp8_status fp8_block_gemm_dgrad(const uint8_t* dyq, const float* sdy, const uint8_t* wqT,
                                const float* sw, void* dx_bf16, int64_t M, int64_t N, int64_t K,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (!dims_ok_gemm(M, K, N, false) || N > FP8_MAX_CONTRACTION_FPROP) return FP8_ERR_SHAPE;
    if (M == 0) return FP8_OK;
    if (!dyq || !sdy || !wqT || !sw || !dx_bf16) return FP8_ERR_NULL;
    if (!aligned16(dyq) || !aligned16(sdy) || !aligned16(wqT) || !aligned16(sw) || !aligned16(dx_bf16) ||
        !aligned16(workspace))
        return FP8_ERR_ALIGN;
    gemm::Params p{};
    p.sa = sdy;
    p.sa_ld = M;                 // sdy [N/128, M]
    p.sb = sw;                   // s_b(output block kb, slab nb) = sw[nb][kb]
    p.sb_sn = 1;
    p.sb_sk = K / 128;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(K);
    p.K = static_cast<int>(N);
    return launch_gemm<gemm::kScaleRowBlock, gemm::kOutBf16>(dyq, wqT, dx_bf16, p, workspace, workspace_bytes,
                                                             static_cast<cudaStream_t>(stream));
}

fp8_status fp8_block_gemm_wgrad(const uint8_t* dyqT, const float* sdyT, const uint8_t* xqT,
                                const float* sxT, void* dw_bf16, int64_t N, int64_t K, int64_t M,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (!dims_ok_gemm(N, K, M, true)) return FP8_ERR_SHAPE;
    if (!dyqT || !sdyT || !xqT || !sxT || !dw_bf16) return FP8_ERR_NULL;
    if (!aligned16(dyqT) || !aligned16(sdyT) || !aligned16(xqT) || !aligned16(sxT) || !aligned16(dw_bf16) ||
        !aligned16(workspace))
        return FP8_ERR_ALIGN;
    return launch_gemm<gemm::kScaleOuter, gemm::kOutBf16>(dyqT, xqT, dw_bf16, wgrad_params(sdyT, sxT, N, K, M),
                                                          workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

fp8_status fp8_block_gemm_wgrad_accum_f32(const uint8_t* dyqT, const float* sdyT, const uint8_t* xqT,
                                          const float* sxT, float* dw_f32, int64_t N, int64_t K, int64_t M,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    if (!dims_ok_gemm(N, K, M, true)) return FP8_ERR_SHAPE;
    if (!dyqT || !sdyT || !xqT || !sxT || !dw_f32) return FP8_ERR_NULL;
    if (!aligned16(dyqT) || !aligned16(sdyT) || !aligned16(xqT) || !aligned16(sxT) || !aligned16(dw_f32) ||
        !aligned16(workspace))
        return FP8_ERR_ALIGN;
    return launch_gemm<gemm::kScaleOuter, gemm::kOutAccF32>(dyqT, xqT, dw_f32, wgrad_params(sdyT, sxT, N, K, M),
                                                            workspace, workspace_bytes,
                                                            static_cast<cudaStream_t>(stream));
}

fp8_status fp8_block_gemm_wgrad_reduce_scatter_f32(const uint8_t* dyqT, const float* sdyT, const uint8_t* xqT,
                                                  const float* sxT, float* const* dw_shards, int nranks,
                                                  int64_t N, int64_t K, int64_t M, void* workspace,
                                                  size_t workspace_bytes, void* stream) {
    if (!dims_ok_gemm(N, K, M, true)) return FP8_ERR_SHAPE;
    if (nranks < 1 || nranks > gemm::kMaxShards || N % nranks) return FP8_ERR_SHAPE;
    if (!dyqT || !sdyT || !xqT || !sxT || !dw_shards) return FP8_ERR_NULL;
    if (!aligned16(dyqT) || !aligned16(sdyT) || !aligned16(xqT) || !aligned16(sxT) || !aligned16(workspace))
        return FP8_ERR_ALIGN;
    gemm::Params p = wgrad_params(sdyT, sxT, N, K, M);
    for (int q = 0; q < nranks; ++q) {
        if (!dw_shards[q]) return FP8_ERR_NULL;
        if (!aligned16(dw_shards[q])) return FP8_ERR_ALIGN;
        p.shards[q] = dw_shards[q];
    }
    p.shard_rows = N / nranks;
    return launch_gemm<gemm::kScaleOuter, gemm::kOutAccF32Shards>(dyqT, xqT, dw_shards[0], p, workspace,
                                                                  workspace_bytes, static_cast<cudaStream_t>(stream));
}

fp8_status fp8_block_gemm_wgrad_static_ws(const uint8_t* dyqT, const float* sdyT, const uint8_t* xqT,
                                          const float* sxT, void* dw_bf16, int64_t N, int64_t K, int64_t M,
                                          void* stream) {
    if (!dims_ok_gemm(N, K, M, true)) return FP8_ERR_SHAPE;
    if (!dyqT || !sdyT || !xqT || !sxT || !dw_bf16) return FP8_ERR_NULL;
    if (!aligned16(dyqT) || !aligned16(sdyT) || !aligned16(xqT) || !aligned16(sxT) || !aligned16(dw_bf16))
        return FP8_ERR_ALIGN;
    int dev = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    void* ws = g_static_ws_ptr[dev].load(std::memory_order_acquire);
    if (!ws) {
        // Set-up, once per device, with that device current: the array's
        // device address (the host-side name is only a stand-in for it) and
        // the number of CTA pairs, which sizes the part of it in use.
        void* ptr = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&ptr, g_static_ws);
        if (e != cudaSuccess || !ptr) return cuda_fail("cudaGetSymbolAddress(static GEMM workspace)", e);
        int sms = 0, pairs = 0;
        if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
        if ((st = gemm_pairs<gemm::kScaleOuter, gemm::kOutBf16, false>(dev, sms, &pairs)) != FP8_OK) return st;
        g_static_ws_pairs[dev].store(pairs, std::memory_order_relaxed);
        g_static_ws_ptr[dev].store(ptr, std::memory_order_release);
        ws = ptr;
    }
    const int pairs = g_static_ws_pairs[dev].load(std::memory_order_relaxed);
    const size_t need = gemm_workspace_bytes(pairs);
    if (need > kStaticWsBytes) {
        snprintf(g_detail, sizeof g_detail,
                 "this GPU's GEMM workspace needs %zu bytes, more than the %zu-byte static one", need,
                 kStaticWsBytes);
        return FP8_ERR_SHAPE;
    }
    // The flags must be zero when a call starts; a call that timed out can
    // leave some set, so they are cleared every time (a memset, not an
    // allocation).
    const size_t flags_off = size_t(pairs) * kPartialFloatsPerPair * sizeof(float);
    const size_t flags_bytes = size_t(pairs) * 2 * gemm::EPI_WARPS * 32 * sizeof(int);
    const cudaError_t e =
        cudaMemsetAsync(static_cast<uint8_t*>(ws) + flags_off, 0, flags_bytes, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail("cudaMemsetAsync(static GEMM workspace flags)", e);
    return launch_gemm<gemm::kScaleOuter, gemm::kOutBf16>(dyqT, xqT, dw_bf16, wgrad_params(sdyT, sxT, N, K, M), ws,
                                                          kStaticWsBytes, static_cast<cudaStream_t>(stream));
}

fp8_status fp8_gemm_workspace_bytes(size_t* bytes) {
    if (!bytes) return FP8_ERR_NULL;
    int dev = 0;
    fp8_status st = current_device(&dev);
    if (st != FP8_OK) return st;
    // Resident CTA pairs of the GEMM kernels (all variants share one shape).
    int sms = 0, pairs = 0;
    if ((st = sm_count(dev, &sms)) != FP8_OK) return st;
    if ((st = gemm_pairs<gemm::kScaleRowBlock, gemm::kOutBf16, false>(dev, sms, &pairs)) != FP8_OK) return st;
    *bytes = gemm_workspace_bytes(pairs);
    return FP8_OK;
}

fp8_status fp8_get_error(void) {
    unsigned int v = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail("cudaDeviceSynchronize", e);
    e = cudaMemcpyFromSymbol(&v, fp8blk::g_error_word, sizeof v);
    if (e != cudaSuccess) return cuda_fail("cudaMemcpyFromSymbol", e);
    return static_cast<fp8_status>(v);
}

fp8_status fp8_clear_error(void) {
    const unsigned int zero = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail("cudaDeviceSynchronize", e);
    e = cudaMemcpyToSymbol(fp8blk::g_error_word, &zero, sizeof zero);
    if (e != cudaSuccess) return cuda_fail("cudaMemcpyToSymbol", e);
    return FP8_OK;
}

const char* fp8_last_cuda_error(void) { return g_detail; }

fp8_status fp8_set_gemm_split_min_work(int64_t units_per_pair) {
    if (units_per_pair < 0) return FP8_ERR_SHAPE;
    g_split_min_units.store(units_per_pair, std::memory_order_relaxed);
    return FP8_OK;
}

fp8_status fp8_set_wait_timeout_ns(uint64_t ns) {
    g_wait_ns.store(ns ? ns : kDefaultWaitNs, std::memory_order_relaxed);
    return FP8_OK;
}

const char* fp8_status_string(fp8_status status) {
    switch (status) {
        case FP8_OK: return "ok";
        case FP8_ERR_NULL: return "a required pointer is NULL";
        case FP8_ERR_SHAPE: return "unsupported shape";
        case FP8_ERR_ALIGN: return "pointer not 16-byte aligned";
        case FP8_ERR_MODE: return "unknown mode";
        case FP8_ERR_CUDA: return "CUDA call or kernel launch failed";
        case FP8_ERR_TIMEOUT: return "a bounded device wait timed out";
    }
    return "unknown status";
}

fp8_status fp8_cast_e4m3_scaled(const float* x, float scale, uint8_t* q, int64_t n, void* stream) {
    if (n < 0) return FP8_ERR_SHAPE;
    if (n == 0) return FP8_OK;
    if (!x || !q) return FP8_ERR_NULL;
    const int64_t blocks = (n + 255) / 256;
    if (blocks > kMaxDim) return FP8_ERR_SHAPE;
    cast_e4m3_scaled_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        x, scale, q, n);
    return last_launch_status("cast launch");
}

fp8_status fp8_selftest_division(unsigned long long* result, void* stream) {
    if (!result) return FP8_ERR_NULL;
    if (!aligned16(result)) return FP8_ERR_ALIGN;
    division_selftest_kernel<<<0x7F7F, 256, 0, static_cast<cudaStream_t>(stream)>>>(result);
    return last_launch_status("division self-test launch");
}

fp8_status fp8_selftest_silu_bf16(uint16_t* out, void* stream) {
    if (!out) return FP8_ERR_NULL;
    if (!aligned16(out)) return FP8_ERR_ALIGN;
    silu_selftest_kernel<<<256, 256, 0, static_cast<cudaStream_t>(stream)>>>(out);
    return last_launch_status("silu self-test launch");
}

fp8_status fp8_selftest_gemm_schedule(int64_t M, int64_t N, int64_t K, int pairs, int split, int32_t* segs,
                                      int64_t max_segs, int64_t* nsegs) {
    if (!segs || !nsegs) return FP8_ERR_NULL;
    if (M <= 0 || N <= 0 || K <= 0 || M % 128 || N % 128 || K % 128 || pairs <= 0 || max_segs < 0 ||
        M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return FP8_ERR_SHAPE;
    gemm::Params p{};
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.tiles_m = static_cast<int>((M + 2 * gemm::BM - 1) / (2 * gemm::BM));
    p.tiles_n = static_cast<int>((N + gemm::BN - 1) / gemm::BN);
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    p.dp_tiles = split ? dp_tiles_for(tiles, pairs, p.K / gemm::BK) : static_cast<int>(tiles);
    const int npairs = p.dp_tiles < tiles ? pairs : static_cast<int>(tiles < pairs ? tiles : pairs);
    const bool split_launch = p.dp_tiles < tiles;
    const int num_kb = p.K / gemm::BK;
    int64_t n = 0;
    for (int q = 0; q < npairs; ++q) {
        gemm::Seg sg;
        for (int idx = 0; split_launch ? gemm::segment<true>(p, q, npairs, idx, sg)
                                       : gemm::segment<false>(p, q, npairs, idx, sg);
             ++idx) {
            if (n >= max_segs) return FP8_ERR_SHAPE;
            int32_t* row = segs + 5 * n;
            row[0] = q;
            row[1] = sg.tile;
            row[2] = sg.kb0;
            row[3] = sg.kb1;
            // the pairs whose partial sums a finalizing segment adds: the
            // first and one past the last (equal when none)
            int32_t first = 0, last = 0;
            if (sg.kb0 == 0 && sg.kb1 < num_kb) {
                const int64_t tile_end =
                    static_cast<int64_t>(sg.tile + 1) * num_kb - static_cast<int64_t>(p.dp_tiles) * num_kb;
                first = q + 1;
                last = q + 1;
                for (int r = q + 1; r < npairs && gemm::split_range_begin(p, r, npairs) < tile_end; ++r)
                    last = r + 1;
            }
            row[4] = (first << 16) | last;
            ++n;
        }
    }
    *nsegs = n;
    return FP8_OK;
}

fp8_status fp8_selftest_stall_next(int which) {
    if (which < 1 || which > 3) return FP8_ERR_MODE;
    g_stall_next.fetch_or(which);
    return FP8_OK;
}

fp8_status fp8_selftest_wait_timeout(void* stream) {
    wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        g_wait_ns.load(std::memory_order_relaxed), static_cast<unsigned int>(FP8_ERR_TIMEOUT));
    return last_launch_status("wait self-test launch");
}

}  // extern "C"
