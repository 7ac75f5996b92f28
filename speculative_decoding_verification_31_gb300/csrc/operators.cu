// operators.cu -- host side of the verify from probabilities, the residual RMS norm and the
// linear product: argument checks and launches.
//
// The C ABI is declared in include/specverify.h; the kernels are in probs.cuh, norm.cuh and
// linear.cuh.  None of these calls uses a workspace.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "internal.h"
#include "linear.cuh"
#include "norm.cuh"
#include "probs.cuh"
#include "specverify.h"

using namespace specverify;

namespace {

constexpr int kMaxDevices = 64;
constexpr int kMaxGamma = 2048;
constexpr int kProbMaxV = 1 << 24;   // chunk sums of a CTA's share fit its shared memory
constexpr int kNormMaxD = 32768;     // a row is held in the registers of one block
constexpr int kLinMaxSide = 1 << 30, kLinMaxK = 1 << 28;  // tile coordinates stay within 32 bits

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// Arrays of 4-byte words (those that are not NULL).
template <class... P>
bool words_aligned(P... p) {
    return (aligned_to(p, 4) && ...);
}

// Raise a kernel's limits (dynamic shared memory, clusters above eight CTAs) once per device.
struct KernelLimits {
    std::mutex mu;
    bool done[kMaxDevices] = {};
    template <class K>
    int raise(K kernel, uint32_t smem, bool wide_cluster) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ECUDA;
        if (dev < 0 || dev >= kMaxDevices) return SPEC_EINVAL;
        std::lock_guard<std::mutex> lock(mu);
        if (done[dev]) return SPEC_OK;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
            cudaSuccess)
            return SPEC_ECUDA;
        if (wide_cluster &&
            cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return SPEC_ECUDA;
        done[dev] = true;
        return SPEC_OK;
    }
};

// Launch with clusters of `cluster` blocks (1: none), as a programmatic dependent of the kernel before
// it on the stream: its blocks are set up while that one drains, and wait for it (grid_dependency)
// before they touch memory.
template <class K, class... A>
int launch(K kernel, unsigned grid, unsigned threads, size_t smem, int cluster, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ECUDA;
    }
    return SPEC_OK;
}

// ---- the verify from probabilities ----

// One instantiation: its limits, how many clusters of it the device holds at once, its launch.
template <class ET, int kChunk, int kBatch, int kMinBlocks>
struct ProbsKernel {
    static int raise() {
        static KernelLimits limits;
        const uint32_t most = static_cast<uint32_t>((kProbMaxV / kProbChunk) * sizeof(PairSum));
        return limits.raise(verify_probs_kernel<ET, kChunk, kBatch, kMinBlocks>, most, true);
    }
    // (a cluster stays within one GPC: fewer than the SMs' blocks / cluster.  Asked once per device.)
    static long long resident(int cluster, int sm_count) {
        if (cluster == 1) return static_cast<long long>(sm_count) * kMinBlocks;
        static std::mutex mu;
        static int known[kMaxDevices][kProbMaxCluster + 1] = {};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices || raise()) return 0;
        std::lock_guard<std::mutex> lock(mu);
        int& n = known[dev][cluster];  // (what it holds and 1)
        if (!n) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(cluster * sm_count));
            cfg.blockDim = dim3(kProbThreads);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int held = 0;
            if (cudaOccupancyMaxActiveClusters(&held, verify_probs_kernel<ET, kChunk, kBatch, kMinBlocks>, &cfg) !=
                cudaSuccess) {
                cudaGetLastError();
                held = 0;
            }
            n = held + 1;
        }
        return n - 1;
    }
    static int launch(ProbParams& p, int cluster, cudaStream_t s) {
        const int rc = raise();
        if (rc) return rc;
        p.share = ((p.V - 1) / kChunk + cluster) / cluster;
        return ::launch(verify_probs_kernel<ET, kChunk, kBatch, kMinBlocks>,
                        static_cast<unsigned>(p.B) * static_cast<unsigned>(cluster), kProbThreads,
                        static_cast<size_t>(p.share) * sizeof(PairSum), cluster, s, p);
    }
};

template <class ET>
int launch_probs(ProbParams& p, int sm_count, cudaStream_t s) {
    constexpr bool wide = sizeof(typename ET::storage) == 4;
    using Two = ProbsKernel<ET, kProbChunk, wide ? 8 : 4, wide ? 2 : 3>;  // (bf16: three a SM already)
    using Three = ProbsKernel<ET, kProbChunk, 4, 3>;
    using Four = ProbsKernel<ET, kProbChunk, wide ? 4 : 2, 4>;
    // Rows of fp32 that half a chunk for every warp of 16 CTAs covers: one step of half the additions,
    // and no search among a warp's chunks (16 x 32000 6.4 us with whole chunks, 5.8 so; bf16: the same).
    if constexpr (wide) {
        using Half = ProbsKernel<ET, kProbChunk / 2, 4, 2>;
        const int halves = (p.V - 1) / (kProbChunk / 2) + 1;
        int c = 1;
        while (c < kProbMaxCluster && c * kProbWarps < halves) c *= 2;
        if (c * kProbWarps >= halves && p.B <= Half::resident(c, sm_count)) return Half::launch(p, c, s);
    }
    // CTAs per sequence: enough for two a SM over the batch, each with a chunk for every warp, but all
    // clusters at once (32 x 128256 fp32: 16.5 us in clusters of 16, four CTAs a SM, 10.7 in clusters of
    // 8; 16 x 128256: 12.7 with two CTAs a SM, of which 16 such clusters do not fit, 8.8 with three), with as
    // many loads in flight as the registers leave room for: a chunk of fp32 is eight vectors of each
    // row a lane, one of bf16 four.  Three CTAs a SM instead of four, where they hold the grid: 200 x
    // 152064 fp32 39 us (44), bf16 33 (42); where they do not, 256 x 152064 fp32 67 us (50).  bf16 with
    // four a SM: two vectors, 256 x 32000 14.7 us (four, with registers spilled: 16.0); fp32: four (two:
    // 53 of 50 us).
    const int chunks = (p.V - 1) / kProbChunk + 1;
    int cluster = 1;
    while (cluster < kProbMaxCluster && static_cast<long long>(p.B) * cluster < 2LL * sm_count &&
           cluster * kProbWarps < chunks)
        cluster *= 2;
    for (; cluster > 1; cluster /= 2) {
        if (p.B <= Two::resident(cluster, sm_count)) return Two::launch(p, cluster, s);
        if constexpr (wide)
            if (p.B <= Three::resident(cluster, sm_count)) return Three::launch(p, cluster, s);
        if (cluster <= 8 && p.B <= Four::resident(cluster, sm_count)) return Four::launch(p, cluster, s);
    }
    if (p.B <= Two::resident(1, sm_count)) return Two::launch(p, 1, s);
    if constexpr (wide)
        if (p.B <= Three::resident(1, sm_count)) return Three::launch(p, 1, s);
    return Four::launch(p, 1, s);
}

// ---- the norm ----

// kValues a thread; a row's threads are as many as that takes (whole warps), or kLanes of a warp.
template <class ET, bool kFp8, int kLanes, int kValues, int kMaxThreads>
int launch_norm_shape(const NormParams& p, cudaStream_t s) {
    constexpr int NV = kValues / ET::kVec;
    const bool whole = p.d % ET::kVec == 0;
    const int threads = kLanes ? kMaxThreads : std::max(32, ((p.d + kValues - 1) / kValues + 31) / 32 * 32);
    const int per_block = kLanes ? kMaxThreads / kLanes : 1;
    const unsigned grid = static_cast<unsigned>((p.rows - 1) / per_block + 1);
    if constexpr (kLanes == 0 || kLanes == 32) {
        if (!whole) return launch(rms_norm_kernel<ET, kFp8, kLanes, NV, kMaxThreads, false>, grid, threads, 0, 1, s, p);
    }
    return launch(rms_norm_kernel<ET, kFp8, kLanes, NV, kMaxThreads, true>, grid, threads, 0, 1, s, p);
}

template <class ET, bool kFp8>
int launch_norm(const NormParams& p, int sm_count, cudaStream_t s) {
    // Up to one row a SM, eight values a thread: the most loads at once (1 x 4096 bf16: 1.9 us).
    // Beyond, sixteen: few enough registers for 1536 to 2048 threads a SM (3328 x 4096 bf16 with
    // residual to e4m3: 17.7 us; 20.6 with eight, 18.5 with 24 or 32), and a warp per short row.
    if (p.rows <= sm_count && p.d <= 8192) return launch_norm_shape<ET, kFp8, 0, 8, 1024>(p, s);
    if (p.d <= 64 && p.d % ET::kVec == 0) return launch_norm_shape<ET, kFp8, 8, 8, 512>(p, s);
    if (p.d <= 128 && p.d % ET::kVec == 0) return launch_norm_shape<ET, kFp8, 16, 8, 512>(p, s);
    if (p.d <= 256) return launch_norm_shape<ET, kFp8, 32, 8, 512>(p, s);
    if (p.d <= 512) return launch_norm_shape<ET, kFp8, 32, 16, 256>(p, s);
    if (p.d <= 1024) return launch_norm_shape<ET, kFp8, 32, 32, 128>(p, s);
    if (p.d <= 16384) return launch_norm_shape<ET, kFp8, 0, 16, 1024>(p, s);
    return launch_norm_shape<ET, kFp8, 0, 32, 1024>(p, s);
}

int norm_check(const void* x, const void* residual, const void* gain, int rows, int d, float eps, int dtype,
               const void* out, const void* out_residual) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EINVAL;
    if (rows < 0 || d < 1 || d > kNormMaxD) return SPEC_EINVAL;
    if (!std::isfinite(eps) || eps < 0.0f) return SPEC_EINVAL;
    if (rows == 0) return SPEC_OK;
    if (!x || !gain || !out || !aligned16(x) || !aligned16(gain) || !aligned16(out)) return SPEC_EINVAL;
    if (residual ? !out_residual : out_residual != nullptr) return SPEC_EINVAL;
    if (!aligned16(residual) || !aligned16(out_residual)) return SPEC_EINVAL;
    return SPEC_OK;
}

int current_sm_count(int* sm_count) {
    static std::mutex mu;
    static int known[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ECUDA;
    if (dev < 0 || dev >= kMaxDevices) return SPEC_EINVAL;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev] && cudaDeviceGetAttribute(&known[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        known[dev] = 0;
        return SPEC_ECUDA;
    }
    *sm_count = known[dev];
    return SPEC_OK;
}

// ---- the linear product ----

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// Row-major [rows, K] of bf16 or 8-bit codes, box of box_rows rows x 128 bytes of K.
int k_slice_map(CUtensorMap* map, const void* base, int rows, int K, bool fp8, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return SPEC_ECUDA;
    const int es = fp8 ? 1 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kLinBK / es), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                           const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPEC_OK : SPEC_EINVAL;
}

// One CTA per tile of 128 channels x BN tokens, `splits` CTAs where K is split.
template <bool kFp8, int BN>
int launch_linear(const void* x, const void* w, int K, LinearParams& p, int splits, int sm_count, cudaStream_t s) {
    p.n_tiles = (p.N - 1) / kLinBM + 1;
    p.bn = BN;
    p.m_tiles = (p.rows + BN - 1) / BN;
    const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
    if (tiles >= (1LL << 27)) return SPEC_EINVAL;
    CUtensorMap map_w, map_x;
    int rc = k_slice_map(&map_w, w, p.N, K, kFp8, kLinBM);
    if (!rc) rc = k_slice_map(&map_x, x, p.rows, K, kFp8, BN);
    if (rc) return rc;
    if (splits > 1) {
        static KernelLimits limits;
        auto kernel = linear_kernel<kFp8, BN, true>;
        rc = limits.raise(kernel, lin_smem(BN), false);
        if (rc) return rc;
        return launch(kernel, static_cast<unsigned>(tiles * splits), lin_threads(BN), lin_smem(BN), splits, s,
                               map_w, map_x, p);
    }
    static KernelLimits limits;
    auto kernel = linear_kernel<kFp8, BN, false>;
    rc = limits.raise(kernel, lin_smem(BN), false);
    if (rc) return rc;
    return launch(kernel, static_cast<unsigned>(std::min<long long>(tiles, sm_count)), lin_threads(BN),
                           lin_smem(BN), 1, s, map_w, map_x, p);
}

template <bool kFp8>
int launch_linear_pairs(const void* x, const void* w, int K, LinearParams& p, int bn, int sm_count, cudaStream_t s) {
    const int pairs = sm_count / 2;
    p.n_tiles = (p.N - 1) / kPairBM + 1;
    p.bn = bn;
    p.m_tiles = (p.rows + p.bn - 1) / p.bn;
    const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
    if (tiles >= (1LL << 30)) return SPEC_EINVAL;
    CUtensorMap map_w, map_x;
    int rc = k_slice_map(&map_w, w, p.N, K, kFp8, kLinBM);
    if (!rc) rc = k_slice_map(&map_x, x, p.rows, K, kFp8, p.bn / 2);
    if (rc) return rc;
    static KernelLimits limits;
    auto kernel = linear_pair_kernel<kFp8>;
    rc = limits.raise(kernel, kPairSmem, false);
    if (rc) return rc;
    const unsigned grid = 2u * static_cast<unsigned>(std::min<long long>(tiles, pairs));
    return launch(kernel, grid, kPairThreads, kPairSmem, 2, s, map_w, map_x, p);
}

template <bool kFp8>
int launch_linear_few(const void* x, const void* w, int K, LinearParams& p, int sm_count, cudaStream_t s) {
    const uint32_t smem = static_cast<uint32_t>(p.rows) * few_stride(kFp8, K);
    static KernelLimits limits;
    auto kernel = linear_few_kernel<kFp8>;
    const int rc = limits.raise(kernel, kFewMaxSmem, false);
    if (rc) return rc;
    // blocks that the SMs hold at once, each striding over the channels, so the tokens are staged once
    const int groups = (p.N - 1) / kFewChannels + 1;
    const int per_sm = std::max(1, std::min(4, static_cast<int>(220u * 1024u / (smem + 8192u))));
    const int grid = std::min(groups, sm_count * per_sm);
    return launch(kernel, static_cast<unsigned>(grid), kFewThreads, smem, 1, s, static_cast<const uint8_t*>(x),
                  static_cast<const uint8_t*>(w), K, p);
}

// Clusters of `size` CTAs of the split kernel (one CTA a SM) that the current device holds at once:
// fewer than SMs / size, since a cluster stays within one GPC.  Asked once per device.
long long resident_clusters(int size, int sm_count) {
    static std::mutex mu;
    static int known[kMaxDevices][4] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    const int slot = size == 2 ? 0 : size == 4 ? 1 : 2;
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev][slot]) {
        auto kernel = linear_kernel<false, 16, true>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(size * (sm_count / size)));
        cfg.blockDim = dim3(lin_threads(16));
        cfg.dynamicSmemBytes = lin_smem(16);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(size);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lin_smem(16))) !=
                cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        known[dev][slot] = n > 0 ? n : std::max(1, sm_count / (2 * size));
    }
    return known[dev][slot];
}

// How a product is done: spec_linear_kind, tokens of a tile, CTAs that share a tile's K.
struct LinearForm {
    int kind, bn, splits;
};

int linear_kblocks(int K, bool fp8) {
    return static_cast<int>((static_cast<long long>(K) * (fp8 ? 1 : 2) + kLinBK - 1) / kLinBK);
}

// The choice, from the sizes and the device alone.  held(size): clusters of that many CTAs that the device
// holds at once.
template <class Held>
LinearForm choose_linear(bool fp8, int rows, int N, int K, int sm_count, Held held) {
    // Up to four tokens, while the channels' tiles are at most a third of the SMs, or for one token
    // and long rows three quarters (1 token, K = 4096, bf16: N = 1024 4.8 us here and 4.8 there, 4096
    // 7.6 and 9.0, 12288 17.9 and 19.1; K = 1024, e4m3: 4096 3.0 and 4.0, 8192 5.8 and 4.1, 12288 7.6
    // and 4.7; 4 tokens, K = 4096, e4m3: 8192 10.2 and 9.7; five tokens would already read twice the
    // shared memory).
    const int kblocks = linear_kblocks(K, fp8);
    const long long n128 = (N - 1) / kLinBM + 1, n256 = (N - 1) / kPairBM + 1;
    const bool few = n128 * 3 <= sm_count || (rows == 1 && K * (fp8 ? 1LL : 2LL) >= 4096 && n128 * 4 <= sm_count * 3LL);
    if (rows <= kFewMaxRows && few && K < (1 << 20) && static_cast<uint32_t>(rows) * few_stride(fp8, K) <= kFewMaxSmem)
        return LinearForm{SPEC_LINEAR_FEW, rows, 1};
    // The tile, the K split and CTA pairs or not, by an estimate in ns that ranks them; its constants are
    // fitted to shapes of 1 to 4096 tokens x 1024 to 16384 channels x K = 1024 and 4096, bf16.  A CTA takes
    // 118 + bn / 5 ns a K slice (a pair 230 + bn / 7), whole waves of tiles; all of them together at
    // most 18.4 KB a ns from L2; the meeting of a split K 1100 + 25 bn.  It is not the call's time: launch,
    // set-up and the operands' way from HBM are left out (256 tokens, N = K = 4096: 9.2 us here, 17.5
    // measured with a weight that is not in L2; 3328 tokens: 51 and 61).
    // (128 tokens, N = 1024, K = 4096: 7.7 us with 32 columns split four ways, 9.8 with 128 split
    // eight ways; 512 tokens, N = K = 4096: 17.2 us with 128 tiles of one CTA, 19.3 with 64 pairs.)
    auto ceil_div = [](long long a, long long b) { return (a + b - 1) / b; };
    long long best = -1;
    LinearForm form{SPEC_LINEAR_TILES, 16, 1};
    auto offer = [&](long long time, LinearForm f) {
        if (best >= 0 && time >= best) return;
        best = time;
        form = f;
    };
    for (int b = 16; b <= 128; b *= 2) {
        const long long tiles = ceil_div(rows, b) * n128;
        const long long traffic = tiles * kblocks * (16 + b / 8) * 1000 / 18400;
        for (int k = 1; k <= 8; k *= 2) {
            if (k > 1 && (kblocks < 4 * k || tiles > held(k))) break;
            const long long waves = ceil_div(tiles * k, sm_count), turns = ceil_div(kblocks, 2 * k);
            offer(std::max(waves * turns * 2 * (118 + b / 5), traffic) + (k > 1 ? 1100 + 25 * b : 0),
                  LinearForm{SPEC_LINEAR_TILES, b, k});
        }
    }
    if (rows > 64)
        for (int b = 256; b >= 64; b -= 32) {
            const long long tiles = ceil_div(rows, b) * n256;
            const long long traffic = 2 * tiles * kblocks * (16 + b / 16) * 1000 / 18400;
            offer(std::max(ceil_div(tiles, sm_count / 2) * kblocks * (230 + b / 7), traffic),
                  LinearForm{SPEC_LINEAR_PAIRS, b, 1});
        }
    return form;
}

template <bool kFp8>
int dispatch_linear(const void* x, const void* w, int K, LinearParams& p, int sm_count, cudaStream_t s) {
    const LinearForm f = choose_linear(kFp8, p.rows, p.N, K, sm_count, [&](int size) { return resident_clusters(size, sm_count); });
    if (f.kind == SPEC_LINEAR_FEW) return launch_linear_few<kFp8>(x, w, K, p, sm_count, s);
    if (f.kind == SPEC_LINEAR_PAIRS) return launch_linear_pairs<kFp8>(x, w, K, p, f.bn, sm_count, s);
    if (f.bn == 16) return launch_linear<kFp8, 16>(x, w, K, p, f.splits, sm_count, s);
    if (f.bn == 32) return launch_linear<kFp8, 32>(x, w, K, p, f.splits, sm_count, s);
    if (f.bn == 64) return launch_linear<kFp8, 64>(x, w, K, p, f.splits, sm_count, s);
    return launch_linear<kFp8, 128>(x, w, K, p, f.splits, sm_count, s);
}

bool linear_sizes_ok(int rows, int N, int K, int in_dtype) {
    if (in_dtype != SPEC_BF16 && in_dtype != SPEC_E4M3) return false;
    return rows >= 0 && rows <= kLinMaxSide && N >= 1 && N <= kLinMaxSide && K >= 1 && K <= kLinMaxK &&
           K % (in_dtype == SPEC_E4M3 ? 16 : 8) == 0 && static_cast<long long>(rows) * N < (1LL << 40);
}

}  // namespace

extern "C" {

int spec_verify_probs(const void* target_probs, const void* draft_probs, const int32_t* draft_tokens,
                      const float* uniforms, const int32_t* draft_lens, int B, int gamma, int V, int dtype,
                      int32_t* out_tokens, int32_t* out_n_accepted, int32_t* d_status, void* stream) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EINVAL;
    if (B < 0 || gamma < 0 || gamma > kMaxGamma || V < 1 || V > kProbMaxV) return SPEC_EINVAL;
    if (static_cast<long long>(B) * (gamma + 1) * static_cast<long long>(V) >= (1LL << 40) || B > (1 << 26))
        return SPEC_EINVAL;
    if (B == 0) return SPEC_OK;
    if (!target_probs || !uniforms || !out_tokens || !out_n_accepted) return SPEC_EINVAL;
    if (gamma > 0 && !draft_tokens) return SPEC_EINVAL;
    if (!aligned16(target_probs) || !aligned16(draft_probs)) return SPEC_EINVAL;
    if (!words_aligned(draft_tokens, uniforms, draft_lens, out_tokens, out_n_accepted, d_status)) return SPEC_EINVAL;
    int32_t* status = nullptr;
    int sm_count = 0;
    int rc = d_status ? current_sm_count(&sm_count) : library_device(&status, &sm_count);
    if (rc) return rc;
    ProbParams p{};
    p.target = target_probs;
    p.draft = gamma > 0 ? draft_probs : nullptr;
    p.tokens = draft_tokens;
    p.uniforms = uniforms;
    p.lens = draft_lens;
    p.B = B;
    p.gamma = gamma;
    p.V = V;
    p.out_tokens = out_tokens;
    p.out_n = out_n_accepted;
    p.status = d_status ? d_status : status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_probs<F32Elem>(p, sm_count, s) : launch_probs<Bf16Elem>(p, sm_count, s);
}

int spec_rms_norm(const void* x, const void* residual, const void* gain, int rows, int d, float eps, int dtype,
                  void* out, void* out_residual, void* stream) {
    int rc = norm_check(x, residual, gain, rows, d, eps, dtype, out, out_residual);
    if (rc || rows == 0) return rc;
    int sm_count = 0;
    rc = current_sm_count(&sm_count);
    if (rc) return rc;
    const NormParams p{x, residual, gain, out, out_residual, nullptr, rows, d, eps};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_norm<F32Elem, false>(p, sm_count, s) : launch_norm<Bf16Elem, false>(p, sm_count, s);
}

int spec_rms_norm_fp8(const void* x, const void* residual, const void* gain, int rows, int d, float eps, int dtype,
                      void* out_codes, float* out_scale, void* out_residual, void* stream) {
    int rc = norm_check(x, residual, gain, rows, d, eps, dtype, out_codes, out_residual);
    if (rc || rows == 0) return rc;
    if (!out_scale || !words_aligned(out_scale)) return SPEC_EINVAL;
    int sm_count = 0;
    rc = current_sm_count(&sm_count);
    if (rc) return rc;
    const NormParams p{x, residual, gain, out_codes, out_residual, out_scale, rows, d, eps};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_norm<F32Elem, true>(p, sm_count, s) : launch_norm<Bf16Elem, true>(p, sm_count, s);
}

int spec_linear(const void* x, const void* weight, const void* bias, const void* residual, const float* x_scale,
                const float* w_scale, int rows, int N, int K, int in_dtype, int out_dtype, int activation, void* out,
                int32_t* d_status, void* stream) {
    if (!linear_sizes_ok(rows, N, K, in_dtype)) return SPEC_EINVAL;
    if (out_dtype != SPEC_F32 && out_dtype != SPEC_BF16) return SPEC_EINVAL;
    if (activation < SPEC_ACT_NONE || activation > SPEC_ACT_SILU) return SPEC_EINVAL;
    const bool fp8 = in_dtype == SPEC_E4M3;
    if (rows == 0) return SPEC_OK;
    if (!x || !weight || !out || !aligned16(x) || !aligned16(weight)) return SPEC_EINVAL;
    if (fp8 ? (!x_scale || !w_scale) : (x_scale || w_scale)) return SPEC_EINVAL;
    if (!words_aligned(x_scale, w_scale, d_status)) return SPEC_EINVAL;
    const size_t os = out_dtype == SPEC_F32 ? 4 : 2;
    if (!aligned_to(out, os) || !aligned_to(bias, os) || !aligned_to(residual, os)) return SPEC_EINVAL;
    int32_t* status = nullptr;
    int sm_count = 0;
    int rc = d_status ? current_sm_count(&sm_count) : library_device(&status, &sm_count);
    if (rc) return rc;
    LinearParams p{};
    p.rows = rows;
    p.N = N;
    p.kblocks = linear_kblocks(K, fp8);
    p.group = 16;
    p.act = activation;
    p.out_f32 = out_dtype == SPEC_F32;
    p.vec = N % 4 == 0 && aligned_to(out, 4 * os) && aligned_to(residual, 4 * os);
    p.x_scale = x_scale;
    p.w_scale = w_scale;
    p.bias = bias;
    p.residual = residual;
    p.out = out;
    p.status = d_status ? d_status : status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return fp8 ? dispatch_linear<true>(x, weight, K, p, sm_count, s) : dispatch_linear<false>(x, weight, K, p, sm_count, s);
}

int spec_linear_form(int rows, int N, int K, int in_dtype, int sm_count, int32_t* clusters, int32_t* out_form) {
    if (!linear_sizes_ok(rows, N, K, in_dtype) || rows < 1 || sm_count < 0 || sm_count == 1 || !out_form ||
        (sm_count > 0 && !clusters))
        return SPEC_EINVAL;
    int32_t held[3];
    if (sm_count == 0) {
        const int rc = current_sm_count(&sm_count);
        if (rc) return rc;
        for (int i = 0; i < 3; ++i) {
            held[i] = static_cast<int32_t>(resident_clusters(2 << i, sm_count));
            if (clusters) clusters[i] = held[i];
        }
    } else {
        for (int i = 0; i < 3; ++i) held[i] = clusters[i];
    }
    const LinearForm f = choose_linear(in_dtype == SPEC_E4M3, rows, N, K, sm_count,
                                       [&](int size) { return static_cast<long long>(held[size == 2 ? 0 : size == 4 ? 1 : 2]); });
    out_form[0] = f.kind;
    out_form[1] = f.bn;
    out_form[2] = f.splits;
    return SPEC_OK;
}

}  // extern "C"
