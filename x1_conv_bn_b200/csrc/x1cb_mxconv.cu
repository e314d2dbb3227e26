// The MX4 1x1 convolution on the tensor cores: out[M, N] = act(x[M, K] w[N, K]^T
// + bias + r), tcgen05.mma kind::mxf4 with one e8m0 scale per 32 elements.
//
// Persistent CTAs, one per SM; a tile is 128 rows (pixels) x kBN channels.
//   warp 0      loads K steps of 256: x and w rows of 128 bytes (TMA, 128-byte
//               swizzle) and their scale tiles (512 bytes per 128 rows x 128 K,
//               stored in the order TMEM wants them) into a ring of stages;
//   warp 1      copies the scales to TMEM (tcgen05.cp) and issues the MMAs, four
//               K = 64 steps a stage.  The scale columns belong to the stage, so
//               they are free exactly when the stage is;
//   warps 4-11  epilogue: two warps per TMEM lane quarter, half the channels
//               each, from two accumulators in turn, so that it runs beside the
//               next tile's MMAs.
// Every wait is bounded: on a timeout the CTA raises an abort flag, records a
// status bit, lets its copies and MMAs land and leaves.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "x1cb_float.cuh"
#include "x1cb_internal.h"
#include "x1cb_plan.h"
#include "x1cb_ptx.cuh"

namespace x1cb {
namespace {

constexpr int kEpiWarps = 8;
constexpr int kMxThreads = 32 * (4 + kEpiWarps);
constexpr int kStageK = 256;             // elements: 128 bytes of codes a row
constexpr int kRowsBytes = 128 * 128;    // codes of 128 rows in a stage
constexpr int kSfBytes = 1024;           // scales of 128 rows in a stage
constexpr int kTmem = 512;
constexpr uint64_t kDrainNs = 200000000ull;

struct MxArgs {
    const uint8_t *xs, *ws;
    const float *bias;
    const void *r;
    void *out;
    unsigned int *status;
    uint64_t wait_ns;
    long long M;
    int K, N, act, inject;
    int stages, k_steps, kt;      // ring depth; K steps of 256; scale tiles per row block
    int m_tiles, n_tiles;
};

template <int BN> struct Shape {
    static constexpr int kW = BN * 128;                       // weight codes of a stage
    static constexpr int kWsf = (BN + 127) / 128 * kSfBytes;  // their scales
    static constexpr int kStage = kRowsBytes + kW + kSfBytes + kWsf;
    static constexpr int kSfCols = 8 + (BN + 127) / 128 * 8;  // TMEM columns a stage's scales take
};

// Tail of the dynamic shared memory behind the ring.
constexpr int kPatch = 32 * 33 * 4;  // an epilogue warp's transposing patch
struct Tail {
    unsigned long long bars[2 * 16 + 2 * 2 + 2];
    uint32_t tmem;
    int abort_flag;
};

template <typename T, int BN>
__global__ void __launch_bounds__(kMxThreads, 1)
    conv_mx4_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                    MxArgs a)
{
    using S = Shape<BN>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    float *patches = reinterpret_cast<float *>(smem + a.stages * S::kStage);
    Tail *tail = reinterpret_cast<Tail *>(smem + a.stages * S::kStage + kEpiWarps * kPatch);
    const uint32_t bars = smem_u32(tail->bars);
    const auto full = [&](int s) { return bars + 8u * s; };
    const auto empty = [&](int s) { return bars + 8u * (a.stages + s); };
    const auto acc_full = [&](int b) { return bars + 8u * (2 * a.stages + b); };
    const auto acc_empty = [&](int b) { return bars + 8u * (2 * a.stages + 2 + b); };
    const uint32_t mma_done = bars + 8u * (2 * a.stages + 4), never = mma_done + 8u;
    volatile int *abort_flag = &tail->abort_flag;
    const WaitCtl ctl{abort_flag, a.status, a.inject == 1 ? 4 * a.wait_ns : a.wait_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = a.m_tiles * a.n_tiles;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), kEpiWarps);
        }
        mbar_init(mma_done, 1);
        mbar_init(never, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem), kTmem);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tail->tmem;
    griddep_wait();  // from here on global memory is touched

    if (warp == 0) {
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const int mt = t / a.n_tiles, nt = t - mt * a.n_tiles;
                const int n0 = nt * BN;
                const uint8_t *xs = a.xs + static_cast<size_t>(mt) * a.kt * 512;
                for (int k = 0; k < a.k_steps; ++k) {
                    if (!mbar_wait(empty(s), ph ^ 1u, ctl, kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = sbase + s * S::kStage;
                    const uint32_t sfb = min(2, a.kt - 2 * k) * 512u;  // one tile at an odd end
                    int wblk = 0;  // blocks of 128 weight rows that exist
#pragma unroll
                    for (int j = 0; j < (BN + 127) / 128; ++j)
                        wblk += n0 + 128 * j < a.N;
                    mbar_arrive_expect_tx(full(s), kRowsBytes + S::kW + sfb * (1 + wblk));
                    tma_load_2d(st, &tmX, full(s), k * 128, mt * 128);
                    tma_load_2d(st + kRowsBytes, &tmW, full(s), k * 128, n0);
                    bulk_load(st + kRowsBytes + S::kW, xs + k * 1024, sfb, full(s));
                    for (int j = 0; j < wblk; ++j)
                        bulk_load(st + kRowsBytes + S::kW + kSfBytes * (1 + j),
                                  a.ws + (static_cast<size_t>(n0 / 128 + j) * a.kt + 2 * k) * 512,
                                  sfb, full(s));
                    ++issued;
                    if (++s == a.stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            // Let every copy still in flight land (after a failed wait elsewhere
            // nobody else waited for the last ones).
            for (int i = max(0, issued - a.stages); i < issued; ++i)
                if (!mbar_drain(full(i % a.stages), (i / a.stages) & 1, kDrainNs))
                    atomicOr(a.status, kDevDrainFailed);
        }
        __syncwarp();
    } else if (warp == 1) {
        bool ok = true;
        if (a.inject == 1) {
            const WaitCtl planted{abort_flag, a.status, a.wait_ns};
            ok = __all_sync(0xffffffffu, mbar_wait(never, 0, planted, kDevTimeoutMma));
        }
        int s = 0, buf = 0;
        uint32_t ph = 0, aph = 0;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            if (!__all_sync(0xffffffffu, mbar_wait(acc_empty(buf), aph ^ 1u, ctl, kDevTimeoutMma))) {
                ok = false;
                break;
            }
            const uint32_t d = tmem + buf * BN;
            // BN = 64: the tile's scales are the lower or upper half of a 128-row block
            const uint32_t half = BN == 64 ? ((t % a.n_tiles) & 1) * 2u : 0u;
            for (int k = 0; k < a.k_steps; ++k) {
                if (!__all_sync(0xffffffffu, mbar_wait(full(s), ph, ctl, kDevTimeoutMma))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = sbase + s * S::kStage;
                const uint32_t sfa = tmem + 2 * BN + s * S::kSfCols, sfw = sfa + 8;
                const int left = min(4, (a.K - k * kStageK + 63) / 64);
                for (int j = 0; j < (left + 1) / 2; ++j) {
                    tmem_cp_scales(sfa + 4 * j, smem_desc_scales(st + kRowsBytes + S::kW + 512 * j));
#pragma unroll
                    for (int i = 0; i < (BN + 127) / 128; ++i)
                        tmem_cp_scales(sfw + (BN + 127) / 128 * 4 * j + 4 * i,
                                       smem_desc_scales(st + kRowsBytes + S::kW +
                                                        kSfBytes * (1 + i) + 512 * j));
                }
                const uint64_t ad = smem_desc_sw128(st), bd = smem_desc_sw128(st + kRowsBytes);
                for (int j = 0; j < left; ++j)
                    mma_mx4(d, ad + 2 * j, bd + 2 * j, idesc_mx4(128, BN, (j & 1) * 2),
                            sfa + 4 * (j >> 1), sfw + (BN + 127) / 128 * 4 * (j >> 1) + half,
                            k > 0 || j > 0);
                mma_commit(empty(s));
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok)
                break;
            mma_commit(acc_full(buf));
            buf ^= 1;
            aph ^= buf == 0;
        }
        // No MMA may still read shared memory or write TMEM behind this point.
        mma_commit(mma_done);
        if (lane == 0 && !mbar_drain(mma_done, 0, kDrainNs))
            atomicOr(a.status, kDevDrainFailed);
        __syncwarp();
    } else if (warp >= 4) {
        const int e = warp - 4, quarter = e & 3, side = e >> 2;
        float *patch = patches + e * (kPatch / 4);
        int buf = 0;
        uint32_t aph = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            const int mt = t / a.n_tiles, nt = t - mt * a.n_tiles;
            if (!__all_sync(0xffffffffu, mbar_wait(acc_full(buf), aph, ctl, kDevTimeoutEpilogue)))
                break;
            tc_fence_after();
            const long long row0 = static_cast<long long>(mt) * 128 + quarter * 32;
            const int rows = static_cast<int>(min(32ll, a.M - row0));
            for (int c0 = side * (BN / 2); c0 < (side + 1) * (BN / 2); c0 += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32_sync(tmem + buf * BN + c0 +
                                            (static_cast<uint32_t>(quarter * 32) << 16),
                                        v);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    patch[lane * 33 + i] = __uint_as_float(v[i]);
                __syncwarp();
                const int o = nt * BN + c0 + lane;
                if (o < a.N) {
                    const float b = a.bias ? a.bias[o] : 0.f;
                    size_t at = static_cast<size_t>(row0) * a.N + o;
                    for (int i = 0; i < rows; ++i, at += a.N) {
                        float y = patch[i * 33 + lane] + b;
                        if (a.r)
                            y += to_f(static_cast<const T *>(a.r)[at]);
                        static_cast<T *>(a.out)[at] = from_f<T>(activate(y, a.act));
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            if (lane == 0)
                mbar_arrive(acc_empty(buf));
            buf ^= 1;
            aph ^= buf == 0;
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

template <typename T, int BN> int run(const Mx4Call &c, int sms, cudaStream_t s)
{
    using S = Shape<BN>;
    MxArgs a{};
    unsigned int *forms = nullptr;
    if (int e = device_words(&a.status, &forms))
        return e;
    a.xs = c.xs;
    a.ws = c.ws;
    a.bias = c.bias;
    a.r = c.r;
    a.out = c.out;
    a.wait_ns = wait_limit_ns();
    a.M = c.M;
    a.K = c.K;
    a.N = c.N;
    a.act = c.act;
    a.inject = debug_inject();
    a.k_steps = (c.K + kStageK - 1) / kStageK;
    a.kt = (c.K + 127) / 128;
    a.m_tiles = static_cast<int>((c.M + 127) / 128);
    a.n_tiles = (c.N + BN - 1) / BN;
    const int fixed = 1024 + kEpiWarps * kPatch + static_cast<int>(sizeof(Tail));
    a.stages = std::min({(232448 - fixed) / S::kStage, (kTmem - 2 * BN) / S::kSfCols, 8});
    const int smem = fixed + a.stages * S::kStage;
    CUtensorMap tmX, tmW;
    const uint64_t str[1] = {static_cast<uint64_t>(c.K) / 2};
    const uint64_t dx[2] = {str[0], static_cast<uint64_t>(c.M)};
    const uint64_t dw[2] = {str[0], static_cast<uint64_t>(c.N)};
    const uint32_t bx[2] = {128, 128}, bw[2] = {128, BN};
    if (int e = encode_map(&tmX, c.x, 2, dx, str, bx, CU_TENSOR_MAP_SWIZZLE_128B))
        return e;
    if (int e = encode_map(&tmW, c.w, 2, dw, str, bw, CU_TENSOR_MAP_SWIZZLE_128B))
        return e;
    if (cudaFuncSetAttribute(conv_mx4_kernel<T, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             232448) != cudaSuccess)
        return X1CB_ERR_CUDA;
    const long long tiles = static_cast<long long>(a.m_tiles) * a.n_tiles;
    if (tiles > 0x7fffffffLL)
        return X1CB_ERR_SHAPE;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(tiles, sms)), 1, 1);
    cfg.blockDim = dim3(kMxThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, conv_mx4_kernel<T, BN>, tmX, tmW, a) == cudaSuccess
               ? X1CB_OK
               : X1CB_ERR_CUDA;
}

template <typename T> int run_bn(const Mx4Call &c, int sms, cudaStream_t s)
{
    return c.N <= 64 ? run<T, 64>(c, sms, s) : run<T, 128>(c, sms, s);
}

}  // namespace

int launch_conv_mx4_tiles(const Mx4Call &c, cudaStream_t s)
{
    int sms = 0;
    if (int e = current_sms(sms))
        return e;
    return c.dtype == X1CB_F32    ? run_bn<float>(c, sms, s)
           : c.dtype == X1CB_BF16 ? run_bn<__nv_bfloat16>(c, sms, s)
                                  : run_bn<__half>(c, sms, s);
}

}  // namespace x1cb
