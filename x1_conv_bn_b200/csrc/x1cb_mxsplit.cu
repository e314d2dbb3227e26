// The MX4 1x1 convolution for few rows or few tiles: the operands change places
// (the weights' 128 channels are the MMA's M, the pixels its N of 16, 32 or 64)
// and K is split over the CTAs of a cluster, so that a handful of rows still
// reads the weights with the whole chip.
//
// A CTA computes 128 channels x NB pixels over its share of K: warp 0 loads the
// codes and scales (TMA ring), warp 1 issues the MMAs, warps 2-5 take the sums
// from TMEM (a lane per channel).  The CTAs of the cluster send each other their
// partial sums through distributed shared memory -- CTA r gets every CTA's sums of
// its share of the pixels -- add them in rank order, and finish: bias, shortcut,
// activation, 32 neighbouring channels to a store.  Bound by latency: a launch,
// one trip to memory for all of the weights, one to the neighbours.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "x1cb_float.cuh"
#include "x1cb_internal.h"
#include "x1cb_plan.h"
#include "x1cb_ptx.cuh"

namespace x1cb {
namespace {

constexpr int kSplitThreads = 192;
constexpr int kRowsBytes = 128 * 128;  // codes of 128 channels, K = 256
constexpr int kSfBytes = 1024;         // scales of 128 rows, K = 256
constexpr int kCols = 128;             // TMEM columns
constexpr uint64_t kDrainNs = 200000000ull;

struct SplitArgs {
    const float *bias;
    const void *r;
    void *out;
    unsigned int *status;
    uint64_t wait_ns;
    int M, N, K, act, inject;
    int k_steps, per;  // K steps of 256 in all, and per CTA
    int ch_tiles;
};

template <int NB> struct SplitShape {
    static constexpr int kX = NB * 128;
    static constexpr int kStage = kRowsBytes + kX + 2 * kSfBytes;
    static constexpr int kAcc = NB < 32 ? 32 : NB;
    // (more than half of an SM's shared memory in any case: no two kernels that
    // hold TMEM share an SM, so none waits there for columns while it keeps a cluster)
    static constexpr int kStages = NB == 64 ? 4 : NB == 32 ? 5 : 6;
    static constexpr int kPart = NB * 128 * 4;  // partial sums received
    static_assert(kAcc + kStages * 16 <= kCols, "TMEM columns");
};
struct SplitTail {
    unsigned long long full[6], empty[6], acc, never;
    uint32_t tmem;
    int abort_flag;
};

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int NB>
__global__ void __launch_bounds__(kSplitThreads)
    conv_mx4_split_kernel(const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmXs,
                          const __grid_constant__ CUtensorMap tmWs, const SplitArgs a)
{
    using S = SplitShape<NB>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(smem);
    float *part = reinterpret_cast<float *>(smem + S::kStages * S::kStage);
    SplitTail *tail =
        reinterpret_cast<SplitTail *>(smem + S::kStages * S::kStage + S::kPart);
    const auto full = [&](int s) { return smem_u32(&tail->full[s]); };
    const auto empty = [&](int s) { return smem_u32(&tail->empty[s]); };
    const uint32_t acc_full = smem_u32(&tail->acc);
    const WaitCtl ctl{&tail->abort_flag, a.status, a.inject == 1 ? 4 * a.wait_ns : a.wait_ns};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t ctas, unit;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(unit));
    const int rank = static_cast<int>(cluster_ctarank());
    const int mt = static_cast<int>(unit) / a.ch_tiles, ct = static_cast<int>(unit) - mt * a.ch_tiles;
    const int m0 = mt * NB, ch0 = ct * 128;
    const int k0 = rank * a.per, steps = max(0, min(a.per, a.k_steps - k0));

    if (threadIdx.x == 0) {
        tail->abort_flag = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(smem_u32(&tail->never), 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmXs);
        tma_prefetch_desc(&tmWs);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tail->tmem), kCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (ctas > 1)  // every CTA of the cluster runs before any writes to another
        cluster_arrive();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tail->tmem, 0);
    griddep_wait();

    bool met = false;  // waited for the others
    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (; issued < steps; ++issued) {
                const int s = issued % S::kStages, k = k0 + issued;
                if (!mbar_wait(empty(s), ((issued / S::kStages) & 1) ^ 1, ctl, kDevTimeoutProducer))
                    break;
                const uint32_t st = ring + s * S::kStage, sf = st + kRowsBytes + S::kX;
                mbar_arrive_expect_tx(full(s), S::kStage);
                tma_load_2d(st, &tmW, full(s), k * 128, ch0);
                tma_load_3d(sf, &tmWs, full(s), 0, 2 * k, ct);
                tma_load_2d(st + kRowsBytes, &tmX, full(s), k * 128, m0);
                tma_load_3d(sf + kSfBytes, &tmXs, full(s), 0, 2 * k, m0 / 128);
            }
            for (int i = max(0, issued - S::kStages); i < issued; ++i)
                if (!mbar_drain(full(i % S::kStages), (i / S::kStages) & 1, kDrainNs))
                    atomicOr(a.status, kDevDrainFailed);
        }
        __syncwarp();
    } else if (warp == 1) {
        bool ok = true;
        if (a.inject == 1) {
            const WaitCtl planted{&tail->abort_flag, a.status, a.wait_ns};
            ok = __all_sync(0xffffffffu,
                            mbar_wait(smem_u32(&tail->never), 0, planted, kDevTimeoutMma));
        }
        // NB = 64: these pixels' scales are the lower or upper half of a 128-row block
        const uint32_t half = NB == 64 ? ((m0 >> 6) & 1) * 2u : 0u;
        for (int i = 0; ok && i < steps; ++i) {
            const int s = i % S::kStages;
            ok = __all_sync(0xffffffffu,
                            mbar_wait(full(s), (i / S::kStages) & 1, ctl, kDevTimeoutMma));
            if (!ok)
                break;
            tc_fence_after();
            const uint32_t st = ring + s * S::kStage, sf = st + kRowsBytes + S::kX;
            const uint32_t sfa = tmem + S::kAcc + s * 16, sfb = sfa + 8;
            const uint64_t ad = smem_desc_sw128(st), bd = smem_desc_sw128(st + kRowsBytes);
            const int left = (a.K - (k0 + i) * 256 + 63) / 64;
            if (left >= 4) {
                mma_mx4_stage<false, 1, 4>(tmem, ad, bd, idesc_mx4(128, NB, 0),
                                           idesc_mx4(128, NB, 2), sfa, sfb, half,
                                           smem_desc_scales(sf), i > 0);
            } else {
                for (int j = 0; j < (left + 1) / 2; ++j) {
                    tmem_cp_scales<false>(sfa + 4 * j, smem_desc_scales(sf + 512 * j));
                    tmem_cp_scales<false>(sfb + 4 * j, smem_desc_scales(sf + kSfBytes + 512 * j));
                }
                for (int j = 0; j < left; ++j)
                    mma_mx4<false>(tmem, ad + 2 * j, bd + 2 * j, idesc_mx4(128, NB, (j & 1) * 2),
                                   sfa + 4 * (j >> 1), sfb + 4 * (j >> 1) + half, i > 0 || j > 0);
            }
            mma_commit(empty(s));
        }
        mma_commit(acc_full);
        // nothing may still read shared memory or write TMEM behind this point
        if (lane == 0 && !mbar_drain(acc_full, 0, kDrainNs))
            atomicOr(a.status, kDevDrainFailed);
        __syncwarp();
    } else {
        const int quarter = warp & 3, ch = ch0 + quarter * 32 + lane;
        const bool ok = __all_sync(0xffffffffu, mbar_wait(acc_full, 0, ctl, kDevTimeoutEpilogue));
        tc_fence_after();
        const int cols = min(NB, a.M - m0);          // pixels of this tile
        const int share = (cols + ctas - 1) / ctas;  // and of each CTA
        const float bias = a.bias && ch < a.N ? __ldg(a.bias + ch) : 0.f;
        if (ctas > 1) {
            cluster_wait();
            met = true;
        }
        const T *r = static_cast<const T *>(a.r);
        T *out = static_cast<T *>(a.out);
        int to = 0, off = 0;  // receiving CTA and place in its share, of column c
        uint32_t dst = 0;
        if (ctas > 1)
            dst = mapa_shared(smem_u32(part + (rank * share * 128 + quarter * 32 + lane)), 0);
#pragma unroll 1
        for (int c0 = 0; c0 < cols; c0 += 16) {
            uint32_t v[16];
            if (steps > 0 && ok) {
                tmem_ld_32x32b_x16_sync(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c0, v);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = 0u;
            }
            if (ctas == 1) {
                size_t at = static_cast<size_t>(m0 + c0) * a.N + ch;
                T rv[16];
                if (r && ch < a.N) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < cols)
                            rv[i] = r[at + static_cast<size_t>(i) * a.N];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i, at += a.N) {
                    if (c0 + i < cols && ch < a.N) {
                        float y = __uint_as_float(v[i]) + bias;
                        if (r)
                            y += to_f(rv[i]);
                        out[at] = from_f<T>(activate(y, a.act));
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (c0 + i < cols) {
                        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(dst + off * 512),
                                     "r"(v[i])
                                     : "memory");
                        if (++off == share) {
                            off = 0;
                            ++to;
                            dst = mapa_shared(
                                smem_u32(part + (rank * share * 128 + quarter * 32 + lane)),
                                min(to, static_cast<int>(ctas) - 1));
                        }
                    }
                }
            }
        }
        if (ctas > 1) {
            const int first = rank * share, mine = max(0, min(share, cols - first));
            // the shortcut of this CTA's pixels is on its way during the exchange
            T rv[8];
            size_t at = static_cast<size_t>(m0 + first) * a.N + ch;
            if (r && ch < a.N) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < mine)
                        rv[c] = r[at + static_cast<size_t>(c) * a.N];
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();
            const float *p = part + quarter * 32 + lane;
            for (int c0 = 0; c0 < mine; c0 += 8) {
                // (a share above eight: two CTAs and more than 16 pixels, or four and 32)
                if (c0 > 0 && r && ch < a.N) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (c0 + c < mine)
                            rv[c] = r[at + static_cast<size_t>(c) * a.N];
                }
#pragma unroll
                for (int c = 0; c < 8; ++c, at += a.N) {
                    if (c0 + c < mine && ch < a.N) {
                        float t[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            t[q] = q < static_cast<int>(ctas) ? p[(q * share + c0 + c) * 128] : 0.f;
                        float y = t[0];
#pragma unroll
                        for (int q = 1; q < 8; ++q)
                            y += t[q];
                        y += bias;
                        if (r)
                            y += to_f(rv[c]);
                        out[at] = from_f<T>(activate(y, a.act));
                    }
                }
            }
        }
    }
    __syncwarp();
    if (ctas > 1 && !met) {  // the other warps keep step with the two barriers
        cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// What a launch of the kernel needs to know once per device: its shared memory,
// opted in to, and how many clusters of 8 and of 4 CTAs the chip holds at once (a
// cluster lies within a GPC, so 8 x 16 CTAs are more than 148 SMs hold).
struct Fit {
    int of8, of4;
};
template <typename T, int NB> struct Kernel {
    using S = SplitShape<NB>;
    static constexpr int kSmem =
        1024 + S::kStages * S::kStage + S::kPart + static_cast<int>(sizeof(SplitTail));
    static_assert(kSmem >= kSmemAlone, "two of these kernels would share an SM");

    static int prepare(Fit &fit)
    {
        static std::mutex mu;
        static Fit known[64];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
            return X1CB_ERR_CUDA;
        std::lock_guard<std::mutex> lk(mu);
        if (!known[dev].of4) {
            const auto kern = conv_mx4_split_kernel<T, NB>;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) !=
                cudaSuccess)
                return X1CB_ERR_CUDA;
            Fit f{};
            for (int split = 8; split >= 4; split /= 2) {
                cudaLaunchConfig_t cfg;
                cudaLaunchAttribute attr[2];
                configure(cfg, attr, 148 / split, split, nullptr);
                if (cudaOccupancyMaxActiveClusters(split == 8 ? &f.of8 : &f.of4, kern, &cfg) !=
                    cudaSuccess)
                    return X1CB_ERR_CUDA;
            }
            if (!f.of4)
                return X1CB_ERR_CUDA;
            known[dev] = f;
        }
        fit = known[dev];
        return X1CB_OK;
    }
    static void configure(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, long long units, int split,
                          cudaStream_t s)
    {
        std::memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3(static_cast<unsigned>(units * split), 1, 1);
        cfg.blockDim = dim3(kSplitThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = split;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = split > 1 ? 2 : 1;
    }
};

long long units_of(const Mx4Call &c, int NB)
{
    return (c.M + NB - 1) / NB * ((c.N + 127) / 128);
}

// CTAs to split K over.  64 x 4096 x 1792: 10.6 us with one, 10.3 with two, 7.9 with
// four, 6.9 with eight; 64 x 4096 x 2048, whose 16 clusters of eight do not run at
// once, 13.0 with eight, 7.9 with four; 64 x 1024 x 512 7.2, 8.6, 7.0, 6.5.  Where
// clusters of four do not run at once either, one against two: 2 x 4096 x 8192 7.7 and
// 6.5, 16 x 4096 x 4800 7.9 and 6.8, 64 x 4096 x 8192 10.6 and 10.6, 64 x 8192 x 9472 15.5
// and 13.0, 64 x 16384 x 8192 24.6 and 18.2.
int split_for(long long units, int k_steps, const Fit &fit)
{
    return k_steps >= 4 && units <= fit.of8   ? 8
           : k_steps >= 4 && units <= fit.of4 ? 4
           : k_steps >= 16 && units <= 74     ? 2
                                              : 1;
}

template <typename T, int NB> int run(const Mx4Call &c, cudaStream_t s)
{
    using Ke = Kernel<T, NB>;
    SplitArgs a{};
    unsigned int *forms = nullptr;
    if (int e = device_words(&a.status, &forms))
        return e;
    Fit fit;
    if (int e = Ke::prepare(fit))
        return e;
    a.bias = c.bias;
    a.r = c.r;
    a.out = c.out;
    a.wait_ns = wait_limit_ns();
    a.M = static_cast<int>(c.M);
    a.N = c.N;
    a.K = c.K;
    a.act = c.act;
    a.inject = debug_inject();
    a.k_steps = (c.K + 255) / 256;
    a.ch_tiles = (c.N + 127) / 128;
    const int kt = (c.K + 127) / 128;
    const long long units = units_of(c, NB);
    const int split = split_for(units, a.k_steps, fit);
    a.per = (a.k_steps + split - 1) / split;
    CUtensorMap tmX, tmW, tmXs, tmWs;
    const uint64_t str[1] = {static_cast<uint64_t>(c.K) / 2};
    const uint64_t dx[2] = {str[0], static_cast<uint64_t>(c.M)};
    const uint64_t dw[2] = {str[0], static_cast<uint64_t>(c.N)};
    const uint32_t bx[2] = {128, NB}, bw[2] = {128, 128};
    if (int e = encode_map(&tmX, c.x, 2, dx, str, bx, CU_TENSOR_MAP_SWIZZLE_128B))
        return e;
    if (int e = encode_map(&tmW, c.w, 2, dw, str, bw, CU_TENSOR_MAP_SWIZZLE_128B))
        return e;
    const uint64_t sstr[2] = {512, static_cast<uint64_t>(kt) * 512};
    const uint64_t dxs[3] = {128, static_cast<uint64_t>(kt), static_cast<uint64_t>((c.M + 127) / 128)};
    const uint64_t dws[3] = {128, static_cast<uint64_t>(kt), static_cast<uint64_t>(a.ch_tiles)};
    const uint32_t bs[3] = {128, 2, 1};
    if (int e = encode_map(&tmXs, c.xs, 3, dxs, sstr, bs, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_DATA_TYPE_UINT32))
        return e;
    if (int e = encode_map(&tmWs, c.ws, 3, dws, sstr, bs, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_DATA_TYPE_UINT32))
        return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    Ke::configure(cfg, attr, units, split, s);
    return cudaLaunchKernelEx(&cfg, conv_mx4_split_kernel<T, NB>, tmX, tmW, tmXs, tmWs, a) ==
                   cudaSuccess
               ? X1CB_OK
               : X1CB_ERR_CUDA;
}

template <typename T> int run_rows(const Mx4Call &c, cudaStream_t s)
{
    return c.M <= 16 ? run<T, 16>(c, s) : c.M <= 32 ? run<T, 32>(c, s) : run<T, 64>(c, s);
}

}  // namespace

// More than 64 rows: the split pays where K is long and the chip holds all of the
// units at once, in us against 128-row tiles: 256 x 2400 x 384 7.2 and 8.8, 100 x 2048 x
// 512 6.5 and 7.2, 196 x 4096 x 1024 (clusters of four) 8.2 and 9.9; but 100 x 1024 x 256
// 6.9 and 5.8, 784 x 2400 x 384 (of two) 9.9 and 8.9.
bool conv_mx4_split_pays(const Mx4Call &c)
{
    const int k_steps = (c.K + 255) / 256;
    const long long units = units_of(c, 64);
    Fit fit;
    if (k_steps < 8 || units > 37 || Kernel<float, 64>::prepare(fit) != X1CB_OK)
        return false;
    const int split = split_for(units, k_steps, fit);
    return split == 8 || (split == 4 && k_steps >= 10);
}

int launch_conv_mx4_split(const Mx4Call &c, cudaStream_t s)
{
    return c.dtype == X1CB_F32    ? run_rows<float>(c, s)
           : c.dtype == X1CB_BF16 ? run_rows<__nv_bfloat16>(c, s)
                                  : run_rows<__half>(c, s);
}

}  // namespace x1cb
