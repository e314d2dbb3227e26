// Group norm + shortcut Sum + activation, channels last, with floating-point,
// int8 NC/32HW32 or MX4 output.
//
// Statistics: a thread owns V neighbouring channels and walks down the pixels.
// Per channel it sums d = x - k and d^2 about the first value k it met, which
// gives its mean and its sum of squares about the mean, M2 = sum d^2 -
// (sum d)^2/n.  k being one of the n values, n (mean - k)^2 <= n M2, so the
// subtraction costs at most a factor n of the relative rounding error, however
// far the data lies from zero; n is kept at or below 64 by folding the sums
// into a running (mean, M2) after 64 pixels.  Partial results are joined in a
// fixed order: the mean of the parts, then M2 + n (mean - joint mean)^2 summed.
//
// This file's first form takes two launches: partial statistics per chunk of
// pixels into the workspace, then the normalisation, which joins them.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>

#include "x1cb_float.cuh"
#include "x1cb_internal.h"
#include "x1cb_ptx.cuh"

namespace x1cb {
namespace {

constexpr int kBlock = 256;
constexpr int kFold = 64;  // pixels a channel's shifted sums run over

struct NormArgs {
    const void *x, *r;
    const float *gamma, *beta;
    void *y;
    uint8_t *sf;
    float2 *part;  // [B][chunks][G] (mean, M2)
    float eps, q_mul;
    int act, B, HW, C, G, cg;
    int nv;             // vectors of V channels per pixel
    int lanes;          // pixels the block takes at a time (kBlock / nv, at least 1)
    int chunks, chunk;  // chunks per image, pixels per chunk
};

// (mean, M2) of the values seen so far, and the shifted sums of the current run.
template <int V> struct Running {
    float mean[V], m2[V], k[V], s[V], q[V];
    int n = 0, run = 0;

    __device__ __forceinline__ void add(const float (&x)[V])
    {
        if (run == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                k[i] = x[i];
                s[i] = q[i] = 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = x[i] - k[i];
                s[i] += d;
                q[i] = fmaf(d, d, q[i]);
            }
        }
        if (++run == kFold)
            fold();
    }
    __device__ __forceinline__ void fold()
    {
        if (run == 0)
            return;
        const float inv = 1.f / static_cast<float>(run);
        const float w = static_cast<float>(run) / static_cast<float>(n + run);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float ms = s[i] * inv;
            const float rm = k[i] + ms;
            const float r2 = fmaxf(fmaf(-ms, s[i], q[i]), 0.f);
            if (n == 0) {
                mean[i] = rm;
                m2[i] = r2;
            } else {
                const float d = rm - mean[i];
                mean[i] = fmaf(d, w, mean[i]);
                m2[i] += r2 + d * d * (static_cast<float>(n) * w);
            }
        }
        n += run;
        run = 0;
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Joins `count` parts of one group, part i of weight cnt(i): the warp's lanes
// take the parts in turn.  All lanes return (mean, M2).
template <typename Get>
__device__ __forceinline__ float2 warp_join(int count, int lane, const Get &get)
{
    float n = 0.f, first = 0.f, sum = 0.f;
    {
        float c;
        first = get(0, c).x;  // the shift of the joint sum
    }
    for (int i = lane; i < count; i += 32) {
        float c;
        const float2 p = get(i, c);
        n += c;
        sum = fmaf(c, c > 0.f ? p.x - first : 0.f, sum);
    }
    n = warp_sum(n);
    sum = warp_sum(sum);
    const float mean = first + sum / n;
    float m2 = 0.f;
    for (int i = lane; i < count; i += 32) {
        float c;
        const float2 p = get(i, c);
        if (c > 0.f) {
            const float d = p.x - mean;
            m2 += fmaf(c * d, d, p.y);
        }
    }
    return make_float2(mean, warp_sum(m2));
}

// Statistics of one chunk of pixels of one image: part[b][chunk][g].
template <typename T, int V> __global__ void __launch_bounds__(kBlock) norm_stats_kernel(NormArgs a)
{
    extern __shared__ float2 buf[];  // [lanes][C] (mean, M2) of each pixel lane and channel
    griddep_wait();
    const int b = blockIdx.y;
    const int p0 = blockIdx.x * a.chunk, p1 = min(a.HW, p0 + a.chunk);
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(b) * a.HW * a.C;
    const int pl = threadIdx.x / a.nv;
    if (pl < a.lanes) {
        for (int cv = threadIdx.x - pl * a.nv; cv < a.nv; cv += kBlock) {
            Running<V> st;
            for (int p = p0 + pl; p < p1; p += a.lanes) {
                const Vec<T, V> v = load_vec<T, V>(x + static_cast<size_t>(p) * a.C + cv * V);
                float f[V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    f[i] = to_f(v.e[i]);
                st.add(f);
            }
            st.fold();
#pragma unroll
            for (int i = 0; i < V; ++i)
                buf[pl * a.C + cv * V + i] =
                    st.n ? make_float2(st.mean[i], st.m2[i]) : make_float2(0.f, 0.f);
        }
    }
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int px = p1 - p0;
    for (int g = warp; g < a.G; g += kBlock / 32) {
        const float2 r = warp_join(a.lanes * a.cg, lane, [&](int i, float &c) {
            const int l = i / a.cg;
            c = static_cast<float>((px - l + a.lanes - 1) / a.lanes);  // pixels of lane l
            return buf[l * a.C + g * a.cg + (i - l * a.cg)];
        });
        if (lane == 0)
            a.part[(static_cast<size_t>(b) * a.chunks + blockIdx.x) * a.G + g] = r;
    }
}

// One vector of V outputs of pixel p (of image b), channels c.. on.
template <typename T, int V, int OUT>
__device__ __forceinline__ void emit(const NormArgs &a, int b, int p, int c, float (&y)[V])
{
    const size_t at = (static_cast<size_t>(b) * a.HW + p) * a.C + c;
    if (OUT == kNormSame) {
        Vec<T, V> v;
#pragma unroll
        for (int i = 0; i < V; ++i)
            v.e[i] = from_f<T>(y[i]);
        store_vec<T, V>(static_cast<T *>(a.y) + at, v);
    } else if (OUT == kNormI8) {
        // NC/32HW32; saturating convert-to-integer, NaN to 0
        Vec<int8_t, V> v;
#pragma unroll
        for (int i = 0; i < V; ++i)
            v.e[i] = static_cast<int8_t>(max(-128, min(127, __float2int_rn(y[i] * a.q_mul))));
        int8_t *q = static_cast<int8_t *>(a.y) +
                    ((static_cast<size_t>(b) * (a.C / 32) + c / 32) * a.HW + p) * 32 + c % 32;
        store_vec<int8_t, V>(q, v);
    } else {
        // The 32 / V neighbouring threads that hold a block agree on its scale
        // (they belong to one pixel, so they are here together).
        constexpr int L = 32 / V;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
        const int lane = threadIdx.x & 31;
        const uint32_t mask = ((L == 32 ? 0u : (1u << (L & 31))) - 1u) << (lane & ~(L - 1));
#pragma unroll
        for (int o = 1; o < L; o <<= 1)
            m = max(m, __shfl_xor_sync(mask, m, o));
        const uint32_t s = mx4_scale_byte(m);
        const float inv = mx4_inverse_scale(min(s, 252u));
#pragma unroll
        for (int i = 0; i < V; ++i)
            y[i] *= inv;
        uint8_t *q = static_cast<uint8_t *>(a.y) + at / 2;
        if constexpr (V == 8)
            *reinterpret_cast<uint32_t *>(q) = s == 255u ? 0u : e2m1x8(y);
        else if constexpr (V == 4)
            *reinterpret_cast<uint16_t *>(q) = s == 255u ? uint16_t{0} : e2m1x4(y);
        if ((lane & (L - 1)) == 0) {
            const int kt = (a.C + 127) / 128, blk = c / 32;
            uint8_t *d = a.sf + mx4_scale_at(static_cast<long long>(b) * a.HW + p, blk, kt);
            *d = static_cast<uint8_t>(s);
            if (blk == a.C / 32 - 1)  // the row's last block: the rest of its tile is padding
                for (int k = 1; k < 4 - (blk & 3); ++k)
                    d[k] = 0;
        }
    }
}

template <typename T, int V, int OUT>
__global__ void __launch_bounds__(kBlock) norm_apply_kernel(NormArgs a)
{
    extern __shared__ float2 buf[];  // [G] (mean, 1/std)
    griddep_wait();
    const int b = blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int g = warp; g < a.G; g += kBlock / 32) {
        const float2 *part = a.part + static_cast<size_t>(b) * a.chunks * a.G + g;
        const float2 r = warp_join(a.chunks, lane, [&](int i, float &c) {
            c = static_cast<float>(min(a.HW, (i + 1) * a.chunk) - i * a.chunk) * a.cg;
            return part[static_cast<size_t>(i) * a.G];
        });
        if (lane == 0)
            buf[g] = make_float2(
                r.x, 1.f / sqrtf(r.y / (static_cast<float>(a.HW) * a.cg) + a.eps));
    }
    if (OUT == kNormMx4 && b == 0 && blockIdx.x == 0)
        mx4_zero_row_padding(a.sf, static_cast<long long>(a.B) * a.HW, (a.C + 127) / 128,
                             threadIdx.x, kBlock);
    __syncthreads();
    const int p0 = blockIdx.x * a.chunk, p1 = min(a.HW, p0 + a.chunk);
    const size_t base = static_cast<size_t>(b) * a.HW * a.C;
    const T *x = static_cast<const T *>(a.x) + base;
    const T *r = a.r ? static_cast<const T *>(a.r) + base : nullptr;
    const int pl = threadIdx.x / a.nv;
    if (pl >= a.lanes)
        return;
    for (int cv = threadIdx.x - pl * a.nv; cv < a.nv; cv += kBlock) {
        float mu[V], sc[V], be[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = cv * V + i;
            const float2 m = buf[c / a.cg];
            mu[i] = m.x;
            sc[i] = a.gamma ? m.y * a.gamma[c] : m.y;
            be[i] = a.beta ? a.beta[c] : 0.f;
        }
        for (int p = p0 + pl; p < p1; p += a.lanes) {
            const size_t at = static_cast<size_t>(p) * a.C + cv * V;
            const Vec<T, V> v = load_vec<T, V>(x + at);
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                y[i] = fmaf(to_f(v.e[i]) - mu[i], sc[i], be[i]);
            if (r) {
                const Vec<T, V> w = load_vec<T, V>(r + at);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    y[i] += to_f(w.e[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                y[i] = activate(y[i], a.act);
            emit<T, V, OUT>(a, b, p, cv * V, y);
        }
    }
}

// Channels per vector: the most that divide C, up to 16 bytes.
int vector_channels(int dtype, int C)
{
    int v = dtype == X1CB_F32 ? 4 : 8;
    while (C % v)
        v /= 2;
    return v;
}

struct Geometry {
    int V, nv, lanes, chunks, chunk;
};

Geometry geometry(int dtype, int B, int HW, int C)
{
    Geometry g;
    g.V = vector_channels(dtype, C);
    g.nv = C / g.V;
    g.lanes = std::max(1, kBlock / g.nv);
    // enough blocks for every SM several times over, at least 8 pixels a thread
    const long long want = std::max(1, 148 * 8 / B);
    const long long most = std::max(1, HW / (g.lanes * 8));
    g.chunks = static_cast<int>(std::min(want, most));
    g.chunk = (HW + g.chunks - 1) / g.chunks;
    g.chunks = (HW + g.chunk - 1) / g.chunk;
    return g;
}

cudaError_t launch(const void *kern, dim3 grid, int threads, size_t smem, cudaStream_t s,
                   void **params)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, params);
}

template <typename T, int V> int run(const NormCall &c, const NormArgs &a0, cudaStream_t s)
{
    NormArgs a = a0;
    const size_t stat_smem = static_cast<size_t>(a.lanes) * a.C * sizeof(float2);
    if (stat_smem > 48 * 1024 &&
        cudaFuncSetAttribute(norm_stats_kernel<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             8192 * static_cast<int>(sizeof(float2))) != cudaSuccess)
        return X1CB_ERR_CUDA;
    const dim3 grid(a.chunks, a.B);
    void *params[] = {&a};
    if (launch(reinterpret_cast<const void *>(norm_stats_kernel<T, V>), grid, kBlock, stat_smem,
               s, params) != cudaSuccess)
        return X1CB_ERR_CUDA;
    const void *k = reinterpret_cast<const void *>(norm_apply_kernel<T, V, kNormSame>);
    if constexpr (V * sizeof(T) == 16) {
        if (c.out == kNormI8)
            k = reinterpret_cast<const void *>(norm_apply_kernel<T, V, kNormI8>);
        else if (c.out == kNormMx4)
            k = reinterpret_cast<const void *>(norm_apply_kernel<T, V, kNormMx4>);
    }
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             8192 * static_cast<int>(sizeof(float2))) != cudaSuccess)
        return X1CB_ERR_CUDA;
    if (launch(k, grid, kBlock, static_cast<size_t>(a.G) * sizeof(float2), s, params) !=
        cudaSuccess)
        return X1CB_ERR_CUDA;
    return X1CB_OK;
}

template <typename T> int run_v(const NormCall &c, const NormArgs &a, int V, cudaStream_t s)
{
    if (V == 8) {
        if constexpr (sizeof(T) == 2)
            return run<T, 8>(c, a, s);
    }
    return V == 4 ? run<T, 4>(c, a, s) : V == 2 ? run<T, 2>(c, a, s) : run<T, 1>(c, a, s);
}

}  // namespace

size_t norm_workspace_floats(int dtype, int B, int HW, int C, int G)
{
    const Geometry g = geometry(dtype, B, HW, C);
    return static_cast<size_t>(B) * g.chunks * G * 2;
}

int launch_norm(const NormCall &c, cudaStream_t s)
{
    if (c.B > 65535)
        return X1CB_ERR_SHAPE;
    const Geometry g = geometry(c.dtype, c.B, c.HW, c.C);
    NormArgs a{};
    a.x = c.x;
    a.r = c.r;
    a.gamma = c.gamma;
    a.beta = c.beta;
    a.y = c.y;
    a.sf = c.sf;
    a.part = reinterpret_cast<float2 *>(c.ws);
    a.eps = c.eps;
    a.q_mul = c.q_mul;
    a.act = c.act;
    a.B = c.B;
    a.HW = c.HW;
    a.C = c.C;
    a.G = c.G;
    a.cg = c.C / c.G;
    a.nv = g.nv;
    a.lanes = g.lanes;
    a.chunks = g.chunks;
    a.chunk = g.chunk;
    if (c.dtype == X1CB_F32)
        return run_v<float>(c, a, g.V, s);
    return c.dtype == X1CB_BF16 ? run_v<__nv_bfloat16>(c, a, g.V, s) : run_v<__half>(c, a, g.V, s);
}

}  // namespace x1cb
