// MX4 (OCP MXFP4: e2m1 elements, one e8m0 scale per 32) conversions, and the
// MX4 1x1 convolution in its plainest form: a warp per output channel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "x1cb_float.cuh"
#include "x1cb_internal.h"
#include "x1cb_ptx.cuh"

namespace x1cb {
namespace {

constexpr int kBlock = 256;

// x -> MX4.  Each thread takes 16 bytes of x; the 32 / V neighbouring threads
// of a block agree on its scale.  Every scale is a power of two, so scaling is
// exact and the only rounding is the one to e2m1.
template <typename T>
__global__ void __launch_bounds__(kBlock)
    quantize_kernel(const T *__restrict__ x, uint8_t *__restrict__ q, uint8_t *__restrict__ sf,
                    long long M, int K)
{
    constexpr int V = 16 / sizeof(T), L = 32 / V;
    griddep_wait();
    const int kt = (K + 127) / 128, nv = K / V;
    const long long n = M * nv;
    const int lane = threadIdx.x & 31;
    const uint32_t mask = ((1u << L) - 1u) << (lane & ~(L - 1));
    const long long t0 = blockIdx.x * static_cast<long long>(kBlock) + threadIdx.x;
    for (long long t = t0; t < n; t += static_cast<long long>(gridDim.x) * kBlock) {
        const long long row = t / nv;
        const int k = static_cast<int>(t - row * nv) * V;
        const Vec<T, V> v = load_vec<T, V>(x + t * V);
        float f[V];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f[i] = to_f(v.e[i]);
            m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1)
            m = max(m, __shfl_xor_sync(mask, m, o));
        const uint32_t s = mx4_scale_byte(m);
        const float inv = mx4_inverse_scale(min(s, 252u));
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] *= inv;
        if constexpr (V == 8)
            reinterpret_cast<uint32_t *>(q)[t] = s == 255u ? 0u : e2m1x8(f);
        else
            reinterpret_cast<uint16_t *>(q)[t] = s == 255u ? uint16_t{0} : e2m1x4(f);
        if ((lane & (L - 1)) == 0) {
            const int blk = k / 32;
            uint8_t *d = sf + mx4_scale_at(row, blk, kt);
            *d = static_cast<uint8_t>(s);
            if (blk == K / 32 - 1)
                for (int j = 1; j < 4 - (blk & 3); ++j)
                    d[j] = 0;
        }
    }
    if (blockIdx.x == 0)
        mx4_zero_row_padding(sf, M, kt, threadIdx.x, kBlock);
}

// MX4 -> values: eight codes a thread.
template <typename T>
__global__ void __launch_bounds__(kBlock)
    dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ sf,
                      T *__restrict__ x, long long M, int K)
{
    griddep_wait();
    const int kt = (K + 127) / 128, nv = K / 8;
    const long long n = M * nv;
    for (long long t = blockIdx.x * static_cast<long long>(kBlock) + threadIdx.x; t < n;
         t += static_cast<long long>(gridDim.x) * kBlock) {
        const long long row = t / nv;
        const int k = static_cast<int>(t - row * nv) * 8;
        __half2 h[4];
        e2m1_to_half(reinterpret_cast<const uint32_t *>(q)[t], h);
        const float s = mx4_scale_value(sf[mx4_scale_at(row, k / 32, kt)]);
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8; j += V) {
            Vec<T, V> v;
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float2 f = __half22float2(h[(j + i) / 2]);
                v.e[i] = from_f<T>(f.x * s);
                v.e[i + 1] = from_f<T>(f.y * s);
            }
            store_vec<T, V>(x + t * 8 + j, v);
        }
    }
}

// out[m, o] for one o per warp and kRows rows m at a time.  A lane takes the
// blocks lane, lane + 32, ... of the row: 32 products of e2m1 values, summed in
// half precision by fours (multiples of 1/4 up to 4 * 36 = 144: exact), then
// scaled and summed in 32 bits.
constexpr int kRows = 4;
template <typename T>
__global__ void __launch_bounds__(kBlock) conv_rows_kernel(Mx4Call c)
{
    griddep_wait();
    const int o = blockIdx.x * (kBlock / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (o >= c.N)
        return;
    const int blocks = c.K / 32, kt = (c.K + 127) / 128;
    const uint4 *w = reinterpret_cast<const uint4 *>(c.w) + static_cast<size_t>(o) * blocks;
    for (long long m0 = static_cast<long long>(blockIdx.y) * kRows; m0 < c.M;
         m0 += static_cast<long long>(gridDim.y) * kRows) {
        float acc[kRows] = {};
        for (int b = lane; b < blocks; b += 32) {
            const uint4 wq = w[b];
            const float wscale = mx4_scale_value(c.ws[mx4_scale_at(o, b, kt)]);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const long long m = m0 + r;
                if (m >= c.M)
                    break;
                const uint4 xq = reinterpret_cast<const uint4 *>(c.x)[m * blocks + b];
                const float xscale = mx4_scale_value(c.xs[mx4_scale_at(m, b, kt)]);
                const uint32_t wa[4] = {wq.x, wq.y, wq.z, wq.w}, xa[4] = {xq.x, xq.y, xq.z, xq.w};
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    __half2 wh[4], xh[4];
                    e2m1_to_half(wa[i], wh);
                    e2m1_to_half(xa[i], xh);
                    __half2 d = __hmul2(wh[0], xh[0]);
#pragma unroll
                    for (int j = 1; j < 4; ++j)
                        d = __hfma2(wh[j], xh[j], d);
                    const float2 f = __half22float2(d);
                    dot += f.x + f.y;
                }
                acc[r] = fmaf(dot * wscale, xscale, acc[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
                acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], d);
            const long long m = m0 + r;
            if (lane == r && m < c.M) {
                float v = acc[r] + (c.bias ? c.bias[o] : 0.f);
                const size_t at = static_cast<size_t>(m) * c.N + o;
                if (c.r)
                    v += to_f(static_cast<const T *>(c.r)[at]);
                static_cast<T *>(c.out)[at] = from_f<T>(activate(v, c.act));
            }
        }
    }
}

cudaError_t launch(const void *kern, dim3 grid, cudaStream_t s, void **params)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kBlock, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kern, params);
}

int blocks_for(long long threads)
{
    return static_cast<int>(std::min<long long>((threads + kBlock - 1) / kBlock, 148 * 32));
}

template <typename T> const void *quantize_fn()
{
    return reinterpret_cast<const void *>(quantize_kernel<T>);
}
template <typename T> const void *dequantize_fn()
{
    return reinterpret_cast<const void *>(dequantize_kernel<T>);
}

}  // namespace

int launch_quantize_mx4(const void *x, int dtype, uint8_t *q, uint8_t *sf, long long M, int K,
                        cudaStream_t s)
{
    const void *k = dtype == X1CB_F32    ? quantize_fn<float>()
                    : dtype == X1CB_BF16 ? quantize_fn<__nv_bfloat16>()
                                         : quantize_fn<__half>();
    void *params[] = {&x, &q, &sf, &M, &K};
    const int V = dtype == X1CB_F32 ? 4 : 8;
    return launch(k, dim3(blocks_for(M * (K / V))), s, params) == cudaSuccess ? X1CB_OK
                                                                              : X1CB_ERR_CUDA;
}

int launch_dequantize_mx4(const uint8_t *q, const uint8_t *sf, void *x, int dtype, long long M,
                          int K, cudaStream_t s)
{
    const void *k = dtype == X1CB_F32    ? dequantize_fn<float>()
                    : dtype == X1CB_BF16 ? dequantize_fn<__nv_bfloat16>()
                                         : dequantize_fn<__half>();
    void *params[] = {&q, &sf, &x, &M, &K};
    return launch(k, dim3(blocks_for(M * (K / 8))), s, params) == cudaSuccess ? X1CB_OK
                                                                              : X1CB_ERR_CUDA;
}

int launch_conv_mx4(const Mx4Call &c, cudaStream_t s)
{
    if (c.M > 8)
        return launch_conv_mx4_tiles(c, s);
    Mx4Call a = c;
    const void *k = c.dtype == X1CB_F32    ? reinterpret_cast<const void *>(conv_rows_kernel<float>)
                    : c.dtype == X1CB_BF16 ? reinterpret_cast<const void *>(conv_rows_kernel<__nv_bfloat16>)
                                           : reinterpret_cast<const void *>(conv_rows_kernel<__half>);
    void *params[] = {&a};
    const long long rows = (c.M + kRows - 1) / kRows;
    const dim3 grid((c.N + kBlock / 32 - 1) / (kBlock / 32),
                    static_cast<unsigned>(std::min<long long>(rows, 4096)));
    return launch(k, grid, s, params) == cudaSuccess ? X1CB_OK : X1CB_ERR_CUDA;
}

}  // namespace x1cb
