// MX4 (OCP MXFP4: e2m1 elements, one e8m0 scale per 32) conversions, and the
// MX4 1x1 convolution of a single row.
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

// The product of a single row: a warp takes kCh channels, its lanes the blocks
// lane, lane + 32, ... of the row, four of them with all loads in flight at
// once.  A block's 32 products of e2m1 values are summed in half precision, eight
// to a sum (multiples of 1/4 up to 8 * 36 = 288: exact), then scaled and summed
// in 32 bits.  Bound by latency (a launch and one trip to memory for weights that
// fit L2 many times over): KKK.
template <typename T, int kCh>
__global__ void __launch_bounds__(kBlock) conv_row_kernel(Mx4Call c)
{
    constexpr int kDeep = 4;
    const int lane = threadIdx.x & 31;
    const int o0 = (blockIdx.x * (kBlock / 32) + threadIdx.x / 32) * kCh;
    griddep_wait();
    if (o0 >= c.N)
        return;
    const int blocks = c.K / 32, kt = (c.K + 127) / 128;
    const uint4 *x = reinterpret_cast<const uint4 *>(c.x);
    float acc[kCh] = {};
    for (int b0 = lane; b0 < blocks; b0 += 32 * kDeep) {
        uint4 xq[kDeep], wq[kDeep][kCh];
        uint32_t xs[kDeep], ws[kDeep][kCh];
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            const int b = b0 + 32 * d;
            if (b < blocks) {
                xq[d] = __ldg(x + b);
                xs[d] = __ldg(c.xs + mx4_scale_at(0, b, kt));
#pragma unroll
                for (int h = 0; h < kCh; ++h) {
                    const int o = min(o0 + h, c.N - 1);
                    wq[d][h] = __ldg(reinterpret_cast<const uint4 *>(c.w) +
                                     static_cast<size_t>(o) * blocks + b);
                    ws[d][h] = __ldg(c.ws + mx4_scale_at(o, b, kt));
                }
            }
        }
#pragma unroll
        for (int d = 0; d < kDeep; ++d) {
            if (b0 + 32 * d < blocks) {
                const uint32_t xa[4] = {xq[d].x, xq[d].y, xq[d].z, xq[d].w};
                __half2 xh[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    e2m1_to_half(xa[i], xh[i]);
                const float xscale = mx4_scale_value(xs[d]);
#pragma unroll
                for (int h = 0; h < kCh; ++h) {
                    const uint32_t wa[4] = {wq[d][h].x, wq[d][h].y, wq[d][h].z, wq[d][h].w};
                    __half2 sum[2];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        __half2 wh[4];
                        e2m1_to_half(wa[i], wh);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sum[i / 2] = i % 2 == 0 && j == 0 ? __hmul2(wh[j], xh[i][j])
                                                              : __hfma2(wh[j], xh[i][j], sum[i / 2]);
                    }
                    const float2 f = __half22float2(sum[0]), g = __half22float2(sum[1]);
                    acc[h] = fmaf((f.x + f.y + (g.x + g.y)) * mx4_scale_value(ws[d][h]), xscale,
                                  acc[h]);
                }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < kCh; ++h) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], d);
        const int o = o0 + h;
        if (lane == h && o < c.N) {
            float v = acc[h] + (c.bias ? c.bias[o] : 0.f);
            if (c.r)
                v += to_f(static_cast<const T *>(c.r)[o]);
            static_cast<T *>(c.out)[o] = from_f<T>(activate(v, c.act));
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
template <typename T> const void *row_fn(int ch)
{
    return ch == 2 ? reinterpret_cast<const void *>(conv_row_kernel<T, 2>)
                   : reinterpret_cast<const void *>(conv_row_kernel<T, 1>);
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

// One row: conv_row_kernel.  Up to 64: the weights as the MMA's rows, K split
// over clusters (4096 x 4096: 16 rows 5.3 us, 64 rows 8.2 us, against 9.9 with
// 128-row tiles; 128 rows 10.6 against 10.2).  More: 128-row tiles.
int launch_conv_mx4(const Mx4Call &c, cudaStream_t s)
{
    if (c.M > 64)
        return launch_conv_mx4_tiles(c, s);
    if (c.M > 1)
        return launch_conv_mx4_split(c, s);
    Mx4Call a = c;
    const int ch = c.N > 148 * 8 * 2 ? 2 : 1;
    const void *k =
        c.dtype == X1CB_F32    ? row_fn<float>(ch)
        : c.dtype == X1CB_BF16 ? row_fn<__nv_bfloat16>(ch)
                               : row_fn<__half>(ch);
    void *params[] = {&a};
    const int per_block = kBlock / 32 * ch;
    return launch(k, dim3((c.N + per_block - 1) / per_block), s, params) == cudaSuccess
               ? X1CB_OK
               : X1CB_ERR_CUDA;
}

}  // namespace x1cb
