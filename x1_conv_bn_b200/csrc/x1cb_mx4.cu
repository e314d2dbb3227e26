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
constexpr int kDepth = 4;  // rows a thread has in flight

// How a block of threads covers an [M, K] matrix in vectors: `rows` rows of nv
// vectors at a time (or one row in pieces of kBlock vectors).
struct Cover {
    int M, K, nv, rows;
};

// 16 bytes of x and the largest magnitude in them, as the bits of a float.
template <typename T, int V> __device__ __forceinline__ uint32_t amax_bits(const Vec<T, V> &v)
{
    if constexpr (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            m = max(m, __float_as_uint(v.e[i]) & 0x7fffffffu);
        return m;
    } else {
        // sign-free 16-bit patterns order as their values do, NaN above infinity
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        m = max(m >> 16, m & 0xffffu);
        if constexpr (std::is_same<T, __half>::value)
            return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(m))));
        else
            return m << 16;
    }
}

// x -> MX4.  Each thread takes 16 bytes of x, of kDepth rows at a time; the 32 / V
// neighbouring threads of a block agree on its scale, and thread d of them stores
// row d's.  Every scale is a power of two, so scaling is exact and the only
// rounding is the one to e2m1.  Bound by memory and, close behind, by
// instructions (the address arithmetic of one row at a time took half of them, 59
// us): 200704 x 512 of bfloat16 45 us, 5.8 TB/s.
template <typename T>
__global__ void __launch_bounds__(kBlock)
    quantize_kernel(const T *__restrict__ x, uint8_t *__restrict__ q, uint8_t *__restrict__ sf,
                    const Cover c)
{
    constexpr int V = 16 / sizeof(T), L = 32 / V;
    static_assert(kDepth <= L, "a thread per row");
    griddep_wait();
    const uint32_t kt = (c.K + 127) / 128;
    const int lane = threadIdx.x & 31;
    // Whole warps go through the loops together, for the shuffles: a thread with
    // nothing to do (behind the last row or vector) loads and stores nothing.
    const int r0 = c.rows > 1 ? threadIdx.x / c.nv : 0;
    const int step = gridDim.x * c.rows;
    const size_t x_step = static_cast<size_t>(step) * c.K;
    for (int v0 = blockIdx.y * kBlock; v0 < c.nv; v0 += gridDim.y * kBlock) {
        const int v = v0 + threadIdx.x - r0 * c.nv;
        const bool active = r0 < c.rows && v < c.nv;
        const int blk = v / L;
        const int pad = blk == c.K / 32 - 1 ? 3 - (blk & 3) : 0;
        uint8_t *scales = sf + static_cast<size_t>(blk >> 2) * 512 + (blk & 3);
        const int first = blockIdx.x * c.rows + r0;
        const size_t at = static_cast<size_t>(first) * c.K + v * V;
        const T *from = x + at;
        uint8_t *to = q + at / 2;
        // (rows count down, so that no row number overflows)
        int left = active ? c.M - first : 0;
        for (int all = c.M - static_cast<int>(blockIdx.x) * c.rows; all > 0;
             all = all > kDepth * step ? all - kDepth * step : 0) {
            Vec<T, V> in[kDepth];
#pragma unroll
            for (int d = 0; d < kDepth; ++d)
                if (left > d * step)
                    in[d] = load_vec<T, V>(from + d * x_step);
            from += kDepth * x_step;
            uint32_t mine = 0;  // exponent bits of the row whose scale this thread stores
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (all > d * step) {
                    uint32_t m = amax_bits<T, V>(in[d]);
#pragma unroll
                    for (int o = 1; o < L; o <<= 1)
                        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const uint32_t e = mx4_exponent(m);
                    const float inv = mx4_inverse_scale(e);
                    mine = (lane & (L - 1)) == d ? e : mine;
                    F2 f[V / 2];
                    unpack<T, V>(in[d], f);
                    float y[V];
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 t = un2(mul2(f[i], f2(inv, inv)));
                        y[2 * i] = t.x;
                        y[2 * i + 1] = t.y;
                    }
                    if (left > d * step) {
                        const bool finite = e != kMx4Bad;
                        if constexpr (V == 8)
                            *reinterpret_cast<uint32_t *>(to + d * (x_step / 2)) =
                                finite ? e2m1x8(y) : 0u;
                        else
                            *reinterpret_cast<uint16_t *>(to + d * (x_step / 2)) =
                                finite ? e2m1x4(y) : uint16_t{0};
                    }
                }
            }
            to += kDepth * (x_step / 2);
            const int d = lane & (L - 1);
            if (d < kDepth && left > d * step) {
                const uint32_t row = static_cast<uint32_t>(c.M - left) + d * step;
                uint8_t *d8 = scales + mx4_scale_row(row, kt);
                *d8 = mx4_scale_byte(mine);
                for (int j = 1; j <= pad; ++j)
                    d8[j] = 0;
            }
            left = left > kDepth * step ? left - kDepth * step : 0;
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0)
        mx4_zero_row_padding(sf, c.M, kt, threadIdx.x, kBlock);
}

// MX4 -> values: eight codes a thread, of kDepth rows at a time.  Bound by memory:
// 200704 x 512 to bfloat16 45 us, 5.7 TB/s of codes read and values written.
template <typename T>
__global__ void __launch_bounds__(kBlock)
    dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ sf,
                      T *__restrict__ x, const Cover c)
{
    griddep_wait();
    const uint32_t kt = (c.K + 127) / 128;
    const int r0 = c.rows > 1 ? threadIdx.x / c.nv : 0;
    if (r0 >= c.rows)
        return;
    const int step = gridDim.x * c.rows;
    const size_t x_step = static_cast<size_t>(step) * c.K;
    for (int v = blockIdx.y * kBlock + threadIdx.x - r0 * c.nv; v < c.nv; v += gridDim.y * kBlock) {
        const int blk = v / 4;
        const uint8_t *scales = sf + static_cast<size_t>(blk >> 2) * 512 + (blk & 3);
        const int first = blockIdx.x * c.rows + r0;
        const size_t at = static_cast<size_t>(first) * c.K + v * 8;
        const uint8_t *from = q + at / 2;
        T *to = x + at;
        for (int left = c.M - first; left > 0;
             left = left > kDepth * step ? left - kDepth * step : 0) {
            uint32_t codes[kDepth], s[kDepth];
            const uint32_t row = static_cast<uint32_t>(c.M - left);
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (left > d * step) {
                    codes[d] = __ldg(reinterpret_cast<const uint32_t *>(from + d * (x_step / 2)));
                    s[d] = __ldg(scales + mx4_scale_row(row + d * step, kt));
                }
            }
            from += kDepth * (x_step / 2);
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                if (left > d * step) {
                    __half2 h[4];
                    e2m1_to_half(codes[d], h);
                    const float scale = mx4_scale_value(s[d]);
                    constexpr int V = 16 / sizeof(T);
#pragma unroll
                    for (int j = 0; j < 8; j += V) {
                        F2 f[V / 2];
#pragma unroll
                        for (int i = 0; i < V / 2; ++i) {
                            const float2 t = __half22float2(h[j / 2 + i]);
                            f[i] = mul2(f2(t.x, t.y), f2(scale, scale));
                        }
                        store_vec<T, V>(to + d * x_step + j, finish<T, V>(f, X1CB_ACT_NONE));
                    }
                }
            }
            to += kDepth * x_step;
        }
    }
}

// The product of a single row: a warp takes kCh channels, its lanes the blocks
// lane, lane + 32, ... of the row, four of them with all loads in flight at
// once.  A block's 32 products of e2m1 values are summed in half precision, eight
// to a sum (multiples of 1/4 up to 8 * 36 = 288: exact), then scaled and summed
// in 32 bits.  The two scales, 2^-127 to 2^127 each, may lie at opposite ends of
// their range: the sum is multiplied by 2^floor(e/2) and 2^ceil(e/2), e the sum of
// their exponents, so that no step leaves the range of a float unless the product
// does (the first step is exact down to 2^-129).  Bound by latency (a launch and one trip to memory for weights that
// fit L2 many times over): 2048 x 1000 2.2 us, 4096 x 4096 4.5 us.
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
                    // scale byte xs + ws in two halves: only their product may overflow
                    const uint32_t both = xs[d] + ws[d][h], low = both >> 1;
                    const float s0 = mx4_scale_value(max(xs[d], ws[d][h]) == 255u ? 255u : low);
                    acc[h] = fmaf((f.x + f.y + (g.x + g.y)) * s0, mx4_scale_value(both - low), acc[h]);
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

Cover cover(long long M, int K, int nv)
{
    return Cover{static_cast<int>(M), K, nv, std::max(1, kBlock / nv)};
}

// Blocks for kDepth rows a thread, but no more than `deep` per SM.  Writing more
// than it reads, dequantisation gains from many short blocks (200704 x 512 to
// bf16: 51.8 us with 8, 45.0 with 32); quantisation does not (45.3 and 49.3).
// Few long rows are cut into pieces besides (quantising 200 x 8192 of float32 7.0 us
// with whole rows, 3.0 so; 1 x 32768 32.1 and 3.7).
dim3 blocks_for(const Cover &c, int deep)
{
    const int all = (c.M + c.rows - 1) / c.rows, pieces = (c.nv + kBlock - 1) / kBlock;
    const int want = (all + kDepth - 1) / kDepth;
    const int x = std::min(std::max(want, std::min(all, 148)), 148 * deep);
    return dim3(x, std::min(pieces, std::max(1, 148 * 8 / x)));
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
    Cover c = cover(M, K, K / (dtype == X1CB_F32 ? 4 : 8));
    void *params[] = {&x, &q, &sf, &c};
    return launch(k, blocks_for(c, 8), s, params) == cudaSuccess ? X1CB_OK : X1CB_ERR_CUDA;
}

int launch_dequantize_mx4(const uint8_t *q, const uint8_t *sf, void *x, int dtype, long long M,
                          int K, cudaStream_t s)
{
    const void *k = dtype == X1CB_F32    ? dequantize_fn<float>()
                    : dtype == X1CB_BF16 ? dequantize_fn<__nv_bfloat16>()
                                         : dequantize_fn<__half>();
    Cover c = cover(M, K, K / 8);
    void *params[] = {&q, &sf, &x, &c};
    return launch(k, blocks_for(c, 32), s, params) == cudaSuccess ? X1CB_OK : X1CB_ERR_CUDA;
}

// One row: conv_row_kernel.  Up to 64, and a few more where K is long: the weights
// as the MMA's rows, K split over clusters (4096 x 4096: 16 rows 5.3 us, 64 rows 8.2
// us, against 9.9 with 128-row tiles).  More: 128-row tiles.
int launch_conv_mx4(const Mx4Call &c, cudaStream_t s)
{
    if (c.M > 64 && !conv_mx4_split_pays(c))
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
