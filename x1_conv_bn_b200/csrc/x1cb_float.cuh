// Device helpers of the floating-point operators: element types, activations,
// and the MX4 number formats.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/x1cb.h"

namespace x1cb {

// N consecutive elements as one load or store of up to 16 bytes.
template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };
template <> struct Raw<1> { using type = uint8_t; };

template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    using raw = typename Raw<sizeof(T) * V>::type;
    T e[V];
};

template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const T *p)
{
    using R = typename Vec<T, V>::raw;
    Vec<T, V> v;
    *reinterpret_cast<R *>(&v) = __ldg(reinterpret_cast<const R *>(p));
    return v;
}

template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &v)
{
    using R = typename Vec<T, V>::raw;
    *reinterpret_cast<R *>(p) = *reinterpret_cast<const R *>(&v);
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v)
{
    return __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// v < 0 is false for NaN, which therefore passes through ReLU.
__device__ __forceinline__ float activate(float v, int act)
{
    if (act == X1CB_ACT_RELU)
        return v < 0.f ? 0.f : v;
    if (act == X1CB_ACT_SILU)
        return __fdividef(v, 1.f + __expf(-v));
    return v;
}

// Byte of the scale of (row, block) in an MX4 scale array whose rows have kt =
// ceil(K/128) tiles.
__host__ __device__ __forceinline__ size_t mx4_scale_at(long long row, int block, int kt)
{
    return (static_cast<size_t>(row >> 7) * kt + (block >> 2)) * 512 + (row & 31) * 16 +
           ((row >> 5) & 3) * 4 + (block & 3);
}

// 2^(s - 127); 255 is NaN, 0 the subnormal 2^-127.
__device__ __forceinline__ float mx4_scale_value(uint32_t s)
{
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// Scale byte of a block whose largest magnitude has the float bits `amax`
// (sign clear): the float's exponent field is floor(log2) + 127, so the byte
// is that less 2 (the exponent of 4, the largest power of two in e2m1);
// subnormals and zeros have field 0 and end at 0 with it.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax)
{
    const int e = static_cast<int>(amax >> 23);
    return e == 255 ? 255u : static_cast<uint32_t>(max(e - 2, 0));
}

// 2^(127 - s) for s <= 252 (a finite block's largest byte): exact.
__device__ __forceinline__ float mx4_inverse_scale(uint32_t s)
{
    return __uint_as_float((254u - s) << 23);
}

// Eight floats -> eight e2m1 codes (round to nearest even, saturating),
// element 0 in the lowest half byte.
__device__ __forceinline__ uint32_t e2m1x8(const float *v)
{
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

__device__ __forceinline__ uint16_t e2m1x4(const float *v)
{
    uint16_t d;
    asm("{\n\t.reg .b8 b0, b1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "mov.b16 %0, {b0, b1};\n\t}"
        : "=h"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
    return d;
}

// Eight e2m1 codes -> four half2 of their values (exact).
__device__ __forceinline__ void e2m1_to_half(uint32_t codes, __half2 (&h)[4])
{
    uint32_t r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = *reinterpret_cast<const __half2 *>(&r[i]);
}

// Zeroes the scale bytes of rows M .. 128*ceil(M/128) - 1 (threads tid of n).
__device__ __forceinline__ void mx4_zero_row_padding(uint8_t *sf, long long M, int kt, int tid,
                                                     int n)
{
    const int rows = static_cast<int>((128 - (M & 127)) & 127);
    for (int i = tid; i < rows * kt; i += n) {
        const size_t at = mx4_scale_at(M + i / kt, (i % kt) * 4, kt);
        *reinterpret_cast<uint32_t *>(sf + at) = 0u;
    }
}

}  // namespace x1cb
