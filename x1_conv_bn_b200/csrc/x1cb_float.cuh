// Device helpers of the floating-point operators: element types, activations,
// and the MX4 number formats.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

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

// Two floats in a 64-bit register: add, multiply-add and multiply work on both
// at once (sm_100), each rounded as the scalar operation.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float x, float y)
{
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 un2(F2 v)
{
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ F2 neg2(F2 a) { return a ^ 0x8000000080000000ull; }

// Pairs of a vector of V elements; an odd single element leaves the upper half 0.
template <int V> constexpr int kPairs = (V + 1) / 2;
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V> &v, F2 (&f)[kPairs<V>])
{
    if constexpr (V == 1) {
        f[0] = f2(to_f(v.e[0]), 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const uint32_t w = reinterpret_cast<const uint32_t *>(&v)[i];
                f[i] = f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 t = __half22float2(reinterpret_cast<const __half2 *>(&v)[i]);
                f[i] = f2(t.x, t.y);
            } else {
                f[i] = f2(v.e[2 * i], v.e[2 * i + 1]);
            }
        }
    }
}

// Two floats -> two elements of 16 bits; RELU: negative results become 0 (NaN stays).
template <typename T, bool RELU> __device__ __forceinline__ uint32_t pack2(float x, float y)
{
    uint32_t d;
    if constexpr (std::is_same<T, __half>::value) {
        if constexpr (RELU)
            asm("cvt.rn.relu.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
        else
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    } else {
        if constexpr (RELU)
            asm("cvt.rn.relu.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
        else
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(y), "f"(x));
    }
    return d;
}

// NaN stays NaN.
__device__ __forceinline__ float relu(float v)
{
    float d;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(d) : "f"(v));
    return d;
}
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

__device__ __forceinline__ float activate(float v, int act)
{
    return act == X1CB_ACT_RELU ? relu(v) : act == X1CB_ACT_SILU ? silu(v) : v;
}

template <int V> __device__ __forceinline__ void activate(float (&y)[V], int act)
{
    if (act == X1CB_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            y[i] = relu(y[i]);
    } else if (act == X1CB_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            y[i] = silu(y[i]);
    }
}

// Largest magnitude, as the bits of a float; NaN if one is.
template <int V> __device__ __forceinline__ uint32_t amax_bits(const float (&y)[V])
{
    static_assert(V == 4 || V == 8, "");
    float m;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(fabsf(y[0])), "f"(fabsf(y[1])), "f"(fabsf(y[2])));
    if constexpr (V == 4) {
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(y[3])));
    } else {
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(y[3])), "f"(fabsf(y[4])));
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(fabsf(y[5])), "f"(fabsf(y[6])));
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(y[7])));
    }
    return __float_as_uint(m);
}

// act(y) rounded to T, in one pass: ReLU is part of the 16-bit conversions.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> finish(const F2 (&f)[kPairs<V>], int act)
{
    Vec<T, V> v;
    if constexpr (V == 1) {
        v.e[0] = from_f<T>(activate(un2(f[0]).x, act));
    } else if constexpr (sizeof(T) == 4) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 t = un2(f[i]);
            y[2 * i] = t.x;
            y[2 * i + 1] = t.y;
        }
        activate(y, act);
#pragma unroll
        for (int i = 0; i < V; ++i)
            v.e[i] = y[i];
    } else {
        uint32_t *w = reinterpret_cast<uint32_t *>(&v);
        if (act == X1CB_ACT_RELU) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 t = un2(f[i]);
                w[i] = pack2<T, true>(t.x, t.y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                float2 t = un2(f[i]);
                if (act == X1CB_ACT_SILU)
                    t = make_float2(silu(t.x), silu(t.y));
                w[i] = pack2<T, false>(t.x, t.y);
            }
        }
    }
    return v;
}

// Copy of N bytes from global to shared memory that completes in the thread's
// bulk of asynchronous copies (commit, then wait).
template <int N> __device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(N)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// A block's exponent bits from the bits of its largest magnitude: the float's
// exponent field e, at least 2, where it stands in the float.  The scale byte is
// e - 2 (e is floor(log2) + 127, and 4, the largest power of two in e2m1, takes
// 2 of it; subnormals and zeros have field 0 and end at byte 0), the inverse
// scale 2^(129 - e), exact; field 255 is a block with an infinity or NaN.
constexpr uint32_t kMx4Bad = 0x7f800000u;
__device__ __forceinline__ uint32_t mx4_exponent(uint32_t amax)
{
    return max(amax & 0x7f800000u, 0x01000000u);
}
__device__ __forceinline__ float mx4_inverse_scale(uint32_t e)
{
    return __uint_as_float(0x80000000u - e);
}
__device__ __forceinline__ uint8_t mx4_scale_byte(uint32_t e)
{
    return static_cast<uint8_t>(e == kMx4Bad ? 255u : (e >> 23) - 2u);
}

// Byte of a row's scales in the array, for the first block of the first tile.
__device__ __forceinline__ size_t mx4_scale_row(uint32_t row, uint32_t kt)
{
    return static_cast<size_t>((row >> 7) * kt) * 512 + ((row & 31) * 16 + ((row >> 5) & 3) * 4);
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

// Zeroes the scale bytes of rows M .. 128*ceil(M/128) - 1 (threads tid of n): of
// each 16 bytes of the last tiles, which hold the rows g, g + 32, g + 64 and g + 96.
__device__ __forceinline__ void mx4_zero_row_padding(uint8_t *sf, long long M, int kt, int tid,
                                                     int n)
{
    const int first = static_cast<int>(M & 127);
    if (first == 0)
        return;
    uint4 *to = reinterpret_cast<uint4 *>(sf + static_cast<size_t>(M >> 7) * kt * 512);
    for (int i = tid; i < kt * 32; i += n) {
        const int g = i & 31;
        if (g >= first) {
            to[i] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            uint32_t *w = reinterpret_cast<uint32_t *>(to + i);
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (g + 32 * q >= first)
                    w[q] = 0u;
        }
    }
}

}  // namespace x1cb
