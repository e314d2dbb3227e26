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
// Two forms.  Where an image (or a slice of its channels that holds whole
// groups) fits the shared memory of a cluster of up to eight CTAs, one launch
// reads it once, keeps it there, joins the statistics over the cluster and
// normalises from shared memory: x in, y out, nothing else.  Larger images take
// two launches, partial statistics per chunk of pixels into the workspace and
// the normalisation, over as many images at a time as stay in L2 between them.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "x1cb_float.cuh"
#include "x1cb_internal.h"
#include "x1cb_ptx.cuh"

namespace x1cb {
namespace {

constexpr int kBlock = 256;
constexpr int kFold = 64;  // pixels a channel's shifted sums run over
constexpr int kBatch = 4;  // vectors a thread has in flight

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
    int b0;             // first image of the launch (two-launch form)
    int Cs, slices;     // channels per slice, slices (cluster form)
    int iters;          // pixels per thread (cluster form)
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

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Joined {
    double mean, m2;
};

// Joins `count` parts of one group, part i of (mean, M2) and weight get(i, c):
// the warp's lanes take the parts in turn.  In 64 bits: there are few parts,
// and what is left of the 32-bit sums' rounding errors averages out over them.
template <typename Get>
__device__ __forceinline__ Joined warp_join(int count, int lane, const Get &get)
{
    double n = 0., sum = 0.;
#pragma unroll 4
    for (int i = lane; i < count; i += 32) {
        float c;
        const float2 p = get(i, c);
        n += c;
        sum += static_cast<double>(c) * p.x;
    }
    n = warp_sum(n);
    const double mean = warp_sum(sum) / n;
    double m2 = 0.;
#pragma unroll 4
    for (int i = lane; i < count; i += 32) {
        float c;
        const float2 p = get(i, c);
        const double d = p.x - mean;
        m2 += c * d * d + p.y;
    }
    return Joined{mean, warp_sum(m2)};
}

// What the normalisation needs of a group: 1/std, and the mean as a float and
// the float's rounding error (which goes into the bias).
struct Coef {
    float mu, mu_low, rstd;
};
__device__ __forceinline__ Coef make_coef(const Joined &j, double n, float eps)
{
    Coef c;
    c.mu = static_cast<float>(j.mean);
    c.mu_low = static_cast<float>(j.mean - c.mu);
    c.rstd = static_cast<float>(1. / sqrt(j.m2 / n + eps));
    return c;
}

// y = (x - mu) * sc + be of V channels from c on; g0 the slice's first channel.
template <int V> struct Affine {
    float mu[V], sc[V], be[V];
    __device__ __forceinline__ Affine(const NormArgs &a, const Coef *coef, int c0, int c)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Coef k = coef[(c + i) / a.cg];
            const float gamma = a.gamma ? a.gamma[c0 + c + i] : 1.f;
            mu[i] = k.mu;
            sc[i] = k.rstd * gamma;
            be[i] = (a.beta ? a.beta[c0 + c + i] : 0.f) - k.mu_low * sc[i];
        }
    }
    template <typename T>
    __device__ __forceinline__ void apply(const NormArgs &a, const Vec<T, V> &x, const Vec<T, V> *r,
                                          float (&y)[V]) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            y[i] = fmaf(to_f(x.e[i]) - mu[i], sc[i], be[i]);
        if (r) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                y[i] += to_f(r->e[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            y[i] = activate(y[i], a.act);
    }
};

// Statistics of one chunk of pixels of one image: part[b][chunk][g].
template <typename T, int V> __global__ void __launch_bounds__(kBlock) norm_stats_kernel(NormArgs a)
{
    extern __shared__ float2 buf[];  // [lanes][C] (mean, M2) of each pixel lane and channel
    griddep_wait();
    const int b = a.b0 + blockIdx.y;
    const int p0 = blockIdx.x * a.chunk, p1 = min(a.HW, p0 + a.chunk);
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(b) * a.HW * a.C;
    const int pl = threadIdx.x / a.nv;
    if (pl < a.lanes) {
        for (int cv = threadIdx.x - pl * a.nv; cv < a.nv; cv += kBlock) {
            Running<V> st;
            const T *xc = x + cv * V;
            for (int p = p0 + pl; p < p1; p += kBatch * a.lanes) {
                Vec<T, V> v[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (p + j * a.lanes < p1)
                        v[j] = load_vec<T, V>(xc + static_cast<size_t>(p + j * a.lanes) * a.C);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (p + j * a.lanes < p1) {
                        float f[V];
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            f[i] = to_f(v[j].e[i]);
                        st.add(f);
                    }
                }
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
        const Joined r = warp_join(a.lanes * a.cg, lane, [&](int i, float &c) {
            const int l = i / a.cg;
            c = static_cast<float>((px - l + a.lanes - 1) / a.lanes);  // pixels of lane l
            return buf[l * a.C + g * a.cg + (i - l * a.cg)];
        });
        if (lane == 0)
            a.part[(static_cast<size_t>(b) * a.chunks + blockIdx.x) * a.G + g] =
                make_float2(static_cast<float>(r.mean), static_cast<float>(r.m2));
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
    extern __shared__ Coef coef[];  // [G]
    griddep_wait();
    const int b = a.b0 + blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int g = warp; g < a.G; g += kBlock / 32) {
        const float2 *part = a.part + static_cast<size_t>(b) * a.chunks * a.G + g;
        const Joined r = warp_join(a.chunks, lane, [&](int i, float &c) {
            c = static_cast<float>(min(a.HW, (i + 1) * a.chunk) - i * a.chunk) * a.cg;
            return part[static_cast<size_t>(i) * a.G];
        });
        if (lane == 0)
            coef[g] = make_coef(r, static_cast<double>(a.HW) * a.cg, a.eps);
    }
    if (OUT == kNormMx4 && b == 0 && blockIdx.x == 0)
        mx4_zero_row_padding(a.sf, static_cast<long long>(a.B) * a.HW, (a.C + 127) / 128,
                             threadIdx.x, kBlock);
    __syncthreads();
    const int p0 = blockIdx.x * a.chunk, p1 = min(a.HW, p0 + a.chunk);
    const size_t base = static_cast<size_t>(b) * a.HW * a.C;
    const int pl = threadIdx.x / a.nv;
    if (pl >= a.lanes)
        return;
    for (int cv = threadIdx.x - pl * a.nv; cv < a.nv; cv += kBlock) {
        const Affine<V> f(a, coef, 0, cv * V);
        const T *x = static_cast<const T *>(a.x) + base + cv * V;
        const T *r = a.r ? static_cast<const T *>(a.r) + base + cv * V : nullptr;
        for (int p = p0 + pl; p < p1; p += kBatch * a.lanes) {
            Vec<T, V> v[kBatch], w[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int q = p + j * a.lanes;
                if (q < p1) {
                    v[j] = load_vec<T, V>(x + static_cast<size_t>(q) * a.C);
                    if (r)
                        w[j] = load_vec<T, V>(r + static_cast<size_t>(q) * a.C);
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int q = p + j * a.lanes;
                if (q < p1) {
                    float y[V];
                    f.apply(a, v[j], r ? &w[j] : nullptr, y);
                    emit<T, V, OUT>(a, b, q, cv * V, y);
                }
            }
        }
    }
}

// The cluster form: CTA `rank` of the cluster (image b, channel slice sl) holds
// the slice's channels of pixels [p0, p1).  A thread keeps its vectors in slots
// of its own (slot i of thread t at (i * threads + t) * 16 bytes), so the data
// itself needs no synchronisation.
template <typename T, int V, int OUT>
__global__ void __launch_bounds__(kBlock, 3) norm_cluster_kernel(NormArgs a)
{
    extern __shared__ uint4 dyn[];
    using Slot = Vec<T, V>;
    Slot *slots = reinterpret_cast<Slot *>(dyn);
    // behind the slots: the joined statistics of this CTA, and the coefficients
    const int groups = a.Cs / a.cg;
    float2 *buf = reinterpret_cast<float2 *>(
        reinterpret_cast<uint8_t *>(dyn) + static_cast<size_t>(a.iters) * kBlock * sizeof(Slot));
    const bool one = a.cg % V == 0;  // a vector lies within one group
    const int per = one ? 1 : V;     // partial results of a thread
    double2 *cta = reinterpret_cast<double2 *>(buf + kBlock * per);
    Coef *coef = reinterpret_cast<Coef *>(cta + groups);
    uint32_t ctas;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const uint32_t rank = cluster_ctarank();
    const int unit = blockIdx.x / ctas, b = unit / a.slices;
    const int c0 = (unit - b * a.slices) * a.Cs;
    const int share = (a.HW + ctas - 1) / ctas;
    const int p0 = min(a.HW, static_cast<int>(rank) * share), p1 = min(a.HW, p0 + share);
    const int pl = threadIdx.x / a.nv, cv = threadIdx.x - pl * a.nv;
    const size_t base = static_cast<size_t>(b) * a.HW * a.C + c0 + cv * V;
    const bool active = pl < a.lanes;

    griddep_wait();
    if (OUT == kNormMx4 && blockIdx.x == 0)
        mx4_zero_row_padding(a.sf, static_cast<long long>(a.B) * a.HW, (a.C + 127) / 128,
                             threadIdx.x, kBlock);
    // Load, keep, and sum about the first value.
    float k[V], s[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        k[i] = s[i] = q[i] = 0.f;
    const int mine = active && p0 + pl < p1 ? (p1 - p0 - pl + a.lanes - 1) / a.lanes : 0;
    {
        const T *x = static_cast<const T *>(a.x) + base + static_cast<size_t>(p0 + pl) * a.C;
        const size_t step = static_cast<size_t>(a.lanes) * a.C;
        for (int i0 = 0; i0 < mine; i0 += kBatch) {
            Slot v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i0 + j < mine)
                    v[j] = load_vec<T, V>(x + (i0 + j) * step);
            if (i0 == 0) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    k[i] = to_f(v[0].e[i]);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (i0 + j < mine) {
                    slots[(i0 + j) * kBlock + threadIdx.x] = v[j];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = to_f(v[j].e[i]) - k[i];
                        s[i] += d;
                        q[i] = fmaf(d, d, q[i]);
                    }
                }
            }
        }
    }
    // (mean, M2) of each channel, or of the thread's whole vector
    {
        const float inv = mine ? 1.f / static_cast<float>(mine) : 0.f;
        float mean = 0.f, m2 = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float ms = s[i] * inv;
            k[i] += ms;
            q[i] = fmaxf(fmaf(-ms, s[i], q[i]), 0.f);
            mean += k[i] - k[0];
        }
        if (one) {
            mean = k[0] + mean * (1.f / V);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = k[i] - mean;
                m2 += fmaf(d * d, static_cast<float>(mine), q[i]);
            }
            buf[threadIdx.x] = make_float2(mean, m2);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                buf[threadIdx.x * V + i] = make_float2(k[i], q[i]);
        }
    }
    __syncthreads();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int px = p1 - p0;
    const int width = one ? a.cg / V : a.cg, pitch = one ? a.nv : a.Cs;
    for (int g = warp; g < groups; g += kBlock / 32) {
        const Joined r = warp_join(a.lanes * width, lane, [&](int i, float &c) {
            const int l = i / width;
            c = px > l ? static_cast<float>((px - l + a.lanes - 1) / a.lanes * (one ? V : 1)) : 0.f;
            return c > 0.f ? buf[l * pitch + g * width + (i - l * width)] : make_float2(0.f, 0.f);
        });
        if (lane == 0) {
            if (ctas == 1)
                coef[g] = make_coef(r, static_cast<double>(a.HW) * a.cg, a.eps);
            else
                cta[g] = make_double2(px > 0 ? r.mean : 0., px > 0 ? r.m2 : 0.);
        }
    }
    if (ctas > 1) {
        cluster_sync_all();
        for (int g = threadIdx.x; g < groups; g += kBlock) {
            // every CTA joins the same parts in the same order
            const uint32_t at = smem_u32(cta + g);
            const double total = static_cast<double>(a.HW) * a.cg;
            double mean = 0., m2 = 0.;
            for (int pass = 0; pass < 2; ++pass) {
                for (uint32_t r = 0; r < ctas; ++r) {
                    double m, v;
                    asm volatile("ld.shared::cluster.v2.f64 {%0, %1}, [%2];"
                                 : "=d"(m), "=d"(v)
                                 : "r"(mapa_shared(at, r))
                                 : "memory");
                    const int q0 = min(a.HW, static_cast<int>(r) * share);
                    const double n = static_cast<double>(min(a.HW, q0 + share) - q0) * a.cg;
                    if (pass == 0)
                        mean += n * m;
                    else if (n > 0.)
                        m2 += v + n * (m - mean) * (m - mean);
                }
                if (pass == 0)
                    mean /= total;
            }
            coef[g] = make_coef(Joined{mean, m2}, total, a.eps);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    __syncthreads();
    if (active) {
        const Affine<V> f(a, coef, c0, cv * V);
        const T *r = a.r ? static_cast<const T *>(a.r) + base + static_cast<size_t>(p0 + pl) * a.C
                         : nullptr;
        const size_t step = static_cast<size_t>(a.lanes) * a.C;
        for (int i0 = 0; i0 < mine; i0 += kBatch) {
            Slot w[kBatch];
            if (r) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (i0 + j < mine)
                        w[j] = load_vec<T, V>(r + (i0 + j) * step);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (i0 + j < mine) {
                    float y[V];
                    f.apply(a, slots[(i0 + j) * kBlock + threadIdx.x], r ? &w[j] : nullptr, y);
                    emit<T, V, OUT>(a, b, p0 + pl + (i0 + j) * a.lanes, c0 + cv * V, y);
                }
            }
        }
    }
    __syncwarp();
    if (ctas > 1)  // no CTA leaves while another may still read its statistics
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- host side ---------------------------------------------------------------

// Channels per vector: the most that divide n, up to 16 bytes.
int vector_channels(int dtype, int n)
{
    int v = dtype == X1CB_F32 ? 4 : 8;
    while (n % v)
        v /= 2;
    return v;
}

// What either form needs to know of a call.
struct Plan {
    int V, nv, lanes;
    int chunks, chunk;                    // two-launch form
    int cluster, Cs, slices, iters, smem;  // cluster form (cluster = 0: two launches)
};

double norm_cost(double ctas, double smem, int segment, int cluster, int iters)
{
    // resident CTAs per SM by shared memory and threads
    const double fit = std::min(3.0, std::floor(227.0 * 1024 / (smem + 1024)));
    double t = std::ceil(ctas / (148 * fit)) * fit * (smem + 3000);  // bytes an SM handles
    t *= 1 + 0.15 * (3 - fit) + (segment < 128 ? 0.1 : 0.0) + (segment < 64 ? 0.4 : 0.0);
    return t + 2000 * (cluster > 1) + 500 * cluster;
}

Plan plan_norm(int dtype, int B, int HW, int C, int G, bool whole_blocks)
{
    Plan p{};
    const int elt = dtype == X1CB_F32 ? 4 : 2, cg = C / G;
    p.V = vector_channels(dtype, C);
    // Slices: multiples of a unit of whole groups, whole vectors and, for
    // outputs in blocks of 32 channels, whole blocks.
    long long unit = cg;
    while (unit % p.V || (whole_blocks && unit % 32))
        unit += cg;
    double best = 1e30;
    for (int n = 1; n * unit <= C; ++n) {
        if (C % (n * unit))
            continue;
        const int Cs = static_cast<int>(n * unit), nv = Cs / p.V;
        if (nv > kBlock)
            break;
        const int lanes = kBlock / nv;
        for (int k = 1; k <= 8; k *= 2) {
            if (k > 1 && HW < k * lanes)
                break;
            const int iters = ((HW + k - 1) / k + lanes - 1) / lanes;
            if (iters > kFold)
                continue;
            const int groups = Cs / cg;
            const long long smem = static_cast<long long>(iters) * kBlock * p.V * elt +
                                   kBlock * (cg % p.V ? p.V : 1) * 8 + groups * (16 + 12);
            if (smem > 220 * 1024)
                continue;
            const double ctas = static_cast<double>(B) * (C / Cs) * k;
            const double cost = norm_cost(ctas, smem, Cs * elt, k, iters);
            if (cost < best) {
                best = cost;
                p.cluster = k;
                p.Cs = Cs;
                p.slices = C / Cs;
                p.nv = nv;
                p.lanes = lanes;
                p.iters = iters;
                p.smem = static_cast<int>(smem);
            }
        }
    }
    if (p.cluster && static_cast<long long>(B) * p.slices * p.cluster <= INT_MAX)
        return p;
    p.cluster = 0;
    p.nv = C / p.V;
    p.lanes = std::max(1, kBlock / p.nv);
    // four blocks per SM at once, at least two batches a thread
    const long long want = std::max(1, 148 * 4 / B);
    const long long most = std::max(1, HW / (p.lanes * kBatch * 2));
    p.chunks = static_cast<int>(std::min(want, most));
    p.chunk = (HW + p.chunks - 1) / p.chunks;
    p.chunks = (HW + p.chunk - 1) / p.chunk;
    return p;
}

// Sets a kernel's shared-memory limit once per device.
struct OptIn {
    std::atomic<bool> done[64];
    int operator()(const void *kern)
    {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
            return X1CB_ERR_CUDA;
        if (!done[dev].load(std::memory_order_acquire)) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 225 * 1024) !=
                cudaSuccess)
                return X1CB_ERR_CUDA;
            done[dev].store(true, std::memory_order_release);
        }
        return X1CB_OK;
    }
};

int launch(const void *kern, dim3 grid, size_t smem, int cluster, cudaStream_t s, NormArgs &a)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kBlock, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    void *params[] = {&a};
    return cudaLaunchKernelExC(&cfg, kern, params) == cudaSuccess ? X1CB_OK : X1CB_ERR_CUDA;
}

template <typename T, int V, int OUT>
int run(const NormCall &c, const Plan &p, NormArgs a, cudaStream_t s)
{
    if (p.cluster) {
        static OptIn opt;
        const void *k = reinterpret_cast<const void *>(norm_cluster_kernel<T, V, OUT>);
        if (int e = opt(k))
            return e;
        return launch(k, dim3(c.B * p.slices * p.cluster), p.smem, p.cluster, s, a);
    }
    static OptIn opt_stats, opt_apply;
    const void *ks = reinterpret_cast<const void *>(norm_stats_kernel<T, V>);
    const void *ka = reinterpret_cast<const void *>(norm_apply_kernel<T, V, OUT>);
    if (int e = opt_stats(ks))
        return e;
    if (int e = opt_apply(ka))
        return e;
    // as many images at a time as L2 (126 MB) holds beside what is written
    const double image = static_cast<double>(c.HW) * c.C * sizeof(T);
    const int most = static_cast<int>(std::min(65535., std::max(1., 40e6 / image)));
    for (a.b0 = 0; a.b0 < c.B; a.b0 += most) {
        const dim3 grid(p.chunks, std::min(most, c.B - a.b0));
        if (int e = launch(ks, grid, static_cast<size_t>(p.lanes) * c.C * sizeof(float2), 1, s, a))
            return e;
        if (int e = launch(ka, grid, static_cast<size_t>(c.G) * sizeof(Coef), 1, s, a))
            return e;
    }
    return X1CB_OK;
}

template <typename T, int V>
int run_out(const NormCall &c, const Plan &p, const NormArgs &a, cudaStream_t s)
{
    if constexpr (V * sizeof(T) == 16) {
        if (c.out == kNormI8)
            return run<T, V, kNormI8>(c, p, a, s);
        if (c.out == kNormMx4)
            return run<T, V, kNormMx4>(c, p, a, s);
    }
    return run<T, V, kNormSame>(c, p, a, s);
}

template <typename T>
int run_v(const NormCall &c, const Plan &p, const NormArgs &a, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2)
        if (p.V == 8)
            return run_out<T, 8>(c, p, a, s);
    return p.V == 4   ? run_out<T, 4>(c, p, a, s)
           : p.V == 2 ? run_out<T, 2>(c, p, a, s)
                      : run_out<T, 1>(c, p, a, s);
}

}  // namespace

// The workspace does not depend on the output's form: the larger of the two.
size_t norm_workspace_floats(int dtype, int B, int HW, int C, int G)
{
    size_t n = 0;
    for (int whole = 0; whole <= (C % 32 == 0 ? 1 : 0); ++whole) {
        const Plan p = plan_norm(dtype, B, HW, C, G, whole != 0);
        if (!p.cluster)
            n = std::max(n, static_cast<size_t>(B) * p.chunks * G * 2);
    }
    return n;
}

int launch_norm(const NormCall &c, cudaStream_t s)
{
    const Plan p = plan_norm(c.dtype, c.B, c.HW, c.C, c.G, c.out != kNormSame);
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
    a.nv = p.nv;
    a.lanes = p.lanes;
    a.chunks = p.chunks;
    a.chunk = p.chunk;
    a.Cs = p.Cs;
    a.slices = p.slices;
    a.iters = p.iters;
    if (c.dtype == X1CB_F32)
        return run_v<float>(c, p, a, s);
    return c.dtype == X1CB_BF16 ? run_v<__nv_bfloat16>(c, p, a, s) : run_v<__half>(c, p, a, s);
}

}  // namespace x1cb
