// Group norm + shortcut Sum + activation, channels last, with floating-point,
// int8 NC/32HW32 or MX4 output.
//
// Statistics: a thread owns V neighbouring channels and walks down up to 64
// pixels.  Per channel it sums d = x - k and d^2 about a value k, which gives its
// mean and its sum of squares about the mean, M2 = sum d^2 - (sum d)^2/n.  k is the
// first value and, behind the first eighth of the pixels, the mean of those
// (norm_stats_kernel: behind the 8th and the 32nd).  k being the mean of m of the n
// values, n (mean - k)^2 <= (n/m) M2, so the subtraction costs at most a factor 8 of
// the relative rounding error, however far the data lies from zero or one value from
// the others (about the first alone, with that one of 64 pixels far off, the results
// were 8 times their tolerance away).  A block joins its threads' (n, mean, M2) about
// the mean R of one of them, S1 = sum n (mean - R) and S2 = sum M2 + n (mean - R)^2,
// and where R lies so far off that S2 - S1^2/n would lose more than four bits, once
// more about the mean found; parts of different blocks are joined in 64 bits.  All in
// a fixed order.
//
// Two forms.  Where an image (or a slice of its channels that holds whole
// groups) fits the shared memory of a cluster of up to eight CTAs, one launch
// reads it once, keeps it there, joins the statistics over the cluster and
// normalises from shared memory: x in, y out, nothing else.  Larger images take
// two launches, partial statistics per chunk of pixels into the workspace and
// the normalisation, over as many images at a time as stay in L2 between them (and
// one between the two that joins the chunks, where there are many).
//
// 256 x 28 x 28 x 512 of bfloat16 with a shortcut: 112 us, 5.5 TB/s, bound by memory
// (without one 74 us, 5.6 TB/s).  To int8 (128 images) 41 us and to MX4 92 us: two CTAs
// fit an SM and go through their phases much together, so that loading and rounding
// come one after the other (to MX4 40 us of bytes and 52 us of instructions; memory at
// 31 % of its peak, the SMs at 57 %).  SiLU adds 28 us of exponentials and divisions.
// Two launches: 1 x 2048 x 2048 x 256 1130 us, x
// read twice and y written at 5.7 TB/s.  1 x 7 x 7 x 2048: 3.8 us, latency.
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
constexpr int kFold = 64;  // pixels a thread's shifted sums run over at most
constexpr int kBatch = 4;  // vectors a thread has in flight

// What the normalisation needs of a group.
struct Coef {
    float mu, mu_low, rstd;  // the mean as a float and that float's rounding error
};

struct NormArgs {
    const void *x, *r;
    const float *gamma, *beta;
    void *y;
    uint8_t *sf;
    float2 *part;  // [B][chunks][G] (mean, M2)
    Coef *coef;    // [B][G], where a launch of its own joins the chunks (else NULL)
    float eps, q_mul;
    int act, B, HW, C, G, cg;
    int nv;             // vectors of V channels per pixel
    int lanes;          // pixels the block takes at a time (kBlock / nv, at least 1)
    int chunks, chunk;  // chunks per image, pixels per chunk
    int b0;             // first image of the launch (two-launch form)
    int Cs, slices;     // channels per slice, slices (cluster form)
    int iters;          // pixels per thread (cluster form)
    int stage_r;        // the shortcut goes through shared memory too
    int log_wl;         // log2 of the threads of a group that share its pixel lanes out
    double inv_count;   // 1 / (HW * cg), the values of a group of an image
    uint32_t div_nv, div_lanes;  // ceil(2^32 / nv), ceil(2^32 / lanes), see quotient()
};

// n / d for n * d < 2^32, from m = ceil(2^32 / d) (d > 1; d = 1 is stored as 0).
__device__ __forceinline__ int quotient(int n, uint32_t m)
{
    return m ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), m)) : n;
}

// Shifted sums of a thread's V channels over n pixels.
template <int V> struct Sums {
    F2 k[kPairs<V>], s[kPairs<V>], q[kPairs<V>];  // -first value, sum d, sum d^2

    template <typename T> __device__ __forceinline__ void start(const Vec<T, V> &v)
    {
        unpack<T, V>(v, k);
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i) {
            const float2 t = un2(k[i]);
            k[i] = f2(-t.x, -t.y);
            s[i] = q[i] = f2(0.f, 0.f);
        }
    }
    template <typename T> __device__ __forceinline__ void add(const Vec<T, V> &v)
    {
        F2 f[kPairs<V>];
        unpack<T, V>(v, f);
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i) {
            const F2 d = add2(f[i], k[i]);
            s[i] = add2(s[i], d);
            q[i] = fma2(d, d, q[i]);
        }
    }
    // Moves k to the mean of the n values so far: by d to k', sum (x - k') = s - n d
    // and sum (x - k')^2 = q - d (s + (s - n d)).
    __device__ __forceinline__ void move(float n, float inv)
    {
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i) {
            const F2 m = fma2(s[i], f2(-inv, -inv), k[i]);  // -k'
            const F2 d = add2(m, neg2(k[i]));              // -d, as m was rounded
            const F2 t = fma2(d, f2(n, n), s[i]);
            q[i] = fma2(d, add2(s[i], t), q[i]);
            s[i] = t;
            k[i] = m;
        }
    }
    // Writes (mean, M2) of each channel, or of all V together (one), to out.
    __device__ __forceinline__ void write(int n, bool one, float2 *out) const
    {
        const float inv = n ? 1.f / static_cast<float>(n) : 0.f;
        float mean[V], m2[V], off = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 kk = un2(k[i / 2]), ss = un2(s[i / 2]), qq = un2(q[i / 2]);
            const float si = i % 2 ? ss.y : ss.x, qi = i % 2 ? qq.y : qq.x;
            const float ms = si * inv;
            mean[i] = (i % 2 ? -kk.y : -kk.x) + ms;
            m2[i] = fmaxf(fmaf(-ms, si, qi), 0.f);
            off += mean[i] - mean[0];
        }
        if (!one) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                out[i] = make_float2(mean[i], m2[i]);
            return;
        }
        const float all = fmaf(off, 1.f / V, mean[0]);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = mean[i] - all;
            sum += fmaf(d * d, static_cast<float>(n), m2[i]);
        }
        out[0] = make_float2(all, sum);
    }
};

// Sum over the `width` lanes (a power of two) around each lane.
template <typename T> __device__ __forceinline__ T lanes_sum(T v, int width)
{
    for (int o = width >> 1; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Joined {
    double mean, m2;
};

// What a group's lanes join (see join_threads).
struct Entries {
    const float2 *buf;
    int filled, base, more, pitch, width, each, w, log_wl;

    // S1 = sum n (mean - at) and S2 = sum M2 + n (mean - at)^2, at = ref + shift.
    __device__ __forceinline__ float2 sums(float ref, float shift) const
    {
        const int lane = threadIdx.x & (w - 1), wl = 1 << log_wl, wv = w >> log_wl;
        float s1 = 0.f, s2 = 0.f;
        for (int l = lane & (wl - 1); l < filled; l += wl) {
            const float n = static_cast<float>((base + (l < more)) * each);
            float t = 0.f, u = 0.f, m = 0.f;
            const float2 *p = buf + l * pitch;
#pragma unroll 2
            for (int v = lane >> log_wl; v < width; v += wv) {
                const float2 e = p[v];
                const float d = e.x - ref - shift;
                t += d;
                u = fmaf(d, d, u);
                m += e.y;
            }
            s1 = fmaf(n, t, s1);
            s2 += fmaf(n, u, m);
        }
        return make_float2(lanes_sum(s1, w), lanes_sum(s2, w));
    }
};
// (seldom called: inlined it costs norm_cluster_kernel registers, 256 x 28 x 28 x 512 to
// MX4 96 us against 90)
__device__ __noinline__ float2 sums_about(Entries e, float ref, float shift)
{
    return e.sums(ref, shift);
}

// Joins the (mean, M2) that a block's threads wrote for one group: entry v of
// pixel lane l at buf[l * pitch + v], v < width, each standing for n * each
// values, n = base (+ 1 for the first `more` lanes).  The w lanes that share the
// group take the pixel lanes in turn, and where those are fewer (many channels) a
// pixel lane's entries; whole warps call it.  The sums are taken about the first
// entry's mean.  Where that lies so far off that S2 - S1^2/n would lose more than
// four bits (of 8191 entries, the first 1000 spreads away: 1e-3 of the variance), the
// group goes through them once more about the mean it found.  (Always twice:
// 256 x 28 x 28 x 512 with a shortcut 119 us, in 64 bits 114, so 110.)
template <bool kInline>
__device__ __forceinline__ Joined join_threads(const float2 *buf, int px, int base, int more,
                                               int lanes, int pitch, int width, int each, int w,
                                               int log_wl, bool active)
{
    const Entries e{buf, !active ? 0 : base ? lanes : more, base, more, pitch, width, each, w, log_wl};
    const float ref = active ? buf[0].x : 0.f;
    const float count = static_cast<float>(px) * static_cast<float>(width * each);
    const float2 s = e.sums(ref, 0.f);
    const float off = __fdividef(s.x, count), rest = fmaf(-s.x, off, s.y);
    Joined r{static_cast<double>(ref) + off, fmaxf(rest, 0.f)};
    const bool again = rest < 0.0625f * s.y;
    if (__builtin_expect(__any_sync(0xffffffffu, again), 0)) {
        const float2 t = kInline ? e.sums(ref, off) : sums_about(e, ref, off);
        const float by = __fdividef(t.x, count);
        if (again)
            r = Joined{static_cast<double>(ref) + off + by, fmaxf(fmaf(-t.x, by, t.y), 0.f)};
    }
    return r;
}

// Lanes per group so that a block's threads cover all groups at once where they can.
__host__ __device__ __forceinline__ int join_width(int groups)
{
    int w = 32;
    while (w > 1 && w * groups > kBlock)
        w >>= 1;
    return w;
}

__device__ __forceinline__ Coef make_coef(const Joined &j, double inv_count, float eps)
{
    Coef c;
    c.mu = static_cast<float>(j.mean);
    c.mu_low = static_cast<float>(j.mean - c.mu);
    // 1/sqrt(v): a 32-bit estimate and one Newton step in 64 bits
    const double v = j.m2 * inv_count + eps;
    double r = rsqrtf(static_cast<float>(v));
    if (v > 1e-30 && v < 1e30)
        r = r * (1.5 - 0.5 * v * r * r);
    else
        r = 1. / sqrt(v);
    c.rstd = static_cast<float>(r);
    return c;
}

// gamma and beta of V channels from c on, loaded ahead of the statistics.
template <int V> struct Params {
    float gamma[V], beta[V];
    __device__ __forceinline__ Params(const NormArgs &a, int c)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            gamma[i] = a.gamma ? __ldg(a.gamma + c + i) : 1.f;
            beta[i] = a.beta ? __ldg(a.beta + c + i) : 0.f;
        }
    }
};

// The normalisation of V channels: y = (x - mu) * sc + be, with what the float mu
// lacks of the mean in be.  (One multiply-add, x * sc + (beta - mu * sc), would
// leave the rounding of mu * sc in y: 0.02 where a constant image of 1000 has to
// come out as beta.)
template <typename T, int V> struct Affine {
    F2 mu[kPairs<V>], sc[kPairs<V>], be[kPairs<V>];
    // p: gamma and beta of the channels; cs: the first of them, counted from the
    // slice's first group
    __device__ __forceinline__ Affine(const NormArgs &a, const Coef *coef, const Params<V> &p, int cs,
                                      bool one)
    {
        float m[V + 1], s[V + 1], b[V + 1];
        m[V] = s[V] = b[V] = 0.f;
        int g = cs / a.cg, left = a.cg - (cs - g * a.cg);
        Coef k = coef[g];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!one && i > 0 && --left == 0) {
                k = coef[++g];
                left = a.cg;
            }
            s[i] = k.rstd * p.gamma[i];
            const float beta = p.beta[i];
            m[i] = -k.mu;
            b[i] = fmaf(-k.mu_low, s[i], beta);
        }
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i) {
            mu[i] = f2(m[2 * i], m[2 * i + 1]);
            sc[i] = f2(s[2 * i], s[2 * i + 1]);
            be[i] = f2(b[2 * i], b[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void apply(const Vec<T, V> &x, const Vec<T, V> *r,
                                          F2 (&y)[kPairs<V>]) const
    {
        unpack<T, V>(x, y);
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i)
            y[i] = fma2(add2(y[i], mu[i]), sc[i], be[i]);
        if (r) {
            F2 f[kPairs<V>];
            unpack<T, V>(*r, f);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i)
                y[i] = add2(y[i], f[i]);
        }
    }
};

// Statistics of one chunk of pixels of one image: part[b][chunk][g].
template <typename T, int V> __global__ void __launch_bounds__(kBlock) norm_stats_kernel(NormArgs a)
{
    extern __shared__ float2 buf[];  // (mean, M2) by pixel lane and vector or channel
    griddep_wait();
    const int b = a.b0 + blockIdx.y;
    const int p0 = blockIdx.x * a.chunk, px = min(a.HW - p0, a.chunk);
    const bool one = a.cg % V == 0;
    const int each = one ? V : 1, width = a.cg / each, pitch = a.C / each;
    const int pl = quotient(threadIdx.x, a.div_nv);
    const int per_lane = quotient(px, a.div_lanes), more = px - per_lane * a.lanes;
    if (pl < a.lanes) {
        const int mine = per_lane + (pl < more);
        const size_t step = static_cast<size_t>(a.lanes) * a.C;
        for (int cv = threadIdx.x - pl * a.nv; cv < a.nv && mine > 0; cv += kBlock) {
            const T *x = static_cast<const T *>(a.x) +
                         (static_cast<size_t>(b) * a.HW + p0 + pl) * a.C + cv * V;
            constexpr int kDeep = 2 * kBatch;
            Sums<V> st;
            Vec<T, V> v[kDeep];
            for (int i0 = 0; i0 < mine; i0 += kDeep) {
#pragma unroll
                for (int j = 0; j < kDeep; ++j)
                    if (i0 + j < mine)
                        v[j] = load_vec<T, V>(x + j * step);
                x += kDeep * step;
                if (i0 == 0)
                    st.start(v[0]);
#pragma unroll
                for (int j = 0; j < kDeep; ++j)
                    if (i0 + j < mine)
                        st.add(v[j]);
                if ((i0 == 0 || i0 == 24) && mine > i0 + kDeep)
                    st.move(i0 + kDeep, i0 ? 1.f / 32 : 1.f / 8);
            }
            st.write(mine, one, buf + (pl * a.nv + cv) * (V / each));
        }
    }
    __syncthreads();
    const int w = join_width(a.G);
    for (int g0 = 0; g0 < a.G; g0 += kBlock / w) {
        const int g = g0 + threadIdx.x / w;
        const Joined r = join_threads<true>(buf + g * width, px, per_lane, more, a.lanes, pitch,
                                      width, each, w, a.log_wl, g < a.G);
        if (g < a.G && threadIdx.x % w == 0)
            a.part[(static_cast<size_t>(b) * a.chunks + blockIdx.x) * a.G + g] =
                make_float2(static_cast<float>(r.mean), static_cast<float>(r.m2));
    }
}

// Joins the chunks' statistics in a launch of its own, a block per group of an
// image, where there are so many of them that each block of the normalisation
// should not repeat it.  In 64 bits and about the first chunk's mean R (equal means
// join to that mean exactly): S1 = sum n (mean - R), S2 = sum M2 + n (mean - R)^2.
__global__ void __launch_bounds__(kBlock) norm_join_kernel(NormArgs a)
{
    __shared__ double sums[2][kBlock / 32];
    griddep_wait();
    const int g = blockIdx.x, b = a.b0 + blockIdx.y;
    const float2 *part = a.part + static_cast<size_t>(b) * a.chunks * a.G + g;
    const double last = static_cast<double>(a.HW - (a.chunks - 1) * a.chunk) * a.cg;
    const double whole = static_cast<double>(a.chunk) * a.cg;
    const double ref = part[0].x;
    double s1 = 0., s2 = 0.;
#pragma unroll 4
    for (int j = threadIdx.x; j < a.chunks; j += kBlock) {
        const float2 p = part[static_cast<size_t>(j) * a.G];
        const double n = j == a.chunks - 1 ? last : whole, e = p.x - ref;
        s1 += n * e;
        s2 += p.y + n * e * e;
    }
    s1 = lanes_sum(s1, 32);
    s2 = lanes_sum(s2, 32);
    if (threadIdx.x % 32 == 0) {
        sums[0][threadIdx.x / 32] = s1;
        sums[1][threadIdx.x / 32] = s2;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        s1 = s2 = 0.;
        for (int i = 0; i < kBlock / 32; ++i) {
            s1 += sums[0][i];
            s2 += sums[1][i];
        }
        const double off = s1 * a.inv_count, m2 = s2 - s1 * off;
        a.coef[static_cast<size_t>(b) * a.G + g] =
            make_coef(Joined{ref + off, m2 < 0. ? 0. : m2}, a.inv_count, a.eps);  // (NaN stays)
    }
}

// Where a thread's outputs go: channels c .. c + V - 1 of pixel p of image b,
// and of every `lanes`-th pixel after it.
template <typename T, int V, int OUT, bool kStream = false> struct Out {
    uint8_t *to;       // the next output, code or int8
    size_t step;       // bytes to the one after it
    uint8_t *scales;   // MX4: the scale array from this block of channels on
    uint32_t row, kt;  // MX4: the pixel, counted over the batch; scale tiles per row
    int pad;           // MX4: bytes of padding behind the row's last block

    __device__ __forceinline__ Out(const NormArgs &a, int b, int p, int c)
    {
        const size_t at = static_cast<size_t>(b) * a.HW + p;
        to = static_cast<uint8_t *>(a.y);
        if constexpr (OUT == kNormSame) {
            to += (at * a.C + c) * sizeof(T);
            step = static_cast<size_t>(a.lanes) * a.C * sizeof(T);
        } else if constexpr (OUT == kNormI8) {
            to += ((static_cast<size_t>(b) * (a.C / 32) + c / 32) * a.HW + p) * 32 + c % 32;
            step = static_cast<size_t>(a.lanes) * 32;
        } else {
            to += (at * a.C + c) / 2;
            step = static_cast<size_t>(a.lanes) * (a.C / 2);
            const int blk = c / 32;
            kt = (a.C + 127) / 128;
            scales = a.sf + static_cast<size_t>(blk >> 2) * 512 + (blk & 3);
            row = static_cast<uint32_t>(at);
            pad = blk == a.C / 32 - 1 ? 3 - (blk & 3) : 0;
        }
    }
    // MX4, the next kBatch pixels (n of them the thread's) at once, so that their
    // shuffles are in flight together (256 x 28 x 28 x 512: 95 us one by one, 88 so):
    // thread j of a block's threads stores the scale of pixel j.  Whole warps call it.
    template <typename Value>
    __device__ __forceinline__ void put_batch(const NormArgs &a, int n, const Value &value)
    {
        if constexpr (OUT == kNormMx4) {
            constexpr int L = 32 / V;
            static_assert(kBatch <= L, "a thread per pixel");
            float y[kBatch][V];
            uint32_t m[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                F2 f[kPairs<V>];
                value(j, f);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 t = un2(f[i]);
                    y[j][2 * i] = t.x;
                    y[j][2 * i + 1] = t.y;
                }
                activate(y[j], a.act);
                m[j] = amax_bits(y[j]);
            }
#pragma unroll
            for (int o = 1; o < L; o <<= 1)
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
            const int lane = threadIdx.x & (L - 1);
            uint32_t mine = 0;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const uint32_t e = mx4_exponent(m[j]);
                const float inv = mx4_inverse_scale(e);
                mine = lane == j ? e : mine;
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 t = un2(mul2(f2(y[j][i], y[j][i + 1]), f2(inv, inv)));
                    y[j][i] = t.x;
                    y[j][i + 1] = t.y;
                }
                if (j < n) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint32_t *>(to) = e == kMx4Bad ? 0u : e2m1x8(y[j]);
                    else
                        *reinterpret_cast<uint16_t *>(to) =
                            e == kMx4Bad ? uint16_t{0} : e2m1x4(y[j]);
                }
                to += step;
            }
            if (lane < min(n, kBatch)) {
                uint8_t *d = scales + mx4_scale_row(row + lane * a.lanes, kt);
                *d = mx4_scale_byte(mine);
                for (int k = 1; k <= pad; ++k)
                    d[k] = 0;
            }
            row += kBatch * a.lanes;
        }
    }
    // MX4: whole warps call it, `valid` says whether this thread has a pixel (a
    // block's threads share one); the others call it with a pixel only.
    static constexpr bool kWhole = OUT == kNormMx4;
    __device__ __forceinline__ void put(const NormArgs &a, const F2 (&f)[kPairs<V>], bool valid)
    {
        if constexpr (OUT == kNormSame) {
            const Vec<T, V> v = finish<T, V>(f, a.act);
            if constexpr (kStream && sizeof(v) == 16)
                __stcs(reinterpret_cast<uint4 *>(to), *reinterpret_cast<const uint4 *>(&v));
            else
                store_vec<T, V>(reinterpret_cast<T *>(to), v);
        } else {
            float y[V];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 t = un2(f[i]);
                y[2 * i] = t.x;
                y[2 * i + 1] = t.y;
            }
            activate(y, a.act);
            if constexpr (OUT == kNormI8) {
                // rounded to an integer (NaN: 0), then packed with saturation
                uint32_t w[V / 4];
#pragma unroll
                for (int i = 0; i < V / 4; ++i) {
                    int n[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        n[j] = __float2int_rn(y[4 * i + j] * a.q_mul);
                    uint32_t hi;
                    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;"
                        : "=r"(hi)
                        : "r"(n[3]), "r"(n[2]), "r"(0));
                    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;"
                        : "=r"(w[i])
                        : "r"(n[1]), "r"(n[0]), "r"(hi));
                }
                if constexpr (V == 8)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
                else
                    *reinterpret_cast<uint32_t *>(to) = w[0];
            } else {
                // The 32 / V neighbouring threads that hold a block agree on its scale.
                // (With a mask of its own for each block, the shuffles of a warp run
                // one after the other: 109 us for 256 x 28 x 28 x 512, 95 with whole
                // warps.)
                constexpr int L = 32 / V;
                uint32_t m = amax_bits(y);
#pragma unroll
                for (int o = 1; o < L; o <<= 1)
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                const uint32_t e = mx4_exponent(m);
                const float inv = mx4_inverse_scale(e);
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const float2 t = un2(mul2(f2(y[i], y[i + 1]), f2(inv, inv)));
                    y[i] = t.x;
                    y[i + 1] = t.y;
                }
                if (valid) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint32_t *>(to) = e == kMx4Bad ? 0u : e2m1x8(y);
                    else
                        *reinterpret_cast<uint16_t *>(to) = e == kMx4Bad ? uint16_t{0} : e2m1x4(y);
                    if ((threadIdx.x & (L - 1)) == 0) {
                        uint8_t *d = scales + mx4_scale_row(row, kt);
                        *d = mx4_scale_byte(e);
                        for (int k = 1; k <= pad; ++k)
                            d[k] = 0;
                    }
                }
                row += a.lanes;
            }
        }
        to += step;
    }
};

template <typename T, int V, int OUT>
__global__ void __launch_bounds__(kBlock) norm_apply_kernel(NormArgs a)
{
    extern __shared__ Coef coef[];  // [G]
    griddep_wait();
    // The last chunks first: they are the ones that the statistics left in L2.
    const int b = a.b0 + gridDim.y - 1 - blockIdx.y;
    const int p0 = (gridDim.x - 1 - blockIdx.x) * a.chunk, px = min(a.HW - p0, a.chunk);
    if (a.coef) {
        for (int g = threadIdx.x; g < a.G; g += kBlock)
            coef[g] = a.coef[static_cast<size_t>(b) * a.G + g];
    } else {
        // Join the chunks, in 64 bits and about the first one's mean (so that equal
        // means join to that mean exactly).
        const int w = join_width(a.G);
        const double last = static_cast<double>(a.HW - (a.chunks - 1) * a.chunk) * a.cg;
        const double whole = static_cast<double>(a.chunk) * a.cg;
        for (int g0 = 0; g0 < a.G; g0 += kBlock / w) {
            const int g = g0 + threadIdx.x / w, lane = threadIdx.x & (w - 1);
            const float2 *part = a.part + static_cast<size_t>(b) * a.chunks * a.G + g;
            constexpr int kKeep = 8;  // parts a lane holds from the first pass to the second
            float2 kept[kKeep];
            double sum = 0., m2 = 0.;
            const int mine = g < a.G && lane < a.chunks ? (a.chunks - lane + w - 1) / w : 0;
            const double ref = g < a.G ? part[0].x : 0.;
#pragma unroll
            for (int j = 0; j < kKeep; ++j)
                if (j < mine)
                    kept[j] = part[static_cast<size_t>(lane + j * w) * a.G];
            const auto weight = [&](int j) { return lane + j * w == a.chunks - 1 ? last : whole; };
#pragma unroll
            for (int j = 0; j < kKeep; ++j)
                if (j < mine)
                    sum += weight(j) * (kept[j].x - ref);
#pragma unroll 4
            for (int j = kKeep; j < mine; ++j)
                sum += weight(j) * (part[static_cast<size_t>(lane + j * w) * a.G].x - ref);
            const double mean = ref + lanes_sum(sum, w) * a.inv_count;
#pragma unroll
            for (int j = 0; j < kKeep; ++j)
                if (j < mine)
                    m2 += kept[j].y + weight(j) * (kept[j].x - mean) * (kept[j].x - mean);
#pragma unroll 4
            for (int j = kKeep; j < mine; ++j) {
                const float2 p = part[static_cast<size_t>(lane + j * w) * a.G];
                m2 += p.y + weight(j) * (p.x - mean) * (p.x - mean);
            }
            m2 = lanes_sum(m2, w);
            if (g < a.G && lane == 0)
                coef[g] = make_coef(Joined{mean, m2}, a.inv_count, a.eps);
        }
    }
    if (OUT == kNormMx4 && b == 0 && blockIdx.x == 0)
        mx4_zero_row_padding(a.sf, static_cast<long long>(a.B) * a.HW, (a.C + 127) / 128,
                             threadIdx.x, kBlock);
    __syncthreads();
    const int pl = quotient(threadIdx.x, a.div_nv);
    const int per_lane = quotient(px, a.div_lanes), more = px - per_lane * a.lanes;
    const int mine = pl < a.lanes ? per_lane + (pl < more) : 0;
    // vectors in flight (64 x 224 x 224 x 64 of bfloat16: 276 us with four, 252 with eight)
    constexpr int kDeep = 2 * kBatch;
    using O = Out<T, V, OUT, true>;  // (results do not push the input out of L2)
    const int most = O::kWhole ? per_lane + (more > 0) : mine;  // of the block
    const size_t step = static_cast<size_t>(a.lanes) * a.C;
    // (C is a multiple of 32 for MX4, and with it the threads of a pixel: a warp's
    // threads leave this loop together but for those without a pixel)
    for (int cv0 = 0; cv0 < a.nv; cv0 += kBlock) {
        const int cv = cv0 + threadIdx.x - pl * a.nv;
        const bool active = mine > 0 && cv < a.nv;
        if (!O::kWhole && !active)
            continue;
        const int c = active ? cv * V : 0, n = active ? mine : 0;
        const Affine<T, V> f(a, coef, Params<V>(a, c), c, a.cg % V == 0);
        const size_t base = (static_cast<size_t>(b) * a.HW + p0 + (active ? pl : 0)) * a.C + c;
        const T *x = static_cast<const T *>(a.x) + base;
        const T *r = a.r ? static_cast<const T *>(a.r) + base : nullptr;
        O out(a, b, p0 + (active ? pl : 0), c);
        for (int i0 = 0; i0 < most; i0 += kDeep) {
            Vec<T, V> v[kDeep], rv[kDeep];
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                if (i0 + j < n) {
                    v[j] = load_vec<T, V>(x + j * step);
                    if (r)
                        rv[j] = load_vec<T, V>(r + j * step);
                }
            }
            x += kDeep * step;
            if (r)
                r += kDeep * step;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                if (O::kWhole ? i0 + j < most : i0 + j < n) {
                    F2 y[kPairs<V>];
                    f.apply(v[j], r ? &rv[j] : nullptr, y);
                    out.put(a, y, i0 + j < n);
                }
            }
        }
    }
}

// The cluster form: CTA `rank` of the cluster (image b, channel slice) holds the
// slice's channels of pixels p0 .. p0 + px - 1.  A thread keeps its vectors in
// slots of its own (slot i of thread t at (i * threads + t)), so the data itself
// needs no synchronisation.
template <typename T, int V, int OUT>
__global__ void __launch_bounds__(kBlock, 3) norm_cluster_kernel(NormArgs a)
{
    extern __shared__ uint4 dyn[];
    using Slot = Vec<T, V>;
    const bool one = a.cg % V == 0;  // a vector lies within one group
    const int each = one ? V : 1, per = V / each;
    const int groups = a.Cs / a.cg;
    // slots of x (and of the shortcut), the threads' statistics, the CTA's, the coefficients
    Slot *slots = reinterpret_cast<Slot *>(dyn) + threadIdx.x;
    float2 *buf = reinterpret_cast<float2 *>(reinterpret_cast<Slot *>(dyn) +
                                             (a.stage_r ? 2 : 1) * a.iters * kBlock);
    double2 *cta = reinterpret_cast<double2 *>(buf + kBlock * per);
    Coef *coef = reinterpret_cast<Coef *>(cta + groups);
    uint32_t ctas;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const uint32_t rank = cluster_ctarank();
    uint32_t unit;
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(unit));
    const int b = unit / static_cast<uint32_t>(a.slices);
    const int share = (a.HW + ctas - 1) / ctas;
    const int p0 = static_cast<int>(rank) * share, px = max(0, min(a.HW - p0, share));
    const int pl = quotient(threadIdx.x, a.div_nv), cv = threadIdx.x - pl * a.nv;
    const int per_lane = quotient(px, a.div_lanes), more = px - per_lane * a.lanes;
    const int c = (static_cast<int>(unit) - b * a.slices) * a.Cs + cv * V;
    const int mine = pl < a.lanes ? per_lane + (pl < more) : 0;
    const size_t base = (static_cast<size_t>(b) * a.HW + p0 + pl) * a.C + c;
    const size_t step = static_cast<size_t>(a.lanes) * a.C;
    const T *r = a.r ? static_cast<const T *>(a.r) + base : nullptr;

    griddep_wait();
    if (OUT == kNormMx4 && blockIdx.x == 0)
        mx4_zero_row_padding(a.sf, static_cast<long long>(a.B) * a.HW, (a.C + 127) / 128,
                             threadIdx.x, kBlock);
    // Every copy of the thread is in flight before the first is used: x in two
    // groups, the pixels before k moves and those behind, then the shortcut.  (k moved
    // behind the 4th and the 16th pixel instead: 117 us for 112 with a shortcut.)
    const int first = (mine + 7) / 8;
    {
        const T *x = static_cast<const T *>(a.x) + base;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int end = h ? mine : first;
            for (int i = h ? first : 0; i < end; ++i, x += step) {
                if constexpr (sizeof(Slot) >= 4)
                    copy_async<sizeof(Slot)>(slots + i * kBlock, x);
                else
                    slots[i * kBlock] = load_vec<T, V>(x);
            }
            copy_commit();
        }
        if (a.stage_r) {
            const T *rr = r;
            for (int i = 0; i < mine; ++i, rr += step) {
                if constexpr (sizeof(Slot) >= 4)
                    copy_async<sizeof(Slot)>(slots + (a.iters + i) * kBlock, rr);
                else
                    slots[(a.iters + i) * kBlock] = load_vec<T, V>(rr);
            }
        }
        copy_commit();
    }
    {
        Sums<V> st;
        copy_wait<2>();
        if (mine > 0) {
            st.start(slots[0]);
            for (int i = 1; i < first; ++i)
                st.add(slots[i * kBlock]);
            if (first > 1)
                st.move(first, __fdividef(1.f, first));
        }
        copy_wait<1>();
        if (mine > 0) {
            for (int i = first; i < mine; ++i)
                st.add(slots[i * kBlock]);
            st.write(mine, one, buf + threadIdx.x * per);
        }
    }
    const bool active = mine > 0;  // (threads without a pixel: any channel of the slice)
    const int cs = active ? cv * V : 0, c1 = active ? c : c - cv * V;
    const Params<V> params(a, c1);
    __syncthreads();
    {
        const int w = join_width(groups), width = a.cg / each, pitch = a.Cs / each;
        for (int g0 = 0; g0 < groups; g0 += kBlock / w) {
            const int g = g0 + threadIdx.x / w;
            const Joined t = join_threads<false>(buf + g * width, px, per_lane, more, a.lanes, pitch,
                                                 width, each, w, a.log_wl, g < groups && px > 0);
            if (g < groups && threadIdx.x % w == 0) {
                if (ctas == 1)
                    coef[g] = make_coef(t, a.inv_count, a.eps);
                else
                    cta[g] = px > 0 ? make_double2(t.mean, t.m2) : make_double2(0., 0.);
            }
        }
    }
    if (ctas > 1) {
        cluster_sync_all();
        // Every CTA joins the same parts in the same order: a lane per CTA.
        for (int g0 = 0; g0 < groups; g0 += kBlock / 8) {
            const int g = g0 + threadIdx.x / 8, q = threadIdx.x & 7;
            double m = 0., v = 0., n = 0.;
            if (g < groups && q < static_cast<int>(ctas)) {
                asm volatile("ld.shared::cluster.v2.f64 {%0, %1}, [%2];"
                             : "=d"(m), "=d"(v)
                             : "r"(mapa_shared(smem_u32(cta + g), q))
                             : "memory");
                n = static_cast<double>(max(0, min(a.HW - q * share, share))) * a.cg;
            }
            const double ref = __shfl_sync(0xffffffffu, m, 0, 8);  // (rank 0 has pixels)
            const double mean = ref + lanes_sum(n * (m - ref), 8) * a.inv_count;
            const double m2 = lanes_sum(n > 0. ? v + n * (m - mean) * (m - mean) : 0., 8);
            if (g < groups && q == 0)
                coef[g] = make_coef(Joined{mean, m2}, a.inv_count, a.eps);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    copy_wait<0>();
    __syncthreads();
    using O = Out<T, V, OUT>;
    const int most = O::kWhole ? per_lane + (more > 0) : mine;  // pixels of the CTA's first lane
    if (most > 0) {
        const Affine<T, V> f(a, coef, params, cs, one);
        O out(a, b, p0 + (active ? pl : 0), c1);
        if (O::kWhole && (a.stage_r || !r)) {
            // (slots past a thread's pixels hold nothing, and nothing of them is stored)
            const int second = r ? a.iters * kBlock : 0;
            for (int i0 = 0; i0 < most; i0 += kBatch)
                out.put_batch(a, mine - i0, [&](int j, F2(&y)[kPairs<V>]) {
                    const int i = min(i0 + j, a.iters - 1) * kBlock;
                    f.apply(slots[i], r ? &slots[second + i] : nullptr, y);
                });
        } else if (a.stage_r || !r) {
            const int second = r ? a.iters * kBlock : 0;
#pragma unroll 2
            for (int i = 0; i < most; ++i) {
                F2 y[kPairs<V>];
                f.apply(slots[i * kBlock], r ? &slots[second + i * kBlock] : nullptr, y);
                out.put(a, y, i < mine);
            }
        } else {
            for (int i0 = 0; i0 < most; i0 += kBatch, r += kBatch * step) {
                Slot rv[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    if (i0 + j < mine)
                        rv[j] = load_vec<T, V>(r + j * step);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    if (i0 + j < most) {
                        F2 y[kPairs<V>];
                        f.apply(slots[(i0 + j) * kBlock], &rv[j], y);
                        out.put(a, y, i0 + j < mine);
                    }
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
    int chunks, chunk, images;            // two-launch form: per image; images at a time
    int joined;                           // the chunks are joined in a launch of their own
    int cluster, Cs, slices, iters, smem;  // cluster form (cluster = 0: two launches)
    int stage_r;
};

constexpr long long kSmemMost = 220 * 1024;

// What a cluster-form plan costs, in us, from measurements on B200: a CTA's
// fixed part of 1.7 us, 17.4 KB/us through an SM, three CTAs at most to an SM
// (registers), and factors for what slows a plan otherwise.  28 x 28 x 512 of
// 16 bits, batch 128: 64 channels (100 KB) per CTA 45.3 us, 128 channels over
// clusters of two (100 KB) 50.2, of four (50 KB) 57.4, 128 channels in one CTA
// (200 KB) 53.2; 56 x 56 x 256, batch 64: 64-byte rows over clusters of two 49.2,
// of 128 bytes over four 52.0.
double norm_cost(double ctas, double smem, int segment, int cluster, bool direct_r)
{
    const double fit = std::min(3.0, std::floor(227.0 * 1024 / (smem + 1024)));
    const double rounds = std::ceil(ctas / (148 * fit));
    // (a shortcut that does not fit beside x is read with little in flight)
    const double bytes = direct_r ? 2.5 * smem : smem;
    double t = rounds * (1.7 + std::min(fit, std::ceil(ctas / 148)) * bytes / 17400.);
    t *= cluster == 1 ? 1. : cluster == 2 ? 1.1 : cluster == 4 ? 1.18 : 1.22;
    t *= segment < 32 ? 1.6 : segment < 64 ? 1.25 : 1.;
    return t * (fit == 1 ? 1.2 : 1.);
}

Plan search_plan(int dtype, int B, int HW, int C, int G, bool whole_blocks, bool res)
{
    Plan p{};
    const int elt = dtype == X1CB_F32 ? 4 : 2, cg = C / G;
    p.V = vector_channels(dtype, C);
    // Slices: multiples of a unit of whole groups, whole vectors and, for
    // outputs in blocks of 32 channels, whole blocks.
    long long unit = cg;
    while (unit % p.V || (whole_blocks && unit % 32))
        unit += cg;
    // The two launches, in us: 28.9 MB of input 21.8, 51.4 MB 30.7, 205 MB 123.  The
    // form is chosen without regard to a shortcut, for the workspace's sake.
    const double two = 10. + 0.55e-6 * B * static_cast<double>(HW) * C * elt;
    double best = 1e30, plain = 1e30;
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
            const long long data = static_cast<long long>(iters) * kBlock * p.V * elt;
            const long long rest = kBlock * (cg % p.V ? p.V : 1) * 8 + groups * (16 + 12);
            if (data + rest > kSmemMost)
                continue;
            const bool stage_r = res && 2 * data + rest <= kSmemMost;
            const long long smem = rest + (stage_r ? 2 : 1) * data;
            const double ctas = static_cast<double>(B) * (C / Cs) * k;
            if (ctas > INT_MAX)
                continue;
            const double cost = norm_cost(ctas, smem, Cs * elt, k, res && !stage_r);
            plain = std::min(plain, res ? norm_cost(ctas, rest + data, Cs * elt, k, false) : cost);
            if (cost < best) {
                best = cost;
                p.cluster = k;
                p.Cs = Cs;
                p.slices = C / Cs;
                p.nv = nv;
                p.lanes = lanes;
                p.iters = iters;
                p.smem = static_cast<int>(smem);
                p.stage_r = stage_r;
            }
        }
    }
    if (p.cluster && plain <= two)
        return p;
    p.cluster = 0;
    p.nv = C / p.V;
    p.lanes = std::max(1, kBlock / p.nv);
    // As many images at a time as L2 (126 MB) holds beside what is written, in
    // equal turns; two blocks per SM (each joins all of its image's chunks: 512 x 512 x
    // 128 51 us with two, 62 with three, 117 with six), at least two batches a thread.
    const double image = static_cast<double>(HW) * C * elt;
    const int turns = static_cast<int>(std::min<double>(B, std::ceil(B * image / 60e6)));
    p.images = std::min((B + turns - 1) / turns, 65535);
    const long long want = std::max(1, 148 * 2 / p.images);
    const long long most = std::max(1, HW / (p.lanes * kBatch * 2));
    p.chunks = static_cast<int>(std::min(want, most));
    p.chunk = std::min((HW + p.chunks - 1) / p.chunks, kFold * p.lanes);
    p.chunks = (HW + p.chunk - 1) / p.chunk;
    // (of 32 groups: 37 chunks 33.0 us joined by every block, 33.5 in a launch of
    // its own; 296 chunks 49.0 and 42.6, 8192 8974 and 1129)
    p.joined = p.chunks > 128;
    return p;
}

// The search takes about a microsecond, as long as the launch of a small call
// takes on the host: each thread keeps the last plans (by shape).
Plan plan_norm(int dtype, int B, int HW, int C, int G, bool whole_blocks, bool res)
{
    struct Entry {
        int key[7];
        Plan plan;
    };
    constexpr int kKept = 8;
    static thread_local Entry kept[kKept];
    static thread_local int used = 0, next = 0;
    const int key[7] = {dtype, B, HW, C, G, whole_blocks, res};
    for (int i = 0; i < used; ++i)
        if (std::memcmp(kept[i].key, key, sizeof(key)) == 0)
            return kept[i].plan;
    Entry &e = kept[next];
    std::memcpy(e.key, key, sizeof(key));
    e.plan = search_plan(dtype, B, HW, C, G, whole_blocks, res);
    next = (next + 1) % kKept;
    used = std::min(used + 1, kKept);
    return e.plan;
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
    for (a.b0 = 0; a.b0 < c.B; a.b0 += p.images) {
        const dim3 grid(p.chunks, std::min(p.images, c.B - a.b0));
        if (int e = launch(ks, grid, static_cast<size_t>(p.lanes) * c.C * sizeof(float2), 1, s, a))
            return e;
        if (p.joined)
            if (int e = launch(reinterpret_cast<const void *>(norm_join_kernel), dim3(c.G, grid.y), 0, 1,
                               s, a))
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

constexpr int kCoefFloats = sizeof(Coef) / sizeof(float);

// The workspace does not depend on the output's form: the larger of the two.
size_t norm_workspace_floats(int dtype, int B, int HW, int C, int G)
{
    size_t n = 0;
    for (int whole = 0; whole <= (C % 32 == 0 ? 1 : 0); ++whole) {
        const Plan p = plan_norm(dtype, B, HW, C, G, whole != 0, false);
        if (!p.cluster)
            n = std::max(n, static_cast<size_t>(B) * G * (static_cast<size_t>(p.chunks) * 2 + p.joined * kCoefFloats));
    }
    return n;
}

int launch_norm(const NormCall &c, cudaStream_t s)
{
    const Plan p = plan_norm(c.dtype, c.B, c.HW, c.C, c.G, c.out != kNormSame, c.r != nullptr);
    NormArgs a{};
    a.x = c.x;
    a.r = c.r;
    a.gamma = c.gamma;
    a.beta = c.beta;
    a.y = c.y;
    a.sf = c.sf;
    a.part = reinterpret_cast<float2 *>(c.ws);
    if (p.joined)
        a.coef = reinterpret_cast<Coef *>(a.part + static_cast<size_t>(c.B) * p.chunks * c.G);
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
    a.stage_r = p.stage_r;
    for (int w = join_width(p.cluster ? p.Cs / a.cg : c.G); 1 << a.log_wl < std::min(w, p.lanes);)
        ++a.log_wl;
    a.inv_count = 1. / (static_cast<double>(c.HW) * a.cg);
    a.div_nv = p.nv > 1 ? static_cast<uint32_t>(((1ull << 32) + p.nv - 1) / p.nv) : 0;
    a.div_lanes = p.lanes > 1 ? static_cast<uint32_t>(((1ull << 32) + p.lanes - 1) / p.lanes) : 0;
    if (c.dtype == X1CB_F32)
        return run_v<float>(c, p, a, s);
    return c.dtype == X1CB_BF16 ? run_v<__nv_bfloat16>(c, p, a, s) : run_v<__half>(c, p, a, s);
}

}  // namespace x1cb
