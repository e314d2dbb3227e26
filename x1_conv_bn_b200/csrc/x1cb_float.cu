// Entry points of the floating-point operators (include/x1cb.h): argument
// checks.  The kernels are in x1cb_norm.cu and x1cb_mx4.cu.
#include <climits>

#include "x1cb_internal.h"

namespace x1cb {
namespace {

bool good_dtype(int d) { return d == X1CB_F32 || d == X1CB_BF16 || d == X1CB_F16; }
bool good_act(int a) { return a >= X1CB_ACT_NONE && a <= X1CB_ACT_SILU; }
size_t elt(int d) { return d == X1CB_F32 ? 4 : 2; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Codes and scales of an [M, K] MX4 matrix.
size_t codes_size(long long M, int K) { return static_cast<size_t>(M) * (K / 2); }

int check_norm_shape(int dtype, int B, int H, int W, int C, int G)
{
    if (!good_dtype(dtype) || B < 0 || H < 0 || W < 0 || C < 1 || C > 8192 || G < 1 || C % G)
        return X1CB_ERR_SHAPE;
    const long long hw = static_cast<long long>(H) * W;
    if (hw > INT_MAX || (hw > 0 && B > INT_MAX / hw))
        return X1CB_ERR_SHAPE;
    return X1CB_OK;
}

int norm_common(NormCall c, size_t ws_bytes, int H, int W, void *stream)
{
    if (int e = check_norm_shape(c.dtype, c.B, H, W, c.C, c.G))
        return e;
    if (!good_act(c.act) || !(c.eps >= 0.f) || (c.out != kNormSame && c.C % 32))
        return X1CB_ERR_SHAPE;
    c.HW = H * W;
    const size_t n = static_cast<size_t>(c.B) * c.HW * c.C;
    if (n == 0)
        return X1CB_OK;
    if (!c.x || !c.y || (c.out == kNormMx4 && !c.sf))
        return X1CB_ERR_NULL;
    const size_t need = norm_workspace_floats(c.dtype, c.B, c.HW, c.C, c.G) * 4;
    if (need > 0 && (!c.ws || ws_bytes < need))
        return X1CB_ERR_WORKSPACE;
    if (!aligned16(c.x) || !aligned16(c.r) || !aligned16(c.y) || !aligned16(c.sf) ||
        (need && !aligned16(c.ws)) || !aligned4(c.gamma) || !aligned4(c.beta))
        return X1CB_ERR_ALIGN;
    const long long M = static_cast<long long>(c.B) * c.HW;
    const size_t in = n * elt(c.dtype), ch = static_cast<size_t>(c.C) * 4;
    const void *outs[3] = {c.y, c.sf, need ? c.ws : nullptr};
    const size_t sizes[3] = {c.out == kNormSame ? in : c.out == kNormI8 ? n : n / 2,
                             c.out == kNormMx4 ? x1cb_mx4_scale_size(M, c.C) : 0, need};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], sizes[i], c.x, in) || overlap(outs[i], sizes[i], c.r, in) ||
            overlap(outs[i], sizes[i], c.gamma, ch) || overlap(outs[i], sizes[i], c.beta, ch))
            return X1CB_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], sizes[i], outs[j], sizes[j]))
                return X1CB_ERR_OVERLAP;
    }
    int sms = 0;
    if (int e = current_sms(sms))
        return e;
    if (int e = check_resident({c.x, c.r, c.gamma, c.beta, c.y, c.sf, need ? c.ws : nullptr}))
        return e;
    return launch_norm(c, static_cast<cudaStream_t>(stream));
}

// (256 rows short of 2^31: the kernels count rows of whole tiles in an int)
int check_mx4_shape(long long M, int K)
{
    return M < 0 || M > INT_MAX - 255 || K < 32 || K % 32 || K > 65536 ? X1CB_ERR_SHAPE : X1CB_OK;
}

// Shared by the two conversions; `values_out`: x is the output.
int convert_common(const void *x, int dtype, const uint8_t *q, const uint8_t *sf, long long M,
                   int K, bool values_out)
{
    if (!good_dtype(dtype))
        return X1CB_ERR_SHAPE;
    if (int e = check_mx4_shape(M, K))
        return e;
    if (M == 0)
        return X1CB_OK;
    if (!x || !q || !sf)
        return X1CB_ERR_NULL;
    if (!aligned16(x) || !aligned16(q) || !aligned16(sf))
        return X1CB_ERR_ALIGN;
    const size_t nx = static_cast<size_t>(M) * K * elt(dtype), nq = codes_size(M, K);
    const size_t ns = x1cb_mx4_scale_size(M, K);
    if (overlap(x, nx, q, nq) || overlap(x, nx, sf, ns) || (!values_out && overlap(q, nq, sf, ns)))
        return X1CB_ERR_OVERLAP;
    int sms = 0;
    if (int e = current_sms(sms))
        return e;
    return check_resident({x, q, sf});
}

}  // namespace
}  // namespace x1cb

using namespace x1cb;

extern "C" {

size_t group_norm_workspace_size(int dtype, int B, int H, int W, int C, int G)
{
    if (check_norm_shape(dtype, B, H, W, C, G) != X1CB_OK || B == 0 || H == 0 || W == 0)
        return 0;
    return norm_workspace_floats(dtype, B, H * W, C, G) * 4;
}

int group_norm_act(const void *x, int dtype, const float *gamma, const float *beta,
                   const void *r, int act, float eps, void *y, void *workspace, size_t ws_bytes,
                   int B, int H, int W, int C, int G, void *stream)
{
    return norm_common(NormCall{x, r, gamma, beta, y, nullptr, static_cast<float *>(workspace),
                                eps, 0.f, dtype, kNormSame, act, B, 0, C, G},
                       ws_bytes, H, W, stream);
}

int group_norm_act_i8(const void *x, int dtype, const float *gamma, const float *beta,
                      const void *r, int act, float eps, float q_mul, int8_t *q, void *workspace,
                      size_t ws_bytes, int B, int H, int W, int C, int G, void *stream)
{
    return norm_common(NormCall{x, r, gamma, beta, q, nullptr, static_cast<float *>(workspace),
                                eps, q_mul, dtype, kNormI8, act, B, 0, C, G},
                       ws_bytes, H, W, stream);
}

int group_norm_act_mx4(const void *x, int dtype, const float *gamma, const float *beta,
                       const void *r, int act, float eps, uint8_t *q, uint8_t *sf,
                       void *workspace, size_t ws_bytes, int B, int H, int W, int C, int G,
                       void *stream)
{
    return norm_common(NormCall{x, r, gamma, beta, q, sf, static_cast<float *>(workspace), eps,
                                0.f, dtype, kNormMx4, act, B, 0, C, G},
                       ws_bytes, H, W, stream);
}

size_t x1cb_mx4_scale_size(long long M, int K)
{
    if (M < 0 || M > INT_MAX || K < 0)
        return 0;
    return static_cast<size_t>((M + 127) / 128) * ((K + 127LL) / 128) * 512;
}

int x1cb_quantize_mx4(const void *x, int dtype, uint8_t *q, uint8_t *sf, long long M, int K,
                      void *stream)
{
    if (int e = convert_common(x, dtype, q, sf, M, K, false))
        return e;
    return M == 0 ? X1CB_OK
                  : launch_quantize_mx4(x, dtype, q, sf, M, K, static_cast<cudaStream_t>(stream));
}

int x1cb_dequantize_mx4(const uint8_t *q, const uint8_t *sf, void *x, int dtype, long long M,
                        int K, void *stream)
{
    if (int e = convert_common(x, dtype, q, sf, M, K, true))
        return e;
    return M == 0 ? X1CB_OK
                  : launch_dequantize_mx4(q, sf, x, dtype, M, K, static_cast<cudaStream_t>(stream));
}

int conv1x1_bias_add_act_mx4(const uint8_t *x, const uint8_t *xs, const uint8_t *w,
                             const uint8_t *ws, const float *bias, const void *r, int act,
                             void *out, int dtype, int B, int H, int W, int Ic, int Oc,
                             void *stream)
{
    if (!good_dtype(dtype) || !good_act(act) || B < 0 || H < 0 || W < 0 || Oc < 1 || Oc > 65536)
        return X1CB_ERR_SHAPE;
    const long long hw = static_cast<long long>(H) * W;
    if (hw > INT_MAX || (hw > 0 && B > INT_MAX / hw))
        return X1CB_ERR_SHAPE;
    const long long M = B * hw;
    if (int e = check_mx4_shape(M, Ic))
        return e;
    if (M == 0)
        return X1CB_OK;
    if (!x || !xs || !w || !ws || !out)
        return X1CB_ERR_NULL;
    if (!aligned16(x) || !aligned16(xs) || !aligned16(w) || !aligned16(ws) || !aligned16(r) ||
        !aligned16(out) || !aligned4(bias))
        return X1CB_ERR_ALIGN;
    const size_t no = static_cast<size_t>(M) * Oc * elt(dtype);
    if (overlap(out, no, x, codes_size(M, Ic)) || overlap(out, no, xs, x1cb_mx4_scale_size(M, Ic)) ||
        overlap(out, no, w, codes_size(Oc, Ic)) ||
        overlap(out, no, ws, x1cb_mx4_scale_size(Oc, Ic)) ||
        overlap(out, no, bias, static_cast<size_t>(Oc) * 4) || overlap(out, no, r, no))
        return X1CB_ERR_OVERLAP;
    int sms = 0;
    if (int e = current_sms(sms))
        return e;
    if (int e = check_resident({x, xs, w, ws, bias, r, out}))
        return e;
    return launch_conv_mx4(Mx4Call{x, xs, w, ws, bias, r, out, dtype, act, M, Ic, Oc},
                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
