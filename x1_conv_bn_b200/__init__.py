"""Python binding of the x1cb C ABI (include/x1cb.h).

Argument marshalling only: tensors become device pointers and sizes, the
current torch CUDA stream becomes the ``void *stream`` argument, and every
step of the computation runs in the library's CUDA kernels.  There is no
fallback: if libx1cb.so is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libx1cb.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "x1cb.h")

X1CB_OK = 0
X1CB_ERR_NULL = -1
X1CB_ERR_SHAPE = -2
X1CB_ERR_ALIGN = -3
X1CB_ERR_ARCH = -4
X1CB_ERR_CUDA = -5
X1CB_ERR_TIMEOUT = -6
X1CB_ERR_WORKSPACE = -7
X1CB_ERR_OVERLAP = -8
X1CB_ERR_DEVICE = -9


class X1cbError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {x1cb_status_string(status)} ({status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libx1cb.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libx1cb.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_size_t
        L.conv1x1_bn_add_relu_i8.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, i, i, i, i, i, vp]
        L.conv3x3_bn_relu_i8.argtypes = [vp, vp, vp, vp, i32, vp, i, i, i, i, i, i, vp]
        L.bottleneck_i8_workspace_size.argtypes = [i, i, i, i]
        L.bottleneck_i8_workspace_size.restype = sz
        L.bottleneck_i8.argtypes = [vp] * 10 + [i32, i32, vp, vp, sz, i, i, i, i, i, vp]
        L.bottleneck_i8_noalloc.argtypes = [vp] * 10 + [i32, i32, vp, i, i, i, i, i, vp]
        L.x1cb_pack_act.argtypes = [vp, vp, i, i, i, i, vp]
        L.x1cb_unpack_act.argtypes = [vp, vp, i, i, i, i, vp]
        L.x1cb_pack_weight.argtypes = [vp, vp, i, i, i, vp]
        L.x1cb_status_string.argtypes = [i]
        L.x1cb_status_string.restype = ctypes.c_char_p
        L.x1cb_last_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), i]
        L.x1cb_last_epilogue_forms.argtypes = [ctypes.POINTER(ctypes.c_uint), i]
        L.x1cb_trace_copy.argtypes = [vp, ctypes.c_longlong, i]
        L.x1cb_trace_copy.restype = ctypes.c_longlong
        L.x1cb_set_block_fusion.argtypes = [i]
        L.x1cb_set_block_fusion.restype = None
        L.x1cb_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        L.x1cb_set_wait_limit_ns.restype = None
        L.x1cb_debug_inject.argtypes = [i]
        L.x1cb_debug_inject.restype = None
        L.x1cb_describe_plan.argtypes = [i, i, i, i, i, i, i, ctypes.c_char_p, sz]
        L.x1cb_version.restype = ctypes.c_char_p
        L.conv3x3s2_bn_relu_i8.argtypes = [vp] * 4 + [i32, vp] + [i] * 5 + [vp]
        L.conv1x1_proj_bn_relu_i8.argtypes = [vp] * 6 + [i32, vp] + [i] * 8 + [vp]
        L.bottleneck_proj_i8_workspace_size.argtypes = [i, i, i, i]
        L.bottleneck_proj_i8_workspace_size.restype = sz
        L.bottleneck_proj_i8.argtypes = [vp] * 11 + [i32, vp, vp, sz] + [i] * 6 + [vp]
        L.x1cb_describe_plan_ex.argtypes = [i] * 10 + [ctypes.c_char_p, sz]
        L.conv_bn_relu_maxpool_i8.argtypes = [vp] * 4 + [i32, vp] + [i] * 7 + [vp]
        L.x1cb_describe_chain.argtypes = [i] * 5 + [ctypes.c_char_p, sz]
        L.conv3x3_conv1x1_bn_add_relu_i8.argtypes = [vp] * 7 + [i32, i32, vp, vp] + [i] * 5 + [vp]
        L.stem_conv_bn_relu_maxpool_i8.argtypes = [vp] * 4 + [i32, vp] + [i] * 4 + [vp]
        L.x1cb_pack_stem.argtypes = [vp, vp] + [i] * 5 + [vp]
        L.x1cb_pack_stem_weight.argtypes = [vp, vp] + [i] * 3 + [vp]
        f, ll = ctypes.c_float, ctypes.c_longlong
        L.group_norm_workspace_size.argtypes = [i] * 6
        L.group_norm_workspace_size.restype = sz
        L.group_norm_act.argtypes = [vp, i, vp, vp, vp, i, f, vp, vp, sz] + [i] * 5 + [vp]
        L.group_norm_act_i8.argtypes = [vp, i, vp, vp, vp, i, f, f, vp, vp, sz] + [i] * 5 + [vp]
        L.group_norm_act_mx4.argtypes = [vp, i, vp, vp, vp, i, f, vp, vp, vp, sz] + [i] * 5 + [vp]
        L.x1cb_mx4_scale_size.argtypes = [ll, i]
        L.x1cb_mx4_scale_size.restype = sz
        L.x1cb_quantize_mx4.argtypes = [vp, i, vp, vp, ll, i, vp]
        L.x1cb_dequantize_mx4.argtypes = [vp, vp, vp, i, ll, i, vp]
        L.conv1x1_bias_add_act_mx4.argtypes = [vp] * 6 + [i, vp, i] + [i] * 5 + [vp]
        _lib = L
    return _lib


def header_functions() -> list:
    """Names of every function declared in include/x1cb.h."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[\w ]+?\**\s*\b(\w+)\s*\(", text, flags=re.M)


def _check(status: int, what: str):
    if status != X1CB_OK:
        raise X1cbError(status, what)


def _dev(t: Optional[torch.Tensor], dtype, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, operands on {device}")
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _same_device(first: torch.Tensor, *others):
    """Every operand must live on the first one's GPU; the call then runs with
    that GPU current (the library launches on the current device)."""
    if not isinstance(first, torch.Tensor) or first.device.type != "cuda":
        raise ValueError("operands must be CUDA tensors")
    for t in others:
        if t is not None and isinstance(t, torch.Tensor) and t.device != first.device:
            raise ValueError(f"operand on {t.device}, expected {first.device}")
    return torch.cuda.device(first.device)


def _act_shape(x: torch.Tensor, name: str):
    if x.dim() != 5 or x.shape[-1] != 32:
        raise ValueError(f"{name} must be NC/32HW32 [B, C/32, H, W, 32], got {tuple(x.shape)}")
    B, C1, H, W, _ = x.shape
    return B, C1 * 32, H, W


def conv1x1_bn_add_relu_i8(x, w, bias, m, m_r: int, S: int, r=None, out=None, stream=None):
    """Fused 1x1 conv + BN (+ shortcut Sum when r is given) + ReLU + int8.

    x [B, Ic/32, H, W, 32] int8; w blocked [Oc/128, Ic/32, 128, 32] int8;
    bias, m [Oc] int32; r, out [B, Oc/32, H, W, 32] int8."""
    B, Ic, H, W = _act_shape(x, "x")
    Oc = bias.numel()
    if out is None:
        out = torch.empty((B, Oc // 32, H, W, 32), dtype=torch.int8, device=x.device)
    with _same_device(x, w, bias, m, r, out):
        st = lib().conv1x1_bn_add_relu_i8(
            _dev(x, torch.int8, "x"), _dev(w, torch.int8, "w"), _dev(bias, torch.int32, "bias"),
            _dev(m, torch.int32, "m"), int(m_r), int(S), _dev(r, torch.int8, "r"),
            _dev(out, torch.int8, "out"), B, H, W, Ic, Oc, _stream(stream, x.device))
    _check(st, "conv1x1_bn_add_relu_i8")
    return out


def conv3x3_bn_relu_i8(x, w, bias, m, S: int, out=None, pad: int = 1, stream=None):
    """Fused 3x3 conv (stride 1, pad 1) + BN + ReLU + int8.

    x [B, Ic/32, H, W, 32]; w [Oc/128, 3, 3, Ic/32, 128, 32]; out [B, Oc/32, H, W, 32]."""
    B, Ic, H, W = _act_shape(x, "x")
    Oc = bias.numel()
    if out is None:
        out = torch.empty((B, Oc // 32, H, W, 32), dtype=torch.int8, device=x.device)
    with _same_device(x, w, bias, m, out):
        st = lib().conv3x3_bn_relu_i8(
            _dev(x, torch.int8, "x"), _dev(w, torch.int8, "w"), _dev(bias, torch.int32, "bias"),
            _dev(m, torch.int32, "m"), int(S), _dev(out, torch.int8, "out"), B, H, W, Ic, Oc,
            int(pad), _stream(stream, x.device))
    _check(st, "conv3x3_bn_relu_i8")
    return out


def bottleneck_i8_workspace_size(B: int, H: int, W: int, Cmid: int) -> int:
    return int(lib().bottleneck_i8_workspace_size(B, H, W, Cmid))


def bottleneck_i8(x, w1, b1, m1, w2, b2, m2, w3, b3, m3, m_r: int, S: int, out=None,
                  workspace=None, stream=None):
    """Res3.x bottleneck: 1x1 (+BN+ReLU), 3x3 (+BN+ReLU), 1x1 (+BN+Sum(x)+ReLU)."""
    B, Cin, H, W = _act_shape(x, "x")
    Cmid = b1.numel()
    if out is None:
        out = torch.empty_like(x)
    need = bottleneck_i8_workspace_size(B, H, W, Cmid)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.int8, device=x.device)
    with _same_device(x, w1, b1, m1, w2, b2, m2, w3, b3, m3, out, workspace):
        st = lib().bottleneck_i8(
            _dev(x, torch.int8, "x"), _dev(w1, torch.int8, "w1"), _dev(b1, torch.int32, "b1"),
            _dev(m1, torch.int32, "m1"), _dev(w2, torch.int8, "w2"), _dev(b2, torch.int32, "b2"),
            _dev(m2, torch.int32, "m2"), _dev(w3, torch.int8, "w3"), _dev(b3, torch.int32, "b3"),
            _dev(m3, torch.int32, "m3"), int(m_r), int(S), _dev(out, torch.int8, "out"),
            _dev(workspace, torch.int8, "workspace"), workspace.numel(), B, H, W, Cin, Cmid,
            _stream(stream, x.device))
    _check(st, "bottleneck_i8")
    return out


def bottleneck_i8_noalloc(x, w1, b1, m1, w2, b2, m2, w3, b3, m3, m_r: int, S: int, out=None,
                          stream=None):
    """bottleneck_i8 without a workspace argument, for callers that cannot
    allocate device memory: the library keeps the two intermediates in a
    built-in 32 MiB device array (problems that need more are rejected).
    Calls share that array, so calls that overlap on the GPU race."""
    B, Cin, H, W = _act_shape(x, "x")
    Cmid = b1.numel()
    if out is None:
        out = torch.empty_like(x)
    with _same_device(x, w1, b1, m1, w2, b2, m2, w3, b3, m3, out):
        st = lib().bottleneck_i8_noalloc(
            _dev(x, torch.int8, "x"), _dev(w1, torch.int8, "w1"), _dev(b1, torch.int32, "b1"),
            _dev(m1, torch.int32, "m1"), _dev(w2, torch.int8, "w2"), _dev(b2, torch.int32, "b2"),
            _dev(m2, torch.int32, "m2"), _dev(w3, torch.int8, "w3"), _dev(b3, torch.int32, "b3"),
            _dev(m3, torch.int32, "m3"), int(m_r), int(S), _dev(out, torch.int8, "out"),
            B, H, W, Cin, Cmid, _stream(stream, x.device))
    _check(st, "bottleneck_i8_noalloc")
    return out


def _half(n: int) -> int:
    """Output extent of a stride-2 3x3 (pad 1) over n pixels."""
    return (n - 1) // 2 + 1 if n > 0 else 0


def conv3x3_conv1x1_bn_add_relu_i8(y1, w2, b2, m2, w3, b3, m3, m_r: int, S: int, r,
                                   out=None, stream=None):
    """Conv2 (3x3 + BN + ReLU) -> Conv3 (1x1 + BN + shortcut r + ReLU) of the
    bottleneck in one launch; conv2's output stays on chip.
    y1 [B, Cmid/32, H, W, 32]; r, out [B, Cout/32, H, W, 32]."""
    B, Cmid, H, W = _act_shape(y1, "y1")
    Cout = b3.numel()
    if out is None:
        out = torch.empty((B, Cout // 32, H, W, 32), dtype=torch.int8, device=y1.device)
    with _same_device(y1, w2, b2, m2, w3, b3, m3, r, out):
        st = lib().conv3x3_conv1x1_bn_add_relu_i8(
            _dev(y1, torch.int8, "y1"), _dev(w2, torch.int8, "w2"), _dev(b2, torch.int32, "b2"),
            _dev(m2, torch.int32, "m2"), _dev(w3, torch.int8, "w3"), _dev(b3, torch.int32, "b3"),
            _dev(m3, torch.int32, "m3"), int(m_r), int(S), _dev(r, torch.int8, "r"),
            _dev(out, torch.int8, "out"), B, H, W, Cmid, Cout, _stream(stream, y1.device))
    _check(st, "conv3x3_conv1x1_bn_add_relu_i8")
    return out


def conv3x3s2_bn_relu_i8(x, w, bias, m, S: int, out=None, stream=None):
    """Fused 3x3 stride-2 conv (pad 1) + BN + ReLU + int8 (a projection
    block's Conv2).  x [B, Ic/32, H, W, 32] -> out [B, Oc/32, Ho, Wo, 32]."""
    B, Ic, H, W = _act_shape(x, "x")
    Oc = bias.numel()
    if out is None:
        out = torch.empty((B, Oc // 32, _half(H), _half(W), 32), dtype=torch.int8,
                          device=x.device)
    with _same_device(x, w, bias, m, out):
        st = lib().conv3x3s2_bn_relu_i8(
            _dev(x, torch.int8, "x"), _dev(w, torch.int8, "w"), _dev(bias, torch.int32, "bias"),
            _dev(m, torch.int32, "m"), int(S), _dev(out, torch.int8, "out"), B, H, W, Ic, Oc,
            _stream(stream, x.device))
    _check(st, "conv3x3s2_bn_relu_i8")
    return out


def conv1x1_proj_bn_relu_i8(y, w3, x, wp, bias, m, S: int, out=None, stream=None):
    """Projection block's Conv3: 1x1 of y plus the stride-2 1x1 of the block
    input x in one accumulator, + BN + ReLU + int8.
    y [B, Cy/32, H, W, 32]; x [B, Cx/32, Hx, Wx, 32]; out [B, Oc/32, H, W, 32]."""
    B, Cy, H, W = _act_shape(y, "y")
    B2, Cx, Hx, Wx = _act_shape(x, "x")
    if B2 != B:
        raise ValueError("y and x must have the same batch")
    Oc = bias.numel()
    if out is None:
        out = torch.empty((B, Oc // 32, H, W, 32), dtype=torch.int8, device=y.device)
    with _same_device(y, w3, x, wp, bias, m, out):
        st = lib().conv1x1_proj_bn_relu_i8(
            _dev(y, torch.int8, "y"), _dev(w3, torch.int8, "w3"), _dev(x, torch.int8, "x"),
            _dev(wp, torch.int8, "wp"), _dev(bias, torch.int32, "bias"),
            _dev(m, torch.int32, "m"), int(S), _dev(out, torch.int8, "out"),
            B, H, W, Cy, Hx, Wx, Cx, Oc, _stream(stream, y.device))
    _check(st, "conv1x1_proj_bn_relu_i8")
    return out


def conv_bn_relu_maxpool_i8(x, w, bias, m, S: int, R: int = 7, stride: int = 2, out=None,
                            stream=None):
    """The stem's conv (R x R, pad (R-1)/2, stride) + BN + ReLU + 3x3 stride-2
    max pooling in one launch; 64 output channels.
    x [B, Ic/32, H, W, 32] -> out [B, 2, Hp, Wp, 32]."""
    B, Ic, H, W = _act_shape(x, "x")
    Oc = bias.numel()
    pad = (R - 1) // 2
    Hc, Wc = (H + 2 * pad - R) // stride + 1, (W + 2 * pad - R) // stride + 1
    if out is None:
        out = torch.empty((B, Oc // 32, _half(Hc), _half(Wc), 32), dtype=torch.int8,
                          device=x.device)
    with _same_device(x, w, bias, m, out):
        st = lib().conv_bn_relu_maxpool_i8(
            _dev(x, torch.int8, "x"), _dev(w, torch.int8, "w"), _dev(bias, torch.int32, "bias"),
            _dev(m, torch.int32, "m"), int(S), _dev(out, torch.int8, "out"), B, H, W, Ic, Oc,
            int(R), int(stride), _stream(stream, x.device))
    _check(st, "conv_bn_relu_maxpool_i8")
    return out


def stem_fold_width(W: int, R: int = 7) -> int:
    """Columns of the folded stem tensor: the stride-2 convolution's outputs."""
    pad = (R - 1) // 2
    return (W + 2 * pad - R) // 2 + 1 if W + 2 * pad >= R else 0


def x1cb_pack_stem(nhwc, R: int = 7, out=None, stream=None):
    """Image [B, H, W, Cin] -> width-folded [B, 1, H, Wc, 32] (R*Cin <= 32),
    Wc = stem_fold_width(W, R)."""
    B, H, W, Cin = nhwc.shape
    if out is None:
        out = torch.empty((B, 1, H, stem_fold_width(W, R), 32), dtype=torch.int8,
                          device=nhwc.device)
    with _same_device(nhwc, out):
        st = lib().x1cb_pack_stem(_dev(nhwc, torch.int8, "nhwc"), _dev(out, torch.int8, "out"),
                                  B, H, W, Cin, int(R), _stream(stream, nhwc.device))
    _check(st, "x1cb_pack_stem")
    return out


def x1cb_pack_stem_weight(oihw, out=None, stream=None):
    """[64, Cin, R, R] -> folded [1, R, 1, 1, 64, 32]."""
    Oc, Cin, R, _ = oihw.shape
    if out is None:
        out = torch.empty((1, R, 1, 1, Oc, 32), dtype=torch.int8, device=oihw.device)
    with _same_device(oihw, out):
        st = lib().x1cb_pack_stem_weight(_dev(oihw, torch.int8, "oihw"),
                                         _dev(out, torch.int8, "out"), Oc, Cin, R,
                                         _stream(stream, oihw.device))
    _check(st, "x1cb_pack_stem_weight")
    return out


def stem_conv_bn_relu_maxpool_i8(folded, wf, bias, m, S: int, R: int = 7, out=None,
                                 stream=None, W: Optional[int] = None):
    """The stem on a width-folded image: R x R stride-2 conv + BN + ReLU +
    3x3 stride-2 max pooling, 64 outputs.  folded [B, 1, H, Wc, 32] from
    x1cb_pack_stem; W is the image width (any width whose folded width is Wc
    gives the same result; default 2*Wc)."""
    B, C, H, Wc = _act_shape(folded, "folded")
    pad = (R - 1) // 2
    if W is None:
        W = 2 * Wc
    if stem_fold_width(W, R) != Wc:
        raise X1cbError(X1CB_ERR_SHAPE, "stem_conv_bn_relu_maxpool_i8: W does not fold to Wc")
    Hc = (H + 2 * pad - R) // 2 + 1
    if out is None:
        out = torch.empty((B, 2, _half(Hc), _half(Wc), 32), dtype=torch.int8,
                          device=folded.device)
    with _same_device(folded, wf, bias, m, out):
        st = lib().stem_conv_bn_relu_maxpool_i8(
            _dev(folded, torch.int8, "folded"), _dev(wf, torch.int8, "wf"),
            _dev(bias, torch.int32, "bias"), _dev(m, torch.int32, "m"), int(S),
            _dev(out, torch.int8, "out"), B, H, W, int(R), _stream(stream, folded.device))
    _check(st, "stem_conv_bn_relu_maxpool_i8")
    return out


def bottleneck_proj_i8_workspace_size(B: int, H: int, W: int, Cmid: int) -> int:
    return int(lib().bottleneck_proj_i8_workspace_size(B, H, W, Cmid))


def bottleneck_proj_i8(x, w1, b1, m1, w2, b2, m2, w3, wp, b3, m3, S: int, out=None,
                       workspace=None, stream=None):
    """Projection bottleneck (Res3.1): 1x1, 3x3 stride 2, 1x1 + stride-2 1x1
    projection of x in one accumulator; BN + ReLU after each."""
    B, Cin, H, W = _act_shape(x, "x")
    Cmid, Cout = b1.numel(), b3.numel()
    if out is None:
        out = torch.empty((B, Cout // 32, _half(H), _half(W), 32), dtype=torch.int8,
                          device=x.device)
    need = bottleneck_proj_i8_workspace_size(B, H, W, Cmid)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.int8, device=x.device)
    with _same_device(x, w1, b1, m1, w2, b2, m2, w3, wp, b3, m3, out, workspace):
        st = lib().bottleneck_proj_i8(
            _dev(x, torch.int8, "x"), _dev(w1, torch.int8, "w1"), _dev(b1, torch.int32, "b1"),
            _dev(m1, torch.int32, "m1"), _dev(w2, torch.int8, "w2"), _dev(b2, torch.int32, "b2"),
            _dev(m2, torch.int32, "m2"), _dev(w3, torch.int8, "w3"), _dev(wp, torch.int8, "wp"),
            _dev(b3, torch.int32, "b3"), _dev(m3, torch.int32, "m3"), int(S),
            _dev(out, torch.int8, "out"), _dev(workspace, torch.int8, "workspace"),
            workspace.numel(), B, H, W, Cin, Cmid, Cout, _stream(stream, x.device))
    _check(st, "bottleneck_proj_i8")
    return out


def x1cb_pack_act(nhwc, out=None, stream=None):
    """[B, H, W, C] int8 -> NC/32HW32 [B, C/32, H, W, 32] on the device."""
    B, H, W, C = nhwc.shape
    if out is None:
        out = torch.empty((B, C // 32, H, W, 32), dtype=torch.int8, device=nhwc.device)
    with _same_device(nhwc, out):
        st = lib().x1cb_pack_act(_dev(nhwc, torch.int8, "nhwc"), _dev(out, torch.int8, "out"),
                                 B, H, W, C, _stream(stream, nhwc.device))
    _check(st, "x1cb_pack_act")
    return out


def x1cb_unpack_act(nc32, out=None, stream=None):
    B, C, H, W = _act_shape(nc32, "nc32")
    if out is None:
        out = torch.empty((B, H, W, C), dtype=torch.int8, device=nc32.device)
    with _same_device(nc32, out):
        st = lib().x1cb_unpack_act(_dev(nc32, torch.int8, "nc32"), _dev(out, torch.int8, "out"),
                                   B, H, W, C, _stream(stream, nc32.device))
    _check(st, "x1cb_unpack_act")
    return out


def x1cb_pack_weight(oihw, out=None, stream=None):
    """[Oc, Ic, R, R] int8 -> blocked [Oc/O2, R, R, Ic/32, O2, 32], O2 = min(Oc, 128)."""
    Oc, Ic, R, R2 = oihw.shape
    O2 = min(Oc, 128)
    if out is None:
        out = torch.empty((Oc // O2, R, R, Ic // 32, O2, 32), dtype=torch.int8,
                          device=oihw.device)
    with _same_device(oihw, out):
        st = lib().x1cb_pack_weight(_dev(oihw, torch.int8, "oihw"),
                                    _dev(out, torch.int8, "out"), Oc, Ic, R,
                                    _stream(stream, oihw.device))
    _check(st, "x1cb_pack_weight")
    return out


# ---- floating-point operators ------------------------------------------------

# Calls in their ordinary form (operands on the current device, results new, on
# the current stream) are marshalled by the compiled module _x1cb_torch, which
# answers None to anything else; the Python below takes that, and names what is
# wrong.  All of them are forward only: operands that require grad are refused while
# grad mode is on.
_fast = None


def _compiled():
    global _fast
    if _fast is None:
        lib()  # raises if nothing is built
        from . import _x1cb_torch

        _fast = _x1cb_torch
    return _fast


DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTS = {"none": 0, "relu": 1, "silu": 2}


def _dtype(t: torch.dtype, name: str) -> int:
    if t not in DTYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t}")
    return DTYPES[t]


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def _forward_only(**operands):
    """Refuses a call that autograd would have to record: there is no backward pass."""
    if torch.is_grad_enabled():
        for name, t in operands.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} requires grad, and this call has no backward pass: "
                                 "detach it or call under torch.no_grad()")


def _sized(t: Optional[torch.Tensor], shape, name: str):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _cuda_index(t, name: str) -> int:
    """Index of the GPU that the call's first operand lives on."""
    d = t.get_device() if isinstance(t, torch.Tensor) else -1
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return d


def _ptr(t, dtype, index: int, name: str):
    """Device address of an operand (None: NULL) after the checks of _dev, and
    that it lives on GPU `index`."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index \
            and t.is_contiguous():
        return t.data_ptr()
    _dev(t, dtype, name)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, operands on cuda:{index}")
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_cuda_devices = {}


def _empty(shape, dtype, index: int, stream):
    """A new tensor, allocated on the stream the call runs on, so that the
    allocator never hands out memory that work on another stream still uses, or
    takes back a workspace too early."""
    device = _cuda_devices.get(index)
    if device is None:
        device = _cuda_devices.setdefault(index, torch.device("cuda", index))
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = _raw_stream(stream, index)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw \
            else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _call(fn, what: str, index: int, *args):
    """Runs the library call with GPU `index` current."""
    if torch._C._cuda_getDevice() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status != X1CB_OK:
        raise X1cbError(status, what)


def group_norm_workspace_size(dtype, B: int, H: int, W: int, C: int, G: int) -> int:
    """Bytes of workspace the group_norm_act calls need (dtype: of x)."""
    return int(lib().group_norm_workspace_size(_dtype(dtype, "dtype"), B, H, W, C, G))


def _norm(fn, what, x, gamma, beta, G, eps, r, act, ys, index, workspace, stream, *q_mul):
    """Shared by the group_norm_act calls, behind the checks of their outputs."""
    shape, xt = x.shape, x.dtype
    B, H, W, C = shape
    dt = DTYPES[xt]
    if gamma is not None and gamma.shape != (C,):
        _sized(gamma, (C,), "gamma")
    if beta is not None and beta.shape != (C,):
        _sized(beta, (C,), "beta")
    if r is not None and r.shape != shape:
        _sized(r, shape, "r")
    need = lib().group_norm_workspace_size(dt, B, H, W, C, G)
    if workspace is None and need:
        workspace = _empty(need, torch.int8, index, stream)
    _call(fn, what, index, _ptr(x, xt, index, "x"), dt, _ptr(gamma, torch.float32, index, "gamma"),
          _ptr(beta, torch.float32, index, "beta"), _ptr(r, xt, index, "r"), _act(act), eps, *q_mul,
          *ys, _ptr(workspace, torch.int8, index, "workspace"),
          0 if workspace is None else workspace.numel(), B, H, W, C, G,
          _raw_stream(stream, index))


def _norm_input(x):
    """(index of x's GPU, shape) of a group norm's input."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError("x must be [B, H, W, C]")
    _dtype(x.dtype, "x")
    return _cuda_index(x, "x"), x.shape


def group_norm_act(x, gamma, beta, G: int, eps: float = 1e-5, r=None, act: str = "relu",
                   out=None, workspace=None, stream=None):
    """Group norm (+ shortcut Sum when r is given) + activation, channels last.

    x, r, out [B, H, W, C] float32, bfloat16 or float16; gamma, beta [C]
    float32 or None; G groups; act "none", "relu" or "silu".  Forward only."""
    if out is None and workspace is None and stream is None:
        y = (_fast or _compiled()).norm(0, x, gamma, beta, G, eps, r, ACTS.get(act, -1), 0.0)
        if y is not None:
            return y
    _forward_only(x=x, gamma=gamma, beta=beta, r=r, out=out)
    index, shape = _norm_input(x)
    if out is None:
        out = _empty(shape, x.dtype, index, stream)
    elif out.shape != shape:
        _sized(out, shape, "out")
    _norm(lib().group_norm_act, "group_norm_act", x, gamma, beta, int(G), eps, r, act,
          (_ptr(out, x.dtype, index, "out"),), index, workspace, stream)
    return out


def group_norm_act_i8(x, gamma, beta, G: int, q_mul: float, eps: float = 1e-5, r=None,
                      act: str = "relu", out=None, workspace=None, stream=None):
    """group_norm_act quantised for the int8 convolutions: clamp(rint(y * q_mul),
    -128, 127) as NC/32HW32 [B, C/32, H, W, 32].  Forward only."""
    if out is None and workspace is None and stream is None:
        y = (_fast or _compiled()).norm(1, x, gamma, beta, G, eps, r, ACTS.get(act, -1), q_mul)
        if y is not None:
            return y
    _forward_only(x=x, gamma=gamma, beta=beta, r=r)
    index, (B, H, W, C) = _norm_input(x)
    shape = (B, C // 32, H, W, 32)
    if out is None:
        out = _empty(shape, torch.int8, index, stream)
    else:
        _sized(out, shape, "out")
    _norm(lib().group_norm_act_i8, "group_norm_act_i8", x, gamma, beta, int(G), eps, r, act,
          (_ptr(out, torch.int8, index, "out"),), index, workspace, stream, q_mul)
    return out


def mx4_scale_shape(M: int, K: int):
    """Shape of the scales of an [M, K] MX4 matrix: [ceil(M/128), ceil(K/128), 32, 16]."""
    return (-(-M // 128), -(-K // 128), 32, 16)


def _mx4_outs(lead, M, K, out, index, stream):
    """Codes [*lead, K/2] and scales for an MX4 result, new or checked."""
    shape, scales = (*lead, K // 2), mx4_scale_shape(M, K)
    if out is None:
        return (_empty(shape, torch.uint8, index, stream),
                _empty(scales, torch.uint8, index, stream))
    q, sf = out
    return (_sized(q, shape, "codes"), _sized(sf, scales, "scales"))


def group_norm_act_mx4(x, gamma, beta, G: int, eps: float = 1e-5, r=None, act: str = "relu",
                       out=None, workspace=None, stream=None):
    """group_norm_act quantised to MX4: (codes [B, H, W, C/2], scales), the
    operand of conv1x1_bias_add_act_mx4.  Forward only."""
    if out is None and workspace is None and stream is None:
        y = (_fast or _compiled()).norm(2, x, gamma, beta, G, eps, r, ACTS.get(act, -1), 0.0)
        if y is not None:
            return y
    _forward_only(x=x, gamma=gamma, beta=beta, r=r)
    index, (B, H, W, C) = _norm_input(x)
    q, sf = _mx4_outs((B, H, W), B * H * W, C, out, index, stream)
    _norm(lib().group_norm_act_mx4, "group_norm_act_mx4", x, gamma, beta, int(G), eps, r, act,
          (_ptr(q, torch.uint8, index, "codes"), _ptr(sf, torch.uint8, index, "scales")), index,
          workspace, stream)
    return q, sf


def x1cb_mx4_scale_size(M: int, K: int) -> int:
    return int(lib().x1cb_mx4_scale_size(int(M), int(K)))


def x1cb_quantize_mx4(x, out=None, stream=None):
    """x [..., K] float32, bfloat16 or float16 -> MX4 (codes [..., K/2] uint8,
    scales [ceil(M/128), ceil(K/128), 32, 16] uint8), M the product of the
    leading sizes; K % 32 == 0.  Forward only."""
    if out is None and stream is None:
        y = (_fast or _compiled()).quantize(x)
        if y is not None:
            return y
    _forward_only(x=x)
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be [..., K]")
    *lead, K = x.shape
    dt, index, M = _dtype(x.dtype, "x"), _cuda_index(x, "x"), x.numel() // K if K else 0
    q, sf = _mx4_outs(lead, M, K, out, index, stream)
    _call(lib().x1cb_quantize_mx4, "x1cb_quantize_mx4", index, _ptr(x, x.dtype, index, "x"), dt,
          _ptr(q, torch.uint8, index, "codes"), _ptr(sf, torch.uint8, index, "scales"), M, K,
          _raw_stream(stream, index))
    return q, sf


def x1cb_dequantize_mx4(q, sf, dtype=torch.bfloat16, out=None, stream=None):
    """MX4 (codes [..., K/2], scales) -> values [..., K] of `dtype`."""
    if out is None and stream is None:
        y = (_fast or _compiled()).dequantize(q, sf, DTYPES.get(dtype, -1))
        if y is not None:
            return y
    _forward_only(out=out)
    if not isinstance(q, torch.Tensor) or q.dim() < 1:
        raise ValueError("codes must be [..., K/2]")
    *lead, half = q.shape
    dt, M, K = _dtype(dtype, "dtype"), q.numel() // half if half else 0, 2 * half
    _sized(sf, mx4_scale_shape(M, K), "scales")
    index = _cuda_index(q, "codes")
    if out is None:
        out = _empty((*lead, K), dtype, index, stream)
    _sized(out, (*lead, K), "out")
    _call(lib().x1cb_dequantize_mx4, "x1cb_dequantize_mx4", index, _ptr(q, torch.uint8, index, "codes"),
          _ptr(sf, torch.uint8, index, "scales"), _ptr(out, dtype, index, "out"), dt, M, K,
          _raw_stream(stream, index))
    return out


def conv1x1_bias_add_act_mx4(x, xs, w, ws, bias=None, r=None, act: str = "relu",
                             dtype=torch.bfloat16, out=None, stream=None):
    """Fused 1x1 conv of MX4 operands + bias (+ shortcut Sum when r is given) +
    activation; with H = W = 1 a fully connected layer.

    x [B, H, W, Ic/2], xs MX4 activations; w [Oc, Ic/2], ws MX4 weights; bias
    [Oc] float32 or None; r, out [B, H, W, Oc] of `dtype` (float32, bfloat16 or
    float16).  Forward only."""
    if out is None and stream is None:
        y = (_fast or _compiled()).conv1x1(x, xs, w, ws, bias, r, ACTS.get(act, -1),
                                           DTYPES.get(dtype, -1))
        if y is not None:
            return y
    _forward_only(bias=bias, r=r, out=out)
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError("x must be [B, H, W, Ic/2]")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be [Oc, Ic/2]")
    B, H, W, half = x.shape
    Oc, Ic, shape = w.shape[0], 2 * half, (B, H, W, w.shape[0])
    dt, a = _dtype(dtype, "dtype"), _act(act)
    _sized(w, (Oc, half), "w")
    _sized(xs, mx4_scale_shape(B * H * W, Ic), "xs")
    _sized(ws, mx4_scale_shape(Oc, Ic), "ws")
    _sized(bias, (Oc,), "bias")
    _sized(r, shape, "r")
    index = _cuda_index(x, "x")
    if out is None:
        out = _empty(shape, dtype, index, stream)
    _sized(out, shape, "out")
    u8 = torch.uint8
    _call(lib().conv1x1_bias_add_act_mx4, "conv1x1_bias_add_act_mx4", index, _ptr(x, u8, index, "x"), _ptr(xs, u8, index, "xs"),
          _ptr(w, u8, index, "w"), _ptr(ws, u8, index, "ws"),
          _ptr(bias, torch.float32, index, "bias"), _ptr(r, dtype, index, "r"), a,
          _ptr(out, dtype, index, "out"), dt, B, H, W, Ic, Oc, _raw_stream(stream, index))
    return out


def x1cb_status_string(status: int) -> str:
    return lib().x1cb_status_string(int(status)).decode()


def x1cb_last_device_error(clear: bool = True):
    """(status, bits) of the sticky device status word; synchronises."""
    bits = ctypes.c_uint(0)
    st = lib().x1cb_last_device_error(ctypes.byref(bits), int(clear))
    return st, bits.value


def x1cb_last_epilogue_forms(clear: bool = True) -> int:
    """Bit set of the exact epilogue forms run since the last clear (bit 0
    generic, 1 64-bit high word, 2 all-32-bit, 3 all-32-bit with the bias in
    the MMA); synchronises."""
    bits = ctypes.c_uint(0)
    _check(lib().x1cb_last_epilogue_forms(ctypes.byref(bits), int(clear)),
           "x1cb_last_epilogue_forms")
    return bits.value


TRACE_SHAPE = (4, 16, 1024)  # [cta][event][n] of SM clock values


def x1cb_trace_copy(clear: bool = True):
    """Timeline table of a trace build as an int64 tensor of TRACE_SHAPE
    (None when the library was built without the trace)."""
    import numpy as np

    words = TRACE_SHAPE[0] * TRACE_SHAPE[1] * TRACE_SHAPE[2]
    buf = np.zeros(words, dtype=np.uint64)
    n = lib().x1cb_trace_copy(buf.ctypes.data, words, int(clear))
    if n < 0:
        raise X1cbError(int(n), "x1cb_trace_copy")
    if n == 0:
        return None
    return torch.from_numpy(buf.view(np.int64).reshape(TRACE_SHAPE).copy())


def x1cb_set_block_fusion(enable: bool):
    """On: bottleneck_i8 runs conv2 -> conv3 as one fused launch where the
    shape allows.  Off (the default, measured faster on B200): separate
    launches.  Same results either way."""
    lib().x1cb_set_block_fusion(int(bool(enable)))


def x1cb_set_wait_limit_ns(ns: int):
    lib().x1cb_set_wait_limit_ns(int(ns))


def x1cb_debug_inject(mode: int):
    lib().x1cb_debug_inject(int(mode))


def x1cb_describe_plan(B, H, W, Ic, Oc, R=1, has_res=True) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(lib().x1cb_describe_plan(B, H, W, Ic, Oc, R, int(has_res), buf, 512),
           "x1cb_describe_plan")
    return buf.value.decode()


def x1cb_describe_plan_ex(B, Hin, Win, Ic, Oc, R=1, stride=1, Ic2=0, has_res=False,
                          pool=False) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(lib().x1cb_describe_plan_ex(B, Hin, Win, Ic, Oc, R, stride, Ic2, int(has_res),
                                       int(pool), buf, 512), "x1cb_describe_plan_ex")
    return buf.value.decode()


def x1cb_describe_chain(B, H, W, Cmid=128, Cout=512) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(lib().x1cb_describe_chain(B, H, W, Cmid, Cout, buf, 512), "x1cb_describe_chain")
    return buf.value.decode()


def x1cb_version() -> str:
    return lib().x1cb_version().decode()
