"""The cases that the floating-point operators are timed on: group norm with an
activation (channels last), microscaled 4-bit (MX4) quantisation, the MX4 1x1
convolution, and the norm that feeds it.

``own`` false: plain torch forms in 32 bits.  ``own`` true: the library's calls.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5
Q_MUL = 32.0  # int8 steps per unit: the range +-4 of a normalised activation


def listed():
    return [
        # one image's last stage: 100 kB in, a call is all latency
        dict(name="norm_tail", op="norm", B=1, H=7, W=7, C=2048, G=32, dtype="bf16", act="relu",
             res=False, out="same"),
        # Res3.2's output, conv -> norm -> Sum -> ReLU over a batch: memory
        dict(name="norm_res3_add", op="norm", B=256, H=28, W=28, C=512, G=32, dtype="bf16",
             act="relu", res=True, out="same"),
        # two large images, groups of 6 channels that no 16-byte vector lines up with
        dict(name="norm_image_odd", op="norm", B=2, H=225, W=223, C=72, G=12, dtype="f32",
             act="silu", res=False, out="same"),
        # the norm in front of an int8 convolution: NC/32HW32 int8 out
        dict(name="norm_res3_i8", op="norm", B=128, H=28, W=28, C=512, G=32, dtype="f16",
             act="relu", res=False, out="i8"),
        # one pooled feature vector on its way to a 4-bit classifier head
        dict(name="quant_row", op="quant", M=1, K=2048, dtype="f32"),
        # a batch of Res3.x activations
        dict(name="quant_res3", op="quant", M=200704, K=512, dtype="bf16"),
        # the classifier head for one image: a product of one row
        dict(name="conv_head", op="conv", B=1, H=1, W=1, Ic=2048, Oc=1000, dtype="f32",
             act="none", res=False),
        # a small batch of odd-sized images, channels that fill no tile
        dict(name="conv_reduce_odd", op="conv", B=7, H=27, W=29, Ic=544, Oc=200, dtype="f16",
             act="relu", res=False),
        # Res3.2 conv3 + Sum + ReLU over a batch: memory
        dict(name="conv_expand_add", op="conv", B=256, H=28, W=28, Ic=128, Oc=512, dtype="bf16",
             act="relu", res=True),
        # the largest product: tensor cores
        dict(name="conv_wide", op="conv", B=256, H=8, W=8, Ic=4096, Oc=4096, dtype="bf16",
             act="silu", res=False),
        # norm -> 4-bit -> 1x1 convolution of two small images
        dict(name="norm_conv_small", op="norm_conv", B=2, H=14, W=14, C=1024, G=32, Oc=256,
             dtype="f16", act="silu"),
        # the same over a batch at Res3.x: Conv1 of the next block behind its norm
        dict(name="norm_conv_res3", op="norm_conv", B=256, H=28, W=28, C=512, G=32, Oc=128,
             dtype="bf16", act="relu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "conv", "conv", "norm_conv"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    act = rng.choice(["none", "relu", "silu"])
    if op == "quant":
        K = 32 * _log(rng, 1, 128)
        return dict(op=op, M=min(_log(rng, 1, 200000), 60_000_000 // K + 1), K=K, dtype=dtype)
    H, W = _log(rng, 1, 112), _log(rng, 1, 112)
    most = _log(rng, 1 << 12, 1 << 25)  # activations of the case
    if op == "conv":
        Ic, Oc = 32 * _log(rng, 1, 128), _log(rng, 8, 4096)
        B = max(1, min(256, most // (H * W * max(Ic, Oc))))
        return dict(op=op, B=B, H=H, W=W, Ic=Ic, Oc=Oc, dtype=dtype, act=act,
                    res=rng.random() < 0.4)
    if op == "norm_conv":
        # 16-bit tensors: behind the 4-bit image no output has 24 good bits
        dtype = rng.choice(["bf16", "f16"])
        G = rng.choice([1, 4, 8, 16, 32])
        C = 32 * _log(rng, 1, 48)
        B = max(1, min(256, most // (H * W * C)))
        return dict(op=op, B=B, H=H, W=W, C=C, G=G, Oc=_log(rng, 8, 1024), dtype=dtype, act=act)
    out = rng.choice(["same", "same", "i8"])
    if out == "i8":
        G = rng.choice([1, 8, 32])
        C = 32 * _log(rng, 1, 64)
    else:
        G = rng.choice([1, 2, 7, 8, 16, 32])
        C = G * _log(rng, 1, 64)
    B = max(1, min(256, most // (H * W * C)))
    return dict(op=op, B=B, H=H, W=W, C=C, G=G, dtype=dtype, act=act,
                res=rng.random() < 0.4, out=out)


# ---- inputs ------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _norm_inputs(c, g, dtype):
    """A convolution's output: each channel with its own mean and spread."""
    C = c["C"]
    x = _normal(g, c["B"], c["H"], c["W"], C)
    x = x.mul_(_normal(g, C).mul_(0.3).exp_()).add_(_normal(g, C).mul_(0.5)).to(dtype)
    return x, 1 + 0.2 * _normal(g, C), 0.2 * _normal(g, C)


def _pack_mx4(x):
    """[M, K] float32 -> (codes [M, K/2] uint8, scales [ceil(M/128), ceil(K/128), 32, 16] uint8)."""
    M, K = x.shape
    blk = x.view(M, K // 32, 32)
    e = _shared_exponent(blk.abs().amax(-1))
    code = _code(blk * _power(-e).unsqueeze(-1)).view(M, K)
    q = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    Mp, Kp = -(-M // 128), -(-K // 128)
    sf = torch.zeros((Mp * 128, Kp * 4), dtype=torch.uint8, device=x.device)
    sf[:M, : K // 32] = (e + 127).to(torch.uint8)
    sf = sf.view(Mp, 4, 32, Kp, 4).permute(0, 3, 2, 1, 4).reshape(Mp, Kp, 32, 16)
    return q.contiguous(), sf.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quant":
        x = _normal(g, case["M"], case["K"]) * _normal(g, case["K"]).mul_(0.5).exp_()
        s["x"] = x.to(_DT[case["dtype"]])
        return s
    dt = _DT[case["dtype"]]
    if case["op"] == "norm":
        s["x"], s["gamma"], s["beta"] = _norm_inputs(case, g, dt)
        s["r"] = None
        if case["res"]:
            s["r"] = _normal(g, case["B"], case["H"], case["W"], case["C"]).to(dt)
        # the value of an int8 step, for the caller's own arithmetic (half: exact)
        s["step"] = torch.tensor(1.0 / Q_MUL, dtype=torch.float16, device="cuda")
        return s
    K = case["C"] if case["op"] == "norm_conv" else case["Ic"]
    s["w"], s["ws"] = _pack_mx4(_normal(g, case["Oc"], K) * K ** -0.5)
    s["bias"] = 0.2 * _normal(g, case["Oc"])
    if case["op"] == "norm_conv":
        s["x"], s["gamma"], s["beta"] = _norm_inputs(case, g, dt)
        return s
    B, H, W = case["B"], case["H"], case["W"]
    x, s["xs"] = _pack_mx4(_normal(g, B * H * W, K) * _normal(g, K).mul_(0.3).exp_())
    s["x"] = x.view(B, H, W, K // 2)
    s["r"] = _normal(g, B, H, W, case["Oc"]).to(dt) if case["res"] else None
    return s


# ---- the plain forms -----------------------------------------------------------

def _shared_exponent(amax):
    """floor(log2 amax) - 2, the MX scale exponent of a block (at least -127; 0 -> -127)."""
    e = torch.frexp(amax)[1] - 3
    return torch.where(amax > 0, e, -127).clamp(-127, 127)


def _power(e):
    """2^e as float32, exactly (-126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _code(v):
    """float32 -> e2m1 code, round to nearest, ties to the even code, saturating."""
    a = v.abs()
    c = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
         + (a >= 3.5) + (a > 5.0))
    return c + 8 * (v < 0)


def _table():
    return torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device="cuda")


def _plain_round_mx4(x):
    """[M, K] float32 -> the values that its MX4 form stands for."""
    M, K = x.shape
    blk = x.view(M, K // 32, 32)
    e = _shared_exponent(blk.abs().amax(-1, keepdim=True))
    return (_table()[_code(blk * _power(-e))] * _power(e.clamp(min=-126))).view(M, K)


def _plain_unpack(q, sf):
    M, K = q.shape[0], 2 * q.shape[1]
    code = torch.stack((q & 15, q >> 4), -1).view(M, K).to(torch.int32)
    s = sf.view(sf.shape[0], sf.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = s.reshape(sf.shape[0] * 128, sf.shape[1] * 4)[:M, : K // 32].to(torch.int32) - 127
    return (_table()[code].view(M, K // 32, 32) * _power(s).unsqueeze(-1)).view(M, K)


def _plain_act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    return v / (1 + torch.exp(-v)) if act == "silu" else v


def _plain_norm(s):
    B, H, W, C = s["x"].shape
    x = s["x"].float().view(B, H * W, s["G"], C // s["G"])
    mu = x.mean((1, 3), keepdim=True)
    d = x - mu
    y = d / torch.sqrt((d * d).mean((1, 3), keepdim=True) + EPS)
    y = y.view(B, H, W, C) * s["gamma"] + s["beta"]
    if s.get("r") is not None:
        y = y + s["r"].float()
    return _plain_act(y, s["act"])


def _plain_conv(s, x, w):
    y = x @ w.T + s["bias"]
    if s.get("r") is not None:
        y = y + s["r"].float().view(y.shape)
    return _plain_act(y, s["act"]).to(_DT[s["dtype"]]).view(s["B"], s["H"], s["W"], s["Oc"])


def _plain(s):
    if s["op"] == "quant":
        return _plain_round_mx4(s["x"].float()).to(torch.bfloat16)
    if s["op"] == "conv":
        x = _plain_unpack(s["x"].view(-1, s["Ic"] // 2), s["xs"])
        return _plain_conv(s, x, _plain_unpack(s["w"], s["ws"]))
    y = _plain_norm(s)
    if s["op"] == "norm_conv":
        return _plain_conv(s, _plain_round_mx4(y.view(-1, s["C"])), _plain_unpack(s["w"], s["ws"]))
    if s["out"] == "i8":
        y = torch.round(y * Q_MUL).clamp(-128, 127) / Q_MUL
        y = y.view(s["B"], s["H"], s["W"], s["C"] // 32, 32).permute(0, 3, 1, 2, 4)
        return y.to(torch.float16).contiguous()
    return y.to(_DT[s["dtype"]])


# ---- one pass --------------------------------------------------------------------

def _own(s):
    import x1_conv_bn_b200 as X

    if s["op"] == "quant":
        q, sf = X.x1cb_quantize_mx4(s["x"])
        return X.x1cb_dequantize_mx4(q, sf, dtype=torch.bfloat16)
    if s["op"] == "conv":
        return X.conv1x1_bias_add_act_mx4(s["x"], s["xs"], s["w"], s["ws"], s["bias"], s["r"],
                                          act=s["act"], dtype=_DT[s["dtype"]])
    if s["op"] == "norm_conv":
        q, sf = X.group_norm_act_mx4(s["x"], s["gamma"], s["beta"], s["G"], eps=EPS, act=s["act"])
        return X.conv1x1_bias_add_act_mx4(q, sf, s["w"], s["ws"], s["bias"],
                                          dtype=_DT[s["dtype"]], act=s["act"])
    if s["out"] == "i8":
        y = X.group_norm_act_i8(s["x"], s["gamma"], s["beta"], s["G"], Q_MUL, eps=EPS, r=s["r"],
                                act=s["act"])
        return y * s["step"]
    return X.group_norm_act(s["x"], s["gamma"], s["beta"], s["G"], eps=EPS, r=s["r"],
                            act=s["act"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    e = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
    if case["op"] == "quant":
        n = case["M"] * case["K"]
        # x in; codes and scales out and in again; bf16 values out
        return {"bytes": n * (e + 2 * 17 / 32 + 2), "flops": 4 * n}
    px = case["B"] * case["H"] * case["W"]
    if case["op"] == "norm":
        n = px * case["C"]
        back = 4 if case["out"] == "i8" else e  # int8 out and in again, its values out
        return {"bytes": n * (e * (2 if case["res"] else 1) + back) + 8 * case["C"],
                "flops": 10 * n}
    N = case["Oc"]
    if case["op"] == "norm_conv":
        K = case["C"]
        n = px * K
        return {"bytes": n * e + N * K * 17 / 32 + 4 * N + px * N * e + 8 * K,
                "flops": 2 * n * N + 14 * n}
    K = case["Ic"]
    return {"bytes": (px + N) * K * 17 / 32 + 4 * N + px * N * e * (2 if case["res"] else 1),
            "flops": 2 * px * N * K}


# ---- 64 bits -----------------------------------------------------------------------

def _exact_round_mx4(x):
    """MX4 of [M, K] float64 by its definition: the spacing of e2m1 numbers around each value."""
    M, K = x.shape
    blk = x.reshape(M, K // 32, 32)
    top = blk.abs().amax(2, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 2)
    # log2 may land on the wrong side of a power of two: put it right by comparison
    scale = torch.where(top >= 8 * scale, scale * 2, scale)
    scale = torch.where(top < 4 * scale, scale / 2, scale).clamp(min=2.0 ** -127)
    v = blk / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(v.dtype)
    return ((torch.round(v / step) * step).clamp(-6, 6) * scale).reshape(M, K)


def _exact_unpack(q, sf):
    """sign * (1 + m/2) * 2^(e-1) (or m/2 where e = 0), times 2^(s - 127)."""
    M, half = q.shape
    code = torch.empty((M, 2 * half), dtype=torch.float64, device=q.device)
    for k in (0, 1):
        n = (q >> (4 * k)) & 15
        m, e = (n & 1).double(), ((n >> 1) & 3).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
        code[:, k::2] = torch.where(n >= 8, -v, v)
    row = torch.arange(M, device=q.device).unsqueeze(1)
    kb = torch.arange(half // 16, device=q.device).unsqueeze(0)
    s = sf[row // 128, kb // 4, row % 32, row % 128 // 32 * 4 + kb % 4].double()
    return code * torch.exp2(s - 127).repeat_interleave(32, 1)


def _exact_act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    return v * torch.sigmoid(v) if act == "silu" else v


def _exact_norm(s):
    x = s["x"].double()
    B, H, W, C = x.shape
    g = x.reshape(B, H * W, s["G"], C // s["G"]).transpose(1, 2).reshape(B, s["G"], -1)
    var, mu = torch.var_mean(g, dim=2, correction=0)
    a = (var + EPS).rsqrt().repeat_interleave(C // s["G"], 1) * s["gamma"].double()
    y = (x - mu.repeat_interleave(C // s["G"], 1)[:, None, None, :]) * a[:, None, None, :]
    y = y + s["beta"].double()
    if s.get("r") is not None:
        y = y + s["r"].double()
    return _exact_act(y, s["act"])


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quant":
        return _exact_round_mx4(s["x"].double())
    if s["op"] in ("norm", "norm_conv"):
        y = _exact_norm(s)
        if s["op"] == "norm":
            if s["out"] == "i8":
                y = torch.round(y * Q_MUL).clamp(-128, 127) / Q_MUL
                y = torch.stack(y.split(32, dim=3), 1)
            return y
        a = _exact_round_mx4(y.reshape(-1, s["C"]))
    else:
        a = _exact_unpack(s["x"].reshape(-1, s["Ic"] // 2), s["xs"])
    y = torch.matmul(a, _exact_unpack(s["w"], s["ws"]).T) + s["bias"].double()
    if s.get("r") is not None:
        y = y + s["r"].double().reshape(y.shape)
    return _exact_act(y, s["act"]).reshape(s["B"], s["H"], s["W"], s["Oc"])
