"""Plain 64-bit forms of the floating-point operators, by their definitions.

TEST INFRASTRUCTURE ONLY, like oracle.py: the library never uses it, and it
shares no code with the CUDA path.  Works on the device of its arguments.
"""
from __future__ import annotations

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
U32 = 2.0 ** -24  # half a step of float32 at 1


def act(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    return v / (1 + torch.exp(-v)) if name == "silu" else v


def group_norm(x, gamma, beta, G, eps, r=None, name="none"):
    """(y, size): y [B, H, W, C] float64, and the magnitude |xhat*gamma| + |beta|
    + |r| of what is added up to it, with a sixteenth of the mean's part
    |mu/std*gamma| (for tolerances)."""
    B, H, W, C = x.shape
    v = x.double().reshape(B, H * W, G, C // G)
    mu = v.mean((1, 3), keepdim=True)
    var = ((v - mu) ** 2).mean((1, 3), keepdim=True)
    std, one = torch.sqrt(var + eps), torch.ones_like(v)
    t = ((v - mu) / std).reshape(B, H, W, C)
    part = (mu.abs() / std * one).reshape(B, H, W, C)
    if gamma is not None:
        t, part = t * gamma.double(), part * gamma.double().abs()
    y, size = t, t.abs() + part / 16
    for a in (beta, r):
        if a is not None:
            y, size = y + a.double(), size + a.double().abs()
    return act(y, name), size


def norm_tolerance(y, size, dtype=torch.float32):
    """How far a 32-bit group norm rounded to `dtype` may be from y.

    Statistics: runs of up to 64 additions, their roundings independent, so 8
    half-steps; the sums run over (x - k), which at most doubles or triples what
    is summed; half of the variance's error reaches 1/std; the shifted sums put
    an error of the same order on the mean, in units of the spread.  With the few
    roundings of the normalisation, bias and shortcut: 64 half-steps of the
    terms' size, plus 1 for the mean.  The mean itself is rounded when its runs
    are formed, joined and subtracted: 4 half-steps of it, the sixteenth in size.
     SiLU: the fast exponential is within 2 + 1.16|v| steps, its
    quotient within 2: 2 * (4 + 1.16|v|) half-steps of |y|, and SiLU's slope is
    at most 1.1."""
    t = 1.1 * 64 * U32 * (size + 1) + 2 * U32 * (4 + 1.16 * size) * y.abs()
    if dtype != torch.float32:
        t = t + (y.abs() + t) * torch.finfo(dtype).eps / 2
        t = t + (2.0 ** -25 if dtype == torch.float16 else 0.0)  # half's subnormals
    return t


def scale_byte(amax):
    """Scale byte of blocks with the largest magnitudes `amax` (float64)."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, m in [1/2, 1)
    s = (e.to(torch.int64) - 1 - 2 + 127).clamp(0, 254)
    s = torch.where(amax > 0, s, torch.zeros_like(s))
    return torch.where(torch.isfinite(amax), s, torch.full_like(s, 255))


def round_e2m1(v):
    """Nearest e2m1 index of |v| (ties to the even index), the sign apart."""
    a = v.abs()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=v.device)
    hi = torch.bucketize(a, grid).clamp(max=7)  # first grid value >= a
    lo = (hi - 1).clamp(min=0)
    dh, dl = grid[hi] - a, a - grid[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up | (a >= 6), hi, lo)


def quantize_mx4(x):
    """x [M, K] -> (codes [M, K] int64, scale bytes [M, K/32] int64)."""
    M, K = x.shape
    b = x.double().reshape(M, K // 32, 32)
    amax = b.abs().amax(-1)
    amax = torch.where(torch.isfinite(b).all(-1), amax, torch.full_like(amax, float("inf")))
    s = scale_byte(amax)
    v = torch.where((s == 255).unsqueeze(-1), torch.zeros_like(b),
                    b * torch.exp2(127.0 - s.double()).unsqueeze(-1))
    c = round_e2m1(v) + 8 * (torch.signbit(v) & (s != 255).unsqueeze(-1))
    return c.reshape(M, K), s


def values_mx4(codes, s):
    """float64 values of (codes [M, K], scale bytes [M, K/32])."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    scale = torch.where(s == 255, torch.full_like(s, 0).double() + float("nan"),
                        torch.exp2(s.double() - 127))
    M, K = codes.shape
    return (table[codes].reshape(M, K // 32, 32) * scale.unsqueeze(-1)).reshape(M, K)


def pack_mx4(codes, s):
    """(codes [M, K], scale bytes [M, K/32]) -> the stored arrays (uint8)."""
    M, K = codes.shape
    q = (codes[:, 0::2] + 16 * codes[:, 1::2]).to(torch.uint8)
    mt, kt = -(-M // 128), -(-K // 128)
    sf = torch.zeros(mt * kt * 512, dtype=torch.uint8, device=codes.device)
    m = torch.arange(M, device=codes.device).unsqueeze(1)
    b = torch.arange(K // 32, device=codes.device).unsqueeze(0)
    at = (m // 128 * kt + b // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + b % 4
    sf[at.reshape(-1)] = s.to(torch.uint8).reshape(-1)
    return q.contiguous(), sf.reshape(mt, kt, 32, 16)


def unpack_mx4(q, sf):
    """The stored arrays (codes [M, K/2], scales) -> (codes [M, K], scale bytes)."""
    M, half = q.shape
    codes = torch.stack((q & 15, q >> 4), -1).reshape(M, 2 * half).long()
    kt = sf.shape[1]
    m = torch.arange(M, device=q.device).unsqueeze(1)
    b = torch.arange(half // 16, device=q.device).unsqueeze(0)
    at = (m // 128 * kt + b // 4) * 512 + m % 32 * 16 + m % 128 // 32 * 4 + b % 4
    return codes, sf.reshape(-1)[at].long()


def conv1x1(x, w, bias, r, name):
    """x [M, K], w [N, K] float64 -> (out [M, N], size) with size = sum |x w| + |bias| + |r|."""
    y, size = x @ w.T, x.abs() @ w.abs().T
    for a in (bias, r):
        if a is not None:
            a = a.double().reshape(-1, y.shape[1])
            y, size = y + a, size + a.abs()
    return act(y, name), size


def conv_tolerance(y, size, K, dtype):
    """How far a product with 32-bit sums rounded to `dtype` may be from y: its
    products are exact, and each of the K/64 + 64 additions a term takes part in
    (64 to a tensor-core step) loses at most a step, 2 half-steps, of the terms'
    size; then bias and shortcut; then the activation as in norm_tolerance."""
    t = 1.1 * 2 * U32 * (K / 64 + 66) * size + 2 * U32 * (4 + 1.16 * size) * y.abs()
    if dtype != torch.float32:
        t = t + (y.abs() + t) * torch.finfo(dtype).eps / 2
        t = t + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    return t
