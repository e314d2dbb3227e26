"""MX4 conversions and the MX4 1x1 convolution against the 64-bit definition,
and the operators as they run together."""
import pytest
import torch

import x1_conv_bn_b200 as X
from oracle import float_ref as F

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from x1_conv_bn_b200 import _build

    _build.build()
    X.lib()
    X.x1cb_debug_inject(0)
    X.x1cb_set_wait_limit_ns(0)
    X.x1cb_last_device_error(clear=True)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _clean():
    torch.cuda.synchronize()
    st, bits = X.x1cb_last_device_error(clear=True)
    assert st == 0, bits


MK = [(1, 32), (1, 2048), (3, 96), (127, 128), (128, 160), (129, 64), (1000, 544), (5, 4096),
      (4096, 32), (2, 65536)]


@pytest.mark.parametrize("M,K", MK)
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_quantize(M, K, dtype):
    g = _gen(M + K)
    x = torch.randn(M, K, generator=g, device=DEV)
    x = x * torch.exp(2 * torch.randn(M, K // 32, generator=g, device=DEV)).repeat_interleave(32, 1)
    x[:, ::7] = 0
    x = x.to(dtype)
    x[0, :32] = 0  # a block of zeros
    q, sf = X.x1cb_quantize_mx4(x)
    codes, s = F.quantize_mx4(x)
    wq, wsf = F.pack_mx4(codes, s)
    assert torch.equal(sf, wsf)
    assert torch.equal(q, wq)
    v = F.values_mx4(codes, s)
    for dt in DTYPES:
        got = X.x1cb_dequantize_mx4(q, sf, dtype=dt)
        assert got.dtype == dt and torch.equal(got, v.to(dt))


def test_quantize_ties_and_borders():
    """Every midpoint of the e2m1 grid and its neighbours, at many scales, each
    beside the block's largest value."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99], device=DEV)
    up = torch.nextafter(mid, torch.full_like(mid, 9.0))
    dn = torch.nextafter(mid, torch.zeros_like(mid))
    row = torch.cat((mid, up, dn, torch.tensor([7.5, 4.0], device=DEV)))
    e = torch.tensor([-140, -130, -128, -127, -126, -100, -1, 0, 1, 50, 124, 125], device=DEV)
    x = torch.cat([row * (2.0 ** int(k)) if k > -120 else (row.double() * 2.0 ** int(k)).float()
                   for k in e.tolist()]).view(len(e), 32)
    x = torch.cat((x, -x))
    q, sf = X.x1cb_quantize_mx4(x)
    wq, wsf = F.pack_mx4(*F.quantize_mx4(x))
    assert torch.equal(sf, wsf) and torch.equal(q, wq)


def test_quantize_not_finite():
    x = torch.randn(4, 96, generator=_gen(1), device=DEV)
    x[1, 40] = float("inf")
    x[2, 0] = float("nan")
    x[3, 95] = -float("inf")
    q, sf = X.x1cb_quantize_mx4(x)
    wq, wsf = F.pack_mx4(*F.quantize_mx4(x))
    assert torch.equal(sf, wsf) and torch.equal(q, wq)
    v = X.x1cb_dequantize_mx4(q, sf, dtype=torch.float32)
    bad = torch.zeros(4, 96, dtype=torch.bool, device=DEV)
    bad[1, 32:64] = bad[2, :32] = bad[3, 64:] = True
    assert torch.equal(torch.isnan(v), bad)


def test_dequantize_every_code_and_scale():
    codes = torch.arange(16, device=DEV).repeat(256, 2)
    s = torch.arange(256, device=DEV).view(256, 1)
    q, sf = F.pack_mx4(codes, s)
    v = F.values_mx4(codes, s)
    for dt in DTYPES:
        got, want = X.x1cb_dequantize_mx4(q, sf, dtype=dt), v.to(dt)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(got[ok], want[ok])


def test_conversions_leave_the_rest_alone():
    """Rows behind the last one are left as they were."""
    x = torch.randn(5, 64, generator=_gen(2), device=DEV)
    buf = torch.full((9, 32), 0xAB, dtype=torch.uint8, device=DEV)
    sf = torch.empty(X.mx4_scale_shape(5, 64), dtype=torch.uint8, device=DEV)
    X.x1cb_quantize_mx4(x, out=(buf[:5], sf))
    assert (buf[5:] == 0xAB).all()
    out = torch.full((9, 64), 7.0, device=DEV)
    X.x1cb_dequantize_mx4(buf[:5], sf, dtype=torch.float32, out=out[:5])
    assert (out[5:] == 7.0).all()


# ---- the product ---------------------------------------------------------------

def _operand(rows, K, g, spread=0.4):
    x = torch.randn(rows, K, generator=g, device=DEV)
    x = x * torch.exp(spread * torch.randn(rows, K // 32, generator=g, device=DEV)).repeat_interleave(32, 1)
    codes, s = F.quantize_mx4(x)
    return F.pack_mx4(codes, s), F.values_mx4(codes, s)


def _conv(shape, dtype, act, bias, res, seed):
    B, H, W, Ic, Oc = shape
    g, M = _gen(seed), B * H * W
    (x, xs), xv = _operand(M, Ic, g)
    (w, ws), wv = _operand(Oc, Ic, g)
    b = torch.randn(Oc, generator=g, device=DEV) if bias else None
    r = torch.randn(B, H, W, Oc, generator=g, device=DEV).to(dtype) if res else None
    y, size = F.conv1x1(xv, wv, b, r, act)
    got = X.conv1x1_bias_add_act_mx4(x.view(B, H, W, Ic // 2), xs, w, ws, b, r, act=act,
                                     dtype=dtype)
    _clean()
    assert got.shape == (B, H, W, Oc) and got.dtype == dtype
    tol = F.conv_tolerance(y, size, Ic, dtype)
    err = (got.double().view(M, Oc) - y).abs()
    worst = (err - tol).max()
    assert not torch.isnan(got).any() and worst <= 0, (float(worst), float(err.max()))


CONV = [  # B, H, W, Ic, Oc
    (1, 1, 1, 32, 1),        # one value
    (1, 1, 1, 2048, 1000),   # a classifier head
    (2, 1, 1, 96, 7),
    (3, 1, 1, 4096, 130),
    (1, 3, 5, 64, 128),
    (1, 4, 4, 1024, 256),    # 16 rows
    (1, 5, 5, 288, 260),     # 25 rows
    (2, 6, 5, 512, 512),     # 60 rows
    (2, 7, 9, 160, 66),      # a K tail of 32, odd channel tail
    (1, 8, 16, 128, 64),     # one whole tile of rows
    (3, 13, 11, 224, 200),
    (7, 27, 29, 544, 200),
    (5, 28, 28, 128, 512),
    (2, 56, 56, 64, 256),
    (1, 17, 19, 2080, 333),
    (9, 16, 16, 1024, 1024),
    (40, 16, 16, 256, 392),
    (16, 32, 32, 512, 2048),
    (1, 129, 127, 32, 8),
    (40, 16, 16, 608, 1000),  # many tiles, ragged in every direction
    (30, 20, 20, 288, 517),   # the same with rows that no 16-byte copy lines up with
    (51, 28, 28, 128, 512),
]


@pytest.mark.parametrize("shape", CONV, ids=[str(s) for s in CONV])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("relu", True, True),
                                          ("silu", True, False)])
def test_conv(shape, dtype, act, bias, res):
    _conv(shape, dtype, act, bias, res, sum(shape))


@pytest.mark.parametrize("shape", [(1, 1, 1, 4096, 256), (1, 7, 7, 4096, 512), (3, 16, 16, 4096, 384),
                                   (9, 16, 16, 608, 1000), (40, 16, 16, 608, 1000),
                                   (30, 20, 20, 2080, 517), (41, 16, 16, 4096, 512)])
def test_conv_exact(shape):
    """Operands whose sums fit 24 bits whatever their order: the result has to
    be exact, so that one wrong scale or element shows."""
    B, H, W, Ic, Oc = shape
    g, M = _gen(sum(shape)), B * H * W
    pair = []
    for rows in (M, Oc):
        codes = torch.randint(0, 16, (rows, Ic), generator=g, device=DEV)
        s = torch.randint(126, 129, (rows, Ic // 32), generator=g, device=DEV)
        pair.append((F.pack_mx4(codes, s), F.values_mx4(codes, s)))
    (x, xs), xv = pair[0]
    (w, ws), wv = pair[1]
    # terms are multiples of 1/16 and at most 6*2*6*2 = 144: 4096 of them stay below 2^20
    got = X.conv1x1_bias_add_act_mx4(x.view(B, H, W, Ic // 2), xs, w, ws, act="none",
                                     dtype=torch.float32)
    _clean()
    assert torch.equal(got.view(M, Oc).double(), xv @ wv.T)


@pytest.mark.parametrize("shape", [(1, 1, 64, 1024, 512), (1, 1, 65, 2400, 384), (2, 1, 50, 1280, 130),
                                   (1, 14, 14, 4096, 1000), (1, 16, 16, 4096, 48), (3, 16, 16, 4096, 48),
                                   (1, 1, 2, 1280, 77), (1, 1, 33, 800, 2048), (1, 1, 40, 4096, 2049),
                                   (1, 1, 64, 4096, 8200)])
def test_conv_split_over_clusters(shape):
    """Few rows, or few tiles and a long K: every split of K, CTAs whose share of
    it is empty among them, and units whose last rows or channels are missing."""
    _conv(shape, torch.float32, "none", True, True, sum(shape))
    _conv(shape, torch.bfloat16, "silu", False, False, sum(shape))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", [(41, 21, 23, 96, 52), (41, 21, 23, 96, 131), (41, 21, 23, 32, 250),
                                   (1, 1, 77, 512, 445), (40, 16, 16, 1024, 1001),
                                   (40, 16, 16, 1024, 1002), (1, 1, 65, 64, 1)])
def test_conv_rows_off_16_bytes(shape, dtype):
    """Rows of no multiple of 16 bytes, several tiles to a CTA, with a shortcut;
    and the elements behind the last row are left as they were."""
    _conv(shape, dtype, "relu", True, True, sum(shape))
    _conv(shape, dtype, "none", False, False, sum(shape))
    B, H, W, Ic, Oc = shape
    g, M = _gen(7), B * H * W
    (x, xs), _ = _operand(M, Ic, g)
    (w, ws), _ = _operand(Oc, Ic, g)
    buf = torch.full((M * Oc + 64,), 7.0, dtype=dtype, device=DEV)
    out = buf[:M * Oc].view(B, H, W, Oc)
    X.conv1x1_bias_add_act_mx4(x.view(B, H, W, Ic // 2), xs, w, ws, dtype=dtype, out=out)
    _clean()
    assert (buf[M * Oc:] == 7.0).all()


def test_conv_row_masks():
    """Zero rows, and blocks whose scale is NaN: their row (or channel) alone is NaN."""
    g = _gen(5)
    (x, xs), xv = _operand(300, 256, g)
    (w, ws), wv = _operand(140, 256, g)
    x[17] = 0
    codes, s = F.unpack_mx4(x, xs)
    s[200, 3] = 255
    x, xs = F.pack_mx4(codes, s)
    wc, wsb = F.unpack_mx4(w, ws)
    wsb[131, 0] = 255
    w, ws = F.pack_mx4(wc, wsb)
    got = X.conv1x1_bias_add_act_mx4(x.view(1, 300, 1, 128), xs, w, ws, act="none",
                                     dtype=torch.float32).view(300, 140)
    _clean()
    bad = torch.zeros(300, 140, dtype=torch.bool, device=DEV)
    bad[200] = True
    bad[:, 131] = True
    assert torch.equal(torch.isnan(got), bad)
    assert (got[17][~bad[17]] == 0).all()


@pytest.mark.parametrize("M,Oc", [(1, 100), (50, 136), (300, 200), (300, 7), (19000, 264)])
def test_conv_leaves_the_rest_alone(M, Oc):
    g = _gen(6)
    (x, xs), _ = _operand(M, 128, g)
    (w, ws), _ = _operand(Oc, 128, g)
    buf = torch.full((M + 140, Oc), 7.0, dtype=torch.bfloat16, device=DEV)
    X.conv1x1_bias_add_act_mx4(x.view(1, M, 1, 64), xs, w, ws, out=buf[:M].view(1, M, 1, Oc))
    _clean()
    assert (buf[M:] == 7.0).all()


def test_conv_empty_and_refused():
    w, ws = X.x1cb_quantize_mx4(torch.ones(64, 128, device=DEV))
    x = torch.empty((0, 4, 4, 64), dtype=torch.uint8, device=DEV)
    xs = torch.empty((0, 1, 32, 16), dtype=torch.uint8, device=DEV)
    assert X.conv1x1_bias_add_act_mx4(x, xs, w, ws).shape == (0, 4, 4, 64)
    x, xs = X.x1cb_quantize_mx4(torch.ones(1, 4, 4, 128, device=DEV))
    for call in (lambda: X.conv1x1_bias_add_act_mx4(x, xs, w[:, :32].contiguous(), ws),
                 lambda: X.conv1x1_bias_add_act_mx4(x, xs[:, :, :, :8], w, ws),
                 lambda: X.conv1x1_bias_add_act_mx4(x, xs, w, ws, dtype=torch.float64),
                 lambda: X.conv1x1_bias_add_act_mx4(x, xs, w, ws, act="gelu"),
                 lambda: X.conv1x1_bias_add_act_mx4(x, xs, w, ws, r=torch.zeros(1, 4, 4, 64, device=DEV)),
                 lambda: X.conv1x1_bias_add_act_mx4(x, xs, w.cpu(), ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(X.X1cbError):
        X.x1cb_quantize_mx4(torch.ones(4, 48, device=DEV))


@pytest.mark.parametrize("shape", [(1, 1, 1, 2048, 1000), (1, 6, 6, 1024, 512),
                                   (3, 28, 28, 256, 384), (40, 16, 16, 256, 512)])
def test_conv_capture_and_streams(shape):
    B, H, W, Ic, Oc = shape
    g, M = _gen(12), B * H * W
    (x, xs), _ = _operand(M, Ic, g)
    (x2, xs2), _ = _operand(M, Ic, g)
    (w, ws), _ = _operand(Oc, Ic, g)
    view = lambda t: t.view(B, H, W, Ic // 2)  # noqa: E731
    want = X.conv1x1_bias_add_act_mx4(view(x), xs, w, ws)
    want2 = X.conv1x1_bias_add_act_mx4(view(x2), xs2, w, ws)
    bx, bs, out = x.clone(), xs.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        X.conv1x1_bias_add_act_mx4(view(bx), bs, w, ws, out=out)
    for a, s, ref in ((x2, xs2, want2), (x, xs, want)):
        bx.copy_(a)
        bs.copy_(s)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a = X.conv1x1_bias_add_act_mx4(view(x), xs, w, ws, stream=one)
    b = X.conv1x1_bias_add_act_mx4(view(x2), xs2, w, ws, stream=two)
    _clean()
    assert torch.equal(a, want) and torch.equal(b, want2)


@pytest.mark.parametrize("shape", [(1, 20, 20, 512, 256), (50, 20, 20, 512, 256)])
def test_conv_bounded_wait(shape):
    """A wait that runs out is reported, and the next call works."""
    B, H, W, Ic, Oc = shape
    g = _gen(13)
    (x, xs), _ = _operand(B * H * W, Ic, g)
    (w, ws), _ = _operand(Oc, Ic, g)
    x = x.view(B, H, W, Ic // 2)
    want = X.conv1x1_bias_add_act_mx4(x, xs, w, ws)
    _clean()
    try:
        X.x1cb_set_wait_limit_ns(20_000_000)
        X.x1cb_debug_inject(1)
        X.conv1x1_bias_add_act_mx4(x, xs, w, ws)
        st, bits = X.x1cb_last_device_error(clear=True)
        assert st == X.X1CB_ERR_TIMEOUT and bits & 2
    finally:
        X.x1cb_debug_inject(0)
        X.x1cb_set_wait_limit_ns(0)
    got = X.conv1x1_bias_add_act_mx4(x, xs, w, ws)
    _clean()
    assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """The last rows of matrices of more than 2^31 elements come out as they do
    alone (rows from a multiple of 128 on keep their scale tiles)."""
    M, K = 2 ** 21 + 200, 1024
    x = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    x.random_(-50, 51, generator=_gen(3))
    q, sf = X.x1cb_quantize_mx4(x)
    tail = 2 ** 21
    q1, sf1 = X.x1cb_quantize_mx4(x[tail:].clone())
    assert torch.equal(q[tail:], q1) and torch.equal(sf[tail // 128:], sf1)
    v = X.x1cb_dequantize_mx4(q, sf)
    assert torch.equal(v[tail:], X.x1cb_dequantize_mx4(q1, sf1))
    del x, v
    q, sf = q[:, :16].contiguous(), sf[:, :1].contiguous()  # K = 32 of it
    (w, ws), _ = _operand(1032, 32, _gen(4))
    got = X.conv1x1_bias_add_act_mx4(q.view(1, M, 1, 16), sf, w, ws, act="none")
    want = X.conv1x1_bias_add_act_mx4(q[tail:].view(1, 200, 1, 16), sf[tail // 128:].contiguous(),
                                      w, ws, act="none")
    _clean()
    assert torch.equal(got[0, tail:], want[0])


def test_conv_own_output():
    """A caller's output gives the same bits as a new one (another way through
    the binding)."""
    g = _gen(14)
    (x, xs), _ = _operand(300, 256, g)
    (w, ws), _ = _operand(72, 256, g)
    x = x.view(3, 10, 10, 128)
    b, r = torch.randn(72, generator=g, device=DEV), torch.randn(3, 10, 10, 72, generator=g, device=DEV)
    want = X.conv1x1_bias_add_act_mx4(x, xs, w, ws, b, r, act="silu", dtype=torch.float32)
    out = torch.empty_like(want)
    assert X.conv1x1_bias_add_act_mx4(x, xs, w, ws, b, r, act="silu", dtype=torch.float32,
                                      out=out) is out
    _clean()
    assert torch.equal(out, want)
    v = torch.randn(5, 64, generator=g, device=DEV)
    q, sf = X.x1cb_quantize_mx4(v)
    mine = (torch.empty_like(q), torch.empty_like(sf))
    X.x1cb_quantize_mx4(v, out=mine)
    assert torch.equal(mine[0], q) and torch.equal(mine[1], sf)
    back = torch.empty_like(v)
    X.x1cb_dequantize_mx4(q, sf, dtype=torch.float32, out=back)
    assert torch.equal(back, X.x1cb_dequantize_mx4(q, sf, dtype=torch.float32))


def test_first_calls_under_capture():
    """In a fresh process the first call of every operator may be captured: nothing
    that a capture forbids happens on the way."""
    import os
    import subprocess
    import sys

    code = """
import torch
import x1_conv_bn_b200 as X
x = torch.randn(2, 9, 8, 128, device="cuda").bfloat16()
one, big = torch.randn(1, 128, device="cuda"), torch.randn(1, 400, 300, 32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = X.group_norm_act(x, None, None, 4)
    z = X.group_norm_act(big, None, None, 4)
    X.group_norm_act_i8(x, None, None, 4, 32.0)
    q, s = X.group_norm_act_mx4(x, None, None, 4)
    w, ws = X.x1cb_quantize_mx4(torch.ones(64, 128, device="cuda"))
    a = X.conv1x1_bias_add_act_mx4(q, s, w, ws)              # 144 rows
    b = X.conv1x1_bias_add_act_mx4(q[:1, :2].contiguous(), s[:1], w, ws)  # 16
    h, hs = X.x1cb_quantize_mx4(one)
    c = X.conv1x1_bias_add_act_mx4(h.view(1, 1, 1, 64), hs, w, ws)
    d = X.x1cb_dequantize_mx4(q, s)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, X.group_norm_act(x, None, None, 4))
assert torch.equal(z, X.group_norm_act(big, None, None, 4))
assert torch.equal(a, X.conv1x1_bias_add_act_mx4(q, s, w, ws))
assert torch.equal(d, X.x1cb_dequantize_mx4(q, s))
assert X.x1cb_last_device_error()[0] == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0 and "captured" in res.stdout, res.stderr[-2000:]


def test_calls_on_two_streams_at_once():
    """The product's kernels hold all of an SM's TMEM: calls that overlap on two
    streams (large, few rows, int8 pairs) still finish, with the right bits."""
    from x1_conv_bn_b200 import synth

    g = _gen(15)
    (x, xs), _ = _operand(20000, 1024, g)
    (few, few_s), _ = _operand(12, 1024, g)
    (w, ws), _ = _operand(1024, 1024, g)
    x, few = x.view(1, 20000, 1, 512), few.view(1, 12, 1, 512)
    inp = synth.conv_inputs(synth.ConvShape(32, 28, 28, 128, 512, 1, True), 5)
    i8 = [X.x1cb_pack_act(inp.x.to(DEV)), X.x1cb_pack_weight(inp.w.to(DEV)), inp.bias.to(DEV),
          inp.m.to(DEV)]
    r = X.x1cb_pack_act(inp.r.to(DEV))
    calls = [lambda: X.conv1x1_bias_add_act_mx4(x, xs, w, ws),
             lambda: X.conv1x1_bias_add_act_mx4(few, few_s, w, ws),
             lambda: X.conv1x1_bn_add_relu_i8(*i8, inp.m_r, inp.S, r)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [None] * len(calls)
    for _ in range(10):
        for i, (c, s) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(s):
                got[i] = c()
    _clean()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_views_off_their_alignment_or_strided():
    """A contiguous view that starts off 16 bytes and a strided one are refused."""
    base = torch.randn(2 * 3 * 3 * 64 + 1, device=DEV).bfloat16()
    off = base[1:].view(2, 3, 3, 64)
    for call in (lambda v: X.group_norm_act(v, None, None, 4),
                 lambda v: X.group_norm_act_i8(v, None, None, 4, 1.0),
                 lambda v: X.group_norm_act_mx4(v, None, None, 4), X.x1cb_quantize_mx4):
        with pytest.raises(X.X1cbError) as e:
            call(off)
        assert e.value.status == X.X1CB_ERR_ALIGN
        with pytest.raises(ValueError):
            call(base[:-1].view(2, 3, 64, 3).transpose(2, 3))
    codes = torch.zeros(4 * 32 + 1, dtype=torch.uint8, device=DEV)
    sf = torch.zeros(X.mx4_scale_shape(4, 64), dtype=torch.uint8, device=DEV)
    with pytest.raises(X.X1cbError) as e:
        X.x1cb_dequantize_mx4(codes[1:].view(4, 32), sf)
    assert e.value.status == X.X1CB_ERR_ALIGN
    w, ws = X.x1cb_quantize_mx4(torch.ones(8, 64, device=DEV))
    with pytest.raises(X.X1cbError) as e:
        X.conv1x1_bias_add_act_mx4(codes[1:].view(1, 2, 2, 32), sf, w, ws)
    assert e.value.status == X.X1CB_ERR_ALIGN
    _clean()


# ---- together --------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(2, 14, 14, 256, 32, 64), (1, 1, 1, 2048, 32, 1000),
                                   (3, 9, 7, 96, 3, 200)])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_norm_then_conv_then_norm(shape, dtype):
    """A pre-activation block: norm + SiLU to MX4, the 1x1 product with a
    shortcut, and a norm of the result; each step against the definition on the
    library's own input to it, so that no rounding is counted twice."""
    B, H, W, C, G, Oc = shape
    g, M = _gen(sum(shape)), B * H * W
    x = (2 * torch.randn(B, H, W, C, generator=g, device=DEV) + 1).to(dtype)
    gamma = 1 + 0.1 * torch.randn(C, generator=g, device=DEV)
    beta = 0.1 * torch.randn(C, generator=g, device=DEV)
    w, ws = X.x1cb_quantize_mx4(torch.randn(Oc, C, generator=g, device=DEV) * C ** -0.5)
    bias = torch.randn(Oc, generator=g, device=DEV)
    r = torch.randn(B, H, W, Oc, generator=g, device=DEV).to(dtype)
    q, sf = X.group_norm_act_mx4(x, gamma, beta, G, act="silu")
    out = X.conv1x1_bias_add_act_mx4(q, sf, w, ws, bias, r, act="none", dtype=dtype)
    xv = F.values_mx4(*F.unpack_mx4(q.view(M, C // 2), sf))
    wv = F.values_mx4(*F.unpack_mx4(w, ws))
    y, size = F.conv1x1(xv, wv, bias, r, "none")
    assert ((out.double().view(M, Oc) - y).abs() <= F.conv_tolerance(y, size, C, dtype)).all()
    # MX4 keeps two to three bits: the values are those of the norm to within a quarter
    ref, _ = F.group_norm(x, gamma, beta, G, 1e-5, None, "silu")
    top = ref.view(M, -1, 32).abs().amax(-1, keepdim=True).expand(-1, -1, 32).reshape(M, C)
    assert ((xv - ref.view(M, C)).abs() <= 0.25 * top + 1e-6).all()
    last = X.group_norm_act(out, None, None, 1, act="relu")
    y2, size2 = F.group_norm(out, None, None, 1, 1e-5, None, "relu")
    assert ((last.double() - y2).abs() <= F.norm_tolerance(y2, size2, dtype)).all()


def test_norm_feeds_the_int8_convolution(oracle):
    """group_norm_act_i8's output is what conv3x3_bn_relu_i8 reads: the chain
    equals the oracle's convolution of the same int8 image, bit for bit."""
    from x1_conv_bn_b200 import synth

    s = synth.ConvShape(2, 14, 14, 128, 128, 3, False)
    inp = synth.conv_inputs(s, 31)
    x = torch.randn(2, 14, 14, 128, generator=_gen(31), device=DEV).bfloat16()
    q = X.group_norm_act_i8(x, None, None, 32, 32.0)
    got = X.conv3x3_bn_relu_i8(q, X.x1cb_pack_weight(inp.w.to(DEV)), inp.bias.to(DEV),
                               inp.m.to(DEV), inp.S)
    _clean()
    img = X.x1cb_unpack_act(q).cpu()
    ref = oracle.pack_act(oracle.conv(img, inp.w, inp.bias, inp.m, inp.S, None, 0))
    assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("rows,Ic,Oc", [(1, 2048, 1000), (1, 4096, 2500), (1, 96, 7), (2, 2048, 1000),
                                        (40, 1024, 130), (300, 544, 200), (300, 96, 50),
                                        (4864, 2048, 1024)])
@pytest.mark.parametrize("swap", [False, True])
def test_conv_opposite_scales(rows, Ic, Oc, swap):
    """Scales at opposite ends of their range (bytes 1 to 253) whose products are
    near 1: only the product itself may overflow, whichever side is the large
    one.  Its sums fit 24 bits in any order, so the result is exact."""
    g, KB = _gen(rows + Ic), Ic // 32
    e = torch.tensor([125, -125, 118, -100, 0], device=DEV).repeat(-(-KB // 5))[:KB]
    if swap:
        e = -e
    pair = []
    for n, sign, spread in ((rows, -1, 1), (Oc, 1, 0)):
        codes = torch.randint(0, 16, (n, Ic), generator=g, device=DEV)
        s = 127 + sign * e + torch.randint(-spread, spread + 1, (n, KB), generator=g, device=DEV)
        pair.append((F.pack_mx4(codes, s), F.values_mx4(codes, s)))
    (x, xs), xv = pair[0]
    (w, ws), wv = pair[1]
    # terms are multiples of 1/8 and at most 36 * 2 = 72: 4096 of them stay below 2^19
    want = xv @ wv.T
    for dtype in (torch.float32, torch.bfloat16):
        got = X.conv1x1_bias_add_act_mx4(x.view(1, rows, 1, Ic // 2), xs, w, ws, act="none", dtype=dtype)
        _clean()
        assert torch.equal(got.view(rows, Oc), want.to(dtype))


@pytest.mark.parametrize("rows", [1, 2, 70])
def test_conv_not_a_number_beside_the_smallest_scale(rows):
    """A block of scale 255 makes its row (or channel) NaN whatever the other
    side's scale is, the smallest (byte 0) among them."""
    g = _gen(8)
    codes, wcodes = (torch.randint(0, 16, (n, 128), generator=g, device=DEV) for n in (rows, 40))
    s = torch.full((rows, 4), 127, device=DEV)
    t = torch.full((40, 4), 127, device=DEV)
    s[rows - 1, 1], t[:, 1] = 255, 0
    t[3, 2], s[:, 2] = 255, 0
    (x, xs), (w, ws) = F.pack_mx4(codes, s), F.pack_mx4(wcodes, t)
    got = X.conv1x1_bias_add_act_mx4(x.view(1, rows, 1, 64), xs, w, ws, act="none",
                                     dtype=torch.float32).view(rows, 40)
    _clean()
    bad = torch.zeros(rows, 40, dtype=torch.bool, device=DEV)
    bad[rows - 1] = True
    bad[:, 3] = True
    assert torch.equal(torch.isnan(got), bad)


@pytest.mark.parametrize("shape,res", [((1, 4, 4, 1024, 256), True), ((2, 6, 5, 512, 512), False),  # K split
                                       ((40, 16, 16, 2048, 1024), False), ((40, 16, 16, 2048, 1024), True),  # pairs
                                       ((40, 16, 16, 2048, 1001), True)])
@pytest.mark.parametrize("limit_ms", [20, 300])
def test_conv_bounded_wait_of_clusters(shape, res, limit_ms):
    """A wait that runs out in a CTA of a cluster: the others are told or come to
    their own end, every copy lands before any of them leaves, and the next call
    works.  (With 300 ms a CTA's other waits last longer than its exit once did.)"""
    B, H, W, Ic, Oc = shape
    g = _gen(14)
    (x, xs), _ = _operand(B * H * W, Ic, g)
    (w, ws), _ = _operand(Oc, Ic, g)
    x = x.view(B, H, W, Ic // 2)
    r = torch.randn(B, H, W, Oc, generator=g, device=DEV).to(torch.bfloat16) if res else None
    want = X.conv1x1_bias_add_act_mx4(x, xs, w, ws, None, r)
    _clean()
    try:
        X.x1cb_set_wait_limit_ns(limit_ms * 1_000_000)
        X.x1cb_debug_inject(1)
        X.conv1x1_bias_add_act_mx4(x, xs, w, ws, None, r)
        st, bits = X.x1cb_last_device_error(clear=True)
    finally:
        X.x1cb_debug_inject(0)
        X.x1cb_set_wait_limit_ns(0)
    assert st == X.X1CB_ERR_TIMEOUT and bits == 2  # the planted wait, and none besides
    got = X.conv1x1_bias_add_act_mx4(x, xs, w, ws, None, r)
    _clean()
    assert torch.equal(got, want)


def test_clusters_on_several_streams():
    """Pairs with the plain epilogue, pairs with TMA boxes and split clusters at
    once on streams of their own, again and again: none keeps TMEM or an SM that
    another waits for with its own, and the results are those of calls alone."""
    calls = []
    for k, (B, H, W, Ic, Oc, res) in enumerate([(40, 16, 16, 2048, 1001, True), (40, 16, 16, 2048, 1001, True),
                                                (40, 16, 16, 2048, 1024, True), (2, 6, 5, 2048, 1500, False)]):
        g = _gen(20 + k)
        (x, xs), _ = _operand(B * H * W, Ic, g)
        (w, ws), _ = _operand(Oc, Ic, g)
        r = torch.randn(B, H, W, Oc, generator=g, device=DEV).to(torch.bfloat16) if res else None
        x = x.view(B, H, W, Ic // 2)
        calls.append(lambda x=x, xs=xs, w=w, ws=ws, r=r, **kw: X.conv1x1_bias_add_act_mx4(x, xs, w, ws, None, r, **kw))
    want = [c() for c in calls]
    _clean()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.empty_like(y) for _ in range(20)] for y in want]
    torch.cuda.synchronize()
    for i in range(20):
        for c, s, o in zip(calls, streams, outs):
            c(out=o[i], stream=s)
    _clean()
    for y, o in zip(want, outs):
        assert all(torch.equal(t, y) for t in o)
