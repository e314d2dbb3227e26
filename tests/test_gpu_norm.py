"""group_norm_act and its int8 and MX4 forms against the 64-bit definition."""
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


def _inputs(shape, dtype, seed, mean=0.5, res=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    C = shape[-1]
    x = torch.randn(shape, generator=g, device=DEV)
    x = x * torch.exp(0.3 * torch.randn(C, generator=g, device=DEV)) + mean
    gamma = 1 + 0.2 * torch.randn(C, generator=g, device=DEV)
    beta = 0.2 * torch.randn(C, generator=g, device=DEV)
    r = torch.randn(shape, generator=g, device=DEV).to(dtype) if res else None
    return x.to(dtype), gamma, beta, r


def _close(got, y, tol):
    err = (got.double() - y).abs()
    worst = (err - tol).max()
    assert not torch.isnan(got).any() and worst <= 0, (float(worst), float(err.max()))


def _check_mx4(q, sf, y, tol):
    """Codes and scales are those of some y' within tol of y."""
    C = y.shape[-1]
    y, tol = y.reshape(-1, C), tol.reshape(-1, C)
    M = y.shape[0]
    codes, s = F.unpack_mx4(q.reshape(M, C // 2), sf)
    a, t = y.abs().reshape(M, -1, 32), tol.reshape(M, -1, 32)
    lo, hi = F.scale_byte((a - t).clamp(min=0).amax(-1)), F.scale_byte((a + t).amax(-1))
    assert ((s >= lo) & (s <= hi)).all()
    scale = torch.exp2(s.double() - 127).repeat_interleave(32, 1)
    grid = torch.tensor(F.E2M1, dtype=torch.float64, device=y.device)

    def q_at(v):
        return torch.where(v < 0, -1.0, 1.0) * grid[F.round_e2m1(v / scale)]

    got = F.values_mx4(codes, torch.full_like(s, 127))
    assert ((got >= q_at(y - tol)) & (got <= q_at(y + tol))).all()
    want = F.pack_mx4(codes, s)[1]  # padding bytes are zero
    assert torch.equal(want, sf)


SHAPES = [  # B, H, W, C, G
    (1, 1, 1, 32, 32),    # one value per group: y = beta
    (2, 1, 1, 64, 32),    # two values per group
    (1, 1, 1, 8192, 1),   # one pixel, one group, the most channels
    (3, 7, 7, 64, 1),
    (2, 5, 3, 7, 7),      # odd channels, a group each
    (2, 9, 11, 30, 6),    # 5 channels a group, 2 to a vector
    (1, 13, 17, 72, 12),  # 6 channels a group: vectors across groups
    (2, 28, 28, 96, 3),
    (5, 14, 14, 256, 32),
    (1, 7, 7, 2048, 32),
    (300, 2, 2, 32, 8),   # many small images
    (2, 112, 112, 64, 32),
    (1, 301, 299, 40, 5),  # more than one chip's worth of pixels per image
    (1, 600, 500, 24, 4),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s) for s in SHAPES])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("act,res", [("none", False), ("relu", True), ("silu", False)])
def test_norm(shape, dtype, act, res):
    *s, G = shape
    x, gamma, beta, r = _inputs(s, dtype, hash(shape) & 0xFFFF, res=res)
    y, size = F.group_norm(x, gamma, beta, G, 1e-5, r, act)
    got = X.group_norm_act(x, gamma, beta, G, eps=1e-5, r=r, act=act)
    assert got.dtype == dtype and got.shape == x.shape
    _close(got, y, F.norm_tolerance(y, size, dtype))


QSHAPES = [(1, 1, 1, 32, 1), (2, 3, 5, 64, 8), (1, 7, 7, 2048, 32), (3, 28, 28, 160, 5),
           (2, 13, 10, 96, 32), (1, 200, 150, 64, 8), (1, 1, 1, 8192, 1)]


@pytest.mark.parametrize("shape", QSHAPES, ids=[str(s) for s in QSHAPES])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("act,res", [("none", True), ("relu", False), ("silu", False)])
def test_norm_i8(shape, dtype, act, res):
    B, H, W, C, G = shape
    x, gamma, beta, r = _inputs((B, H, W, C), dtype, 3, res=res)
    y, size = F.group_norm(x, gamma, beta, G, 1e-5, r, act)
    q = X.group_norm_act_i8(x, gamma, beta, G, 37.5, r=r, act=act)
    assert q.shape == (B, C // 32, H, W, 32) and q.dtype == torch.int8
    got = X.x1cb_unpack_act(q)
    t = (y * 37.5).clamp(-128, 127)
    # half a step of the integer rounding, and the 32-bit product's own
    _close(got, t, 0.5 + 37.5 * F.norm_tolerance(y, size) + t.abs() * F.U32)


@pytest.mark.parametrize("shape", QSHAPES, ids=[str(s) for s in QSHAPES])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("act,res", [("none", True), ("relu", False), ("silu", False)])
def test_norm_mx4(shape, dtype, act, res):
    B, H, W, C, G = shape
    x, gamma, beta, r = _inputs((B, H, W, C), dtype, 4, res=res)
    y, size = F.group_norm(x, gamma, beta, G, 1e-5, r, act)
    q, sf = X.group_norm_act_mx4(x, gamma, beta, G, r=r, act=act)
    assert q.shape == (B, H, W, C // 2) and tuple(sf.shape) == X.mx4_scale_shape(B * H * W, C)
    _check_mx4(q, sf, y, F.norm_tolerance(y, size))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_without_gamma_and_beta(dtype):
    x, _, _, _ = _inputs((2, 6, 5, 48), dtype, 5)
    y, size = F.group_norm(x, None, None, 6, 1e-3)
    _close(X.group_norm_act(x, None, None, 6, eps=1e-3, act="none"), y,
           F.norm_tolerance(y, size, dtype))


@pytest.mark.parametrize("shape", [(1, 60, 50, 32, 4), (1, 600, 500, 24, 4)])
@pytest.mark.parametrize("mean", [1000.0, -30000.0])
def test_far_from_zero(shape, mean):
    """Data whose mean is many times its spread: sums of squares about zero
    would lose every digit."""
    *s, G = shape
    x, gamma, beta, _ = _inputs(s, torch.float32, 6, mean=mean)
    y, size = F.group_norm(x, gamma, beta, G, 1e-5)
    got = X.group_norm_act(x, gamma, beta, G, act="none")
    _close(got, y, F.norm_tolerance(y, size))


def test_one_outlier():
    """The first pixel of an image is far off: the shifted sums start there."""
    x, gamma, beta, _ = _inputs((1, 40, 30, 32), torch.float32, 7)
    x[0, 0, 0, :] = 1e4
    y, size = F.group_norm(x, gamma, beta, 4, 1e-5)
    got = X.group_norm_act(x, gamma, beta, 4, act="none")
    # the outlier carries the variance and its run's sums cancel by up to the
    # run's length, 64: 64 more half-steps of the statistics
    _close(got, y, 64 * F.norm_tolerance(y, size))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape", [(2, 33, 31, 64), (1, 500, 400, 32)])
@pytest.mark.parametrize("value", [3.0, 1000.0, -0.0078125])
def test_constant_image(dtype, shape, value):
    """Zero variance: every 1/std is 1/sqrt(eps), every output beta."""
    x = torch.full(shape, value, device=DEV).to(dtype)
    beta = torch.arange(shape[-1], device=DEV, dtype=torch.float32)
    got = X.group_norm_act(x, None, beta, 8, act="none")
    assert torch.equal(got, beta.to(dtype).expand_as(got))


def test_not_a_number_and_infinity():
    """A NaN or infinity makes its group of its image NaN, and nothing else;
    ReLU keeps NaN; int8 turns it to 0, MX4 to NaN blocks."""
    x, gamma, beta, _ = _inputs((2, 9, 8, 128), torch.float32, 8)
    x[0, 3, 2, 5] = float("nan")   # group 0 of image 0
    x[1, 0, 0, 127] = float("inf")  # group 3 of image 1
    clean = x.clone()
    clean[0, :, :, :32] = 0
    clean[1, :, :, 96:] = 0
    want = X.group_norm_act(clean, gamma, beta, 4, act="relu")
    got = X.group_norm_act(x, gamma, beta, 4, act="relu")
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[0, :, :, :32] = True
    bad[1, :, :, 96:] = True
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[~bad], want[~bad])
    q = X.x1cb_unpack_act(X.group_norm_act_i8(x, gamma, beta, 4, 32.0))
    assert (q[bad] == 0).all()
    assert torch.equal(q[~bad], X.x1cb_unpack_act(X.group_norm_act_i8(clean, gamma, beta, 4, 32.0))[~bad])
    codes, sf = X.group_norm_act_mx4(x, gamma, beta, 4)
    v = X.x1cb_dequantize_mx4(codes, sf, dtype=torch.float32)
    assert torch.equal(torch.isnan(v), bad)


def test_empty_and_refused():
    x = torch.empty((0, 4, 4, 64), device=DEV)
    assert X.group_norm_act(x, None, None, 8).shape == x.shape
    assert X.group_norm_act_i8(x, None, None, 8, 1.0).shape == (0, 2, 4, 4, 32)
    q, sf = X.group_norm_act_mx4(x, None, None, 8)
    assert q.shape == (0, 4, 4, 32) and sf.numel() == 0
    y = torch.zeros((1, 4, 4, 64), device=DEV)
    for call in (lambda: X.group_norm_act(y, None, None, 5),
                 lambda: X.group_norm_act(y, None, None, 8, out=y),
                 lambda: X.group_norm_act_i8(y[..., :48].contiguous(), None, None, 8, 1.0)):
        with pytest.raises(X.X1cbError):
            call()
    for call in (lambda: X.group_norm_act(y[..., :32], None, None, 8),  # strided
                 lambda: X.group_norm_act(y, torch.zeros(64), None, 8),  # on the host
                 lambda: X.group_norm_act(y, None, None, 8, r=y.bfloat16())):
        with pytest.raises(ValueError):
            call()


def test_same_result_every_time():
    """Sums are joined in a fixed order: the same bits on every call."""
    x, gamma, beta, _ = _inputs((2, 333, 251, 72), torch.float32, 9)
    first = X.group_norm_act(x, gamma, beta, 12, act="silu")
    for _ in range(4):
        assert torch.equal(first, X.group_norm_act(x, gamma, beta, 12, act="silu"))


@pytest.mark.parametrize("shape", [(2, 28, 28, 128, 32), (1, 600, 500, 24, 4)])
def test_capture_and_other_stream(shape):
    *s, G = shape
    x, gamma, beta, _ = _inputs(s, torch.bfloat16, 10)
    want = X.group_norm_act(x, gamma, beta, G)
    x2, _, _, _ = _inputs(s, torch.bfloat16, 11)
    want2 = X.group_norm_act(x2, gamma, beta, G)
    out = torch.empty_like(x)
    need = X.group_norm_workspace_size(x.dtype, *s, G)
    ws = torch.empty(need, dtype=torch.int8, device=DEV) if need else None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        X.group_norm_act(x, gamma, beta, G, out=out, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        X.group_norm_act(buf, gamma, beta, G, out=out, workspace=ws)
    for src, ref in ((x2, want2), (x, want), (x2, want2)):
        buf.copy_(src)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    # the stream argument, as an object and as a raw handle
    torch.cuda.synchronize()
    got = X.group_norm_act(x, gamma, beta, G, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    got = X.group_norm_act(x, gamma, beta, G, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want)


def test_many_chunks():
    """An image of more than 128 chunks: the statistics are joined by a launch of
    their own.  The data lies far from zero, in each channel elsewhere."""
    for dtype, shape, G in ((torch.bfloat16, (2, 700, 513, 128), 32), (torch.float32, (1, 999, 1001, 36), 3)):
        x, gamma, beta, _ = _inputs(shape, dtype, 40, mean=torch.arange(shape[-1], device=DEV) / 4.0)
        y, size = F.group_norm(x, gamma, beta, G, 1e-5)
        got = X.group_norm_act(x, gamma, beta, G, act="none")
        _close(got, y, F.norm_tolerance(y, size, dtype))
        assert torch.equal(got, X.group_norm_act(x, gamma, beta, G, act="none"))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("shape,G", [((2, 301, 299, 96), 3), ((1, 700, 513, 128), 32),
                                     ((40, 150, 160, 32), 8)])
def test_large_images_every_output(shape, G, dtype):
    """Images that do not fit a cluster, several at a time and in several turns, to
    each form of output, with a shortcut."""
    x, gamma, beta, r = _inputs(shape, dtype, 50, res=True)
    y, size = F.group_norm(x, gamma, beta, G, 1e-5, r, "relu")
    tol = F.norm_tolerance(y, size)
    _close(X.group_norm_act(x, gamma, beta, G, r=r), y, F.norm_tolerance(y, size, dtype))
    q, sf = X.group_norm_act_mx4(x, gamma, beta, G, r=r)
    _check_mx4(q, sf, y, tol)
    got = X.x1cb_unpack_act(X.group_norm_act_i8(x, gamma, beta, G, 37.5, r=r))
    t = (y * 37.5).clamp(-128, 127)
    _close(got, t, 0.5 + 37.5 * tol + t.abs() * F.U32)


def test_more_than_two_to_the_31_elements():
    """Offsets pass 32 bits: the last images come out as they do alone, to a step
    of bfloat16 (another plan may join the statistics in another order)."""
    for shape, G in (((5600, 28, 28, 512), 32), ((11, 1024, 1024, 192), 8)):
        x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
        x.random_(-8, 9, generator=torch.Generator(device=DEV).manual_seed(2))
        got = X.group_norm_act(x, None, None, G, act="none")
        last = X.group_norm_act(x[-2:].clone(), None, None, G, act="none")
        assert (got[-2:].float() - last.float()).abs().max() <= 2.0 ** -7 * last.float().abs().max()
        y, size = F.group_norm(x[-1:], None, None, G, 1e-5)
        _close(got[-1:], y, F.norm_tolerance(y, size, torch.bfloat16))
        del x, got


def test_own_output_and_workspace():
    """A caller's tensors give the same bits as new ones (another way through the
    binding), and a workspace of a byte too few is refused."""
    for shape, G in (((3, 14, 14, 96), 3), ((1, 600, 500, 24), 4)):
        x, gamma, beta, r = _inputs(shape, torch.float16, 21, res=True)
        want = X.group_norm_act(x, gamma, beta, G, r=r, act="silu")
        need = X.group_norm_workspace_size(x.dtype, *shape, G)
        ws = torch.empty(max(need, 1), dtype=torch.int8, device=DEV)
        out = torch.empty_like(x)
        assert X.group_norm_act(x, gamma, beta, G, r=r, act="silu", out=out, workspace=ws) is out
        assert torch.equal(out, want)
        if need:
            with pytest.raises(X.X1cbError) as e:
                X.group_norm_act(x, gamma, beta, G, r=r, workspace=ws[:need - 1].clone())
            assert e.value.status == X.X1CB_ERR_WORKSPACE


def test_threads_at_once():
    """Calls from several threads, each on its own stream and shapes."""
    import threading

    cases = [((2, 28, 28, 128), 32), ((1, 13, 17, 72), 12), ((4, 7, 7, 512), 16), ((1, 300, 200, 40), 5)]
    data = [(_inputs(s, torch.bfloat16, 30 + i), G) for i, (s, G) in enumerate(cases)]
    want = [X.group_norm_act(x, g, b, G, act="silu") for (x, g, b, _), G in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        (x, g, b, _), G = data[i]
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = X.group_norm_act(x, g, b, G, act="silu")
            stream.synchronize()
        if not torch.equal(got, want[i]):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


OFF_CENTRE = [  # B, H, W, C, G: groups of many values, kept on chip or in two launches
    (1, 1, 1, 8191, 1),   # a channel to an entry of the join
    (1, 1, 1, 8192, 1),   # four channels to one
    (1, 7, 7, 2050, 1),
    (1, 16, 16, 4, 1),
    (1, 40, 30, 32, 4),
    (2, 28, 28, 256, 1),
    (1, 112, 112, 64, 1),
    (1, 301, 299, 40, 5),
    (1, 600, 500, 24, 4),
]


@pytest.mark.parametrize("shape", OFF_CENTRE, ids=[str(s) for s in OFF_CENTRE])
@pytest.mark.parametrize("where", ["channel", "pixel", "column"])
@pytest.mark.parametrize("far", [30.0, 100.0, 1000.0])
def test_first_values_far_off(shape, where, far):
    """The values that the sums start from lie away from all others: the first
    channel, the first pixel or the first column of every image."""
    *s, G = shape
    g = torch.Generator(device=DEV).manual_seed(11)
    x = torch.randn(s, generator=g, device=DEV)
    x[{"channel": (..., 0), "pixel": (slice(None), 0, 0), "column": (slice(None), slice(None), 0)}[where]] += far
    y, size = F.group_norm(x, None, None, G, 1e-5)
    got = X.group_norm_act(x, None, None, G, act="none")
    _close(got, y, F.norm_tolerance(y, size))


@pytest.mark.parametrize("shape", [(1000, 48, 48, 7, 7), (1, 148, 128, 1031, 1031)])
@pytest.mark.parametrize("far", [30.0, 1000.0])
def test_first_of_a_long_run_far_off(shape, far):
    """One thread's 64 pixels hold an image's only far value, their first."""
    *s, G = shape
    g = torch.Generator(device=DEV).manual_seed(12)
    x = torch.randn(s, generator=g, device=DEV)
    x[:, 0, 0] += far
    y, size = F.group_norm(x, None, None, G, 1e-5)
    got = X.group_norm_act(x, None, None, G, act="none")
    _close(got, y, F.norm_tolerance(y, size))
