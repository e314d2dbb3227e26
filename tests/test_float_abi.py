"""Argument checks of the floating-point entry points: every bad call is
refused on the host, before any device is touched (the pointers are fake and
never dereferenced), and empty calls succeed without a device."""
import ctypes
import math

import pytest
import torch

import x1_conv_bn_b200 as X

BIG = 1 << 36  # fake 16-byte aligned addresses, far apart


@pytest.fixture(scope="module")
def L():
    from x1_conv_bn_b200 import _build

    _build.build()
    return X.lib()


def _p(k):
    return ctypes.c_void_p(k) if k else None


def _norm(L, kind="same", x=BIG, dtype=1, gamma=2 * BIG, beta=3 * BIG, r=0, act=1, eps=1e-5,
          y=5 * BIG, sf=6 * BIG, ws=7 * BIG, ws_bytes=1 << 34, B=2, H=28, W=28, C=128, G=32):
    head = [_p(x), dtype, _p(gamma), _p(beta), _p(r), act, eps]
    tail = [_p(ws), ws_bytes, B, H, W, C, G, None]
    if kind == "same":
        return L.group_norm_act(*head, _p(y), *tail)
    if kind == "i8":
        return L.group_norm_act_i8(*head, 32.0, _p(y), *tail)
    return L.group_norm_act_mx4(*head, _p(y), _p(sf), *tail)


@pytest.mark.parametrize("kind", ["same", "i8", "mx4"])
def test_norm_refusals(L, kind):
    S, N, A, O = X.X1CB_ERR_SHAPE, X.X1CB_ERR_NULL, X.X1CB_ERR_ALIGN, X.X1CB_ERR_OVERLAP
    for bad in (dict(dtype=3), dict(dtype=-1), dict(act=3), dict(act=-1), dict(B=-1), dict(H=-2),
                dict(C=0), dict(C=8224), dict(G=0), dict(G=-1), dict(G=3), dict(eps=-1e-5),
                dict(eps=math.nan), dict(H=65536, W=65536), dict(B=4, H=32768, W=32768)):
        assert _norm(L, kind, **bad) == S, bad
    if kind != "same":
        assert _norm(L, kind, C=48, G=4) == S
    for bad in (dict(x=0), dict(y=0)):
        assert _norm(L, kind, **bad) == N, bad
    for bad in (dict(x=BIG + 8), dict(y=5 * BIG + 4), dict(r=4 * BIG + 2), dict(gamma=2 * BIG + 2),
                dict(beta=3 * BIG + 1)):
        assert _norm(L, kind, **bad) == A, bad
    for bad in (dict(y=BIG), dict(y=BIG + 4096), dict(r=4 * BIG, y=4 * BIG), dict(y=2 * BIG)):
        assert _norm(L, kind, **bad) == O, bad
    for empty in (dict(B=0), dict(H=0), dict(W=0)):
        assert _norm(L, kind, **empty) == X.X1CB_OK
        assert _norm(L, kind, x=0, y=0, sf=0, ws=0, ws_bytes=0, **empty) == X.X1CB_OK
    if kind == "mx4":
        assert _norm(L, kind, sf=0) == N
        assert _norm(L, kind, sf=6 * BIG + 8) == A
        assert _norm(L, kind, sf=5 * BIG) == O


def test_norm_workspace(L):
    # a shape whose statistics leave the chip
    shape = dict(B=1, H=2048, W=2048, C=64, G=8)
    need = X.group_norm_workspace_size(torch.bfloat16, *shape.values())
    assert need > 0
    assert _norm(L, ws=0, ws_bytes=0, **shape) == X.X1CB_ERR_WORKSPACE
    assert _norm(L, ws_bytes=need - 1, **shape) == X.X1CB_ERR_WORKSPACE
    assert _norm(L, ws=BIG, ws_bytes=need, **shape) == X.X1CB_ERR_OVERLAP
    assert _norm(L, ws=7 * BIG + 4, ws_bytes=need, **shape) == X.X1CB_ERR_ALIGN
    # sizes that mean nothing, or nothing to do, need none
    for bad in ((0, 28, 28, 128, 32), (2, 0, 28, 128, 32), (2, 28, 28, 128, 3), (-1, 1, 1, 32, 1)):
        assert X.group_norm_workspace_size(torch.float32, *bad) == 0


@pytest.mark.parametrize("back", [False, True])
def test_conversion_refusals(L, back):
    def call(x=BIG, dtype=1, q=2 * BIG, sf=3 * BIG, M=100, K=256):
        if back:
            return L.x1cb_dequantize_mx4(_p(q), _p(sf), _p(x), dtype, M, K, None)
        return L.x1cb_quantize_mx4(_p(x), dtype, _p(q), _p(sf), M, K, None)

    for bad in (dict(dtype=3), dict(M=-1), dict(M=1 << 31), dict(M=(1 << 31) - 255), dict(K=0), dict(K=16), dict(K=-32),
                dict(K=65568)):
        assert call(**bad) == X.X1CB_ERR_SHAPE, bad
    for bad in (dict(x=0), dict(q=0), dict(sf=0)):
        assert call(**bad) == X.X1CB_ERR_NULL, bad
    for bad in (dict(x=BIG + 8), dict(q=2 * BIG + 1), dict(sf=3 * BIG + 4)):
        assert call(**bad) == X.X1CB_ERR_ALIGN, bad
    for bad in (dict(q=BIG), dict(sf=BIG + 512)):
        assert call(**bad) == X.X1CB_ERR_OVERLAP, bad
    if not back:
        assert call(sf=2 * BIG) == X.X1CB_ERR_OVERLAP
    assert call(M=0) == X.X1CB_OK
    assert call(x=0, q=0, sf=0, M=0) == X.X1CB_OK


def test_scale_size(L):
    assert X.x1cb_mx4_scale_size(0, 32) == 0
    assert X.x1cb_mx4_scale_size(1, 32) == 512
    assert X.x1cb_mx4_scale_size(129, 160) == 2 * 2 * 512
    assert X.x1cb_mx4_scale_size(-1, 32) == 0
    for M in (1 << 31, (1 << 63) - 1):
        assert X.x1cb_mx4_scale_size(M, 32) == 0
    assert X.x1cb_mx4_scale_size((1 << 31) - 1, 65536) == (1 << 24) * 512 * 512


def test_conv_refusals(L):
    def call(x=BIG, xs=2 * BIG, w=3 * BIG, ws=4 * BIG, bias=5 * BIG, r=6 * BIG, act=1,
             out=7 * BIG, dtype=1, B=2, H=28, W=28, Ic=128, Oc=512):
        return L.conv1x1_bias_add_act_mx4(_p(x), _p(xs), _p(w), _p(ws), _p(bias), _p(r), act,
                                          _p(out), dtype, B, H, W, Ic, Oc, None)

    for bad in (dict(dtype=7), dict(act=9), dict(B=-1), dict(H=-1), dict(W=-1), dict(Ic=48),
                dict(Ic=0), dict(Ic=65568), dict(Oc=0), dict(Oc=65537), dict(H=65536, W=65536),
                dict(B=3, H=32768, W=32768), dict(B=1, H=(1 << 31) - 255, W=1)):
        assert call(**bad) == X.X1CB_ERR_SHAPE, bad
    for bad in (dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(out=0)):
        assert call(**bad) == X.X1CB_ERR_NULL, bad
    for bad in (dict(x=BIG + 8), dict(xs=2 * BIG + 4), dict(w=3 * BIG + 1), dict(ws=4 * BIG + 8),
                dict(r=6 * BIG + 2), dict(out=7 * BIG + 8), dict(bias=5 * BIG + 2)):
        assert call(**bad) == X.X1CB_ERR_ALIGN, bad
    for at in (BIG, 2 * BIG, 3 * BIG, 4 * BIG, 5 * BIG, 6 * BIG):
        assert call(out=at) == X.X1CB_ERR_OVERLAP, at
    for empty in (dict(B=0), dict(H=0), dict(W=0)):
        assert call(**empty) == X.X1CB_OK
        assert call(x=0, xs=0, w=0, ws=0, out=0, **empty) == X.X1CB_OK


def test_binding_refusals():
    """The binding names what is wrong before it calls the library."""
    x = torch.zeros(1, 2, 2, 32)
    with pytest.raises(ValueError):
        X.group_norm_act(x, None, None, 4)  # not on a GPU
    with pytest.raises(ValueError):
        X.group_norm_act(x.double(), None, None, 4)
    with pytest.raises(ValueError):
        X.group_norm_act(x, None, None, 4, act="gelu")
    with pytest.raises(ValueError):
        X.group_norm_act(x[0], None, None, 4)
    with pytest.raises(ValueError):
        X.group_norm_act(x, torch.zeros(31), None, 4)
    with pytest.raises(ValueError):
        X.x1cb_quantize_mx4(x.to(torch.int8))
    q = torch.zeros(1, 2, 2, 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        X.x1cb_dequantize_mx4(q, torch.zeros(1, 1, 32, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        X.conv1x1_bias_add_act_mx4(q, None, torch.zeros(8, 32, dtype=torch.uint8), None)


def test_marshalling_module_leaves_the_unusual_alone():
    """The compiled marshalling answers None (the Python way then says what is
    wrong) to anything but plain CUDA tensors; no call here has a device."""
    from x1_conv_bn_b200 import _build

    _build.build()
    f = X._compiled()
    x, q = torch.zeros(1, 2, 2, 32), torch.zeros(1, 2, 2, 16, dtype=torch.uint8)
    s = torch.zeros(1, 1, 32, 16, dtype=torch.uint8)
    assert f.norm(0, x, None, None, 4, 1e-5, None, 1, 0.0) is None
    assert f.norm(0, None, None, None, 4, 1e-5, None, 1, 0.0) is None
    assert f.norm(0, x, None, None, "4", 1e-5, None, 1, 0.0) is None
    assert f.norm(0, x) is None
    assert f.quantize(x) is None and f.quantize(3) is None and f.quantize(x, x) is None
    assert f.dequantize(q, s, 1) is None and f.dequantize(q, s, -1) is None
    assert f.dequantize(q, s, "bf16") is None
    assert f.conv1x1(q, s, q, s, None, None, 1, 1) is None
    assert f.conv1x1(q, s, q, s, None, None, -1, 7) is None


_CHILD = """
import sys
sys.path.insert(0, {root!r})
import torch
import x1_conv_bn_b200 as X
f = X._compiled()
assert f.raises(16) is None and f.raises(torch.zeros(3)) is None
try:
    f.raises(1 << 62)  # no allocator has this
except (RuntimeError, MemoryError) as e:
    print("allocation:", type(e).__name__)
def inside(t):
    try:
        f.raises(t)  # a vmap's tensors have no storage of their own
    except RuntimeError as e:
        print("address:", type(e).__name__)
    return t
torch.vmap(inside)(torch.zeros(2, 3))
"""


def test_marshalling_module_raises():
    """A C++ exception in the compiled marshalling arrives as a Python one."""
    import os
    import subprocess
    import sys

    from x1_conv_bn_b200 import _build

    _build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CHILD.format(root=root)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr)
    assert r.stdout.split("\n")[:2] == ["allocation: RuntimeError", "address: RuntimeError"], r.stdout


def test_binding_refuses_gradients():
    """No call has a backward pass: what autograd would have to record is refused
    by name, and runs (here as far as the check for a GPU) without grad mode."""
    x, q = torch.zeros(1, 2, 2, 32), torch.zeros(1, 2, 2, 16, dtype=torch.uint8)
    s, v = torch.zeros(1, 1, 32, 16, dtype=torch.uint8), torch.zeros(32)
    p = lambda t: torch.nn.Parameter(t.clone())  # noqa: E731
    norms = (X.group_norm_act, lambda *a, **k: X.group_norm_act_i8(*a, 1.0, **k), X.group_norm_act_mx4)
    calls = [("x", lambda: X.x1cb_quantize_mx4(p(x))),
             ("out", lambda: X.x1cb_dequantize_mx4(q, s, dtype=torch.float32, out=p(x))),
             ("bias", lambda: X.conv1x1_bias_add_act_mx4(q, s, q[0, 0], s, p(v[:2]))),
             ("r", lambda: X.conv1x1_bias_add_act_mx4(q, s, q[0, 0], s, None, p(x))),
             ("out", lambda: X.group_norm_act(x, None, None, 4, out=p(x)))]
    for n in norms:
        calls += [("x", lambda n=n: n(p(x), None, None, 4)), ("gamma", lambda n=n: n(x, p(v), None, 4)),
                  ("beta", lambda n=n: n(x, None, p(v), 4)), ("r", lambda n=n: n(x, None, None, 4, r=p(x)))]
    for name, call in calls:
        with pytest.raises(ValueError, match=f"^{name} requires grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError) as e:
            call()
        assert "requires grad" not in str(e.value)


def test_marshalling_module_of_another_torch_is_rebuilt(tmp_path, monkeypatch):
    """The module is out of date where it was built for another torch, whatever
    its times; the built one says what it was built for."""
    import shutil

    from x1_conv_bn_b200 import _build

    _build.build()
    assert _build.binding_up_to_date()
    assert torch.__version__ in X._compiled().built_for
    copy = tmp_path / "_x1cb_torch.so"
    shutil.copy2(_build.BINDING, copy)
    monkeypatch.setattr(_build, "BINDING", str(copy))
    assert _build.binding_up_to_date()
    ran = []
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".1")
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or _Failed)
    assert not _build.binding_up_to_date()
    with pytest.raises(RuntimeError):
        _build.build_binding()
    assert ran and any(torch.__version__ in a for a in ran[0])


class _Failed:
    returncode, stdout, stderr = 1, "", ""
