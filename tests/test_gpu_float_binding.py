"""The floating-point calls where the binding cannot serve them: no memory for
a result, tensors without memory of their own.  In child processes, which have
to end normally."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from x1_conv_bn_b200 import _build

    _build.build()


def _child(code):
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr)


def test_out_of_memory():
    """Within 1 GiB (the allocator's own limit), every call whose result does not
    fit raises torch's error, and the next one that fits works."""
    _child("""
import torch
import x1_conv_bn_b200 as X
total = torch.cuda.get_device_properties(0).total_memory
torch.cuda.set_per_process_memory_fraction((1 << 30) / total)
u8 = dict(dtype=torch.uint8, device="cuda")
x = torch.ones(1, 475, 1024, 512, device="cuda")  # 950 MiB
g = torch.ones(512, device="cuda")
calls = [lambda: X.group_norm_act(x, g, g, 32), lambda: X.group_norm_act_i8(x, g, g, 32, 1.0),
         lambda: X.group_norm_act_mx4(x, g, g, 32), lambda: X.x1cb_quantize_mx4(x)]
def fails(call):
    try:
        call()
    except torch.OutOfMemoryError:
        return
    raise SystemExit("no error")
for c in calls:
    fails(c)
small = x[:, :1].clone()
del x, calls
q, sf = X.x1cb_quantize_mx4(small)
w, ws = X.x1cb_quantize_mx4(g.expand(1 << 16, 512).contiguous().to(torch.bfloat16))
q = q.view(1, 1024, 1, 256).expand(16, 1024, 1, 256).contiguous()
sf = sf.expand(16, *sf.shape).reshape(-1, *sf.shape[1:]).contiguous()
fails(lambda: X.conv1x1_bias_add_act_mx4(q, sf, w, ws))  # 2 GiB
del w, ws
q = torch.zeros(1 << 20, 512, **u8)
sf = torch.zeros(X.mx4_scale_shape(1 << 20, 1024), **u8)
fails(lambda: X.x1cb_dequantize_mx4(q, sf))  # 2 GiB
assert (X.group_norm_act(small, None, g, 32) == 1).all()
torch.cuda.synchronize()
""")


def test_tensors_without_memory():
    """Inside vmap, and for sparse and nested tensors, the calls raise."""
    _child("""
import torch
import x1_conv_bn_b200 as X
x = torch.ones(2, 1, 4, 4, 64, device="cuda")
q, sf = X.x1cb_quantize_mx4(x[0])
qq, ss = torch.stack((q, q)), torch.stack((sf, sf))
w, ws = X.x1cb_quantize_mx4(torch.ones(32, 64, device="cuda"))
for f, args in ((lambda t: X.group_norm_act(t, None, None, 8), (x,)),
                (lambda t: X.group_norm_act_i8(t, None, None, 8, 1.0), (x,)),
                (lambda t: X.group_norm_act_mx4(t, None, None, 8), (x,)),
                (lambda t: X.group_norm_act(x[0], None, None, 8, r=t), (x,)),
                (X.x1cb_quantize_mx4, (x,)),
                (X.x1cb_dequantize_mx4, (qq, ss)),
                (lambda a, b: X.conv1x1_bias_add_act_mx4(a, b, w, ws), (qq, ss))):
    try:
        torch.vmap(f)(*args)
    except RuntimeError as e:
        assert "storage" in str(e), e
    else:
        raise SystemExit("no error")
for t in (x[0].to_sparse(), torch.nested.nested_tensor([x[0, 0], x[1, 0]])):
    for f in (X.x1cb_quantize_mx4, lambda t: X.group_norm_act(t, None, None, 8)):
        try:
            f(t)
        except (RuntimeError, ValueError, NotImplementedError):
            continue
        raise SystemExit("no error")
torch.cuda.synchronize()
""")


def test_gradients_are_refused():
    """An operand that requires grad is refused while grad mode is on, and served
    without it with the same results."""
    import x1_conv_bn_b200 as X

    p = lambda t: torch.nn.Parameter(t.clone())  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(2, 5, 5, 64, generator=g, device="cuda")
    v = torch.randn(64, generator=g, device="cuda")
    q, sf = X.x1cb_quantize_mx4(x)
    w, ws = X.x1cb_quantize_mx4(torch.randn(64, 64, generator=g, device="cuda"))
    conv = lambda b, r: X.conv1x1_bias_add_act_mx4(q, sf, w, ws, b, r, dtype=torch.float32)  # noqa: E731
    cases = [(lambda a: X.group_norm_act(a, v, v, 8), x), (lambda a: X.group_norm_act(x, a, v, 8), v),
             (lambda a: X.group_norm_act(x, v, a, 8), v), (lambda a: X.group_norm_act(x, v, v, 8, r=a), x),
             (lambda a: X.group_norm_act_i8(a, v, v, 8, 30.0), x),
             (lambda a: X.group_norm_act_mx4(x, a, v, 8)[0], v), (lambda a: X.x1cb_quantize_mx4(a)[1], x),
             (lambda a: conv(a, None), v), (lambda a: conv(None, a), x)]
    for f, t in cases:
        want = f(t)
        with pytest.raises(ValueError, match="requires grad"):
            f(p(t))
        for off in (torch.no_grad, torch.inference_mode):
            with off():
                got = f(p(t))
                assert not got.requires_grad and torch.equal(got, want)
        assert torch.equal(f(p(t).detach()), want)
