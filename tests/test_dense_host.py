"""The dense product with its backward pass and the experts' layer for a few
tokens on the host (no GPU): every argument error is found before anything is
enqueued, an empty call succeeds without touching a pointer, the Python layer
refuses wrong dtypes, shapes and devices.  The 64-bit implementations that the
GPU tests compare with are checked against differences and each other."""
import ctypes

import pytest
import torch

import dense_ref
from combine_dispatch_layout_02_amd import ep

P = ctypes.c_void_p
FAKE, ODD = P(0x1000), P(0x1008)   # never dereferenced: the host checks come first
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    return ep.load()


def _few(T=4, H=256, I=128, E=8, k=2, fmt=ep.EP_FMT_FP8_S128):   # noqa: E741
    return ep.ep_few_shape(T, H, I, E, k, fmt)


def _few_args(lib, sh, ws=FAKE, nbytes=BIG, **bad):
    args = dict(x=FAKE, idx=FAKE, w=FAKE, up=FAKE, up_s=FAKE, down=FAKE, down_s=FAKE, r=None, y=FAKE)
    args.update(bad)
    return lib.ep_moe_few(None if sh is None else ctypes.byref(sh), *args.values(), ws, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=65), dict(E=0), dict(E=4097), dict(k=0), dict(k=33), dict(H=0), dict(H=64), dict(H=192),
    dict(I=0), dict(I=200), dict(H=2 ** 20 + 128), dict(I=2 ** 20 + 128), dict(fmt=2), dict(fmt=-1),
    dict(fmt=ep.EP_FMT_BF16, H=12), dict(fmt=ep.EP_FMT_BF16, I=4), dict(T=64, k=32, I=2 ** 17)])
def test_few_shapes_refused(lib, bad):
    sh, n = _few(**bad), ctypes.c_size_t()
    assert _few_args(lib, sh) == ep.EP_EINVAL
    assert lib.ep_moe_few_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == ep.EP_EINVAL


def test_few_arguments(lib):
    sh = _few()
    assert _few_args(lib, None) == ep.EP_EINVAL
    assert lib.ep_moe_few(ctypes.byref(_few(T=0)), *[None] * 10, 0, None) == ep.EP_OK
    for name in ("x", "idx", "w", "up", "up_s", "down", "down_s", "y"):
        assert _few_args(lib, sh, **{name: None}) == ep.EP_EINVAL, name
    for name in ("x", "up", "down", "r", "y"):
        assert _few_args(lib, sh, **{name: ODD}) == ep.EP_EALIGN, name
    bf = _few(fmt=ep.EP_FMT_BF16)
    assert _few_args(lib, bf) == ep.EP_EINVAL                       # scales with bf16 weights
    assert _few_args(lib, bf, up_s=None, down_s=None, ws=None) == ep.EP_EWORKSPACE
    n = ctypes.c_size_t()
    assert lib.ep_moe_few_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == ep.EP_OK
    assert n.value == ep.moe_few_workspace_bytes(4, 256, 128, 8, 2) >= 4 * 2 * 128 * 4
    assert lib.ep_moe_few_workspace_bytes(ctypes.byref(sh), None) == ep.EP_EINVAL
    assert _few_args(lib, sh, nbytes=n.value - 1) == ep.EP_EWORKSPACE
    assert _few_args(lib, sh, ws=P(0x1080)) == ep.EP_EALIGN


def _linear(M=4, K=64, N=32, act=0, gated=0, f32=0, w32=0):
    return ep.ep_linear_shape(M, K, N, act, gated, f32, w32)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(K=0), dict(K=4), dict(K=60), dict(N=0), dict(N=12), dict(K=2 ** 20 + 8), dict(N=2 ** 20 + 8),
    dict(act=-1), dict(act=5), dict(gated=2), dict(f32=-1), dict(w32=2), dict(M=2 ** 29, K=64), dict(M=2 ** 40),
    dict(M=2 ** 16, N=2 ** 20), dict(M=2 ** 15, N=2 ** 19, K=64, gated=1), dict(M=2 ** 16, K=2 ** 20), dict(K=2 ** 18, N=2 ** 18)])
def test_linear_shapes_refused(lib, bad):
    sh, n = _linear(**bad), ctypes.c_size_t()
    assert lib.ep_linear(ctypes.byref(sh), *[FAKE] * 6, None) == ep.EP_EINVAL
    assert lib.ep_linear_backward(ctypes.byref(sh), *[FAKE] * 8, BIG, None) == ep.EP_EINVAL
    assert lib.ep_linear_backward_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == ep.EP_EINVAL


def test_linear_limits(lib):
    """Shapes just inside the launch limits are accepted (an odd pointer tells them from refused ones)."""
    for d in (dict(M=2 ** 21, N=7168, K=7168), dict(M=2 ** 15, N=2 ** 19), dict(M=2 ** 27, K=64, N=64)):
        assert lib.ep_linear(ctypes.byref(_linear(**d)), ODD, *[FAKE] * 5, None) == ep.EP_EALIGN, d


def test_linear_arguments(lib):
    sh = _linear(act=2)
    assert lib.ep_linear(None, *[FAKE] * 6, None) == ep.EP_EINVAL
    assert lib.ep_linear(ctypes.byref(_linear(M=0)), *[None] * 7) == ep.EP_OK
    for i in (0, 1, 4):                     # x, w, y
        args = [FAKE] * 6
        args[i] = None
        assert lib.ep_linear(ctypes.byref(sh), *args, None) == ep.EP_EINVAL
    for i in range(6):
        args = [FAKE] * 6
        args[i] = ODD
        assert lib.ep_linear(ctypes.byref(sh), *args, None) == ep.EP_EALIGN
    back = lib.ep_linear_backward
    assert back(None, *[FAKE] * 8, BIG, None) == ep.EP_EINVAL
    # dy, x, w, z, grad_x, grad_w, grad_bias, ws
    for drop in ([0], [1], [2], [3]):
        args = [FAKE] * 8
        for i in drop:
            args[i] = None
        assert back(ctypes.byref(sh), *args, BIG, None) == ep.EP_EINVAL, drop
    for i in (0, 1, 2, 3, 4, 5):
        args = [FAKE] * 8
        args[i] = ODD
        assert back(ctypes.byref(sh), *args, BIG, None) == ep.EP_EALIGN, i
    assert back(ctypes.byref(sh), *[FAKE] * 7, None, BIG, None) == ep.EP_EWORKSPACE
    assert back(ctypes.byref(sh), *[FAKE] * 7, P(0x1010), BIG, None) == ep.EP_EALIGN
    n = ctypes.c_size_t()
    assert lib.ep_linear_backward_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == ep.EP_OK
    assert n.value == ep.linear_backward_workspace_bytes(4, 64, 32, "silu") >= 4 * 32 * 2
    assert back(ctypes.byref(sh), *[FAKE] * 8, n.value - 1, None) == ep.EP_EWORKSPACE
    assert lib.ep_linear_backward_workspace_bytes(ctypes.byref(sh), None) == ep.EP_EINVAL
    # nothing asked for: nothing is launched
    assert back(ctypes.byref(sh), *[FAKE] * 4, None, None, None, FAKE, BIG, None) == ep.EP_OK


def test_python_layer_refuses():
    f32, bf, u8, i32, i64 = torch.float32, torch.bfloat16, torch.uint8, torch.int32, torch.int64
    z = lambda *s, d=bf: torch.zeros(*s, dtype=d)   # noqa: E731
    few = dict(x=z(4, 128), topk_idx=z(4, 2, d=i64), topk_w=z(4, 2, d=f32), gate_up=z(3, 256, 128, d=u8),
               gate_up_scales=z(3, 2, 1, d=f32), down=z(3, 128, 128, d=u8), down_scales=z(3, 1, 1, d=f32), residual=None,
               y=z(4, 128), ws=z(1024, d=u8))
    for bad in (dict(x=z(4, 128, d=f32)), dict(x=z(4, 120)), dict(x=z(128)), dict(topk_idx=z(4, 2, d=i32)),
                dict(topk_idx=z(3, 2, d=i64)), dict(topk_w=z(4, 2)), dict(topk_w=z(4, 3, d=f32)),
                dict(gate_up=z(3, 255, 128, d=u8)), dict(gate_up=z(3, 256, 128)), dict(gate_up=z(256, 128, d=u8)),
                dict(gate_up_scales=None), dict(down_scales=None), dict(gate_up_scales=z(3, 2, 2, d=f32)),
                dict(down=z(3, 128, 64, d=u8)), dict(down_scales=z(3, 1, 1)), dict(residual=z(4, 120)),
                dict(residual=z(4, 128, d=f32)), dict(y=z(4, 128, d=f32)), dict(y=z(3, 128)), dict(ws=z(1024)), {}):
        with pytest.raises(ValueError):   # {}: tensors of the host
            ep.ep_moe_few(**dict(few, **bad))
    lin = dict(x=z(4, 64), w=z(32, 64), bias=None, residual=None, y=z(4, 32))
    for bad in (dict(x=z(4, 64, d=f32)), dict(x=z(64)), dict(w=z(32, 56)), dict(w=z(32, 64, d=f32)),
                dict(bias=z(32)), dict(bias=z(16, d=f32)), dict(residual=z(4, 32, d=f32)), dict(residual=z(3, 32)),
                dict(y=z(4, 32, d=torch.float16)), dict(y=z(4, 16)), dict(z=z(4, 16)), dict(z=z(4, 32, d=f32)),
                dict(gated=True), dict(activation="tanh"), dict(w=z(31, 64), gated=True), {}):
        with pytest.raises(ValueError):
            ep.ep_linear(**dict(lin, **bad))
    back = dict(dy=z(4, 32), x=z(4, 64), w=z(32, 64), z=None, grad_x=z(4, 64), grad_w=z(32, 64),
                grad_bias=z(32, d=f32), ws=z(4096, d=u8))
    for bad in (dict(dy=z(4, 16)), dict(dy=z(4, 32, d=torch.float16)), dict(activation="silu"), dict(gated=True),
                dict(z=z(4, 16), activation="silu"), dict(grad_x=z(4, 64, d=f32)), dict(grad_w=z(64, 32)),
                dict(grad_w=z(32, 64, d=torch.float16)), dict(grad_bias=z(32)), dict(ws=z(4096)), {}):
        with pytest.raises(ValueError):
            ep.ep_linear_backward(**dict(back, **bad))


def test_reference_slopes_against_differences():
    z = torch.linspace(-9, 9, 181, dtype=torch.float64) + 0.013
    h = 1e-5
    for act in dense_ref.ACTIVATIONS:
        diff = (dense_ref.value(z + h, act) - dense_ref.value(z - h, act)) / (2 * h)
        # h^2 / 6 of third derivatives below 4, and the rounding of values below 10 over 2 h
        assert ((diff - dense_ref.slope(z, act)).abs() < 1e-9).all(), act


def test_reference_values_against_torch():
    z = torch.linspace(-6, 6, 121, dtype=torch.float64)
    F = torch.nn.functional
    for act, want in (("relu", F.relu(z)), ("silu", F.silu(z)), ("gelu", F.gelu(z)),
                      ("gelu_tanh", F.gelu(z, approximate="tanh"))):
        assert torch.allclose(dense_ref.value(z, act), want, rtol=1e-12, atol=1e-14)


def test_reference_gradients_against_autograd():
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    for act, gated in ((None, False), ("silu", True), ("gelu", False), ("relu", True), ("gelu_tanh", False), (None, True)):
        x, w, b = rand(5, 16), rand(24 if gated else 12, 16), rand(24 if gated else 12)
        x, w, b = (t.double().requires_grad_() for t in (x, w, b))
        z = x @ w.T + b
        y = dense_ref.value(z[:, :12], act) * z[:, 12:] if gated else dense_ref.value(z, act)
        dy = rand(5, 12)
        want = torch.autograd.grad(y, (x, w, b), dy.double())
        got = dense_ref.linear_backward(dy, x.detach(), w.detach(), z.detach(), act, gated, 0)
        for (v, _), t in zip(got, want):
            assert torch.allclose(v, t, rtol=1e-10, atol=1e-10)


def test_reference_few_against_linear():
    """One expert for all tokens with weight 1 is two dense products."""
    g = torch.Generator().manual_seed(1)
    x, up, down = (torch.randn(*s, generator=g) for s in ((6, 32), (1, 48, 32), (1, 32, 24)))
    idx, w = torch.zeros(6, 1, dtype=torch.int64), torch.ones(6, 1)
    y, _ = dense_ref.moe_few(x, idx, w, up, None, down, None, x)
    h = dense_ref.linear(x, up[0], None, None, "silu", True)[0]
    assert torch.allclose(y, dense_ref.linear(h, down[0], None, x, None, False)[0], rtol=1e-12)
