"""The lower tails of the activations, where e^z leaves binary32's normal
numbers: by a large factor (a gate's, a gradient) they come back into them, and
keep their precision on the way.  And a closed relu gate beside a large
gradient."""
import math

import pytest

import dense_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# on both sides of where the tail's own form starts, to where e^(z / 2) (or its like) is still a normal number
TAILS = {"silu": [-60.0, -79.5, -80.5, -87.5, -89.0, -96.0, -100.0, -103.0, -104.5, -120.0, -150.0, -173.0],
         "gelu": [-8.0, -11.5, -11.9, -12.1, -12.9, -13.25, -14.0, -14.5, -16.0, -18.5],
         "gelu_tanh": [-8.0, -9.6, -9.75, -10.0, -10.25, -10.5, -11.0, -12.0, -12.75]}
FACTORS = [1.0, -3.0, 1e8, 1e20, -3e38]


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _grid(act):
    """Every tail value beside every factor, as bf16 values; their number is a multiple of 8."""
    z = torch.tensor(TAILS[act]).to(BF).repeat_interleave(len(FACTORS))
    u = torch.tensor(FACTORS).to(BF).repeat(len(TAILS[act]))
    pad = -len(z) % 8
    return torch.cat((z, z[:pad])), torch.cat((u, u[:pad]))


def _error(z, act):
    """Relative.  16 steps of the result: 5 of the library's function at most, twice 1 of the exponential, half of
    each of 4 products and a sum, the rest for the derivative's second term.  And the rounded argument's: erfc's is
    off by 2 halves of a step, which moves it by 2 t^2 = z^2 times that (the exponential's z^2 is exact for a bf16
    z); the cubic's a is off by 7 halves, which moves e^a by |a| times that."""
    cond = torch.zeros_like(z)
    if act == "gelu":
        cond = z * z + 1
    if act == "gelu_tanh":
        cond = 6 * (z.abs() + 0.044715 * z.abs() ** 3)
    return ref.STEP * (16 + cond)


def _close(got, want, rel, half):
    got, err = got.double().cpu(), rel * want.abs()
    # one step of the smallest subnormals, and the rounding to the output's type (bf16's subnormal step is 2^-133)
    tiny = 2.0 ** -149 if half == ref.F32_HALF else 2.0 ** -134 + 2.0 ** -149
    ok = (got - want).abs() <= err + half * (want.abs() + err) + tiny
    assert ok.all(), [(float(got.flatten()[i]), float(want.flatten()[i])) for i in torch.nonzero(~ok.flatten())[:5, 0]]


@pytest.mark.parametrize("act", list(TAILS))
@pytest.mark.parametrize("M", [1, 70])
@pytest.mark.parametrize("dtype,half", [(F32, ref.F32_HALF), (BF, ref.BF16_HALF)], ids=["fp32", "bf16"])
def test_forward(ep, act, M, dtype, half):
    """x picks one weight, so z and u are exactly the weights."""
    z, u = _grid(act)
    x = torch.zeros(M, 8)
    x[:, 3] = 1
    w = torch.zeros(2 * len(z), 8)
    w[:, 3] = torch.cat((z, u)).float()
    x, w = x.to(BF).cuda(), w.to(BF).cuda()
    zd, ud = z.double(), u.double()
    f, rel = ref.value(zd, act), _error(zd, act)
    y = ep.linear(x, w, activation=act, gated=True, out_dtype=dtype)
    _close(y, (f * ud).expand(M, -1), rel, half)
    y = ep.linear(x, w[:len(z)], activation=act, out_dtype=dtype)
    _close(y, f.expand(M, -1), rel, half)


@pytest.mark.parametrize("act", list(TAILS))
@pytest.mark.parametrize("dtype", [F32, BF], ids=["fp32", "bf16"])
def test_backward(ep, act, dtype):
    """The bias' gradient of a single row is dz itself."""
    z, u = _grid(act)
    N = len(z)
    x, w = torch.ones(1, 8, dtype=BF, device="cuda"), torch.ones(2 * N, 8, dtype=BF, device="cuda")
    zd, ud = z.double(), u.double()
    f, d, rel = ref.value(zd, act), ref.slope(zd, act), _error(zd, act)
    for scale in (1.0, 2.0 ** 40, -3.0 * 2.0 ** -20):
        dy = torch.full((1, N), scale, dtype=dtype, device="cuda")
        zz = torch.cat((z, u))[None].cuda()
        ws = torch.empty(ep.linear_backward_workspace_bytes(1, 8, N, act, True, y_dtype=dtype), dtype=torch.uint8,
                         device="cuda")
        gb = torch.empty(2 * N, device="cuda")
        ep.ep_linear_backward(dy, x, w, zz, None, None, gb, ws, act, True)
        got = gb.cpu()
        inside = ((ud * scale).abs() < 3e38) | (zd < {"silu": -80, "gelu": -12, "gelu_tanh": -9.7}[act])
        _close(got[:N][inside], (scale * ud * d)[inside], rel[inside], ref.F32_HALF)
        _close(got[N:], scale * f, rel, ref.F32_HALF)
        gb = torch.empty(N, device="cuda")
        ep.ep_linear_backward(dy, x, w[:N], zz[:, :N].contiguous(), None, None, gb, ws, act)
        _close(gb, scale * d, rel, ref.F32_HALF)


def test_lowest_values(ep):
    """Down to bf16's lowest number the tails and their slopes are 0, not NaN, whatever is beside them."""
    z = torch.tensor([-20.0, -200.0, -1e4, -1e13, -1e20, -3.38e38, -9.75, -174.0]).to(BF)
    u = torch.full((8,), 3e38).to(BF)
    x = torch.ones(1, 8, dtype=BF, device="cuda")
    w = torch.zeros(16, 8, dtype=BF)
    w[:, 0] = torch.cat((z, u))
    for act in TAILS:
        far = (torch.arange(8) < 6) & (torch.arange(8) >= (1 if act == "silu" else 0))
        y = ep.linear(x, w.cuda(), activation=act, gated=True, out_dtype=F32).cpu()[0]
        assert torch.isfinite(y).all()
        assert (y[far] == 0).all()
        dy = torch.full((1, 8), 1e30, device="cuda")
        _, gw, gb = ep.linear_backward(dy, x, w.cuda(), torch.cat((z, torch.ones(8).to(BF)))[None].cuda(), act, True,
                                       bias=True)
        assert torch.isfinite(gb).all() and torch.isfinite(gw).all()
        assert (gb.cpu()[:8][far] == 0).all() and (gb.cpu()[8:][far] == 0).all()


def test_closed_relu_gate(ep):
    """dy u past binary32 behind a closed gate: the gradient is 0, not NaN."""
    z = torch.tensor([-1.0, 0.0, -0.0, -3e38, 2.0, 1e-30, -1e-30, 1.0])
    u = torch.tensor([1e30, -1e30, 3e38, 1e30, 1e5, 1e5, 1e30, -2.0])
    dy = torch.full((1, 8), 1e20, device="cuda")
    x, w = torch.ones(1, 8, dtype=BF, device="cuda"), torch.ones(16, 8, dtype=BF, device="cuda")
    zu = torch.cat((z, u)).to(BF)
    gx, gw, gb = ep.linear_backward(dy, x, w, zu[None].cuda(), "relu", True, bias=True)
    zd, ud = zu[:8].double(), zu[8:].double()
    want = torch.cat((torch.where(zd > 0, 1e20 * ud, 0), 1e20 * zd.clamp(min=0)))
    _close(gb, want, torch.full_like(want, 2 * ref.STEP), ref.F32_HALF)
    assert torch.isfinite(gx).all() and torch.isfinite(gw).all()
