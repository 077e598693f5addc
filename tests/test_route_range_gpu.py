"""The router at the ends of its ranges: scores at the bottom of binary64, one
rounding of the gradient to bf16, and the largest batches."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

F32_HALF, BF16_HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _shares(z):
    """e^z over its sum, in 64 bits: what renormalised weights are where 1 + e^z is 1, and for a softmax always."""
    e = np.exp(z - z.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _low_logits(E):
    """Logits where e^-z has left binary64 (from -709.8 on) and e^z has not (until -745), and the three best experts."""
    z = np.full((4, E), -2000.0, np.float32)
    z[0, :6] = [-720, -715, -712, -718, -711, -730]
    z[1, :6] = [-744, -743, -742, -741, -740, -739]
    z[2, 6:12] = [-700, -709, -709.5, -710, -710.5, -725]
    z[3, :6] = [-2000, -740, -2000, -742, -2000, -735]
    return z, np.array([[4, 2, 1], [5, 4, 3], [6, 7, 8], [5, 1, 3]])


@pytest.mark.parametrize("E", [12, 1500])   # scores kept in registers, and computed again
def test_order_of_the_smallest_sigmoid_scores(ep, E):
    z, want = _low_logits(E)
    idx, w = ep.route(torch.from_numpy(z).cuda(), ep.make_router(E, 3, "sigmoid"))
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    assert (w == 0).all()                            # below all of binary32


@pytest.mark.parametrize("E", [12, 1500])
def test_shares_of_the_smallest_sigmoid_scores(ep, E):
    z, want = _low_logits(E)
    idx, w = ep.route(torch.from_numpy(z).cuda(), ep.make_router(E, 3, "sigmoid", renormalize=True))
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    ref = _shares(np.take_along_axis(z, want, 1).astype(np.float64))
    assert (np.abs(w.cpu().double().numpy() - ref) <= F32_HALF * ref + 1e-12).all()


@pytest.mark.parametrize("E", [40, 1500])
def test_softmax_shares_of_experts_far_below_the_largest(ep, E):
    """A bias takes experts whose scores are subnormal, or 0, against the largest logit; their shares stay exact."""
    z = np.full((5, E), -3000.0, np.float32)
    z[:, 0] = 0
    z[:, 30:33] = [[-600, -601, -602.5], [-700, -701, -702.5], [-735, -737, -738.5], [-743, -744, -744.5],
                   [-800, -801, -802]]
    bias = torch.zeros(E)
    bias[30:33] = torch.tensor([4.0, 3.0, 2.0])
    r = ep.make_router(E, 3, "softmax", renormalize=True)
    idx, w = ep.route(torch.from_numpy(z).cuda(), r, bias.cuda())
    assert (idx.cpu() == torch.tensor([30, 31, 32])).all()
    ref = _shares(z[:, 30:33].astype(np.float64))
    assert (np.abs(w.cpu().double().numpy() - ref) <= F32_HALF * ref + 1e-12).all()


@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
def test_gradient_of_shares_at_the_bottom_of_binary64(ep, score):
    """With shares q the gradient is q (g - <g, q>): 1 - p is 1 here for a sigmoid."""
    z = np.array([[-720, -715, -712], [-744, -743, -742.5], [-700, -709.5, -712], [-600, -602, -601]], np.float32)
    g = np.array([[1, -2, 0.5], [3, 1, -1], [0.25, 1, 2], [1, 2, 3]], np.float32)
    idx = torch.arange(3).repeat(4, 1)
    r = ep.make_router(3, 3, score, renormalize=True)
    dz = ep.route_backward(torch.from_numpy(g).cuda(), torch.from_numpy(z).cuda(), idx.cuda(), r)
    q = _shares(z.astype(np.float64))
    ref = q * (g - (g * q).sum(1, keepdims=True))
    assert (np.abs(dz.cpu().double().numpy() - ref) <= F32_HALF * np.abs(ref) + 1e-12).all()


def _bf16_nearest(x):
    """Positive binary64 values to the nearest bf16, ties to even, in one rounding."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256), e - 8)         # 8 bits; rint goes to even


def test_bf16_gradient_is_rounded_once(ep):
    """Gradients just above and just below the middle of two bf16 values, by less than a step of binary32."""
    rng = np.random.default_rng(3)
    g, s = rng.uniform(1, 2, 1 << 21).astype(np.float32), np.float32(1 + 5 * 2.0 ** -23)
    x = g.astype(np.float64) * float(s) / 4          # z = 0: p (1 - p) = 1 / 4, exact
    twice = _bf16_nearest(x.astype(np.float32).astype(np.float64))
    g = np.concatenate([g[twice != _bf16_nearest(x)], [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]]).astype(np.float32)
    want = _bf16_nearest(g.astype(np.float64) * float(s) / 4)
    assert g.size > 4                                # the draw holds such values
    z = torch.zeros(g.size, 2, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(g.size, 1, dtype=torch.int64, device="cuda")
    for sign in (1, -1):
        r = ep.make_router(2, 1, "sigmoid", scale=sign * float(s))
        dz = ep.route_backward(torch.from_numpy(g)[:, None].cuda(), z, idx, r).cpu().double().numpy()
        np.testing.assert_array_equal(dz[:, 0], sign * want)
        assert (dz[:, 1] == 0).all()
    # the ends of bf16: subnormals, overflow, infinities and NaN
    g = torch.tensor([2.0 ** -131, 1.25 * 2.0 ** -131, 3 * 2.0 ** -132, 2.0 ** -136, 3.3e38, math.inf, -math.inf,
                      math.nan, 0.0]).cuda()
    r = ep.make_router(2, 1, "sigmoid", scale=4.0)
    dz = ep.route_backward(g[:, None].contiguous(), z[:9], idx[:9], r)[:, 0]
    want = g.to(torch.bfloat16)
    assert torch.equal(dz.isnan(), want.isnan()) and torch.equal(dz.nan_to_num(), want.nan_to_num())
    r = ep.make_router(2, 1, "sigmoid", scale=8.0)
    assert torch.isinf(ep.route_backward(g[4:5, None].contiguous(), z[:1], idx[:1], r)[0, 0])


@pytest.mark.parametrize("T", [2 ** 26 - 4, 2 ** 26 - 3, 2 ** 26 - 1])
def test_largest_batches(ep, T):
    """Every documented number of tokens: launches of up to 2^32 threads less some."""
    z = torch.empty(T, 2, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    r = ep.make_router(2, 1, "softmax")
    idx, w = ep.route(z, r)
    assert torch.equal(idx[:, 0], (z[:, 1] > z[:, 0]).long())
    d = (z[:, 0].double() - z[:, 1].double()).abs()
    p = 1 / (1 + torch.exp(-d))
    assert ((w[:, 0].double() - p).abs() <= F32_HALF * p + 1e-14).all()
    del idx, w, p, d
    g = torch.ones(T, 1, device="cuda")
    idx = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    dz = ep.route_backward(g, z, idx, r)
    d = z[:, 0].double() - z[:, 1].double()
    want = 1 / (1 + torch.exp(-d)) / (1 + torch.exp(d))
    del d, idx, g
    for i, sign in ((0, 1), (1, -1)):
        assert ((dz[:, i].double() - sign * want).abs() <= BF16_HALF * (1 + 1e-6) * want + 2.0 ** -133).all()
