"""A gradient given in fp32 enters every product with its precision: sums that
cancel show what is lost of their terms.  In each launch form of the products."""
import pytest

import dense_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LOST = 2.0 ** -17   # of a term, in two bf16 parts that are both rounded to nearest


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _inputs(M, K, N, gated, act, seed=0):
    """Neighbouring columns of dy nearly alike, weights of opposite signs for them; the same over rows, for x."""
    g = torch.Generator().manual_seed(seed + M + 3 * K + 7 * N)
    rand = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    wide = 2 * N if gated else N
    dy = (1 + torch.rand((M + 1) // 2, N // 2, generator=g)).repeat_interleave(2, 0)[:M].repeat_interleave(2, 1)
    dy = dy * (1 + 2.0 ** -12 * rand(M, N))
    w = rand(wide // 2, K).sign().repeat_interleave(2, 0)
    w[1::2] *= -1
    x = rand((M + 1) // 2, K).sign().repeat_interleave(2, 0)
    x[1::2] *= -1
    z = rand(1, wide).expand(M, wide).contiguous().to(BF) if act or gated else None
    return dy, x[:M].to(BF), w.to(BF), z


def _want(dy, x, w, z, act, gated, lost_x, lost_w):
    (gx, ex), (gw, ew), (gb, eb) = ref.linear_backward(dy, x, w, z, act, gated, 0)
    d = dy.double()
    if gated:
        n = dy.shape[1]
        g, u = z.double()[:, :n], z.double()[:, n:]
        d = torch.cat((d * u * ref.slope(g, act), d * ref.value(g, act)), 1)
    elif act is not None:
        d = d * ref.slope(z.double(), act)
    # the parts follow each other in the sums: up to three times the steps
    ax, aw = d.abs() @ w.double().abs(), d.abs().T @ x.double().abs()
    ex = ex + lost_x * ax + ref.sum_error(ax, 3 * w.shape[0])
    ew = ew + lost_w * aw + ref.sum_error(aw, 3 * x.shape[0])
    return (gx, ex), (gw, ew), (gb, eb)


SIZES = [(1, 8, 8), (6, 64, 32), (100, 520, 136), (130, 264, 1032), (341, 72, 64), (700, 1048, 264), (1500, 2056, 520),
         (2048, 5128, 264)]


@pytest.mark.parametrize("M,K,N", SIZES, ids=str)
@pytest.mark.parametrize("act,gated", [(None, False), ("silu", True), ("gelu", False), (None, True)])
@pytest.mark.parametrize("w32", [False, True], ids=["bf16", "fp32"])
def test_fp32_gradient(ep, M, K, N, act, gated, w32):
    dy, x, w, z = _inputs(M, K, N, gated, act)
    kw = dict(activation=act, gated=gated)
    dtype = F32 if w32 else BF
    c = [None if t is None else t.cuda() for t in (dy, x, w, z)]
    got = ep.linear_backward(*c, bias=True, grad_w_dtype=dtype, **kw)
    want = _want(dy, x, w, z, act, gated, LOST, 0 if w32 else LOST)
    for v, (t, e), half in zip(got, want, (ref.BF16_HALF, ref.F32_HALF if w32 else ref.BF16_HALF, ref.F32_HALF)):
        ref.check(v.cpu(), t, e, half)
    # each by itself has the same bits, of a type that the others do not change
    ws = torch.empty(ep.linear_backward_workspace_bytes(M, K, N, act, gated, F32, dtype), dtype=torch.uint8,
                     device="cuda")
    for i in range(3):
        out = [None, None, None]
        out[i] = torch.full_like(got[i], 7)
        ws.random_()
        ep.ep_linear_backward(*c, *out, ws, act, gated)
        assert torch.equal(out[i], got[i])


def test_far_apart(ep):
    """Values of every size, at the ends of the types: the parts stay finite where the gradient is."""
    vals = torch.tensor([3.4e38, -3.4e38, 1e-38, -1e-40, 1.0, 3.3961775e38, 2.0 ** -126, 0.0])
    N = len(vals)
    w = torch.zeros(N, 8)
    w[torch.arange(N), torch.arange(N)] = 2.0 ** -8
    gx, gw = ep.linear_backward(vals[None].cuda(), torch.ones(1, 8, dtype=BF, device="cuda"), w.to(BF).cuda())
    want = vals.double() * 2.0 ** -8
    ok = (gx.cpu().double()[0] - want).abs() <= (LOST + ref.BF16_HALF) * want.abs() + 2.0 ** -132
    assert ok.all(), gx
    small = vals.abs() < 1e38   # the others round to bf16's infinity or its largest number
    ref.check(gw.cpu()[small], vals[small, None].double().expand(-1, 8), 0.0, LOST + ref.BF16_HALF)
