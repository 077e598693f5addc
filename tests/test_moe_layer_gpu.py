"""The router, the dispatch, the experts' products and the combine together, as
a layer uses them, forward and back: every stage against its 64-bit
implementation on the data the stage before delivered; the same run captured
into a graph, on other streams, and two at once."""
import numpy as np
import pytest

import moe_ref
import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


class Layer:
    """One layer's weights, buffers and plan; `run` is its forward pass with no allocation."""

    def __init__(self, ep, T, H, I, E, R, k, seed=0, capacity=0, score="sigmoid", device="cuda"):
        self.ep, self.T, self.H, self.I, self.E, self.k = ep, T, H, I, E, k
        g = torch.Generator(device=device).manual_seed(seed)
        e = lambda *s, d=torch.float32: torch.empty(s, dtype=d, device=device)   # noqa: E731

        def q(*s):
            x = torch.randn(*s, generator=g, device=device) * 100
            return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.w1, self.w2 = q(E, 2 * I, H), q(E, H, I)
        self.s1 = (torch.rand(E, 2 * I // 128, H // 128, generator=g, device=device) + 0.5) / (100 * H ** 0.5)
        self.s2 = (torch.rand(E, (H + 127) // 128, I // 128, generator=g, device=device) + 0.5) / (100 * I ** 0.5)
        self.bias = torch.randn(E, generator=g, device=device) * 0.05
        self.router = ep.make_router(E, k, score, num_groups=4, topk_groups=2, renormalize=True, scale=1.5)
        self.shape = ep.make_shape(T, H, E, R, 1, k, ep.EP_FMT_FP8_S128, ep.EP_FMT_BF16, capacity)
        self.R, self.M = R, capacity
        self.ws = ep.Workspace(self.shape, device)
        rows = self.shape.rows
        self.x, self.z = e(T, H, d=torch.bfloat16), e(T, E)
        self.idx, self.w = e(T, k, d=torch.int64), e(T, k)
        self.xq, self.xs = e(T, H, d=torch.uint8), e(T, H // 128)
        self.recv, self.recv_s = torch.zeros(rows, H, dtype=torch.uint8, device=device), e(rows, H // 128)
        self.src, self.rw = e(rows, d=torch.int32), e(rows)
        self.slot, self.off = e(T, k, d=torch.int32), e(E + 1, d=torch.int32)
        self.h, self.hs = torch.zeros(rows, I, dtype=torch.uint8, device=device), e(rows, I // 128)
        self.y = torch.zeros(rows, H, dtype=torch.bfloat16, device=device)
        self.out = e(T, H, d=torch.bfloat16)
        self.dy, self.dexp = e(T, H, d=torch.bfloat16), torch.zeros(rows, H, dtype=torch.bfloat16, device=device)
        self.dw, self.dz = e(T, k), e(T, E)

    def fill(self, seed, masked=0.0):
        g = torch.Generator(device=self.x.device).manual_seed(seed + 77)
        self.x.copy_(torch.randn(self.T, self.H, generator=g, device=self.x.device))
        self.z.copy_(torch.randn(self.T, self.E, generator=g, device=self.x.device))
        self.z[torch.rand(self.T, generator=g, device=self.x.device) < masked] = -float("inf")
        self.dy.copy_(torch.randn(self.T, self.H, generator=g, device=self.x.device))

    def run(self, stream=None):
        ep, kw = self.ep, dict(num_ranks=self.R, rank_capacity=self.M, stream=stream)
        ep.ep_route(self.router, self.z, self.bias, self.idx, self.w, stream)
        ep.ep_quant_fp8_s128(self.x, self.xq, self.xs, stream)
        ep.ep_dispatch(self.shape, self.xq, self.xs, self.idx, self.w, self.recv, self.recv_s, self.src, self.rw,
                       self.slot, self.off, self.ws, stream)
        ep.ep_expert_gated(self.off, self.recv, self.recv_s, self.w1, self.s1, self.h, self.hs, **kw)
        ep.ep_expert_gemm(self.off, self.h, self.hs, self.w2, self.s2, self.y, **kw)
        ep.ep_combine(self.shape, self.y, None, self.slot, self.w, self.out, stream)
        ep.ep_combine_backward(self.shape, self.dy, self.y, self.slot, self.w, self.dexp, self.dw, stream)
        ep.ep_route_backward(self.router, self.z, self.idx, self.dw, self.dz, stream)

    def results(self):
        live = self.slot[self.slot >= 0].long()
        return [t.clone() for t in (self.idx, self.w, self.out, self.dw, self.dz, self.y[live], self.dexp[live])]


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


SIZES = [dict(T=1, H=256, I=128, E=8, R=2, k=2), dict(T=57, H=384, I=256, E=16, R=4, k=3),
         dict(T=300, H=512, I=384, E=32, R=4, k=4), dict(T=90, H=256, I=128, E=16, R=4, k=3, capacity=40),
         dict(T=3000, H=256, I=256, E=8, R=1, k=4, score="softmax")]


@pytest.mark.parametrize("size", SIZES, ids=lambda d: f"T{d['T']}E{d['E']}M{d.get('capacity', 0)}")
@pytest.mark.parametrize("masked", [0.0, 0.2])
def test_layer_stage_by_stage(ep, size, masked):
    L = Layer(ep, seed=size["T"], **size)
    L.fill(size["T"], masked)
    L.run()
    torch.cuda.synchronize()
    n = lambda t: t.cpu().numpy()   # noqa: E731
    score = size.get("score", "sigmoid")
    z = n(L.z).astype(np.float64)
    idx, w = moe_ref.route(z, L.k, score, n(L.bias).astype(np.float64), 4, 2, 2, True, 1.5)
    np.testing.assert_array_equal(n(L.idx), idx)
    assert (np.abs(n(L.w) - w) <= moe_ref.F32_HALF * w * 1.0001).all()

    h, err, valid = moe_ref.gated(n(L.off), n(L.recv), n(L.recv_s), n(L.w1), n(L.s1), L.R, L.M)
    moe_ref.check_quantised(n(L.h), n(L.hs), h, err, valid)
    assert valid.sum() == (n(L.slot) >= 0).sum() and (masked or L.M or valid.sum() == L.T * L.k)
    y, mag, _ = moe_ref.product(n(L.off), n(L.h), n(L.hs), n(L.w2), n(L.s2), L.R, L.M)
    err = moe_ref.sum_error_8bit(mag, L.I)
    got = L.y.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - y) <= moe_ref.BF16_HALF * (np.abs(y) + err) + err)[valid].all()
    assert (got[~valid] == 0).all()
    want = oracle.combine_bf16(_bits(L.y), n(L.slot), n(L.w))
    np.testing.assert_array_equal(_bits(L.out), want)
    # the tokens' rows and their experts fit together: every token's row is the dispatch of its own row
    live = n(L.slot) >= 0
    assert (n(L.recv)[n(L.slot)[live]] == n(L.xq)[np.nonzero(live)[0]]).all()

    dy = L.dy.double().cpu().numpy()
    at = np.clip(n(L.slot), 0, None)
    p = dy[:, None] * got[at]
    gw = np.where(live, p.sum(2), 0)
    assert (np.abs(n(L.dw) - gw) <= L.H * moe_ref.F32_HALF * np.abs(p).sum(2)).all()
    dz = moe_ref.route_backward(z, n(L.idx), n(L.dw).astype(np.float64), score, True, 1.5)
    noise = 1e-13 * 1.5 * np.abs(n(L.dw)).sum(1, keepdims=True)
    assert (np.abs(n(L.dz) - dz) <= moe_ref.F32_HALF * np.abs(dz) + noise + 2.0 ** -150).all()


@pytest.mark.parametrize("size", [SIZES[1], SIZES[2], SIZES[4]], ids=lambda d: f"T{d['T']}")
def test_layer_in_a_graph(ep, size):
    """Captured once, replayed over new inputs (all tokens masked among them), with eager work and
    synchronisations between the replays; every replay equals the eager run to the bit."""
    L = Layer(ep, seed=3, **size)
    ref = Layer(ep, seed=3, **size)
    L.fill(0)
    L.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        L.run()
    torch.cuda.synchronize()
    for i, masked in enumerate((0.0, 0.3, 1.0, 0.0, 0.1, 0.0)):
        L.fill(i, masked)
        ref.fill(i, masked)
        torch.cuda.synchronize()
        g.replay()
        ref.run()
        torch.cuda.synchronize()
        for a, b in zip(L.results(), ref.results()):
            assert torch.equal(a, b), i
        ref.x.normal_()
        torch.cuda.synchronize()


def test_two_graphs_and_two_streams_at_once(ep):
    """Layers that share nothing but the library run on two streams and from two graphs at the same
    time; nothing of one reaches the other."""
    size = dict(T=200, H=512, I=256, E=16, R=4, k=3)
    A, B = Layer(ep, seed=1, **size), Layer(ep, seed=2, **size)
    want = []
    for L, seed in ((A, 10), (B, 11)):
        L.fill(seed, 0.1)
        L.run()
        torch.cuda.synchronize()
        want.append(L.results())
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        A.run(sa)
        B.run(sb)
    torch.cuda.synchronize()
    for L, ref in ((A, want[0]), (B, want[1])):
        assert all(torch.equal(a, b) for a, b in zip(L.results(), ref))
    graphs = []
    for L, s in ((A, sa), (B, sb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            L.run()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(4):
        for t in (A.out, B.out, A.dz, B.dz):
            t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, (sa, sb)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for L, ref in ((A, want[0]), (B, want[1])):
            assert all(torch.equal(a, b) for a, b in zip(L.results(), ref))


def test_allocating_forms_on_another_stream(ep):
    """The allocating forms with a stream of their own: results equal those of the current stream."""
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(64, 32, generator=g, device="cuda")
    r = ep.make_router(32, 4, "softmax")
    a = (torch.randn(64, 256, generator=g, device="cuda") * 100).to(torch.float8_e4m3fn).view(torch.uint8)
    w = (torch.randn(2, 256, 256, generator=g, device="cuda") * 100).to(torch.float8_e4m3fn).view(torch.uint8)
    a_s, w_s = torch.rand(64, 2, device="cuda") / 100, torch.rand(2, 2, 2, device="cuda") / 100
    off = torch.tensor([0, 20, 64], dtype=torch.int32, device="cuda")
    shape = ep.make_shape(32, 256, 2, 1, 1, 2)
    slot = torch.arange(64, dtype=torch.int32, device="cuda").view(32, 2)
    tw = torch.rand(32, 2, device="cuda")
    dy = torch.randn(32, 256, generator=g, device="cuda").to(torch.bfloat16)

    def everything(stream):
        idx, wt = ep.route(z, r, stream=stream)
        dz = ep.route_backward(wt, z, idx, r, stream=stream)
        y = ep.expert_gemm(off, a, a_s, w, w_s, stream=stream)
        q, s = ep.expert_gated(off, a, a_s, w, w_s, stream=stream)
        ge, gw = ep.combine_backward(dy, y, ep.Handle(shape, slot, off, tw), stream=stream)
        return idx, wt, dz, y, q, s, ge, gw
    want = everything(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = everything(side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_refusals_on_the_device(ep):
    """Strided tensors and tensors of the host among device ones are refused."""
    r = ep.make_router(16, 2)
    z = torch.randn(8, 32, device="cuda")[:, ::2]
    with pytest.raises(ValueError, match="contiguous"):
        ep.route(z, r)
    z = torch.randn(8, 16, device="cuda")
    with pytest.raises(ValueError, match="device tensor"):
        ep.ep_route(r, z, torch.zeros(16), torch.zeros(8, 2, dtype=torch.int64).cuda(), torch.zeros(8, 2).cuda())
    with pytest.raises(RuntimeError, match="invalid argument"):
        ep.route(torch.randn(8, 15, device="cuda"), ep.make_router(15, 2, num_groups=4, topk_groups=2))
    a = torch.zeros(10, 256, dtype=torch.uint8, device="cuda")
    x = torch.zeros(10 * 256 + 8, dtype=torch.uint8, device="cuda")[8:].view(10, 256)
    a_s, w_s = torch.ones(10, 2, device="cuda"), torch.ones(2, 2, 2, device="cuda")
    w = torch.zeros(2, 256, 256, dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 5, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError, match="aligned"):
        ep.expert_gemm(off, x, a_s, w, w_s)
    with pytest.raises(RuntimeError, match="invalid argument"):
        ep.expert_gemm(off, a, a_s, w, w_s, num_ranks=2, rank_capacity=4)
    assert (ep.expert_gemm(off, a, a_s, w, w_s) == 0).all()
