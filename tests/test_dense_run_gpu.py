"""The dense products and the experts' layer for a few tokens together, as a
layer uses them: the router's logits, the choice, the experts and a shared
expert that joins them, for decoding and with its backward pass for training;
every stage against its 64-bit implementation on what the stage before
delivered.  The same runs captured and replayed, on other streams, two at once,
with a workspace in common; tensors past 32 bits; the framework's other chain."""
import pytest

import dense_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


class Block:
    """Router, experts and a shared expert; every buffer of a forward pass for a few tokens, its backward
    pass for the dense parts, and no allocation in either."""

    def __init__(self, ep, T, H, I, S, E, k, fp8, seed=0):   # noqa: E741
        self.ep, self.T = ep, T
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
        e = lambda *s, d=BF: torch.empty(s, dtype=d, device="cuda")   # noqa: E731
        self.router = ep.make_router(E, k, "softmax", renormalize=True)
        self.wr = (rand(E, H) / H ** 0.5).to(BF)
        self.s1, self.s2 = (rand(2 * S, H) / H ** 0.5).to(BF), (rand(H, S) / S ** 0.5).to(BF)
        self.b1 = rand(2 * S) * 0.1
        self.w, self.sc = [], []
        for N, K in ((2 * I, H), (H, I)):
            if fp8:
                self.w.append((rand(E, N, K) * 100).clamp(-448, 448).to(F8).view(torch.uint8))
                self.sc.append((torch.rand(E, -(-N // 128), K // 128, generator=g, device="cuda") + 0.5) / (100 * K ** 0.5))
            else:
                self.w.append((rand(E, N, K) / K ** 0.5).to(BF))
                self.sc.append(None)
        self.x, self.dy, self.dw = e(T, H), e(T, H), e(T, k, d=F32)
        self.z, self.idx, self.tw = e(T, E, d=F32), e(T, k, d=torch.int64), e(T, k, d=F32)
        self.h, self.hz, self.shared, self.y = e(T, S), e(T, 2 * S), e(T, H), e(T, H)
        fmt = ep.EP_FMT_FP8_S128 if fp8 else ep.EP_FMT_BF16
        self.ws = e(ep.moe_few_workspace_bytes(T, H, I, E, k, fmt), d=torch.uint8)
        self.gz = e(T, E, d=F32)
        self.gx = [e(T, H), e(T, H)]
        self.gh = e(T, S)
        self.gwr, self.gs1, self.gs2, self.gb1 = e(E, H, d=F32), e(2 * S, H), e(H, S), e(2 * S, d=F32)
        need = ep.linear_backward_workspace_bytes
        self.bws = e(max(need(T, H, E, y_dtype=F32, grad_w_dtype=F32), need(T, S, H), need(T, H, S, "silu", True)),
                     d=torch.uint8)

    def fill(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed + 99)
        for t in (self.x, self.dy, self.dw):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    def forward(self, stream=None):
        ep = self.ep
        ep.ep_linear(self.x, self.wr, None, None, self.z, stream=stream)
        ep.ep_route(self.router, self.z, None, self.idx, self.tw, stream)
        ep.ep_linear(self.x, self.s1, self.b1, None, self.h, self.hz, "silu", True, stream=stream)
        ep.ep_linear(self.h, self.s2, None, self.x, self.shared, stream=stream)
        ep.ep_moe_few(self.x, self.idx, self.tw, self.w[0], self.sc[0], self.w[1], self.sc[1], self.shared, self.y,
                      self.ws, stream)

    def backward(self, stream=None):
        ep = self.ep
        ep.ep_route_backward(self.router, self.z, self.idx, self.dw, self.gz, stream)
        ep.ep_linear_backward(self.gz, self.x, self.wr, None, self.gx[0], self.gwr, None, self.bws, stream=stream)
        ep.ep_linear_backward(self.dy, self.h, self.s2, None, self.gh, self.gs2, None, self.bws, stream=stream)
        ep.ep_linear_backward(self.gh, self.x, self.s1, self.hz, self.gx[1], self.gs1, self.gb1, self.bws, "silu", True,
                              stream)

    def run(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def outputs(self):
        return [self.z, self.idx, self.tw, self.h, self.hz, self.shared, self.y, self.gz, *self.gx, self.gh, self.gwr,
                self.gs1, self.gs2, self.gb1]

    def results(self):
        return [t.clone() for t in self.outputs()]


#        T, H, I, S, E, k, fp8
SIZES = [(1, 256, 128, 128, 8, 2, True), (5, 384, 256, 136, 24, 3, True), (17, 328, 88, 264, 16, 4, False),
         (33, 512, 128, 1032, 40, 6, True), (64, 1032, 200, 320, 8, 8, False)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_stage_by_stage(ep, size):
    L = Block(ep, *size, seed=size[0])
    L.fill(size[0])
    L.run()
    c = lambda t: None if t is None else t.cpu()   # noqa: E731
    x, h, hz = c(L.x), c(L.h), c(L.hz)
    y, err, _, _ = ref.linear(x, c(L.wr), None, None, None, False)
    ref.check(c(L.z), y, err, ref.F32_HALF)
    best = c(L.z).topk(size[5], 1)
    assert torch.equal(c(L.z).gather(1, c(L.idx)), best.values)
    w = best.values.double().softmax(1)
    assert ((c(L.tw) - w).abs() <= ref.F32_HALF * w * 1.0001).all()
    y, err, z, ez = ref.linear(x, c(L.s1), c(L.b1), None, "silu", True)
    ref.check(h, y, err, ref.BF16_HALF)
    ref.check(hz, z, ez, ref.BF16_HALF)
    y, err, _, _ = ref.linear(h, c(L.s2), None, x, None, False)
    ref.check(c(L.shared), y, err, ref.BF16_HALF)
    y, err = ref.moe_few(x, c(L.idx), c(L.tw), c(L.w[0]), c(L.sc[0]), c(L.w[1]), c(L.sc[1]), c(L.shared))
    ref.check(c(L.y), y, err, ref.BF16_HALF)

    # the router's gradient, in 64 bits: w = softmax over the chosen logits
    dw = c(L.dw).double()
    gz = torch.zeros(size[0], size[4], dtype=torch.float64)
    gz.scatter_(1, c(L.idx), w * (dw - (w * dw).sum(1, keepdim=True)))
    assert ((c(L.gz) - gz).abs() <= ref.F32_HALF * gz.abs() + 1e-13 * dw.abs().sum(1, keepdim=True)).all()
    (gx, ex), (gw, ew), _ = ref.linear_backward(c(L.gz), x, c(L.wr), None, None, False, 3)
    ref.check(c(L.gx[0]), gx, ex, ref.BF16_HALF)
    ref.check(c(L.gwr), gw, ew, ref.F32_HALF)
    (gx, ex), (gw, ew), _ = ref.linear_backward(c(L.dy), h, c(L.s2), None, None, False, 0)
    ref.check(c(L.gh), gx, ex, ref.BF16_HALF)
    ref.check(c(L.gs2), gw, ew, ref.BF16_HALF)
    (gx, ex), (gw, ew), (gb, eb) = ref.linear_backward(c(L.gh), x, c(L.s1), hz, "silu", True, 1)
    ref.check(c(L.gx[1]), gx, ex, ref.BF16_HALF)
    ref.check(c(L.gs1), gw, ew, ref.BF16_HALF)
    ref.check(c(L.gb1), gb, eb, ref.F32_HALF)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_in_a_graph(ep, size):
    """Captured once, replayed over new inputs with eager work on the same memory's neighbours and synchronisations
    between the replays; every replay equals the eager run to the bit."""
    L, other = Block(ep, *size, seed=3), Block(ep, *size, seed=3)
    L.fill(0)
    L.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        L.run()
    for seed in range(1, 5):
        L.fill(seed)
        for t in L.outputs():
            t.fill_(7)
        L.ws.random_()
        L.bws.random_()
        g.replay()
        got = L.results()
        other.fill(seed)
        other.run()
        torch.cuda.synchronize()
        for a, b in zip(got, other.results()):
            assert torch.equal(a, b)


def test_two_graphs_with_one_workspace(ep):
    """Two sizes captured into two graphs over one workspace each; replayed in turn, on one stream."""
    a, b = Block(ep, 64, 256, 128, 136, 24, 4, True, seed=1), Block(ep, 5, 256, 128, 136, 24, 4, True, seed=2)
    assert a.ws.numel() >= b.ws.numel() and a.bws.numel() >= b.bws.numel()
    want, graphs = [], []
    for L in (a, b):
        L.fill(11)
        L.run()
        want.append(L.results())
    b.ws, b.bws = a.ws, a.bws
    torch.cuda.synchronize()
    for L in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            L.run()
        graphs.append(g)
    for _ in range(3):
        for L, g, w in zip((a, b), graphs, want):
            for t in L.outputs():
                t.zero_()
            g.replay()
            for p, q in zip(L.results(), w):
                assert torch.equal(p, q)
        torch.cuda.synchronize()


def test_streams(ep):
    """Two runs at once on two streams, given as arguments, each with its own buffers; the allocating calls on a stream."""
    size = (33, 512, 256, 520, 32, 4, True)
    Ls = [Block(ep, *size, seed=i) for i in range(2)]
    want = []
    for i, L in enumerate(Ls):
        L.fill(i)
        L.run()
        want.append(L.results())
        for t in L.outputs():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ls]
    for _ in range(6):
        for L, s in zip(Ls, streams):
            L.run(s)
    for L, s, w in zip(Ls, streams, want):
        s.synchronize()
        for a, b in zip(L.results(), w):
            assert torch.equal(a, b)
    L, s = Ls[0], streams[0]
    y = ep.moe_few(L.x, L.idx, L.tw, L.w[0], L.w[1], L.sc[0], L.sc[1], residual=L.shared, stream=s)
    h, z = ep.linear(L.x, L.s1, L.b1, activation="silu", gated=True, save=True, stream=s)
    gx, gw, gb = ep.linear_backward(L.gh, L.x, L.s1, z, "silu", True, bias=True, stream=s)
    s.synchronize()
    for a, b in ((y, L.y), (h, L.h), (z, L.hz), (gx, L.gx[1]), (gw, L.gs1), (gb, L.gb1)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,K,N,act,gated", [(1020, 512, 1000, None, False), (1024, 264, 520, "silu", True),
                                             (100, 1536, 1016, "relu", False), (1023, 128, 1024, None, False),
                                             (340, 200, 256, "gelu", False), (2000, 72, 64, "silu", True)], ids=str)
@pytest.mark.parametrize("w32", [False, True])
def test_a_gradient_by_itself(ep, M, K, N, act, gated, w32):
    """At the edges between the launches: each gradient alone has the bits that it has among all three."""
    g = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    wide = 2 * N if gated else N
    x, w, dy = rand(M, K).to(BF), rand(wide, K).to(BF), rand(M, N).to(BF)
    z = rand(M, wide).to(BF) if act else None
    kw = dict(activation=act, gated=gated)
    dtype = F32 if w32 else BF
    full = ep.linear_backward(dy, x, w, z, bias=True, grad_w_dtype=dtype, **kw)
    ws = torch.empty(ep.linear_backward_workspace_bytes(M, K, N, act, gated, grad_w_dtype=dtype), dtype=torch.uint8,
                     device="cuda")
    for i, like in enumerate(full):
        out = [None, torch.empty_like(full[1]), None]   # its type is part of the shape
        out[i] = torch.full_like(like, 7)
        if i != 1:
            ep.ep_linear_backward(dy, x, w, z, *out, ws, **kw)
            assert torch.equal(out[i], like) and torch.equal(out[1], full[1])
            out[1] = None
            out[i].fill_(7)
        ep.ep_linear_backward(dy, x, w, z, *out, ws, **kw)
        assert torch.equal(out[i], like)
    (wx, ex), (ww, ew), (wb, eb) = ref.linear_backward(dy.cpu(), x.cpu(), w.cpu(), None if z is None else z.cpu(), act,
                                                       gated, 0 if not act else (3 if w32 else 1))
    ref.check(full[0].cpu(), wx, ex, ref.BF16_HALF)
    ref.check(full[1].cpu(), ww, ew, ref.F32_HALF if w32 else ref.BF16_HALF)
    ref.check(full[2].cpu(), wb, eb, ref.F32_HALF)


def _rows(M, n=70):
    return torch.cat((torch.arange(n), torch.arange(M // 2, M // 2 + n), torch.arange(M - n, M))).cuda()


def test_past_32_bits(ep):
    """More than 2^31 elements in y, z, residual and dy: the first, middle and last rows, and sums over all of them."""
    M, K, N = 530001, 64, 4104
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF)
    w = (torch.randn(N, K, generator=g, device="cuda") / 8).to(BF)
    r = torch.empty(M, N, dtype=BF, device="cuda")
    r.copy_(x[:, :1].expand(M, N))
    assert r.numel() > 2 ** 31
    y, z = ep.linear(x, w, residual=r, activation="relu", save=True)
    at = _rows(M)
    wy, ey, wz, ez = ref.linear(x[at].cpu(), w.cpu(), None, r[at].cpu(), "relu", False)
    ref.check(y[at].cpu(), wy, ey, ref.BF16_HALF)
    ref.check(z[at].cpu(), wz, ez, ref.BF16_HALF)
    del r
    gx, gw, gb = ep.linear_backward(y, x, w, z, activation="relu", bias=True)
    (wx, ex), _, _ = ref.linear_backward(y[at].cpu(), x[at].cpu(), w.cpu(), z[at].cpu(), "relu", False, 1)
    ref.check(gx[at].cpu(), wx, ex, ref.BF16_HALF)
    cols = torch.tensor([0, 1, 63, 64, 2047, 4095, 4096, N - 1], device="cuda")
    dz = torch.where(z[:, cols] > 0, y[:, cols], 0).double()
    part, tiny = 2.0 ** -134, ref.BF16_HALF
    want, mag = dz.T @ x.double(), dz.T.abs() @ x.double().abs()   # dz is y's bf16, exactly
    ref.check(gw[cols].cpu(), want.cpu(), ref.sum_error(mag, M).cpu() + part, tiny)
    s = dz.sum(0).cpu()
    ref.check(gb[cols].cpu(), s, ref.STEP * (64 + M / 64 + 17) * dz.abs().sum(0).cpu(), ref.F32_HALF)
    # and as the longer operand of the other products: x and grad_x past 32 bits
    del y, gx
    x2 = z   # [M, N] taken as an input of N features
    w2 = (torch.randn(72, N, generator=g, device="cuda") / 64).to(BF)
    y2 = ep.linear(x2, w2, out_dtype=F32)
    wy, ey, _, _ = ref.linear(x2[at].cpu(), w2.cpu(), None, None, None, False)
    ref.check(y2[at].cpu(), wy, ey, ref.F32_HALF)
    dy = y2.to(BF)
    gx, gw = ep.linear_backward(dy, x2, w2, grad_w_dtype=F32)
    (wx, ex), _, _ = ref.linear_backward(dy[at].cpu(), x2[at].cpu(), w2.cpu(), None, None, False, 0)
    ref.check(gx[at].cpu(), wx, ex, ref.BF16_HALF)
    xc = x2[:, cols].double()
    want, mag = dy.double().T @ xc, dy.double().T.abs() @ xc.abs()
    ref.check(gw[:, cols].cpu(), want.cpu(), ref.sum_error(mag, M).cpu(), ref.F32_HALF)


@pytest.mark.parametrize("fp8", [True, False])
def test_experts_past_32_bits(ep, fp8):
    """Weights of more than 2^32 bytes: the last experts' results are those of the same experts in a small layer."""
    E, H, I, T, k = 300, 4096, 1024, 9, 3   # noqa: E741
    if not fp8:
        E = 270
    g = torch.Generator(device="cuda").manual_seed(6)
    ids = torch.tensor([E - 1, E - 2, E // 2, 0])
    up, down, s1, s2 = None, None, None, None
    if fp8:
        up = torch.empty(E, 2 * I, H, dtype=torch.uint8, device="cuda").fill_(0x7F)   # NaN wherever nothing is written
        down = torch.empty(E, H, I, dtype=torch.uint8, device="cuda").fill_(0x7F)
        s1 = torch.rand(E, 2 * I // 128, H // 128, generator=g, device="cuda") / 4096
        s2 = torch.rand(E, H // 128, I // 128, generator=g, device="cuda") / 4096
        new = lambda t: torch.randn(t.shape, generator=g, device="cuda").mul(50).clamp(-448, 448).to(F8).view(torch.uint8)   # noqa: E731
        assert up.numel() > 2 ** 31
    else:
        up = torch.full((E, 2 * I, H), float("nan"), dtype=BF, device="cuda")
        down = torch.full((E, H, I), float("nan"), dtype=BF, device="cuda")
        new = lambda t: (torch.randn(t.shape, generator=g, device="cuda") / 32).to(BF)   # noqa: E731
        assert up.numel() * 2 > 2 ** 32
    for e in ids.tolist():
        up[e], down[e] = new(up[e]), new(down[e])
    small = torch.randint(0, 4, (T, k), generator=torch.Generator().manual_seed(1))
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    tw = torch.rand(T, k, generator=g, device="cuda")
    at = ids.cuda()
    y = ep.moe_few(x, at[small.cuda()], tw, up, down, s1, s2)
    want, err = ref.moe_few(x.cpu(), small, tw.cpu(), up[at].cpu(), None if s1 is None else s1[at].cpu(), down[at].cpu(),
                            None if s2 is None else s2[at].cpu(), None)
    ref.check(y.cpu(), want, err, ref.BF16_HALF)


@pytest.mark.parametrize("T,H,I,E,k", [(3, 256, 128, 8, 2), (40, 384, 256, 16, 4), (64, 512, 384, 32, 6)])   # noqa: E741
def test_beside_the_chain(ep, T, H, I, E, k):   # noqa: E741
    """The layer for a few tokens against dispatch, products and combine on rows that e4m3 holds exactly.  The chain
    rounds the gated product to e4m3 (half a step 2^-4 of a value, and of the smallest ones 2^-10 of the largest
    over 448) and each expert's row to bf16; the rest are both sides' own errors."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    up, down = ((rand(E, *s) * 100).clamp(-448, 448).to(F8).view(torch.uint8) for s in ((2 * I, H), (H, I)))
    s1 = (torch.rand(E, 2 * I // 128, H // 128, generator=g, device="cuda") + 0.5) / (100 * H ** 0.5)
    s2 = (torch.rand(E, H // 128, I // 128, generator=g, device="cuda") + 0.5) / (100 * I ** 0.5)
    x = torch.randint(-8, 9, (T, H), generator=g, device="cuda").to(BF)
    x[:, ::128] = 7   # so that a block's largest is 7 times a power of two and its scale exact: 448 = 7 * 64
    x.clamp_(-7, 7)
    router = ep.make_router(E, k, "softmax", renormalize=True)
    idx, tw = ep.route(rand(T, E), router)
    y = ep.moe_few(x, idx, tw, up, down, s1, s2)
    q, s = ep.quant_fp8_s128(x)
    assert torch.equal(q.view(F8).double().view(T, -1, 128) * s.double()[:, :, None], x.double().view(T, -1, 128))
    shape = ep.make_shape(T, H, E, 1, 1, k, ep.EP_FMT_FP8_S128, ep.EP_FMT_BF16)
    rows, rows_s, _, _, h = ep.dispatch(q, idx, tw, shape, ep.Workspace(shape), x_scales=s)
    a, sa = ep.expert_gated(h.expert_offset, rows, rows_s, up, s1)
    z = ep.combine(ep.expert_gemm(h.expert_offset, a, sa, down, s2), h)
    want, err = ref.moe_few(x.cpu(), idx.cpu(), tw.cpu(), up.cpu(), s1.cpu(), down.cpu(), s2.cpu(), None)
    ref.check(y.cpu(), want, err, ref.BF16_HALF)
    off = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            v = x[t].cpu().double() @ ref.weights(up[e].cpu(), s1[e].cpu()).T
            p = (ref.value(v[:I], "silu") * v[I:]).abs()
            top = p.view(-1, 128).amax(1).repeat_interleave(128)
            d = ref.weights(down[e].cpu(), s2[e].cpu()).abs()
            loss = d @ (1.01 * p / 16 + top / 448 / 1024)   # 1.01: the errors before that rounding
            row = d @ p
            off[t] += float(tw[t, j]) * (loss + 2 * ref.BF16_HALF * row)
    ref.check(z.cpu(), want, off + 2 * err, ref.BF16_HALF)
