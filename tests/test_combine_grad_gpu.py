"""The combine's backward pass on the GPU against 64 bits and against the
forward pass itself."""
import numpy as np
import pytest

import moe_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _inputs(rng, T, H, k, rows, masked):
    slot = np.full((T, k), -1, np.int32)
    flat = rng.permutation(rows)[:T * k].astype(np.int32)
    slot.reshape(-1)[:len(flat)] = flat
    slot[rng.random((T, k)) < masked] = -1
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    w = torch.from_numpy(rng.uniform(-1, 1, (T, k)).astype(np.float32))
    return bf(T, H), bf(rows, H), torch.from_numpy(slot), w


def _check(ep, shape, dy, out, slot, w):
    H = dy.shape[1]
    g = torch.full(out.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    gw = torch.full(w.shape, 7.0, device="cuda")
    ep.ep_combine_backward(shape, dy.cuda(), out.cuda(), slot.cuda(), w.cuda(), g, gw)
    want = torch.full(out.shape, 7.0, dtype=torch.bfloat16)
    ref, mag = np.zeros(w.shape), np.zeros(w.shape)
    for t in range(w.shape[0]):
        for j in range(w.shape[1]):
            s = int(slot[t, j])
            if 0 <= s < out.shape[0]:
                want[s] = (w[t, j] * dy[t].float()).to(torch.bfloat16)
                p = dy[t].double() * out[s].double()
                ref[t, j], mag[t, j] = float(p.sum()), float(p.abs().sum())
    assert torch.equal(g.cpu(), want)
    # exact products, at most H - 1 roundings of partial sums
    assert (np.abs(gw.cpu().double().numpy() - ref) <= H * moe_ref.F32_HALF * mag).all()
    return g, gw


@pytest.mark.parametrize("T,H,k,masked", [(1, 8, 1, 0), (3, 16, 2, 0), (5, 1000, 3, 0.3), (2, 2048, 8, 0), (9, 2056, 4, 0.2),
                                          (7, 7168, 8, 0.1), (2, 7176, 32, 0.5), (4, 512, 8, 1.0), (3, 20000, 2, 0),
                                          (300, 64, 2, 0.1), (2, 65536, 3, 0)])
def test_gradients(ep, T, H, k, masked):
    rng = np.random.default_rng(T + H + k)
    shape = ep.make_shape(T, H, 64, 4, 1, k)
    _check(ep, shape, *_inputs(rng, T, H, k, T * k, masked))


def test_rank_major_rows_and_slots_outside(ep):
    rng = np.random.default_rng(3)
    shape = ep.make_shape(20, 256, 8, 4, 1, 2, rank_capacity=15)
    dy, out, slot, w = _inputs(rng, 20, 256, 2, 60, 0.2)
    slot[0, 0], slot[1, 1] = 60, 2 ** 31 - 1
    _check(ep, shape, dy, out, slot, w)


def test_inf_and_nan_stay_in_their_rows(ep):
    rng = np.random.default_rng(4)
    shape = ep.make_shape(6, 128, 8, 1, 1, 2)
    dy, out, slot, w = _inputs(rng, 6, 128, 2, 12, 0)
    ref = _check(ep, shape, dy, out, slot, w)
    out[int(slot[2, 1]), 5] = float("inf")
    dy[4, 7] = float("nan")
    h = ep.Handle(shape, slot.cuda(), None, w.cuda())
    g, gw = ep.combine_backward(dy.cuda(), out.cuda(), h)
    assert torch.isinf(gw[2, 1]) and torch.isnan(gw[4]).all()
    keep = [s for t in range(6) if t != 4 for s in slot[t].tolist()]
    assert torch.equal(g[keep], ref[0][keep])
    assert torch.equal(gw[[0, 1, 3, 5]], ref[1][[0, 1, 3, 5]])
    assert torch.isnan(g[slot[4].tolist(), 7]).all()


def test_against_differences_of_the_combine(ep):
    """Small whole numbers make every rounding of the forward pass exact, so
    its differences are the gradient exactly."""
    rng = np.random.default_rng(5)
    T, H, k = 5, 16, 3
    shape = ep.make_shape(T, H, 8, 1, 1, k)
    slot = torch.from_numpy(rng.permutation(T * k).reshape(T, k).astype(np.int32)).cuda()
    w = torch.from_numpy(rng.integers(-3, 4, (T, k)).astype(np.float32)).cuda()
    out = torch.from_numpy(rng.integers(-3, 4, (T * k, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    dy = torch.from_numpy(rng.integers(-3, 4, (T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    h = ep.Handle(shape, slot, None, w)
    g, gw = ep.combine_backward(dy, out, h)

    def loss(o, ww):
        y = ep.combine(o, ep.Handle(shape, slot, None, ww))
        return float((y.double() * dy.double()).sum())
    base = loss(out, w)
    for t in range(T):
        for j in range(k):
            w2 = w.clone()
            w2[t, j] += 1
            assert loss(out, w2) - base == float(gw[t, j])
    for s in range(0, T * k, 4):
        o2 = out.clone()
        o2[s, 3] += 1
        assert loss(o2, w) - base == float(g[s, 3])


def test_large_batch(ep):
    """The exchange's own handle at T = 600, H = 7168, and the result repeated to the bit."""
    from combine_dispatch_layout_02_amd import workloads as W
    inp = W.make_inputs("prefill2n", T=600, mask_frac=0.1)
    shape = ep.make_shape(600, 7168, 256, 16, 2, 8)
    ws = ep.Workspace(shape)
    x = torch.from_numpy(inp["x"].view(np.int16)).view(torch.bfloat16).cuda()
    idx, w = torch.from_numpy(inp["topk_idx"]).cuda(), torch.from_numpy(inp["topk_w"]).cuda()
    recv, _, _, _, h = ep.dispatch(x, idx, w, shape, ws)
    dy = torch.randn(600, 7168, device="cuda").to(torch.bfloat16)
    n = int(h.expert_offset[-1])
    recv[n:] = 0
    g, gw = ep.combine_backward(dy, recv, h)
    live = h.token_slot >= 0
    at = h.token_slot.clamp(min=0).long()
    want = (w[:, :, None] * dy[:, None].float()).to(torch.bfloat16)
    assert torch.equal(g[at][live], want[live])
    p = dy.double()[:, None] * recv.double()[at]
    err = (gw.double() - p.sum(2)).abs()
    assert (err[live] <= 7168 * moe_ref.F32_HALF * p.abs().sum(2)[live]).all() and (gw[~live] == 0).all()
    g2, gw2 = ep.combine_backward(dy, recv, h)
    assert torch.equal(g2[:n], g[:n]) and torch.equal(gw2, gw)


def test_no_tokens(ep):
    shape = ep.make_shape(0, 64, 8, 1, 1, 2)
    e = lambda *s, d=torch.bfloat16: torch.empty(s, dtype=d, device="cuda")  # noqa: E731
    h = ep.Handle(shape, e(0, 2, d=torch.int32), None, e(0, 2, d=torch.float32))
    g, gw = ep.combine_backward(e(0, 64), e(0, 64), h)
    assert g.shape == (0, 64) and gw.shape == (0, 2)


@pytest.mark.parametrize("T,H,k", [(1024, 264, 3), (1100, 2056, 4), (1500, 40, 9)])
def test_one_wave_a_token(ep, T, H, k):
    rng = np.random.default_rng(T)
    shape = ep.make_shape(T, H, 64, 4, 1, k)
    _check(ep, shape, *_inputs(rng, T, H, k, T * k, 0.1))
