"""ep_moe_few against its 64-bit implementation: both weight formats, one token
to the limit, masked slots and tokens, experts named twice, all tokens on one
expert, odd sizes, values at the ends of the types; in place."""
import pytest

import dense_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def draw(T, H, I, E, k, fp8, seed=0, masked=0.0, residual=False, spread=None):   # noqa: E741
    """Inputs on the CPU; spread: only the first so many experts are chosen."""
    g = torch.Generator().manual_seed(seed + 3 * T + H + I + 7 * E)
    rand = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    d = dict(x=rand(T, H).to(BF), tw=rand(T, k).softmax(1))
    n = E if spread is None else spread
    idx = torch.rand(T, n, generator=g).argsort(1)[:, :k]
    if n < k:
        idx = torch.randint(0, n, (T, k), generator=g)
    d["idx"] = torch.where(torch.rand(T, k, generator=g) < masked, -1, idx)
    for name, N, K in (("up", 2 * I, H), ("down", H, I)):
        if fp8:
            d[name] = (rand(E, N, K) * 100).clamp(-448, 448).to(F8).view(torch.uint8)
            d[name + "_s"] = (torch.rand(E, -(-N // 128), K // 128, generator=g) + 0.5) / (100 * K ** 0.5)
        else:
            d[name], d[name + "_s"] = (rand(E, N, K) / K ** 0.5).to(BF), None
    d["r"] = rand(T, H).to(BF) if residual else None
    return d


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def call(ep, c, **kw):
    return ep.moe_few(c["x"], c["idx"], c["tw"], c["up"], c["down"], c["up_s"], c["down_s"], residual=c["r"], **kw)


def check(d, y):
    want, err = ref.moe_few(d["x"], d["idx"], d["tw"], d["up"], d["up_s"], d["down"], d["down_s"], d["r"])
    ref.check(y.cpu(), want, err, ref.BF16_HALF)


FP8 = [(1, 128, 128, 1, 1), (1, 256, 128, 8, 8), (2, 128, 256, 4, 2), (3, 896, 384, 6, 3), (7, 256, 640, 16, 4),
       (8, 384, 128, 5, 2), (9, 640, 256, 12, 3), (16, 256, 384, 40, 8), (17, 128, 128, 7, 4), (31, 384, 256, 64, 6),
       (33, 256, 128, 9, 2), (48, 128, 384, 24, 5), (64, 256, 256, 96, 8)]
BF16 = [(1, 8, 8, 1, 1), (1, 72, 24, 8, 8), (2, 1000, 712, 6, 2), (5, 520, 136, 9, 3), (13, 64, 1032, 4, 4),
        (16, 200, 40, 30, 7), (29, 328, 88, 10, 3), (40, 96, 64, 3, 2), (64, 136, 200, 33, 6)]
CASES = [(c, True) for c in FP8] + [(c, False) for c in BF16]


@pytest.mark.parametrize("size,fp8", CASES, ids=str)
@pytest.mark.parametrize("masked,residual", [(0.0, False), (0.3, True)])
def test_few(ep, size, fp8, masked, residual):
    d = draw(*size, fp8, masked=masked, residual=residual)
    y = call(ep, cuda(d))
    check(d, y)
    assert torch.equal(y, call(ep, cuda(d)))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("T,k,spread", [(64, 1, 1), (64, 8, 8), (40, 2, 2), (33, 4, 5), (17, 2, 1), (12, 2, 1),
                                        (2, 32, 1), (9, 32, 1), (64, 32, 3)])
def test_crowded(ep, T, k, spread, fp8):
    """Few experts for many tokens (several row tiles each), slots that name one expert again and again."""
    d = draw(T, 256, 128, 8, k, fp8, seed=5, masked=0.1, residual=True, spread=spread)
    check(d, call(ep, cuda(d)))


def test_masks(ep):
    """Masked slots add nothing whatever their weight, ids past the end count as masked, empty tokens get their
    residual or +0."""
    d = draw(6, 128, 128, 4, 3, True, residual=True)
    d["idx"][0] = -1
    d["idx"][3] = torch.tensor([-5, 4, 2 ** 40])
    d["idx"][4, 1] = -1
    for bad in (float("nan"), float("inf")):
        d["tw"][0], d["tw"][3], d["tw"][4, 1] = bad, bad, bad
        y = call(ep, cuda(d))
        clean = dict(d, tw=torch.where((d["idx"] < 0) | (d["idx"] >= 4), torch.zeros(()), d["tw"]))
        check(clean, y)
        assert torch.equal(y[0].cpu(), d["r"][0]) and torch.equal(y[3].cpu(), d["r"][3])
    bare = dict(d, r=None)
    y = call(ep, cuda(bare)).cpu()
    for t in (0, 3):
        assert (y[t].view(torch.int16) == 0).all()
    d["idx"][:] = -1
    assert torch.equal(call(ep, cuda(d)).cpu(), d["r"])
    assert (call(ep, cuda(dict(d, r=None))) == 0).all()


def test_unused_experts_are_not_touched(ep):
    """NaN weights and scales of experts that no token names reach nothing; one token's NaN stays its own."""
    d = draw(20, 256, 128, 6, 2, True, seed=9, spread=4)
    want = call(ep, cuda(d))
    for e in (4, 5):
        d["up"][e] = 0x7F
        d["down"][e] = 0x7F
        d["up_s"][e] = float("nan")
    assert torch.equal(call(ep, cuda(d)), want)
    d["x"][7, 3] = float("nan")
    y = call(ep, cuda(d))
    keep = (torch.arange(20) != 7).cuda()
    assert torch.isnan(y[7]).all() and torch.equal(y[keep], want[keep])
    d = draw(20, 256, 128, 6, 2, True, seed=9, spread=4)
    d["down"][0] = 0x7F          # an expert's NaN reaches the tokens that name it and no others
    y = call(ep, cuda(d))
    hit = (d["idx"] == 0).any(1).cuda()
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], want[~hit])


def test_large_values(ep):
    """h past bf16's largest value (3.39e38) but inside binary32's: its first part stays finite."""
    d = draw(1, 8, 8, 1, 1, False)
    d["x"][:] = 0
    d["x"][0, 0] = 2.0 ** 64
    d["tw"][:] = 1
    d["up"][:] = 0
    d["up"][0, 0, 0] = 1
    d["up"][0, 8, 0] = 1.9921875 * 2.0 ** -1         # g u = 2^128 (1 - 2^-8): above the largest bf16 by rounding only
    d["down"][:] = 0
    d["down"][0, 0, 0] = 2.0 ** -10
    y = call(ep, cuda(d)).cpu()
    assert float(y[0, 0]) == 2.0 ** 118 * (1 - 2.0 ** -8)


def test_shared_buffers(ep):
    """y in x's buffer and in the residual's, a workspace with anything in it, nothing written around y."""
    d = cuda(draw(11, 256, 128, 7, 3, True, residual=True))
    want = call(ep, d)
    n = ep.moe_few_workspace_bytes(11, 256, 128, 7, 3)
    for name in ("x", "r"):
        c = {k: None if v is None else v.clone() for k, v in d.items()}
        ws = torch.randint(0, 256, (n + 256,), dtype=torch.uint8, device="cuda")
        tail = ws[n:].clone()
        ep.ep_moe_few(c["x"], c["idx"], c["tw"], c["up"], c["up_s"], c["down"], c["down_s"], c["r"], c[name], ws[:n])
        assert torch.equal(c[name], want) and torch.equal(ws[n:], tail)
    buf = torch.full((64 + 11 * 256 + 64,), 5.0, dtype=BF, device="cuda")
    ep.ep_moe_few(d["x"], d["idx"], d["tw"], d["up"], d["up_s"], d["down"], d["down_s"], d["r"],
                  buf[64:-64].view(11, 256), torch.empty(n, dtype=torch.uint8, device="cuda"))
    assert torch.equal(buf[64:-64].view(11, 256), want) and (buf[:64] == 5).all() and (buf[-64:] == 5).all()


def test_empty(ep):
    d = cuda(draw(1, 128, 128, 2, 1, True))
    d = dict(d, x=d["x"][:0], idx=d["idx"][:0], tw=d["tw"][:0])
    assert call(ep, d).shape == (0, 128)


def test_refusals(ep):
    d = cuda(draw(4, 256, 128, 3, 2, True))
    with pytest.raises(RuntimeError, match="invalid argument"):
        c = cuda(draw(65, 256, 128, 3, 2, True))
        call(ep, c)
    with pytest.raises(RuntimeError, match="workspace"):
        call(ep, d, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        call(ep, dict(d, tw=torch.rand(4, 4, device="cuda")[:, ::2]))
    with pytest.raises(ValueError, match="scales"):
        call(ep, dict(d, down_s=None))
    with pytest.raises(ValueError, match="device tensor"):
        call(ep, dict(d, down=d["down"].cpu()))
