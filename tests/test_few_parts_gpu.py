"""What of the gated product reaches the second half of the layer for a few
tokens: sums in which it cancels show what its two bf16 parts lose, 2^-17 of it
at most."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _parts(v):
    """A binary32 value of 24 bits as three bf16 values, exactly."""
    a = v.to(BF)
    b = (v - a.double()).to(BF)
    c = (v - a.double() - b.double()).to(BF)
    assert (a.double() + b.double() + c.double() == v).all()
    return a, b, c


@pytest.mark.parametrize("T", [1, 9, 40])
def test_two_parts(ep, T):
    """h[4 n] = v and h[4 n + 1 .. 4 n + 3] its three exact parts; y[n] = their difference is what h lost."""
    g = torch.Generator().manual_seed(T)
    n = 512
    v = 1 + torch.randint(0, 2 ** 23, (n,), generator=g).double() * 2.0 ** -23
    # among them those whose cut, or rounded, first part leaves the longest rest
    v[:64] = 1 + torch.arange(64) * 2.0 ** -7 + 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -20
    v[64:128] = 1 + torch.arange(64) * 2.0 ** -7 + 2.0 ** -8 - 2.0 ** -17 - 2.0 ** -20
    p = _parts(v)
    H, I = n, 4 * n   # noqa: E741
    up = torch.zeros(1, 2 * I, H)
    up[0, :I, 0] = 128                      # silu(128) is 128: the gate is exact
    for i in range(3):                      # x[0 .. 2] are 1: u is v, and each of its parts
        up[0, I + 0:2 * I:4, i] = p[i].float()
        up[0, I + 1 + i:2 * I:4, i] = p[i].float()
    down = torch.zeros(1, H, I)
    at = torch.arange(n)
    down[0, at, 4 * at] = 1
    for i in range(3):
        down[0, at, 4 * at + 1 + i] = -1
    x = torch.zeros(T, H)
    x[:, :3] = 1
    y = ep.moe_few(x.to(BF).cuda(), torch.zeros(T, 1, dtype=torch.int64, device="cuda"), torch.ones(T, 1, device="cuda"),
                   up.to(BF).cuda(), down.to(BF).cuda()).cpu().double()
    # 128 v goes in; a step of fp32 for each of the products' 4 terms, in both parts, and u's own 3; y is rounded to bf16
    most = 128 * v * (2.0 ** -17 + 11 * 2.0 ** -23) * (1 + 2.0 ** -8)
    assert (y.abs() <= most).all(), float((y.abs() / (128 * v)).max()) * 2 ** 17
