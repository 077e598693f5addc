"""The layer for a few tokens at the widths where the second kernel's columns
have one block each: its sums go straight to y.  Beside them the widest that is
cut, and a ragged last block."""
import pytest

import dense_ref as ref
from test_few_gpu import call, cuda, draw

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


@pytest.mark.parametrize("H,fp8", [(4096, True), (4224, True), (7168, True), (4096, False), (4104, False), (7176, False),
                                   (8200, False)])
@pytest.mark.parametrize("T,k", [(2, 2), (9, 3), (17, 2), (33, 3), (64, 2)])
@pytest.mark.parametrize("masked,residual", [(0.0, False), (0.3, True)])
def test_wide(ep, H, fp8, T, k, masked, residual):
    d = draw(T, H, 128 if fp8 else 40, 5, k, fp8, seed=7, masked=masked, residual=residual)
    y = call(ep, cuda(d))
    want, err = ref.moe_few(d["x"], d["idx"], d["tw"], d["up"], d["up_s"], d["down"], d["down_s"], d["r"])
    ref.check(y.cpu(), want, err, ref.BF16_HALF)
    if not residual:
        assert torch.equal(y, call(ep, cuda(d)))
    none = (d["idx"] < 0).all(1)
    assert torch.equal(y.cpu()[none], d["r"][none]) if residual else not none.any()


def test_wide_guards(ep):
    """Nothing is written around y, nor past the workspace; y in the residual's buffer."""
    for H in (4104, 7176):
        d = cuda(draw(17, H, 40, 4, 2, False, residual=True))
        want = call(ep, d)
        n = ep.moe_few_workspace_bytes(17, H, 40, 4, 2, ep.EP_FMT_BF16)
        ws = torch.full((n + 256,), 9, dtype=torch.uint8, device="cuda")
        buf = torch.full((64 + 17 * H + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        y = buf[64:-64].view(17, H)
        y.copy_(d["r"])
        ep.ep_moe_few(d["x"], d["idx"], d["tw"], d["up"], None, d["down"], None, y, y, ws[:n])
        assert torch.equal(y, want) and (buf[:64] == 5).all() and (buf[-64:] == 5).all() and (ws[n:] == 9).all()
