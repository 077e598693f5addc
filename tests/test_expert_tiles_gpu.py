"""The gated product's tiles over buffers that are only partly in use, with more
experts than a block has threads, and with offsets that do not ascend."""
import numpy as np
import pytest

import moe_ref
import moe_strict
from test_expert_strict_gpu import _draw, _product64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _off(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _gated(ep, off, a, a_s, w, w_s, R=1, M=0):
    q = torch.full((a.shape[0], w.shape[1] // 2), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((a.shape[0], w.shape[1] // 256), 7.0, device="cuda")
    ep.ep_expert_gated(_off(off), a, a_s, w, w_s, q, s, R, M)
    return q, s


def test_parts_of_a_buffer(ep):
    """Every slice of the experts, and the first rows alone, give the whole buffer's rows and touch no others."""
    counts = [2000, 0, 1900, 2311, 3000, 1, 2700, 2500]
    off = [0] + np.cumsum(counts).tolist()
    a, a_s, w, w_s = _draw(3, off[-1], 8, 384, 768)
    q, s = _gated(ep, off, a, a_s, w, w_s)
    for e0, e1 in ((0, 1), (2, 4), (3, 8), (5, 6), (7, 8)):
        q2, s2 = _gated(ep, off[e0:e1 + 1], a, a_s, w[e0:e1].contiguous(), w_s[e0:e1].contiguous())
        lo, hi = off[e0], off[e1]
        assert torch.equal(q2[lo:hi], q[lo:hi]) and torch.equal(s2[lo:hi], s[lo:hi])
        rest = torch.ones(off[-1], dtype=torch.bool, device="cuda")
        rest[lo:hi] = False
        assert (q2[rest] == 0x55).all() and (s2[rest] == 7.0).all()
    none, _ = _gated(ep, [700] * 9, a, a_s, w, w_s)
    assert (none == 0x55).all()


def test_rank_blocks_with_room_to_spare(ep):
    """RANK_MAJOR blocks that are a third full, one of them empty: the rows of the same segments side by side."""
    counts = [900, 700, 800, 5, 0, 0, 1200, 433]
    off, R, M = [0] + np.cumsum(counts).tolist(), 4, 5000
    a, a_s, w, w_s = _draw(4, R * M, 8, 256, 512)
    q, s = _gated(ep, off, a, a_s, w, w_s, R, M)
    rows = np.concatenate([np.arange(lo, hi) for _, lo, hi in moe_ref.segments(off, R * M, R, M)])
    at = torch.from_numpy(rows).cuda()
    pad = torch.zeros(20000 - rows.size, 256, dtype=torch.uint8, device="cuda")
    q2, s2 = _gated(ep, off, torch.cat((a[at], pad)), torch.cat((a_s[at], pad[:, :2].float())), w, w_s)
    assert torch.equal(q2[:rows.size], q[at]) and torch.equal(s2[:rows.size], s[at])
    rest = torch.ones(R * M, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (q[rest] == 0x55).all() and (s[rest] == 7.0).all()


@pytest.mark.parametrize("E", [512, 513, 1100])
def test_more_experts_than_threads(ep, E):
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 330, E)
    counts[rng.integers(0, E, E // 4)] = 0
    counts[E - 1] += 141 * E - counts.sum() if counts.sum() < 141 * E else 0
    off = [3] + (3 + np.cumsum(counts)).tolist()
    x = _draw(5, off[-1] + 2, E, 128, 256)
    q, s = _gated(ep, off, *x)
    y, mag, valid = _product64(off, *x, 1, 0)
    h, err = moe_strict.gated(y, mag, 128)
    q, s = q.cpu().numpy(), s.cpu().double().numpy()
    moe_strict.check_quantised(q, s, h, err, valid)
    assert (q[~valid] == 0x55).all() and (s[~valid] == 7.0).all()


def test_offsets_that_do_not_ascend_stay_in_the_buffers(ep):
    rows, E = 22000, 4
    a, a_s, w, w_s = _draw(6, rows, E, 128, 512)
    for bad in ([-5, 9000, 12000, 40000, 90000], [0, rows, 0, rows, 0], [rows, 12000, 500, 20, 0], [0, 9000, 300, 15000, 7],
                [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1]):
        q = torch.full((rows + 300, 256), 0x55, dtype=torch.uint8, device="cuda")
        s = torch.full((rows + 300, 2), 7.0, device="cuda")
        ep.ep_expert_gated(_off(bad), a, a_s, w, w_s, q[:rows], s[:rows])
        assert (q[rows:] == 0x55).all() and (s[rows:] == 7.0).all()
