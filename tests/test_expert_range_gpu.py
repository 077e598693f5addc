"""The gated product at the ends of binary32: groups whose largest value, or
whose scale, is subnormal, and gates far below zero.

Every sum here is a single exact product (the gate comes from the first block
of K alone, the up value from the second), so g and u are known exactly and h
is off by the gate's own evaluation only: at most 5 steps (2 of e^(g/2) squared
or 1 of e^g, 1 of the reciprocal, half of the sum and of three products), and
half the smallest subnormal where h itself falls below 2^-126."""
import numpy as np
import pytest

import moe_ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

STEP, TINY = 2.0 ** -23, 2.0 ** -149
UPS = np.array([0, 1, -1, 1.5, -7, 11, 15, 0.125, -0.25, 3, -13, 2, 0, 5, -10, 14])   # exact in e4m3


@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from combine_dispatch_layout_02_amd import ep as mod
    mod.load()
    return mod


def _run(ep, gates, ups, copies):
    """Row r has the gate gates[r] in every column and the up value ups[r] times UPS (columns 0-127: all of them;
    128-255: one of them, 0 elsewhere; 256-383: 0).  copies: each row that often (more rows: the tiled form)."""
    g, s = np.repeat(np.float32(gates), copies), np.repeat(np.float32(ups), copies)
    rows = g.size
    v = np.zeros(384)
    v[:128] = np.resize(UPS, 128)
    v[200] = 15
    a = torch.zeros((rows, 256), dtype=torch.uint8)
    a[:, 0] = a[:, 128] = 0x38                       # 1 in both blocks of K
    w = torch.zeros((1, 768, 256), dtype=torch.uint8)
    w[0, :384, 0] = 0x38
    w[0, 384:, 128] = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8)
    a_s = torch.from_numpy(np.stack([g, s], 1))
    off = torch.tensor([0, rows], dtype=torch.int32)
    q, scale = ep.expert_gated(off.cuda(), a.cuda(), a_s.cuda(), w.cuda(), torch.ones(1, 6, 2, device="cuda"))
    q, scale = q.cpu().numpy(), scale.cpu().double().numpy()
    g, u = g.astype(np.float64), s.astype(np.float64)[:, None] * v
    assert (u.astype(np.float32) == u).all()         # exact, subnormals too
    h = (g / (1 + np.exp(-g)))[:, None] * u
    return q, scale, h, 5 * STEP * np.abs(h) + TINY / 2


def _check(q, scale, h, err):
    """Scale: the largest magnitude / 448 in binary32, at least the smallest subnormal, 1 for a group of zeros.
    Bytes: h over that scale, saturated, to the nearest."""
    assert ((q & 0x7F) != 0x7F).all(), "NaN bytes"
    groups = np.abs(h).reshape(len(h), -1, 128)
    top, slack = groups.max(2), err.reshape(groups.shape).max(2)
    fine = np.abs(scale - np.maximum(top / 448, TINY)) <= slack / 448 + 2.0 ** -24 * top / 448 + TINY / 2
    fine |= (top <= slack) & (scale == 1.0)          # all zero in binary32
    assert fine.all(), "scales"
    wide = np.repeat(scale, 128, 1)
    want = np.clip(h, -448 * wide, 448 * wide)
    got = moe_ref.e4m3_value(q) * wide
    # half a step of e4m3 (at least half of its smallest, 2^-9), and the rounding of the quotient
    tol = moe_ref.E4M3_HALF * (np.abs(want) + err) + 2.0 ** -10 * wide + err + STEP * np.abs(want)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("copies", [1, 300])
def test_scales_down_to_the_smallest_subnormal(ep, copies):
    """Groups whose largest value runs from far above 448 times the smallest subnormal down to below it."""
    ups = 2.0 ** -np.arange(128.0, 147.0)
    ups = np.concatenate([ups, 1.375 * ups[:14], -1.25 * ups[:14]])
    for gate in (1.0, -3.0, 40.0):
        _check(*_run(ep, np.full(ups.size, gate), ups, copies))


@pytest.mark.parametrize("copies", [1, 300])
@pytest.mark.parametrize("up,deepest", [(1.0, 116.0), (2.0 ** -6, 112.0), (2.0 ** 20, 130.0), (2.0 ** 100, 173.0)])
def test_deep_gates(ep, up, deepest, copies):
    """Every gate of a group far below zero, where e^g is subnormal or below all of binary32: h is not, or just so."""
    gates = -np.linspace(78.0, deepest, 41)
    _check(*_run(ep, gates, np.full(gates.size, up), copies))
