"""The comparisons of moe_strict.py (CPU): correctly rounded results pass, NaN and values a step off do not."""
import numpy as np
import pytest
import torch

import moe_ref
import moe_strict


def _h(rng):
    h = rng.standard_normal((20, 256)) * 2.0 ** rng.integers(-20, 20, (20, 1))
    h[3], h[5, :128], h[6] = 0, 0, h[6] * 2.0 ** -130
    return h


def _rows(h):
    """The rule on h in binary32: bytes and scales."""
    h = torch.from_numpy(h.astype(np.float32))
    top = h.view(20, -1, 128).abs().amax(2)
    s = torch.where(top == 0, 1.0, (top / 448).clamp(min=2.0 ** -149))
    q = (h.view(20, -1, 128) / s[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(20, 256)
    return q.numpy().copy(), s.double().numpy()


def test_quantised_rows():
    rng = np.random.default_rng(1)
    h = _h(rng)
    q, s = _rows(h)
    err = 2.0 ** -24 * np.abs(h) + 2.0 ** -149
    valid = np.ones(20, bool)
    valid[9] = False
    moe_strict.check_quantised(q, s, h, err, valid)
    moe_strict.check_quantised(np.where(valid[:, None], q, 0x7F), np.where(valid[:, None], s, np.nan), h, err, valid)
    for r, c in ((0, 0), (3, 17), (6, 40), (19, 255)):
        for byte in (0x7F, 0xFF):
            bad = q.copy()
            bad[r, c] = byte
            with pytest.raises(AssertionError):
                moe_strict.check_quantised(bad, s, h, err, valid)
    for r, g in ((0, 0), (3, 1), (6, 0)):
        for v in (np.nan, np.inf, s[r, g] * (1 + 2.0 ** -20), 0.0):
            bad = s.copy()
            bad[r, g] = v
            with pytest.raises(AssertionError), np.errstate(all="ignore"):
                moe_strict.check_quantised(q, bad, h, err, valid)
    # a byte one step up or down, wherever that is not the other neighbour of a middle
    x = np.abs(h) / np.repeat(s, 128, 1)
    for step in (-1, 1):
        for r, c in rng.integers(0, (20, 256), (200, 2)):
            code = int(q[r, c] & 0x7F) + step
            if r in (3, 5, 6, 9) or not 1 <= code <= 0x7E:
                continue
            v = moe_ref.e4m3_value(np.array(code))
            half = moe_strict.half_step(x[r, c], 3, -6)
            if abs(v - x[r, c]) < half * 1.01:
                continue
            bad = q.copy()
            bad[r, c] = (bad[r, c] & 0x80) | code
            with pytest.raises(AssertionError):
                moe_strict.check_quantised(bad, s, h, err, valid)


def test_bf16_rows():
    rng = np.random.default_rng(2)
    ref = _h(rng)
    got = torch.from_numpy(ref).float().bfloat16().double().numpy()
    err = 2.0 ** -24 * np.abs(ref) + 2.0 ** -140
    valid = np.ones(20, bool)
    valid[9] = False
    moe_strict.check_product(got, ref, err, valid)
    moe_strict.check_product(np.where(valid[:, None], got, np.nan), ref, err, valid)
    for r, c in ((0, 0), (3, 5), (19, 255)):
        for v in (np.nan, np.inf, got[r, c] * (1 + 2.0 ** -6) + 2.0 ** -100):
            bad = got.copy()
            bad[r, c] = v
            with pytest.raises(AssertionError):
                moe_strict.check_product(bad, ref, err, valid)
