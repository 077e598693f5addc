"""Comparisons of the experts' products with their 64-bit values that hold every
element to its own rounding, and that a NaN cannot pass: each says what has to
be true, not what must not be."""
import numpy as np

import moe_ref

STEP = 2.0 ** -23


def half_step(x, bits, lowest):
    """Half the distance of the values of a format with `bits` mantissa bits, and subnormals below 2^lowest, at |x|."""
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(x)))
    return 2.0 ** (np.maximum(e, lowest) - bits - 1)


def gated(y, mag, K):
    """h and a bound of its error, from the two products, their terms' magnitudes and K: silu' is below 1.1, the gate's
    own evaluation within 5 steps, and half a smallest subnormal lost before and after the product with u."""
    N = y.shape[1] // 2
    g, u = y[:, :N], y[:, N:]
    dg, du = moe_ref.sum_error(mag[:, :N], K), moe_ref.sum_error(mag[:, N:], K)
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    h = silu * u
    return h, 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 5 * STEP * np.abs(h) + 2.0 ** -149 * (1 + np.abs(u))


def check_product(got, ref, err, valid):
    """bf16 values (as float64) of ref, whose sums are off by err at most."""
    got, ref, err = got[valid], ref[valid], err[valid]
    ok = np.abs(got - ref) <= err + half_step(np.abs(ref) + err, 7, -126)
    assert ok.all(), (np.argwhere(~ok)[:5], int((~ok).sum()))


def check_quantised(q, s, h, err, valid):
    """e4m3 bytes q and scales s (float64) of h, which is off by err at most."""
    q, s, h, err = q[valid], s[valid], h[valid], err[valid]
    top, slack = (x.reshape(len(x), -1, 128).max(2) for x in (np.abs(h), err))
    ok = np.abs(s - np.maximum(top / 448, 2.0 ** -149)) <= slack / 448 + 2.0 ** -24 * (top + slack) / 448 + 2.0 ** -150
    ok |= (top <= slack) & (s == 1.0)                # all zero in binary32
    assert ok.all(), ("scales", np.argwhere(~ok)[:5], int((~ok).sum()))
    wide = np.repeat(s, 128, 1)
    x, dx = h / wide, err / wide + STEP * np.abs(h) / wide    # before its rounding to 8 bits
    want = np.clip(x, -448, 448)
    ok = np.abs(moe_ref.e4m3_value(q) - want) <= dx + half_step(np.minimum(np.abs(x) + dx, 448), 3, -6)
    assert ok.all(), ("bytes", np.argwhere(~ok)[:5], int((~ok).sum()))
