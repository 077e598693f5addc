"""Plain 64-bit implementations of the router, the experts' products and the
combine's backward pass, written from their definitions in include/ep.h, and
the error bounds the GPU results are held to."""
import math

import numpy as np

F32_HALF, BF16_HALF, E4M3_HALF = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4   # half a step, relative


# --------------------------------------------------------------------------- router

def scores(z, score):
    """Scores of one token's logits (float64 list), 0 where the logit is -inf or NaN."""
    live = [x == x and x > -math.inf for x in z]
    if score == "sigmoid":
        return [0.0 if not ok else (1 / (1 + math.exp(-x)) if x > -700 else math.exp(max(x, -1e4)))
                for x, ok in zip(z, live)], live
    top = max([x for x, ok in zip(z, live) if ok], default=0.0)
    e = [0.0 if not ok else (1.0 if x == top else math.exp(x - top)) for x, ok in zip(z, live)]
    s = sum(e)
    return [x / s if s else 0.0 for x in e], live


def route(z, k, score, bias=None, G=1, Gk=None, gtop=1, renorm=False, scale=1.0):
    """z [T, E] float64 -> idx [T, k], w [T, k] (float64), by sorting."""
    T, E = z.shape
    Gk = G if Gk is None else Gk
    idx, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        p, live = scores(z[t].tolist(), score)
        key = [(-math.inf if not ok else x + (float(bias[e]) if bias is not None else 0.0))
               for e, (x, ok) in enumerate(zip(p, live))]
        key = [-math.inf if x != x else x for x in key]
        if G > 1:
            per = E // G
            mark = []
            for g in range(G):
                m = sum(sorted(key[g * per:(g + 1) * per], reverse=True)[:gtop])
                mark.append(-math.inf if m != m else m)
            keep = set(sorted(range(G), key=lambda g: (-mark[g], g))[:Gk])
            key = [x if e // per in keep else -math.inf for e, x in enumerate(key)]
        best = [e for e in sorted(range(E), key=lambda e: (-key[e], e))[:k] if key[e] > -math.inf]
        idx[t, :len(best)] = best
        w[t, :len(best)] = weights(z[t], best, score, renorm, scale)
    return idx, w


def weights(z, chosen, score, renorm, scale):
    """Weights of one token's chosen experts."""
    p, _ = scores(z.tolist(), score)
    v = [p[e] for e in chosen]
    if renorm:
        if score == "softmax":
            v, _ = scores([float(z[e]) for e in chosen], "softmax")
        s = sum(v)
        v = [x / s if s > 0 else 0.0 for x in v]
    return [scale * x for x in v]


def route_backward(z, idx, g, score, renorm=False, scale=1.0):
    """Gradient [T, E] by the Jacobian of `weights`, written out entry by entry."""
    T, E = z.shape
    out = np.zeros((T, E))
    for t in range(T):
        p, live = scores(z[t].tolist(), score)
        slots = [(j, int(e)) for j, e in enumerate(idx[t]) if 0 <= e < E and live[int(e)]]
        if not slots:
            continue
        q = [x / scale for x in weights(z[t], [e for _, e in slots], score, True, scale)]
        for a, (j, e) in enumerate(slots):
            c = scale * float(g[t, j])
            if score == "softmax" and not renorm:
                for i in range(E):
                    out[t, i] += c * p[e] * ((1.0 if i == e else 0.0) - p[i])
            elif score == "softmax":
                for b, (_, i) in enumerate(slots):
                    out[t, i] += c * q[a] * ((1.0 if a == b else 0.0) - q[b])
            elif not renorm:
                out[t, e] += c * p[e] * rest(z[t, e])
            else:
                for b, (_, i) in enumerate(slots):
                    out[t, i] += c * q[a] * ((1.0 if a == b else 0.0) - q[b]) * rest(z[t, i])
    return out


def rest(x):
    """1 - sigmoid(x) without cancellation."""
    return 1 / (1 + math.exp(x)) if x < 700 else 0.0


# --------------------------------------------------------------------------- formats

def e4m3_value(b):
    """Values of e4m3 bytes (OCP fn)."""
    b = np.asarray(b, np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def dequant_rows(q, s):
    return e4m3_value(q) * np.repeat(np.asarray(s, np.float64), 128, axis=1)


def dequant_weights(q, s):
    N, K = q.shape
    return e4m3_value(q) * np.repeat(np.repeat(np.asarray(s, np.float64), 128, 0)[:N], 128, 1)


# --------------------------------------------------------------------------- products

def segments(offset, rows, R=1, M=0):
    """[(expert, first row, end)] of every expert's rows."""
    E = len(offset) - 1
    out = []
    for e in range(E):
        lo, hi = int(offset[e]), int(offset[e + 1])
        if M > 0:
            r = e // (E // R)
            first = int(offset[r * (E // R)])
            lo, hi = (min(x - first + r * M, (r + 1) * M) for x in (lo, hi))
        out.append((e, lo, max(lo, hi)))
    return out


def product(offset, a, a_s, w, w_s, R=1, M=0):
    """y, the sum of the magnitudes of its terms (both [rows, N], float64), and the mask of rows that are written."""
    rows, N = a.shape[0], w.shape[1]
    y, mag, valid = np.zeros((rows, N)), np.zeros((rows, N)), np.zeros(rows, bool)
    for e, lo, hi in segments(offset, rows, R, M):
        if hi > lo:
            x, v = dequant_rows(a[lo:hi], a_s[lo:hi]), dequant_weights(w[e], w_s[e])
            y[lo:hi], mag[lo:hi], valid[lo:hi] = x @ v.T, np.abs(x) @ np.abs(v).T, True
    return y, mag, valid


def sum_error(mag, K):
    """How far an fp32 evaluation of `product` may be: 128 products and their
    sum in fp32 (at most a whole step, 2^-23, lost at each of 127 additions),
    one rounding of the two scales' product, one of each block's multiply-add,
    and 16 additions of the parts of a split K."""
    return mag * (127 * 2.0 ** -23 + 2.0 ** -24 * (1 + K // 128 + 16)) * 1.01


def sum_error_8bit(mag, K):
    """The same with the 8-bit matrix instruction, which adds 8 products at a
    time after cutting them at 2^-13 of the power of two of the largest.  A
    product of two e4m3 values has 8 bits, so the largest loses nothing and
    each of the 7 others less than 2^-13 of it: a group loses less than 7 * 2^-13
    of its largest product, and all groups together less than 7 * 2^-13 of the
    sum of the magnitudes."""
    return sum_error(mag, K) + 7 * 2.0 ** -13 * mag


def gated(offset, a, a_s, w, w_s, R=1, M=0):
    """h and a bound of its fp32 error, both [rows, N], and the mask of rows."""
    K = a.shape[1]
    y, mag, valid = product(offset, a, a_s, w, w_s, R, M)
    N = y.shape[1] // 2
    g, u = y[:, :N], y[:, N:]
    dg, du = sum_error(mag[:, :N], K), sum_error(mag[:, N:], K)
    with np.errstate(over="ignore"):
        silu = g / (1 + np.exp(-g))
    h = silu * u
    # |silu'| < 1.1; expf, the sum, the division and the product: at most 8 half steps of h; a negative g below the
    # range of expf gives 0 where the definition gives less than 2^-120 |u|
    err = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + 8 * F32_HALF * np.abs(h) + 2.0 ** -120 * np.abs(u)
    return h, err, valid


def check_quantised(q, s, h, err, valid):
    """e4m3 rows q and scales s against h with fp32 error err."""
    rows, N = h.shape
    hg, eg = np.abs(h).reshape(rows, -1, 128), err.reshape(rows, -1, 128)
    top = hg.max(2)
    slack = eg.max(2)
    want = np.where(top == 0, 1.0, top / 448)
    s64 = np.asarray(s, np.float64)
    ok = np.abs(s64 - want) <= slack / 448 + F32_HALF * want * 2
    ok |= (top <= slack) & (s64 == 1.0)   # all zero in fp32
    assert ok[valid].all(), "scales"
    wide = np.repeat(s64, 128, 1)
    got = e4m3_value(q) * wide
    # half a step of e4m3 (2^-4 of the value, or of its smallest step 2^-9 below 2^-6), one rounding of the division
    tol = E4M3_HALF * (np.abs(h) + err) * (1 + 2 * F32_HALF) + 2.0 ** -10 * wide + err + 2 * F32_HALF * np.abs(h)
    bad = np.abs(got - h) > tol
    assert not bad[valid].any(), np.argwhere(bad & valid[:, None])[:5]
