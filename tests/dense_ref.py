"""Plain 64-bit implementations of the dense product with its backward pass and
of the experts' layer for a few tokens, written from their definitions in
include/ep.h, with a bound of the error of an evaluation in the precision that
stands there.  Each takes and gives CPU tensors."""
import math

import torch

STEP, BF16_HALF, F32_HALF = 2.0 ** -23, 2.0 ** -8, 2.0 ** -24
ACTIVATIONS = (None, "relu", "silu", "gelu", "gelu_tanh")


def value(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":   # 1 + tanh(a) as twice a sigmoid, which keeps the lower tail
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        a = c * (z + 0.044715 * z ** 3)
        p = torch.sigmoid(a)
        return p + z * p * torch.sigmoid(-a) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def sum_error(mag, K):
    """A sum of K products of bf16 values in fp32: a product is exact, and on
    its way passes at most 31 additions inside its matrix instruction, K / 32
    from one to the next and 16 of parts of K, and loses a step at most at
    each (half where it is rounded, one where it is cut)."""
    return mag * STEP * (31 + K / 32 + 16)


def activation_error(z, act, dz):
    """Error of act(z) from z's own error dz and the fp32 evaluation.  No
    activation is steeper than 1.13.  The evaluation: at most 16 steps of the
    result (a library function within 4, a division, and the products), and for
    those with an argument that is itself rounded (the erfc's and the cubic's)
    what 4 steps of that argument move the result by: below 4 z^2 steps of it for
    gelu (erfc falls by at most about 2 a + 1 times itself for a unit of a > 0) and
    4 |a| for the cubic's a.  Results below the smallest normal number lose at most a step of the subnormals."""
    f = value(z, act).abs()
    cond = torch.zeros_like(z)
    if act == "gelu":
        cond = 4 * (z * z + z.abs() + 1)
    if act == "gelu_tanh":
        cond = 8 * (z.abs() + 0.044715 * z.abs() ** 3)
    # far below, where the result is smaller than binary32's normal numbers (2^-126 |z|), all of it may be lost
    return 1.13 * dz + torch.minimum(STEP * (16 + cond) * f, f) + 2.0 ** -120


def linear(x, w, bias, residual, act, gated):
    """y, z and bounds of their errors before the last rounding."""
    x, w = x.double(), w.double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    dz = sum_error(mag, x.shape[1]) + STEP * z.abs()
    if gated:
        n = z.shape[1] // 2
        g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
        f, df = value(g, act), activation_error(g, act, dg)
        y, dy = f * u, df * (u.abs() + du) + f.abs() * du + STEP * (f * u).abs()
    else:
        y, dy = value(z, act), activation_error(z, act, dz)
    if residual is not None:
        y = y + residual.double()
        dy = dy + STEP * y.abs()
    return y, dy, z, dz


def check(got, want, err, half):
    """got (rounded to a type whose half step is `half`, relative) of want, which is off by err at most."""
    got = got.double()
    ok = (got - want).abs() <= err + half * (want.abs() + err) + 2.0 ** -134
    assert ok.all(), (torch.nonzero(~ok)[:5].tolist(), int((~ok).sum()), float((got - want).abs().max()))


def slope_error(z, act):
    """Of act' in fp32: its terms are below 1.2 in all, 24 steps of that and the argument's part as above."""
    cond = torch.zeros_like(z)
    if act == "gelu":
        cond = 4 * (z * z + z.abs() + 1) * (0.5 * torch.special.erfc(z.abs() / math.sqrt(2)) + torch.exp(-z * z / 2) * z.abs())
    if act == "gelu_tanh":
        cond = 8 * (z.abs() + 0.044715 * z.abs() ** 3) * torch.sigmoid(-z.abs()) * (1 + z.abs() * (1 + z * z))
    return STEP * (1.2 * 24 + cond)


def linear_backward(dy, x, w, z, act, gated, parts):
    """(grad_x, its error), (grad_w, ...), (grad_bias, ...); parts: how grad_w takes dz (0: as it is, 1: bf16, 3: three
    bf16 parts, exactly; grad_x takes the first)."""
    dy, x, w = dy.double(), x.double(), w.double()
    if gated:
        n = dy.shape[1]
        g, u = z.double()[:, :n], z.double()[:, n:]
        f, d = value(g, act), slope(g, act)
        dz = torch.cat((dy * u * d, dy * f), 1)
        e = torch.cat((dy.abs() * (u.abs() * slope_error(g, act) + 2 * STEP * (u * d).abs()),
                       dy.abs() * (activation_error(g, act, 0.0) + STEP * f.abs())), 1)
    elif act is not None:
        z = z.double()
        dz = dy * slope(z, act)
        e = dy.abs() * (slope_error(z, act) + STEP)
    else:
        dz, e = dy, torch.zeros_like(dy)
    tiny = 2.0 ** -134
    ex = e + (0 if parts == 0 else BF16_HALF * (dz.abs() + e) + tiny)
    ew = e + (BF16_HALF if parts == 1 else 0) * (dz.abs() + e) + (tiny if parts else 0)
    gx, gw = dz @ w, dz.T @ x
    mx, mw = (dz.abs() + ex) @ w.abs(), (dz.abs() + ew).T @ x.abs()
    ex = ex @ w.abs() + sum_error(mx, w.shape[0])
    ew = ew.T @ x.abs() + sum_error(mw, max(parts, 1) * x.shape[0])
    gb, mb = dz.sum(0), dz.abs().sum(0)
    # runs of 4 to 64 rows, added in some order, then 16 parts of the runs
    eb = e.sum(0) + STEP * (64 + len(dz) / 64 + 1 + 16) * (mb + e.sum(0))
    return (gx, ex), (gw, ew), (gb, eb)


# --------------------------------------------------------------------------- a few tokens

def e4m3(b):
    return b.view(torch.float8_e4m3fn).double()


def weights(q, s):
    """[N, K] weights in 64 bits."""
    if s is None:
        return q.double()
    N, K = q.shape
    return e4m3(q) * s.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)


def moe_few(x, idx, tw, up, up_s, down, down_s, residual):
    """y and the bound of its error before the last rounding."""
    T, H = x.shape
    E, I = up.shape[0], up.shape[1] // 2   # noqa: E741
    x, tw = x.double(), tw.double()
    y = torch.zeros(T, H, dtype=torch.float64) if residual is None else residual.double().clone()
    err, mag, terms = torch.zeros_like(y), y.abs(), 0
    for e in sorted(set(int(i) for i in idx.flatten() if 0 <= i < E)):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        u1, d1 = weights(up[e], None if up_s is None else up_s[e]), weights(down[e], None if down_s is None else down_s[e])
        z, m = x[t] @ u1.T, x[t].abs() @ u1.abs().T
        # the scales: a rounding at each block's multiply-add
        dz = sum_error(m, H) + m * F32_HALF * (H / 128)
        g, u, dg, du = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
        f = value(g, "silu")
        h = f * u * tw[t, j, None]
        # 1.1: the slope; 5 steps of the gate's evaluation, one of the weight's product; 2^-17 of the two parts, and one
        # step of bf16's subnormals for each
        dh = tw[t, j, None].abs() * (1.1 * dg * (u.abs() + du) + f.abs() * du) + 6 * STEP * h.abs()
        dh = dh + 2.0 ** -16 * (h.abs() + dh) + 2.0 ** -132
        y.index_add_(0, t, h @ d1.T)
        mag.index_add_(0, t, (h.abs() + dh) @ d1.abs().T)
        err.index_add_(0, t, dh @ d1.abs().T)
        terms += 1
    # a token's sum: inside an expert's K, a rounding for each scaled block, the experts and the waves' parts in turn
    return y, err + mag * STEP * (31 + I / 32 + I / 128 + 2 + terms + 16 + 2)
