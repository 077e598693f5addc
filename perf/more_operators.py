"""The products around the experts that are measured: the matrix product with
bias, activation and residual (the router's logits, the shared expert), its
backward pass, and the whole experts' layer for a few tokens.

``run`` computes them in their plain form (elementary torch operations) or,
with ``own`` set, through the package's calls; both take what ``prepare``
draws.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
BF = torch.bfloat16


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token at a device that holds 32 experts of the exchange's headline hidden size
        dict(name="few_token", op="few", T=1, E=32, k=8, H=7168, I=2048, fp8=True, masked=0.0, residual=False),
        # a decode batch that reaches all of 64 experts; the shared expert's result comes in as the residual
        dict(name="few_batch", op="few", T=32, E=64, k=8, H=7168, I=2048, fp8=True, masked=0.0, residual=True),
        # small bf16 experts of odd sizes, tokens with masked slots
        dict(name="few_odd", op="few", T=7, E=20, k=4, H=1000, I=712, fp8=False, masked=0.1, residual=True),
        # the largest batch, over many smaller experts
        dict(name="few_most", op="few", T=64, E=96, k=6, H=2048, I=1408, fp8=True, masked=0.02, residual=False),
        # the router's logits of one decoded token: all latency
        dict(name="linear_logits", op="linear", M=1, K=7168, N=256, act=None, gated=False, bias=False, residual=False,
             f32=True, save=False),
        # the shared expert's first half in a decode batch
        dict(name="linear_decode", op="linear", M=16, K=7168, N=2048, act="silu", gated=True, bias=False,
             residual=False, f32=False, save=False),
        # odd sizes, every part of the epilogue at work, the products kept for the backward pass
        dict(name="linear_odd", op="linear", M=777, K=1000, N=1112, act="gelu", gated=False, bias=True, residual=True,
             f32=False, save=True),
        # the shared expert of a prefill batch: gate and up
        dict(name="linear_up", op="linear", M=4096, K=7168, N=2048, act="silu", gated=True, bias=False,
             residual=False, f32=False, save=False),
        # and down, onto the routed experts' result
        dict(name="linear_down", op="linear", M=4096, K=2048, N=7168, act=None, gated=False, bias=False,
             residual=True, f32=False, save=False),
        # a small fine-tuning batch, back
        dict(name="back_small", op="back", M=100, K=1000, N=512, act="gelu_tanh", gated=False, bias=True, f32=False,
             w32=False),
        # the router's logits back: fp32 gradients in, fp32 weights' gradient out
        dict(name="back_logits", op="back", M=4096, K=7168, N=256, act=None, gated=False, bias=False, f32=True,
             w32=True),
        # the shared expert's first half back, at a training batch
        dict(name="back_up", op="back", M=4096, K=7168, N=2048, act="silu", gated=True, bias=False, f32=False,
             w32=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("few", "linear", "back"))
    if op == "few":
        fp8 = rng.random() < 0.6
        E = _spread(rng, 1, 60 if fp8 else 30)
        unit, most = (128, (56, 16)) if fp8 else (8, (896, 256))
        return dict(op=op, T=_spread(rng, 1, 64), E=E, k=rng.randint(1, min(8, E)), H=unit * _spread(rng, 1, most[0]),
                    I=unit * _spread(rng, 1, most[1]), fp8=fp8, masked=rng.choice((0.0, 0.1)),
                    residual=rng.random() < 0.5)
    gated = rng.random() < 0.4
    N = 8 * _spread(rng, 1, 256 if gated else 512)
    case = dict(op=op, M=_spread(rng, 1, 4096), K=8 * _spread(rng, 1, 896), N=N,
                act=rng.choice(("relu", "silu", "gelu", "gelu_tanh") + (() if gated else (None, None))), gated=gated,
                bias=rng.random() < 0.5)
    if op == "linear":
        return dict(case, residual=rng.random() < 0.5, f32=rng.random() < 0.3, save=rng.random() < 0.4)
    return dict(case, f32=rng.random() < 0.3, w32=rng.random() < 0.3)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 6151 + 5)


def _fp8_weights(E, N, K, g):
    """e4m3 weights [E, N, K] whose blocks of 128 by 128 fill the format's range, with the scale of each."""
    q = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    for e in range(E):
        q[e] = torch.randn(N, K, generator=g, device=DEV).mul_(105.0).clamp_(-448, 448).to(F8).view(torch.uint8)
    s = torch.rand(E, -(-N // 128), K // 128, generator=g, device=DEV) + 0.5
    return q, s / (105.0 * math.sqrt(K))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    if c["op"] == "few":
        T, E, k, H, I = (c[n] for n in "TEkHI")
        s["x"] = torch.randn(T, H, generator=g, device=DEV).to(BF)
        idx = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].contiguous()
        if c["masked"]:
            idx = torch.where(torch.rand(T, k, generator=g, device=DEV) < c["masked"], -1, idx)
        s["idx"], s["w"] = idx, torch.randn(T, k, generator=g, device=DEV).softmax(1)
        if c["fp8"]:
            s["up"], s["up_s"] = _fp8_weights(E, 2 * I, H, g)
            s["down"], s["down_s"] = _fp8_weights(E, H, I, g)
        else:
            s["up"] = (torch.randn(E, 2 * I, H, generator=g, device=DEV) / math.sqrt(H)).to(BF)
            s["down"] = (torch.randn(E, H, I, generator=g, device=DEV) / math.sqrt(I)).to(BF)
            s["up_s"] = s["down_s"] = None
        s["r"] = torch.randn(T, H, generator=g, device=DEV).to(BF) if c["residual"] else None
        return s
    M, K, N = c["M"], c["K"], c["N"]
    wide = 2 * N if c["gated"] else N
    s["x"] = torch.randn(M, K, generator=g, device=DEV).to(BF)
    s["w"] = (torch.randn(wide, K, generator=g, device=DEV) / math.sqrt(K)).to(BF)
    s["b"] = torch.randn(wide, generator=g, device=DEV) * 0.1 if c["bias"] else None
    if c["op"] == "linear":
        s["r"] = torch.randn(M, N, generator=g, device=DEV).to(BF) if c["residual"] else None
        return s
    # a gradient of the size that a mean loss over the batch has, and the products that the forward pass kept
    s["dy"] = (torch.randn(M, N, generator=g, device=DEV) / M).to(torch.float32 if c["f32"] else BF)
    s["z"] = None
    if c["act"] is not None:
        z = s["x"].float() @ s["w"].float().t()
        s["z"] = (z if s["b"] is None else z + s["b"]).to(BF)
    return s


# --------------------------------------------------------------------------- one pass

def run(state):
    return {"few": _few, "linear": _linear, "back": _back}[state["op"]](state)


def _few(s):
    if own:
        from combine_dispatch_layout_02_amd import ep
        return ep.moe_few(s["x"], s["idx"], s["w"], s["up"], s["down"], s["up_s"], s["down_s"], residual=s["r"])
    x = s["x"].float()
    T, H = x.shape
    y = torch.zeros_like(x) if s["r"] is None else s["r"].float()
    for e in range(s["E"]):   # every expert over every token, weighted by what the token gives it
        share = torch.where(s["idx"] == e, s["w"], 0).sum(1, keepdim=True)
        up, down = (_wide(s[n][e], None if s[n + "_s"] is None else s[n + "_s"][e]) for n in ("up", "down"))
        gate, lin = (x @ up.t()).chunk(2, 1)
        y = y + share * ((gate / (1 + torch.exp(-gate)) * lin) @ down.t())
    return y.to(BF)


def _wide(w, scales):
    """Weights in fp32."""
    if scales is None:
        return w.float()
    N, K = w.shape
    v = w.view(F8).float().view(N, K // 128, 128)
    return (v * scales.repeat_interleave(128, 0)[:N, :, None]).view(N, K)


def _act(z, act):
    """An activation and its derivative."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0), (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(z * -math.sqrt(0.5))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    # gelu_tanh: (1 + tanh(a)) / 2 is the sigmoid of 2 a
    a = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    p = 1 / (1 + torch.exp(-a))
    return z * p, p + z * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    out = torch.float32 if s["f32"] else BF
    if own:
        from combine_dispatch_layout_02_amd import ep
        return ep.linear(s["x"], s["w"], s["b"], s["r"], activation=s["act"], gated=s["gated"], out_dtype=out,
                         save=s["save"])
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    if s["gated"]:
        gate, lin = z.chunk(2, 1)
        y = _act(gate, s["act"])[0] * lin
    else:
        y = _act(z, s["act"])[0]
    if s["r"] is not None:
        y = y + s["r"].float()
    return (y.to(out), z.to(BF)) if s["save"] else y.to(out)


def _back(s):
    w_type = torch.float32 if s["w32"] else BF
    if own:
        from combine_dispatch_layout_02_amd import ep
        return ep.linear_backward(s["dy"], s["x"], s["w"], s["z"], activation=s["act"], gated=s["gated"],
                                  bias=s["bias"], grad_w_dtype=w_type)
    dz = s["dy"].float()
    if s["gated"]:
        gate, lin = s["z"].float().chunk(2, 1)
        a, da = _act(gate, s["act"])
        dz = torch.cat((dz * lin * da, dz * a), 1)
    elif s["act"] is not None:
        dz = dz * _act(s["z"].float(), s["act"])[1]
    dx = (dz @ s["w"].float()).to(BF)
    dw = (dz.t() @ s["x"].float()).to(w_type)
    return (dx, dw, dz.sum(0)) if s["bias"] else (dx, dw)


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "few":
        T, E, k, H, I = (c[n] for n in "TEkHI")
        used = E * (1 - (1 - k * (1 - c["masked"]) / E) ** T)   # experts that get a token, on average
        b = used * 3 * H * I * (1 if c["fp8"] else 2)
        if c["fp8"]:
            b += used * 4 * (-(-2 * I // 128) * (H // 128) + -(-H // 128) * (I // 128))
        b += T * H * (6 if c["residual"] else 4) + T * k * 12
        return dict(bytes=b, flops=6 * T * k * (1 - c["masked"]) * H * I)
    M, K, N = c["M"], c["K"], c["N"]
    wide = 2 * N if c["gated"] else N
    b = 2 * M * K + 2 * wide * K + M * N * (4 if c["f32"] else 2)
    if c["op"] == "linear":
        b += (4 * wide if c["bias"] else 0) + (2 * M * N if c["residual"] else 0) + (2 * M * wide if c["save"] else 0)
        return dict(bytes=b, flops=2 * M * wide * K)
    b += 2 * M * K + wide * K * (4 if c["w32"] else 2) + (4 * wide if c["bias"] else 0)
    b += 0 if c["act"] is None else 2 * M * wide
    return dict(bytes=b, flops=4 * M * wide * K)


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"few": _exact_few, "linear": _exact_linear, "back": _exact_back}[case["op"]](s)


def _exact_few(s):
    x = s["x"].double()
    y = torch.zeros_like(x)
    idx = s["idx"].cpu()
    for e in idx[idx >= 0].unique().tolist():
        t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
        rows, I = x[t], s["I"]
        w1, w2 = s["up"][e], s["down"][e]
        if s["fp8"]:
            tile = torch.ones(128, 128, dtype=torch.float64, device=DEV)
            w1 = w1.view(F8).double() * torch.kron(s["up_s"][e].double(), tile)
            w2 = w2.view(F8).double() * torch.kron(s["down_s"][e].double(), tile)[:s["H"]]
        w1, w2 = w1.double(), w2.double()
        g = torch.matmul(rows, w1[:I].t())
        h = g * torch.sigmoid(g) * torch.matmul(rows, w1[I:].t())
        y.index_add_(0, t, s["w"][t, j].double()[:, None] * torch.matmul(h, w2.t()))
    return y if s["r"] is None else y + s["r"].double()


_EXACT_ACT = {
    None: lambda z: z,
    "relu": torch.relu,
    "silu": lambda z: z * torch.sigmoid(z),
    "gelu": lambda z: 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0)),
    "gelu_tanh": lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))),
}


def _exact_linear(s):
    z = torch.matmul(s["x"].double(), s["w"].double().t())
    if s["b"] is not None:
        z += s["b"].double()
    f = _EXACT_ACT[s["act"]]
    y = f(z[:, :s["N"]]) * z[:, s["N"]:] if s["gated"] else f(z)
    if s["r"] is not None:
        y = y + s["r"].double()
    return (y, z) if s["save"] else y


def _exact_back(s):
    dy = s["dy"].double()
    dz = dy
    if s["act"] is not None:   # by automatic differentiation of the definition
        z = s["z"].double().requires_grad_()
        f = _EXACT_ACT[s["act"]]
        y = f(z[:, :s["N"]]) * z[:, s["N"]:] if s["gated"] else f(z)
        dz, = torch.autograd.grad(y, z, dy)
    out = (torch.matmul(dz, s["w"].double()), torch.matmul(dz.t(), s["x"].double()))
    return out + (dz.sum(0),) if s["bias"] else out
