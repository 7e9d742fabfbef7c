"""The transformer block's operators around its attention, case by case: layer
normalisation (forward and backward), the gated feed-forward (forward and
backward) and the projection with low-rank adapters.

`run` computes one pass of a case: with `own` false in plain 32-bit torch
operations, with `own` true by the library's calls.  `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}
EPS = 1e-5


def _norm(op, dtype, T, C, name=None):
    c = {"op": op, "dtype": dtype, "T": T, "C": C}
    return c if name is None else {"name": name, **c}


def _ff(op, dtype, T, C, F, name=None):
    c = {"op": op, "dtype": dtype, "T": T, "C": C, "F": F}
    return c if name is None else {"name": name, **c}


def _adapter(dtype, G, N, C, K, R, L, bias, name=None):
    c = {"op": "adapter_linear", "dtype": dtype, "G": G, "N": N, "C": C, "K": K, "R": R, "L": L, "bias": bias}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # the block's norms at the UNet's 64x64 level, a guidance pair of images
        _norm("layer_norm", "fp16", 8192, 320, "norm 64x64 pair"),
        # the text encoding of one prompt pair: few rows, latency
        _norm("layer_norm", "bf16", 154, 768, "norm text pair"),
        # the same norm's backward pass when the block is fine-tuned
        _norm("layer_norm_backward", "bf16", 8192, 320, "norm backward 64x64 pair"),
        # a training batch of 16 images, 32-bit residual stream
        _norm("layer_norm_backward", "fp32", 65536, 320, "norm backward 64x64 batch"),
        # the feed-forward's gated projection at the 64x64 level
        _ff("gated_ff", "fp16", 8192, 320, 1280, "gated 64x64 pair"),
        # the mid block: few rows against wide weights
        _ff("gated_ff", "bf16", 128, 1280, 5120, "gated 8x8 pair"),
        # 16 images at once
        _ff("gated_ff", "fp16", 65536, 320, 1280, "gated 64x64 batch"),
        # fine-tuning: gradients of the input, the weight and the bias
        _ff("gated_ff_backward", "bf16", 8192, 320, 1280, "gated backward 64x64 pair"),
        # a cropped image at the 16x16 level: rows that fill no tile
        _ff("gated_ff_backward", "fp16", 500, 1280, 5120, "gated backward ragged"),
        # cross-attention's key projection of the text of one prompt pair
        _adapter("fp16", 2, 77, 768, 320, 8, 2, False, "adapters text keys"),
        # self-attention's projection for 16 users' images, each with its own style adapter
        _adapter("bf16", 16, 4096, 320, 320, 16, 8, True, "adapters 64x64 batch"),
        # the time embedding's projection: one row a request
        _adapter("fp16", 48, 1, 1280, 1280, 32, 12, True, "adapters one row each"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "gated_ff", "gated_ff_backward", "adapter_linear"])
    if op.startswith("layer_norm"):
        C = _log(rng, 8, 4096)
        T = max(1, min(_log(rng, 1, 65536), 65536 * 320 // C))
        return _norm(op, rng.choice(["fp16", "bf16", "fp32"]), T, C)
    dtype = rng.choice(["fp16", "bf16"])
    if op.startswith("gated_ff"):
        C, F = 8 * _log(rng, 4, 200), 8 * _log(rng, 4, 640)
        most = 65536 * 320 * 1280 // (3 if op.endswith("backward") else 1)
        return _ff(op, dtype, max(1, min(_log(rng, 1, 16384), most // (C * F))), C, F)
    G, C, K = _log(rng, 1, 64), 8 * _log(rng, 4, 200), 8 * _log(rng, 4, 320)
    N = max(1, min(_log(rng, 1, 4096), 65536 * 320 // (G * max(C, K))))
    return _adapter(dtype, G, N, C, K, rng.choice([8, 16, 24, 32, 64, 128]), _log(rng, 1, 32), rng.random() < 0.5)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"op": op, "dtype": dt}
    if op.startswith("layer_norm"):
        T, C = case["T"], case["C"]
        # a residual stream: rows of their own scale and offset, a few wide channels
        x = normal(T, C) * torch.exp(0.5 * normal(T, 1)) + 0.5 * normal(T, 1)
        x[:, :: 97] *= 8.0
        s["x"] = x.to(dt)
        s["gamma"], s["beta"] = 1.0 + 0.2 * normal(C), 0.2 * normal(C)
        if op.endswith("backward"):
            s["dy"] = (0.1 * normal(T, C)).to(dt)
            # what the forward pass left: mean and 1 / sqrt(var + eps) of each row
            x64 = s["x"].double()
            mean, var = x64.mean(1), x64.var(1, unbiased=False)
            s["stats"] = torch.stack([mean, 1.0 / torch.sqrt(var + EPS)], 1).float()
    elif op.startswith("gated_ff"):
        T, C, F = case["T"], case["C"], case["F"]
        s["x"] = normal(T, C).to(dt)
        s["w"] = (normal(2 * F, C) / math.sqrt(C)).to(dt)
        s["bias"] = 0.1 * normal(2 * F)
        if op.endswith("backward"):
            s["dy"] = (0.1 * normal(T, F)).to(dt)
    else:
        G, N, C, K, R, L = (case[k] for k in ("G", "N", "C", "K", "R", "L"))
        s["x"] = normal(G, N, C).to(dt)
        s["w"] = (normal(K, C) / math.sqrt(C)).to(dt)
        s["bias"] = 0.1 * normal(K) if case["bias"] else None
        s["down"] = (normal(L, R, C) / math.sqrt(C)).to(dt)
        s["up"] = (normal(L, K, R) / math.sqrt(R)).to(dt)
        s["scale"] = 0.25 + 0.75 * torch.rand(L, generator=g, device="cuda")
        # an adapter for each request, none (-1) for some
        s["ids"] = torch.randint(-1, L, (G,), generator=g, device="cuda", dtype=torch.int32)
    return s


def _plain_layer_norm(s):
    x = s["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    return (d * rstd * s["gamma"] + s["beta"]).to(s["dtype"])


def _plain_layer_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xhat = (x - mean) * rstd
    dg = dy * s["gamma"]
    dx = rstd * (dg - dg.mean(1, keepdim=True) - xhat * (dg * xhat).mean(1, keepdim=True))
    return dx.to(s["dtype"]), (dy * xhat).sum(0), dy.sum(0)


def _halves(s):
    p = s["x"].float() @ s["w"].float().t() + s["bias"]
    F = p.shape[1] // 2
    h, g = p[:, :F], p[:, F:]
    return h, g, 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))


def _plain_gated_ff(s):
    h, g, cdf = _halves(s)
    return (h * g * cdf).to(s["dtype"])


def _plain_gated_ff_backward(s):
    h, g, cdf = _halves(s)
    dy = s["dy"].float()
    slope = cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    dp = torch.cat([dy * g * cdf, dy * h * slope], 1)
    return (dp @ s["w"].float()).to(s["dtype"]), (dp.t() @ s["x"].float()).to(s["dtype"]), dp.sum(0)


def _plain_adapter_linear(s):
    x, ids = s["x"].float(), s["ids"].long()
    y = x @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    at = ids.clamp(min=0)
    scale = torch.where(ids >= 0, s["scale"][at], torch.zeros_like(s["scale"][at]))
    u = torch.bmm(x, s["down"][at].float().transpose(1, 2)) * scale[:, None, None]
    return (y + torch.bmm(u, s["up"][at].float().transpose(1, 2))).to(s["dtype"])


_PLAIN = {"layer_norm": _plain_layer_norm, "layer_norm_backward": _plain_layer_norm_backward,
          "gated_ff": _plain_gated_ff, "gated_ff_backward": _plain_gated_ff_backward,
          "adapter_linear": _plain_adapter_linear}


def run(s):
    op = s["op"]
    if not own:
        return _PLAIN[op](s)
    import diffusion_unet_attention_b200 as sd
    if op == "layer_norm":
        return sd.layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS)
    if op == "layer_norm_backward":
        return sd.layer_norm_backward(s["dy"], s["x"], s["stats"], s["gamma"])
    if op == "gated_ff":
        return sd.gated_ff(s["x"], s["w"], s["bias"])
    if op == "gated_ff_backward":
        return sd.gated_ff_backward(s["dy"], s["x"], s["w"], s["bias"])
    return sd.adapter_linear(s["x"], s["w"], s["bias"], s["down"], s["up"], s["scale"], s["ids"])


def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op.startswith("layer_norm"):
        T, C = case["T"], case["C"]
        if op == "layer_norm":
            return {"bytes": 2 * T * C * b + 8 * C, "flops": 8 * T * C}
        return {"bytes": 3 * T * C * b + 8 * T + 12 * C, "flops": 14 * T * C}
    if op.startswith("gated_ff"):
        T, C, F = case["T"], case["C"], case["F"]
        product = 2 * T * C * 2 * F
        if op == "gated_ff":
            return {"bytes": b * (T * C + 2 * F * C + T * F) + 8 * F, "flops": product}
        # the projection again, then its two transposed products
        return {"bytes": b * (2 * T * C + 4 * F * C + T * F) + 16 * F, "flops": 3 * product}
    G, N, C, K, R, L = (case[k] for k in ("G", "N", "C", "K", "R", "L"))
    used = L * (1.0 - (1.0 - 1.0 / (L + 1)) ** G)      # adapters that at least one request names, on average
    part = L / (L + 1.0)                               # requests with an adapter, on average
    return {"bytes": b * (G * N * (C + K) + K * C + used * R * (C + K)) + 4 * G + (4 * K if case["bias"] else 0),
            "flops": 2 * G * N * (C * K + part * R * (C + K))}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    x = s["x"].to(torch.float64)
    if op == "layer_norm":
        n = x.shape[1]
        mean = x.sum(1) / n
        var = (x.square().sum(1) - n * mean.square()) / n
        return (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * s["gamma"].double() + s["beta"].double()
    if op == "layer_norm_backward":
        dy, gamma, n = s["dy"].double(), s["gamma"].double(), x.shape[1]
        mean, rstd = s["stats"].double().unbind(1)
        z = torch.einsum("tc,t->tc", x - mean[:, None], rstd)
        a, b = dy @ gamma / n, torch.einsum("tc,tc,c->t", dy, z, gamma) / n
        dx = (torch.einsum("tc,c->tc", dy, gamma) - a[:, None] - z * b[:, None]) * rstd[:, None]
        return dx, torch.einsum("tc,tc->c", dy, z), dy.sum(0)
    if op.startswith("gated_ff"):
        w, F = s["w"].double(), case["F"]
        h = torch.addmm(s["bias"][:F].double(), x, w[:F].t())
        g = torch.addmm(s["bias"][F:].double(), x, w[F:].t())
        act = g * torch.special.ndtr(g)
        if op == "gated_ff":
            return h * act
        dy = s["dy"].double()
        dh = dy * act
        del act
        dg = dy * h * (torch.special.ndtr(g) + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi))
        return dh @ w[:F] + dg @ w[F:], torch.cat([dh.t() @ x, dg.t() @ x]), torch.cat([dh.sum(0), dg.sum(0)])
    y = torch.einsum("gnc,kc->gnk", x, s["w"].double())
    if s["bias"] is not None:
        y += s["bias"].double()
    for r, i in enumerate(s["ids"].tolist()):
        if i >= 0:
            y[r] += s["scale"][i].double() * (x[r] @ s["down"][i].double().t() @ s["up"][i].double().t())
    return y
