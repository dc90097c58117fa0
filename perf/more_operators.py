"""The operators around and in place of the feed-forward block as they are
timed and compared: each in its plain form (elementary torch operations) and
through this library.

  linear       residual + act(x W + bias), bf16 operands (inference)
  linear train the same, and the gradients of x, W and bias
  norm         s = residual + scale * gate * post-norm(y), n = pre-norm(s)
  norm train   the same, and the gradients of y, residual, gate and weights
  moe          router, top-k, gated experts and their weighted sum, few tokens

A case's sizes: M rows (tokens), K inputs, N outputs, F gated outputs of an
expert, E experts of which each token takes ``top``; ``pad`` is the number of
unused elements behind each stored row of the operands; ``groups`` the number
of gate rows, each for M / groups consecutive rows (0: no gate).
"""

import math

import torch

own = False


def listed():
    return [
        # single token through an attention block's output projection
        {"name": "linear token 1x5120x5120", "op": "linear", "M": 1, "N": 5120, "K": 5120,
         "act": "none", "bias": True, "res": True, "out": "bf16", "pad": 0},
        # a decode batch through the up projection of a block without a gate
        {"name": "linear decode 48x16384x4096", "op": "linear", "M": 48, "N": 16384, "K": 4096,
         "act": "gelu_tanh", "bias": True, "res": False, "out": "bf16", "pad": 0},
        # a prompt of odd length through the down projection, onto an fp32 residual stream
        {"name": "linear prompt 2047x5120x13824", "op": "linear", "M": 2047, "N": 5120, "K": 13824,
         "act": "none", "bias": True, "res": True, "out": "fp32", "pad": 8},
        # a training step on few tokens, ragged in both directions
        {"name": "linear train 333x1000x520", "op": "linear", "train": True, "M": 333, "N": 1000,
         "K": 520, "act": "silu", "bias": True, "res": True, "out": "bf16", "pad": 8},
        # a training step on a full micro-batch
        {"name": "linear train 4096x13824x5120", "op": "linear", "train": True, "M": 4096,
         "N": 13824, "K": 5120, "act": "gelu_tanh", "bias": True, "res": False, "out": "bf16",
         "pad": 0},
        # one step of a small decode batch, between two blocks
        {"name": "norm decode 8x5120", "op": "norm", "M": 8, "K": 5120, "post": True, "groups": 1,
         "res": "bf16", "pad": 0},
        # a prompt's rows
        {"name": "norm prompt 8192x5120", "op": "norm", "M": 8192, "K": 5120, "post": True,
         "groups": 1, "res": "bf16", "pad": 0},
        # ragged rows of an odd length, one gate per sequence of a batch, fp32 residual stream
        {"name": "norm train 1113x2049", "op": "norm", "train": True, "M": 1113, "K": 2049,
         "post": True, "groups": 7, "res": "fp32", "pad": 3},
        # a full micro-batch, a learned gate per channel
        {"name": "norm train 8192x4096", "op": "norm", "train": True, "M": 8192, "K": 4096,
         "post": True, "groups": 1, "res": "bf16", "pad": 0},
        # single token, many small experts
        {"name": "moe token 1 of 64x2048x1024", "op": "moe", "M": 1, "K": 2048, "F": 1024, "E": 64,
         "top": 8, "act": "silu", "pad": 0},
        # a ragged decode batch, few large experts
        {"name": "moe decode 13 of 8x4096x13824", "op": "moe", "M": 13, "K": 4096, "F": 13824,
         "E": 8, "top": 2, "act": "silu", "pad": 0},
        # the largest decode batch, most experts hit
        {"name": "moe decode 64 of 128x2048x768", "op": "moe", "M": 64, "K": 2048, "F": 768,
         "E": 128, "top": 8, "act": "silu", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: mostly a multiple of 16, one in four any number."""
    k = _log_int(rng, lo, hi)
    return k if rng.random() < 0.25 else max(16, k // 16 * 16)


def draw(rng):
    kind = rng.choice(["linear", "linear train", "norm", "norm train", "moe"])
    pad = rng.choice([0, 0, 8, 16, 3])
    if kind == "moe":
        c = {"op": "moe", "M": _log_int(rng, 1, 64), "K": _width(rng, 64, 4096),
             "F": _width(rng, 32, 4096), "E": _log_int(rng, 2, 128),
             "act": rng.choice(["silu", "gelu_tanh"]), "pad": pad}
        c["top"] = rng.randint(1, min(8, c["E"]))
        c["E"] = max(c["top"], min(c["E"], (1 << 30) // (3 * c["K"] * c["F"])))
        return c
    if kind.startswith("norm"):
        c = {"op": "norm", "M": _log_int(rng, 1, 8192), "K": _width(rng, 16, 13824),
             "post": rng.random() < 0.75, "groups": rng.choice([0, 1, 1, 3, -1]),
             "res": rng.choice(["bf16", "bf16", "fp32"]), "pad": pad}
        if c["groups"] == 3:  # sequences of one batch
            c["M"] = max(3, c["M"] // 3 * 3)
        if c["groups"] < 0:  # a gate per token
            c["M"] = min(c["M"], 2048)
            c["groups"] = c["M"]
    else:
        c = {"op": "linear", "M": _log_int(rng, 1, 4096), "N": _width(rng, 16, 13824),
             "K": _width(rng, 32, 5120), "act": rng.choice(["none", "relu", "silu", "gelu_tanh"]),
             "bias": rng.random() < 0.75, "res": rng.random() < 0.5,
             "out": rng.choice(["bf16", "bf16", "fp32"]), "pad": pad}
    if kind.endswith("train"):
        c["train"] = True
    return c


def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    train = case.get("train", False)
    if op == "norm":
        G, r = case["groups"], 2 if case["res"] == "bf16" else 4
        w = 2 * K * (1 + case["post"]) + 2 * G * K
        # y, residual in; s, n out
        b, f = M * K * (2 + r + r + 2) + w, 12 * M * K
        if train:  # dn, ds in; dy, dresidual and the sums out
            b += M * K * (2 + r + 2 + r) + 4 * K * (1 + case["post"]) + 4 * G * K
            f += 24 * M * K
        return {"bytes": b, "flops": f}
    if op == "moe":
        E, F, k = case["E"], case["F"], case["top"]
        hit = E * (1.0 - (1.0 - k / E) ** M)  # experts that some token takes
        return {"bytes": int(hit * 6 * K * F) + 2 * E * K + 4 * M * K + 8 * M * k,
                "flops": 6 * M * k * K * F + 2 * M * E * K}
    N, o = case["N"], 2 if case["out"] == "bf16" else 4
    b = 2 * (M * K + K * N) + o * M * N * (1 + case["res"]) + 2 * N * case["bias"]
    if train:  # dy in; dx, dw, db out
        return {"bytes": b + 2 * M * N + 2 * (M * K + K * N) + 4 * N * case["bias"],
                "flops": 6 * M * N * K}
    return {"bytes": b, "flops": 2 * M * N * K}


# ---- inputs ------------------------------------------------------------------


def _rows(g, M, K, pad, std=1.0, dtype=torch.bfloat16):
    """[M, K] with ``pad`` unused elements behind each row."""
    x = torch.randn(M, K + pad, generator=g, device="cuda", dtype=torch.float32).mul_(std)
    return x.to(dtype)[:, :K]


def _vector(g, K, mean, std):
    return (mean + std * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)


def _experts(g, E, rows, K, pad, std):
    w = torch.empty(E, rows, K + pad, dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        w[e] = _rows(g, rows, K + pad, 0, std)
    return w[:, :, :K]


_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, M, K, pad = case["op"], case["M"], case["K"], case["pad"]
    train = case.get("train", False)
    s = dict(case, train=train)
    if op == "linear":
        N, out = case["N"], _TYPES[case["out"]]
        s["x"] = _rows(g, M, K, pad)
        s["w"] = _rows(g, N, K, pad, 1.0 / math.sqrt(K))
        s["b"] = _vector(g, N, 0.0, 0.5) if case["bias"] else None
        s["r"] = _rows(g, M, N, pad, 2.0, out) if case["res"] else None
        if train:
            s["dy"] = _rows(g, M, N, pad)
        return s
    if op == "norm":
        res = _TYPES[case["res"]]
        s["y"] = _rows(g, M, K, pad)
        s["h"] = _rows(g, M, K, pad, 2.0, res)
        # a few channels far above the rest, as hidden states have them, and a
        # padding row of zeros
        s["h"][:, :: max(1, K // 7)] *= 20.0
        if M > 2:
            s["y"][M // 2] = 0.0
            s["h"][M // 2] = 0.0
        s["wn"] = _vector(g, K, 1.0, 0.1)
        s["wp"] = _vector(g, K, 1.0, 0.1) if case["post"] else None
        G = case["groups"]
        s["g"] = _vector(g, G * K, 0.3, 0.1).view(G, K) if G else None
        s["scale"], s["eps"] = 0.5, 1e-6
        if train:
            s["dn"] = _rows(g, M, K, pad)
            s["ds"] = _rows(g, M, K, pad, 1.0, res)
        return s
    E, F = case["E"], case["F"]
    s["x"] = _rows(g, M, K, pad)
    if M > 2:
        s["x"][M // 2] = 0.0  # a padding token: every expert ties
    s["router"] = _rows(g, E, K, pad, 1.5 / math.sqrt(K))
    s["w1"] = _experts(g, E, 2 * F, K, pad, 1.0 / math.sqrt(K))
    s["w2"] = _experts(g, E, K, F, pad, 1.0 / math.sqrt(F))
    return s


# ---- one pass ----------------------------------------------------------------


def _act(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    t = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return 0.5 * z * (1.0 + torch.tanh(t))


def _act_grad(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).float()
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z)


def _linear(s):
    x, w = s["x"].float(), s["w"].float()
    z = torch.mm(x, w.t())
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(_TYPES[s["out"]])
    if not s["train"]:
        return y
    dz = s["dy"].float() * _act_grad(z, s["act"])
    o = {"y": y, "dx": torch.mm(dz, w).to(torch.bfloat16), "dw": torch.mm(dz.t(), x).to(torch.bfloat16)}
    if s["b"] is not None:
        o["db"] = dz.sum(dim=0)
    return o


def _norm(s):
    y, h, wn = s["y"].float(), s["h"].float(), s["wn"].float()
    M, K = y.shape
    ry = None
    p = y
    if s["wp"] is not None:
        ry = 1.0 / torch.sqrt((y * y).mean(dim=1, keepdim=True) + s["eps"])
        p = y * ry * s["wp"].float()
    a = s["scale"]
    if s["g"] is not None:
        a = a * s["g"].float().repeat_interleave(M // s["groups"], dim=0)
    t = h + a * p
    rs = 1.0 / torch.sqrt((t * t).mean(dim=1, keepdim=True) + s["eps"])
    o = {"n": (t * rs * wn).to(torch.bfloat16), "s": t.to(s["h"].dtype)}
    if not s["train"]:
        return o
    dn = s["dn"].float()
    dt = dn * wn
    dt = s["ds"].float() + rs * dt - t * (rs * rs * rs / K) * (dt * t).sum(dim=1, keepdim=True)
    o["dwn"] = (dn * t * rs).sum(dim=0)
    o["dh"] = dt.to(s["h"].dtype)
    if s["g"] is not None:
        o["dg"] = (s["scale"] * dt * p).view(s["groups"], -1, K).sum(dim=1)
    dp = a * dt
    if s["wp"] is not None:
        o["dwp"] = (dp * y * ry).sum(dim=0)
        dp = dp * s["wp"].float()
        dp = ry * dp - y * (ry * ry * ry / K) * (dp * y).sum(dim=1, keepdim=True)
    o["dy"] = dp.to(torch.bfloat16)
    return o


def _moe(s):
    x, F = s["x"].float(), s["F"]
    # (64 bits: which experts a token takes must not depend on the order of a sum)
    logits = torch.mm(s["x"].double(), s["router"].double().t())
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :s["top"]], ids[:, :s["top"]]
    p = torch.exp((top - top[:, :1]).float())
    p = p / p.sum(dim=1, keepdim=True)
    M, E = logits.shape
    if ids.numel() < E:  # the experts of each choice
        gu = torch.bmm(s["w1"][ids.reshape(-1)].float(),
                       x.repeat_interleave(s["top"], dim=0)[:, :, None])
        a = _act(gu[:, :F], s["act"]) * gu[:, F:]
        y = torch.bmm(s["w2"][ids.reshape(-1)].float(), a)[:, :, 0]
        y = (p[:, :, None] * y.view(M, s["top"], -1)).sum(dim=1)
    else:  # every token through every expert, with a share of 0 where it takes others
        gu = torch.mm(s["w1"].float().reshape(E * 2 * F, -1), x.t().contiguous()).view(E, 2 * F, M)
        a = _act(gu[:, :F], s["act"]) * gu[:, F:]
        share = torch.zeros(M, E, dtype=torch.float32, device=x.device).scatter_(1, ids, p)
        y = torch.bmm(s["w2"].float(), a * share.t()[:, None, :]).sum(dim=0).t()
    return {"y": y.to(torch.bfloat16), "ids": ids.int(), "p": p}


def run(s):
    if own:
        return _run_own(s)
    return {"linear": _linear, "norm": _norm, "moe": _moe}[s["op"]](s)


def _run_own(s):
    from layout_aware_gemm_amd import tgemm

    if s["op"] == "linear":
        kw = {"bias": s["b"], "act": s["act"], "residual": s["r"], "out_dtype": _TYPES[s["out"]]}
        if not s["train"]:
            return tgemm.linear(s["x"], s["w"].t(), **kw)
        y, z = tgemm.linear(s["x"], s["w"].t(), save=True, **kw)
        dx, dw, db = tgemm.linear_backward(s["dy"], s["x"], s["w"].t(), z, act=s["act"],
                                           bias=s["b"] is not None)
        o = {"y": y, "dx": dx, "dw": dw.t()}
        if db is not None:
            o["db"] = db
        return o
    if s["op"] == "norm":
        kw = {"post_weight": s["wp"], "gate": s["g"], "scale": s["scale"]}
        if not s["train"]:
            n, t = tgemm.block_norm(s["y"], s["h"], s["wn"], eps=s["eps"], **kw)
            return {"n": n, "s": t}
        n, t, rstd = tgemm.block_norm(s["y"], s["h"], s["wn"], eps=s["eps"], save=True, **kw)
        dh, dy, dwn, dwp, dg = tgemm.block_norm_backward(s["dn"], s["y"], s["h"], rstd, s["wn"],
                                                         ds=s["ds"], **kw)
        o = {"n": n, "s": t, "dwn": dwn, "dh": dh, "dy": dy}
        if dg is not None:
            o["dg"] = dg
        if dwp is not None:
            o["dwp"] = dwp
        return o
    y, ids, p = tgemm.moe(s["x"], s["router"].t(), s["w1"].transpose(1, 2),
                          s["w2"].transpose(1, 2), s["top"], act=s["act"], routing=True)
    return {"y": y, "ids": ids, "p": p}


# ---- 64 bits, from the definitions -------------------------------------------


def _exact_act(z, kind):
    """act(z) and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0.0), (z > 0).double()
    c = 2.0 * math.sqrt(2.0 / math.pi)
    v, dv = (z, 1.0) if kind == "silu" else (c * z * (1.0 + 0.044715 * z ** 2),
                                             c * (1.0 + 0.134145 * z ** 2))
    e = torch.exp(-v.abs())
    up, down = 1.0 / (1.0 + e), e / (1.0 + e)  # the sigmoid's two sides
    p, q = torch.where(v >= 0, up, down), torch.where(v >= 0, down, up)
    return z * p, p + z * p * q * dv


def _exact_linear(s):
    x, w = s["x"].double(), s["w"].double()
    z = torch.mm(x, w.t())
    if s["b"] is not None:
        z += s["b"].double()[None, :]
    y, slope = _exact_act(z, s["act"])
    if s["r"] is not None:
        y = y + s["r"].double()
    if not s["train"]:
        return y
    dz = slope * s["dy"].double()
    o = {"y": y, "dx": torch.mm(dz, w), "dw": torch.mm(dz.t(), x)}
    if s["b"] is not None:
        o["db"] = torch.mv(dz.t(), torch.ones(dz.shape[0], dtype=dz.dtype, device=dz.device))
    return o


def _exact_rms(v, w, eps, d=None):
    """v / rms(v) * w; with d, the gradients of v and w for d on the result."""
    rms = torch.sqrt(v.square().sum(dim=1, keepdim=True) / v.shape[1] + eps)
    unit = v / rms
    if d is None:
        return unit * w
    e = d * w
    along = (e * unit).sum(dim=1, keepdim=True) / v.shape[1]
    return (e - unit * along) / rms, (d * unit).sum(dim=0)


def _exact_norm(s):
    y, h, wn = s["y"].double(), s["h"].double(), s["wn"].double()
    wp = None if s["wp"] is None else s["wp"].double()
    (M, K), G = y.shape, s["groups"]
    p = y if wp is None else _exact_rms(y, wp, s["eps"])
    by_group = (lambda v: v.reshape(G, M // G, K)) if G else None
    gate = s["g"].double()[:, None, :] if G else None
    t = h + s["scale"] * ((by_group(p) * gate).reshape(M, K) if G else p)
    o = {"n": _exact_rms(t, wn, s["eps"]), "s": t}
    if not s["train"]:
        return o
    dt, o["dwn"] = _exact_rms(t, wn, s["eps"], s["dn"].double())
    dt = dt + s["ds"].double()
    o["dh"] = dt
    dp = s["scale"] * dt
    if G:
        o["dg"] = (by_group(dp) * by_group(p)).sum(dim=1)
        dp = (by_group(dp) * gate).reshape(M, K)
    o["dy"] = dp
    if wp is not None:
        o["dy"], o["dwp"] = _exact_rms(y, wp, s["eps"], dp)
    return o


def _exact_moe(s):
    x, F, k = s["x"].double(), s["F"], s["top"]
    logits = torch.mm(x, s["router"].double().t())
    left, ids, y = logits.clone(), [], torch.zeros_like(x)
    for _ in range(k):  # the largest that is left, the first of equals
        best = left == left.max(dim=1, keepdim=True).values
        ids.append(best.int().argmax(dim=1))
        left[torch.arange(x.shape[0], device=x.device), ids[-1]] = -math.inf
    ids = torch.stack(ids, dim=1)
    p = torch.softmax(logits.gather(1, ids), dim=1)
    for e in range(s["E"]):
        share = (p * (ids == e)).sum(dim=1)  # of each token, 0 where it takes others
        rows = share.nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        w1 = s["w1"][e].double()
        g, u = torch.mm(x[rows], w1[:F].t()), torch.mm(x[rows], w1[F:].t())
        a = _exact_act(g, s["act"])[0] * u * share[rows, None]
        y[rows] += torch.mm(a, s["w2"][e].double().t())
    return {"y": y, "ids": ids.int(), "p": p}


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "norm": _exact_norm, "moe": _exact_moe}[s["op"]](s)
