"""The operators of a token step, as measured: the root-mean-square norm with
the residual's addition (forward, forward into block-scaled 8 bits, backward),
products with 4-bit weights and group scales, and sampling from given random
numbers.

``run`` computes them in their plain form (elementary torch operations in 32
or 64 bits, rounded once at the end) where ``own`` is false, and through the
framework's entry points (``fgemm.rms_norm``, ``rms_norm_mx``,
``rms_norm_backward``, ``matmul_w4``, ``sample``) where it is true.
``exact`` restates each operator in 64 bits on the host.

Sizes: widths and products come from the token-projection and FFN shapes the
benchmark uses (4096, 14336, 28672 = gate | up, 2048 .. 16384), batches from
one token to a prompt; vocabularies are generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LOGIT_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
EPS = 1e-5


def listed():
    return [
        # one token of a decode step: nothing but latency
        {"name": "norm, one token", "op": "norm", "rows": 1, "width": 4096, "type": "bf16", "residual": True},
        # a ragged batch of an odd width, as after pruning, without a residual (a query / key norm)
        {"name": "norm, odd width", "op": "norm", "rows": 1537, "width": 5127, "type": "f16", "residual": False},
        # a prompt's tokens into the 8-bit product's input
        {"name": "norm to 8 bits, prompt", "op": "norm_mx", "rows": 8192, "width": 4096, "type": "bf16", "residual": True,
         "format": "e4m3"},
        # a training step's tokens, with the gradient that the residual stream brings
        {"name": "norm backward, training", "op": "norm_back", "rows": 8192, "width": 4096, "type": "bf16", "residual": True},
        # a small fine-tuning batch at the width of an FFN's inner norm
        {"name": "norm backward, small batch", "op": "norm_back", "rows": 300, "width": 14336, "type": "f16", "residual": False},
        # one token through a square projection
        {"name": "w4, one token", "op": "w4", "rows": 1, "n": 4096, "k": 4096, "type": "bf16", "group": 128, "zeros": False,
         "epilogue": "none"},
        # a few sequences through gate | up with SwiGLU, weights with zero points
        {"name": "w4, gate and up, 5 tokens", "op": "w4", "rows": 5, "n": 28672, "k": 4096, "type": "bf16", "group": 128,
         "zeros": True, "epilogue": "swiglu"},
        # a serving batch, fine groups
        {"name": "w4, batch of 48", "op": "w4", "rows": 48, "n": 8192, "k": 8192, "type": "f16", "group": 64, "zeros": False,
         "epilogue": "scale_bias"},
        # a prompt through the down projection
        {"name": "w4, prompt", "op": "w4", "rows": 2048, "n": 4096, "k": 14336, "type": "bf16", "group": 128, "zeros": False,
         "epilogue": "none"},
        # one sequence, the usual chat settings
        {"name": "sample, one row", "op": "sample", "rows": 1, "vocab": 32000, "type": "bf16", "top_k": 50, "top_p": 0.95,
         "min_p": 0.0, "masked": 0.0},
        # a serving batch with a large vocabulary, nucleus sampling over all of it
        {"name": "sample, nucleus, batch", "op": "sample", "rows": 64, "vocab": 131072, "type": "f32", "top_k": 0, "top_p": 0.9,
         "min_p": 0.0, "masked": 0.0},
        # constrained decoding: half of an odd vocabulary masked, one row left with nothing; no truncation but min-p
        {"name": "sample, constrained, batch", "op": "sample", "rows": 200, "vocab": 50257, "type": "f16", "top_k": 0,
         "top_p": 1.0, "min_p": 0.02, "masked": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_mx", "norm_back", "w4", "w4", "sample", "sample"])
    if op.startswith("norm"):
        width = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        rows = _log(rng, 1, max(2, min(16384, 8192 * 4096 // width)))
        c = {"op": op, "rows": rows, "width": width, "type": rng.choice(["bf16", "f16"]), "residual": rng.random() < 0.7}
        if op == "norm_mx":
            c["format"] = rng.choice(["e4m3", "e5m2"])
        return c
    if op == "w4":
        n = _log(rng, 256, 28672) // 32 * 32
        k = _log(rng, 256, 16384)
        if rng.random() < 0.8:
            k = k // 128 * 128
        most = max(1, min(2048, 2048 * 4096 * 14336 // (n * k)))
        return {"op": op, "rows": min(most, _log(rng, 1, 512)), "n": n, "k": k, "type": rng.choice(["bf16", "f16"]),
                "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "epilogue": rng.choice(["none", "scale_bias", "silu", "swiglu"])}
    vocab = _log(rng, 1000, 200000)
    return {"op": op, "rows": _log(rng, 1, max(2, min(256, 64 * 131072 // vocab))), "vocab": vocab,
            "type": rng.choice(["bf16", "f16", "f32"]), "top_k": rng.choice([0, 0, 1, 20, 50, 1000]),
            "top_p": rng.choice([1.0, 1.0, 0.5, 0.9, 0.95, 0.999]), "min_p": rng.choice([0.0, 0.0, 0.05]),
            "masked": rng.choice([0.0, 0.0, 0.3])}


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)

    op, rows = case["op"], case["rows"]
    s = {"case": case}
    if op.startswith("norm"):
        t, width = TYPES[case["type"]], case["width"]
        # a residual stream has channels far larger than the rest
        channels = torch.exp(0.5 * normal(width))
        s["gain"] = (1.0 + 0.2 * normal(width)).to(t)
        if op == "norm_back":
            s["total"] = (normal(rows, width) * channels).to(t)
            s["inv_rms"] = torch.rsqrt(s["total"].double().square().mean(1) + EPS).float()
            s["dy"] = (0.1 * normal(rows, width)).to(t)
            s["dtotal"] = (0.1 * normal(rows, width)).to(t) if case["residual"] else None
        else:
            s["x"] = normal(rows, width).to(t)
            s["residual"] = (normal(rows, width) * channels).to(t) if case["residual"] else None
    elif op == "w4":
        t, n, k, group = TYPES[case["type"]], case["n"], case["k"], case["group"]
        groups = -(-k // group)
        s["a"] = normal(rows, -(-k // 8) * 8).to(t)[:, :k]  # rows of whole 16 bytes
        # 4-bit values of weights ~ N(0, 1/k): two to a byte, the even one low
        ld = -(-k // 32) * 16
        lo = torch.clamp(torch.round(8 + 2.7 * normal(n, ld)), 0, 15).to(torch.uint8)
        hi = torch.clamp(torch.round(8 + 2.7 * normal(n, ld)), 0, 15).to(torch.uint8)
        s["w"] = (lo | (hi << 4))[:, :(k + 1) // 2]
        s["scales"] = ((1 + 0.3 * torch.rand((n, groups), generator=g, device=DEV)) / (2.7 * math.sqrt(k))).to(t)
        s["zeros"] = (torch.randint(5, 12, (n, groups), generator=g, device=DEV, dtype=torch.uint8)
                      if case["zeros"] else None)
        s["bias"] = (0.02 * normal(n)).to(t) if case["epilogue"] in ("scale_bias", "silu") else None
        s["alpha"] = 1.0 if case["epilogue"] != "scale_bias" else 0.5
    else:
        t, vocab = LOGIT_TYPES[case["type"]], case["vocab"]
        x = 2.5 * normal(rows, vocab)
        # a few likely continuations in each row
        likely = torch.randint(0, vocab, (rows, 16), generator=g, device=DEV)
        x.scatter_add_(1, likely, 3 + 2.0 * normal(rows, 16))
        if case["masked"]:
            x.masked_fill_(torch.rand((rows, vocab), generator=g, device=DEV) < case["masked"], -math.inf)
            if rows > 1:
                x[rows // 2] = -math.inf
        s["logits"] = x.to(t)
        # every request has settings of its own
        each = torch.rand((4, rows), generator=g, device=DEV)
        s["temperature"] = 0.6 + 0.8 * each[0]
        s["top_k"] = torch.full((rows,), case["top_k"], dtype=torch.int32, device=DEV)
        s["top_p"] = (case["top_p"] - 0.05 * each[1]) if case["top_p"] < 1 else torch.ones(rows, device=DEV)
        s["min_p"] = case["min_p"] * (0.5 + each[2])
        s["u"] = torch.rand(rows, generator=g, device=DEV)
    return s


# -------------------------------------------------------------- plain forms


def _plain_norm(s):
    x = s["x"]
    total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    t = total.float()
    inv = torch.rsqrt(t.double().square().mean(1).float() + EPS)
    return total, inv, t * inv[:, None] * s["gain"].float()


def _plain_mx(y, fmt):
    """Blocks of 32 along each row: scale 2^(floor(log2 max|y|) - emax) with
    its exponent held to E8M0's range, elements y / scale clamped to the
    largest finite value and rounded to nearest even."""
    rows, width = y.shape
    blocks = -(-width // 32)
    y = torch.nn.functional.pad(y, (0, blocks * 32 - width)).view(rows, blocks, 32)
    emax, top = (8, 448.0) if fmt == "e4m3" else (15, 57344.0)
    amax = y.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - emax, -127).clamp(-127, 127)
    q = (y.double() * torch.exp2(-e.double())[:, :, None]).clamp(-top, top).float()
    q = q.reshape(rows, blocks * 32)[:, :width].to(F8[fmt])
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_norm_back(s):
    dy, t, inv, gain = s["dy"].float(), s["total"].float(), s["inv_rms"][:, None], s["gain"].float()
    gdy = dy * gain
    dot = (gdy * t).double().mean(1, keepdim=True).float()
    dx = inv * gdy - t * (inv * inv * inv * dot)
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    dgain = (dy * t * inv).double().sum(0).float()
    return dx.to(s["dy"].dtype), dgain


def _epilogue(v, kind):
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "swiglu":
        half = v.shape[1] // 2
        gate = v[:, :half]
        return gate / (1 + torch.exp(-gate)) * v[:, half:]
    return v


def _weights(w, scales, zeros, k, group, to):
    q = torch.stack((w & 15, w >> 4), 2).flatten(1)[:, :k].to(to)
    z = torch.full_like(scales, 8) if zeros is None else zeros
    each = torch.arange(k, device=w.device) // group
    return (q - z.to(to)[:, each]) * scales.to(to)[:, each]


def _plain_w4(s):
    c = s["case"]
    w = _weights(s["w"], s["scales"], s["zeros"], c["k"], c["group"], torch.float32)
    v = s["alpha"] * (s["a"].float() @ w.t())
    if s["bias"] is not None:
        v = v + s["bias"].float()
    return _epilogue(v, c["epilogue"]).to(s["a"].dtype)


def _plain_sample(s):
    x = s["logits"].double()
    rows, vocab = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    m = x.amax(1, keepdim=True)
    t = s["temperature"].double()[:, None]
    w = torch.where(x == m, 1.0, torch.exp((x - m) / t))
    w = torch.where(x == -math.inf, 0.0, w)
    ws, order = torch.sort(x, dim=1, descending=True, stable=True)
    ws = w.gather(1, order)
    rank = torch.arange(vocab, device=x.device)[None]
    k = s["top_k"].long()[:, None]
    keep = (k <= 0) | (rank < k)
    ws = torch.where(keep, ws, 0.0)
    cum = ws.cumsum(1)
    p = s["top_p"].double()[:, None]
    before = cum - ws
    keep &= (p >= 1) | (before < p * cum[:, -1:])
    keep &= (ws >= s["min_p"].double()[:, None])
    keep |= rank == 0
    keep &= x.gather(1, order) > -math.inf
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0.0))
    cum = kept.cumsum(1)
    z = cum[:, -1:]
    hit = (cum > s["u"].double()[:, None] * z) & (kept > 0)
    first = torch.where(hit, rank, vocab).amin(1)
    last = torch.where(kept > 0, rank, -1).amax(1)
    token = torch.where(first < vocab, first, last)
    prob = kept.gather(1, token.clamp(min=0)[:, None])[:, 0] / z[:, 0]
    empty = token < 0
    return token.to(torch.int32), torch.where(empty, 0.0, prob).float()


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        return _own(s, c, op)
    if op == "norm":
        total, inv, y = _plain_norm(s)
        return {"y": y.to(total.dtype), "total": total, "inv_rms": inv}
    if op == "norm_mx":
        total, inv, y = _plain_norm(s)
        q, scales = _plain_mx(y, c["format"])
        return {"q": q, "scales": scales, "total": total, "inv_rms": inv}
    if op == "norm_back":
        dx, dgain = _plain_norm_back(s)
        return {"dx": dx, "dgain": dgain}
    if op == "w4":
        return {"c": _plain_w4(s)}
    token, prob = _plain_sample(s)
    return {"token": token, "prob": prob}


def _own(s, c, op):
    from complexity_matmul_tcgen05_gb300 import fgemm
    if op == "norm":
        y, total, inv = fgemm.rms_norm(s["x"], s["gain"], residual=s["residual"], eps=EPS)
        return {"y": y, "total": total, "inv_rms": inv}
    if op == "norm_mx":
        q, scales, total, inv = fgemm.rms_norm_mx(s["x"], s["gain"], residual=s["residual"], eps=EPS, fmt=c["format"])
        # 8-bit codes and scales as the values they stand for
        return {"q": q.view(F8[c["format"]]), "scales": scales.view(torch.float8_e8m0fnu), "total": total, "inv_rms": inv}
    if op == "norm_back":
        dx, dgain = fgemm.rms_norm_backward(s["dy"], s["total"], s["gain"], s["inv_rms"], dtotal=s["dtotal"])
        return {"dx": dx, "dgain": dgain}
    if op == "w4":
        return {"c": fgemm.matmul_w4(s["a"], s["w"], s["scales"], zeros=s["zeros"], group=c["group"], bias=s["bias"],
                                     alpha=s["alpha"], epilogue=c["epilogue"])}
    token, prob = fgemm.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])
    return {"token": token, "prob": prob}


# --------------------------------------------------------------------- work


def work(case):
    op, rows = case["op"], case["rows"]
    if op == "w4":
        n, k = case["n"], case["k"]
        groups = -(-k // case["group"])
        n_out = n // 2 if case["epilogue"] == "swiglu" else n
        b = n * ((k + 1) // 2) + n * groups * (3 if case["zeros"] else 2) + rows * (k + n_out) * 2
        return {"bytes": b + (2 * n if case["epilogue"] in ("scale_bias", "silu") else 0), "flops": 2 * rows * n * k}
    if op == "sample":
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": rows * (case["vocab"] * size + 28), "flops": 2 * rows * case["vocab"]}
    width = case["width"]
    each = rows * width
    if op == "norm_back":  # dy, total and the stream's gradient in, dx out; gains and their gradient
        return {"bytes": each * 2 * (3 + case["residual"]) + rows * 4 + width * 6, "flops": 10 * each}
    # x in, y out; with a residual that in and the sum out; gains in, 1/rms out
    out = each + rows * -(-width // 32) if op == "norm_mx" else 2 * each
    return {"bytes": each * 2 * (3 if case["residual"] else 1) + out + rows * 4 + width * 2, "flops": 5 * each}


# -------------------------------------------------------------------- exact


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def exact(case, seed):
    op = case["op"]
    if op == "w4" and 2.0 * case["rows"] * case["n"] * case["k"] > 5e11:
        return None
    s = prepare(case, seed)
    if op.startswith("norm"):
        gain = _np(s["gain"])
        if op == "norm_back":
            dy, h, inv = _np(s["dy"]), _np(s["total"]), _np(s["inv_rms"])[:, None]
            unit = h * inv
            g = dy * gain
            dx = inv * (g - unit * np.mean(g * unit, axis=1, keepdims=True))
            if s["dtotal"] is not None:
                dx += _np(s["dtotal"])
            return {"dx": dx, "dgain": np.einsum("ij,ij->j", dy, unit)}
        total = s["x"] if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
        h = _np(total)
        inv = 1.0 / np.sqrt(np.mean(h * h, axis=1) + EPS)
        y = h * inv[:, None] * gain
        if op == "norm":
            return {"y": y, "total": h, "inv_rms": inv}
        rows, width = y.shape
        emax, bits, low, top = (8, 3, -6, 448.0) if case["format"] == "e4m3" else (15, 2, -14, 57344.0)
        q, scales = np.empty_like(y), np.empty((rows, -(-width // 32)))
        for b in range(scales.shape[1]):
            v = y[:, 32 * b:32 * b + 32]
            most = np.max(np.abs(v), axis=1)
            e = np.where(most > 0, np.frexp(most)[1] - 1 - emax, -127).clip(-127, 127)
            scales[:, b] = np.ldexp(1.0, e)
            v = np.ldexp(v, -e[:, None])
            step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - 1, low) - bits)  # spacing of 8-bit values around v
            q[:, 32 * b:32 * b + 32] = np.clip(np.rint(v / step) * step, -top, top)
        return {"q": q, "scales": scales, "total": h, "inv_rms": inv}
    if op == "w4":
        # 64-bit products on the device: on the host they would take minutes
        n, k, group = case["n"], case["k"], case["group"]
        a = s["a"].double()
        v = torch.zeros((case["rows"], n), dtype=torch.float64, device=a.device)
        for k0 in range(0, k, group):
            k1 = min(k, k0 + group)
            codes = torch.empty((n, k1 - k0), dtype=torch.float64, device=a.device)
            part = s["w"][:, k0 // 2:(k1 + 1) // 2]
            codes[:, 0::2] = (part % 16).double()
            codes[:, 1::2] = (part // 16).double()[:, :(k1 - k0) // 2]
            codes -= 8.0 if s["zeros"] is None else s["zeros"][:, k0 // group, None].double()
            v += (a[:, k0:k1] @ codes.t()) * s["scales"][:, k0 // group].double()
        v = s["alpha"] * v.cpu().numpy()
        if s["bias"] is not None:
            v = v + _np(s["bias"])
        if case["epilogue"] == "silu":
            v = v / (1 + np.exp(-v))
        elif case["epilogue"] == "swiglu":
            gate, up = np.split(v, 2, axis=1)
            v = gate * up / (1 + np.exp(-gate))
        return {"c": v}
    x = _np(s["logits"])
    t, top_k, top_p, min_p, u = (_np(s[name]) for name in ("temperature", "top_k", "top_p", "min_p", "u"))
    probs = np.zeros(x.shape[0])
    for i in range(x.shape[0]):
        ids = np.argsort(-x[i], kind="stable")
        ids = ids[x[i][ids] > -math.inf]
        if not ids.size:
            continue
        if top_k[i] > 0:
            ids = ids[:int(top_k[i])]
        w = np.exp((x[i][ids] - x[i][ids[0]]) / t[i])
        n = len(ids)
        if top_p[i] < 1:
            n = min(n, 1 + int(np.searchsorted(np.cumsum(w), top_p[i] * w.sum(), side="left")))
        n = max(1, min(n, int(np.count_nonzero(w >= min_p[i]))))
        chosen = np.argsort(ids[:n])
        w = w[:n][chosen]
        at = min(int(np.searchsorted(np.cumsum(w), u[i] * w.sum(), side="right")), n - 1)
        probs[i] = w[at] / w.sum()
    return {"token": None, "prob": probs}
