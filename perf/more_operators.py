"""The operators of a token step with a cache, as measured: rotary positions
with the write into a paged key-value cache, attention of one new token over
that cache, attention over packed prompts, and log probabilities of given
tokens with entropy and top alternatives.

``run`` computes them in their plain form (elementary torch operations in 32
or 64 bits, rounded once at the end) where ``own`` is false, and through the
framework's entry points (``fgemm.rotary_cache``, ``attention_paged``,
``attention``, ``logprobs``) where it is true.  ``exact`` restates each
operator in 64 bits.

Sizes: 32 heads of 128 are the width 4096 of the benchmark's projections; the
rest (groups, pages, contexts, vocabularies) is generic.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step: nothing but latency
        {"name": "rotary, one token", "op": "rotary", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "page": 16, "type": "bf16"},
        # a prompt's tokens on their way into the cache, three quarters of each head rotated
        {"name": "rotary, prompt", "op": "rotary", "tokens": 8191, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 96,
         "interleaved": True, "page": 64, "type": "f16"},
        # one sequence of a chat
        {"name": "decode, one sequence", "op": "paged", "seqs": 1, "longest": 4097, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "type": "bf16"},
        # a serving batch of very different lengths
        {"name": "decode, ragged batch", "op": "paged", "seqs": 64, "longest": 16384, "ragged": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "type": "bf16"},
        # a few documents, small heads in groups of an odd size
        {"name": "decode, long context", "op": "paged", "seqs": 3, "longest": 131071, "ragged": False, "heads": 28,
         "kv_heads": 4, "dim": 64, "page": 64, "window": 0, "type": "f16"},
        # a short question
        {"name": "prompt, 37 tokens", "op": "prompt", "seqs": 1, "tokens": 37, "prefix": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "causal": True, "window": 0, "type": "bf16"},
        # packed prompts of different lengths
        {"name": "prompts, packed", "op": "prompt", "seqs": 13, "tokens": 12345, "prefix": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "causal": True, "window": 0, "type": "bf16"},
        # a long document
        {"name": "prompt, long", "op": "prompt", "seqs": 1, "tokens": 16384, "prefix": 0, "heads": 32, "kv_heads": 8,
         "dim": 128, "causal": True, "window": 0, "type": "bf16"},
        # next parts of prompts whose beginnings are known, narrow heads, a sliding window
        {"name": "prompts, window behind a prefix", "op": "prompt", "seqs": 5, "tokens": 7001, "prefix": 2000,
         "heads": 24, "kv_heads": 24, "dim": 80, "causal": True, "window": 1024, "type": "f16"},
        # one answer's next token with its alternatives
        {"name": "logprobs, one row", "op": "logprobs", "rows": 1, "vocab": 32000, "top": 5, "type": "bf16", "masked": 0.0},
        # a serving batch with a large vocabulary
        {"name": "logprobs, batch", "op": "logprobs", "rows": 64, "vocab": 131072, "top": 20, "type": "f32", "masked": 0.0},
        # scoring a prompt's tokens, an odd vocabulary with masked entries
        {"name": "logprobs, prompt", "op": "logprobs", "rows": 4096, "vocab": 50257, "top": 0, "type": "f16", "masked": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "paged", "paged", "prompt", "prompt", "logprobs"])
    kind = rng.choice(["bf16", "f16"])
    if op == "logprobs":
        vocab = _log(rng, 1000, 200000)
        return {"op": op, "rows": _log(rng, 1, max(2, min(4096, 4096 * 50257 // vocab))), "vocab": vocab,
                "top": rng.choice([0, 1, 5, 20, 32]), "type": rng.choice(["bf16", "f16", "f32"]),
                "masked": rng.choice([0.0, 0.0, 0.3])}
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 16) if g * kv_heads <= 64])
    c = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": rng.choice([64, 128, 128, 32, 72, 80, 96]), "type": kind}
    if op == "rotary":
        c["rot"] = c["dim"] if rng.random() < 0.7 else max(2, int(c["dim"] * rng.random()) // 2 * 2)
        return {**c, "tokens": _log(rng, 1, min(8192, 8192 * 40 * 128 // ((heads + kv_heads) * c["dim"]))),
                "interleaved": rng.random() < 0.4, "page": rng.choice([8, 16, 24, 64])}
    if op == "paged":
        longest = _log(rng, 1, 131072)
        most = max(1, 32 * 16384 * 8 * 128 // (longest * kv_heads * c["dim"]))
        return {**c, "seqs": _log(rng, 1, min(512, most)), "longest": longest, "ragged": rng.random() < 0.6,
                "page": rng.choice([8, 16, 24, 64, 256]), "window": rng.choice([0, 0, 0, 512, 4000])}
    tokens = _log(rng, 1, 16384)
    prefix = rng.choice([0, 0, 0, 1, 100, 2000])
    causal = rng.random() < 0.8
    seqs = _log(rng, 1, max(1, min(100, tokens // 8, 8192 // max(1, prefix))))
    # a product of all queries and keys of a sequence costs at most the long prompt's
    tokens = min(tokens, int(16384 * math.sqrt(min(1.0, 32 * 128 / (heads * c["dim"])) / (1 if causal else 2))) - prefix)
    return {**c, "seqs": min(seqs, tokens), "tokens": tokens, "prefix": prefix, "causal": causal,
            "window": rng.choice([0, 0, 100, 2048]) if causal else 0}


def _lengths(case):
    """Lengths of a case's sequences: its sizes alone say them."""
    rng = random.Random(7919 * case["seqs"] + case.get("longest", 0) + case.get("tokens", 0))
    if case["op"] == "paged":
        if not case["ragged"]:
            return [case["longest"]] * case["seqs"]
        return [max(1, int(case["longest"] * rng.random() ** 2)) for _ in range(case["seqs"])]
    left, n = case["tokens"], case["seqs"]
    if n == 1:
        return [left]
    share = [0.1 + rng.random() ** 2 for _ in range(n)]
    lengths = [max(1, int(s / sum(share) * (left - n))) for s in share[:-1]]
    return lengths + [left - sum(lengths)]


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, type=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=type)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    op, t = case["op"], TYPES[case["type"]]
    s = {"case": case}
    if op == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        x = 2.5 * normal(rows, vocab)
        # a few likely continuations in each row, one of them the given token as a rule
        likely = torch.randint(0, vocab, (rows, 16), generator=g, device=DEV)
        x.scatter_add_(1, likely, 4 + 3.0 * normal(rows, 16))
        if case["masked"]:
            x.masked_fill_(torch.rand((rows, vocab), generator=g, device=DEV) < case["masked"], -math.inf)
        s["logits"] = x.to(t)
        s["tokens"] = likely[:, 0].to(torch.int32)
        return s
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if op == "rotary":
        n, page = case["tokens"], case["page"]
        # queries, keys and values side by side, as one projection leaves them
        wide = normal(n, (heads + 2 * kv_heads) * dim).to(t)
        s["q"], s["k"], s["v"] = (part.unflatten(1, (-1, dim)) for part in
                                  wide.split((heads * dim, kv_heads * dim, kv_heads * dim), 1))
        pages = 2 * (-(-n // page)) + 1
        s["k_cache"] = torch.zeros((pages, page, kv_heads, dim), dtype=t, device=DEV)
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        # tokens of sequences anywhere in their contexts, each at a place of its own
        s["positions"] = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV, dtype=torch.int32)
        s["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:n].to(torch.int32)
        half = torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64)
        s["inv_freq"] = (500000.0 ** (-2 * half / case["rot"])).float()
        return s
    lengths = _lengths(case)
    # keys have channels of their own; some queries look for one key above all
    channel = normal(kv_heads, dim)
    if op == "paged":
        n, page = case["seqs"], case["page"]
        need = [-(-length // page) for length in lengths]
        total = sum(need) + 3
        s["q"] = (1.5 * normal(n, heads, dim)).to(t)
        s["k_cache"] = normal(total, page, kv_heads, dim, type=t)
        s["k_cache"] += channel.to(t)
        s["v_cache"] = normal(total, page, kv_heads, dim, type=t)
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros((n, max(need)), dtype=torch.int32, device=DEV)
        at = 0
        for i, count in enumerate(need):
            table[i, :count] = order[at:at + count]
            at += count
        s["page_table"], s["lengths"], s["host_lengths"] = table, ints(lengths), lengths
        return s
    k_lengths = [length + case["prefix"] for length in lengths]
    starts, k_starts = [0], [0]
    for a, b in zip(lengths, k_lengths):
        starts.append(starts[-1] + a)
        k_starts.append(k_starts[-1] + b)
    s["q"] = (1.5 * normal(starts[-1], heads, dim)).to(t)
    s["k"] = (normal(k_starts[-1], kv_heads, dim) + channel).to(t)
    s["v"] = normal(k_starts[-1], kv_heads, dim).to(t)
    s["starts"], s["host_starts"] = ints(starts), starts
    s["k_starts"], s["host_k_starts"] = (ints(k_starts) if case["prefix"] else None), k_starts
    return s


# -------------------------------------------------------------- plain forms


def _plain_rotary(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x):
        y = x.float().clone()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., :half].clone(), y[..., half:rot].clone()
            y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    where = s["slots"].long()
    s["k_cache"].flatten(0, 1)[where] = turned(s["k"])
    s["v_cache"].flatten(0, 1)[where] = s["v"]
    return turned(s["q"])


def _weighted(scores, v):
    """softmax(scores) @ v and the log of the sums; scores are -inf where masked."""
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    w = torch.exp(scores - m)
    z = w.sum(-1, keepdim=True)
    out = (w @ v) / torch.where(z == 0, 1.0, z)
    return out, (m + torch.log(z))[..., 0]


def _plain_paged(s):
    c = s["case"]
    kv_heads, dim, group = c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    outs, lses = [], []
    for i, length in enumerate(s["host_lengths"]):
        pages = s["page_table"][i, :-(-length // c["page"])].long()
        first = max(0, length - c["window"]) if c["window"] else 0
        k, v = (x[pages].flatten(0, 1)[first:length].float().transpose(0, 1) for x in (s["k_cache"], s["v_cache"]))
        q = s["q"][i].float().view(kv_heads, group, dim)
        out, lse = _weighted((q @ k.transpose(1, 2)) / math.sqrt(dim), v)
        outs.append(out.reshape(1, -1, dim))
        lses.append(lse.reshape(1, -1))
    return torch.cat(outs).to(s["q"].dtype), torch.cat(lses)


def _plain_prompt(s):
    c = s["case"]
    kv_heads, group = c["kv_heads"], c["heads"] // c["kv_heads"]
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    for i in range(c["seqs"]):
        q0, q1 = s["host_starts"][i:i + 2]
        k0, k1 = s["host_k_starts"][i:i + 2]
        ahead = (k1 - k0) - (q1 - q0)
        for a in range(q0, q1, 2048):  # queries of a block, keys up to its last
            b = min(q1, a + 2048)
            most = ahead + b - q0 if c["causal"] else k1 - k0
            at = torch.arange(ahead + a - q0, ahead + b - q0, device=DEV)[:, None]
            key = torch.arange(most, device=DEV)[None]
            hidden = (key > at) if c["causal"] else torch.zeros_like(key > at)
            if c["window"]:
                hidden = hidden | (key <= at - c["window"])
            for h in range(kv_heads):
                q = s["q"][a:b, h * group:(h + 1) * group].float().transpose(0, 1)
                k, v = s["k"][k0:k0 + most, h].float(), s["v"][k0:k0 + most, h].float()
                scores = (q @ k.t()) / math.sqrt(c["dim"])
                o, z = _weighted(scores.masked_fill_(hidden, -math.inf), v)
                out[a:b, h * group:(h + 1) * group] = o.transpose(0, 1).to(out.dtype)
                lse[a:b, h * group:(h + 1) * group] = z.t()
    return out, lse


def _plain_logprobs(s):
    top = s["case"]["top"]
    x = s["logits"].double()
    m = x.amax(1, keepdim=True)
    w = torch.exp(x - m)
    z = w.sum(1, keepdim=True)
    logp = x - m - torch.log(z)
    given = logp.gather(1, s["tokens"].long()[:, None])[:, 0]
    entropy = -(w / z * torch.where(w == 0, 0.0, logp)).sum(1)
    order = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :top] if top else x[:, :0].long()
    return given.float(), entropy.float(), order.to(torch.int32), logp.gather(1, order).float()


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "rotary":
        return {"q": _plain_rotary(state), "k_cache": state["k_cache"], "v_cache": state["v_cache"]}
    if op == "logprobs":
        given, entropy, top, top_logprobs = _plain_logprobs(state)
        return {"logprob": given, "entropy": entropy, "top": top, "top_logprobs": top_logprobs}
    out, lse = _plain_paged(state) if op == "paged" else _plain_prompt(state)
    return {"out": out, "lse": lse}


def _own(s, op):
    from complexity_matmul_tcgen05_gb300 import fgemm
    c = s["case"]
    if op == "rotary":
        q = fgemm.rotary_cache(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"],
                               s["v_cache"], interleaved=c["interleaved"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "logprobs":
        given, entropy, top, top_logprobs = fgemm.logprobs(s["logits"], s["tokens"], top=c["top"])
        return {"logprob": given, "entropy": entropy, "top": top, "top_logprobs": top_logprobs}
    if op == "paged":
        out, lse = fgemm.attention_paged(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lengths"],
                                         window=c["window"])
    else:
        out, lse = fgemm.attention(s["q"], s["k"], s["v"], s["starts"], k_starts=s["k_starts"], causal=c["causal"],
                                   window=c["window"])
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------- work


def _seen(length, ahead, causal, window):
    """Pairs of a query and a key that it sees, of a sequence."""
    if not causal:
        return length * (length + ahead)
    pairs = length * ahead + length * (length + 1) // 2
    if window:  # queries at positions p >= window see `window` keys, the others p + 1
        first = max(ahead, window)
        count = max(0, ahead + length - first)
        pairs -= count * (first - window + 1) + count * (count - 1) // 2
    return pairs


def work(case):
    op = case["op"]
    if op == "logprobs":
        size = 4 if case["type"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 12 + 8 * case["top"]), "flops": 6 * case["rows"] * case["vocab"]}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    if op == "rotary":  # queries, keys and values in and out
        n = case["tokens"]
        return {"bytes": n * ((heads + 2 * kv_heads) * dim * 4 + 8) + case["rot"] * 2,
                "flops": 3 * n * (heads + kv_heads) * case["rot"]}
    lengths = _lengths(case)
    if op == "paged":
        seen = sum(min(length, case["window"]) if case["window"] else length for length in lengths)
        pages = sum(-(-length // case["page"]) for length in lengths)
        return {"bytes": seen * kv_heads * dim * 4 + case["seqs"] * heads * (dim * 4 + 4) + 4 * pages + 4 * case["seqs"],
                "flops": 4 * seen * heads * dim}
    pairs = sum(_seen(length, case["prefix"], case["causal"], case["window"]) for length in lengths)
    n, n_k = sum(lengths), sum(lengths) + case["prefix"] * len(lengths)
    return {"bytes": n * heads * (dim * 4 + 4) + n_k * kv_heads * dim * 4, "flops": 4 * pairs * heads * dim}


# -------------------------------------------------------------------- exact


def exact(case, seed):
    """In 64 bits, on the device: on the host the larger cases would take minutes."""
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "logprobs":
        given, entropy, values = [], [], []
        for a in range(0, case["rows"], 256):
            x = s["logits"][a:a + 256].double()
            lse = torch.logsumexp(x, 1, keepdim=True)
            x -= lse
            given.append(x.gather(1, s["tokens"][a:a + 256, None].long())[:, 0])
            entropy.append(torch.special.entr(x.exp()).sum(1))
            values.append(x.topk(case["top"], dim=1).values)
        return {"logprob": torch.cat(given).cpu().numpy(), "entropy": torch.cat(entropy).cpu().numpy(), "top": None,
                "top_logprobs": torch.cat(values).cpu().numpy()}
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    group = heads // kv_heads
    if op == "rotary":
        rot = case["rot"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None, None] * s["inv_freq"].double())

        def turned(x):
            y = x.double()
            pairs = y[..., :rot].unflatten(-1, (-1, 2) if case["interleaved"] else (2, -1))
            axis = -1 if case["interleaved"] else -2
            z = torch.complex(pairs.select(axis, 0).contiguous(), pairs.select(axis, 1).contiguous()) * turn
            y[..., :rot] = torch.stack((z.real, z.imag), axis).flatten(-2)
            return y

        at = s["slots"].long()
        k, v = (torch.zeros(x.shape, dtype=torch.float64, device=DEV) for x in (s["k_cache"], s["v_cache"]))
        k.view(-1, kv_heads, dim)[at], v.view(-1, kv_heads, dim)[at] = turned(s["k"]), s["v"].double()
        return {"q": turned(s["q"]).cpu().numpy(), "k_cache": k.cpu().numpy(), "v_cache": v.cpu().numpy()}
    n = s["q"].shape[0]
    out = torch.zeros((n, heads, dim), dtype=torch.float64, device=DEV)
    lse = torch.zeros((n, heads), dtype=torch.float64, device=DEV)

    def fill(a, b, k, v, first, last):
        """Queries a .. b over keys k (n_k x kv_heads x dim); query i sees keys first[i] .. last[i] - 1."""
        key = torch.arange(k.shape[0], device=DEV)
        seen = (key >= first[:, None]) & (key < last[:, None])
        for h in range(heads):
            x = s["q"][a:b, h].double() @ k[:, h // group].double().t() * dim ** -0.5
            x = torch.where(seen, x, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[a:b, h] = z
            out[a:b, h] = torch.where(seen, torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None]), 0.0) @ v[:, h // group].double()

    if op == "paged":
        for i, length in enumerate(s["host_lengths"]):
            token = torch.arange(length, device=DEV)
            page = s["page_table"][i].long()[token // case["page"]]
            k, v = (x[page, token % case["page"]] for x in (s["k_cache"], s["v_cache"]))
            last = torch.tensor([length], device=DEV)
            fill(i, i + 1, k, v, last - (case["window"] or length), last)
    else:
        for i in range(case["seqs"]):
            (q0, q1), (k0, k1) = s["host_starts"][i:i + 2], s["host_k_starts"][i:i + 2]
            for a in range(q0, q1, 1024):
                b = min(q1, a + 1024)
                last = torch.arange(a, b, device=DEV) + 1 + (k1 - q1) - k0
                first = last - (case["window"] or k1)
                if not case["causal"]:
                    first, last = torch.zeros_like(last), torch.full_like(last, k1 - k0)
                most = int(last[-1])
                fill(a, b, s["k"][k0:k0 + most], s["v"][k0:k0 + most], first, last)
    return {"out": out.cpu().numpy(), "lse": lse.cpu().numpy()}
