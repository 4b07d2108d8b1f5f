"""Prompts into a paged cache and tokens out of it, on one GPU.

A small transformer with random weights: its attention is fgemm.rotary_cache,
fgemm.attention over the packed prompts and fgemm.attention_paged for every new
token; norms, products, sampling and log probabilities stand around it.

    python examples/cached_decode.py [--width 4096 --depth 4 --steps 32]

The prompts of all sequences go through the model packed together; then every step
adds a token to each sequence, eagerly or as one replayed CUDA graph, with the same
tokens.  Last, the prompt and what was generated are scored in one pass.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from complexity_matmul_tcgen05_gb300 import fgemm  # noqa: E402


class Cache:
    """Pages of keys and values for every layer, and which of them a sequence has."""

    def __init__(self, depth, seqs, longest, kv_heads, dim, page=16, dtype=torch.bfloat16, seed=0):
        width = -(-longest // page)
        self.page = page
        shape = (seqs * width, page, kv_heads, dim)
        self.k = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(depth)]
        self.v = [torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(depth)]
        order = torch.randperm(seqs * width, generator=torch.Generator().manual_seed(seed))
        self.table = order.view(seqs, width).to("cuda", torch.int32)

    def slots(self, seq, position):
        """Slots of tokens (vectors of their sequences and positions)."""
        return (self.table[seq, position // self.page] * self.page + position % self.page).to(torch.int32)


class Model:
    def __init__(self, width=512, heads=8, kv_heads=2, hidden=1024, depth=2, vocab=8000, dtype=torch.bfloat16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def matrix(k, n):
            return (torch.randn(k, n, generator=g, device="cuda") * k ** -0.5).to(dtype)

        self.heads, self.kv_heads, self.dim = heads, kv_heads, width // heads
        self.embedding = torch.randn(vocab, width, generator=g, device="cuda").to(dtype)
        self.gain = torch.ones(width, dtype=dtype, device="cuda")
        self.qkv = [matrix(width, (heads + 2 * kv_heads) * self.dim) for _ in range(depth)]
        self.out = [matrix(width, width) for _ in range(depth)]
        self.up = [matrix(width, 2 * hidden) for _ in range(depth)]
        self.down = [matrix(hidden, width) for _ in range(depth)]
        self.head = matrix(width, vocab)
        half = torch.arange(self.dim // 2, dtype=torch.float64, device="cuda")
        self.inv_freq = (10000.0 ** (-2 * half / self.dim)).float()

    def forward(self, tokens, positions, slots, cache, attend):
        """Logits of tokens; attend(layer, q, k, v) is a layer's attention, with
        queries turned to their positions and keys and values in the cache."""
        part, stream = self.embedding[tokens.long()], None
        parts = (self.heads * self.dim, self.kv_heads * self.dim, self.kv_heads * self.dim)
        for layer in range(len(self.qkv)):
            y, stream, _ = fgemm.rms_norm(part, self.gain, residual=stream)
            q, k, v = (x.unflatten(1, (-1, self.dim)) for x in fgemm.matmul(y, self.qkv[layer]).split(parts, 1))
            q = fgemm.rotary_cache(q, k, v, positions, slots, self.inv_freq, cache.k[layer], cache.v[layer])
            part = fgemm.matmul(attend(layer, q, v).flatten(1), self.out[layer])
            y, stream, _ = fgemm.rms_norm(part, self.gain, residual=stream)
            part = fgemm.matmul(fgemm.matmul(y, self.up[layer], epilogue="swiglu"), self.down[layer])
        y, _, _ = fgemm.rms_norm(part, self.gain, residual=stream)
        return fgemm.matmul(y, self.head)

    def prompts(self, tokens, starts, cache):
        """Logits of packed prompts, starts the borders of the sequences (a list)."""
        lengths = torch.tensor(starts).diff()
        seq = torch.repeat_interleave(torch.arange(len(lengths)), lengths).cuda()
        at = torch.cat([torch.arange(n) for n in lengths.tolist()]).cuda()
        slots, border = cache.slots(seq, at), torch.tensor(starts, dtype=torch.int32, device="cuda")

        def attend(layer, q, v):  # the turned keys are in the cache
            k = cache.k[layer].flatten(0, 1)[slots.long()]
            return fgemm.attention(q, k, v, border)[0]

        return self.forward(tokens, at.to(torch.int32), slots, cache, attend)

    def step(self, tokens, lengths, cache):
        """Logits of one new token of each sequence; lengths (int32) with it."""
        at = lengths - 1
        slots = cache.slots(torch.arange(len(tokens), device="cuda"), at)

        def attend(layer, q, v):
            return fgemm.attention_paged(q, cache.k[layer], cache.v[layer], cache.table, lengths)[0]

        return self.forward(tokens, at, slots, cache, attend)


def generate(model, cache, prompts, uniform, graph=True, **kept):
    """(tokens, their log probabilities), steps x sequences, behind the prompts (a
    list of vectors); uniform: steps x sequences random numbers."""
    starts = [0]
    for x in prompts:
        starts.append(starts[-1] + len(x))
    logits = model.prompts(torch.cat(prompts), starts, cache)[torch.tensor(starts[1:], device="cuda") - 1]
    lengths = torch.tensor(starts, device="cuda").diff().to(torch.int32)
    token, _ = fgemm.sample(logits, uniform[0], **kept)
    logprob = fgemm.logprobs(logits, token)[0]
    out, scores = [token.clone()], [logprob.clone()]
    u = uniform[0].clone()

    def step():
        lengths.add_(1)
        logits = model.step(token, lengths, cache)
        token.copy_(fgemm.sample(logits, u, **kept)[0])
        logprob.copy_(fgemm.logprobs(logits, token, top=5)[0])

    if graph:
        before = lengths.clone(), token.clone()
        step()  # what a first call sets up is not captured
        lengths.copy_(before[0])
        token.copy_(before[1])
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
    for row in uniform[1:]:
        u.copy_(row)
        captured.replay() if graph else step()
        out.append(token.clone())
        scores.append(logprob.clone())
    return torch.stack(out), torch.stack(scores)


def score(model, cache, sequences):
    """Log probabilities of sequences' tokens (a list of vectors) behind each one's first."""
    starts = [0]
    for x in sequences:
        starts.append(starts[-1] + len(x))
    logits = model.prompts(torch.cat(sequences), starts, cache)
    follows = torch.cat([torch.cat((x[1:], x.new_full((1,), -1))) for x in sequences])
    scores = fgemm.logprobs(logits, follows)[0]
    return [scores[a:b - 1] for a, b in zip(starts, starts[1:])]


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("width", 4096), ("heads", 32), ("kv_heads", 8), ("hidden", 14336), ("depth", 4),
                        ("vocab", 128000), ("steps", 32)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    model = Model(a.width, a.heads, a.kv_heads, a.hidden, a.depth, a.vocab)
    g = torch.Generator("cuda").manual_seed(1)
    prompts = [torch.randint(0, a.vocab, (n,), generator=g, device="cuda", dtype=torch.int32) for n in (700, 37, 2000, 1)]
    uniform = torch.rand(a.steps, len(prompts), generator=g, device="cuda")
    longest = max(len(x) for x in prompts) + a.steps
    for graph in (False, True):
        cache = Cache(a.depth, len(prompts), longest, a.kv_heads, a.width // a.heads)
        generate(model, cache, prompts, uniform, graph, temperature=0.8, top_p=0.95)
        torch.cuda.synchronize()
        t = time.perf_counter()
        tokens, scores = generate(model, cache, prompts, uniform, graph, temperature=0.8, top_p=0.95)
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t) * 1e3
        print(f"{'graph' if graph else 'eager'}: prompts and {a.steps} steps in {ms:.2f} ms, {tokens[:6, 0].tolist()}")
    whole = [torch.cat((x, tokens[:, i])) for i, x in enumerate(prompts)]
    again = score(model, Cache(a.depth, len(prompts), longest, a.kv_heads, a.width // a.heads), whole)
    print("mean log probability of what was generated: "
          f"{float(scores.mean()):.4f}, scored in one pass {float(torch.stack([x[-a.steps:] for x in again]).mean()):.4f}")
    status = fgemm.default_handle().get_error()
    if status != fgemm.OK:
        raise SystemExit(fgemm.status_string(status))


if __name__ == "__main__":
    main()
