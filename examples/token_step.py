"""A token step from the operators around a product, on one GPU.

Residual blocks of RMS norm, a gated projection and one back, all with 4-bit
weights; a last norm, the projection to the vocabulary and sampling:

    python examples/token_step.py [--width 4096 --depth 4 --rows 4 --steps 32]

Steps run eagerly or as one replayed CUDA graph, with the same tokens.  The
first block's gain is then fitted for a few steps with the norm's backward
pass, and the same norm gives 8-bit blocks to the block-scaled product.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from complexity_matmul_tcgen05_gb300 import fgemm  # noqa: E402


def quantise_w4(W, group=128):
    """(codes, scales) of an N x K matrix (K even) as matmul_w4 takes them,
    zero point 8: the scale takes the group's largest value to 7."""
    n, k = W.shape
    groups = -(-k // group)
    V = torch.zeros(n, groups * group, dtype=torch.float32, device=W.device)
    V[:, :k] = W.float()
    V = V.view(n, groups, group)
    scales = (V.abs().amax(2) / 7).clamp_min(1e-6).to(W.dtype)
    q = (V / scales.float()[:, :, None]).round().clamp(-8, 7).view(n, -1)[:, :k].to(torch.int16) + 8
    return (q[:, 0::2] + 16 * q[:, 1::2]).to(torch.uint8), scales


class Model:
    """Random weights of the given sizes; `embedding` is vocab x width."""

    def __init__(self, width=1024, hidden=2816, depth=2, vocab=32000, group=128, dtype=torch.bfloat16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def matrix(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).to(dtype)

        self.group = group
        self.embedding = torch.randn(vocab, width, generator=g, device="cuda").to(dtype)
        self.gains = [torch.ones(width, dtype=dtype, device="cuda") for _ in range(depth + 1)]
        self.up = [quantise_w4(matrix(2 * hidden, width), group) for _ in range(depth)]  # gate, then up
        self.down = [quantise_w4(matrix(width, hidden), group) for _ in range(depth)]
        self.head = quantise_w4(matrix(vocab, width), group)

    def logits(self, x):
        """Logits of the rows x; a block's output meets the residual stream in
        the next norm, which adds the two."""
        part, stream = x, None
        for gain, up, down in zip(self.gains, self.up, self.down):
            y, stream, _ = fgemm.rms_norm(part, gain, residual=stream)
            h = fgemm.matmul_w4(y, *up, group=self.group, epilogue="swiglu")
            part = fgemm.matmul_w4(h, *down, group=self.group)
        y, _, _ = fgemm.rms_norm(part, self.gains[-1], residual=stream)
        return fgemm.matmul_w4(y, *self.head, group=self.group)

    def step(self, token, u, **kept):
        """(next token, its probability, logits); token is int32, one a row."""
        logits = self.logits(self.embedding[token.long()])
        return (*fgemm.sample(logits, u, **kept), logits)


def generate(model, token, uniform, graph=True, **kept):
    """Tokens (steps + 1) x rows from the first ones and steps x rows uniform
    numbers.  With graph, one captured step is replayed."""
    out = [token.clone()]
    if not graph:
        for u in uniform:
            out.append(model.step(out[-1], u, **kept)[0])
        return torch.stack(out)
    state, u = token.clone(), uniform[0].clone()
    model.step(state, u, **kept)  # what a first call sets up is not captured
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        state.copy_(model.step(state, u, **kept)[0])
    for row in uniform:
        u.copy_(row)
        g.replay()
        out.append(state.clone())
    return torch.stack(out)


def fit_gain(x, target, gain, steps=10, rate=0.5):
    """Mean square errors of `steps` descents of a norm's gain towards a target."""
    losses = []
    gain32 = gain.float()
    for _ in range(steps):
        y, total, inv = fgemm.rms_norm(x, gain32.to(gain.dtype))
        error = y.float() - target.float()
        losses.append(error.square().mean())
        _, dgain = fgemm.rms_norm_backward((2 * error / len(x)).to(x.dtype), total, gain32.to(gain.dtype), inv)
        gain32 -= rate * dgain
    return torch.stack(losses).tolist()


def norm_into_mx(x, gain, B, scale_b):
    """rms_norm(x) @ B with both operands in block-scaled 8 bits."""
    q, scales, _, _ = fgemm.rms_norm_mx(x, gain)
    return fgemm.matmul_mx(q, scales, B, scale_b)


def main():
    ap = argparse.ArgumentParser()
    for name, value in (("width", 4096), ("hidden", 14336), ("depth", 4), ("vocab", 128000), ("rows", 4), ("steps", 32)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    model = Model(a.width, a.hidden, a.depth, a.vocab)
    token = torch.arange(a.rows, dtype=torch.int32, device="cuda")
    uniform = torch.rand(a.steps, a.rows, device="cuda")
    kept = dict(temperature=0.8, top_k=50, top_p=0.95)
    for graph in (False, True):
        generate(model, token, uniform, graph, **kept)
        torch.cuda.synchronize()
        t = time.perf_counter()
        tokens = generate(model, token, uniform, graph, **kept)
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t) * 1e3
        print(f"{'graph' if graph else 'eager'}: {a.steps} steps in {ms:.2f} ms, first row {tokens[:8, 0].tolist()}")
    x = model.embedding[:512]
    gain = model.gains[0]
    target = fgemm.rms_norm(x, gain * 1.5)[0]
    losses = fit_gain(x, target, gain)
    print(f"gain: mean square error {losses[0]:.4f} -> {losses[-1]:.6f}")
    n = a.width
    B = torch.full((n, 64), 0x38, dtype=torch.uint8, device="cuda")  # 1.0 in E4M3
    C = norm_into_mx(x, gain, B, torch.full((-(-n // 32), 64), 127, dtype=torch.uint8, device="cuda"))
    print(f"8-bit blocks into a product: {tuple(C.shape)} {C.dtype}")
    status = fgemm.default_handle().get_error()
    if status != fgemm.OK:
        raise SystemExit(fgemm.status_string(status))


if __name__ == "__main__":
    main()
