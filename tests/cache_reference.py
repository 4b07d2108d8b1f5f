"""The operators around a key-value cache in 64 bits (torch on the CPU), and
bounds on what the kernels may differ from them.

Bounds count roundings: storing to a 16-bit type is off by half a step
(``torch.finfo(t).eps / 2`` of the value, plus half the subnormal step), one
fp32 operation by 2^-24, and one addition inside a matrix instruction, which
may truncate, by 2^-23 of the terms' magnitudes.
"""
import math

import torch

U32 = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double()


def store(v, dtype):
    """Bound of one rounding of v to dtype."""
    info = torch.finfo(dtype)
    return v.abs() * info.eps / 2 + info.tiny * info.eps / 2


# ------------------------------------------------------------------ attention


def attend(q, k, v, seen, scale, dtype):
    """(out, lse, bound of out, bound of lse) of queries q (n x heads x dim) over
    keys and values (m x key heads x dim); seen: n x m truth values.

    Bounds.  A score sums dim products in an order of the kernel's; scaling by
    scale * log2 e, the maximum's subtraction and the exponential add a few
    roundings of the largest score: relative error `d` of a weight.  Weights are
    rounded to dtype (half a step of themselves; in fp16 at least 2^-25 of the
    largest one's scale), sums of weights and of weights times values go through
    at most m / 16 + 16 truncating additions.  Everything moves an output by its
    relative size times sum p |v|, twice where numerator and sum both carry it."""
    n, heads, dim = q.shape
    m, kv_heads, _ = k.shape
    group = heads // kv_heads
    out = torch.zeros(n, heads, dim, dtype=torch.float64)
    lse = torch.full((n, heads), -math.inf, dtype=torch.float64)
    b_out, b_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for h in range(heads):
        kk, vv = k[:, h // group], v[:, h // group]
        x = (q[:, h] @ kk.t()) * scale
        x = torch.where(seen, x, -math.inf)
        any_seen = (x > -math.inf).any(1)
        z = torch.logsumexp(x, 1)
        p = torch.where(seen, torch.exp(x - torch.where(any_seen, z, 0.0)[:, None]), 0.0)
        # (a value that no query sees may be anything)
        finite = torch.where(seen.any(0)[:, None], vv, 0.0)
        o = p @ finite
        out[:, h], lse[:, h] = o, z
        if m == 0:
            continue
        most = torch.where(seen, x.abs(), 0.0).amax(1)
        terms = torch.where(seen, (q[:, h].abs() @ torch.where(seen.any(0)[:, None], kk, 0.0).abs().t()) * scale, 0.0).amax(1)
        d = 2 * (dim / 8 + 4) * U32 * terms + 12 * U32 * most + 8 * U32
        sums = 2 * (m / 16 + 16) * U32
        mass = p @ finite.abs()
        half = torch.finfo(dtype).eps / 2
        b = mass * (half + sums + 2 * d[:, None] + sums)
        if dtype == torch.float16:
            b = b + 2.0 ** -25 * (seen.double() @ finite.abs())
        b_out[:, h] = b + store(o, dtype)
        b_lse[:, h] = torch.where(any_seen, 2 * d + sums + 4 * U32 * (z.abs() + most), 0.0)
    return out, lse, b_out, b_lse


def seen_by(n, m, causal, window):
    """n x m truth values: which keys the last n of m positions see."""
    at = torch.arange(n)[:, None] + (m - n)
    key = torch.arange(m)[None]
    seen = torch.ones(n, m, dtype=torch.bool)
    if causal:
        seen &= key <= at
    if window:
        seen &= key > at - window
    return seen


# --------------------------------------------------------------------- rotary


def rotate(x, positions, inv_freq, interleaved):
    """(values, bound before the rounding of the store) of heads x (T x heads x dim)."""
    half = inv_freq.shape[0]
    angle = positions.double()[:, None, None] * inv_freq.double()
    y, b = x.clone(), torch.zeros_like(x)
    a_at, b_at = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else
                  (slice(0, half), slice(half, 2 * half)))
    u, v = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin()
    # the reduced angle is at most pi and off by 2^-24 of itself, cosine and
    # sine by two roundings more, the products and their sum by three
    b[..., a_at] = b[..., b_at] = (u.abs() + v.abs()) * ((math.pi + 2) + 3) * U32
    return y, b


# ------------------------------------------------------------------- logprobs


def logprobs(x, tokens, top):
    """(logprob, entropy, top tokens, top logprobs, bounds of the first, second
    and fourth) of rows x (64 bits, NaN counting as -inf).

    A weight e^(x - m) carries 2^-24 |x - m| log2 e of its argument and 4
    roundings; weights below e^-40 do not count beside the first.  The sum is one
    of at most vocab / 128 + 40 additions a thread and its neighbours.  log z is
    then off by the sum's error over z."""
    rows, vocab = x.shape
    x = torch.where(torch.isnan(x), -math.inf, x)
    given = torch.full((rows,), -math.inf, dtype=torch.float64)
    entropy = torch.zeros(rows, dtype=torch.float64)
    tops = torch.full((rows, top), -1, dtype=torch.int64)
    top_lp = torch.full((rows, top), -math.inf, dtype=torch.float64)
    b_given, b_entropy, b_top = torch.zeros(rows), torch.zeros(rows), torch.zeros(rows, top)
    rel = (vocab / 128 + 40 + 4 + 2 * 40 * 1.5) * U32
    for i in range(rows):
        m = x[i].max() if vocab else torch.tensor(-math.inf)
        if m == -math.inf:
            continue
        below = torch.where(x[i] == m, 0.0, x[i] - m)  # 0 for the largest, infinite ones too
        w = torch.exp(below)
        rest = w.sum() - 1 if (w == 1).sum() > 1 else torch.where(x[i] == m, 0.0, w).sum()
        log_z = torch.log1p(rest)
        z = 1 + rest
        t = torch.where(w > 0, w * torch.where(w > 0, below, 0.0), 0.0).sum() / z
        lp = below - log_z
        entropy[i] = log_z - t
        off = rel * rest / z + 4 * U32 * log_z
        b_entropy[i] = off + (2 * rel + 4 * U32) * t.abs()
        if 0 <= tokens[i] < vocab:
            given[i] = lp[tokens[i]]
            b_given[i] = off + (4 * U32 * below[tokens[i]].abs() if given[i] > -math.inf else 0)
        order = torch.sort(x[i], descending=True, stable=True)[1][:top]
        order = order[x[i][order] > -math.inf]
        tops[i, :len(order)] = order
        top_lp[i, :len(order)] = lp[order]
        b_top[i, :len(order)] = off + 4 * U32 * below[order].abs()
    return given, entropy, tops, top_lp, b_given, b_entropy, b_top
