"""The operators of a token step in 64 bits (numpy), and bounds on what the
kernels may differ from them.

Bounds count roundings: storing to a 16-bit type is off by half a step
(``torch.finfo(t).eps / 2`` of the value, plus half the subnormal step), one
fp32 operation by 2^-24, and an fp32 sum of a chain of c additions by
c * 2^-24 of the sum of the terms' magnitudes.
"""
import math

import numpy as np
import torch

U32 = 2.0 ** -24
F8 = {"e4m3": (8, 3, -6, 448.0), "e5m2": (15, 2, -14, 57344.0)}  # emax, mantissa bits, least exponent, largest


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def store(v, dtype):
    """Bound of one rounding of v to dtype."""
    info = torch.finfo(dtype)
    return np.abs(v) * info.eps / 2 + info.tiny * info.eps / 2


def norm_chain(n):
    """Additions a row's sum goes through: at most 64 columns a thread (more
    only for rows above 65536), then ten doublings."""
    return max(64, n / 1024 + 8) + 10


def norm(t, gain, eps):
    """(inv, y) of rows t."""
    inv = 1.0 / np.sqrt(np.mean(t * t, axis=1) + eps)
    return inv, t * inv[:, None] * gain


def norm_bound(y, n):
    """fp32 error of y: the sum's, halved by the root, and six operations."""
    return np.abs(y) * (norm_chain(n) / 2 + 6) * U32


def mx(y, fmt):
    """(elements, scales) of rows y in block-scaled 8 bits."""
    emax, bits, low, top = F8[fmt]
    rows, n = y.shape
    q, scales = np.empty_like(y), np.empty((rows, -(-n // 32)))
    for b in range(scales.shape[1]):
        v = y[:, 32 * b:32 * b + 32]
        most = np.max(np.abs(v), axis=1)
        e = np.where(most > 0, np.frexp(most)[1] - 1 - emax, -127).clip(-127, 127)
        scales[:, b] = np.ldexp(1.0, e)
        v = np.ldexp(v, -e[:, None])
        step = np.ldexp(1.0, np.maximum(np.frexp(v)[1] - 1, low) - bits)
        q[:, 32 * b:32 * b + 32] = np.clip(np.rint(v / step) * step, -top, top)
    return q, scales


def norm_backward(dy, t, gain, inv, dtotal):
    u = t * inv[:, None]
    a = dy * gain
    mean = np.mean(a * u, axis=1, keepdims=True)
    dx = inv[:, None] * (a - u * mean)
    if dtotal is not None:
        dx = dx + dtotal
    return dx, np.sum(dy * u, axis=0)


def norm_backward_bound(dy, t, gain, inv, dtotal, rows_a_cta, ctas):
    """fp32 errors of (dx, dgain)."""
    n = t.shape[1]
    u = np.abs(t * inv[:, None])
    a = np.abs(dy * gain)
    mean = np.mean(a * u, axis=1, keepdims=True)
    dx = np.abs(inv)[:, None] * ((norm_chain(n) + 8) * u * mean + 6 * a) * U32
    if dtotal is not None:
        dx = dx + (np.abs(dtotal) + np.abs(inv)[:, None] * (a + u * mean)) * U32
    return dx, (rows_a_cta + ctas / 32 + 32 + 4) * U32 * np.sum(np.abs(dy) * u, axis=0)


def w4_codes(W, k):
    return np.stack((W & 15, W >> 4), axis=2).reshape(W.shape[0], -1)[:, :k].astype(np.float64)


def w4(A, W, scales, zeros, group, alpha, bias, epilogue, dtype, silu_err=True):
    """(C, bound) for A, scales, bias in float64 and W, zeros in uint8."""
    k, n = A.shape[1], W.shape[0]
    at = np.arange(k) // group
    s = scales[:, at]
    z = np.full_like(s, 8.0) if zeros is None else zeros.astype(np.float64)[:, at]
    q = w4_codes(W, k)
    v = A @ ((q - z) * s).T
    # the kernel adds (1 + q/16) x and takes (1 + z/16) x off, 16 s of each;
    # the tensor core adds 16 terms a step, each step off by 2^-23 at most
    mag = np.abs(A) @ ((32 + q + z) * np.abs(s)).T
    err = mag * 2.0 ** -23 * (group / 16 + k / group / 2 + 16)
    v, err = alpha * v, abs(alpha) * err + np.abs(alpha * v) * U32
    if bias is not None:
        v = v + bias
        err = err + np.abs(v) * U32

    def silu(x, e):
        with np.errstate(over="ignore"):
            y = x / (1 + np.exp(-x))
        # |silu'| < 1.1; exp is off by (2 + 1.2 |x|) 2^-23, the quotient by 2^-22
        return y, 1.1 * e + np.abs(y) * (2 + 1.2 * np.abs(x) + 4) * 2.0 ** -23

    if epilogue == "silu":
        v, err = silu(v, err)
    elif epilogue == "swiglu":
        g, eg = silu(v[:, :n // 2], err[:, :n // 2])
        up, eu = v[:, n // 2:], err[:, n // 2:]
        v, err = g * up, eg * np.abs(up) + eu * np.abs(g) + eg * eu + np.abs(g * up) * U32
    return v, err + store(v, dtype)


def sample_row(x, u, temperature, top_k, top_p, min_p):
    """(token, prob, gap) of one row: gap is the distance of the nearest
    border that decided anything, relative to the sum it divides (a kernel
    whose sums are off by less must give this token)."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    if not x.size or np.max(x) == -np.inf:
        return -1, 0.0, np.inf
    ids = np.argsort(-x, kind="stable")
    if not temperature > 0:
        return int(ids[0]), 1.0, np.inf
    ids = ids[x[ids] > -np.inf]
    if top_k > 0:
        ids = ids[:top_k]
    m = x[ids[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x[ids] == m, 1.0, np.exp((x[ids] - m) / temperature))
    gap = np.inf
    n = len(ids)
    if top_p < 1:
        cum = np.cumsum(w)
        t = max(top_p, 0.0) * cum[-1]
        n = min(n, 1 + int(np.searchsorted(cum, t, side="left")))
        near = np.abs(cum - t)
        near = near[near > 0]  # sums that hit the border exactly are exact in the kernel as well
        gap = min(gap, float(near.min()) / cum[-1]) if near.size else gap
    if min_p > 0:
        n = max(1, min(n, int(np.count_nonzero(w >= min_p))))
        near = np.abs(w - min_p)
        gap = min(gap, float(near[near > 0].min(initial=np.inf)))
    order = np.argsort(ids[:n])
    w = w[:n][order]
    cum = np.cumsum(w)
    u = 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0 ** -24)  # the nearest float in [0, 1)
    t = u * cum[-1]
    at = int(np.searchsorted(cum, t, side="right"))
    if at >= n:
        at = int(np.max(np.nonzero(w)))
    near = np.abs(cum - t)
    near = near[near > 0]
    gap = min(gap, float(near.min()) / cum[-1]) if near.size else gap
    return int(ids[:n][order][at]), float(w[at] / cum[-1]), gap
