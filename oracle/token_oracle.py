"""Plain CPU oracle for the token operators (embedding and norm, with their
gradients and dropout), in float64.

TEST INFRASTRUCTURE ONLY, as fsdp_oracle: written from the formulas, it
imports nothing from the product package.  Activations are [rows, cols] float64
arrays holding the exact values of the tested types; round_to(a, name) rounds
float64 values to one of them, once, to nearest even.
"""

from __future__ import annotations

import numpy as np

MANTISSA = {"f32": 24, "bf16": 8, "f16": 11}  # significand bits
MIN_EXP = {"f32": -126, "bf16": -126, "f16": -14}  # exponent of the smallest normal number


def round_to(a: np.ndarray, name: str) -> np.ndarray:
    """a (float64, within range) rounded to the type's grid, ties to even;
    denormals keep the type's smallest step."""
    a = np.asarray(a, dtype=np.float64)
    _, e = np.frexp(a)  # a = m * 2^e, 0.5 <= |m| < 1
    step = np.exp2(np.maximum(e - 1, MIN_EXP[name]) - (MANTISSA[name] - 1.0))
    with np.errstate(invalid="ignore"):
        r = np.rint(a / step) * step
    return np.where(np.isfinite(a), r, a)


# --- dropout ----------------------------------------------------------------

def philox4x32(counter, key, rounds: int = 7):
    """Philox4x32 of Salmon, Moraes, Dror, Shaw (SC 2011): four 32-bit words
    from a counter of four and a key of two, with Python's integers."""
    x0, x1, x2, x3 = (int(c) for c in counter)
    k0, k1 = (int(k) for k in key)
    for _ in range(rounds):
        hi0, lo0 = divmod(0xD2511F53 * x0, 1 << 32)
        hi1, lo1 = divmod(0xCD9E8D57 * x2, 1 << 32)
        x0, x1, x2, x3 = hi1 ^ x1 ^ k0, lo1, hi0 ^ x3 ^ k1, lo0
        k0 = (k0 + 0x9E3779B9) % (1 << 32)
        k1 = (k1 + 0xBB67AE85) % (1 << 32)
    return x0, x1, x2, x3


def dropout_factors(rows: int, cols: int, p: float, seed: int, step: int, site: int) -> np.ndarray:
    """[rows, cols]: 0 where an element is dropped, else 1 / (1 - p), p a
    multiple of 2^-16."""
    cut = int(p * 65536 + 0.5)
    out = np.zeros((rows, cols))
    for t in range(rows):
        for j in range((cols + 7) // 8):
            words = philox4x32((j, t, site, step % (1 << 32)), (seed % (1 << 32), seed >> 32))
            for k in range(min(8, cols - 8 * j)):
                lane = words[k // 2] >> (16 * (k % 2)) & 0xFFFF
                if lane >= cut:
                    out[t, 8 * j + k] = 65536 / (65536 - cut)
    return out


def _times(a, factors):
    """a * factors, with 0 (not NaN) where the factor is 0."""
    if factors is None:
        return a
    with np.errstate(invalid="ignore"):
        return np.where(factors == 0, 0.0, a * factors)


# --- embedding --------------------------------------------------------------

def embedding(tokens, table, scale=1.0, factors=None):
    out = np.zeros((len(tokens), table.shape[1]))
    for t, v in enumerate(tokens):
        if 0 <= v < table.shape[0]:
            out[t] = scale * table[v]
    return _times(out, factors)


def embedding_grad(tokens, dout, vocab, scale=1.0, factors=None):
    """The gradient of the table of one rank, and what its rounding in any
    order of fp32 sums scales with: the sums of the terms' magnitudes."""
    d = _times(dout, factors)
    grad, size = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1]))
    for t, v in enumerate(tokens):
        if 0 <= v < vocab:
            grad[v] += d[t]
            size[v] += np.abs(d[t])
    return scale * grad, abs(scale) * size


# --- norm -------------------------------------------------------------------

def norm_input(x, residual, factors, act):
    """h = residual + drop(x), rounded to the activations' type."""
    h = _times(x, factors)
    return round_to(h if residual is None else residual + h, act)


def norm(h, weight, bias, eps, rms):
    """y, mean, rstd of the rows of h."""
    mean = np.zeros(h.shape[0]) if rms else h.mean(1)
    d = h - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None] * weight
    return (y if bias is None else y + bias), mean, rstd


def norm_grad(dy, h, mean, rstd, weight, dh, rms):
    """dres, the gradients of weight and bias, and the sums of the magnitudes
    of their terms."""
    xhat = (h - mean[:, None]) * rstd[:, None]
    g = dy * weight
    d = g - xhat * (g * xhat).mean(1, keepdims=True)
    if not rms:
        d = d - g.mean(1, keepdims=True)
    d = d * rstd[:, None]
    if dh is not None:
        d = d + dh
    return d, (dy * xhat).sum(0), dy.sum(0), np.abs(dy * xhat).sum(0), np.abs(dy).sum(0)
