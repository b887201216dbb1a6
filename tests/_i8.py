"""Plain 64-bit forms of the 8-bit integer operators and of the router by groups,
written from their definitions (numpy, on the CPU), with the bounds their
tests use.

Bounds.  fp32 rounds to nearest: at most 2^-24 of a normal value.  A product is an
exact whole number that is rounded when it becomes fp32, when it meets the row's
scale and when it meets the column's; a bf16 result once more (2^-8)."""
from __future__ import annotations

import numpy as np

from tests._moe import HALF_STEP, TINY, gate_bound, gathered, silu

__all__ = ["quant", "product", "product_bound", "moe_product", "scaled_bound", "gate_bound", "silu", "choose", "weights",
           "grouped_grad", "HALF_STEP", "TINY"]

HALF_F32 = 2.0 ** -24


def quant(x: np.ndarray):
    """codes and scales (64 bits; the scale before its rounding to fp32).  fp32
    magnitudes times 127 or 254 and a quotient of them: ties are seen exactly."""
    codes, scales = np.zeros(x.shape, dtype=np.int64), np.zeros(len(x))
    for m, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scales[m] = np.nan
            continue
        amax = np.abs(row).max()
        scales[m] = amax / 127
        if amax > 0:
            whole = np.floor(127 * np.abs(row) / amax)
            # 254 |x| and (2 whole + 1) amax have at most 33 bits: exact
            whole -= 2 * whole * amax > 254 * np.abs(row)          # (a quotient rounded up to a whole number)
            d = 254 * np.abs(row) - (2 * whole + 1) * amax
            up = (d > 0) | ((d == 0) & (whole % 2 == 1))
            codes[m] = np.sign(row) * (whole + up)
    return codes, scales


def product(A, sA, B, sB):
    """Codes as whole numbers in fp64: sums below 2^31 are exact."""
    return (A @ B.T) * sA[:, None] * sB[None, :]


def scaled_bound(D):
    """Three roundings to fp32 (and a last place for their products), or a subnormal's."""
    return 3.01 * HALF_F32 * np.abs(D) + 2.0 ** -140


def product_bound(D, bf16: bool):
    b = scaled_bound(D)
    return b + HALF_STEP * (np.abs(D) + b) + TINY if bf16 else b


def moe_product(X, sX, W, sW, offsets, rows):
    x, s = gathered(X, rows), gathered(sX[:, None], rows)
    D = np.zeros((len(x), W.shape[1]))
    for e in range(W.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        D[lo:hi] = (x[lo:hi] @ W[e].T) * s[lo:hi] * sW[e][None, :]
    return D


# ---------------------------------------------------------------- the router

BIG = float(np.finfo(np.float32).max)


def _open(x):
    return np.where(np.isnan(x), -np.inf, np.minimum(x, BIG))


def scores(x: np.ndarray, kind: str):
    """Of one token's opened logits; closed experts 0."""
    s = np.zeros_like(x)
    there = x > -np.inf
    if not there.any():
        return s
    z = x[there]
    if kind == "sigmoid":
        e = np.exp(-np.abs(z))
        s[there] = np.where(z >= 0, 1 / (1 + e), e / (1 + e))
    else:
        p = np.exp(z - z.max())
        s[there] = p / p.sum()
    return s


def choose(logits, k, bias, groups, kept, best, kind):
    """experts (T, k), -1: none."""
    T, E = logits.shape
    per = E // groups
    out = np.full((T, k), -1)
    b = np.zeros(E) if bias is None else _open(bias)
    for t in range(T):
        x = np.where(b > -np.inf, _open(logits[t]), -np.inf)
        s = scores(_open(logits[t]), kind)
        c = [s[e] + b[e] for e in range(E)]
        there = [e for e in range(E) if x[e] > -np.inf]
        if kept < groups:
            rank = []
            for g in range(groups):
                mine = sorted((c[e] for e in there if e // per == g), reverse=True)[:best]
                if mine:
                    rank.append((-sum(mine), g))
            keep = [g for _, g in sorted(rank)[:kept]]
            there = [e for e in there if e // per in keep]
        for j, e in enumerate(sorted(there, key=lambda e: (-c[e], e))[:k]):
            out[t, j] = e
    return out


def weights(logits, experts, kind, renorm, scale):
    """(weights, how many roundings' worth of 2^-23 each may be off)."""
    w, steps = np.zeros(experts.shape), np.zeros(experts.shape)
    for t in range(len(experts)):
        on = experts[t] >= 0
        e = experts[t][on]
        if not len(e):
            continue
        x = _open(logits[t])
        if renorm:
            # ratios of scores, from their logarithms: sums of scores may be below fp64's range
            y = x[e]
            if kind == "sigmoid":
                low, rest = np.minimum(y, 0), 1 / (1 + np.exp(-np.abs(y)))
            else:
                low, rest = y, np.ones_like(y)
            v = np.exp(low - low.max()) * rest
            w[t, on] = scale * v / v.sum()
            steps[t, on] = np.minimum(low.max() - low, 200)
        else:
            w[t, on] = scale * scores(x, kind)[e]
            steps[t, on] = np.minimum(x.max() - x[e], 200) if kind == "softmax" else 0
    return w, steps


def grouped_grad(logits, experts, dweights, kind, renorm, scale):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        on = experts[t] >= 0
        e, u = experts[t][on], dweights[t][on] * scale
        if not len(e):
            continue
        x = _open(logits[t])
        if kind == "softmax":
            z = np.full(E, -np.inf)
            if renorm:
                z[e] = x[e]
            else:
                z = x
            p = np.exp(z - z.max())
            p /= p.sum()
            full = np.zeros(E)
            full[e] = u
            out[t] = p * (full - (p * full).sum())
            continue
        y = x[e]
        small = np.exp(-np.abs(y))
        s = np.where(y >= 0, 1, small) / (1 + small)
        rest = np.where(y >= 0, small, 1) / (1 + small)
        if renorm:
            low = np.minimum(y, 0)
            v = np.exp(low - low.max()) / (1 + small)
            w = v / v.sum()
            out[t, e] = w * (u - (w * u).sum()) * rest
        else:
            out[t, e] = u * s * rest
    return out
