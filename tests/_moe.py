"""Plain 64-bit forms of the mixture-of-experts operators, written from their
definitions (numpy, on the CPU), with the bounds their tests use.

Bounds.  bf16 rounds to nearest: half a step is at most 2^-8 of a normal value.  A sum
of K exact products in fp32 is off by at most K steps of 2^-23 of the sum of
their magnitudes (one step per addition, whichever way it is rounded)."""
from __future__ import annotations

import numpy as np
import torch

HALF_STEP = 2.0 ** -8       # seven stored significand bits: a step is 2^-7 of 2^e <= |x|
TINY = 2.0 ** -126          # below bf16's normal range steps no longer shrink


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def routing(experts: np.ndarray, E: int):
    """offsets, rows, slots of the stable order by expert, pair by pair."""
    T, k = experts.shape
    lists = [[] for _ in range(E)]
    for t in range(T):
        for j in range(k):
            if experts[t, j] >= 0:
                lists[experts[t, j]].append((t, j))
    offsets, rows, slots = [0], np.full(T * k, -1), np.full((T, k), -1)
    at = 0
    for e in range(E):
        for t, j in lists[e]:
            rows[at], slots[t, j] = t, at
            at += 1
        offsets.append(at)
    return np.array(offsets), rows, slots


def route(logits: np.ndarray, k: int, renorm: bool):
    T, E = logits.shape
    experts, weights = np.full((T, k), -1), np.zeros((T, k))
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        x = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], big))
        order = sorted(range(E), key=lambda e: (-x[e], e))
        order = [e for e in order if x[e] > -np.inf]
        if not order:
            continue
        p = np.exp(x - x[order[0]])
        chosen = order[:k]
        whole = p[chosen].sum() if renorm else p.sum()
        for j, e in enumerate(chosen):
            experts[t, j], weights[t, j] = e, p[e] / whole
    return experts, weights


def route_grad(logits: np.ndarray, experts: np.ndarray, dweights: np.ndarray, renorm: bool) -> np.ndarray:
    T, E = logits.shape
    out = np.zeros((T, E))
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        x = np.where(np.isnan(logits[t]), -np.inf, np.minimum(logits[t], big))
        u = np.zeros(E)
        chosen = [e for e in experts[t] if e >= 0]
        for j, e in enumerate(experts[t]):
            if e >= 0:
                u[e] = dweights[t, j]
        if renorm:
            x = np.array([x[e] if e in chosen else -np.inf for e in range(E)])
        if not np.any(x > -np.inf):
            continue
        p = np.exp(x - x.max())
        p /= p.sum()
        out[t] = p * (u - (p * u).sum())
    return out


def gathered(X: np.ndarray, rows) -> np.ndarray:
    """X's rows by index; an index outside X stands for a zero row."""
    if rows is None:
        return X
    out = np.zeros((len(rows), X.shape[1]))
    for i, r in enumerate(rows):
        if 0 <= r < X.shape[0]:
            out[i] = X[r]
    return out


def product(X, W, offsets, rows, mn: bool):
    """The products and, per output, the sum of magnitudes behind it."""
    x = gathered(X, rows)
    E, N = W.shape[0], W.shape[2] if mn else W.shape[1]
    D, S = np.zeros((len(x), N)), np.zeros((len(x), N))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        w = W[e] if mn else W[e].T
        D[lo:hi] = x[lo:hi] @ w
        S[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w)
    return D, S


def product_bound(D, S, K: int):
    acc = K * 2.0 ** -23 * S
    return HALF_STEP * (np.abs(D) + acc) + acc + TINY


def silu(g):
    return g / (1 + np.exp(-g))


def gate_bound(g, u, eg, eu):
    """Bound of bf16(silu(g) u) in fp32 arithmetic, g and u off by eg and eu:
    silu's slope is at most 1.1; the exponential's relative error grows with
    its argument (a step of 2^-23 of |g|), the other operations take one step
    each (eight in all, the reciprocal's last place among them)."""
    a = np.abs(silu(g) * u)
    moved = 1.1 * eg * np.abs(u) + np.abs(silu(g)) * eu + 1.1 * eg * eu
    rel = (8 + np.abs(g)) * 2.0 ** -22 * (a + moved)
    return moved + rel + HALF_STEP * (a + moved + rel) + TINY


def dw(dY, X, offsets, rows):
    x = gathered(X, rows)
    E = len(offsets) - 1
    D = np.zeros((E, dY.shape[1], X.shape[1]))
    S = np.zeros_like(D)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        D[e] = dY[lo:hi].T @ x[lo:hi]
        S[e] = np.abs(dY[lo:hi]).T @ np.abs(x[lo:hi])
    return D, S
